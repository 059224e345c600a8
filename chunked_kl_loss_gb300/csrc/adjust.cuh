// Logits adjusted by a request's rules before they are scored: penalties for repeated tokens, biases of
// given tokens and a mask of allowed tokens; and the gradient through that.
//
// With z a row's logits, its history h_0..h_{L-1} (the entries before `prompt` were given, the others
// generated; -1 is an empty slot), seen_v: v stands in the history, c_v: how often v was generated,
//   z1 = z / r  where seen_v and z > 0,  z r  where seen_v and z <= 0,  z  otherwise
//   z' = z1 - f c_v - p [c_v > 0] + (sum of v's biases);  -inf where v is not allowed
//   dz = 0 where v is not allowed, otherwise g times dz1/dz
// Arithmetic is fp32, rounded once to the logits' type; a place that no rule touches keeps its bits.
#pragma once

#include "score.cuh"

namespace fckl {

constexpr int ADJUST_THREADS = 256;
constexpr int ADJUST_UNROLL = 4;

// What a token's word in shared memory holds: how often it was generated, whether it stands in the
// prompt, and one more than the bias slot that carries the sum of its biases (0: none).
constexpr uint32_t ADJ_COUNT = 0xfffffu;
constexpr uint32_t ADJ_GIVEN = 1u << 20;
constexpr uint32_t ADJ_SEEN = ADJ_COUNT | ADJ_GIVEN;
constexpr int ADJ_SLOT_SHIFT = 21;
constexpr int ADJUST_HISTORY_MAX = 0xfffff;

struct AdjustParams {
  const void* z;   // logits
  const void* g;   // upstream gradient (gradient kernel only)
  void* out;
  int64_t ld_z, ld_g, ld_out;
  const int32_t* history;
  int64_t ld_h;
  int L;
  const int32_t* lengths;  // NULL: L
  const int32_t* prompt;   // NULL: 0
  const float *r, *f, *p;  // per row, or NULL and the one value for all
  float r1, f1, p1;
  const int32_t* bias_tokens;
  const float* bias;
  int B;
  const uint32_t* allowed;  // NULL: all
  int64_t ld_allowed;
  int V;
  int segs, seg_vecs;  // segments of a row, vectors of a segment
  unsigned* status;
};

template <typename T, int VE>
struct AdjustVec {
  T v[VE];
};

// One block per (row, segment of seg_vecs vectors). The segment's words are gathered in shared memory
// from the row's whole history, then the segment is walked once.
template <typename T, int VE, bool GRAD, bool IN_PLACE>
__global__ void __launch_bounds__(ADJUST_THREADS) adjust_kernel(const AdjustParams p) {
  extern __shared__ __align__(16) uint32_t adj_smem[];
  const int64_t row = blockIdx.x / p.segs;
  const int seg = blockIdx.x % p.segs;
  const int tid = threadIdx.x;
  const T* x = GRAD ? static_cast<const T*>(p.g) + row * p.ld_g : static_cast<const T*>(p.z) + row * p.ld_z;
  const T* z = static_cast<const T*>(p.z) + row * p.ld_z;
  T* out = static_cast<T*>(p.out) + row * p.ld_out;
  const int mis = VE == 1 ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T));
  const int nvec = (p.V + mis + VE - 1) / VE;
  const int v0 = seg * p.seg_vecs, v1 = min(nvec, v0 + p.seg_vecs);
  if (v0 >= v1) return;
  const int base = v0 * VE - mis;  // column of the segment's first word
  const int words = p.seg_vecs * VE;
  uint32_t* word = adj_smem;
  int* btok = reinterpret_cast<int*>(adj_smem + words);
  float* bsum = reinterpret_cast<float*>(btok + p.B);
  float* bval = bsum + p.B;

  for (int i = tid; i < words; i += ADJUST_THREADS) word[i] = 0;
  for (int b = tid; b < p.B; b += ADJUST_THREADS) {
    btok[b] = p.bias_tokens[row * p.B + b];
    bval[b] = p.bias[row * p.B + b];
  }
  __syncthreads();
  const int len = p.lengths ? min(max(p.lengths[row], 0), p.L) : p.L;
  const int prompt = p.prompt ? p.prompt[row] : 0;
  const int32_t* h = p.history + row * p.ld_h;
  bool bad = false;
  for (int i = tid; i < len; i += ADJUST_THREADS) {
    const int t = h[i];
    if (t < 0 || t >= p.V) {
      bad |= t != -1;
      continue;
    }
    const unsigned at = static_cast<unsigned>(t - base);
    if (at < static_cast<unsigned>(words)) {
      if (!GRAD && i >= prompt) atomicAdd(&word[at], 1u);
      else atomicOr(&word[at], ADJ_GIVEN);
    }
  }
  // The first slot of a token takes the sum over its slots, in their order.
  for (int b = tid; b < p.B; b += ADJUST_THREADS) {
    const int t = btok[b];
    if (t < 0 || t >= p.V) {
      bad |= t != -1;
      continue;
    }
    const unsigned at = static_cast<unsigned>(t - base);
    if (at >= static_cast<unsigned>(words)) continue;
    float sum = 0.f;
    bool first = true;
    for (int j = 0; j < p.B; ++j) {
      if (btok[j] != t) continue;
      if (j < b) {
        first = false;
        break;
      }
      sum += bval[j];
    }
    if (first) {
      bsum[b] = sum;
      atomicOr(&word[at], static_cast<uint32_t>(b + 1) << ADJ_SLOT_SHIFT);
    }
  }
  if (bad) atomicOr(p.status, ST_BAD_INDEX);
  __syncthreads();

  const float r = p.r ? p.r[row] : p.r1;
  const float f = p.f ? p.f[row] : p.f1;
  const float pr = p.p ? p.p[row] : p.p1;
  const uint32_t* allowed = p.allowed ? p.allowed + row * p.ld_allowed : nullptr;
  const float none = GRAD ? 0.f : -INFINITY;
  // value at column c with word w
  auto value = [&](float v, uint32_t w, int c) -> float {
    if constexpr (GRAD) {
      if (w) v = to_f32(z[c]) > 0.f ? v / r : v * r;
    } else {
      if (w & ADJ_SEEN) v = v > 0.f ? v / r : v * r;
      const uint32_t n = w & ADJ_COUNT;
      if (n) v = v - f * static_cast<float>(n) - pr;
      const uint32_t slot = w >> ADJ_SLOT_SHIFT;
      if (slot) v += bsum[slot - 1];
    }
    return v;
  };
  auto bit = [&](int c) { return !allowed || ((allowed[c >> 5] >> (c & 31)) & 1u); };
  for (int i = v0 + tid; i < v1; i += ADJUST_THREADS) {
    const int c = i * VE - mis;
    const uint32_t* w = word + (i - v0) * VE;
    if (c < 0 || c + VE > p.V) {  // an end of the row
      for (int j = 0; j < VE; ++j) {
        if (c + j < 0 || c + j >= p.V) continue;
        if (!bit(c + j)) out[c + j] = from_f32<T>(none);
        else if (w[j]) out[c + j] = from_f32<T>(value(to_f32(x[c + j]), w[j], c + j));
        else if (!IN_PLACE) out[c + j] = x[c + j];
      }
      continue;
    }
    constexpr uint32_t ALL = (1u << VE) - 1u;
    uint32_t m = ALL;
    if (allowed) {
      const int lo = c >> 5, hi = (c + VE - 1) >> 5;
      m = __funnelshift_r(allowed[lo], hi > lo ? allowed[hi] : 0u, c & 31) & ALL;
    }
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < VE; ++j) any |= w[j];
    if (IN_PLACE && !any && m == ALL) continue;
    using Vec = AdjustVec<T, VE>;
    struct alignas(VE * sizeof(T)) Raw {
      Vec v;
    };
    Raw d;
    if (m) {
      d = *reinterpret_cast<const Raw*>(x + c);
      if (any) {
#pragma unroll
        for (int j = 0; j < VE; ++j)
          if (w[j]) d.v.v[j] = from_f32<T>(value(to_f32(d.v.v[j]), w[j], c + j));
      }
    }
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (!((m >> j) & 1u)) d.v.v[j] = from_f32<T>(none);
    *reinterpret_cast<Raw*>(out + c) = d;
  }
}

}  // namespace fckl
