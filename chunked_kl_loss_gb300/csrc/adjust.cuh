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

#include <type_traits>

#include "adjust_plan.h"
#include "bulk.cuh"
#include "score.cuh"

namespace fckl {

constexpr int ADJUST_UNROLL = 8;      // vectors that a thread has under way
constexpr int ADJUST_AHEAD = 8;       // history entries that a thread has under way

// What shared memory holds for a token that a rule touches: how often it was generated, whether it stands
// in the prompt, and TOKENS_MAX less the bias slot that carries the sum of its biases (0: none).
constexpr uint32_t ADJ_COUNT = 0xfffffu;
constexpr uint32_t ADJ_GIVEN = 1u << 20;
constexpr uint32_t ADJ_SEEN = ADJ_COUNT | ADJ_GIVEN;
constexpr uint32_t ADJ_POSITIVE = 1;  // gradient: the logit is above 0
constexpr int ADJ_SLOT_SHIFT = 21;
constexpr int ADJ_SEVERAL = static_cast<int>(0x80000000u);  // of a bias token in shared memory: it has several slots
constexpr int ADJ_TOKEN = 0x7fffffff;
constexpr int ADJUST_HISTORY_MAX = 0xfffff;
constexpr uint32_t ADJ_NO_KEY = ~0u;

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
  int stages;          // of a warp's ring in the staged kernel
  int slots_log2;      // of the table of touched tokens; < 0: one word for every token of the segment
  unsigned* status;
};

// Word k of a 16-byte vector with what is not allowed replaced: -inf, or 0 in a gradient.
template <typename T, bool GRAD>
__device__ __forceinline__ uint32_t masked_word(uint32_t w, uint32_t m, int k) {
  const uint32_t none = GRAD ? 0u : fill_word<T>(-INFINITY);
  if constexpr (sizeof(T) == 4) {
    return (m >> k) & 1u ? w : none;
  } else {
    const uint32_t keep = ((m >> (2 * k)) & 1u ? 0xffffu : 0u) | ((m >> (2 * k + 1)) & 1u ? 0xffff0000u : 0u);
    return (w & keep) | (none & ~keep);
  }
}

// A row's segment and the shared memory of its touched tokens.
struct AdjustSegment {
  int mis, v0, v1;     // values from the 16-byte boundary below the row's start; first and last vector
  int c0, columns;     // its columns
  int first;           // column of the first vector's first value (below 0 before a row's start)
  bool table;
  int words, bits;     // 32-bit words of the table or array, and of one set of bits
  uint32_t *seen, *positive;  // bits by value from `first` on
  uint32_t *word, *key;
  int* btok;
  float *bsum, *bval;
};

// Sets of bits, then words and keys, then biases: as much of it as the kernel and the kind of rules need.
template <typename T, int VE, AdjustKind KIND, bool STAGED>
__device__ __forceinline__ AdjustSegment adjust_segment(const AdjustParams& p, const T* out, int seg, uint32_t* smem) {
  AdjustSegment s;
  s.mis = VE == 1 ? 0 : static_cast<int>((reinterpret_cast<uintptr_t>(out) & 15u) / sizeof(T));
  const int nvec = (p.V + s.mis + VE - 1) / VE;
  s.v0 = seg * p.seg_vecs;
  s.v1 = min(nvec, s.v0 + p.seg_vecs);
  s.first = s.v0 * VE - s.mis;
  s.c0 = max(s.first, 0);
  s.columns = min(s.v1 * VE - s.mis, p.V) - s.c0;
  s.table = p.slots_log2 >= 0;
  s.bits = STAGED || !s.table ? (p.seg_vecs * VE + 127) / 128 * 4 : 0;
  s.words = STAGED && KIND != ADJUST_COUNTS ? 0 : s.table ? 1 << p.slots_log2 : p.seg_vecs * VE;
  s.seen = smem;
  s.positive = smem + s.bits;
  s.word = smem + (STAGED && KIND == ADJUST_GRAD ? 2 : 1) * s.bits;
  s.key = s.word + s.words;
  s.btok = reinterpret_cast<int*>(s.word + (s.table ? 2 : 1) * s.words);
  s.bsum = reinterpret_cast<float*>(s.btok + p.B);
  s.bval = s.bsum + p.B;
  return s;
}

__device__ __forceinline__ uint32_t adjust_hash(int token, int log2) {
  return (static_cast<uint32_t>(token) * 0x9E3779B1u) >> (32 - log2);
}

// Gathers the segment's touched tokens from the row's history and biases. Counts and bias slots are kept in
// a hash table of token ids where those are few, so that its size does not depend on V, else in a word for
// every token. A set of bits says which tokens are touched (not beside the table of the kernel that is not
// staged), and in a staged gradient a second one which logits are above 0. Complete after the caller's next
// barrier.
template <typename T, AdjustKind KIND, bool STAGED, int NT>
__device__ __forceinline__ void adjust_gather(const AdjustParams& p, const AdjustSegment& s, int64_t row, const T* z) {
  const int tid = threadIdx.x;
  const int32_t* h = p.history + row * p.ld_h;
  // The first history entries (whether or not they count: that is known when lengths[row] is here) and
  // biases are under way while shared memory is cleared, later entries while earlier ones are gathered.
  constexpr int A = ADJUST_AHEAD;
  int ahead[A];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < A; ++u) ahead[u] = i0 + u * NT < p.L ? h[i0 + u * NT] : -1;
  };
  fetch(tid);
  const int len = p.lengths ? min(max(p.lengths[row], 0), p.L) : p.L;
  const int prompt = KIND == ADJUST_COUNTS && p.prompt ? p.prompt[row] : 0;
  const uint4 zero = make_uint4(0, 0, 0, 0), no_key = make_uint4(ADJ_NO_KEY, ADJ_NO_KEY, ADJ_NO_KEY, ADJ_NO_KEY);
  const int clear = ((STAGED && KIND == ADJUST_GRAD ? 2 : 1) * s.bits + s.words) / 4;
  int first_token = -1;
  float first_bias = 0.f;
  if (tid < p.B) {
    first_token = p.bias_tokens[row * p.B + tid];
    first_bias = p.bias[row * p.B + tid];
  }
  for (int i = tid; i < clear; i += NT) reinterpret_cast<uint4*>(s.seen)[i] = zero;
  if (s.table)
    for (int i = tid; i < s.words / 4; i += NT) reinterpret_cast<uint4*>(s.key)[i] = no_key;
  bool bad = false;
  for (int b = tid; b < p.B; b += NT) {
    const int t = b == tid ? first_token : p.bias_tokens[row * p.B + b];
    const bool in = static_cast<unsigned>(t) < static_cast<unsigned>(p.V);
    bad |= !in && t != -1;
    s.btok[b] = in ? t : -1;  // what is not a token is an empty slot from here on
    s.bval[b] = b == tid ? first_bias : p.bias[row * p.B + b];
  }
  __syncthreads();
  // The word of a token of the segment. The table has room for every history entry and bias.
  auto place = [&](int t) -> uint32_t* {
    if (!s.table) return s.word + (t - s.c0);
    uint32_t at = adjust_hash(t, p.slots_log2);
    for (;;) {
      const uint32_t k = *static_cast<volatile uint32_t*>(s.key + at);
      if (k == static_cast<uint32_t>(t)) break;
      if (k == ADJ_NO_KEY) {
        const uint32_t old = atomicCAS(s.key + at, ADJ_NO_KEY, static_cast<uint32_t>(t));
        if (old == ADJ_NO_KEY || old == static_cast<uint32_t>(t)) break;
      }
      at = (at + 1) & (s.words - 1);
    }
    return s.word + at;
  };
  // Sets a token's bit; whether it was not set before.
  auto mark = [&](uint32_t* bits, int t) {
    const uint32_t one = 1u << ((t - s.first) & 31);
    return !(atomicOr(bits + ((t - s.first) >> 5), one) & one);
  };
  for (int i0 = tid; i0 < len; i0 += A * NT) {
    int t[A];
    T sign[A];
#pragma unroll
    for (int u = 0; u < A; ++u) t[u] = i0 + u * NT < len ? ahead[u] : -1;
    if (i0 + A * NT < len) fetch(i0 + A * NT);
#pragma unroll
    for (int u = 0; u < A; ++u) {
      if (static_cast<unsigned>(t[u]) >= static_cast<unsigned>(p.V)) {
        bad |= t[u] != -1;
        t[u] = -1;
      } else if (static_cast<unsigned>(t[u] - s.c0) >= static_cast<unsigned>(s.columns)) {
        t[u] = -1;
      } else if (KIND == ADJUST_COUNTS) {
        if (STAGED || s.bits) mark(s.seen, t[u]);
        uint32_t* w = place(t[u]);
        if (i0 + u * NT >= prompt) atomicAdd(w, 1u);
        else atomicOr(w, ADJ_GIVEN);
      } else {
        if (!STAGED && s.bits) mark(s.seen, t[u]);
        const bool is_new = STAGED ? mark(s.seen, t[u]) : atomicOr(place(t[u]), ADJ_GIVEN) == 0;
        if (KIND == ADJUST_GRAD && is_new) sign[u] = z[t[u]];
        else t[u] = -1;
      }
    }
    if (KIND == ADJUST_GRAD) {
#pragma unroll
      for (int u = 0; u < A; ++u) {
        if (t[u] < 0 || !(to_f32(sign[u]) > 0.f)) continue;
        if (STAGED) mark(s.positive, t[u]);
        else atomicOr(place(t[u]), ADJ_POSITIVE);
      }
    }
  }
  // The first slot of a token takes the sum over its slots, in their order: found by the largest of their
  // numbers counted down, in the word's upper bits; only a token with several slots looks through all.
  if (p.B) {
    __syncthreads();  // the words' lower bits are complete
    // whether slot b's token lies in the segment; its word then holds a slot's number from the first loop on
    auto inside = [&](int b) {
      return s.btok[b] != -1 && static_cast<unsigned>((s.btok[b] & ADJ_TOKEN) - s.c0) < static_cast<unsigned>(s.columns);
    };
    for (int b = tid; b < p.B; b += NT) {
      const int t = s.btok[b];
      if (!inside(b)) continue;
      if (STAGED || s.bits) mark(s.seen, t);
      uint32_t* w = place(t);
      atomicMax(w, (*static_cast<volatile uint32_t*>(w) & ((1u << ADJ_SLOT_SHIFT) - 1u)) |
                       static_cast<uint32_t>(TOKENS_MAX - b) << ADJ_SLOT_SHIFT);
    }
    __syncthreads();
    auto owner = [&](int t) { return TOKENS_MAX - static_cast<int>(*place(t) >> ADJ_SLOT_SHIFT); };
    for (int b = tid; b < p.B; b += NT) {
      if (!inside(b)) continue;
      const int first = owner(s.btok[b] & ADJ_TOKEN);
      if (first != b) atomicOr(&s.btok[first], ADJ_SEVERAL);
    }
    __syncthreads();
    for (int b = tid; b < p.B; b += NT) {
      const int t = s.btok[b] & ADJ_TOKEN;
      if (!inside(b) || owner(t) != b) continue;
      float sum = s.bval[b];
      if (s.btok[b] & ADJ_SEVERAL)
        for (int j = b + 1; j < p.B; ++j)
          if ((s.btok[j] & ADJ_TOKEN) == t) sum += s.bval[j];
      s.bsum[b] = sum;
    }
  }
  if (bad) atomicOr(p.status, ST_BAD_INDEX);
}

// A row's penalties, and a value under what its word says.
struct AdjustRow {
  float r, f, p;
  __device__ __forceinline__ AdjustRow(const AdjustParams& q, int64_t row)
      : r(q.r ? q.r[row] : q.r1), f(q.f ? q.f[row] : q.f1), p(q.p ? q.p[row] : q.p1) {}
  __device__ __forceinline__ float repeated(float v, bool positive) const { return positive ? v / r : v * r; }
  template <AdjustKind KIND>
  __device__ __forceinline__ float value(float v, uint32_t w, const float* bsum) const {
    if constexpr (KIND == ADJUST_GRAD) {
      return repeated(v, w & ADJ_POSITIVE);
    } else {
      if (w & ADJ_SEEN) v = repeated(v, v > 0.f);
      const uint32_t n = w & ADJ_COUNT;
      if (n) v = v - f * static_cast<float>(n) - p;
      const uint32_t slot = w >> ADJ_SLOT_SHIFT;
      if (slot) v += bsum[TOKENS_MAX - slot];
      return v;
    }
  }
};

// Into rows that lie alike to the 16-byte boundaries, or in place under a mask. One block per (row, segment of
// seg_vecs vectors). The segment streams through shared memory by bulk copies, which are under way while
// the threads gather the segment's touched tokens: every warp has a ring of stages of its own, so that no
// barrier of the block stands in the stream. The threads change the touched and the masked places in the
// stages: what no rule touches passes through no register, and a touched place costs no access to
// memory. Two blocks an SM: one gathers while the other streams.
// Bound by memory: 4096 x 128256 bf16 without rules 306 us (a plain copy's time), with a mask 317, with 1024
// history entries, 16 biases and a mask 328 (floor 325); the gradient, which reads the logits at the history's
// tokens from all over the row before it streams, 372 (374 with those read before the first barrier).
// Before: a word in shared memory for every token 1070 us; rows through registers with the touched places
// written again afterwards 437 to 451; one ring to a block with a barrier for every stage 418; the touched
// and masked places of each vector for itself instead of the lane's three vectors at once 362. Of 96 vectors
// and 3 stages: 2 stages 15% more, 64 vectors 5%, 4 stages of 128 vectors (one block an SM less) 30%.
template <typename T, AdjustKind KIND, int NT>
__global__ void __launch_bounds__(NT) adjust_staged_kernel(const AdjustParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int WARPS = NT / 32, TV = ADJUST_STAGE_VECS;
  constexpr int U = TV / 32;
  constexpr uint32_t ALL = (1u << VE) - 1u;
  constexpr bool GRAD = KIND == ADJUST_GRAD;
  extern __shared__ __align__(128) uint8_t adj_stage[];
  __shared__ uint64_t bars[WARPS][ADJUST_STAGES];
  const int64_t row = blockIdx.x / p.segs;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const T* x = GRAD ? static_cast<const T*>(p.g) + row * p.ld_g : static_cast<const T*>(p.z) + row * p.ld_z;
  const T* z = static_cast<const T*>(p.z) + row * p.ld_z;
  T* out = static_cast<T*>(p.out) + row * p.ld_out;
  uint32_t* after_rings = reinterpret_cast<uint32_t*>(adj_stage + p.stages * WARPS * ADJUST_STAGE_BYTES);
  const AdjustSegment s = adjust_segment<T, VE, KIND, true>(p, out, blockIdx.x % p.segs, after_rings);
  if (s.v0 >= s.v1) return;
  // Whole vectors [wa, wb), in tiles of a stage that the warps take in turn; the row's ends, if they are
  // ragged, go value by value.
  const int wa = s.v0 + (s.first < 0), wb = max(wa, s.v1 - (s.v1 * VE - s.mis > p.V));
  const int all_tiles = (wb - wa + TV - 1) / TV;
  const int tiles = all_tiles > warp ? (all_tiles - warp + WARPS - 1) / WARPS : 0;  // of this warp
  const int stages = p.stages;
  uint64_t* full = bars[warp];
  uint8_t* ring = adj_stage + warp * stages * TV * 16;
  auto column = [&](int v) { return v * VE - s.mis; };
  auto tile_at = [&](int k) { return wa + (k * WARPS + warp) * TV; };
  auto tile_bytes = [&](int k) { return static_cast<uint32_t>(min(TV, wb - tile_at(k))) * 16; };
  auto load_tile = [&](int k, int stage) {
    mbar_arrive_expect_tx(&full[stage], tile_bytes(k));
    bulk_load(ring + stage * TV * 16, x + column(tile_at(k)), tile_bytes(k), &full[stage]);
  };
  if (lane == 0) {
    for (int k = 0; k < stages; ++k) mbar_init(&full[k], 1);
    fence_mbar_init();
    for (int k = 0; k < min(stages, tiles); ++k) load_tile(k, k);
  }
  adjust_gather<T, KIND, true, NT>(p, s, row, z);
  const uint32_t* allowed = p.allowed ? p.allowed + row * p.ld_allowed : nullptr;
  // A lane's vectors lie 32 apart, a multiple of 32 values: one shift serves them all, for the mask's bits
  // and for the touched ones, and their words are at fixed distances.
  const int own = column(tile_at(0) + lane), mask_shift = own & 31;
  const bool two_words = mask_shift + VE > 32;  // the mask's bits of the lane's vectors
  const uint32_t* mask = allowed + (own >> 5);
  constexpr int STEP = WARPS * U * VE;  // words from a tile of the warp to its next
  const int seen_at = (tile_at(0) - s.v0 + lane) * VE, seen_shift = seen_at & 31;
  const uint32_t* seen = s.seen + (seen_at >> 5);
  uint32_t lo[U], hi[U];
  auto fetch_bits = [&](int left) {  // of the lane's vectors of the tile at `mask`, if they lie before the end
#pragma unroll
    for (int u = 0; u < U; ++u) {
      lo[u] = u * 32 < left ? mask[u * VE] : 0;
      hi[u] = two_words && u * 32 < left ? mask[u * VE + 1] : 0;
    }
  };
  if (allowed && tiles) fetch_bits(wb - tile_at(0) - lane);
  const AdjustRow rules(p, row);
  __syncthreads();
  auto value = [&](float v, int c) -> float {  // of a touched place
    if constexpr (KIND == ADJUST_COUNTS) {
      uint32_t at = c - s.c0;
      if (s.table) {
        at = adjust_hash(c, p.slots_log2);
        while (s.key[at] != static_cast<uint32_t>(c)) at = (at + 1) & (s.words - 1);
      }
      return rules.value<KIND>(v, s.word[at], s.bsum);
    } else if constexpr (GRAD) {
      return rules.repeated(v, (s.positive[(c - s.first) >> 5] >> ((c - s.first) & 31)) & 1u);
    } else {
      return rules.repeated(v, v > 0.f);
    }
  };
  int k = 0, stage = 0, before = stages - 1;
  uint32_t phase = 0;
  for (; k < tiles; ++k) {
    uint4* data = reinterpret_cast<uint4*>(ring + stage * TV * 16);
    // The lane's places of the tile, a bit each: those that are not allowed, and of the others the touched ones.
    static_assert(U * VE <= 32, "");
    const int left = wb - tile_at(k) - lane;
    uint32_t off = 0, touched = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * 32 >= left) break;
      if (allowed) off |= (~__funnelshift_r(lo[u], hi[u], mask_shift) & ALL) << (u * VE);
      touched |= ((seen[u * VE] >> seen_shift) & ALL) << (u * VE);
    }
    touched &= ~off;
    mask += STEP;
    if (allowed && k + 1 < tiles) fetch_bits(wb - tile_at(k + 1) - lane);
    const bool ok = drain_phase(&full[stage], phase, p.status);
    T* mine = reinterpret_cast<T*>(data + lane);  // place i at value i / VE * 32 VE + i % VE
    for (; touched; touched &= touched - 1) {
      const int i = __ffs(touched) - 1, e = i / VE * 32 * VE + i % VE;
      mine[e] = from_f32<T>(value(to_f32(mine[e]), column(tile_at(k) + lane) + e));
    }
    if (__popc(off) <= 4) {
      for (; off; off &= off - 1) {
        const int i = __ffs(off) - 1;
        mine[i / VE * 32 * VE + i % VE] = from_f32<T>(GRAD ? 0.f : -INFINITY);
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t m = (off >> (u * VE)) & ALL;
        if (!m) continue;
        uint4 d = m == ALL ? make_uint4(0, 0, 0, 0) : data[u * 32 + lane];
        d.x = masked_word<T, GRAD>(d.x, ~m, 0);
        d.y = masked_word<T, GRAD>(d.y, ~m, 1);
        d.z = masked_word<T, GRAD>(d.z, ~m, 2);
        d.w = masked_word<T, GRAD>(d.w, ~m, 3);
        data[u * 32 + lane] = d;
      }
    }
    seen += STEP;
    fence_proxy_async_smem();
    if (!__all_sync(0xffffffffu, ok)) break;
    if (lane == 0) {
      bulk_store(out + column(tile_at(k)), data, tile_bytes(k));
      bulk_commit();
      if (k >= 1 && k - 1 + stages < tiles) {  // once the store of the stage before this one has read it
        bulk_wait_read<1>();
        load_tile(k - 1 + stages, before);
      }
    }
    before = stage;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1;
    }
  }
  if (k < tiles && lane == 0) {  // a copy did not come: leave none under way
    for (int j = k + 1; j < min(tiles, max(k - 1, 0) + stages); ++j)
      drain_phase(&full[j % stages], (j / stages) & 1, p.status);
  }
  const int head = min(column(wa), p.V) - s.c0;  // values before the whole vectors, and after them
  const int tail0 = max(column(wb), s.c0 + head), tail = max(0, s.c0 + s.columns - tail0);
  if (tid < head + tail) {
    const int c = tid < head ? s.c0 + tid : tail0 + tid - head, b = c - s.first;
    T v = x[c];
    if ((s.seen[b >> 5] >> (b & 31)) & 1u) v = from_f32<T>(value(to_f32(v), c));
    if (allowed && !((allowed[c >> 5] >> (c & 31)) & 1u)) v = from_f32<T>(GRAD ? 0.f : -INFINITY);
    out[c] = v;
  }
  if (lane == 0) bulk_wait_read<0>();
}

// In place without a mask, or into rows that lie differently: the segment is copied under the mask (in place
// there is nothing to copy), then the touched places are written again, each by one thread, from the logits as
// they came in. In place a call is all latency: 1 x 201088 with 1500 history entries 5.5 us in 8 segments or so
// (8.9 in one), 256 x 128256 with 16000 62 us (154 with every token's word looked through instead of a set
// of bits).
template <typename T, int VE, AdjustKind KIND, bool IN_PLACE>
__global__ void __launch_bounds__(ADJUST_THREADS, 2) adjust_kernel(const AdjustParams p) {
  static_assert(IN_PLACE || VE == 1, "");
  extern __shared__ __align__(16) uint32_t adj_smem[];
  const int64_t row = blockIdx.x / p.segs;
  const int tid = threadIdx.x;
  constexpr bool GRAD = KIND == ADJUST_GRAD;
  const T* x = GRAD ? static_cast<const T*>(p.g) + row * p.ld_g : static_cast<const T*>(p.z) + row * p.ld_z;
  const T* z = static_cast<const T*>(p.z) + row * p.ld_z;
  T* out = static_cast<T*>(p.out) + row * p.ld_out;
  const AdjustSegment s = adjust_segment<T, VE, KIND, false>(p, out, blockIdx.x % p.segs, adj_smem);
  if (s.v0 >= s.v1) return;
  adjust_gather<T, KIND, false, ADJUST_THREADS>(p, s, row, z);
  if (GRAD) __syncthreads();  // the logits' signs are read: out may be the logits

  const uint32_t* allowed = !IN_PLACE && p.allowed ? p.allowed + row * p.ld_allowed : nullptr;
  const T none = from_f32<T>(GRAD ? 0.f : -INFINITY);
  auto bit = [&](int c) { return !allowed || ((allowed[c >> 5] >> (c & 31)) & 1u); };
  constexpr int U = ADJUST_UNROLL;
  if constexpr (!IN_PLACE) {
    for (int c0 = s.v0 + tid; c0 < s.v1; c0 += U * ADJUST_THREADS) {
      // Every load of the step is issued before any of them is used.
      T d[U];
      uint32_t m[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * ADJUST_THREADS;
        m[u] = ~0u;
        if (c < s.v1) {
          d[u] = x[c];
          if (allowed) m[u] = allowed[c >> 5];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int c = c0 + u * ADJUST_THREADS;
        if (c < s.v1) out[c] = (m[u] >> (c & 31)) & 1u ? d[u] : none;
      }
    }
  }
  __syncthreads();

  const AdjustRow rules(p, row);
  // Up to U touched places of the thread at a time (no word: none), from their words to the result.
  uint32_t w[U];
  int c[U];
  auto write = [&]() {
    float v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (w[u]) {
        v[u] = to_f32(x[c[u]]);
        if (!bit(c[u])) w[u] = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (w[u]) out[c[u]] = from_f32<T>(rules.value<KIND>(v[u], w[u], s.bsum));
  };
  if (s.table) {
    for (int i0 = tid; i0 < s.words; i0 += U * ADJUST_THREADS) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * ADJUST_THREADS;
        w[u] = i < s.words ? s.word[i] : 0;
        c[u] = w[u] ? static_cast<int>(s.key[i]) : 0;
      }
      write();
    }
  } else {
    for (int i = tid; i < s.bits; i += ADJUST_THREADS) {
      for (uint32_t left = s.seen[i]; left;) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          c[u] = left ? s.first + i * 32 + __ffs(left) - 1 : s.c0;
          w[u] = left ? s.word[c[u] - s.c0] : 0;
          left &= left - 1;
        }
        write();
      }
    }
  }
}

}  // namespace fckl
