// Scoring kernels over logits that are at hand: log-probabilities of given tokens, entropy and
// top alternatives of a row of logits in one pass over it, and the gradient of the
// log-probabilities and the entropy.
//
// With z the logits of a row, m = max z and the row's tokens t_1..t_T (an id of -1 is an empty
// slot):
//   s       = sum_v exp(z_v - m),  u = sum_v (z_v - m) exp(z_v - m)
//   logp_t  = (z_t - m) - log s                    (empty slot: 0)
//   entropy = log s - u / s                        (= - sum_v q_v log q_v, q = softmax(z))
//   dz_v    = sum_t g_t [v = t] - q_v (sum_t g_t + g_e (log q_v + entropy))
// The pair (m, log s) is kept, not their sum: where a mask leaves a row with nothing but the
// type's lowest value, log s is lost in the rounding of m + log s.
// A row whose logits are all -inf has m = -inf, log s = 0, log-probabilities -inf, entropy 0 and
// a zero gradient. A NaN or +inf among a row's logits makes its results NaN.
#pragma once

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "simt.cuh"

namespace fckl {

constexpr int SCORE_THREADS = 256;
constexpr int SCORE_GV = 4;            // 16-byte vectors of a group
constexpr int SCORE_MAX_GROUPS = 8192; // group maxima that one block keeps in shared memory
constexpr int TOKENS_MAX = 1024;       // given tokens, and alternatives, of a row

// ---------------------------------------------------------------- values of a row
// max that keeps a NaN (fmaxf drops it, and a row with one would pass for a good row)
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}

// The two values of a 32-bit word, lower address first.
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __nv_bfloat16) {
  a = __uint_as_float(w << 16);
  b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  a = f.x;
  b = f.y;
}

template <typename T>
__device__ __forceinline__ void unpack16(uint4 w, float (&x)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    x[0] = __uint_as_float(w.x);
    x[1] = __uint_as_float(w.y);
    x[2] = __uint_as_float(w.z);
    x[3] = __uint_as_float(w.w);
  } else {
    unpack2(w.x, x[0], x[1], T{});
    unpack2(w.y, x[2], x[3], T{});
    unpack2(w.z, x[4], x[5], T{});
    unpack2(w.w, x[6], x[7], T{});
  }
}

// A row seen as aligned 16-byte vectors: vector i covers columns [VE i - mis, VE i - mis + VE),
// where mis is the row's distance, in values, from the 16-byte boundary below it. Rows of any
// alignment (odd V, sliced views) so keep wide loads; columns outside [0, V) are never read.
template <typename T>
struct RowVecs {
  static constexpr int VE = 16 / sizeof(T);
  const T* row;
  int V, mis, nvec;
  __device__ __forceinline__ RowVecs(const T* r, int V_) : row(r), V(V_) {
    mis = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15u) / sizeof(T));
    nvec = (V + mis + VE - 1) / VE;
  }
  __device__ __forceinline__ int col(int i) const { return i * VE - mis; }
  __device__ __forceinline__ bool whole(int i) const {
    const int c = col(i);
    return c >= 0 && c + VE <= V;
  }
  __device__ __forceinline__ uint4 raw(int i) const {
    return *reinterpret_cast<const uint4*>(row + static_cast<int64_t>(col(i)));
  }
  // Vector i as it lies in memory; -inf outside the row.
  __device__ __forceinline__ uint4 words(int i) const;
  // Values of vector i; -inf outside the row.
  __device__ __forceinline__ void load(int i, float (&x)[VE]) const {
    if (i < nvec && whole(i)) {
      unpack16<T>(raw(i), x);
    } else {
      const int c = col(i);
#pragma unroll
      for (int j = 0; j < VE; ++j) x[j] = (i < nvec && c + j >= 0 && c + j < V) ? to_f32(row[c + j]) : -INFINITY;
    }
  }
};

template <typename T>
__device__ __forceinline__ uint32_t fill_word(float v);

template <typename T>
__device__ __forceinline__ uint4 RowVecs<T>::words(int i) const {
  if (i < nvec && whole(i)) return raw(i);
  const uint32_t none = fill_word<T>(-INFINITY);
  uint4 w = make_uint4(none, none, none, none);
  if (i < nvec) {  // an end of the row
    __align__(16) T v[VE];
    *reinterpret_cast<uint4*>(v) = w;
    const int c = col(i);
#pragma unroll
    for (int j = 0; j < VE; ++j)
      if (c + j >= 0 && c + j < V) v[j] = row[c + j];
    w = *reinterpret_cast<const uint4*>(v);
  }
  return w;
}

// ---------------------------------------------------------------- running statistics
// m: maximum so far, l = sum exp(z - m), t = sum (z - m) exp(z - m).
// Both sums are formed from the difference z - m, which is exact near the maximum; it is held at or
// above -256, where the exponential is zero, so that values far below the maximum and masked ones
// add 0 * -256 rather than 0 * -inf.
struct RowStat {
  float m = -INFINITY, l = 0.f, t = 0.f;
};
constexpr float DIFF_FLOOR = -256.f;
__device__ __forceinline__ float exp_diff(float d) { return ex2_approx(d * LOG2E); }

__device__ __forceinline__ RowStat merge(const RowStat& a, const RowStat& b) {
  RowStat r;
  r.m = fmaxf(a.m, b.m);
  if (r.m == -INFINITY) {  // nothing yet on either side (or only a NaN, which the sums keep)
    r.l = a.l + b.l;
    r.t = a.t + b.t;
    return r;
  }
  const float da = fmaxf(a.m - r.m, DIFF_FLOOR), db = fmaxf(b.m - r.m, DIFF_FLOOR);
  const float fa = exp_diff(da), fb = exp_diff(db);
  // products and sums that are written out, so that every kernel rounds them alike
  r.l = fmaf(a.l, fa, __fmul_rn(b.l, fb));
  r.t = fmaf(fa, fmaf(da, a.l, a.t), __fmul_rn(fb, fmaf(db, b.l, b.t)));
  return r;
}

// Adds one vector's values, whose maximum is at most s.m (or NaN).
template <int VE>
__device__ __forceinline__ void add_values(RowStat& s, const float (&x)[VE]) {
#pragma unroll
  for (int j = 0; j < VE; ++j) {
    const float d = max_nan(x[j] - s.m, DIFF_FLOOR);
    const float e = exp_diff(d);
    s.l += e;
    s.t = fmaf(d, e, s.t);
  }
}

// The fast form of the same sums, for whole groups of 16-byte vectors: two values at a time through
// the packed fp32 instructions. Values are raised to at least low() first, which stands in for the
// floor on the difference: far below any maximum but one that is itself masked. A block whose maximum
// ends below low_limit() is summed again by add_values. Differences are halved, in the same
// instruction: half the difference of two finite numbers is finite, and finite times an exponential
// of zero is zero. (Its product with log2(e) may overflow; only the exponential takes that.)
template <typename T>
__device__ __forceinline__ float low();
template <>
__device__ __forceinline__ float low<__half>() {
  return -6e4f;
}
template <>
__device__ __forceinline__ float low<__nv_bfloat16>() {
  return -1e30f;
}
template <>
__device__ __forceinline__ float low<float>() {
  return -1e30f;
}
template <typename T>
__device__ __forceinline__ float low_limit() {
  return low<T>() * 0.5f;
}

__device__ __forceinline__ unsigned long long pack2(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2f(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Per 32-bit word of a row: the larger of two words (by value; a NaN stays), the values of a word
// raised to low(), and the word that stands for -inf.
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, __nv_bfloat16) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, __half) {
  uint32_t r;
  asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_words(uint32_t a, uint32_t b, float) {
  return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
}
__device__ __forceinline__ float max_of_word(uint32_t w, float) { return __uint_as_float(w); }
template <typename T>
__device__ __forceinline__ float max_of_word(uint32_t w, T) {
  float a, b;
  unpack2(w, a, b, T{});
  return max_nan(a, b);
}
template <typename T>
__device__ __forceinline__ uint32_t fill_word(float v) {  // v in every value of a word
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(v);
  } else {
    const T t = from_f32<T>(v);
    const uint16_t h = *reinterpret_cast<const uint16_t*>(&t);
    return h | (static_cast<uint32_t>(h) << 16);
  }
}

struct FastStat {
  float m = -INFINITY;           // maximum so far, at least low()
  unsigned long long l, t;       // l and t / 2 of RowStat, two interleaved parts each
  __device__ __forceinline__ FastStat() : l(pack2(0.f, 0.f)), t(pack2(0.f, 0.f)) {}
  __device__ __forceinline__ void raise(float to) {  // brings the sums to a new maximum
    const float d = fmaxf(m - to, DIFF_FLOOR), f = exp_diff(d);
    t = mul2(pack2(f, f), fma2(pack2(0.5f * d, 0.5f * d), l, t));
    l = mul2(pack2(f, f), l);
    m = to;
  }
  __device__ __forceinline__ void add(float a, float b) {
    const unsigned long long h = fma2(pack2(a, b), pack2(0.5f, 0.5f), pack2(-0.5f * m, -0.5f * m));
    float ya, yb;
    unpack2f(mul2(h, pack2(2.f * LOG2E, 2.f * LOG2E)), ya, yb);
    const unsigned long long e = pack2(ex2_approx(ya), ex2_approx(yb));
    l = add2(l, e);
    t = fma2(h, e, t);
  }
  __device__ __forceinline__ RowStat stat() const {
    RowStat s;
    float a, b;
    unpack2f(l, a, b);
    s.l = a + b;
    unpack2f(t, a, b);
    s.t = 2.f * (a + b);
    s.m = m;
    return s;
  }
};

// Order of (logit, id) pairs in one 64-bit number: larger logit first, then smaller id.
__device__ __forceinline__ uint32_t logit_key(float z) { return order_key(z + 0.f); }  // -0 counts as +0
__device__ __forceinline__ unsigned long long pair_key(float z, int id) {
  return (static_cast<unsigned long long>(logit_key(z)) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

// Sum over the block of one int per thread; every thread gets it. `buf` holds one int per warp.
template <int NT>
__device__ __forceinline__ int block_sum(int v, int* buf) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) s += buf[w];
  return s;
}

// Descending bitonic sort of n (a power of two) 64-bit keys in shared memory.
template <int NT>
__device__ __forceinline__ void block_sort(unsigned long long* a, int n) {
  for (int k = 2; k <= n; k <<= 1) {
    for (int j = k >> 1; j > 0; j >>= 1) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += NT) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const unsigned long long x = a[lo], y = a[hi];
        if ((x < y) == ((lo & k) == 0)) {
          a[lo] = y;
          a[hi] = x;
        }
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ int pow2_at_least(int n) { return n <= 1 ? 1 : 1 << (32 - __clz(n - 1)); }

// Orders n distinct keys in shared memory, largest first. Up to ORDER_MAX keys each one's place is the
// number of larger ones (n reads and two barriers instead of a sort's dozens); `a` has room for the
// next power of two.
constexpr int ORDER_MAX = 256;
template <int NT>
__device__ __forceinline__ void block_order(unsigned long long* a, int n) {
  const int tid = threadIdx.x;
  if (n <= ORDER_MAX) {
    constexpr int PER = ORDER_MAX / NT;
    __syncthreads();
    unsigned long long mine[PER];
    int place[PER];
#pragma unroll
    for (int b = 0; b < PER; ++b) {
      const int i = b * NT + tid;
      mine[b] = i < n ? a[i] : 0ull;
      place[b] = 0;
      if ((i & ~31) < n) {  // warps that hold a key
        const ulonglong2* two = reinterpret_cast<const ulonglong2*>(a);
#pragma unroll 4
        for (int j = 0; j < n / 2; ++j) {
          const ulonglong2 v = two[j];
          place[b] += (v.x > mine[b]) + (v.y > mine[b]);
        }
        if (n & 1) place[b] += a[n - 1] > mine[b];
      }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < PER; ++b)
      if (b * NT + tid < n) a[place[b]] = mine[b];
    __syncthreads();
    return;
  }
  const int n2 = pow2_at_least(n);
  for (int i = n + tid; i < n2; i += NT) a[i] = 0ull;
  block_sort<NT>(a, n2);
}

// 16 bytes from global to shared memory, asynchronously; the groups of copies finish in order.
__device__ __forceinline__ void copy_async16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_async_wait() {  // all but the last PENDING groups are there
  asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
}

struct ScoreParams {
  const void* logits;
  int64_t ld;
  const int32_t* tokens;
  int V, T, top;
  int cand_cap;  // candidates that fit in shared memory (a power of two)
  int groups;    // group maxima kept per block
  int gshift;    // 2^gshift steps of SCORE_GV vectors per thread make up a group
  int split;     // blocks (of a cluster) per row
  float* logp;
  float* entropy;
  float* norm;
  int32_t* top_idx;
  float* top_logp;
  unsigned* status;
};

// One block of NT threads per row, or a cluster of `split` blocks that share a row's vectors in order.
//
// Statistics: each thread runs over its vectors once and keeps (m, l, t); the block and then the
// cluster merge them in a fixed order.
// Alternatives: the pass also leaves in shared memory the maximum of every group of vectors (the
// ones that one thread took in one step). tau is a lower bound on the block's K-th largest logit:
// at least K threads, or groups, have their maximum at or above it (or tau = -inf).
// Only groups whose maximum reaches tau can hold a logit at or above it; there are about K, and they
// are read again (from L2) to collect those logits. They are K or more, and the set is among them.
// Where they are more than there is room for (equal logits, masked rows):
//   the logits above tau, C of them, are collected instead. C < K: the K-th largest logit is tau
//   itself, and the first K - C ids with logit tau, found by a scan in id order, complete the set.
//   C above the room: tau is raised by bisection over the listed groups' logits until the logits at
//   or above it fit, or it is the K-th largest itself, which is the case before.
// The set is sorted by (logit, id). Each block of a cluster does this for its share of the row,
// and block 0 sorts the blocks' sets together. Exact for every input, ties included.
//
// What bounds it: with many rows HBM. 4096 x 128256 bf16 takes 170 us without alternatives (6.2 TB/s,
// 0.91 of the copy bandwidth), 189 with one and 225 with 100: the listed groups are read again
// when part of the 600 rows in flight (155 MB) has left L2, and a block's selection is about 8 us of
// latency beside the other blocks' streams. A thread's loads run a step ahead of its sums, and two
// values share an instruction where they can (310 us without either). fp32 rows have half the
// arithmetic per byte and want more bytes on their way than registers hold: with many long rows the
// loads go through shared memory, two steps ahead (RING; 2048 x 128256, one alternative: 202 to 178 us; bf16 loses 5%). With few rows it is latency:
// 6.5 us for one row of 201088 over eight blocks, 12 us with 20 alternatives. With many short rows it is
// the latency of a row's steps too: smaller blocks put more rows on an SM (launch_token_logprobs).
template <typename T, int NT, int RING>
__global__ void __launch_bounds__(NT) token_logprobs_kernel(const ScoreParams p) {
  namespace cg = cooperative_groups;
  constexpr int VE = 16 / sizeof(T);
  constexpr int WARPS = NT / 32;
  constexpr int SETS = NT < SCORE_THREADS ? 2 : 1;  // maxima of a thread that bound the alternatives
  constexpr int BINS = SETS * NT;
  extern __shared__ __align__(16) unsigned char score_smem[];
  unsigned long long* cand = reinterpret_cast<unsigned long long*>(score_smem);  // [cand_cap]
  uint32_t* gkey = reinterpret_cast<uint32_t*>(cand + (p.top ? p.cand_cap : 0));  // [groups]
  uint16_t* live = reinterpret_cast<uint16_t*>(gkey + p.groups);                 // [groups]
  uint4* ring = nullptr;  // [RING][SCORE_GV][NT]
  if constexpr (RING > 0) {  // the candidates and the listed groups take the ring's place after the row
    gkey = reinterpret_cast<uint32_t*>(score_smem);
    ring = reinterpret_cast<uint4*>(gkey + (p.top ? p.groups : 0));
    cand = reinterpret_cast<unsigned long long*>(ring);
    live = reinterpret_cast<uint16_t*>(cand + p.cand_cap);
  }
  __shared__ RowStat sstat[WARPS];
  __shared__ RowStat bstat;  // this block's share of the row
  __shared__ int ibuf[WARPS];
  __shared__ uint32_t tkey[BINS], tau_s;
  __shared__ int n_cand, n_live;

  cg::cluster_group cluster = cg::this_cluster();
  const int rank = p.split > 1 ? static_cast<int>(cluster.block_rank()) : 0;
  const int64_t row = blockIdx.x / p.split;
  const RowVecs<T> rv(static_cast<const T*>(p.logits) + row * p.ld, p.V);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // this block's vectors [v0, v1) and columns [c0, c1)
  const int per = (rv.nvec + p.split - 1) / p.split;
  const int v0 = min(rank * per, rv.nvec), v1 = min(v0 + per, rv.nvec);
  const int c0 = max(0, rv.col(v0)), c1 = min(p.V, rv.col(v1));

  // ---- statistics and group maxima
  constexpr int STEP = NT * SCORE_GV;
  const int steps = (v1 - v0 + STEP - 1) / STEP;
  float tmax[SETS];  // this thread's largest logits (two sets: of even and of odd vectors)
#pragma unroll
  for (int b = 0; b < SETS; ++b) tmax[b] = -INFINITY;
  RowStat s;
  {
    FastStat f;
    float gmax = -INFINITY;
    const uint32_t lo = fill_word<T>(low<T>());
    uint4 next[SCORE_GV];
    auto fetch = [&](int st) {
#pragma unroll
      for (int j = 0; j < SCORE_GV; ++j) {
        const int i = v0 + st * STEP + j * NT + tid;
        if constexpr (RING == 0) {
          next[j] = rv.words(i < v1 ? i : rv.nvec);
        } else if (i < v1 && rv.whole(i)) {  // a thread reads what it copies: no barrier
          copy_async16(ring + (st % RING * SCORE_GV + j) * NT + tid, rv.row + static_cast<int64_t>(rv.col(i)));
        }
      }
      if constexpr (RING > 0) copy_async_commit();  // steps past the last one are empty
    };
#pragma unroll
    for (int st = 0; st < (RING ? RING : 1); ++st) fetch(st);
    for (int st = 0, in_group = 0, g = tid; st < steps; ++st) {
      uint32_t w[4 * SCORE_GV];
      if constexpr (RING > 0) copy_async_wait<RING - 1>();
#pragma unroll
      for (int j = 0; j < SCORE_GV; ++j) {
        if constexpr (RING > 0) {
          const int i = v0 + st * STEP + j * NT + tid;
          next[j] = i < v1 && rv.whole(i) ? ring[(st % RING * SCORE_GV + j) * NT + tid]
                                          : rv.words(i < v1 ? i : rv.nvec);
        }
        w[4 * j] = next[j].x;
        w[4 * j + 1] = next[j].y;
        w[4 * j + 2] = next[j].z;
        w[4 * j + 3] = next[j].w;
      }
      if (RING > 0 || st + 1 < steps) fetch(st + (RING ? RING : 1));  // on its way while this step is summed
      float m = 0.f;
#pragma unroll
      for (int b = 0; b < SETS; ++b) {
        uint32_t wm = w[4 * b];
#pragma unroll
        for (int j = 4 * b + 1; j < 4 * SCORE_GV; ++j)
          if (j / 4 % SETS == b) wm = max_words(wm, w[j], T{});
        const float mb = max_of_word(wm, T{});
        tmax[b] = fmaxf(tmax[b], mb);
        m = b ? max_nan(m, mb) : mb;
      }
      const float mc = fmaxf(m, low<T>());
      if (mc > f.m) f.raise(mc);
#pragma unroll
      for (int j = 0; j < 4 * SCORE_GV; j += sizeof(T) / 2) {
        float a, b;
        if constexpr (sizeof(T) == 4) {
          a = __uint_as_float(max_words(w[j], lo, T{}));
          b = __uint_as_float(max_words(w[j + 1], lo, T{}));
        } else {
          unpack2(max_words(w[j], lo, T{}), a, b, T{});
        }
        f.add(a, b);
      }
      if (p.top) {
        gmax = fmaxf(gmax, m);
        if (++in_group == 1 << p.gshift || st == steps - 1) {
          gkey[g] = logit_key(gmax);
          g += NT;
          gmax = -INFINITY;
          in_group = 0;
        }
      }
    }
    s = f.stat();
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    RowStat b;
    b.m = __shfl_xor_sync(0xffffffffu, s.m, o);
    b.l = __shfl_xor_sync(0xffffffffu, s.l, o);
    b.t = __shfl_xor_sync(0xffffffffu, s.t, o);
    s = merge(s, b);
  }
  if (lane == 0) sstat[warp] = s;
  if (tid == 0) n_cand = n_live = 0;
  __syncthreads();
  s = sstat[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) s = merge(s, sstat[w]);
  if (s.m < low_limit<T>()) {  // masked throughout (the same for the whole block)
    const bool nan = s.l != s.l;
    s = RowStat();
    if (!__syncthreads_or(fmaxf(tmax[0], tmax[SETS - 1]) > -INFINITY || nan)) {
      // with -inf alone: nothing is left
    } else {  // exact sums
      for (int i0 = v0 + tid; i0 < v1; i0 += STEP) {
        uint4 w[SCORE_GV];
#pragma unroll
        for (int j = 0; j < SCORE_GV; ++j) {
          const int i = i0 + j * NT;
          w[j] = rv.words(i < v1 ? i : rv.nvec);
        }
#pragma unroll
        for (int j = 0; j < SCORE_GV; ++j) {
          float x[VE];
          unpack16<T>(w[j], x);
          float m = x[0];
#pragma unroll
          for (int e = 1; e < VE; ++e) m = max_nan(m, x[e]);
          if (!(m <= s.m)) {
            RowStat none;
            none.m = m;
            s = merge(s, none);
          }
          if (s.m != -INFINITY || m != m) add_values<VE>(s, x);
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      RowStat b;
      b.m = __shfl_xor_sync(0xffffffffu, s.m, o);
      b.l = __shfl_xor_sync(0xffffffffu, s.l, o);
      b.t = __shfl_xor_sync(0xffffffffu, s.t, o);
      s = merge(s, b);
    }
    __syncthreads();
    if (lane == 0) sstat[warp] = s;
    __syncthreads();
    s = sstat[0];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) s = merge(s, sstat[w]);
  }
  if (tid == 0) bstat = s;

  // ---- this block's alternatives: cand[0..k), sorted
  const int k = min(p.top, c1 - c0);
  if (k > 0 && !(s.l != s.l)) {
    static_assert(SCORE_GV == 4 && (NT & (NT - 1)) == 0, "shifts in item_vec");
    const int item_bits = p.gshift + 2;  // of an item's number: its place in the group
    const int ng = ((steps - 1 >> p.gshift) + 1) * NT;
    uint32_t tau = order_key(-INFINITY);
    if (k <= BINS / 2) {
      // the k-th largest of the threads' maxima, or a little less, by one warp. Each is the largest of
      // many logits where rows are long, so few more than k logits lie above it.
#pragma unroll
      for (int b = 0; b < SETS; ++b) tkey[b * NT + tid] = logit_key(tmax[b]);
      __syncthreads();
      if (warp == 0) {
        uint32_t key[BINS / 32], lo = 0xffffffffu, hi = 0;
#pragma unroll
        for (int j = 0; j < BINS / 32; ++j) {
          key[j] = tkey[32 * j + lane];
          lo = min(lo, key[j]);
          hi = max(hi, key[j]);
        }
        lo = __reduce_min_sync(0xffffffffu, lo);      // reached by all
        hi = __reduce_max_sync(0xffffffffu, hi) + 1;  // reached by none (a key is never the largest uint32)
        // a little more, but not so much that nearly every thread counts
        const int bins = min(BINS, v1 - v0);
        const int enough = k + min(k / 16 + 4, max(0, bins - k) / 4);
        // keys of 16-bit logits lie at least KEY_STEP apart: finer differences decide nothing
        constexpr uint32_t KEY_STEP = sizeof(T) == 4 ? 1u : 1u << 13;
        while (hi - lo > KEY_STEP) {
          const uint32_t mid = lo + (hi - lo) / 2;
          int n = 0;
#pragma unroll
          for (int j = 0; j < BINS / 32; ++j) n += key[j] >= mid;
          n = __reduce_add_sync(0xffffffffu, n);
          if (n >= k) {
            lo = mid;
            if (n <= enough) break;
          } else {
            hi = mid;
          }
        }
        if (lane == 0) tau_s = lo;
      }
      __syncthreads();
      tau = max(tau, tau_s);
    } else if (ng >= k) {
      // the largest prefix of key bits that at least k group maxima reach, refined only until few
      // more than k do
      const int enough = k + k / 4 + 16;
      uint32_t prefix = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const uint32_t c = prefix | (1u << bit);
        int n = 0;
        for (int g = tid; g < ng; g += NT) n += gkey[g] >= c;
        n = block_sum<NT>(n, ibuf);
        if (n >= k) {
          prefix = c;
          if (n <= enough) break;
        }
      }
      tau = max(prefix, tau);
    }
    auto list = [&](uint32_t cut) {  // groups that hold a logit at or above cut
      __syncthreads();
      if (tid == 0) n_live = n_cand = 0;
      __syncthreads();
      for (int g = tid; g < ng; g += NT)
        if (gkey[g] >= cut) live[atomicAdd(&n_live, 1)] = static_cast<uint16_t>(g);
      __syncthreads();
    };
    auto item_vec = [&](int it) {  // vector of item it of the listed groups
      const uint32_t g = live[it >> item_bits], j = it & ((1 << item_bits) - 1);
      return v0 + static_cast<int>(((g / NT << item_bits) + j) * NT + g % NT);
    };
    // logits at or above cut into cand, as many as fit; n_cand counts them all. Columns outside the
    // row read as -inf, which no cut above it takes.
    auto collect = [&](uint32_t cut) {
      const int items = n_live << item_bits;
      constexpr int AT_ONCE = 4;  // vectors of a thread whose loads are issued together
      for (int it0 = tid; it0 < items; it0 += AT_ONCE * NT) {
        uint4 w[AT_ONCE];
        int vec[AT_ONCE];
#pragma unroll
        for (int b = 0; b < AT_ONCE; ++b) {
          const int it = it0 + b * NT;
          const int i = it < items ? item_vec(it) : v1;
          vec[b] = i < v1 ? i : rv.nvec;  // no such vector: -inf
          w[b] = rv.words(vec[b]);
        }
#pragma unroll
        for (int b = 0; b < AT_ONCE; ++b) {
          const uint32_t top2 = max_words(max_words(w[b].x, w[b].y, T{}), max_words(w[b].z, w[b].w, T{}), T{});
          if (logit_key(max_of_word(top2, T{})) < cut) continue;  // most of a group's vectors
          float x[VE];
          unpack16<T>(w[b], x);
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            if (logit_key(x[e]) >= cut) {
              const int at = atomicAdd(&n_cand, 1);
              if (at < p.cand_cap) cand[at] = pair_key(x[e], rv.col(vec[b]) + e);
            }
          }
        }
      }
      __syncthreads();
    };
    const uint32_t none = order_key(-INFINITY);
    list(tau);
    if (tau > none && n_live <= p.cand_cap) collect(tau);
    if (tau == none || n_live > p.cand_cap || n_cand > p.cand_cap) {
      // too many at tau (equal logits, or a mask): those above it, and then the first ones at it
      list(tau + 1);
      collect(tau + 1);
      if (n_cand > p.cand_cap) {
        // bisect: lo is reached by at least k logits; stop when those at or above it fit
        const int items = n_live << item_bits;
        uint32_t lo = tau, hi = 0xffffffffu;
        bool fits = false;
        while (!fits && hi - lo > 1) {
          const uint32_t mid = lo + (hi - lo) / 2;
          int n = 0;
          for (int it = tid; it < items; it += NT) {
            const int i = item_vec(it);
            if (i >= v1) continue;
            float x[VE];
            rv.load(i, x);
#pragma unroll
            for (int e = 0; e < VE; ++e) n += logit_key(x[e]) >= mid;
          }
          n = block_sum<NT>(n, ibuf);
          if (n >= k) {
            lo = mid;
            fits = n <= p.cand_cap;
          } else {
            hi = mid;
          }
        }
        tau = lo;
        __syncthreads();
        if (tid == 0) n_cand = 0;
        __syncthreads();
        collect(fits ? tau : tau + 1);
      }
    }
    int c = min(n_cand, p.cand_cap);  // more only if the logits changed while they were read
    if (c < k) {
      // ids in order whose logit is tau, until the set is complete
      for (int base = v0; base < v1 && c < k; base += NT) {
        const int i = base + tid;
        uint32_t hit = 0;
        float x[VE];
        if (i < v1) {
          rv.load(i, x);
          const int col = rv.col(i);
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (col + e >= 0 && col + e < p.V && logit_key(x[e]) == tau) hit |= 1u << e;
        }
        const int mine = __popc(hit);
        int before = mine;  // inclusive prefix within the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, before, o);
          if (lane >= o) before += v;
        }
        __syncthreads();
        if (lane == 31) ibuf[warp] = before;
        __syncthreads();
        int total = 0, at = c + before - mine;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          if (w < warp) at += ibuf[w];
          total += ibuf[w];
        }
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (hit & (1u << e)) {
            if (at < k) cand[at] = pair_key(x[e], rv.col(i) + e);
            ++at;
          }
        c += total;
      }
      c = min(c, k);
    }
    block_order<NT>(cand, c);
  }

  // ---- the whole row, in block 0 of the cluster
  if (p.split > 1) {
    cluster.sync();
    if (rank == 0) {
      const RowStat mine = s;
      s = mine;
      for (int r = 1; r < p.split; ++r) s = merge(s, *cluster.map_shared_rank(&bstat, r));
      if (p.top && !(s.l != s.l)) {
        int n = k;
        for (int r = 1; r < p.split; ++r) {
          const int a = max(0, rv.col(min(r * per, rv.nvec)));
          const int b = min(p.V, rv.col(min(min(r * per, rv.nvec) + per, rv.nvec)));
          const int kr = min(p.top, max(0, b - a));
          const unsigned long long* theirs = cluster.map_shared_rank(cand, r);
          for (int i = tid; i < kr; i += NT) cand[n + i] = theirs[i];
          n += kr;
        }
        block_order<NT>(cand, n);
      }
    }
    cluster.sync();  // the others' shared memory has been read
    if (rank != 0) return;
  }

  const bool nothing = s.m == -INFINITY && s.l == 0.f;
  const float log_s = nothing ? 0.f : logf(s.l);
  if (tid == 0) {
    const float ent = nothing ? 0.f : log_s - s.t / s.l;
    p.entropy[row] = ent < 0.f ? 0.f : ent;  // rounding may leave a sharp row just below zero
    p.norm[2 * row] = s.m;
    p.norm[2 * row + 1] = log_s;
  }
  for (int t = tid; t < p.T; t += NT) {
    const int id = p.tokens[row * p.T + t];
    float lp = 0.f;
    if (id < -1 || id >= p.V) {
      atomicOr(p.status, ST_BAD_INDEX);
      lp = NAN;
    } else if (id >= 0) {
      lp = nothing ? -INFINITY : (to_f32(rv.row[id]) - s.m) - log_s;
    }
    p.logp[row * p.T + t] = lp;
  }
  const bool bad = s.l != s.l;
  for (int i = tid; i < p.top; i += NT) {
    int id = i;
    float lp = NAN;
    if (!bad) {
      const unsigned long long c = cand[i];
      id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(c));
      lp = nothing ? -INFINITY : (order_key_inv(static_cast<uint32_t>(c >> 32)) - s.m) - log_s;
    }
    p.top_idx[row * p.top + i] = id;
    p.top_logp[row * p.top + i] = lp;
  }
}

// ---------------------------------------------------------------- gradient
struct ScoreGradParams {
  const void* logits;  // may be the same array as dlogits
  int64_t ld, ld_out;
  const int32_t* tokens;
  int V, T, segs;
  const float* norm;
  const float* entropy;
  const float* g_logp;
  const float* g_entropy;  // null: zero
  void* dlogits;
  unsigned* status;
};
constexpr int SCORE_GRAD_VECS = 8;  // vectors per thread of a segment
constexpr int SCORE_GRAD_RESIDENT = 5;  // blocks of 256 threads, of 47 registers each, on an SM
constexpr int SCORE_GRAD_TOKENS = TOKENS_MAX / SCORE_THREADS;  // given tokens per thread

// HBM-bound: 345 us at 4096 x 128256 bf16, read and written once (6.1 TB/s).
// A block takes one segment of a row: dense part first, then the (few) tokens of the row that
// fall into the segment, each written once with all its slots' gradients. Their logits are read
// before anything is written, so dlogits may be logits itself. A row without any upstream
// gradient is written as zeros without being read (positions that a loss masks out may hold
// anything).
template <typename T, int NT>
__global__ void __launch_bounds__(NT, SCORE_GRAD_RESIDENT * SCORE_THREADS / NT) token_logprobs_grad_kernel(const ScoreGradParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int WARPS = NT / 32;
  constexpr int PER = SCORE_GRAD_TOKENS;
  __shared__ int ids[PER * NT];
  __shared__ float gs[PER * NT];
  __shared__ float wsum[WARPS];
  __shared__ int wany[WARPS];
  const int64_t row = blockIdx.x / p.segs;
  const int seg = static_cast<int>(blockIdx.x % p.segs);
  const T* zrow = static_cast<const T*>(p.logits) + row * p.ld;
  T* orow = static_cast<T*>(p.dlogits) + row * p.ld_out;
  const RowVecs<T> ov(orow, p.V);  // vectors of the output: every store is wide but the ends
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (ov.nvec + p.segs - 1) / p.segs;  // at most SCORE_GRAD_VECS NT
  const int v0 = seg * per;
  if (v0 >= ov.nvec) return;
  const int v1 = min(v0 + per, ov.nvec);
  const int c0 = max(0, ov.col(v0)), c1 = min(p.V, ov.col(v1));

  // the row's tokens and their gradients
  float sg = 0.f;
  int any = 0;
  float zt[PER];
#pragma unroll
  for (int a = 0; a < PER; ++a) {
    const int t = a * NT + tid;
    zt[a] = 0.f;
    if (t < p.T) {
      const int id = p.tokens[row * p.T + t];
      const bool ok = id >= 0 && id < p.V;
      if (id < -1 || id >= p.V) atomicOr(p.status, ST_BAD_INDEX);
      const float g = ok ? p.g_logp[row * p.T + t] : 0.f;
      ids[t] = ok ? id : -1;
      gs[t] = g;
      sg += g;
      any |= g != 0.f;
      if (ok && id >= c0 && id < c1) zt[a] = to_f32(zrow[id]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sg += __shfl_xor_sync(0xffffffffu, sg, o);
  any = __any_sync(0xffffffffu, any);
  if (lane == 0) {
    wsum[warp] = sg;
    wany[warp] = any;
  }
  __syncthreads();
  sg = 0.f;
  any = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    sg += wsum[w];
    any |= wany[w];
  }
  const float ge = p.g_entropy ? p.g_entropy[row] : 0.f, ent = p.entropy[row];
  const float m = p.norm[2 * row], log_s = p.norm[2 * row + 1];
  // nothing upstream, or nothing left by the mask (log s is 0 there, and NaN if a NaN is among the -inf)
  const bool zero = (!any && ge == 0.f) || (m == -INFINITY && log_s == 0.f);
  // taken from memory beside ge (behind it: 406 us for 346 at 4096 x 128256), left out where it plays no part
  const float a0 = ge == 0.f ? sg : sg + ge * ent;
  // dense part: - q (a0 + ge log q)
  auto dense = [&](float z) {
    const float lq = max_nan((z - m) - log_s, DIFF_FLOOR);  // q is 0 below: 0 * finite, for any ge
    return -exp_diff(lq) * fmaf(ge, lq, a0);
  };
  const int shift = static_cast<int>((reinterpret_cast<uintptr_t>(zrow) & 15u) / sizeof(T)) - ov.mis;
  const bool same = shift == 0;  // logits and output vectors line up
  constexpr int GB = 4;  // vectors whose loads are issued together (stores may be to the same array)
  uint4 ahead[GB];
#pragma unroll
  for (int j = 0; j < SCORE_GRAD_VECS; ++j) {
    const int i = v0 + j * NT + tid;
    if (j % GB == 0) {
#pragma unroll
      for (int b = 0; b < GB; ++b) {
        const int ib = i + b * NT;
        if (same && !zero && ib < v1 && ov.whole(ib)) ahead[b] = *reinterpret_cast<const uint4*>(zrow + ov.col(ib));
      }
    }
    if (i >= v1) continue;
    const int c = ov.col(i);
    if (ov.whole(i)) {
      float x[VE];
      if (zero) {
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = 0.f;
      } else {
        if (same) {
          unpack16<T>(ahead[j % GB], x);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e) x[e] = to_f32(zrow[c + e]);
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) x[e] = dense(x[e]);
      }
      __align__(16) T y[VE];
#pragma unroll
      for (int e = 0; e < VE; ++e) y[e] = from_f32<T>(x[e]);
      *reinterpret_cast<uint4*>(orow + c) = *reinterpret_cast<const uint4*>(y);
    } else {
#pragma unroll
      for (int e = 0; e < VE; ++e)
        if (c + e >= 0 && c + e < p.V) orow[c + e] = from_f32<T>(zero ? 0.f : dense(to_f32(zrow[c + e])));
    }
  }
  if (zero) return;
  __syncthreads();  // the dense values are written; the tokens' entries replace theirs
#pragma unroll
  for (int a = 0; a < PER; ++a) {
    const int t = a * NT + tid;
    if (t >= p.T) continue;
    const int id = ids[t];
    if (id < c0 || id >= c1) continue;
    float g = 0.f;
    bool first = true;
    for (int u = 0; u < p.T; ++u) {
      if (ids[u] != id) continue;
      if (u < t) {
        first = false;
        break;
      }
      g += gs[u];
    }
    if (first) orow[id] = from_f32<T>(dense(zt[a]) + g);
  }
}

}  // namespace fckl
