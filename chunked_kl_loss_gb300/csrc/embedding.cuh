// The tied embedding: rows of W [V, d] for given tokens times a scale, and the gradient of W.
//
//   y_n   = s W[t_n]                               (t_n = -1: a row of zeros)
//   dW[v] = (dW[v] +) s sum over n with t_n = v of g_n
//
// The gradient's positions are first put in the order of their tokens, equal tokens in the order of
// their positions (a radix sort by one cluster). Blocks then walk tiles of the ordered list, each over
// its own columns: the rows of a token that begins and ends within a tile are summed in registers and
// written once; a token that crosses a tile's edge leaves one partial sum per tile, and those are added
// in the order of the tiles by a second kernel. So every row of dW has one writer, and the sums, all in
// fp32, one order: the same call gives the same bits.
#pragma once

#include <cooperative_groups.h>

#include "score.cuh"

namespace fckl {

// E values that are loaded or stored together (a power of two, at most 16 bytes of T).
template <typename T, int E>
struct alignas(E * sizeof(T)) Pack {
  T v[E];
};

// ---------------------------------------------------------------- lookup
constexpr int EMBED_THREADS = 256;

// TPR threads to a row, E values at a time.
template <typename T, int E, int TPR>
__global__ void __launch_bounds__(EMBED_THREADS)
    embedding_kernel(const T* __restrict__ W, int64_t ldw, const int32_t* __restrict__ tokens, int64_t N, int d, int V,
                     float scale, T* __restrict__ out, int64_t ld_out, unsigned* status) {
  const int lane = threadIdx.x % TPR;
  const int64_t n = int64_t(blockIdx.x) * (EMBED_THREADS / TPR) + threadIdx.x / TPR;
  if (n >= N) return;
  const int t = tokens[n];
  const bool in = t >= 0 && t < V;
  if (!in && t != -1 && lane == 0) atomicOr(status, ST_BAD_INDEX);
  const T* src = W + int64_t(in ? t : 0) * ldw;
  T* dst = out + n * ld_out;
  using P = Pack<T, E>;
  const float fill = t == -1 ? 0.f : NAN;
  constexpr int U = 4;
  for (int c0 = lane * E; c0 < d; c0 += U * TPR * E) {
    P x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * TPR * E;
      if (in && c < d) x[u] = *reinterpret_cast<const P*>(src + c);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int c = c0 + u * TPR * E;
      if (c >= d) break;
#pragma unroll
      for (int j = 0; j < E; ++j) x[u].v[j] = from_f32<T>(in ? to_f32(x[u].v[j]) * scale : fill);
      *reinterpret_cast<P*>(dst + c) = x[u];
    }
  }
}

// ---------------------------------------------------------------- positions in the order of their tokens
constexpr int SORT_THREADS = 1024;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 8;                        // per thread and tile
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;
constexpr int SORT_BITS = 9;                         // of a digit at most
constexpr int SORT_BINS = 1 << SORT_BITS;

struct SortParams {
  const int32_t* tokens;
  int N, V;
  int passes, bits;     // digits and bits of each
  int per_cta;          // positions of one block of the cluster, a multiple of SORT_TILE or all
  uint2* a;             // (token, position), written by the even passes
  uint2* b;             // and by the odd ones
  unsigned* status;
};

// Least significant digit first; one cluster. Empty slots and bad ids take the key V, so that they come
// last. Each pass: the digits' numbers per block, their places over the whole cluster, then tile by tile
// the items' ranks among equal digits (in the order of the warps, of a warp's rounds and of its lanes).
__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ unsigned hist[SORT_BINS];                    // this block's numbers
  __shared__ unsigned place[SORT_BINS];                   // where its next item of a digit goes
  __shared__ unsigned sums[SORT_WARPS];
  __shared__ unsigned short wcount[SORT_WARPS][SORT_BINS];  // a tile's numbers per warp, then their ranks
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = cluster.block_rank(), blocks = cluster.num_blocks();
  const int64_t begin64 = int64_t(rank) * p.per_cta;
  const int begin = static_cast<int>(min(begin64, int64_t(p.N)));
  const int end = static_cast<int>(min(begin64 + p.per_cta, int64_t(p.N)));
  if (rank == 0 && tid == 0) *p.status = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits;
    const unsigned dmask = (1u << p.bits) - 1u;
    const uint2* from = pass & 1 ? p.a : p.b;
    uint2* to = pass & 1 ? p.b : p.a;
    auto item = [&](int i) -> uint2 {
      if (pass) return from[i];
      const int t = p.tokens[i];
      return make_uint2(t >= 0 && t < p.V ? t : p.V, i);
    };
    if (tid < SORT_BINS) hist[tid] = 0;
    __syncthreads();
    for (int i = begin + tid; i < end; i += SORT_THREADS) atomicAdd(&hist[(item(i).x >> shift) & dmask], 1u);
    cluster.sync();
    // place = items of smaller digits anywhere + items of this digit in earlier blocks
    unsigned total = 0, before = 0;
    if (tid < SORT_BINS) {
      for (int b = 0; b < blocks; ++b) {
        const unsigned c = *cluster.map_shared_rank(&hist[tid], b);
        if (b < rank) before += c;
        total += c;
      }
    }
    unsigned run = total;  // inclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const unsigned up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    if (tid < SORT_BINS) {
      unsigned lower = 0;
      for (int w = 0; w < warp; ++w) lower += sums[w];
      place[tid] = lower + run - total + before;
    }
    for (int t0 = begin; t0 < end; t0 += SORT_TILE) {
      for (int i = tid; i < SORT_WARPS * SORT_BINS / 2; i += SORT_THREADS) reinterpret_cast<unsigned*>(wcount)[i] = 0;
      __syncthreads();
      uint2 x[SORT_ITEMS];
      unsigned short order[SORT_ITEMS];
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        const int i = t0 + (warp * SORT_ITEMS + k) * 32 + lane;
        if (i < end) x[k] = item(i);
      }
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        const int i = t0 + (warp * SORT_ITEMS + k) * 32 + lane;
        const unsigned digit = i < end ? (x[k].x >> shift) & dmask : ~0u;
        const unsigned same = __match_any_sync(0xffffffffu, digit);
        unsigned old = 0;
        if (digit != ~0u) old = wcount[warp][digit];
        __syncwarp();
        order[k] = static_cast<unsigned short>(old + __popc(same & ((1u << lane) - 1u)));
        if (digit != ~0u && lane == __ffs(same) - 1)
          wcount[warp][digit] = static_cast<unsigned short>(old + __popc(same));
        __syncwarp();
      }
      __syncthreads();
      unsigned in_tile = 0;
      if (tid < SORT_BINS) {
        for (int w = 0; w < SORT_WARPS; ++w) {
          const unsigned c = wcount[w][tid];
          wcount[w][tid] = static_cast<unsigned short>(in_tile);
          in_tile += c;
        }
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        const int i = t0 + (warp * SORT_ITEMS + k) * 32 + lane;
        if (i < end) {
          const unsigned digit = (x[k].x >> shift) & dmask;
          to[place[digit] + wcount[warp][digit] + order[k]] = x[k];
        }
      }
      __syncthreads();
      if (tid < SORT_BINS) place[tid] += in_tile;
    }
    __threadfence();
    cluster.sync();  // the pass is written, and every block has read the others' numbers
  }
  // ids outside [-1, V), once
  bool bad = false;
  for (int i = begin + tid; i < end; i += SORT_THREADS) {
    const int t = p.tokens[i];
    bad |= t < -1 || t >= p.V;
  }
  if (bad) atomicOr(p.status, ST_BAD_INDEX);
}

// ---------------------------------------------------------------- sums by token
constexpr int GSUM_THREADS = 128;
constexpr int GSUM_TILE_MAX = 64;  // entries of a tile at most
constexpr int GSUM_AHEAD = 8;      // rows loaded ahead

struct EmbedGradParams {
  const uint2* list;  // (token, position) in order
  int N, V, d;
  const void* g;
  int64_t ldg;
  void* dW;
  float scale;
  int tile, tiles;     // entries of a tile, tiles
  int slices;          // column slices
  int64_t sum_blocks;  // blocks that sum; the others write zeros
  int fill_rows;       // rows of one of those
  float* partial;      // [tiles][2][ldp]: what a tile adds to a token begun before it; what it begins
  int64_t ldp;
};

template <typename O, int E, bool ADD>
__device__ __forceinline__ void write_gradient(O* at, const float (&acc)[E], float scale) {
  using P = Pack<O, (E * sizeof(O) > 16 ? 16 / sizeof(O) : E)>;
  constexpr int EP = sizeof(P) / sizeof(O);
#pragma unroll
  for (int q = 0; q < E; q += EP) {
    P x;
    if constexpr (ADD) x = *reinterpret_cast<const P*>(at + q);
#pragma unroll
    for (int j = 0; j < EP; ++j) {
      if constexpr (ADD) x.v[j] = from_f32<O>(fmaf(scale, acc[q + j], to_f32(x.v[j])));
      else x.v[j] = from_f32<O>(scale * acc[q + j]);
    }
    *reinterpret_cast<P*>(at + q) = x;
  }
}

// First entry of the list whose token is at least v.
__device__ __forceinline__ int lower_bound(const uint2* list, int N, unsigned v) {
  int lo = 0, hi = N;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (list[mid].x < v) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <typename T, typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS) embedding_grad_kernel(const EmbedGradParams p) {
  __shared__ uint2 entry[GSUM_TILE_MAX + 2];
  __shared__ unsigned char present[GSUM_THREADS];
  const int tid = threadIdx.x;
  O* dW = static_cast<O*>(p.dW);
  if (blockIdx.x >= p.sum_blocks) {  // zeros for the rows of tokens that do not occur
    const int64_t r0 = (blockIdx.x - p.sum_blocks) * p.fill_rows;
    const int rows = static_cast<int>(min(int64_t(p.fill_rows), p.V - r0));
    if (tid < rows) {
      const int at = lower_bound(p.list, p.N, static_cast<unsigned>(r0) + tid);
      present[tid] = at < p.N && p.list[at].x == static_cast<unsigned>(r0) + tid;
    }
    __syncthreads();
    float zero[E];
#pragma unroll
    for (int j = 0; j < E; ++j) zero[j] = 0.f;
    for (int r = 0; r < rows; ++r) {
      if (present[r]) continue;
      for (int c = tid * E; c < p.d; c += GSUM_THREADS * E)
        write_gradient<O, E, false>(dW + (r0 + r) * p.d + c, zero, 0.f);
    }
    return;
  }
  const int tile = static_cast<int>(blockIdx.x / p.slices), slice = static_cast<int>(blockIdx.x % p.slices);
  const int e0 = tile * p.tile, count = min(p.tile, p.N - e0);
  // entry[1 + i]: the tile's; entry[0] and entry[count + 1]: its neighbours (no token: V)
  const uint2 no_entry = make_uint2(p.V, 0);
  for (int i = tid; i < count + 2; i += GSUM_THREADS) {
    const int at = e0 + i - 1;
    entry[i] = at >= 0 && at < p.N ? p.list[at] : no_entry;
  }
  __syncthreads();
  const int c = (slice * GSUM_THREADS + tid) * E;
  if (c >= p.d) return;
  const T* g = static_cast<const T*>(p.g) + c;
  using P = Pack<T, E>;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  const unsigned none = p.V;
  bool begun = entry[1].x != entry[0].x;  // whether the running token begins in this tile
  for (int i0 = 0; i0 < count; i0 += GSUM_AHEAD) {
    P x[GSUM_AHEAD];
#pragma unroll
    for (int u = 0; u < GSUM_AHEAD; ++u) {
      const int i = i0 + u;
      if (i < count && entry[1 + i].x != none)
        x[u] = *reinterpret_cast<const P*>(g + static_cast<int64_t>(entry[1 + i].y) * p.ldg);
    }
#pragma unroll
    for (int u = 0; u < GSUM_AHEAD; ++u) {
      const int i = i0 + u;
      if (i >= count) break;
      const unsigned v = entry[1 + i].x, next = entry[2 + i].x;
      if (v == none) return;  // empty slots come last
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] += to_f32(x[u].v[j]);
      if (next == v && i + 1 < count) continue;
      const bool ends = next != v;
      if (begun && ends) {
        write_gradient<O, E, ADD>(dW + int64_t(v) * p.d + c, acc, p.scale);
      } else {
        float* part = p.partial + (int64_t(tile) * 2 + (begun ? 1 : 0)) * p.ldp + c;
        write_gradient<float, E, false>(part, acc, 1.f);
      }
      begun = true;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] = 0.f;
    }
  }
}

// Tokens that cross tiles: the block of the tile where such a token begins adds what the tiles left.
template <typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS) embedding_grad_join_kernel(const EmbedGradParams p) {
  const int tile = static_cast<int>(blockIdx.x / p.slices), slice = static_cast<int>(blockIdx.x % p.slices);
  const int e0 = tile * p.tile, e1 = e0 + p.tile;
  if (e1 >= p.N) return;
  const unsigned v = p.list[e1 - 1].x;
  if (v == static_cast<unsigned>(p.V) || p.list[e1].x != v) return;     // nothing crosses the end
  if (p.list[e0].x == v && e0 > 0 && p.list[e0 - 1].x == v) return;     // it began before
  const int c = (slice * GSUM_THREADS + threadIdx.x) * E;
  if (c >= p.d) return;
  float acc[E];
  const float* part = p.partial + (int64_t(tile) * 2 + 1) * p.ldp + c;
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = part[j];
  for (int t = tile + 1; t < p.tiles && p.list[int64_t(t) * p.tile].x == v; ++t) {
    part = p.partial + int64_t(t) * 2 * p.ldp + c;
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] += part[j];
  }
  write_gradient<O, E, ADD>(static_cast<O*>(p.dW) + int64_t(v) * p.d + c, acc, p.scale);
}

}  // namespace fckl
