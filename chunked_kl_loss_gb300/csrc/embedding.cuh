// The tied embedding: rows of W [V, d] for given tokens times a scale, and the gradient of W.
//
//   y_n   = s W[t_n]                               (t_n = -1: a row of zeros)
//   dW[v] = (dW[v] +) s sum over n with t_n = v of g_n
//
// The gradient's positions are first put in the order of their tokens, equal tokens in the order of
// their positions (a radix sort by one cluster). Blocks then walk tiles of the ordered list, each over
// its own columns: the rows of a token that begins and ends within a tile are summed in registers and
// written once; a token that crosses a tile's edge leaves one partial sum per tile, and those are added
// in a fixed order by a second kernel. So every row of dW has one writer, and the sums, all in
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
  int passes, bits;  // digits and bits of each
  int cluster;       // blocks that sort: the first cluster of the grid; the others write zeros
  int per_cta;       // positions of one of them
  uint2* a;          // (token, position), written by the even passes
  uint2* b;          // and by the odd ones
  unsigned* status;
  uint8_t* zero;     // what the other blocks clear, from a 16-byte boundary, and its size
  int64_t zero_bytes;
};

// Clears p.zero with the blocks behind the sorting ones.
__device__ __forceinline__ void clear_beside(const SortParams& p) {
  const int64_t step = int64_t(gridDim.x - p.cluster) * SORT_THREADS;
  const int64_t n = p.zero_bytes / 16;
  uint4* at = reinterpret_cast<uint4*>(p.zero);
  int64_t i = int64_t(blockIdx.x - p.cluster) * SORT_THREADS + threadIdx.x;
  for (; i + 3 * step < n; i += 4 * step) {
#pragma unroll
    for (int u = 0; u < 4; ++u) at[i + u * step] = make_uint4(0, 0, 0, 0);
  }
  for (; i < n; i += step) at[i] = make_uint4(0, 0, 0, 0);
  const int64_t rest = n * 16 + (int64_t(blockIdx.x - p.cluster) * SORT_THREADS + threadIdx.x) * 2;
  if (rest < p.zero_bytes) *reinterpret_cast<uint16_t*>(p.zero + rest) = 0;
}

// Least significant digit first; one cluster. Empty slots and bad ids take the key V, so that they come
// last. A pass counts each digit's items per warp, which also gives an item's rank among its equals (in the
// order of the warps, of a warp's rounds and of its lanes); the blocks exchange their numbers through
// distributed shared memory, and every item goes to its place. A block with more items than one tile
// counts them first and then takes tile after tile.
// The sort is bound by latency (two passes over 32768 positions move 1 MB): where all of dW is written,
// the rest of the GPU clears it meanwhile.
__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortParams p) {
  namespace cg = cooperative_groups;
  if (blockIdx.x >= p.cluster) return clear_beside(p);
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ unsigned hist[SORT_BINS];                    // this block's numbers
  __shared__ unsigned place[SORT_BINS];                   // where its next item of a digit goes
  __shared__ unsigned sums[SORT_WARPS];
  __shared__ unsigned short wcount[SORT_WARPS][SORT_BINS];  // a tile's numbers per warp, then their ranks
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = cluster.block_rank(), blocks = p.cluster;
  const int64_t begin64 = int64_t(rank) * p.per_cta;
  const int begin = static_cast<int>(min(begin64, int64_t(p.N)));
  const int end = static_cast<int>(min(begin64 + p.per_cta, int64_t(p.N)));
  const bool one_tile = p.per_cta <= SORT_TILE;
  const int items = one_tile ? (p.per_cta + SORT_THREADS - 1) / SORT_THREADS : SORT_ITEMS;  // rounds of a tile
  bool bad = false;
  if (rank == 0 && tid == 0) *p.status = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits, bins = 1 << p.bits;
    const unsigned dmask = bins - 1;
    const uint2* from = pass & 1 ? p.a : p.b;
    uint2* to = pass & 1 ? p.b : p.a;
    auto item = [&](int i) -> uint2 {
      if (pass) return from[i];
      const int t = p.tokens[i];
      bad |= t < -1 || t >= p.V;
      return make_uint2(t >= 0 && t < p.V ? t : p.V, i);
    };
    uint2 x[SORT_ITEMS];
    unsigned short order[SORT_ITEMS];
    unsigned in_tile = 0;  // of digit tid
    // Items of the tile at t0, their ranks within their warp, and the warps' numbers before each warp.
    auto rank_tile = [&](int t0) {
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        const int i = t0 + (warp * items + k) * 32 + lane;
        if (k < items && i < end) x[k] = item(i);
      }
      for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<unsigned*>(wcount[warp])[i] = 0;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        if (k >= items) break;
        const int i = t0 + (warp * items + k) * 32 + lane;
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
      in_tile = 0;
      if (tid < bins) {
#pragma unroll 8
        for (int w = 0; w < SORT_WARPS; ++w) {
          const unsigned c = wcount[w][tid];
          wcount[w][tid] = static_cast<unsigned short>(in_tile);
          in_tile += c;
        }
      }
    };
    auto scatter_tile = [&](int t0) {
#pragma unroll
      for (int k = 0; k < SORT_ITEMS; ++k) {
        const int i = t0 + (warp * items + k) * 32 + lane;
        if (k < items && i < end) {
          const unsigned digit = (x[k].x >> shift) & dmask;
          to[place[digit] + wcount[warp][digit] + order[k]] = x[k];
        }
      }
    };
    if (one_tile) {
      rank_tile(begin);
      if (tid < bins) hist[tid] = in_tile;
    } else {
      if (tid < bins) hist[tid] = 0;
      __syncthreads();
      for (int i = begin + tid; i < end; i += SORT_THREADS) atomicAdd(&hist[(item(i).x >> shift) & dmask], 1u);
    }
    cluster.sync();
    // place = items of smaller digits anywhere + items of this digit in earlier blocks
    unsigned total = 0, before = 0;
    if (tid < bins) {
#pragma unroll 8
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
    if (tid < bins) {
      unsigned lower = 0;
#pragma unroll
      for (int w = 0; w < SORT_BINS / 32; ++w) lower += w < warp ? sums[w] : 0;
      place[tid] = lower + run - total + before;
    }
    __syncthreads();
    if (one_tile) {
      scatter_tile(begin);
    } else {
      for (int t0 = begin; t0 < end; t0 += SORT_TILE) {
        rank_tile(t0);
        __syncthreads();
        scatter_tile(t0);
        __syncthreads();
        if (tid < bins) place[tid] += in_tile;
      }
    }
    __threadfence();
    cluster.sync();  // the pass is written, and every block has read the others' numbers
  }
  if (bad) atomicOr(p.status, ST_BAD_INDEX);
}

// ---------------------------------------------------------------- sums by token
constexpr int GSUM_THREADS = 128;
constexpr int GSUM_TILE_MAX = 64;  // entries of a tile at most
#ifndef GS_A
#define GS_A 4
#endif
constexpr int GSUM_AHEAD = GS_A;  // rows loaded ahead
constexpr int GJOIN_GROUPS = 4;    // of threads that share a crossing token's tiles

struct EmbedGradParams {
  const uint2* list;  // (token, position) in order
  int N, V, d;
  const void* g;
  int64_t ldg;
  void* dW;
  float scale;
  int tile, tiles;  // entries of a tile, tiles
  int slices;       // column slices
  float* partial;   // [tiles][2][ldp]: what a tile adds to a token begun before it; what it begins
  int64_t ldp;
};

// A row's values of dW, in packs of at most 16 bytes.
template <typename O, int E>
struct GradPacks {
  static constexpr int EP = E * sizeof(O) > 16 ? 16 / sizeof(O) : E;
  Pack<O, EP> v[E / EP];
  __device__ __forceinline__ void load(const O* at) {
#pragma unroll
    for (int q = 0; q < E / EP; ++q) v[q] = reinterpret_cast<const Pack<O, EP>*>(at)[q];
  }
  __device__ __forceinline__ void store(O* at) const {
#pragma unroll
    for (int q = 0; q < E / EP; ++q) reinterpret_cast<Pack<O, EP>*>(at)[q] = v[q];
  }
};

// One block per (tile of the list, column slice).
template <typename T, typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS) embedding_grad_kernel(const EmbedGradParams p) {
  __shared__ uint2 entry[GSUM_TILE_MAX + 2];
  const int tid = threadIdx.x;
  O* dW = static_cast<O*>(p.dW);
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
    // The rows of the step, and where a token ends in it the row of dW that it is added to, all under way
    // at once.
    P x[GSUM_AHEAD];
    GradPacks<O, E> old[GSUM_AHEAD];
#pragma unroll
    for (int u = 0; u < GSUM_AHEAD; ++u) {
      const int i = i0 + u;
      if (i < count && entry[1 + i].x != none) {
        x[u] = *reinterpret_cast<const P*>(g + static_cast<int64_t>(entry[1 + i].y) * p.ldg);
        if (ADD && entry[2 + i].x != entry[1 + i].x) old[u].load(dW + int64_t(entry[1 + i].x) * p.d + c);
      }
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
      if (begun && next != v) {
        GradPacks<O, E> y;
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const float to = ADD ? to_f32(old[u].v[j / y.EP].v[j % y.EP]) : 0.f;
          y.v[j / y.EP].v[j % y.EP] = from_f32<O>(ADD ? fmaf(p.scale, acc[j], to) : p.scale * acc[j]);
        }
        y.store(dW + int64_t(v) * p.d + c);
      } else {
        GradPacks<float, E> y;
#pragma unroll
        for (int j = 0; j < E; ++j) y.v[j / y.EP].v[j % y.EP] = acc[j];
        y.store(p.partial + (int64_t(tile) * 2 + (begun ? 1 : 0)) * p.ldp + c);
      }
      begun = true;
#pragma unroll
      for (int j = 0; j < E; ++j) acc[j] = 0.f;
    }
  }
}

// Tokens that cross tiles: the block of the tile where such a token begins adds what the tiles left, in
// four runs of tiles and then those in order.
template <typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS * GJOIN_GROUPS) embedding_grad_join_kernel(const EmbedGradParams p) {
  __shared__ float part[GJOIN_GROUPS - 1][GSUM_THREADS * E];
  const int tile = static_cast<int>(blockIdx.x / p.slices), slice = static_cast<int>(blockIdx.x % p.slices);
  const int e0 = tile * p.tile, e1 = e0 + p.tile;
  if (e1 >= p.N) return;
  const unsigned v = p.list[e1 - 1].x;
  if (v == static_cast<unsigned>(p.V) || p.list[e1].x != v) return;  // nothing crosses the end
  if (p.list[e0].x == v && e0 > 0 && p.list[e0 - 1].x == v) return;  // it began before
  // tiles that begin with the token: they follow each other
  int more = 0;
  for (int t0 = tile + 1; t0 < p.tiles; t0 += GSUM_THREADS * GJOIN_GROUPS) {
    const int t = t0 + threadIdx.x;
    const int n = __syncthreads_count(t < p.tiles && p.list[int64_t(t) * p.tile].x == v);
    more += n;
    if (n < GSUM_THREADS * GJOIN_GROUPS) break;
  }
  const int lane = threadIdx.x % GSUM_THREADS, group = threadIdx.x / GSUM_THREADS;
  const int c = (slice * GSUM_THREADS + lane) * E;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
  if (c < p.d) {
    auto take = [&](int i) {  // partial sum i of the token: what it began, then the tiles' first ones
      GradPacks<float, E> x;
      x.load(p.partial + (int64_t(tile + i) * 2 + (i == 0 ? 1 : 0)) * p.ldp + c);
      return x;
    };
    const int all = more + 1, per = (all + GJOIN_GROUPS - 1) / GJOIN_GROUPS;
    const int i1 = min(all, (group + 1) * per);
    for (int i = group * per; i < i1; i += 4) {
      GradPacks<float, E> x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u < i1) x[u] = take(i + u);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (i + u >= i1) break;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] += x[u].v[j / x[u].EP].v[j % x[u].EP];
      }
    }
  }
  if (group > 0) {
#pragma unroll
    for (int j = 0; j < E; ++j) part[group - 1][j * GSUM_THREADS + lane] = acc[j];
  }
  __syncthreads();
  if (group > 0 || c >= p.d) return;
  for (int r = 0; r < GJOIN_GROUPS - 1; ++r) {
#pragma unroll
    for (int j = 0; j < E; ++j) acc[j] += part[r][j * GSUM_THREADS + lane];
  }
  O* at = static_cast<O*>(p.dW) + int64_t(v) * p.d + c;
  GradPacks<O, E> y;
  if (ADD) y.load(at);
#pragma unroll
  for (int j = 0; j < E; ++j) {
    O& o = y.v[j / y.EP].v[j % y.EP];
    o = from_f32<O>(ADD ? fmaf(p.scale, acc[j], to_f32(o)) : p.scale * acc[j]);
  }
  y.store(at);
}

}  // namespace fckl
