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

#include "bulk.cuh"
#include "score.cuh"

namespace fckl {

// E values that are loaded or stored together (a power of two, at most 16 bytes of T).
template <typename T, int E>
struct alignas(E * sizeof(T)) Pack {
  T v[E];
};

// ---------------------------------------------------------------- lookup
constexpr int EMBED_THREADS = 256;
constexpr int EMBED_BLOCKS = 8;  // of an SM: 32 registers a thread

// TPR threads to a row, E values at a time and U of those under way. Bound by memory at random rows of W:
// many threads with few registers keep more under way than fewer with more (65536 x 2880 bf16 in blocks
// of 256 threads: 96 us at 4 blocks an SM, 87 at 6, 81 at 8; floor 75), and streaming stores leave L2 to W's
// frequent rows (103 -> 93 us at 4 blocks). Rows through shared memory by bulk copies took 95.
template <typename T, int E, int TPR, int U>
__global__ void __launch_bounds__(EMBED_THREADS, EMBED_BLOCKS)
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
      if constexpr (sizeof(P) == 16)
        __stcs(reinterpret_cast<uint4*>(dst + c), *reinterpret_cast<const uint4*>(&x[u]));
      else
        *reinterpret_cast<P*>(dst + c) = x[u];
    }
  }
}

// ---------------------------------------------------------------- positions in the order of their tokens
constexpr int SORT_THREADS = 512;
constexpr int SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ITEMS = 16;  // per thread and tile
constexpr int SORT_TILE = SORT_THREADS * SORT_ITEMS;
constexpr int SORT_BITS = 9;    // of a digit at most
constexpr int SORT_BINS = 1 << SORT_BITS;
constexpr int SORT_CLUSTER_MAX = 16;

static_assert(SORT_THREADS >= SORT_BINS, "a thread for every digit");

struct SortParams {
  const int32_t* tokens;
  int N, V;
  int passes, bits;  // digits and bits of each
  int cluster;       // blocks that sort: the first cluster of the grid; the others write zeros
  int per_log2;      // positions of one of them: a power of two
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
// The sort is bound by latency (two passes over 32768 positions move 1 MB): 17 us there, 20 with 8 blocks
// instead of 16, 2 more with match.any instead of ballots, 4 more with the items between the passes in
// global memory. Where all of dW is written, the rest of the GPU clears it meanwhile (525 MB beside 16384
// positions: 90 us; rows that do not occur, looked up and cleared after the sort, took 108).
__global__ void __launch_bounds__(SORT_THREADS) sort_tokens_kernel(const SortParams p) {
  namespace cg = cooperative_groups;
  let_next_begin();
  if (blockIdx.x >= p.cluster) return clear_beside(p);
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ unsigned hist[SORT_BINS];                    // this block's numbers
  __shared__ unsigned place[SORT_BINS];                   // where its next item of a digit goes
  __shared__ unsigned sums[SORT_WARPS];
  __shared__ unsigned short wcount[SORT_WARPS][SORT_BINS];  // a tile's numbers per warp, then their ranks
  extern __shared__ uint2 kept[];  // the items between two passes, if they fit
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int rank = cluster.block_rank(), blocks = p.cluster;
  const int64_t begin64 = int64_t(rank) << p.per_log2;
  const int begin = static_cast<int>(min(begin64, int64_t(p.N)));
  const int end = static_cast<int>(min(begin64 + (int64_t(1) << p.per_log2), int64_t(p.N)));
  const int per = 1 << p.per_log2;
  const bool one_tile = per <= SORT_TILE;
  const int items = one_tile ? (per + SORT_THREADS - 1) / SORT_THREADS : SORT_ITEMS;  // rounds of a tile
  bool bad = false;
  if (rank == 0 && tid == 0) *p.status = 0;
  for (int pass = 0; pass < p.passes; ++pass) {
    const int shift = pass * p.bits, bins = 1 << p.bits;
    const unsigned dmask = bins - 1;
    const uint2* from = pass & 1 ? p.a : p.b;
    uint2* to = pass & 1 ? p.b : p.a;
    const bool last = pass + 1 == p.passes;
    auto item = [&](int i) -> uint2 {
      if (pass) return one_tile ? kept[i - begin] : from[i];
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
        unsigned same = __ballot_sync(0xffffffffu, i < end);  // lanes with the same digit
#pragma unroll
        for (int b = 0; b < SORT_BITS; ++b) {
          const bool set = (digit >> b) & 1u;
          const unsigned lanes = __ballot_sync(0xffffffffu, set);
          same &= set ? lanes : ~lanes;
        }
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
          const unsigned at = place[digit] + wcount[warp][digit] + order[k];
          if (last || !one_tile) to[at] = x[k];
          else cluster.map_shared_rank(kept, at >> p.per_log2)[at & (per - 1)] = x[k];
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
    if (!one_tile) __threadfence();
    cluster.sync();  // the pass is written, and every block has read the others' numbers
  }
  if (bad) atomicOr(p.status, ST_BAD_INDEX);
}

// ---------------------------------------------------------------- sums by token
constexpr int GSUM_THREADS = 128;
constexpr int GSUM_TILE_MAX = 64;  // entries of a tile at most
constexpr int GSUM_AHEAD = 2;      // rows loaded ahead
constexpr int GJOIN_GROUPS = 4;    // of threads that share a long run's tiles

struct EmbedGradParams {
  const uint2* list;  // (token, position) in order
  int N, V, d;
  const void* g;
  int64_t ldg;
  void* dW;
  float scale;
  int tile, tiles;  // entries of a tile, tiles
  int slices;       // column slices
  int slice_vecs;   // 16-byte vectors of g in one (ring kernel)
  unsigned* status;
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

// One block per (tile of the list, column slice), rows through registers: for rows that do not lie on
// 16-byte boundaries.
template <typename T, typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS) embedding_grad_kernel(const EmbedGradParams p) {
  __shared__ uint2 entry[GSUM_TILE_MAX + 2];
  const int tid = threadIdx.x;
  O* dW = static_cast<O*>(p.dW);
  const int tile = static_cast<int>(blockIdx.x / p.slices), slice = static_cast<int>(blockIdx.x % p.slices);
  const int e0 = tile * p.tile, count = min(p.tile, p.N - e0);
  // entry[1 + i]: the tile's; entry[0] and entry[count + 1]: its neighbours (no token: V)
  const unsigned none = p.V;
  let_next_begin();
  wait_for_previous();
  for (int i = tid; i < count + 2; i += GSUM_THREADS) {
    const int at = e0 + i - 1;
    entry[i] = at >= 0 && at < p.N ? p.list[at] : make_uint2(none, 0);
  }
  __syncthreads();
  const int c = (slice * GSUM_THREADS + tid) * E;
  if (c >= p.d) return;
  const T* g = static_cast<const T*>(p.g) + c;
  using P = Pack<T, E>;
  float acc[E];
#pragma unroll
  for (int j = 0; j < E; ++j) acc[j] = 0.f;
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

// The same sums where rows of g and dW lie on 16-byte boundaries. A block takes (a tile of the list, a
// column chunk of up to 96 vectors), each of its warps a quarter of the tile, one entry to a lane. The
// entries' rows, and the rows of dW that sums are added to, come by bulk copies into rings of the warp's own
// in shared memory: what is under way does not depend on registers, and no barrier stands in the stream.
// Tokens that cross from warp to warp are then joined in shared memory.
// Bound by memory: 32768 x 2880 bf16 added to fp32 rows, 482 MB in 75 us (6.4 TB/s). Rows through registers
// took 98 us with the rows of dW loaded ahead and 160 without; 6 or 8 rows of g or 3 of dW under way
// 3 to 14% more (fewer blocks fit an SM), 3 rows of g 4%.
constexpr int GRING_WARPS = 4;
constexpr int GRING_STAGES = 4;  // rows of g
constexpr int GRING_OLD = 2;     // rows of dW
constexpr int GRING_VECS = 96;      // 16-byte vectors of g in a chunk at most
constexpr int GRING_TILE_MAX = 32 * GRING_WARPS;

// Shared memory of a warp: its rings, which later hold its two partial sums.
template <typename T, typename O, bool ADD>
__host__ __device__ constexpr int gring_warp_bytes() {
  const int rings = GRING_VECS * 16 * (GRING_STAGES + (ADD ? GRING_OLD * int(sizeof(O)) / int(sizeof(T)) : 0));
  const int sums = 2 * GRING_VECS * 16 / int(sizeof(T)) * 4;
  return rings > sums ? rings : sums;
}

template <typename T, typename O, bool ADD>
__global__ void __launch_bounds__(32 * GRING_WARPS) embedding_grad_ring_kernel(const EmbedGradParams p) {
  constexpr int VE = 16 / sizeof(T), U = GRING_VECS / 32, S = GRING_STAGES, SO = GRING_OLD;
  constexpr int STAGE = GRING_VECS * 16, OLD = STAGE * int(sizeof(O)) / int(sizeof(T));
  constexpr int WARP_BYTES = gring_warp_bytes<T, O, ADD>();
  constexpr unsigned ALL = 0xffffffffu;
  extern __shared__ __align__(128) uint8_t gring[];
  __shared__ uint64_t bars[GRING_WARPS][S + SO];
  // a warp's first and last token, and whether sums came in (which may end in it) and went out
  __shared__ unsigned token_in[GRING_WARPS], token_out[GRING_WARPS];
  __shared__ bool has_in[GRING_WARPS], in_ends[GRING_WARPS], has_out[GRING_WARPS];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int tile = static_cast<int>(blockIdx.x / p.slices), slice = static_cast<int>(blockIdx.x % p.slices);
  const int own = p.tile / GRING_WARPS;  // entries of a warp
  const int64_t e0 = int64_t(tile) * p.tile + warp * own;
  const int count = static_cast<int>(max(int64_t(0), min(int64_t(own), p.N - e0)));
  const unsigned none = p.V;
  uint64_t *full = bars[warp], *old_full = bars[warp] + S;
  if (lane == 0) {
    for (int k = 0; k < S + SO; ++k) mbar_init(&full[k], 1);
    fence_mbar_init();
  }
  let_next_begin();
  wait_for_previous();
  // an entry to a lane, and its neighbours' tokens
  const uint2 mine = lane < count ? p.list[e0 + lane] : make_uint2(none, 0);
  unsigned before = __shfl_up_sync(ALL, mine.x, 1), after = __shfl_down_sync(ALL, mine.x, 1);
  if (lane == 0) before = e0 > 0 && e0 <= p.N ? p.list[e0 - 1].x : none;
  if (lane == count - 1) after = e0 + count < p.N ? p.list[e0 + count].x : none;
  const bool live = lane < count && mine.x != none;
  const int entries = __popc(__ballot_sync(ALL, live));  // empty slots come last
  const unsigned ends = __ballot_sync(ALL, live && after != mine.x);
  const unsigned breaks = entries ? ends | 1u << (entries - 1) : 0u;  // where a sum is written, whole or in part
  const bool comes_in = __shfl_sync(ALL, live && before == mine.x, 0);
  unsigned adds = ends;  // sums that belong to dW: they begin and end in this warp
  if (comes_in && ends) adds &= ends - 1;
  const int vecs = p.d / VE, v0 = slice * p.slice_vecs, nv = min(p.slice_vecs, vecs - v0);
  const T* g = static_cast<const T*>(p.g) + int64_t(v0) * VE;
  O* dW = static_cast<O*>(p.dW) + int64_t(v0) * VE;
  uint8_t* ring = gring + warp * WARP_BYTES;
  uint8_t* old_ring = ring + S * STAGE;
  const uint32_t bytes = static_cast<uint32_t>(nv) * 16, old_bytes = bytes / sizeof(T) * sizeof(O);
  auto load_row = [&](int i) {  // all lanes
    const int pos = __shfl_sync(ALL, static_cast<int>(mine.y), i);
    if (lane == 0) {
      mbar_arrive_expect_tx(&full[i % S], bytes);
      bulk_load(ring + (i % S) * STAGE, g + int64_t(pos) * p.ldg, bytes, &full[i % S]);
    }
  };
  unsigned to_load = ADD ? adds : 0u;  // rows of dW not yet asked for
  int asked = 0, used = 0;
  auto load_old = [&]() {
    if (!to_load) return;
    const unsigned v = __shfl_sync(ALL, mine.x, __ffs(to_load) - 1);
    to_load &= to_load - 1;
    if (lane == 0) {
      mbar_arrive_expect_tx(&old_full[asked % SO], old_bytes);
      bulk_load(old_ring + (asked % SO) * OLD, dW + int64_t(v) * p.d, old_bytes, &old_full[asked % SO]);
    }
    ++asked;
  };
  __syncwarp();
  for (int i = 0; i < min(S, entries); ++i) load_row(i);
  for (int k = 0; k < SO; ++k) load_old();
  float acc[U][VE], in[U][VE];  // the running sum; the one of the token that comes in
  auto clear = [&](float (&x)[U][VE]) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < VE; ++j) x[u][j] = 0.f;
  };
  clear(acc);
  bool ok = true;
  int i = 0;
  for (; i < entries; ++i) {
    ok = drain_phase(&full[i % S], (i / S) & 1, p.status);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int q = u * 32 + lane;
      if (q < nv) {
        float f[VE];
        unpack16<T>(reinterpret_cast<const uint4*>(ring + (i % S) * STAGE)[q], f);
#pragma unroll
        for (int j = 0; j < VE; ++j) acc[u][j] += f[j];
      }
    }
    if (!__all_sync(ALL, ok)) break;  // (and the stage has been read)
    if (i + S < entries) load_row(i + S);
    if (!((breaks >> i) & 1u)) continue;
    if ((adds >> i) & 1u) {
      const unsigned v = __shfl_sync(ALL, mine.x, i);
      if (ADD) ok = drain_phase(&old_full[used % SO], (used / SO) & 1, p.status);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int q = u * 32 + lane;
        if (q >= nv) continue;
        GradPacks<O, VE> y;
        if (ADD) y.load(reinterpret_cast<const O*>(old_ring + (used % SO) * OLD) + q * VE);
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          O& o = y.v[j / y.EP].v[j % y.EP];
          o = from_f32<O>(ADD ? fmaf(p.scale, acc[u][j], to_f32(o)) : p.scale * acc[u][j]);
        }
        y.store(dW + int64_t(v) * p.d + q * VE);
      }
      if (!__all_sync(ALL, ok)) break;
      ++used;
      load_old();
    } else if (comes_in && !(breaks & ((1u << i) - 1u))) {  // the first sum written: it began before
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < VE; ++j) in[u][j] = acc[u][j];
    } else {
      continue;  // the last sum, which goes on: it stays in acc
    }
    clear(acc);
  }
  if (i < entries && lane == 0) {  // a copy did not come: leave none under way
    for (int k = i + 1; k < min(i + S, entries); ++k) drain_phase(&full[k % S], (k / S) & 1, p.status);
    if (ADD)
      for (int k = used; k < asked; ++k) drain_phase(&old_full[k % SO], (k / SO) & 1, p.status);
  }
  // What crosses the warps' edges, through shared memory: a sum that came in, and one that goes on.
  const bool one_run = comes_in && !ends && entries;          // covers the warp: it counts as coming in
  const bool goes_on = entries && !((ends >> (entries - 1)) & 1u) && !one_run;
  float* sums = reinterpret_cast<float*>(ring);
  __syncwarp();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int q = u * 32 + lane;
    if (q >= nv) continue;
    GradPacks<float, VE> y;
    if (comes_in) {
#pragma unroll
      for (int j = 0; j < VE; ++j) y.v[j / y.EP].v[j % y.EP] = in[u][j];
      y.store(sums + q * VE);
    }
    if (goes_on) {
#pragma unroll
      for (int j = 0; j < VE; ++j) y.v[j / y.EP].v[j % y.EP] = acc[u][j];
      y.store(sums + GRING_VECS * VE + q * VE);
    }
  }
  const unsigned last = __shfl_sync(ALL, mine.x, max(entries - 1, 0));
  if (lane == 0) {
    token_in[warp] = mine.x;
    token_out[warp] = last;
    has_in[warp] = comes_in;
    in_ends[warp] = ends != 0;
    has_out[warp] = goes_on;
  }
  __syncthreads();
  for (int c = threadIdx.x * 4; c < nv * VE; c += 128 * GRING_WARPS) {  // four columns a thread
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
    bool running = false, began = false;
    auto add = [&](const float* x) {
      const float4 f = *reinterpret_cast<const float4*>(x + c);
      run.x += f.x, run.y += f.y, run.z += f.z, run.w += f.w;
    };
    auto leave = [&](int which) {  // for the other blocks' part of this token
      *reinterpret_cast<float4*>(p.partial + (int64_t(tile) * 2 + which) * p.ldp + int64_t(v0) * VE + c) = run;
    };
    for (int w = 0; w < GRING_WARPS; ++w) {
      const float* x = reinterpret_cast<const float*>(gring + w * WARP_BYTES);
      if (has_in[w]) {
        add(x);
        running = true;
        if (in_ends[w]) {
          if (began) {
            O* to = dW + int64_t(token_in[w]) * p.d + c;
            const float f[4] = {run.x, run.y, run.z, run.w};
            GradPacks<O, 4> y;
            if (ADD) y.load(to);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              O& o = y.v[j / y.EP].v[j % y.EP];
              o = from_f32<O>(ADD ? fmaf(p.scale, f[j], to_f32(o)) : p.scale * f[j]);
            }
            y.store(to);
          } else {
            leave(0);
          }
          running = began = false;
          run = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      if (has_out[w]) {
        add(x + GRING_VECS * VE);
        running = began = true;
      }
    }
    if (running) leave(began ? 1 : 0);
  }
}

// Tokens that cross tiles: the block of the tile where such a token begins adds what the tiles left. Of
// a few tiles every group of threads takes a column slice; of many the groups share the tiles of each
// slice, a stretch of them each, and add their sums in order. 7 us at 32768 x 2880, all of it latency. A token that
// holds most positions is still joined by one block: 65536 x 2880 added to fp32 rows take 283 us without one,
// 261 with a token that holds half of them (floor 160) and 178 where one holds all (floor 56).
template <typename O, int E, bool ADD>
__global__ void __launch_bounds__(GSUM_THREADS * GJOIN_GROUPS) embedding_grad_join_kernel(const EmbedGradParams p) {
  constexpr int NT = GSUM_THREADS * GJOIN_GROUPS;
  __shared__ float part[GJOIN_GROUPS - 1][GSUM_THREADS * E];
  const int tile = static_cast<int>(blockIdx.x), tid = threadIdx.x;
  const int64_t e0 = int64_t(tile) * p.tile, e1 = e0 + p.tile;
  wait_for_previous();
  if (e1 >= p.N) return;
  const unsigned v = p.list[e1 - 1].x, next = p.list[e1].x, first = p.list[e0].x, earlier = p.list[max(e0 - 1, int64_t(0))].x;
  if (v == static_cast<unsigned>(p.V) || next != v) return;  // nothing crosses the end
  if (first == v && e0 > 0 && earlier == v) return;          // it began before
  int more = 0;  // tiles that begin with the token follow each other
  for (int t0 = tile + 1; t0 < p.tiles; t0 += NT) {
    const int t = t0 + tid;
    const int n = __syncthreads_count(t < p.tiles && p.list[int64_t(t) * p.tile].x == v);
    more += n;
    if (n < NT) break;
  }
  const int lane = tid % GSUM_THREADS, group = tid / GSUM_THREADS, all = more + 1;
  // acc += partial sums [k, k1): what the token's first tile began, then the other tiles' first ones
  auto add = [&](float (&acc)[E], int k, int k1, int c) {
    for (; k < k1; k += 4) {
      GradPacks<float, E> x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (k + u < k1) x[u].load(p.partial + (int64_t(tile + k + u) * 2 + (k + u == 0 ? 1 : 0)) * p.ldp + c);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (k + u >= k1) break;
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] += x[u].v[j / x[u].EP].v[j % x[u].EP];
      }
    }
  };
  auto finish = [&](const float (&acc)[E], int c) {
    O* to = static_cast<O*>(p.dW) + int64_t(v) * p.d + c;
    GradPacks<O, E> y;
    if (ADD) y.load(to);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      O& o = y.v[j / y.EP].v[j % y.EP];
      o = from_f32<O>(ADD ? fmaf(p.scale, acc[j], to_f32(o)) : p.scale * acc[j]);
    }
    y.store(to);
  };
  if (all <= 16) {
    for (int slice = group; slice < p.slices; slice += GJOIN_GROUPS) {
      const int c = (slice * GSUM_THREADS + lane) * E;
      if (c >= p.d) return;
      float acc[E] = {};
      add(acc, 0, all, c);
      finish(acc, c);
    }
    return;
  }
  const int per = (all + GJOIN_GROUPS - 1) / GJOIN_GROUPS;
  for (int slice = 0; slice < p.slices; ++slice) {
    const int c = (slice * GSUM_THREADS + lane) * E;
    float acc[E] = {};
    if (c < p.d) add(acc, group * per, min(all, (group + 1) * per), c);
    if (group > 0) {
#pragma unroll
      for (int j = 0; j < E; ++j) part[group - 1][j * GSUM_THREADS + lane] = acc[j];
    }
    __syncthreads();
    if (group == 0 && c < p.d) {
      for (int r = 0; r < GJOIN_GROUPS - 1; ++r) {
#pragma unroll
        for (int j = 0; j < E; ++j) acc[j] += part[r][j * GSUM_THREADS + lane];
      }
      finish(acc, c);
    }
    __syncthreads();
  }
}

}  // namespace fckl
