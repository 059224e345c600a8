// Host side of the tied embedding (embedding.cuh): argument checks, workspace, launch shapes and the C
// entry points declared in include/fckl.h. Part of the translation unit of fckl.cu.
#pragma once

#include "embedding.cuh"
#include "score_host.cuh"

namespace fckl {
namespace {

int embed_shape(int64_t N, int d, int V, int dt) {
  if (N < 0 || d < 1 || V < 1 || !known_dtype(dt)) return FCKL_ERR_ARG;
  if (V > (1 << 30) || N > (int64_t(1) << 30) || d > (1 << 20)) return FCKL_ERR_UNSUPPORTED;
  return FCKL_OK;
}

// The most values, at most 16 bytes of them, that every row's start keeps together: d, the pitch and the
// address are multiples of them.
int pack_of(const void* p, int64_t ld, int64_t rows, int d, size_t bytes) {
  int e = static_cast<int>(16 / bytes);
  while (e > 1 && (d % e || (rows > 1 && ld % e) || !aligned(p, e * bytes))) e /= 2;
  return e;
}

template <typename T, int E>
int launch_embedding(const void* W, int64_t ldw, const int32_t* tokens, int64_t N, int d, int V, float scale, void* out,
                     int64_t ld_out, unsigned* status, cudaStream_t s) {
  auto go = [&](auto tpr, auto u) {
    constexpr int TPR = decltype(tpr)::value, U = decltype(u)::value;
    const unsigned grid = static_cast<unsigned>(cdiv(N, EMBED_THREADS / TPR));
    return launch(KIND_EMBEDDING, s, "embedding", [&] {
      embedding_kernel<T, E, TPR, U><<<grid, EMBED_THREADS, 0, s>>>(static_cast<const T*>(W), ldw, tokens, N, d, V, scale,
                                                                    static_cast<T*>(out), ld_out, status);
    });
  };
  // As many loads of a thread at once as spread a row evenly over its steps.
  auto with = [&](auto tpr) {
    constexpr int TPR = decltype(tpr)::value;
    const int64_t each = cdiv(cdiv(d, E), TPR), u = cdiv(each, cdiv(each, 4));
    if constexpr (E * sizeof(T) == 16) {
      if (u == 1) return go(tpr, std::integral_constant<int, 1>{});
      if (u == 2) return go(tpr, std::integral_constant<int, 2>{});
      if (u == 3) return go(tpr, std::integral_constant<int, 3>{});
    }
    return go(tpr, std::integral_constant<int, 4>{});
  };
  const int64_t packs = cdiv(d, E);
  if (packs <= 32) return with(std::integral_constant<int, 8>{});
  if (packs <= 128) return with(std::integral_constant<int, 32>{});
  return with(std::integral_constant<int, 128>{});
}

template <typename T>
int launch_embedding_pack(int e, const void* W, int64_t ldw, const int32_t* tokens, int64_t N, int d, int V, float scale,
                          void* out, int64_t ld_out, unsigned* status, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (e == 8) return launch_embedding<T, 8>(W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
  if (e >= 4) return launch_embedding<T, 4>(W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
  if (e == 2) return launch_embedding<T, 2>(W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
  return launch_embedding<T, 1>(W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
}

// ------------------------------------------------------------------ gradient
constexpr int GSUM_TILE_MIN = 8;
constexpr int SORT_CTA_ITEMS = 1024;  // positions of a sorting block, as long as the cluster can grow
// SMs that tiles are cut for: a constant, so that the workspace's size and the order of the sums do not depend
// on the device that is current.
constexpr int GSUM_SMS = 152;

struct EmbedGradPlan {
  int passes, bits;
  int64_t ldp;
  int tiles;  // that the partial sums have room for
  size_t off_a, off_b, off_partial, total;
};

// Entries of a tile: as many as leave blocks for the GPU several times over, between GSUM_TILE_MIN and
// `most`. More slices never give smaller tiles.
int grad_tile(int64_t N, int64_t slices, int most) {
  int tile = GSUM_TILE_MIN;
  while (tile < most && cdiv(N, 2 * tile) * slices >= 4 * GSUM_SMS) tile *= 2;
  return tile;
}

EmbedGradPlan embed_grad_plan(int64_t N, int d, int V) {
  EmbedGradPlan q{};
  int bits = 1;
  while ((int64_t(1) << bits) <= V) ++bits;  // keys 0..V
  q.passes = static_cast<int>(cdiv(bits, SORT_BITS));
  q.bits = static_cast<int>(cdiv(bits, q.passes));
  q.ldp = rup(d, 8);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t r = o;
    o = static_cast<size_t>(rup(static_cast<int64_t>(o + bytes), 256));
    return r;
  };
  take(STATUS_WS_BYTES);
  q.off_a = take(size_t(N) * 8);
  q.off_b = take(size_t(N) * 8);
  // two partial sums for every tile, at the smallest tiles that any alignment of the rows leads to
  const int least = grad_tile(N, cdiv(d, 8 * GRING_VECS), GSUM_TILE_MAX);
  q.tiles = static_cast<int>(cdiv(N, least));
  q.off_partial = take(size_t(q.tiles) * 2 * q.ldp * 4);
  q.total = o;
  return q;
}

// Sorts p.tokens with a cluster of up to SORT_CLUSTER_MAX blocks (as many as the device takes).
int launch_sort_tokens(const DevInfo* di, SortParams p, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(SORT_THREADS);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  static int most[64] = {};
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!most[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           SORT_TILE * int(sizeof(uint2)));
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(sort_tokens_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      int clusters = 0;
      cfg.gridDim = dim3(SORT_CLUSTER_MAX);
      cfg.dynamicSmemBytes = SORT_TILE * sizeof(uint2);
      attr[0].val.clusterDim.x = SORT_CLUSTER_MAX;
      if (e == cudaSuccess) e = cudaOccupancyMaxActiveClusters(&clusters, sort_tokens_kernel, &cfg);
      if (e != cudaSuccess) {
        set_error("set-up of sort_tokens", e);
        return FCKL_ERR_CUDA;
      }
      most[di->id] = clusters > 0 ? SORT_CLUSTER_MAX : 8;
    }
  }
  p.cluster = 1;
  while (p.cluster < most[di->id] && int64_t(p.cluster) * SORT_CTA_ITEMS < p.N) p.cluster *= 2;
  p.per_log2 = 5;
  while ((int64_t(p.cluster) << p.per_log2) < p.N) ++p.per_log2;
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.cluster);
  cfg.dynamicSmemBytes = (1 << p.per_log2) <= SORT_TILE ? sizeof(uint2) << p.per_log2 : 0;
  // two blocks for every SM (one runs at a time, with the sort's 128 registers a thread), and no more than
  // have 64 KB to clear
  const int64_t clear = std::min<int64_t>(cdiv(p.zero_bytes, 65536), 2 * int64_t(di->sms) - p.cluster);
  cfg.gridDim = dim3(static_cast<unsigned>(p.cluster + rup(clear, p.cluster)));
  return launch(KIND_SORT_TOKENS, s, "sort_tokens", [&] { cudaLaunchKernelEx(&cfg, sort_tokens_kernel, p); });
}

template <typename T, typename O, int E, bool ADD>
int launch_embedding_grad(const DevInfo* di, EmbedGradParams p, cudaStream_t s) {
  const int room = p.tiles;  // of the partial sums
  const int64_t join_slices = cdiv(p.d, GSUM_THREADS * E);
  int64_t blocks;
  int st;
  if constexpr (E * sizeof(T) == 16) {
    const int64_t vecs = p.d / E;
    p.slices = static_cast<int>(cdiv(vecs, GRING_VECS));
    p.slice_vecs = static_cast<int>(cdiv(vecs, p.slices));
    p.tile = grad_tile(p.N, p.slices, GRING_TILE_MAX);
    p.tiles = static_cast<int>(cdiv(p.N, p.tile));
    blocks = int64_t(p.tiles) * p.slices;
    if (blocks > INT_MAX || p.tiles > room) return FCKL_ERR_UNSUPPORTED;
    constexpr int SMEM = GRING_WARPS * gring_warp_bytes<T, O, ADD>();
    auto k = embedding_grad_ring_kernel<T, O, ADD>;
    {
      static bool done[64] = {};
      std::lock_guard<std::mutex> lk(g_setup_mu);
      if (!done[di->id]) {
        cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) {
          set_error("cudaFuncSetAttribute(embedding_grad)", e);
          return FCKL_ERR_CUDA;
        }
        done[di->id] = true;
      }
    }
    st = launch_after(KIND_EMBEDDING_GRAD, s, "embedding_grad", static_cast<unsigned>(blocks), 32 * GRING_WARPS, SMEM, k, p);
  } else {
    p.slices = static_cast<int>(join_slices);
    p.tile = grad_tile(p.N, p.slices, GSUM_TILE_MAX);
    p.tiles = static_cast<int>(cdiv(p.N, p.tile));
    blocks = int64_t(p.tiles) * p.slices;
    if (blocks > INT_MAX || p.tiles > room) return FCKL_ERR_UNSUPPORTED;
    st = launch_after(KIND_EMBEDDING_GRAD, s, "embedding_grad", static_cast<unsigned>(blocks), GSUM_THREADS, 0,
                      embedding_grad_kernel<T, O, E, ADD>, p);
  }
  if (st || p.tiles < 2) return st;
  p.slices = static_cast<int>(join_slices);
  return launch_after(KIND_EMBEDDING_JOIN, s, "embedding_grad_join", static_cast<unsigned>(p.tiles - 1),
                      GSUM_THREADS * GJOIN_GROUPS, 0, embedding_grad_join_kernel<O, E, ADD>, p);
}

template <typename T, typename O, bool ADD>
int launch_embedding_grad_pack(const DevInfo* di, int e, const EmbedGradParams& p, cudaStream_t s) {
  if constexpr (sizeof(T) == 2)
    if (e == 8) return launch_embedding_grad<T, O, 8, ADD>(di, p, s);
  if (e >= 4) return launch_embedding_grad<T, O, 4, ADD>(di, p, s);
  if (e == 2) return launch_embedding_grad<T, O, 2, ADD>(di, p, s);
  return launch_embedding_grad<T, O, 1, ADD>(di, p, s);
}

template <typename T>
int launch_embedding_grad_type(const DevInfo* di, int e, int dt, int out_dt, bool add, const EmbedGradParams& p, cudaStream_t s) {
  if (out_dt == FCKL_F32)
    return add ? launch_embedding_grad_pack<T, float, true>(di, e, p, s)
               : launch_embedding_grad_pack<T, float, false>(di, e, p, s);
  if constexpr (sizeof(T) == 2)
    return add ? launch_embedding_grad_pack<T, T, true>(di, e, p, s) : launch_embedding_grad_pack<T, T, false>(di, e, p, s);
  return FCKL_ERR_ARG;
}

}  // namespace
}  // namespace fckl

extern "C" {

int fckl_embedding(const void* W, int dtype, int64_t ldw, const int32_t* tokens, int64_t N, int d, int V, float scale,
                   void* out, int64_t ld_out, void* ws, size_t ws_bytes, void* stream) {
  return guarded("fckl_embedding", [&]() -> int {
    int st = embed_shape(N, d, V, dtype);
    if (st) return st;
    if (ldw < d || ld_out < d) return FCKL_ERR_ARG;
    if (ldw > (int64_t(1) << 40) || ld_out > (int64_t(1) << 40)) return FCKL_ERR_UNSUPPORTED;
    if ((st = status_ws_checks(ws, ws_bytes))) return st;
    if (N == 0) return FCKL_OK;
    const size_t b = value_bytes(dtype);
    if (!W || !tokens || !out || !aligned(W, b) || !aligned(out, b) || !aligned(tokens, 4)) return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    const int e = std::min(pack_of(W, ldw, V, d, b), pack_of(out, ld_out, N, d, b));
    unsigned* status = static_cast<unsigned*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FCKL_BF16)
      return launch_embedding_pack<__nv_bfloat16>(e, W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
    if (dtype == FCKL_F16)
      return launch_embedding_pack<__half>(e, W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
    return launch_embedding_pack<float>(e, W, ldw, tokens, N, d, V, scale, out, ld_out, status, s);
  });
}

size_t fckl_embedding_backward_workspace_bytes(int64_t N, int d, int V) {
  if (embed_shape(N, d, V, FCKL_BF16) != FCKL_OK) return 0;
  return embed_grad_plan(N, d, V).total;
}

int fckl_embedding_backward(const void* g, int dtype, int64_t ldg, const int32_t* tokens, int64_t N, int d, int V,
                            float scale, void* dW, int dW_dtype, int accumulate, void* ws, size_t ws_bytes,
                            void* stream) {
  return guarded("fckl_embedding_backward", [&]() -> int {
    int st = embed_shape(N, d, V, dtype);
    if (st) return st;
    if (ldg < d || (dW_dtype != FCKL_F32 && dW_dtype != dtype)) return FCKL_ERR_ARG;
    if (ldg > (int64_t(1) << 40)) return FCKL_ERR_UNSUPPORTED;
    if (!ws || !aligned(ws, 256)) return FCKL_ERR_ARG;
    const EmbedGradPlan q = embed_grad_plan(N, d, V);
    if (ws_bytes < q.total) return FCKL_ERR_WORKSPACE;
    const size_t b = value_bytes(dtype), bo = value_bytes(dW_dtype);
    if (!dW || !aligned(dW, bo)) return FCKL_ERR_ARG;
    if (N > 0 && (!g || !tokens || !aligned(g, b) || !aligned(tokens, 4))) return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* w = static_cast<uint8_t*>(ws);
    unsigned* status = static_cast<unsigned*>(ws);
    if (N == 0) {
      cudaError_t e = cudaMemsetAsync(status, 0, sizeof(unsigned), s);
      if (e == cudaSuccess && !accumulate) e = cudaMemsetAsync(dW, 0, size_t(V) * d * bo, s);
      if (e != cudaSuccess) {
        set_error("cudaMemsetAsync", e);
        return FCKL_ERR_CUDA;
      }
      return FCKL_OK;
    }
    SortParams sp{};
    sp.tokens = tokens;
    sp.N = static_cast<int>(N);
    sp.V = V;
    sp.passes = q.passes;
    sp.bits = q.bits;
    sp.a = reinterpret_cast<uint2*>(w + q.off_a);
    sp.b = reinterpret_cast<uint2*>(w + q.off_b);
    sp.status = status;
    if (!accumulate) {
      // whole 16-byte vectors from the first boundary on; what lies before it is short
      sp.zero = static_cast<uint8_t*>(dW);
      sp.zero_bytes = int64_t(V) * d * int64_t(bo);
      const int64_t ahead = std::min<int64_t>(-reinterpret_cast<uintptr_t>(dW) & 15u, sp.zero_bytes);
      if (ahead) {
        cudaError_t e = cudaMemsetAsync(dW, 0, size_t(ahead), s);
        if (e != cudaSuccess) {
          set_error("cudaMemsetAsync", e);
          return FCKL_ERR_CUDA;
        }
        sp.zero += ahead;
        sp.zero_bytes -= ahead;
      }
    }
    if ((st = launch_sort_tokens(di, sp, s))) return st;
    EmbedGradParams p{};
    p.list = q.passes & 1 ? sp.a : sp.b;
    p.N = static_cast<int>(N);
    p.V = V;
    p.d = d;
    p.g = g;
    p.ldg = ldg;
    p.dW = dW;
    p.scale = scale;
    p.status = status;
    p.tiles = q.tiles;
    p.partial = reinterpret_cast<float*>(w + q.off_partial);
    p.ldp = q.ldp;
    const int e_out = pack_of(dW, d, V, d, bo);
    int e = pack_of(g, ldg, N, d, b);
    if (e_out * bo < 16) e = std::min(e, e_out);  // 16 bytes of dW: several of its packs make one of g's
    if (dtype == FCKL_BF16) return launch_embedding_grad_type<__nv_bfloat16>(di, e, dtype, dW_dtype, accumulate != 0, p, s);
    if (dtype == FCKL_F16) return launch_embedding_grad_type<__half>(di, e, dtype, dW_dtype, accumulate != 0, p, s);
    return launch_embedding_grad_type<float>(di, e, dtype, dW_dtype, accumulate != 0, p, s);
  });
}

}  // extern "C"
