// Host side of the 8-bit projection (block_scaled.cuh): argument checks, launches and the C entry
// points declared in include/fckl.h. Part of the translation unit of fckl.cu.
#pragma once

#include "block_scaled.cuh"
#include "score_host.cuh"
#include "skinny.cuh"

namespace fckl {
namespace {

constexpr int64_t BS_MAX_ROWS = int64_t(1) << 30;  // rows are TMA coordinates (int32)
constexpr int64_t BS_MAX_COLS = int64_t(1) << 20;  // the framework's limit of d

template <typename T>
int launch_quantize(const QuantParams& p, int block_rows, cudaStream_t s) {
  if (block_rows == 1) {
    const unsigned grid = static_cast<unsigned>(cdiv(p.rows, QUANT_ROWS) * cdiv(p.kblocks, QUANT_UNROLL));
    return launch(KIND_BLOCK_QUANTIZE, s, "block_quantize",
                  [&] { quantize_rows_kernel<T><<<grid, QUANT_THREADS, 0, s>>>(p); });
  }
  const unsigned grid = static_cast<unsigned>(cdiv(p.rows, QB) * p.kblocks);
  return launch(KIND_BLOCK_QUANTIZE, s, "block_quantize",
                [&] { quantize_blocks_kernel<T><<<grid, QUANT_THREADS, 0, s>>>(p); });
}

template <typename TC>
int launch_block_matmul(DevInfo* di, const BlockMatmulParams& p, cudaStream_t s) {
  auto k = block_matmul_kernel<TC>;
  static_assert(BS_SMEM <= 232448, "shared memory budget");
  static int max_pairs[64] = {};
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(BS_THREADS);
  cfg.dynamicSmemBytes = BS_SMEM;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs;
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!max_pairs[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(BS_SMEM));
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(block_matmul)", e);
        return FCKL_ERR_CUDA;
      }
      int n = di->sms / 2, m = 0;
      cfg.gridDim = dim3(static_cast<unsigned>(2 * n));
      if (cudaOccupancyMaxActiveClusters(&m, k, &cfg) == cudaSuccess && m > 0) n = std::min(n, m);
      cudaGetLastError();
      max_pairs[di->id] = n;
    }
    pairs = max_pairs[di->id];
  }
  cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min(p.num_units, pairs)));
  cfg.stream = s;
  return launch(KIND_BLOCK_MATMUL, s, "block_scaled_matmul", [&] { cudaLaunchKernelEx(&cfg, k, p); });
}

size_t skinny_matmul_smem(int NG, int K) {
  return size_t(8 * NG) * skinny_pitch(K) + size_t(2) * SK_WARPS * SK8_ROWS * 8 * NG * 4 +
         size_t(cdiv(K, QB)) * 8 * NG * 4;
}

template <int NG, typename TC>
int launch_matmul_skinny(DevInfo* di, SkinnyMatmulParams p, cudaStream_t s) {
  auto k = block_matmul_skinny_kernel<NG, TC>;
  static bool done[64] = {};
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!done[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SK8_SMEM_MAX);
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(block_matmul_skinny)", e);
        return FCKL_ERR_CUDA;
      }
      done[di->id] = true;
    }
  }
  p.tiles = static_cast<int>(cdiv(p.N, SK8_ROWS));
  const unsigned grid = static_cast<unsigned>(std::min(p.tiles, 2 * di->sms));
  const size_t smem = skinny_matmul_smem(NG, p.K);
  return launch(KIND_MATMUL_SKINNY, s, "block_matmul_skinny", [&] { k<<<grid, SK_THREADS, smem, s>>>(p); });
}
template <typename TC>
int launch_matmul_skinny_any(DevInfo* di, const SkinnyMatmulParams& p, cudaStream_t s) {
  switch (cdiv(p.M, 8)) {
    case 1: return launch_matmul_skinny<1, TC>(di, p, s);
    default: return launch_matmul_skinny<2, TC>(di, p, s);
  }
}

}  // namespace
}  // namespace fckl

extern "C" {

int fckl_block_quantize(const void* x, int dtype, int64_t ldx, int64_t rows, int64_t cols, int block_rows, void* q,
                        int64_t ldq, float* scale, int64_t scale_rs, int64_t scale_cs, void* stream) {
  return guarded("fckl_block_quantize", [&]() -> int {
    if (rows < 0 || cols < 1 || !known_dtype(dtype) || (block_rows != 1 && block_rows != QB)) return FCKL_ERR_ARG;
    if (ldx < cols || ldq < cols || scale_rs < 1 || scale_cs < 1) return FCKL_ERR_ARG;
    if (rows > BS_MAX_ROWS || cols > BS_MAX_COLS || ldx > (int64_t(1) << 40) || ldq > (int64_t(1) << 40))
      return FCKL_ERR_UNSUPPORTED;
    if (ldq % 16 != 0) return FCKL_ERR_UNSUPPORTED;
    if (rows == 0) return FCKL_OK;
    if (!x || !q || !scale || !aligned(x, value_bytes(dtype)) || !aligned(q, 16) || !aligned(scale, 4))
      return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    int st = device_info(&di);
    if (st) return st;
    QuantParams p{};
    p.x = x;
    p.ldx = ldx;
    p.rows = rows;
    p.cols = static_cast<int>(cols);
    p.kblocks = static_cast<int>(cdiv(cols, QB));
    p.wide = aligned(x, 16) && ldx * value_bytes(dtype) % 16 == 0;
    p.q = static_cast<uint8_t*>(q);
    p.ldq = ldq;
    p.scale = scale;
    p.rs = scale_rs;
    p.cs = scale_cs;
    // one grid of up to 2^31 - 1 thread blocks
    if ((block_rows == 1 ? cdiv(rows, QUANT_ROWS) * cdiv(p.kblocks, QUANT_UNROLL) : cdiv(rows, QB) * p.kblocks) >
        INT_MAX)
      return FCKL_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FCKL_BF16) return launch_quantize<__nv_bfloat16>(p, block_rows, s);
    if (dtype == FCKL_F16) return launch_quantize<__half>(p, block_rows, s);
    return launch_quantize<float>(p, block_rows, s);
  });
}

int fckl_block_scaled_matmul(const void* a, int64_t lda, const float* sa, int64_t sa_rs, int64_t sa_cs, const void* b,
                             int64_t ldb, const float* sb, int64_t sb_rs, int64_t sb_cs, int64_t M, int64_t N,
                             int64_t K, void* c, int c_dtype, int64_t ldc, void* ws, size_t ws_bytes, void* stream) {
  return guarded("fckl_block_scaled_matmul", [&]() -> int {
    if (M < 0 || N < 1 || K < 1 || (c_dtype != FCKL_BF16 && c_dtype != FCKL_F32)) return FCKL_ERR_ARG;
    if (lda < K || ldb < K || ldc < N || sa_rs < 1 || sa_cs < 1 || sb_rs < 1 || sb_cs < 1) return FCKL_ERR_ARG;
    if (M > BS_MAX_ROWS || N > BS_MAX_ROWS || K > BS_MAX_COLS) return FCKL_ERR_UNSUPPORTED;
    // pitches of the tensor maps: multiples of 16 bytes below 2^40
    if (lda % 16 != 0 || ldb % 16 != 0 || lda >= (int64_t(1) << 40) || ldb >= (int64_t(1) << 40) ||
        ldc >= (int64_t(1) << 38))
      return FCKL_ERR_UNSUPPORTED;
    int st = status_ws_checks(ws, ws_bytes);
    if (st) return st;
    if (M == 0) return FCKL_OK;
    if (!a || !b || !sa || !sb || !c || !aligned(a, 16) || !aligned(b, 16) || !aligned(sa, 4) || !aligned(sb, 4) ||
        !aligned(c, value_bytes(c_dtype)))
      return FCKL_ERR_ARG;
    BlockMatmulParams p;
    memset(&p, 0, sizeof(p));
    const int64_t mb = cdiv(M, 2 * BM), nb = cdiv(N, 256);
    if (mb * nb > INT_MAX - 1024) return FCKL_ERR_UNSUPPORTED;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (M <= SK_MAX_POS && skinny_matmul_smem(static_cast<int>(cdiv(M, 8)), static_cast<int>(K)) <= SK8_SMEM_MAX) {
      SkinnyMatmulParams q{};
      q.a = static_cast<const uint8_t*>(a);
      q.lda = lda;
      q.sa = sa;
      q.sa_rs = sa_rs;
      q.sa_cs = sa_cs;
      q.b = static_cast<const uint8_t*>(b);
      q.ldb = ldb;
      q.sb = sb;
      q.sb_rs = sb_rs;
      q.sb_cs = sb_cs;
      q.M = static_cast<int>(M);
      q.K = static_cast<int>(K);
      q.k_blocks = static_cast<int>(cdiv(K, QB));
      q.N = N;
      q.c = c;
      q.ldc = ldc;
      return c_dtype == FCKL_BF16 ? launch_matmul_skinny_any<__nv_bfloat16>(di, q, s)
                                  : launch_matmul_skinny_any<float>(di, q, s);
    }
    if ((st = make_map(&p.tmA, a, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, M, lda, QB, BM))) return st;
    if ((st = make_map(&p.tmB, b, CU_TENSOR_MAP_DATA_TYPE_UINT8, K, N, ldb, QB, BM))) return st;
    p.m_blocks = static_cast<int>(mb);
    p.n_blocks = static_cast<int>(nb);
    p.k_blocks = static_cast<int>(cdiv(K, QB));
    p.num_units = static_cast<int>(mb * nb);
    p.M = M;
    p.N = N;
    p.sa = sa;
    p.sa_rs = sa_rs;
    p.sa_cs = sa_cs;
    p.sb = sb;
    p.sb_rs = sb_rs;
    p.sb_cs = sb_cs;
    p.c = c;
    p.ldc = ldc;
    const size_t cb = value_bytes(c_dtype);
    p.wide = aligned(c, 16) && ldc * cb % 16 == 0;
    if (p.wide && (st = make_map(&p.tmC, c, c_dtype == FCKL_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                                                : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                 N, M, ldc * cb, static_cast<uint32_t>(128 / cb), 32)))
      return st;
    p.status = static_cast<unsigned*>(ws);
    return c_dtype == FCKL_BF16 ? launch_block_matmul<__nv_bfloat16>(di, p, s) : launch_block_matmul<float>(di, p, s);
  });
}

}  // extern "C"
