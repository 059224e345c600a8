// Products with few positions (decoding): W streams once through the SMs at memory speed.
//
// With at most 16 positions a projection reads W [V, d] and does next to nothing with it: 2 N flops
// per value. What counts is that W comes from HBM in long contiguous runs. The tiles of the large
// products do the opposite (256 rows, 128 or 256 bytes of each at a time): they read W at 4.0 of
// 6.8 TB/s. Here a block takes 16 whole rows, contiguous in memory, at a time; its eight warps share
// the rows' length and read 512 bytes of each row together.
//
// The values go straight from global memory into the operand registers of the warp-level MMAs (m16:
// rows of W, n8: positions). Such an MMA wants a lane's values from two places of a row; since a sum
// over k may be taken in any order, a lane's 16 loaded bytes are used for both, and the hidden states
// are picked from shared memory in the same order. Its rate does not matter: at 8 positions
// the tensor pipe is 9% busy. 2880 x 201088: 177 us in bf16 (6.5 TB/s, 0.96 of the copy bandwidth) up to 8
// positions against 210 to 320 with the large product's tiles; in 8 bits 94 us (0.91), and 116 at 16
// positions, against 150. Per block and 16 rows the warps' partial sums meet in shared memory (one
// barrier, two buffers), where the epilogue takes over: a thread always serves the same position.
#pragma once

#include <cuda_bf16.h>
#include <cstdint>

#include "score.cuh"

namespace fckl {

constexpr int SK_WARPS = 8;
constexpr int SK_THREADS = 32 * SK_WARPS;
constexpr int SK_ROWS = 16;        // rows of W per block and step
constexpr int SK_MAX_POS = 16;     // positions
constexpr int SK_MAX_TOKENS = 32;  // given tokens per position
constexpr int SK_BATCH = 4;        // loads in flight per lane and row
// Shared memory of a block, two to an SM: what they leave of the SM's 256 KB is what loads pass
// through. At 16 x 2880 x 201088 (bf16; 110 KB a block) the kernel takes 345 us, at 8 positions (55 KB)
// 189, the large product 217 at either.
constexpr int SK_SMEM_MAX = 64 * 1024;
// The 8-bit kernel's rows are half as long, and its room for partial sums twice as large.
constexpr int SK8_SMEM_MAX = 96 * 1024;
constexpr int SK_MAX_BLOCKS = 1024;

__device__ __forceinline__ uint4 load_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Bytes between the positions' rows in shared memory: 64 more than a multiple of 128, so that the
// 16-byte reads of two positions fall into different banks.
__host__ __device__ constexpr int skinny_pitch(int row_bytes) { return (row_bytes + 127) / 128 * 128 + 64; }

struct HeadSkinnyParams {
  const __nv_bfloat16* H;
  const __nv_bfloat16* W;
  const int32_t* tokens;
  int N, d, V, T;
  int tiles;  // of SK_ROWS rows
  float *pm, *pl, *pt;  // [blocks][ld]
  int ld;
  float* zt;  // [N][T] logits of the tokens
  unsigned* status;
};

// Scoring of up to 8 NG positions: logits of 16 rows of W at a time, folded into each position's
// running statistics (one set per block, merged by head_combine_kernel).
template <int NG>
__global__ void __launch_bounds__(SK_THREADS, 2) head_skinny_kernel(const HeadSkinnyParams p) {
  constexpr int POS = 8 * NG;
  constexpr int VALUES = SK_ROWS * POS;                               // logits per step
  constexpr int PER = (VALUES + SK_THREADS - 1) / SK_THREADS;         // of one thread
  extern __shared__ __align__(16) uint8_t sk_smem[];
  const int pitch = skinny_pitch(p.d * 2);
  uint8_t* hs = sk_smem;                                              // [POS][pitch]
  float* part = reinterpret_cast<float*>(sk_smem + POS * pitch);      // [2][SK_WARPS][VALUES]
  int* toks = reinterpret_cast<int*>(part + 2 * SK_WARPS * VALUES);   // [N][T]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

  // hidden states, zero beyond N and d
  const int vecs = pitch / 16;
  for (int i = tid; i < POS * vecs; i += SK_THREADS) {
    const int n = i / vecs, k = (i - n * vecs) * 8;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n < p.N && k < p.d) v = *reinterpret_cast<const uint4*>(p.H + static_cast<int64_t>(n) * p.d + k);
    *reinterpret_cast<uint4*>(hs + n * pitch + k * 2) = v;
  }
  for (int i = tid; i < p.N * p.T; i += SK_THREADS) {
    const int id = p.tokens[i];
    toks[i] = id;
    if (blockIdx.x == 0 && (id < -1 || id >= p.V)) atomicOr(p.status, ST_BAD_INDEX);
  }
  __syncthreads();

  const int chunks = (p.d + 31) / 32;  // of 32 values: 64 bytes of a row, 16 per lane
  const int batches = (chunks + SK_WARPS * SK_BATCH - 1) / (SK_WARPS * SK_BATCH);
  uint4 cur[SK_BATCH][2], nxt[SK_BATCH][2];
  auto fetch = [&](uint4 (&to)[SK_BATCH][2], int tile, int b) {
    const int r0 = tile * SK_ROWS + g;
#pragma unroll
    for (int u = 0; u < SK_BATCH; ++u) {
      const int k = ((b * SK_BATCH + u) * SK_WARPS + warp) * 32 + 8 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = r0 + 8 * h;
        to[u][h] = (k < p.d && r < p.V) ? load_stream(p.W + static_cast<int64_t>(r) * p.d + k) : make_uint4(0, 0, 0, 0);
      }
    }
  };

  RowStat s[PER];
  if (static_cast<int>(blockIdx.x) < p.tiles) fetch(cur, blockIdx.x, 0);
  int buf = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, buf ^= 1) {
    float c[NG][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) c[n][0] = c[n][1] = c[n][2] = c[n][3] = 0.f;
    for (int b = 0; b < batches; ++b) {
      const bool last = b + 1 == batches;  // the next batch, of this step or the next one
      const int nt = last ? tile + static_cast<int>(gridDim.x) : tile;
      if (nt < p.tiles) fetch(nxt, nt, last ? 0 : b + 1);
#pragma unroll
      for (int u = 0; u < SK_BATCH; ++u) {
        const int ch = (b * SK_BATCH + u) * SK_WARPS + warp;
        if (ch >= chunks) break;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const uint4 h = *reinterpret_cast<const uint4*>(hs + (8 * n + g) * pitch + ch * 64 + 16 * t);
          mma_bf16(c[n], cur[u][0].x, cur[u][1].x, cur[u][0].y, cur[u][1].y, h.x, h.y);
          mma_bf16(c[n], cur[u][0].z, cur[u][1].z, cur[u][0].w, cur[u][1].w, h.z, h.w);
        }
      }
#pragma unroll
      for (int u = 0; u < SK_BATCH; ++u) {
        cur[u][0] = nxt[u][0];
        cur[u][1] = nxt[u][1];
      }
    }
    // partial sums [position][row]
    float* mine = part + (buf * SK_WARPS + warp) * VALUES;
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      float* at = mine + (8 * n + 2 * t) * SK_ROWS + g;
      at[0] = c[n][0];
      at[SK_ROWS] = c[n][1];
      at[8] = c[n][2];
      at[SK_ROWS + 8] = c[n][3];
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int v = j * SK_THREADS + tid;
      if (v >= VALUES) break;
      const float* from = part + buf * SK_WARPS * VALUES + v;
      float z = from[0];
#pragma unroll
      for (int w = 1; w < SK_WARPS; ++w) z += from[w * VALUES];
      const int n = v / SK_ROWS, r = tile * SK_ROWS + v % SK_ROWS;
      if (n < p.N && r < p.V) {
        if (z > s[j].m) {
          RowStat top;
          top.m = z;
          s[j] = merge(s[j], top);
        }
        const float x[1] = {z};
        add_values<1>(s[j], x);
        for (int q = 0; q < p.T; ++q)
          if (toks[n * p.T + q] == r) p.zt[n * p.T + q] = z;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {  // the 16 rows of a step
      RowStat b;
      b.m = __shfl_xor_sync(0xffffffffu, s[j].m, o);
      b.l = __shfl_xor_sync(0xffffffffu, s[j].l, o);
      b.t = __shfl_xor_sync(0xffffffffu, s[j].t, o);
      s[j] = merge(s[j], b);
    }
    const int v = j * SK_THREADS + tid, n = v / SK_ROWS;
    if (v < VALUES && v % SK_ROWS == 0 && n < p.N) {
      const size_t o = static_cast<size_t>(blockIdx.x) * p.ld + n;
      p.pm[o] = s[j].m;
      p.pl[o] = s[j].l;
      p.pt[o] = s[j].t;
    }
  }
}

// ---------------------------------------------------------------- 8 bits
__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SkinnyMatmulParams {
  const uint8_t* a;  // [M, K] e4m3, rows lda bytes apart
  int64_t lda;
  const float* sa;
  int64_t sa_rs, sa_cs;
  const uint8_t* b;  // [N, K]
  int64_t ldb;
  const float* sb;
  int64_t sb_rs, sb_cs;
  int M, K, k_blocks;
  int64_t N;
  int tiles;
  void* c;
  int64_t ldc;
};

// C of up to 8 NG rows of A. A warp takes whole K-blocks of 128 bytes (two loads of 16 bytes per lane
// and row), scales each one's sums and adds them up; a block takes 32 rows of B at a time, so that
// one K-block per warp keeps 4 KB in flight (with 16 rows and two K-blocks the second one is mostly
// past a row of 2880: 144 us, against 109 with 32 rows, at 8 x 2880 x 201088).
constexpr int SK8_ROWS = 32;
template <int NG, typename TC>
__global__ void __launch_bounds__(SK_THREADS, 2) block_matmul_skinny_kernel(const SkinnyMatmulParams p) {
  constexpr int POS = 8 * NG;
  constexpr int VALUES = SK8_ROWS * POS;
  constexpr int PER = (VALUES + SK_THREADS - 1) / SK_THREADS;
  extern __shared__ __align__(16) uint8_t sk_smem[];
  const int pitch = skinny_pitch(p.K);
  uint8_t* as = sk_smem;                                             // [POS][pitch]
  float* part = reinterpret_cast<float*>(sk_smem + POS * pitch);     // [2][SK_WARPS][VALUES]
  float* sas = part + 2 * SK_WARPS * VALUES;                         // [k_blocks][POS]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;

  const int vecs = pitch / 16;
  for (int i = tid; i < POS * vecs; i += SK_THREADS) {
    const int n = i / vecs, k = (i - n * vecs) * 16;
    uint4 v = make_uint4(0, 0, 0, 0);
    if (n < p.M && k < p.K) {
      const uint8_t* from = p.a + n * p.lda + k;
      if (k + 16 <= p.K) {
        v = *reinterpret_cast<const uint4*>(from);
      } else {  // zeros past K: the row's padding may hold anything
        __align__(16) uint8_t x[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] = k + j < p.K ? from[j] : 0;
        v = *reinterpret_cast<const uint4*>(x);
      }
    }
    *reinterpret_cast<uint4*>(as + n * pitch + k) = v;
  }
  for (int i = tid; i < POS * p.k_blocks; i += SK_THREADS) {
    const int n = i % POS, kb = i / POS;
    sas[i] = n < p.M ? p.sa[n * p.sa_rs + kb * p.sa_cs] : 0.f;
  }
  __syncthreads();

  const int batches = (p.k_blocks + SK_WARPS - 1) / SK_WARPS;
  uint4 cur[2][4], nxt[2][4];  // [half of a K-block][row g + 8 h]
  auto fetch = [&](uint4 (&to)[2][4], int tile, int b) {
    const int64_t r0 = static_cast<int64_t>(tile) * SK8_ROWS + g;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int k = (b * SK_WARPS + warp) * 128 + u * 64 + 16 * t;
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int64_t r = r0 + 8 * h;
        // 16 bytes that start before K lie within the row (its pitch is a multiple of 16); what is
        // past K in them meets the zeros of `as`, but as e4m3 it may be a NaN: cleared below
        to[u][h] = (k < p.K && r < p.N) ? load_stream(p.b + r * p.ldb + k) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  const int tail = p.K & 15;  // bytes of the last vector that count, 0: all
  auto clear_tail = [&](uint4& v) {
    uint32_t* w = &v.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int left = tail - 4 * j;
      w[j] = left >= 4 ? w[j] : left <= 0 ? 0u : w[j] & ((1u << (8 * left)) - 1u);
    }
  };

  if (static_cast<int>(blockIdx.x) < p.tiles) fetch(cur, blockIdx.x, 0);
  int buf = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x, buf ^= 1) {
    const float* sb = p.sb + static_cast<int64_t>(tile) * SK8_ROWS / 128 * p.sb_rs;
    float c[2][NG][4];  // [rows 16 m + ...]
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NG; ++n) c[m][n][0] = c[m][n][1] = c[m][n][2] = c[m][n][3] = 0.f;
    for (int b = 0; b < batches; ++b) {
      const bool last = b + 1 == batches;  // the next batch, of this step or the next one
      const int nt = last ? tile + static_cast<int>(gridDim.x) : tile;
      if (nt < p.tiles) fetch(nxt, nt, last ? 0 : b + 1);
      const int kb = b * SK_WARPS + warp;
      if (kb < p.k_blocks) {
        const float sw = __ldg(sb + kb * p.sb_cs);
        float x[2][NG][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int n = 0; n < NG; ++n) x[m][n][0] = x[m][n][1] = x[m][n][2] = x[m][n][3] = 0.f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int k = kb * 128 + u * 64;
          if (k >= p.K) break;
          if (tail && k + 16 * t < p.K && k + 16 * t + 16 > p.K) {
#pragma unroll
            for (int h = 0; h < 4; ++h) clear_tail(cur[u][h]);
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const uint4 h = *reinterpret_cast<const uint4*>(as + (8 * n + g) * pitch + k + 16 * t);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint4 &lo = cur[u][2 * m], &hi = cur[u][2 * m + 1];
              mma_e4m3(x[m][n], lo.x, hi.x, lo.y, hi.y, h.x, h.y);
              mma_e4m3(x[m][n], lo.z, hi.z, lo.w, hi.w, h.z, h.w);
            }
          }
        }
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const float2 sh = *reinterpret_cast<const float2*>(sas + kb * POS + 8 * n + 2 * t);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            c[m][n][0] = fmaf(x[m][n][0], sh.x * sw, c[m][n][0]);
            c[m][n][1] = fmaf(x[m][n][1], sh.y * sw, c[m][n][1]);
            c[m][n][2] = fmaf(x[m][n][2], sh.x * sw, c[m][n][2]);
            c[m][n][3] = fmaf(x[m][n][3], sh.y * sw, c[m][n][3]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int h = 0; h < 4; ++h) cur[u][h] = nxt[u][h];
    }
    float* mine = part + (buf * SK_WARPS + warp) * VALUES;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        float* at = mine + (8 * n + 2 * t) * SK8_ROWS + 16 * m + g;
        at[0] = c[m][n][0];
        at[SK8_ROWS] = c[m][n][1];
        at[8] = c[m][n][2];
        at[SK8_ROWS + 8] = c[m][n][3];
      }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int v = j * SK_THREADS + tid;
      if (v >= VALUES) break;
      const float* from = part + buf * SK_WARPS * VALUES + v;
      float z = from[0];
#pragma unroll
      for (int w = 1; w < SK_WARPS; ++w) z += from[w * VALUES];
      const int n = v / SK8_ROWS;
      const int64_t r = static_cast<int64_t>(tile) * SK8_ROWS + v % SK8_ROWS;
      if (n < p.M && r < p.N) static_cast<TC*>(p.c)[n * p.ldc + r] = from_f32<TC>(z);
    }
  }
}

}  // namespace fckl
