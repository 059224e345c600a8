// Output projection in 8-bit floating point (e4m3) with a scale for each block of 128.
//
// block_quantize_kernel: x [R, C] to e4m3 values and one fp32 scale per block_rows x 128 block
// (block_rows 1: hidden states, one scale per position and 128 channels; 128: output matrices):
//   s = max(amax / 448, 2^-126),   q = e4m3(x / s)
// 448 is the largest e4m3 value. Both quotients are rounded to nearest in fp32 before anything
// else is done with them, so the values are the same wherever the definition is followed.
//
// block_matmul_kernel: C[m, n] = sum_kb sa[m, kb] sb[n / 128, kb] sum_{k in kb} A[m, k] B[n, k],
// with A [M, K] and B [N, K] in e4m3. The tensor cores sum one K-block of 128 at a time in fp32
// (TMEM); the epilogue warps scale each K-block's sums and add them up in fp32 registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cstdint>

#include "score.cuh"
#include "tc_gemm.cuh"

namespace fckl {

constexpr int QB = 128;  // values of a scale block along K
constexpr float E4M3_MAX = 448.f;
constexpr float SCALE_MIN = 1.17549435e-38f;  // 2^-126: a block of zeros, or of tiny values

// ---------------------------------------------------------------- quantisation
// 8 values as they lie in memory; zeros for those that are not there.
template <typename T>
struct Eight {
  static constexpr int WORDS = 2 * sizeof(T);
  uint32_t w[WORDS];
};

template <typename T>
__device__ __forceinline__ Eight<T> load8(const T* p, int left, bool wide) {
  Eight<T> v;
  if (wide && left >= 8) {
#pragma unroll
    for (int i = 0; i < Eight<T>::WORDS / 4; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + 4 * i);
      v.w[4 * i] = u.x;
      v.w[4 * i + 1] = u.y;
      v.w[4 * i + 2] = u.z;
      v.w[4 * i + 3] = u.w;
    }
  } else {
    __align__(16) T x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < left ? p[e] : from_f32<T>(0.f);
#pragma unroll
    for (int i = 0; i < Eight<T>::WORDS; ++i) v.w[i] = reinterpret_cast<const uint32_t*>(x)[i];
  }
  return v;
}

__device__ __forceinline__ void values_of_words(const uint32_t* w, float& a, float& b, float) {
  a = __uint_as_float(w[0]);
  b = __uint_as_float(w[1]);
}
template <typename T>
__device__ __forceinline__ void values_of_words(const uint32_t* w, float& a, float& b, T) {
  unpack2(w[0], a, b, T{});
}

// Largest magnitude of a value in words, as words again (NaNs drop out).
__device__ __forceinline__ uint32_t absmax_words(uint32_t m, uint32_t w, __nv_bfloat16) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ uint32_t absmax_words(uint32_t m, uint32_t w, __half) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(w & 0x7fff7fffu));
  return r;
}
__device__ __forceinline__ uint32_t absmax_words(uint32_t m, uint32_t w, float) {
  return __float_as_uint(fmaxf(__uint_as_float(m), fabsf(__uint_as_float(w))));
}
template <typename T>
__device__ __forceinline__ uint32_t absmax8(uint32_t m, const Eight<T>& v) {
#pragma unroll
  for (int i = 0; i < Eight<T>::WORDS; ++i) m = absmax_words(m, v.w[i], T{});
  return m;
}
template <typename T>
__device__ __forceinline__ float absmax_value(uint32_t m) {
  if constexpr (sizeof(T) == 4) {
    return __uint_as_float(m);
  } else {
    float a, b;
    unpack2(m, a, b, T{});
    return fmaxf(a, b);
  }
}

// The scale of a block and how to divide by it. The quotient has to be the nearest fp32 number: with
// r the reciprocal rounded to nearest, q = x r and e = x - q s (exact in an FMA), q + e r rounds to
// the correctly rounded quotient (P. Markstein, IBM J. Res. Dev. 34, 1990). Its steps neither over-
// nor underflow where s is in the range below, except in quotients too small to be anything but 0
// in 8 bits; outside the range (a block with an infinity, or of nothing above 1e-27) the division
// operator does it.
struct BlockScale {
  float s, r;
  bool plain;  // plain division
  __device__ __forceinline__ explicit BlockScale(float amax) {
    s = fmaxf(__fdiv_rn(amax, E4M3_MAX), SCALE_MIN);
    plain = !(s > 2.5e-30f && s < 1e36f);
    r = __frcp_rn(s);
  }
};

template <typename T>
__device__ __forceinline__ void store8(uint8_t* q, int left, const Eight<T>& v, const BlockScale& bs) {
  union {
    __nv_fp8x2_storage_t h[4];
    uint8_t b[8];
    uint2 v;
  } u;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    values_of_words(v.w + e * Eight<T>::WORDS / 4, a, b, T{});
    if (bs.plain) {
      a = __fdiv_rn(a, bs.s);
      b = __fdiv_rn(b, bs.s);
    } else {
      const unsigned long long x = pack2(a, b), r = pack2(bs.r, bs.r);
      const unsigned long long q0 = mul2(x, r);
      unpack2f(fma2(fma2(q0, pack2(-bs.s, -bs.s), x), r, q0), a, b);
    }
    u.h[e] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  }
  if (left >= 8) {
    *reinterpret_cast<uint2*>(q) = u.v;  // rows of q start on 16-byte boundaries
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < left) q[e] = u.b[e];
  }
}

struct QuantParams {
  const void* x;
  int64_t ldx, rows;
  int cols, kblocks;
  int wide;  // x's rows start on 16-byte boundaries
  uint8_t* q;
  int64_t ldq;
  float* scale;
  int64_t rs, cs;  // element (row block, K-block) of scale at rb * rs + kb * cs
};

constexpr int QUANT_THREADS = 256;

// One scale per row and 128 columns: 16 lanes a row, 8 values each. A thread block takes 16 rows and
// QUANT_UNROLL adjacent scale blocks of them, whose loads are issued together (65536 x 2880 bf16:
// 115 us, 4.9 TB/s; one block at a time 150).
constexpr int QUANT_UNROLL = 4;
constexpr int QUANT_ROWS = QUANT_THREADS / 16;
template <typename T>
__global__ void __launch_bounds__(QUANT_THREADS) quantize_rows_kernel(const QuantParams p) {
  const int l = threadIdx.x & 15;
  const unsigned kgroups = (p.kblocks + QUANT_UNROLL - 1) / QUANT_UNROLL;
  const int64_t row = static_cast<int64_t>(blockIdx.x / kgroups) * QUANT_ROWS + threadIdx.x / 16;
  const int kb0 = static_cast<int>(blockIdx.x % kgroups) * QUANT_UNROLL;
  const bool on = row < p.rows;
  const T* x0 = static_cast<const T*>(p.x) + (on ? row : 0) * p.ldx;
  Eight<T> x[QUANT_UNROLL];
  int left[QUANT_UNROLL];
#pragma unroll
  for (int j = 0; j < QUANT_UNROLL; ++j) {
    const int c = (kb0 + j) * QB + 8 * l;
    left[j] = on ? p.cols - c : 0;
    x[j] = load8(x0 + c, left[j], p.wide);
  }
#pragma unroll
  for (int j = 0; j < QUANT_UNROLL; ++j) {
    float m = absmax_value<T>(absmax8(0u, x[j]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const BlockScale s(m);
    if (left[j] > 0) store8(p.q + row * p.ldq + (kb0 + j) * QB + 8 * l, left[j], x[j], s);
    // lane 0's values are there whenever its block is
    if (left[j] > 0 && l == 0) p.scale[row * p.rs + (kb0 + j) * p.cs] = s.s;
  }
}

// One scale per 128 x 128 block: a thread block each, the values held in registers between the
// maximum and the conversion. 201088 x 2880 bf16: 320 us (5.4 TB/s, 0.80 of the copy bandwidth) with
// four blocks per SM (two, at 100 registers: 497; with the division operator and values held as
// fp32: 980). Loads past L1, 512 threads or five blocks gave nothing.
template <typename T>
__global__ void __launch_bounds__(QUANT_THREADS, sizeof(T) == 4 ? 2 : 4) quantize_blocks_kernel(const QuantParams p) {
  constexpr int RSTEP = QUANT_THREADS / 16, STEPS = QB / RSTEP;
  __shared__ float wmax[QUANT_THREADS / 32];
  const int l = threadIdx.x & 15, r = threadIdx.x / 16;
  const int64_t rb = blockIdx.x / p.kblocks;
  const int kb = static_cast<int>(blockIdx.x - rb * p.kblocks);
  const int c = kb * QB + 8 * l;
  const T* x = static_cast<const T*>(p.x);
  Eight<T> v[STEPS];
  uint32_t mw = 0;
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int64_t row = rb * QB + j * RSTEP + r;
    const int left = row < p.rows ? p.cols - c : 0;
    v[j] = load8(x + (row < p.rows ? row : 0) * p.ldx + c, left, p.wide);
  }
#pragma unroll
  for (int j = 0; j < STEPS; ++j) mw = absmax8(mw, v[j]);
  float m = absmax_value<T>(mw);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < QUANT_THREADS / 32; ++w) m = fmaxf(m, wmax[w]);
  const BlockScale s(m);
#pragma unroll
  for (int j = 0; j < STEPS; ++j) {
    const int64_t row = rb * QB + j * RSTEP + r;
    if (row < p.rows && c < p.cols) store8(p.q + row * p.ldq + c, p.cols - c, v[j], s);
  }
  if (threadIdx.x == 0) p.scale[rb * p.rs + kb * p.cs] = s.s;
}

// ---------------------------------------------------------------- product
// Instruction descriptor for kind::f8f6f4 with e4m3 A and B (format 0), fp32 D, both K-major.
__host__ __device__ constexpr uint32_t make_idesc_e4m3(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem of both CTAs] (+)= A * B^T over the CTA pair, e4m3 operands, K = 32 per instruction.
__device__ __forceinline__ void umma_e4m3_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Bounded wait that leaves shared memory alone while it waits: each try may suspend the thread for up
// to 20 us, where the default polls on (2% of the product at 8192 x 2880 x 201088: its operands
// keep shared memory's bandwidth busy). After POLLS tries wait_phase applies its time limit.
constexpr int POLLS = 512;
__device__ __forceinline__ bool mbar_try_wait_20us(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool poll_phase(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                           unsigned* status) {
#pragma unroll 1
  for (int i = 0; i < POLLS; ++i)
    if (mbar_try_wait_20us(bar, parity)) return true;
  return wait_phase(bar, parity, abort_flag, status);
}

// 32 lanes x 64 consecutive 32-bit columns, as tmem_ld32: two such loads read a thread's share of a
// K-block, 3.56 ms against 4.25 ms with 16 columns at a time (8192 x 2880 x 201088).
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, "
      "%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31]), "=f"(v[32]),
        "=f"(v[33]), "=f"(v[34]), "=f"(v[35]), "=f"(v[36]), "=f"(v[37]), "=f"(v[38]), "=f"(v[39]), "=f"(v[40]),
        "=f"(v[41]), "=f"(v[42]), "=f"(v[43]), "=f"(v[44]), "=f"(v[45]), "=f"(v[46]), "=f"(v[47]), "=f"(v[48]),
        "=f"(v[49]), "=f"(v[50]), "=f"(v[51]), "=f"(v[52]), "=f"(v[53]), "=f"(v[54]), "=f"(v[55]), "=f"(v[56]),
        "=f"(v[57]), "=f"(v[58]), "=f"(v[59]), "=f"(v[60]), "=f"(v[61]), "=f"(v[62]), "=f"(v[63])
      : "r"(taddr)
      : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_lane() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}

// Arrive on an mbarrier of another CTA of the cluster. Only TMEM is handed over with it, which the
// tcgen05 fences order: no memory of this thread has to be made visible to the other SM (with
// cluster-wide release and acquire on this hand-off a K-block took 2400 cycles rather than 1400).
__device__ __forceinline__ void arrive_peer(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar_cluster) : "memory");
}

constexpr int BS_EPI_WARPS = 8;  // two per TMEM lane quarter: 128 fp32 sums per thread
constexpr int BS_THREADS = 128 + 32 * BS_EPI_WARPS;
// Registers per thread: a block of 384 threads is launched with 168 (65536 / 384, rounded down to 8);
// the first four warps give up what the epilogue's 128 sums and 64 values read at once need.
constexpr int BS_REGS_FEW = 56, BS_REGS_EPI = 224;
static_assert(128 * BS_REGS_FEW + 32 * BS_EPI_WARPS * BS_REGS_EPI <= BS_THREADS * 168, "registers at launch");
constexpr int BS_STAGES = 5;
constexpr uint32_t BS_A_BYTES = BM * QB, BS_B_BYTES = BM * QB;
constexpr uint32_t BS_STAGE_BYTES = BS_A_BYTES + BS_B_BYTES;
constexpr uint32_t BS_OUT_OFF = BS_STAGES * BS_STAGE_BYTES;  // two staging boxes per epilogue warp
constexpr uint32_t BS_BAR_OFF = BS_OUT_OFF + BS_EPI_WARPS * 2 * EPI_BUF_BYTES;
constexpr uint32_t BS_SMEM = BS_BAR_OFF + (2 * BS_STAGES + 5) * 8 + 16 + 1024;

struct BlockMatmulParams {
  CUtensorMap tmA;  // A [M, K] e4m3, 128 x 128 boxes
  CUtensorMap tmB;  // B [N, K]
  CUtensorMap tmC;  // C, boxes of 32 rows x 128 bytes (wide)
  int m_blocks, n_blocks, k_blocks, num_units;
  int64_t M, N;
  const float* sa;
  int64_t sa_rs, sa_cs;
  const float* sb;
  int64_t sb_rs, sb_cs;
  void* c;
  int64_t ldc;
  int wide;  // c's rows start on 16-byte boundaries
  unsigned* status;
};

// Persistent, one CTA per SM, SM pairs: a pair computes 256 x 256 of C (each CTA 128 rows). Warp 0
// fills a ring of K-blocks (16 KB of A, 16 KB of B per CTA), warp 1 of the even CTA issues four
// MMAs per K-block into one of two 256-column TMEM buffers, and the eight epilogue warps of both
// CTAs fold each buffer into their registers while the next K-block is multiplied into the other.
//
// What bounds it: a K-block is 512 cycles of MMA at the 8-bit rate, and TMEM holds two. Measured inside
// the kernel, a K-block's round is 1600 cycles from the issue of its MMAs to their commit (behind the
// other buffer's), 300 to read the sums and 400 until the buffer is free again at the MMA warp, so a
// K-block takes 900 to 1100. With one hand-off per tile instead of one per K-block, which cannot apply
// the scales, the same loop takes 2.7 ms at 8192 x 2880 x 201088. Steps at that size (bf16 C; single
// launches, before the power cap sets in: in a sequence of them the last one takes 4.0 ms):
// 9.7 ms with cluster-scope release and acquire on the hand-off; 5.8 ms without; 4.25 ms with the
// MMA warp converged (its loop was 1000 cycles) and C staged and stored with TMA; 3.7 ms with half
// the reads, twice as wide; 3.6 ms with the next tile's scales fetched early and longer suspended
// waits. Slower: four 128-column buffers (4.5 ms, A is read twice from shared memory), tiles of 128
// columns with four K-blocks in TMEM (5.6 ms), sixteen epilogue warps (3.9 ms), two K-blocks per
// ring stage (3.9 ms), one lane waiting for a warp (3.9 ms).
template <typename TC>
__global__ void __launch_bounds__(BS_THREADS, 1) block_matmul_kernel(const __grid_constant__ BlockMatmulParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + BS_BAR_OFF);
  uint64_t* empty = full + BS_STAGES;
  uint64_t* tfull = empty + BS_STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x / 2, num_pairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < BS_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * BS_EPI_WARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tmA);
    prefetch_tmap(&p.tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers exist before anyone signals them
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(BS_REGS_FEW));
    if (warp == 0 && lane == 0) {
      // -------------------------------------------------------- TMA producer (each CTA)
      uint32_t cnt = 0, armed = 0, armed_par = 0;
      bool ok = true;
      const uint32_t full_base = mapa_shared(smem_u32(full), 0);
      for (int u = pair; ok && u < p.num_units; u += num_pairs) {
        const int nb = u / p.m_blocks, mb = u - nb * p.m_blocks;
        const int arow = (2 * mb + static_cast<int>(rank)) * BM;
        const int brow = (2 * nb + static_cast<int>(rank)) * BM;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++cnt) {
          const uint32_t s = cnt % BS_STAGES, ph = (cnt / BS_STAGES) & 1u;
          if (!poll_phase(&empty[s], ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&full[s], 2 * BS_STAGE_BYTES);
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | (ph << s);
          }
          uint8_t* a = smem + s * BS_STAGE_BYTES;
          const uint32_t fb = full_base + s * 8u;
          tma_load_2d_pair(a, &p.tmA, fb, kb * QB, arow);
          tma_load_2d_pair(a + BS_A_BYTES, &p.tmB, fb, kb * QB, brow);
        }
      }
      // every copy this pair started lands before a CTA may exit (see tc_gemm.cuh)
      if (leader) {
        for (int s = 0; s < BS_STAGES; ++s)
          if (armed & (1u << s)) drain_phase(&full[s], (armed_par >> s) & 1u, p.status);
      } else if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    } else if (warp == 1 && leader) {
      // -------------------------------------------------------- MMA issuer (leader CTA)
      // The whole warp walks the loop and one elected lane issues: converged, the compiler keeps
      // descriptors and addresses in uniform registers, which the MMAs take.
      constexpr uint32_t IDESC = make_idesc_e4m3(2 * BM, 256);
      const uint64_t a0 = make_sdesc_sw128(smem_u32(smem), 16, 1024);
      uint32_t cnt = 0;
      bool ok = true;
      for (int u = pair; ok && u < p.num_units; u += num_pairs) {
        for (int kb = 0; kb < p.k_blocks; ++kb, ++cnt) {
          const uint32_t acc = cnt & 1u, use = cnt >> 1;
          const uint32_t s = cnt % BS_STAGES, ph = (cnt / BS_STAGES) & 1u;
          ok = poll_phase(&full[s], ph, abort_flag, p.status) &&
               poll_phase(&tempty[acc], (use & 1u) ^ 1u, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
          if (elect_lane()) {
            const uint64_t ad = a0 + static_cast<uint64_t>(s * (BS_STAGE_BYTES >> 4));
            const uint32_t d = tmem_base + acc * ACC_STRIDE;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              umma_e4m3_pair(d, ad + 2 * kk, ad + (BS_A_BYTES >> 4) + 2 * kk, IDESC, kk > 0);
            umma_commit_pair(&tfull[acc], 0x3);
            umma_commit_pair(&empty[s], 0x3);
          }
          __syncwarp();
        }
      }
      // all MMAs finish before TMEM is released; committed by the lane that issued them
      if (elect_lane()) umma_commit_pair(drain, 0x1);
      __syncwarp();
      if (lane == 0) drain_phase(drain, 0, p.status);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(BS_REGS_EPI));
    // ---------------------------------------------------------- epilogue (each CTA)
    const int q = warp & 3;           // TMEM lane quarter this warp may access
    const int half = (warp - 4) / 4;  // columns [128 half, 128 half + 128) of the tile
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    uint8_t* obuf = smem + BS_OUT_OFF + (warp - 4) * 2 * EPI_BUF_BYTES;
    uint32_t cnt = 0, ocnt = 0;
    bool ok = true;
    // This thread's row and first column of C and their scales. A tile's first scales are fetched
    // before the tile ahead of it is written out, later ones a K-block ahead.
    int64_t row = 0, col = 0;
    bool live = false;
    const float *sa = p.sa, *sb = p.sb;
    float a_next = 0.f, b_next = 0.f;
    auto enter = [&](int u) {
      const int nb = u / p.m_blocks, mb = u - nb * p.m_blocks;
      row = (2 * mb + static_cast<int64_t>(rank)) * BM + 32 * q + lane;
      col = static_cast<int64_t>(nb) * 256 + 128 * half;
      live = row < p.M && col < p.N;
      sa = p.sa + (live ? row : 0) * p.sa_rs;
      sb = p.sb + (live ? col / QB : 0) * p.sb_rs;
      a_next = live ? __ldg(sa) : 0.f;
      b_next = live ? __ldg(sb) : 0.f;
    };
    if (pair < p.num_units) enter(pair);
    for (int u = pair; ok && u < p.num_units; u += num_pairs) {
      float sum[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int t = 0; t < 32; ++t) sum[c][t] = 0.f;
      for (int kb = 0; kb < p.k_blocks; ++kb, ++cnt) {
        const uint32_t acc = cnt & 1u, use = cnt >> 1;
        const float sc = a_next * b_next;
        if (live && kb + 1 < p.k_blocks) {  // the next K-block's scales, while this one is awaited
          a_next = __ldg(sa + (kb + 1) * p.sa_cs);
          b_next = __ldg(sb + (kb + 1) * p.sb_cs);
        }
        ok = __all_sync(0xffffffffu, poll_phase(&tfull[acc], use & 1u, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * ACC_STRIDE + 128 * half;
        float x[64];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          tmem_ld64(taddr + 64 * c, x);
          if (c == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (!leader)
                arrive_peer(tempty_leader + acc * 8u);
              else
                mbar_arrive(&tempty[acc]);
            }
          }
#pragma unroll
          for (int t = 0; t < 64; ++t) sum[2 * c + t / 32][t % 32] = fmaf(x[t], sc, sum[2 * c + t / 32][t % 32]);
        }
      }
      if (!ok) break;
      const int64_t orow = row, ocol = col;
      if (u + num_pairs < p.num_units) enter(u + num_pairs);
      constexpr int VE = 16 / sizeof(TC), BOX = 128 / sizeof(TC);  // values of 16 bytes, of a box's row
      // Staged 32 rows x 128 bytes at a time (128-byte swizzle). TMA stores a box where C's rows start on
      // 16-byte boundaries; it leaves out what lies beyond C, but only in steps of 16 bytes along a
      // row, so that a ragged end takes the other way: a row at a time, its values by adjacent lanes.
      const bool tma = p.wide && (ocol + 128 <= p.N || p.N % VE == 0);
      const int64_t row0 = orow - lane;
      const int rows = static_cast<int>(max(int64_t(0), min(int64_t(32), p.M - row0)));
#pragma unroll
      for (int bx = 0; bx < 128 / BOX; ++bx, ++ocnt) {
        uint8_t* buf = obuf + (ocnt & 1u) * EPI_BUF_BYTES;
        if (lane == 0) {
          if (tma)
            bulk_wait_read<1>();  // the store of the box before last has read this buffer
          else
            bulk_wait_read<0>();
        }
        __syncwarp();
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          __align__(16) TC y[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) y[e] = from_f32<TC>(sum[(BOX * bx + VE * v) / 32][(BOX * bx + VE * v) % 32 + e]);
          *reinterpret_cast<uint4*>(buf + lane * 128 + (v ^ (lane & 7)) * 16) = *reinterpret_cast<const uint4*>(y);
        }
        const int64_t c0 = ocol + BOX * bx;
        if (tma) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (row0 < p.M && c0 < p.N) tma_store_2d(&p.tmC, buf, static_cast<int>(c0), static_cast<int>(row0));
            bulk_commit();
          }
        } else {
          __syncwarp();
          TC* out = static_cast<TC*>(p.c) + row0 * p.ldc + c0;
#pragma unroll
          for (int h = 0; h < BOX / 32; ++h) {
            const int e = 32 * h + lane;
            if (c0 + e < p.N) {
#pragma unroll 4
              for (int r = 0; r < rows; ++r)
                out[r * p.ldc + e] = *reinterpret_cast<const TC*>(buf + r * 128 + ((e / VE) ^ (r & 7)) * 16 +
                                                                  (e % VE) * sizeof(TC));
            }
          }
          __syncwarp();  // read before the buffer is staged again
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the leader's MMAs into this CTA's TMEM are done
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

}  // namespace fckl
