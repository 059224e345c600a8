// Scoring of given tokens straight from hidden states: the logits z = H W^T live in TMEM only.
//
// head_score_kernel is the logits product of tc_gemm.cuh (persistent, one CTA per SM, SM pairs,
// TMA ring, two TMEM accumulators; K-major operands) with two epilogues of its own:
//   HEAD_STATS : per row and 256-column tile the statistics (m, l, t) of score.cuh, and the logits
//                of the row's given tokens
//   HEAD_GRAD  : G = sum_t g_t [v = t] - q_v (sum_t g_t + g_e (log q_v + entropy)) from the row's
//                log-partition, rounded to bf16 and stored with TMA into the chunk's gradient
//                slab, which the dH and dW products read. As in the loss, G is rounded to bf16
//                because the tensor cores take both operands in one type (half a step, 2^-8 of
//                each entry, independent over the V or N entries that a product sums). A few
//                entries, those at the given tokens, are most of a gradient, and their rounding
//                alone would double its error: with up to REST_TOKENS tokens what the rounding
//                left of them is kept in fp32 and added to dH and dW (dh_rest_kernel, dw_rest_kernel).
// Bound by the tensor cores at large d: 2048 x 2880 x 65536 takes 392 us (1.97 PFLOP/s, tensor pipe 90%
// busy) with HEAD_STATS and 411 us (86%) with HEAD_GRAD; below d of about 1000 by the epilogue, whose
// exponentials alone are 2048 cycles per 128 x 256 tile and SM (2048 x 512 x 128256: 191 us and 223,
// 141 at the tensor rate).
#pragma once

#include <cfloat>

#include "score.cuh"
#include "tc_gemm.cuh"

namespace fckl {

enum { HEAD_STATS = 0, HEAD_GRAD = 1 };

// Up to this many tokens per position are compared with every tile's columns as they are; more are
// ordered first (token_order_kernel), and a cursor walks them. Ordering is a launch of 6 us, the
// comparisons are hidden behind the product.
constexpr int DIRECT_TOKENS = 2;

constexpr int REST_TOKENS = 8;

__device__ __forceinline__ float rounding_left(float v) { return v - __bfloat162float(__float2bfloat16_rn(v)); }

struct HeadParams {
  CUtensorMap tmA;  // H rows of the chunk
  CUtensorMap tmB;  // W
  CUtensorMap tmC;  // gradient slab (HEAD_GRAD)
  Sched sch;
  int num_units;
  int a_3d, b_3d;  // one copy fetches a stage's two K-blocks
  unsigned* status;
  int rows, V, T;
  const int32_t* tokens;  // [rows][T] as given, for T <= DIRECT_TOKENS
  const float* g_logp;    // [rows][T] (HEAD_GRAD)
  const int* sid;         // else: [rows][T] tokens of the chunk, ascending per row
  const int* sslot;       // [rows][T] the slot each came from
  // HEAD_STATS
  float* pm;  // [tiles][ld_part]
  float* pl;
  float* pt;
  int ld_part;
  float* zt;  // [rows][T] logits of the tokens, by slot
  // HEAD_GRAD
  const float* sgrad;  // [rows][T] upstream gradients in the order of sid
  const float* gsum;   // [rows] their sum
  const float* lse;
  const float* entropy;
  const float* g_entropy;  // or null
  float* rest;             // or null; [rows][T] by slot: what the rounding of G left of its entry at a token
};

// Eight epilogue warps, two per TMEM lane quarter (the loss's product has four): each takes 128 of a
// tile's columns, a statistics tile of its own. With four, one per scheduler, nothing hid a warp's
// latencies and the epilogue outlasted the product below d of about 1000.
constexpr int HEAD_EPI_WARPS = 8;
constexpr int HEAD_THREADS = 64 + 32 * HEAD_EPI_WARPS;
constexpr int HEAD_COLS = VOCAB_TILE / 2;  // columns of a warp, and of a statistics tile
static_assert(HEAD_EPI_WARPS * EPI_BUF_BYTES == EPI_WARPS * 2 * EPI_BUF_BYTES, "one staging box per warp");

template <int EPI, bool TF32>
__global__ void __launch_bounds__(HEAD_THREADS, 1) head_score_kernel(const __grid_constant__ HeadParams p) {
  constexpr int CGS = 2, BN = VOCAB_TILE, BN_CTA = BN / CGS;
  constexpr int KPS = TF32 ? 1 : 2;
  using L = TcSmem<CGS, BN, KPS>;
  constexpr int NST = L::STAGES;
  constexpr int KE = TF32 ? BK / 2 : BK;  // K elements per K-block (128 bytes of each row)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t* empty = full + NST;
  uint64_t* tfull = empty + NST;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair = blockIdx.x / CGS;
  const int num_pairs = gridDim.x / CGS;

  if (threadIdx.x == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], HEAD_EPI_WARPS * CGS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tmA);
    prefetch_tmap(&p.tmB);
    if (EPI == HEAD_GRAD) prefetch_tmap(&p.tmC);
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

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer (each CTA)
    if (lane == 0) {
      uint32_t cnt = 0, armed = 0, armed_par = 0;
      bool ok = true;
      const uint32_t full_base = mapa_shared(smem_u32(full), 0);
      for (int u = pair; ok && u < p.num_units; u += num_pairs) {
        int mb, nb, sp, kb0, kb1;
        decode_unit(p.sch, u, mb, nb, sp, kb0, kb1);
        const int arow = (mb * CGS + static_cast<int>(rank)) * BM;
        const int brow = nb * BN + static_cast<int>(rank) * BN_CTA;
        for (int kb = kb0; kb < kb1; kb += KPS, ++cnt) {
          const uint32_t s = cnt % NST, ph = (cnt / NST) & 1u;
          if (!wait_phase(&empty[s], ph ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&full[s], CGS * L::STAGE_BYTES);
            armed |= 1u << s;
            armed_par = (armed_par & ~(1u << s)) | (ph << s);
          }
          uint8_t* a = smem + s * L::STAGE_BYTES;
          uint8_t* b = a + L::A_BYTES;
          const uint32_t fb = full_base + s * 8u;
          if (!TF32 && p.a_3d) {
            tma_load_3d_pair(a, &p.tmA, fb, 0, arow, kb);
          } else {
#pragma unroll
            for (int j = 0; j < KPS; ++j) tma_load_2d_pair(a + j * L::A_KB, &p.tmA, fb, (kb + j) * KE, arow);
          }
          if (!TF32 && p.b_3d) {
            tma_load_3d_pair(b, &p.tmB, fb, 0, brow, kb);
          } else {
#pragma unroll
            for (int j = 0; j < KPS; ++j) tma_load_2d_pair(b + j * L::B_KB, &p.tmB, fb, (kb + j) * KE, brow);
          }
        }
      }
      // every copy this pair started lands before a CTA may exit (see tc_gemm.cuh)
      if (leader) {
        for (int s = 0; s < NST; ++s)
          if (armed & (1u << s)) drain_phase(&full[s], (armed_par >> s) & 1u, p.status);
      } else if (!ok) {
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000ull) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t IDESC =
          TF32 ? make_idesc_tf32(BM * CGS, BN) : make_idesc_bf16(BM * CGS, BN, false, false);
      uint32_t cnt = 0, it = 0;
      bool ok = true;
      for (int u = pair; ok && u < p.num_units; u += num_pairs, ++it) {
        int mb, nb, sp, kb0, kb1;
        decode_unit(p.sch, u, mb, nb, sp, kb0, kb1);
        const uint32_t acc = it & 1u, use = it >> 1;
        if (!wait_phase_cluster(&tempty[acc], (use & 1u) ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * ACC_STRIDE;
        for (int kb = kb0; kb < kb1; kb += KPS, ++cnt) {
          const uint32_t s = cnt % NST, ph = (cnt / NST) & 1u;
          if (!wait_phase(&full[s], ph, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + s * L::STAGE_BYTES);
          const uint32_t b_addr = a_addr + L::A_BYTES;
#pragma unroll
          for (int q = 0; q < KPS * (BK / 16); ++q) {
            const int j = q / (BK / 16), kk = q % (BK / 16);
            if (KPS > 1 && kb + j >= kb1) break;
            const uint64_t ad = make_sdesc_sw128(a_addr + j * L::A_KB + kk * 32, 16, 1024);
            const uint64_t bd = make_sdesc_sw128(b_addr + j * L::B_KB + kk * 32, 16, 1024);
            const uint32_t accum = (kb > kb0 || q > 0) ? 1u : 0u;
            if constexpr (TF32)
              umma_tf32_pair(d_tmem, ad, bd, IDESC, accum);
            else
              umma_bf16_pair(d_tmem, ad, bd, IDESC, accum);
          }
          umma_commit_pair(&empty[s], 0x3);
        }
        if (!ok) break;
        umma_commit_pair(&tfull[acc], 0x3);
      }
      umma_commit_pair(drain, 0x1);  // all MMAs finish before TMEM is released
      drain_phase(drain, 0, p.status);
    }
  } else {
    // ------------------------------------------------------------ epilogue (each CTA)
    const int q = warp & 3;  // TMEM lane quarter this warp may access
    const int half = (warp - 2) / 4;  // columns [HEAD_COLS half, + HEAD_COLS) of a tile
    uint8_t* buf = smem + L::EPI_OFF + (warp - 2) * EPI_BUF_BYTES;
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty), 0);
    auto release_acc = [&](uint32_t acc) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (!leader)
          mbar_arrive_cluster(tempty_leader + acc * 8u);
        else
          mbar_arrive(&tempty[acc]);
      }
    };
    uint32_t it = 0;
    bool stored = false;
    for (int u = pair; u < p.num_units; u += num_pairs, ++it) {
      int mb, nb, sp, kb0, kb1;
      decode_unit(p.sch, u, mb, nb, sp, kb0, kb1);
      const uint32_t acc = it & 1u, use = it >> 1;
      const uint32_t taddr = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + acc * ACC_STRIDE + half * HEAD_COLS;
      const int row0 = (mb * CGS + static_cast<int>(rank)) * BM + 32 * q;  // first row of this warp
      const int row = row0 + lane;
      const bool valid = row < p.rows;
      const int v0 = nb * BN + half * HEAD_COLS;  // this warp's first column; may lie past V
      const size_t tk = static_cast<size_t>(valid ? row : 0) * p.T;
      const bool direct = p.T <= DIRECT_TOKENS;
      // few tokens: each one's place in this tile, or -1, and its gradient
      int rel[DIRECT_TOKENS];
      float gt[DIRECT_TOKENS], gsum = 0.f;
      // more: a cursor over the row's ordered tokens, at the first one of this tile (empty slots,
      // -1, sort before every tile)
      const int* ids = p.sid + tk;
      int k = p.T, nxt = INT_MAX;
      if (direct) {
#pragma unroll
        for (int q = 0; q < DIRECT_TOKENS; ++q) {
          const int id = valid && q < p.T ? __ldg(p.tokens + tk + q) : -1;
          const bool in = id >= 0 && id < p.V;
          if (v0 == 0 && !in && id != -1) atomicOr(p.status, ST_BAD_INDEX);
          rel[q] = in && id >= v0 && id < v0 + HEAD_COLS ? id - v0 : -1;
          if constexpr (EPI == HEAD_GRAD) {
            gt[q] = in ? __ldg(p.g_logp + tk + q) : 0.f;
            gsum += gt[q];
          }
        }
      } else if (valid) {
        k = lower_bound_ids(ids, p.T, v0);
        nxt = k < p.T ? __ldg(ids + k) : INT_MAX;
        if constexpr (EPI == HEAD_GRAD) gsum = __ldg(p.gsum + row);
      }
      if constexpr (EPI == HEAD_STATS) {
        if (!warp_wait_phase(&tfull[acc], use & 1u, abort_flag, p.status)) break;
        tc_fence_after();
        FastStat s[2];  // two sets of sums, for their latency; one maximum
#pragma unroll 1
        for (int j = 0; j < HEAD_COLS / 32; ++j) {
          float x[32];
          __syncwarp();
          tmem_ld32(taddr + 32 * j, x);
          if (j == HEAD_COLS / 32 - 1) release_acc(acc);
          const int cb = v0 + 32 * j;
          if (direct) {
#pragma unroll
            for (int t = 0; t < DIRECT_TOKENS; ++t)
              if (rel[t] >> 5 == j) p.zt[tk + t] = pick32(x, rel[t] & 31);
          }
          while (nxt < cb + 32) {  // nxt < V or INT_MAX: ids past the vocabulary were put last
            p.zt[tk + __ldg(p.sslot + tk + k)] = pick32(x, nxt - cb);
            ++k;
            nxt = k < p.T ? __ldg(ids + k) : INT_MAX;
          }
          if (cb + 32 > p.V) {
#pragma unroll
            for (int t = 0; t < 32; ++t)
              if (cb + t >= p.V) x[t] = -FLT_MAX;  // not above any finite logit, and no 0 * -inf
          }
          const float cm = max32(x);
          if (cm > s[0].m) {
            s[0].raise(cm);
            s[1].raise(cm);
          }
#pragma unroll
          for (int t = 0; t < 32; t += 4) {
            s[0].add(x[t], x[t + 1]);
            s[1].add(x[t + 2], x[t + 3]);
          }
        }
        if (valid && v0 < p.V) {
          const RowStat a = s[0].stat(), b = s[1].stat();  // of the same maximum
          const size_t o = static_cast<size_t>(2 * nb + half) * p.ld_part + row;
          p.pm[o] = a.m;
          p.pl[o] = a.l + b.l;
          p.pt[o] = a.t + b.t;
        }
      } else {
        const float ge = valid && p.g_entropy ? __ldg(p.g_entropy + row) : 0.f;
        const float lse = valid ? __ldg(p.lse + row) : 0.f;
        const float ent = valid ? __ldg(p.entropy + row) : 0.f;
        const float a0 = ge == 0.f ? gsum : fmaf(ge, ent, gsum);  // left out where it plays no part
        const float nge = -2.f * ge, nlse = -0.5f * lse;
        if (!warp_wait_phase(&tfull[acc], use & 1u, abort_flag, p.status)) break;
        tc_fence_after();
#pragma unroll 1
        for (int jj = 0; jj < HEAD_COLS / 64; ++jj) {
          if (stored && lane == 0) bulk_wait_read<0>();
          __syncwarp();
          stored = true;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int j = 2 * jj + h;
            float x[32];
            __syncwarp();
            tmem_ld32(taddr + 32 * j, x);
            if (j == HEAD_COLS / 32 - 1) release_acc(acc);
            const int cb = v0 + 32 * j;
#pragma unroll
            for (int t = 0; t < 32; t += 2) {
              // -q (a0 + ge log q) as (-2 ge q) (log q / 2) - a0 q: half the difference of two finite numbers
              // is finite, and where q is 0 each product is 0
              const unsigned long long hq = fma2(pack2(x[t], x[t + 1]), pack2(0.5f, 0.5f), pack2(nlse, nlse));
              float y0, y1;
              unpack2f(mul2(hq, pack2(2.f * LOG2E, 2.f * LOG2E)), y0, y1);
              const unsigned long long q = pack2(ex2_approx(y0), ex2_approx(y1));
              unpack2f(fma2(mul2(q, pack2(nge, nge)), hq, mul2(q, pack2(-a0, -a0))), x[t], x[t + 1]);
            }
            if (direct) {
#pragma unroll
              for (int t = 0; t < DIRECT_TOKENS; ++t)
                if (rel[t] >> 5 == j) sub32(x, rel[t] & 31, -gt[t]);
#pragma unroll
              for (int t = 0; t < DIRECT_TOKENS; ++t)
                if (rel[t] >> 5 == j && p.rest) {
                  bool first = true;  // a repeated token's entry counts once
#pragma unroll
                  for (int o = 0; o < t; ++o) first &= rel[o] != rel[t];
                  p.rest[tk + t] = first ? rounding_left(pick32(x, rel[t] & 31)) : 0.f;
                }
            }
            while (nxt < cb + 32) {
              const int id = nxt;
              sub32(x, id - cb, -__ldg(p.sgrad + tk + k));
              nxt = k + 1 < p.T ? __ldg(ids + k + 1) : INT_MAX;
              if (p.rest) p.rest[tk + __ldg(p.sslot + tk + k)] = nxt == id ? 0.f : rounding_left(pick32(x, id - cb));
              ++k;
            }
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
              uint4 w;
              w.x = pack_bf16x2(x[8 * cc + 0], x[8 * cc + 1]);
              w.y = pack_bf16x2(x[8 * cc + 2], x[8 * cc + 3]);
              w.z = pack_bf16x2(x[8 * cc + 4], x[8 * cc + 5]);
              w.w = pack_bf16x2(x[8 * cc + 6], x[8 * cc + 7]);
              const int chunk16 = (4 * h + cc) ^ (lane & 7);
              *reinterpret_cast<uint4*>(buf + lane * 128 + chunk16 * 16) = w;
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int sx = v0 + 64 * jj;
            if (sx < p.V && row0 < p.rows) tma_store_2d(&p.tmC, buf, sx, row0);
            bulk_commit();
          }
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

// One warp per position: the row's tokens in ascending order (by id, then slot) with the slot and
// the upstream gradient of each, and the sum of the gradients. An id outside [0, V), -1 aside,
// is reported and put last, where no tile reaches it, without a gradient.
__global__ void __launch_bounds__(32 * PRE_WARPS) token_order_kernel(
    const int32_t* __restrict__ tokens, const float* __restrict__ g, int rows, int T, int V, int* __restrict__ sid,
    int* __restrict__ sslot, float* __restrict__ sgrad, float* __restrict__ gsum, unsigned* __restrict__ status) {
  extern __shared__ int order_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x * PRE_WARPS + warp;
  if (row >= rows) return;  // warp-uniform; no block barrier below
  int* ids = order_smem + warp * T;
  const size_t o = static_cast<size_t>(row) * T;
  int bad = 0;
  for (int t = lane; t < T; t += 32) {
    int i = tokens[o + t];
    if (i < -1 || i >= V) {
      bad = 1;
      i = INT_MAX;
    }
    ids[t] = i;
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, ST_BAD_INDEX);
  __syncwarp();
  float s = 0.f;
  for (int t = lane; t < T; t += 32) {
    const int key = ids[t];
    int r = 0;
    for (int j = 0; j < T; ++j) {
      const int i = ids[j];
      r += (i < key) | ((i == key) & (j < t));
    }
    sid[o + r] = key;
    sslot[o + r] = t;
    if (g) {
      const float gt = key >= 0 && key != INT_MAX ? g[o + t] : 0.f;
      sgrad[o + r] = gt;
      s += gt;
    }
  }
  if (g) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane == 0) gsum[row] = s;
  }
}

// dH of a chunk: the K-splits' partials and the tokens' rests, rest_t W[t], summed in fp32 in a fixed
// order. Four columns per thread.
template <typename TO>
__global__ void __launch_bounds__(256) dh_rest_kernel(const float* __restrict__ partial, int splits, int64_t stride,
                                                      int rows, int d, const int32_t* __restrict__ tokens,
                                                      const float* __restrict__ rest, int T, int V,
                                                      const __nv_bfloat16* __restrict__ W, TO* __restrict__ out) {
  const int64_t n4 = static_cast<int64_t>(rows) * (d / 4);
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n4; i += gridDim.x * 256ll) {
    const int64_t row = i / (d / 4);
    const int c = static_cast<int>(i - row * (d / 4)) * 4;
    float4 a = *reinterpret_cast<const float4*>(partial + row * d + c);
    for (int s = 1; s < splits; ++s) {
      const float4 b = *reinterpret_cast<const float4*>(partial + s * stride + row * d + c);
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    for (int t = 0; t < T; ++t) {
      const int id = __ldg(tokens + row * T + t);
      if (id < 0 || id >= V) continue;
      const float g = __ldg(rest + row * T + t);
      const uint2 w = __ldg(reinterpret_cast<const uint2*>(W + static_cast<int64_t>(id) * d + c));
      float w0, w1, w2, w3;
      unpack2(w.x, w0, w1, __nv_bfloat16{});
      unpack2(w.y, w2, w3, __nv_bfloat16{});
      a.x = fmaf(g, w0, a.x), a.y = fmaf(g, w1, a.y), a.z = fmaf(g, w2, a.z), a.w = fmaf(g, w3, a.w);
    }
    TO* o = out + row * d + c;
    if constexpr (sizeof(TO) == 4) {
      *reinterpret_cast<float4*>(o) = a;
    } else {
      uint2 v;
      v.x = pack_bf16x2(a.x, a.y);
      v.y = pack_bf16x2(a.z, a.w);
      *reinterpret_cast<uint2*>(o) = v;
    }
  }
}

// dW rounded to bf16, four values per thread and step: runs on a second stream beside the last chunk's
// dH product, which leaves most of HBM's bandwidth free.
__global__ void __launch_bounds__(256) dw_round_kernel(const float4* __restrict__ dW, uint2* __restrict__ out,
                                                       int64_t n4) {
  constexpr int B = 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i0 = blockIdx.x * 256ll + threadIdx.x; i0 < n4; i0 += B * step) {
    float4 v[B];
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (i0 + b * step < n4) v[b] = __ldcs(dW + i0 + b * step);
#pragma unroll
    for (int b = 0; b < B; ++b)
      if (i0 + b * step < n4)
        out[i0 + b * step] = make_uint2(pack_bf16x2(v[b].x, v[b].y), pack_bf16x2(v[b].z, v[b].w));
  }
}

// dW[id] += sum of rest h over a window of a chunk's entries (position, slot) with that token, in order.
// A block per entry looks through the window's tokens: the first entries with an id share that row's
// columns, REST_COLS at a time, and each adds up all of the id's entries in them, so that every element
// of dW has one writer; the others leave. (Sorting the entries first, in one block, took 25 us for 2048
// of them; this takes 12.) 2048 x 2880 entries of different tokens take 26 us, of one token 104 us
// (with one block for all of an id: 24 and 1930).
constexpr int REST_WINDOW = 4096;
constexpr int REST_THREADS = 256;
__global__ void __launch_bounds__(REST_THREADS) dw_rest_kernel(const int32_t* __restrict__ tokens,
                                                               const float* __restrict__ rest, int first, int entries,
                                                               int T, int V, const __nv_bfloat16* __restrict__ H,
                                                               int d, float* __restrict__ dW) {
  constexpr int PER = REST_WINDOW / REST_THREADS;
  constexpr int REST_COLS = 2 * REST_THREADS;
  __shared__ int2 list[REST_WINDOW];  // position and rest of the id's entries
  __shared__ int wsum[REST_THREADS / 32];
  __shared__ int rank_s;
  const int own = first + blockIdx.x;  // entries of the window: [first, entries)
  const int id = tokens[own];
  if (id < 0 || id >= V) return;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t hit = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = first + tid * PER + j;
    if (e < entries && __ldg(tokens + e) == id) hit |= 1u << j;
  }
  int at = __popc(hit);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += v;
  }
  if (lane == 31) wsum[warp] = at;
  __syncthreads();
  int n = 0;
  at -= __popc(hit);
#pragma unroll
  for (int w = 0; w < REST_THREADS / 32; ++w) {
    if (w < warp) at += wsum[w];
    n += wsum[w];
  }
  if (tid == (own - first) / PER) rank_s = at + __popc(hit & ((1u << (own - first) % PER) - 1u));
  __syncthreads();
  const int rank = rank_s, share = min(n, (d + REST_COLS - 1) / REST_COLS);
  if (rank >= share) return;
  while (hit) {
    const int e = first + tid * PER + __ffs(hit) - 1;
    list[at++] = make_int2(e / T, __float_as_int(__ldg(rest + e)));
    hit &= hit - 1;
  }
  __syncthreads();
  for (int c = rank * REST_COLS + tid * 2; c < d; c += share * REST_COLS) {
    float* o = dW + static_cast<int64_t>(id) * d + c;
    float2 a = *reinterpret_cast<const float2*>(o);
#pragma unroll 16
    for (int i = 0; i < n; ++i) {
      const int2 e = list[i];
      const float g = __int_as_float(e.y);
      float h0, h1;
      unpack2(__ldg(reinterpret_cast<const uint32_t*>(H + static_cast<int64_t>(e.x) * d + c)), h0, h1, __nv_bfloat16{});
      a.x = fmaf(g, h0, a.x);
      a.y = fmaf(g, h1, a.y);
    }
    *reinterpret_cast<float2*>(o) = a;
  }
}

// Merges the tiles' statistics of R positions per block into the log-partition, the entropy and the
// tokens' log-probabilities (logp holds the tokens' logits on entry). 1024 / R threads share a
// position's tiles. R = 32 reads whole lines; with few positions R = 4 keeps more of a position's loads
// in flight (786 tiles of one position: 16 us with R = 32, 10 with R = 4). The order of the merges is
// one, so that a position's result does not depend on how many share its chunk: tile t goes to part
// t mod 256, in ascending order, and the parts are merged in halves. A thread holds 256 R / 1024 parts
// (2048 positions of 1571 tiles: 20 us, 18 with parts of its own order).
constexpr int COMBINE_THREADS = 1024;
constexpr int COMBINE_PARTS = 256;
template <int R>
__global__ void __launch_bounds__(COMBINE_THREADS) head_combine_kernel(
    const float* __restrict__ pm, const float* __restrict__ pl, const float* __restrict__ pt, int ld, int tiles,
    int rows, const int32_t* __restrict__ tokens, int T, int V, float* __restrict__ logp,
    float* __restrict__ entropy, float* __restrict__ lse) {
  constexpr int STEP = COMBINE_THREADS / R;      // threads of a position
  constexpr int OWN = COMBINE_PARTS / STEP;      // parts of a thread: STEP apart
  __shared__ RowStat part[COMBINE_THREADS];
  __shared__ float rm[R], rs[R];
  const int tid = threadIdx.x;
  const int row0 = blockIdx.x * R, row = row0 + tid % R;
  RowStat own[OWN];
  if (row < rows) {
    constexpr int B = 8;  // the loads of 8 tiles are issued before any of them is merged
    static_assert(B % OWN == 0, "whole rounds of the parts");
    for (int t0 = tid / R; t0 < tiles; t0 += STEP * B) {
      RowStat x[B];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int t = t0 + STEP * b;
        if (t < tiles) {
          const size_t o = static_cast<size_t>(t) * ld + row;
          x[b].m = pm[o];
          x[b].l = pl[o];
          x[b].t = pt[o];
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) own[b % OWN] = merge(own[b % OWN], x[b]);
    }
  }
#pragma unroll
  for (int h = OWN / 2; h > 0; h /= 2) {
#pragma unroll
    for (int b = 0; b < h; ++b) own[b] = merge(own[b], own[b + h]);
  }
  RowStat s = own[0];
  part[tid] = s;
  for (int o = COMBINE_THREADS / 2; o >= R; o >>= 1) {
    __syncthreads();
    if (tid < o) part[tid] = merge(part[tid], part[tid + o]);
  }
  if (tid < R) {
    s = part[tid];
    const float log_s = logf(s.l);
    rm[tid] = s.m;
    rs[tid] = log_s;
    if (row < rows) {
      const float e = log_s - s.t / s.l;
      entropy[row] = e < 0.f ? 0.f : e;
      lse[row] = s.m + log_s;
    }
  }
  __syncthreads();
  const int n = min(R, rows - row0) * T;
  const size_t o = static_cast<size_t>(row0) * T;
  for (int i = tid; i < n; i += COMBINE_THREADS) {
    const int id = tokens[o + i], r = i / T;
    float lp = 0.f;
    if (id < -1 || id >= V)
      lp = NAN;
    else if (id >= 0)
      lp = (logp[o + i] - rm[r]) - rs[r];
    logp[o + i] = lp;
  }
}

}  // namespace fckl
