// Host side of the scoring from hidden states (score_gemm.cuh): workspace, chunk loop and the C
// entry points declared in include/fckl.h. Part of the translation unit of fckl.cu; the gradient
// products are the loss's own (chunk_products).
#pragma once

#include "score_gemm.cuh"
#include "score_host.cuh"
#include "skinny.cuh"

namespace fckl {
namespace {

// A chunk of fewer positions is copied to this many rows, zeros after it, before the product: with
// fewer than 24 rows behind the tensor map every SM fetches the same few lines again and again, and
// the product takes 235 to 300 us where it takes 200 with 24 and more (2880 x 201088).
constexpr int HEAD_MIN_ROWS = 32;

int head_shape(int64_t N, int d, int V, int T, int chunk, int dt) {
  if (N < 0 || T < 0) return FCKL_ERR_ARG;
  if (T > TOKENS_MAX) return FCKL_ERR_UNSUPPORTED;
  return check_shape(std::max<int64_t>(N, 1), d, V, 1, chunk, dt);
}

// K-splits (over V) of the dH product: the least estimated time, waves of 256 x 256 tiles over the 76 SM
// pairs at a K-block's 0.34 us each (1900 TFLOP/s) plus the fp32 partials written and read back
// (6.8 TB/s). With chunks of 512 rows at d = 1024 the loss's limit of 4 keeps 32 pairs busy (44 us);
// 9 splits take 28.
constexpr int HEAD_MAX_SPLITS = 16;
int head_splits(int rows, int d, int V) {
  const int64_t kb = cdiv(V, BK), tiles = cdiv(rows, TILE_M) * cdiv(d, 256), pairs = 76;
  int best = 1;
  double least = 1e30;
  for (int sp = 1; sp <= HEAD_MAX_SPLITS && sp <= kb; ++sp) {
    const int64_t per = cdiv(kb, sp);
    if (cdiv(kb, per) != sp) continue;
    const double us = double(cdiv(tiles * sp, pairs)) * double(per) * 0.34 + 8.0 * sp * rows * double(d) / 6.8e6;
    if (us < least) {
      least = us;
      best = sp;
    }
  }
  return best;
}

// The loss's plan with the regions that scoring uses: ordered tokens in sidx, their slots in T
// (rows x T ints), their gradients in sp, the sums of those in S, the tiles' statistics, and for the
// backward pass the gradient slab and dH partials.
Plan head_plan(int64_t N, int d, int V, int T, int chunk, int dt, bool backward) {
  Plan p = make_plan(std::max<int64_t>(N, 1), d, V, 1, chunk, dt);
  p.K = T;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    size_t r = o;
    o = static_cast<size_t>(rup(static_cast<int64_t>(o + bytes), 1024));
    return r;
  };
  const size_t R = p.rows_alloc, D = d;
  p.off_status = take(256);
  p.off_sidx = take(R * T * 4);
  p.off_T = take(R * T * 4);
  p.off_sp = take(backward ? R * T * 4 : 0);
  // rests of the tokens' entries, in pm's place
  const size_t rests = backward && T <= REST_TOKENS ? R * T : 0;
  p.off_S = take(backward ? R * 4 : 0);
  // statistics: of every HEAD_COLS columns and row of a chunk, or of every block of the skinny kernel
  const size_t skinny = N <= SK_MAX_POS ? size_t(std::min<int64_t>(cdiv(V, SK_ROWS), SK_MAX_BLOCKS)) * N : 0;
  const size_t stat = backward ? 0 : std::max(size_t(cdiv(V, HEAD_COLS)) * R, skinny) * 4;
  p.off_pm = take(stat + rests * 4);
  p.off_pl = take(stat);
  p.off_pc = take(stat);
  p.off_G = take(backward ? R * p.ldG * 2 : 0);
  p.off_dhp = take(backward ? std::max(MAX_SPLITS, head_splits(p.chunk, d, V)) * R * D * 4 : 0);
  const bool f32 = dt == FCKL_F32;
  p.off_Hb = take(f32 && backward ? R * D * 2 : 0);
  p.off_Wb = take(f32 && backward ? size_t(V) * D * 2 : 0);
  p.off_Ht = take(f32 ? R * D * 4 : size_t(HEAD_MIN_ROWS) * D * 2);
  p.off_Wt = take(f32 ? size_t(V) * D * 4 : 0);
  p.total = p.total_overlap = o;
  return p;
}

int head_setup(Run& r, const void* H, const void* W, int dt, const int32_t* tokens, int64_t N, int d, int V, int T,
               int chunk, bool backward, void* ws, size_t ws_bytes, void* stream) {
  int st = head_shape(N, d, V, T, chunk, dt);
  if (st) return st;
  if (!ws || !aligned(ws, 256)) return FCKL_ERR_ARG;
  if (N > 0 && (!H || !aligned(H, 16) || (T > 0 && (!tokens || !aligned(tokens, 4))))) return FCKL_ERR_ARG;
  if (!W || !aligned(W, 16)) return FCKL_ERR_ARG;
  r.pl = head_plan(N, d, V, T, chunk, dt, backward);
  if (ws_bytes < r.pl.total) return FCKL_ERR_WORKSPACE;
  r.s = static_cast<cudaStream_t>(stream);
  r.w = static_cast<uint8_t*>(ws);
  r.status = reinterpret_cast<unsigned*>(r.w + r.pl.off_status);
  r.H = H;
  r.Wraw = W;
  r.Wb = W;
  r.dtype = dt;
  r.idx = tokens;
  return FCKL_OK;
}

// Orders the chunk's tokens and returns its hidden states as the products read them (as
// chunk_prepare does for the loss).
int head_prepare(Run& r, int64_t r0, int rows, const float* g, const void** Hl, const void** Hc, bool backward) {
  const Plan& pl = r.pl;
  const int T = pl.K;
  int st;
  if (T > DIRECT_TOKENS) {
    const unsigned blocks = static_cast<unsigned>(cdiv(rows, PRE_WARPS));
    cudaStream_t s = r.s;
    uint8_t* w = r.w;
    unsigned* status = r.status;
    const int32_t* tok = r.idx + r0 * T;
    st = launch(KIND_TOKEN_ORDER, s, "token_order", [&] {
      token_order_kernel<<<blocks, 32 * PRE_WARPS, size_t(PRE_WARPS) * T * 4, s>>>(
          tok, g, rows, T, pl.V, reinterpret_cast<int*>(w + pl.off_sidx), reinterpret_cast<int*>(w + pl.off_T),
          reinterpret_cast<float*>(w + pl.off_sp), reinterpret_cast<float*>(w + pl.off_S), status);
    });
    if (st) return st;
  }
  const size_t esz = r.dtype == FCKL_F32 ? 4 : 2;
  *Hl = static_cast<const uint8_t*>(r.H) + static_cast<size_t>(r0) * pl.d * esz;
  *Hc = *Hl;
  if (r.dtype == FCKL_F32) {
    if ((st = launch_cvt(static_cast<const float*>(*Hl), r.w + pl.off_Ht, backward ? r.w + pl.off_Hb : nullptr,
                         int64_t(rows) * pl.d, r.di, r.s)))
      return st;
    *Hl = r.w + pl.off_Ht;
    *Hc = r.w + pl.off_Hb;
  } else if (rows < HEAD_MIN_ROWS) {
    uint8_t* pad = r.w + pl.off_Ht;
    const size_t have = size_t(rows) * pl.d * 2, all = size_t(HEAD_MIN_ROWS) * pl.d * 2;
    cudaError_t e = cudaMemcpyAsync(pad, *Hl, have, cudaMemcpyDeviceToDevice, r.s);
    if (e == cudaSuccess) e = cudaMemsetAsync(pad + have, 0, all - have, r.s);
    if (e != cudaSuccess) {
      set_error("short chunk", e);
      return FCKL_ERR_CUDA;
    }
    *Hl = pad;
  }
  return FCKL_OK;
}

// Adds the rests of a chunk's tokens to dW.
int launch_dw_rest(Run& r, const int32_t* tokens, const float* rest, int rows, const __nv_bfloat16* Hc) {
  const int T = r.pl.K, d = r.pl.d, V = r.pl.V, entries = rows * T;
  cudaStream_t s = r.s;
  float* dW = r.dW;
  for (int first = 0; first < entries; first += REST_WINDOW) {
    const int end = std::min(entries, first + REST_WINDOW);
    int st = launch(KIND_DW_REST, s, "dw_rest", [&] {
      dw_rest_kernel<<<static_cast<unsigned>(end - first), REST_THREADS, 0, s>>>(tokens, rest, first, end, T, V, Hc, d,
                                                                                  dW);
    });
    if (st) return st;
  }
  return FCKL_OK;
}

// Rounds dW to bf16 on the caller's stream or, with side, on the side stream after what the caller's
// holds so far; the caller then joins with `side->join`.
int launch_dw_round(Run& r, SideStream* side, void* out) {
  const int64_t n4 = int64_t(r.pl.V) * r.pl.d / 4;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(cdiv(n4, 1024), int64_t(r.di->sms) * (side ? 4 : 8)));
  const float4* dW = reinterpret_cast<const float4*>(r.dW);
  uint2* to = static_cast<uint2*>(out);
  if (!side) {
    cudaStream_t s = r.s;
    return launch(KIND_DW_ROUND, s, "dw_round", [&] { dw_round_kernel<<<grid, 256, 0, s>>>(dW, to, n4); });
  }
  static bool done[64] = {};
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!done[r.di->id]) {  // the product's shared-memory split, so that both run on an SM
      cudaError_t e = cudaFuncSetAttribute(dw_round_kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                                           cudaSharedmemCarveoutMaxShared);
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(dw_round)", e);
        return FCKL_ERR_CUDA;
      }
      done[r.di->id] = true;
    }
  }
  cudaError_t e = cudaEventRecord(side->fork, r.s);
  if (e == cudaSuccess) e = cudaStreamWaitEvent(side->s, side->fork, 0);
  if (e != cudaSuccess) {
    set_error("fork to the side stream", e);
    return FCKL_ERR_CUDA;
  }
  cudaStream_t s = side->s;
  const int st = launch(KIND_DW_ROUND, s, "dw_round", [&] { dw_round_kernel<<<grid, 256, 0, s>>>(dW, to, n4); });
  e = cudaEventRecord(side->join, s);  // whatever failed: nothing of the call stays outside its stream
  if (e != cudaSuccess && !st) {
    set_error("join from the side stream", e);
    return FCKL_ERR_CUDA;
  }
  return st;
}

// Persistent launch of one instance: as many SM pairs as can be resident, capped by the units.
template <int EPI, bool TF32>
int launch_head(int kind, DevInfo* di, const HeadParams& p, cudaStream_t s, const char* what) {
  auto k = head_score_kernel<EPI, TF32>;
  constexpr uint32_t smem = TcSmem<2, VOCAB_TILE, TF32 ? 1 : 2>::DYN_BYTES;
  static int max_pairs[64] = {};
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(HEAD_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int pairs;
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!max_pairs[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(head_score)", e);
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
  return launch(kind, s, what, [&] { cudaLaunchKernelEx(&cfg, k, p); });
}

// One block per 32 positions, or per 4 where that leaves most SMs without one.
int launch_head_combine(const float* pm, const float* pl, const float* pt, int ld, int tiles, int rows,
                        const int32_t* tokens, int T, int V, float* logp, float* entropy, float* lse,
                        cudaStream_t s) {
  return launch(KIND_HEAD_COMBINE, s, "head_combine", [&] {
    if (rows > 512)
      head_combine_kernel<32><<<static_cast<unsigned>(cdiv(rows, 32)), COMBINE_THREADS, 0, s>>>(
          pm, pl, pt, ld, tiles, rows, tokens, T, V, logp, entropy, lse);
    else
      head_combine_kernel<4><<<static_cast<unsigned>(cdiv(rows, 4)), COMBINE_THREADS, 0, s>>>(
          pm, pl, pt, ld, tiles, rows, tokens, T, V, logp, entropy, lse);
  });
}

// Few positions, few tokens each, and hidden states that fit beside two steps' partial sums.
size_t skinny_smem(int NG, int d, int64_t N, int T) {
  return size_t(8 * NG) * skinny_pitch(d * 2) + size_t(2) * SK_WARPS * SK_ROWS * 8 * NG * 4 + size_t(N) * T * 4;
}
bool head_is_skinny(const Run& r, int64_t N, int d, int T) {
  return r.dtype == FCKL_BF16 && N <= SK_MAX_POS && T <= SK_MAX_TOKENS &&
         skinny_smem(static_cast<int>(cdiv(N, 8)), d, N, T) <= SK_SMEM_MAX;
}

template <int NG>
int launch_head_skinny(DevInfo* di, HeadSkinnyParams p, cudaStream_t s, int* blocks) {
  auto k = head_skinny_kernel<NG>;
  const size_t smem = skinny_smem(NG, p.d, p.N, p.T);
  static bool done[64] = {};
  {
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!done[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SK_SMEM_MAX);
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(head_skinny)", e);
        return FCKL_ERR_CUDA;
      }
      done[di->id] = true;
    }
  }
  p.tiles = static_cast<int>(cdiv(p.V, SK_ROWS));
  *blocks = std::min({p.tiles, 2 * di->sms, SK_MAX_BLOCKS});
  const unsigned grid = static_cast<unsigned>(*blocks);
  return launch(KIND_HEAD_SKINNY, s, "head_skinny", [&] { k<<<grid, SK_THREADS, smem, s>>>(p); });
}

// What both passes over a chunk's logits share.
int head_params(Run& r, const void* Hl, int rows, HeadParams* p) {
  const Plan& pl = r.pl;
  memset(p, 0, sizeof(*p));
  int st = map_logits_A(r, &p->tmA, Hl, std::max(rows, r.dtype == FCKL_BF16 ? HEAD_MIN_ROWS : 1), &p->a_3d);
  if (st) return st;
  p->tmB = r.tmW_k;
  p->b_3d = r.w_k_3d;
  const int kb = logits_kblocks(r);
  p->sch = {static_cast<int>(cdiv(rows, TILE_M)), pl.tiles_v, kb, 1, kb, 1};
  p->num_units = p->sch.m_blocks * p->sch.n_blocks;
  p->status = r.status;
  p->rows = rows;
  p->V = pl.V;
  p->T = pl.K;
  p->sid = reinterpret_cast<const int*>(r.w + pl.off_sidx);
  p->sslot = reinterpret_cast<const int*>(r.w + pl.off_T);
  return FCKL_OK;
}

}  // namespace
}  // namespace fckl

extern "C" {

size_t fckl_projected_logprobs_workspace_bytes(int64_t N, int d, int V, int T, int chunk, int dtype, int backward) {
  if (head_shape(N, d, V, T, chunk, dtype) != FCKL_OK) return 0;
  return head_plan(N, d, V, T, chunk, dtype, backward != 0).total;
}

int fckl_projected_logprobs(const void* H, const void* W, int dtype, const int32_t* tokens, int64_t N, int d, int V,
                            int T, int chunk, float* logp, float* entropy, float* lse, void* ws, size_t ws_bytes,
                            void* stream) {
  return guarded("fckl_projected_logprobs", [&]() -> int {
    Run r;
    int st = head_setup(r, H, W, dtype, tokens, N, d, V, T, chunk, false, ws, ws_bytes, stream);
    if (st) return st;
    if (N > 0 && (!entropy || !lse || (T > 0 && !logp))) return FCKL_ERR_ARG;
    if (!aligned(logp, 4) || !aligned(entropy, 4) || !aligned(lse, 4)) return FCKL_ERR_ARG;
    if ((st = device_info(&r.di))) return st;
    if (N == 0) return cudaMemsetAsync(r.status, 0, 4, r.s) == cudaSuccess ? FCKL_OK : FCKL_ERR_CUDA;
    if ((st = run_begin(r, false))) return st;
    const Plan& pl = r.pl;
    cudaStream_t s = r.s;
    if (head_is_skinny(r, N, d, T)) {
      HeadSkinnyParams p{};
      p.H = static_cast<const __nv_bfloat16*>(H);
      p.W = static_cast<const __nv_bfloat16*>(W);
      p.tokens = tokens;
      p.N = static_cast<int>(N);
      p.d = d;
      p.V = V;
      p.T = T;
      p.pm = reinterpret_cast<float*>(r.w + pl.off_pm);
      p.pl = reinterpret_cast<float*>(r.w + pl.off_pl);
      p.pt = reinterpret_cast<float*>(r.w + pl.off_pc);
      p.ld = p.N;
      p.zt = logp;
      p.status = r.status;
      int blocks = 0;
      switch (cdiv(N, 8)) {
        case 1: st = launch_head_skinny<1>(r.di, p, s, &blocks); break;
        default: st = launch_head_skinny<2>(r.di, p, s, &blocks); break;
      }
      if (st) return st;
      return launch_head_combine(p.pm, p.pl, p.pt, p.ld, blocks, p.N, tokens, T, V, logp, entropy, lse, s);
    }
    for (int64_t r0 = 0; r0 < N; r0 += pl.chunk) {
      const int rows = static_cast<int>(std::min<int64_t>(pl.chunk, N - r0));
      const void *Hl = nullptr, *Hc = nullptr;
      if ((st = head_prepare(r, r0, rows, nullptr, &Hl, &Hc, false))) return st;
      HeadParams p;
      if ((st = head_params(r, Hl, rows, &p))) return st;
      p.pm = reinterpret_cast<float*>(r.w + pl.off_pm);
      p.pl = reinterpret_cast<float*>(r.w + pl.off_pl);
      p.pt = reinterpret_cast<float*>(r.w + pl.off_pc);
      p.ld_part = pl.rows_alloc;
      p.tokens = tokens + r0 * T;
      p.zt = logp + r0 * T;
      st = dtype == FCKL_F32 ? launch_head<HEAD_STATS, true>(KIND_HEAD_LOGITS, r.di, p, s, "head_logits_stats")
                             : launch_head<HEAD_STATS, false>(KIND_HEAD_LOGITS, r.di, p, s, "head_logits_stats");
      if (st) return st;
      st = launch_head_combine(p.pm, p.pl, p.pt, p.ld_part, static_cast<int>(cdiv(V, HEAD_COLS)), rows, tokens + r0 * T, T, V, p.zt,
                               entropy + r0, lse + r0, s);
      if (st) return st;
    }
    return FCKL_OK;
  });
}

int fckl_projected_logprobs_backward(const void* H, const void* W, int dtype, const int32_t* tokens, int64_t N, int d,
                                     int V, int T, int chunk, const float* lse, const float* entropy,
                                     const float* g_logp, const float* g_entropy, void* dH, float* dW,
                                     void* dW_bf16, void* ws, size_t ws_bytes, void* stream) {
  return guarded("fckl_projected_logprobs_backward", [&]() -> int {
    Run r;
    int st = head_setup(r, H, W, dtype, tokens, N, d, V, T, chunk, true, ws, ws_bytes, stream);
    if (st) return st;
    if ((!dH && !dW) || !aligned(dW, 16) || (dW_bf16 && (!dW || !aligned(dW_bf16, 16)))) return FCKL_ERR_ARG;
    if (N > 0 && (!lse || !entropy || (T > 0 && !g_logp))) return FCKL_ERR_ARG;
    if (!aligned(lse, 4) || !aligned(entropy, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4) || !aligned(dH, 16))
      return FCKL_ERR_ARG;
    if ((st = device_info(&r.di))) return st;
    if (N == 0) {
      cudaError_t e = cudaMemsetAsync(r.status, 0, 4, r.s);
      if (e == cudaSuccess && dW) e = cudaMemsetAsync(dW, 0, size_t(V) * d * 4, r.s);
      if (e == cudaSuccess && dW_bf16) e = cudaMemsetAsync(dW_bf16, 0, size_t(V) * d * 2, r.s);
      if (e == cudaSuccess) return FCKL_OK;
      set_error("cudaMemsetAsync", e);
      return FCKL_ERR_CUDA;
    }
    r.dH = dH;
    r.dW = dW;
    if ((st = run_begin(r, true))) return st;
    const Plan& pl = r.pl;
    if (!std::getenv("FCKL_SPLITS")) r.splits = head_splits(pl.chunk, d, V);
    for (int64_t r0 = 0; r0 < N; r0 += pl.chunk) {
      const int rows = static_cast<int>(std::min<int64_t>(pl.chunk, N - r0));
      const void *Hl = nullptr, *Hc = nullptr;
      if ((st = head_prepare(r, r0, rows, g_logp + r0 * T, &Hl, &Hc, true))) return st;
      HeadParams p;
      if ((st = head_params(r, Hl, rows, &p))) return st;
      if ((st = make_map(&p.tmC, r.w + pl.off_G, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, V, rows, uint64_t(pl.ldG) * 2, 64,
                         32)))
        return st;
      p.tokens = tokens + r0 * T;
      p.g_logp = g_logp + r0 * T;
      p.sgrad = reinterpret_cast<const float*>(r.w + pl.off_sp);
      p.gsum = reinterpret_cast<const float*>(r.w + pl.off_S);
      p.lse = lse + r0;
      p.entropy = entropy + r0;
      p.g_entropy = g_entropy ? g_entropy + r0 : nullptr;
      const bool rest = T > 0 && T <= REST_TOKENS;
      if (rest) {
        p.rest = reinterpret_cast<float*>(r.w + pl.off_pm);
        r.rest = p.rest;
        r.rest_tokens = p.tokens;
      }
      st = dtype == FCKL_F32 ? launch_head<HEAD_GRAD, true>(KIND_HEAD_GRAD, r.di, p, r.s, "head_logit_grad")
                             : launch_head<HEAD_GRAD, false>(KIND_HEAD_GRAD, r.di, p, r.s, "head_logit_grad");
      if (st) return st;
      // dW first, so that its rounding can run beside the last chunk's dH
      Run part = r;
      part.dH = nullptr;
      if (dW && (st = chunk_products(part, 0, r0, rows, Hc))) return st;
      if (rest && dW &&
          (st = launch_dw_rest(r, p.tokens, p.rest, rows, static_cast<const __nv_bfloat16*>(Hc))))
        return st;
      SideStream* side = nullptr;
      if (dW_bf16 && r0 + rows >= N) {
        // beside dH where that is long enough to cover it (as for the loss's side work); at 777 x 1024 x
        // 32000 the rounding alone takes 25 us, beside a dH of 28 us 70
        if (dH && overlap_pays(rows, d, V, false) && (st = side_stream(r.di->id, &side))) return st;
        st = launch_dw_round(r, side, dW_bf16);
      }
      part = r;
      part.dW = nullptr;
      if (!st && dH) st = chunk_products(part, 0, r0, rows, Hc);
      if (side) {
        const int sj = wait_event(r.s, side->join);
        if (!st) st = sj;
      }
      if (st) return st;
    }
    return FCKL_OK;
  });
}

}  // extern "C"
