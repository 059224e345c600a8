// Host side of the logit rules (adjust.cuh): argument checks, launch shapes and the C entry points
// declared in include/fckl.h. Part of the translation unit of fckl.cu.
#pragma once

#include "adjust.cuh"
#include "score_host.cuh"

namespace fckl {
namespace {

int adjust_checks(const void* x, int dt, int64_t ld, const AdjustParams& p, int64_t N) {
  if (N < 0 || p.V < 1 || p.L < 0 || p.B < 0 || ld < p.V || p.ld_out < p.V || p.ld_h < p.L || !known_dtype(dt))
    return FCKL_ERR_ARG;
  if (p.V > (1 << 30) || N > (int64_t(1) << 40) || ld > (int64_t(1) << 40) || p.ld_out > (int64_t(1) << 40) ||
      p.ld_h > (int64_t(1) << 40) || p.ld_allowed > (int64_t(1) << 40))
    return FCKL_ERR_UNSUPPORTED;
  if (p.L > ADJUST_HISTORY_MAX || p.B > TOKENS_MAX) return FCKL_ERR_UNSUPPORTED;
  if (p.allowed && p.ld_allowed != 0 && p.ld_allowed < cdiv(p.V, 32)) return FCKL_ERR_ARG;
  if (N == 0) return FCKL_OK;
  if (!x || !p.out || !aligned(x, value_bytes(dt)) || !aligned(p.out, value_bytes(dt))) return FCKL_ERR_ARG;
  if (p.L > 0 && (!p.history || !aligned(p.history, 4))) return FCKL_ERR_ARG;
  if (p.B > 0 && (!p.bias_tokens || !p.bias)) return FCKL_ERR_ARG;
  if (!aligned(p.bias_tokens, 4) || !aligned(p.bias, 4) || !aligned(p.allowed, 4) || !aligned(p.lengths, 4) ||
      !aligned(p.prompt, 4) || !aligned(p.r, 4) || !aligned(p.f, 4) || !aligned(p.p, 4))
    return FCKL_ERR_ARG;
  if (x == p.out && ld != p.ld_out) return FCKL_ERR_ARG;
  return FCKL_OK;
}

template <typename T, int VE, AdjustKind KIND, bool IN_PLACE, bool STAGED>
int launch_adjust_kernel(DevInfo* di, AdjustParams p, int64_t N, cudaStream_t s) {
  constexpr bool GRAD = KIND == ADJUST_GRAD;
  const AdjustPlan plan = adjust_plan<VE, KIND, STAGED>(di->sms, N, p.V, p.L, p.B, !IN_PLACE);
  if (!plan.threads) return FCKL_ERR_UNSUPPORTED;
  p.segs = plan.segs;
  p.seg_vecs = plan.seg_vecs;
  p.stages = plan.stages;
  p.slots_log2 = plan.slots_log2;
  void (*k)(AdjustParams);
  if constexpr (STAGED)
    k = plan.threads == ADJUST_STAGED_FEW ? adjust_staged_kernel<T, KIND, ADJUST_STAGED_FEW>
                                          : adjust_staged_kernel<T, KIND, ADJUST_STAGED_THREADS>;
  else
    k = adjust_kernel<T, VE, KIND, IN_PLACE>;
  {
    static bool done[64][2] = {};
    bool& set = done[di->id][plan.threads == ADJUST_STAGED_FEW];
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!set) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(ADJUST_SMEM));
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(adjust)", e);
        return FCKL_ERR_CUDA;
      }
      set = true;
    }
  }
  const int64_t rows_max = INT_MAX / p.segs;  // rows of one launch
  for (int64_t r0 = 0; r0 < N; r0 += rows_max) {
    const int64_t rows = std::min(rows_max, N - r0);
    AdjustParams q = p;
    q.z = static_cast<const T*>(p.z) + r0 * p.ld_z;
    if (GRAD) q.g = static_cast<const T*>(p.g) + r0 * p.ld_g;
    q.out = static_cast<T*>(p.out) + r0 * p.ld_out;
    q.history = p.history + r0 * p.ld_h;
    if (p.lengths) q.lengths = p.lengths + r0;
    if (p.prompt) q.prompt = p.prompt + r0;
    if (p.r) q.r = p.r + r0;
    if (p.f) q.f = p.f + r0;
    if (p.p) q.p = p.p + r0;
    q.bias_tokens = p.bias_tokens + r0 * p.B;
    q.bias = p.bias + r0 * p.B;
    if (p.allowed) q.allowed = p.allowed + r0 * p.ld_allowed;
    const unsigned grid = static_cast<unsigned>(rows * p.segs);
    int st = launch(GRAD ? KIND_ADJUST_GRAD : KIND_ADJUST, s, GRAD ? "adjust_logits_grad" : "adjust_logits",
                    [&] { k<<<grid, plan.threads, plan.smem, s>>>(q); });
    if (st) return st;
  }
  return FCKL_OK;
}

// Through shared memory where every row of the input and of the output lies alike to the 16-byte boundaries;
// in place too if there is a mask (2000 x 50000 bf16 with 2% masked, 1000 history entries and 8 biases: 97 us,
// 1024 x 50000 fp32 with 0.4% left: 78; writing the masked places for themselves, without reading the others,
// took 111 and 72). Without a history those 2000 rows take 63 us (floor 62), with 1024 entries anywhere in the
// row and a frequency penalty 105 (floor 63): the gathering, as into a new tensor (63 and 106). Rows that lie
// differently go value by value: 4096 rows of 50257 out of 50304 bf16 into a dense tensor, 1024 history entries,
// 16 biases and a mask, 456 us; into rows that lie alike 260 (floor 129); fp32 476 and 323 (252).
template <typename T, AdjustKind KIND>
int launch_adjust(DevInfo* di, const AdjustParams& p, int64_t N, cudaStream_t s) {
  constexpr bool GRAD = KIND == ADJUST_GRAD;
  constexpr AdjustKind FULL = GRAD ? ADJUST_GRAD : ADJUST_COUNTS;
  const void* x = GRAD ? p.g : p.z;
  const int64_t ld = GRAD ? p.ld_g : p.ld_z;
  constexpr int VE = 16 / sizeof(T);
  if (x == p.out && !p.allowed) return launch_adjust_kernel<T, VE, FULL, true, false>(di, p, N, s);
  const bool alike = (reinterpret_cast<uintptr_t>(x) & 15u) == (reinterpret_cast<uintptr_t>(p.out) & 15u) &&
                     (N == 1 || (ld - p.ld_out) % VE == 0);
  if (alike) return launch_adjust_kernel<T, VE, KIND, false, true>(di, p, N, s);
  return launch_adjust_kernel<T, 1, FULL, false, false>(di, p, N, s);
}

template <AdjustKind KIND>
int launch_adjust_type(DevInfo* di, int dt, const AdjustParams& p, int64_t N, cudaStream_t s) {
  if (dt == FCKL_BF16) return launch_adjust<__nv_bfloat16, KIND>(di, p, N, s);
  if (dt == FCKL_F16) return launch_adjust<__half, KIND>(di, p, N, s);
  return launch_adjust<float, KIND>(di, p, N, s);
}

}  // namespace
}  // namespace fckl

extern "C" {

int fckl_adjust_logits(const void* logits, int dtype, int64_t ld, int64_t N, int V, const int32_t* history, int64_t ld_h,
                       int L, const int32_t* lengths, const int32_t* prompt, const float* repetition,
                       float repetition_all, const float* frequency, float frequency_all, const float* presence,
                       float presence_all, const int32_t* bias_tokens, const float* bias, int B,
                       const uint32_t* allowed, int64_t ld_allowed, void* out, int64_t ld_out, void* ws,
                       size_t ws_bytes, void* stream) {
  return guarded("fckl_adjust_logits", [&]() -> int {
    AdjustParams p{};
    p.z = logits;
    p.out = out;
    p.ld_z = ld;
    p.ld_out = ld_out;
    p.history = history;
    p.ld_h = ld_h;
    p.L = L;
    p.lengths = lengths;
    p.prompt = prompt;
    p.r = repetition;
    p.f = frequency;
    p.p = presence;
    p.r1 = repetition_all;
    p.f1 = frequency_all;
    p.p1 = presence_all;
    p.bias_tokens = bias_tokens;
    p.bias = bias;
    p.B = B;
    p.allowed = allowed;
    p.ld_allowed = ld_allowed;
    p.V = V;
    p.status = static_cast<unsigned*>(ws);
    int st = adjust_checks(logits, dtype, ld, p, N);
    if (st) return st;
    if (!repetition && !(repetition_all > 0.f)) return FCKL_ERR_ARG;
    if ((st = status_ws_checks(ws, ws_bytes))) return st;
    if (N == 0) return FCKL_OK;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool counts = frequency || presence || frequency_all != 0.f || presence_all != 0.f || B > 0;
    return counts ? launch_adjust_type<ADJUST_COUNTS>(di, dtype, p, N, s) : launch_adjust_type<ADJUST_SEEN>(di, dtype, p, N, s);
  });
}

int fckl_adjust_logits_backward(const void* g, int dtype, int64_t ld_g, const void* logits, int64_t ld, int64_t N, int V,
                                const int32_t* history, int64_t ld_h, int L, const int32_t* lengths,
                                const float* repetition, float repetition_all, const uint32_t* allowed,
                                int64_t ld_allowed, void* out, int64_t ld_out, void* ws, size_t ws_bytes,
                                void* stream) {
  return guarded("fckl_adjust_logits_backward", [&]() -> int {
    AdjustParams p{};
    p.z = logits;
    p.g = g;
    p.out = out;
    p.ld_z = ld;
    p.ld_g = ld_g;
    p.ld_out = ld_out;
    p.history = history;
    p.ld_h = ld_h;
    p.L = L;
    p.lengths = lengths;
    p.r = repetition;
    p.r1 = repetition_all;
    p.allowed = allowed;
    p.ld_allowed = ld_allowed;
    p.V = V;
    p.status = static_cast<unsigned*>(ws);
    int st = adjust_checks(g, dtype, ld_g, p, N);
    if (st) return st;
    if (ld < V || (!repetition && !(repetition_all > 0.f))) return FCKL_ERR_ARG;
    if (ld > (int64_t(1) << 40)) return FCKL_ERR_UNSUPPORTED;
    if ((st = status_ws_checks(ws, ws_bytes))) return st;
    if (N == 0) return FCKL_OK;
    if (!logits || !aligned(logits, value_bytes(dtype))) return FCKL_ERR_ARG;
    if (logits == out && ld != ld_out) return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    return launch_adjust_type<ADJUST_GRAD>(di, dtype, p, N, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
