// Host side of the scoring operators (score.cuh): argument checks, launch shapes and the C
// entry points declared in include/fckl.h. Part of the translation unit of fckl.cu.
#pragma once

#include <new>

#include "score.cuh"

namespace fckl {
namespace {

constexpr size_t STATUS_WS_BYTES = 256;  // workspace that holds only the status word

// Runs a C entry's body: nothing that it throws crosses the C boundary.
template <class F>
int guarded(const char* where, F&& body) noexcept {
  try {
    return body();
  } catch (...) {
    snprintf(g_last_error, sizeof(g_last_error), "%s: out of host memory or a system error", where);
    return FCKL_ERR_CUDA;
  }
}

// Launches a kernel that may begin, up to its wait_for_previous(), while the stream's last kernel ends.
template <class... P, class... A>
int launch_after(int kind, cudaStream_t s, const char* what, unsigned grid, unsigned block, size_t smem, void (*k)(P...),
                 const A&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return launch(kind, s, what, [&] { cudaLaunchKernelEx(&cfg, k, args...); });
}

size_t value_bytes(int dt) { return dt == FCKL_F32 ? 4 : 2; }
bool known_dtype(int dt) { return dt == FCKL_BF16 || dt == FCKL_F32 || dt == FCKL_F16; }

// Shape and pointers of the calls that take logits. `top` is 0 where there are no alternatives.
int score_checks(const void* logits, int dt, int64_t ld, const int32_t* tokens, int64_t N, int V, int T, int top) {
  if (N < 0 || V < 1 || T < 0 || top < 0 || ld < V || !known_dtype(dt)) return FCKL_ERR_ARG;
  if (V > (1 << 30) || N > (int64_t(1) << 40) || ld > (int64_t(1) << 40)) return FCKL_ERR_UNSUPPORTED;
  if (T > TOKENS_MAX || top > TOKENS_MAX || top > V) return FCKL_ERR_UNSUPPORTED;
  if (N == 0) return FCKL_OK;
  if (!logits || !aligned(logits, value_bytes(dt))) return FCKL_ERR_ARG;
  if (T > 0 && (!tokens || !aligned(tokens, 4))) return FCKL_ERR_ARG;
  return FCKL_OK;
}

int status_ws_checks(const void* ws, size_t ws_bytes) {
  if (!ws || !aligned(ws, 256)) return FCKL_ERR_ARG;
  return ws_bytes < STATUS_WS_BYTES ? FCKL_ERR_WORKSPACE : FCKL_OK;
}

template <typename T, int NT, int RING = 0>
int launch_token_logprobs_block(DevInfo* di, ScoreParams p, int64_t N, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int STEP = NT * SCORE_GV;
  const int64_t nvec = cdiv(p.V, VE) + 1;  // one more where rows start off a 16-byte boundary
  // A row goes to a cluster of blocks where rows alone would leave SMs idle, while each block
  // keeps at least half a step of vectors per thread.
  p.split = 1;
  while (p.split < 8 && N * p.split * 2 <= 2 * int64_t(di->sms) && nvec / (2 * p.split) >= STEP / 2) p.split *= 2;
  const int64_t steps = cdiv(cdiv(nvec, p.split), STEP);
  p.gshift = 0;
  while (cdiv(steps, int64_t(1) << p.gshift) > SCORE_MAX_GROUPS / NT) ++p.gshift;
  p.groups = static_cast<int>(cdiv(steps, int64_t(1) << p.gshift)) * NT;
  // twice the alternatives, so that ordinary rows' candidates fit; and the blocks' sets together
  p.cand_cap = 512;
  while (p.cand_cap < 2 * p.top || (p.split > 1 && p.cand_cap < p.split * p.top)) p.cand_cap *= 2;
  const size_t ring = size_t(std::min<int64_t>(RING, steps)) * STEP * 16;
  const size_t smem =
      p.top ? size_t(p.groups) * 4 + std::max(ring, size_t(p.cand_cap) * 8 + size_t(p.groups) * 2) : ring;
  constexpr size_t SMEM_MAX =
      SCORE_MAX_GROUPS * 4 + std::max<size_t>(RING * STEP * 16, 8 * TOKENS_MAX * 8 + SCORE_MAX_GROUPS * 2);
  auto k = token_logprobs_kernel<T, NT, RING>;
  {
    static bool done[64] = {};
    std::lock_guard<std::mutex> lk(g_setup_mu);
    if (!done[di->id]) {
      cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(SMEM_MAX));
      if (e != cudaSuccess) {
        set_error("cudaFuncSetAttribute(token_logprobs)", e);
        return FCKL_ERR_CUDA;
      }
      done[di->id] = true;
    }
  }
  const int64_t rows_max = INT_MAX / p.split;  // rows of one launch
  for (int64_t r0 = 0; r0 < N; r0 += rows_max) {
    const int64_t rows = std::min(rows_max, N - r0);
    ScoreParams q = p;
    q.logits = static_cast<const T*>(p.logits) + r0 * p.ld;
    q.tokens = p.tokens + r0 * p.T;
    q.logp = p.logp + r0 * p.T;
    q.entropy = p.entropy + r0;
    q.norm = p.norm + 2 * r0;
    q.top_idx = p.top_idx + r0 * p.top;
    q.top_logp = p.top_logp + r0 * p.top;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.split);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(static_cast<unsigned>(rows * p.split));
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = p.split > 1 ? 1 : 0;
    int st = launch(KIND_TOKEN_LOGPROBS, s, "token_logprobs", [&] { cudaLaunchKernelEx(&cfg, k, q); });
    if (st) return st;
  }
  return FCKL_OK;
}

template <typename T>
int launch_token_logprobs(DevInfo* di, const ScoreParams& p, int64_t N, cudaStream_t s) {
  // Blocks of 128 or 64 threads where there are rows for all SMs and a row is short: more rows are then
  // under way on an SM, and a row's selection keeps fewer warps waiting. 4096 rows, bf16, one alternative,
  // with 256 / 128 / 64 threads: V = 1000 48 / 25 / 18 us, 8000 45 / 30 / 27, 64000 118 / 103 / 121, 128256
  // 191 / 201 / 255; with 100 alternatives 2000 75 / 53 / 95, 32000 108 / 107 / 121. 600 rows: 16000
  // 11.1 / 9.6 / 11.6; 300 rows: 4000 7.3 / 6.6 / 6.8, 16000 8.1 / 8.5 / 10.5.
  const int64_t nvec = cdiv(p.V, 16 / sizeof(T)) + 1;
  const bool few = p.top <= 64;
  int64_t longest = 0;  // row, in vectors, for 128 threads
  if (N > 4 * int64_t(di->sms)) longest = few ? 8192 : 4096;
  else if (2 * N > 5 * int64_t(di->sms)) longest = few ? 4096 : 1024;
  else if (N > di->sms && few) longest = 1024;
  if (2 * N > 5 * int64_t(di->sms) && few && nvec <= 512) return launch_token_logprobs_block<T, 64>(di, p, N, s);
  if (p.top <= 128 && nvec <= longest) return launch_token_logprobs_block<T, 128>(di, p, N, s);
  // fp32 rows through the ring in shared memory where an SM has work for several blocks after each other,
  // or fewer blocks than fit; its three blocks an SM instead of four otherwise cost a wave (one
  // alternative, without / with: 2048 x 128256 202 / 178 us, 4096 x 50001 155 / 141, 300 x 201088 53 / 45;
  // 600 x 128256 60 / 75, 1000 x 201088 142 / 149).
  if constexpr (sizeof(T) == 4) {
    if ((N >= 8 * int64_t(di->sms) && nvec >= 12000) || (N > di->sms && N <= 3 * int64_t(di->sms) && nvec >= 25000))
      return launch_token_logprobs_block<T, SCORE_THREADS, 2>(di, p, N, s);
  }
  return launch_token_logprobs_block<T, SCORE_THREADS>(di, p, N, s);
}

template <typename T, int NT>
int launch_token_logprobs_grad_block(DevInfo* di, ScoreGradParams p, int64_t N, cudaStream_t s) {
  constexpr int VE = 16 / sizeof(T), STEP = NT * SCORE_GRAD_VECS;
  // Segments of at most STEP vectors; up to twice as many where that fills the last wave
  // of blocks better (301 x 50001 fp16: 4 segments a row leave 0.4 of a second wave idle, 17.5 us;
  // 5 segments, 12.5).
  const int least = static_cast<int>(cdiv(cdiv(p.V, VE) + 1, STEP));
  const int64_t slots = int64_t(di->sms) * (SCORE_GRAD_RESIDENT * SCORE_THREADS / NT);
  double best = 0.0;
  for (int segs = least; segs <= 2 * least; ++segs) {
    const int64_t blocks = N * segs;
    const double fill = double(blocks) / double(cdiv(blocks, slots) * slots);
    if (fill > 1.02 * best) {
      best = fill;
      p.segs = segs;
    }
  }
  const int64_t rows_max = INT_MAX / p.segs;
  for (int64_t r0 = 0; r0 < N; r0 += rows_max) {
    const int64_t rows = std::min(rows_max, N - r0);
    ScoreGradParams q = p;
    q.logits = static_cast<const T*>(p.logits) + r0 * p.ld;
    q.dlogits = static_cast<T*>(p.dlogits) + r0 * p.ld_out;
    q.tokens = p.tokens + r0 * p.T;
    q.g_logp = p.g_logp + r0 * p.T;
    q.norm = p.norm + 2 * r0;
    q.entropy = p.entropy + r0;
    if (p.g_entropy) q.g_entropy = p.g_entropy + r0;
    const unsigned grid = static_cast<unsigned>(rows * p.segs);
    int st = launch(KIND_TOKEN_LOGPROBS_GRAD, s, "token_logprobs_grad",
                    [&] { token_logprobs_grad_kernel<T, NT><<<grid, NT, 0, s>>>(q); });
    if (st) return st;
  }
  return FCKL_OK;
}

template <typename T>
int launch_token_logprobs_grad(DevInfo* di, const ScoreGradParams& p, int64_t N, cudaStream_t s) {
  // Blocks of 128 threads but for long rows: 4096 rows, bf16, with 256 / 128 / 64 threads: V = 1000
  // 28 / 9.5 / 9.8 us, 8000 46 / 27 / 27, 64000 174 / 173 / 195, 128256 344 / 377 / 382.
  constexpr int SMALL = 128;
  if (p.T <= SMALL * SCORE_GRAD_TOKENS && cdiv(p.V, 16 / sizeof(T)) + 1 <= 8192)
    return launch_token_logprobs_grad_block<T, SMALL>(di, p, N, s);
  return launch_token_logprobs_grad_block<T, SCORE_THREADS>(di, p, N, s);
}

}  // namespace
}  // namespace fckl

extern "C" {

int fckl_token_logprobs(const void* logits, int dtype, int64_t ld, const int32_t* tokens, int64_t N, int V, int T,
                        int top, float* logp, float* entropy, float* norm, int32_t* top_idx, float* top_logp,
                        void* ws, size_t ws_bytes, void* stream) {
  return guarded("fckl_token_logprobs", [&]() -> int {
    int st = score_checks(logits, dtype, ld, tokens, N, V, T, top);
    if (st) return st;
    if ((st = status_ws_checks(ws, ws_bytes))) return st;
    if (N == 0) return FCKL_OK;
    if (!entropy || !norm || (T > 0 && !logp) || (top > 0 && (!top_idx || !top_logp))) return FCKL_ERR_ARG;
    if (!aligned(entropy, 4) || !aligned(norm, 4) || !aligned(logp, 4) || !aligned(top_idx, 4) ||
        !aligned(top_logp, 4))
      return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    ScoreParams p{};
    p.logits = logits;
    p.ld = ld;
    p.tokens = tokens;
    p.V = V;
    p.T = T;
    p.top = top;
    p.logp = logp;
    p.entropy = entropy;
    p.norm = norm;
    p.top_idx = top_idx;
    p.top_logp = top_logp;
    p.status = static_cast<unsigned*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FCKL_BF16) return launch_token_logprobs<__nv_bfloat16>(di, p, N, s);
    if (dtype == FCKL_F16) return launch_token_logprobs<__half>(di, p, N, s);
    return launch_token_logprobs<float>(di, p, N, s);
  });
}

int fckl_token_logprobs_backward(const void* logits, int dtype, int64_t ld, const int32_t* tokens, int64_t N, int V,
                                 int T, const float* norm, const float* entropy, const float* g_logp,
                                 const float* g_entropy, void* dlogits, int64_t ld_out, void* ws, size_t ws_bytes,
                                 void* stream) {
  return guarded("fckl_token_logprobs_backward", [&]() -> int {
    int st = score_checks(logits, dtype, ld, tokens, N, V, T, 0);
    if (st) return st;
    if (ld_out < V) return FCKL_ERR_ARG;
    if (ld_out > (int64_t(1) << 40)) return FCKL_ERR_UNSUPPORTED;
    if ((st = status_ws_checks(ws, ws_bytes))) return st;
    if (N == 0) return FCKL_OK;
    if (!norm || !entropy || !dlogits || (T > 0 && !g_logp)) return FCKL_ERR_ARG;
    if (!aligned(norm, 4) || !aligned(entropy, 4) || !aligned(g_logp, 4) || !aligned(g_entropy, 4) ||
        !aligned(dlogits, value_bytes(dtype)))
      return FCKL_ERR_ARG;
    if (logits == dlogits && ld != ld_out) return FCKL_ERR_ARG;
    DevInfo* di = nullptr;
    if ((st = device_info(&di))) return st;
    ScoreGradParams p{};
    p.logits = logits;
    p.ld = ld;
    p.ld_out = ld_out;
    p.tokens = tokens;
    p.V = V;
    p.T = T;
    p.norm = norm;
    p.entropy = entropy;
    p.g_logp = g_logp;
    p.g_entropy = g_entropy;
    p.dlogits = dlogits;
    p.status = static_cast<unsigned*>(ws);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == FCKL_BF16) return launch_token_logprobs_grad<__nv_bfloat16>(di, p, N, s);
    if (dtype == FCKL_F16) return launch_token_logprobs_grad<__half>(di, p, N, s);
    return launch_token_logprobs_grad<float>(di, p, N, s);
  });
}

}  // extern "C"
