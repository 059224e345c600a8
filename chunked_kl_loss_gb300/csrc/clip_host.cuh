// Host side of the gradients' norm (clip.cuh): argument checks, the tables of tensors and the C entry
// points declared in include/fckl.h. Part of the translation unit of fckl.cu.
#pragma once

#include "clip.cuh"
#include "score_host.cuh"

namespace fckl {
namespace {

constexpr int CLIP_CAP_SMALL = 32, CLIP_CAP = 896;  // tensors of a launch; the larger table takes 26 KB of arguments
constexpr int64_t CLIP_COUNT_MAX = 1 << 20;

struct ClipList {
  const void* const* in;
  void* const* out;  // NULL: the norm alone
  const int64_t* n;
  const int* types;
  const int* out_types;
  int count;
};

size_t clip_workspace(int64_t count) {
  return STATUS_WS_BYTES + size_t(std::max<int64_t>(1, cdiv(count, CLIP_CAP))) * CLIP_BLOCKS * sizeof(double);
}

// Whether a tensor that is written overlaps another one's input or output (its own input apart). Inputs
// that are only read may overlap each other.
bool clip_overlaps(const ClipList& l) {
  struct Span {
    uintptr_t a, b;
    bool written;
  };
  std::vector<Span> v;
  v.reserve(2 * size_t(l.count));
  bool sorted = true;
  auto add = [&](const void* p, int64_t bytes, bool written) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (!v.empty() && v.back().a > a) sorted = false;
    v.push_back({a, a + uintptr_t(bytes), written});
  };
  for (int i = 0; i < l.count; ++i)
    if (l.n[i]) add(l.out[i], l.n[i] * int64_t(value_bytes(l.out_types[i])), true);
  for (int i = 0; i < l.count; ++i)
    if (l.n[i] && l.in[i] != l.out[i]) add(l.in[i], l.n[i] * int64_t(value_bytes(l.types[i])), false);
  if (!sorted) std::sort(v.begin(), v.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t written_to = 0, any_to = 0;  // where the spans so far end
  for (const Span& x : v) {
    if (x.a < (x.written ? any_to : written_to)) return true;
    if (x.written) written_to = std::max(written_to, x.b);
    any_to = std::max(any_to, x.b);
  }
  return false;
}

int clip_checks(const ClipList& l) {
  if (l.count < 0) return FCKL_ERR_ARG;
  if (l.count > CLIP_COUNT_MAX) return FCKL_ERR_UNSUPPORTED;
  if (l.count && (!l.in || !l.n || !l.types)) return FCKL_ERR_ARG;
  int64_t units = 0;
  for (int i = 0; i < l.count; ++i) {
    if (l.n[i] < 0 || !known_dtype(l.types[i])) return FCKL_ERR_ARG;
    if (l.n[i] > (int64_t(1) << 40) || (units += l.n[i] / CLIP_UNIT + 2) > INT_MAX) return FCKL_ERR_UNSUPPORTED;
    if (l.n[i] && (!l.in[i] || !aligned(l.in[i], value_bytes(l.types[i])))) return FCKL_ERR_ARG;
    if (l.out) {
      if (!known_dtype(l.out_types[i])) return FCKL_ERR_ARG;
      if (l.n[i] && (!l.out[i] || !aligned(l.out[i], value_bytes(l.out_types[i])))) return FCKL_ERR_ARG;
      if (l.in[i] == l.out[i] && l.types[i] != l.out_types[i] && l.n[i]) return FCKL_ERR_ARG;
    }
  }
  if (l.out && clip_overlaps(l)) return FCKL_ERR_ARG;
  return FCKL_OK;
}

// Tensors [i0, i0 + taken) of the list as a table; returns `taken`.
template <int CAP>
int fill_table(ClipTable<CAP>& t, const ClipList& l, int i0) {
  t.count = 0;
  int64_t units = 0;
  int i = i0;
  for (; i < l.count && t.count < CAP; ++i) {
    if (!l.n[i]) continue;
    const int64_t mis = int64_t((reinterpret_cast<uintptr_t>(l.in[i]) & 15u) / value_bytes(l.types[i]));
    const int64_t more = cdiv(l.n[i] + mis, CLIP_UNIT);
    t.first[t.count] = static_cast<int>(units);
    t.in[t.count] = l.in[i];
    t.out[t.count] = l.out ? l.out[i] : nullptr;
    t.n[t.count] = l.n[i];
    t.type[t.count] = static_cast<uint8_t>(l.types[i] | (l.out ? l.out_types[i] << 4 : 0));
    units += more;
    ++t.count;
  }
  t.first[t.count] = static_cast<int>(units);
  t.units = static_cast<int>(units);
  return i - i0;
}

int clip_grid(const DevInfo* di, int units) {
  return std::max(1, std::min({units, CLIP_BLOCKS, di->sms * 4}));
}

template <int CAP>
int run_clip(DevInfo* di, const ClipList& l, float max_norm, float* norm, unsigned* status, double* partial,
             cudaStream_t s) {
  static thread_local ClipTable<CAP> t;
  int partials = 0, launches = 0;
  for (int i = 0; i < l.count || launches == 0; ++launches) {
    i += fill_table(t, l, i);
    const int grid = clip_grid(di, t.units);
    double* at = partial + partials;
    unsigned* st0 = launches ? nullptr : status;
    int st = launch(KIND_SQUARES, s, "gradient_squares",
                    [&] { squares_kernel<CAP><<<grid, CLIP_THREADS, 0, s>>>(t, at, st0); });
    if (st) return st;
    partials += grid;
  }
  if (!l.out)
    return launch_after(KIND_NORM, s, "gradient_norm", 1, CLIP_THREADS, 0, norm_kernel,
                        static_cast<const double*>(partial), partials, norm);
  for (int i = 0, n = 0; i < l.count || n == 0; ++n) {
    if (launches > 1) i += fill_table(t, l, i);  // of one table: it is still there
    else i = l.count;
    const int grid = clip_grid(di, t.units);
    float* to = n ? nullptr : norm;
    int st = launch_after(KIND_CLIP, s, "clip_gradients", static_cast<unsigned>(grid), CLIP_THREADS, 0, clip_kernel<CAP>, t,
                          static_cast<const double*>(partial), partials, max_norm, to);
    if (st) return st;
  }
  return FCKL_OK;
}

int clip_entry(const ClipList& l, float max_norm, float* norm, void* ws, size_t ws_bytes, void* stream) {
  int st = clip_checks(l);
  if (st) return st;
  if (!norm || !aligned(norm, 4) || !ws || !aligned(ws, 256)) return FCKL_ERR_ARG;
  if (ws_bytes < clip_workspace(l.count)) return FCKL_ERR_WORKSPACE;
  DevInfo* di = nullptr;
  if ((st = device_info(&di))) return st;
  unsigned* status = static_cast<unsigned*>(ws);
  double* partial = reinterpret_cast<double*>(static_cast<uint8_t*>(ws) + STATUS_WS_BYTES);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (l.count <= CLIP_CAP_SMALL) return run_clip<CLIP_CAP_SMALL>(di, l, max_norm, norm, status, partial, s);
  return run_clip<CLIP_CAP>(di, l, max_norm, norm, status, partial, s);
}

}  // namespace
}  // namespace fckl

extern "C" {

size_t fckl_gradient_norm_workspace_bytes(int64_t count) {
  return count < 0 || count > fckl::CLIP_COUNT_MAX ? 0 : fckl::clip_workspace(count);
}

int fckl_gradient_norm(const void* const* grads, const int64_t* sizes, const int* dtypes, int count, float* norm,
                       void* ws, size_t ws_bytes, void* stream) {
  return fckl::guarded("fckl_gradient_norm", [&]() -> int {
    return fckl::clip_entry({grads, nullptr, sizes, dtypes, nullptr, count}, 0.f, norm, ws, ws_bytes, stream);
  });
}

int fckl_clip_gradients(const void* const* grads, const int64_t* sizes, const int* dtypes, int count, float max_norm,
                        void* const* out, const int* out_dtypes, float* norm, void* ws, size_t ws_bytes,
                        void* stream) {
  return fckl::guarded("fckl_clip_gradients", [&]() -> int {
    if (!(max_norm >= 0.f) || (count > 0 && (!out || !out_dtypes))) return FCKL_ERR_ARG;
    static void* const no_out[1] = {nullptr};  // an empty list is still one that is written
    return fckl::clip_entry({grads, count > 0 ? out : no_out, sizes, dtypes, out_dtypes, count}, max_norm, norm, ws,
                            ws_bytes, stream);
  });
}

}  // extern "C"
