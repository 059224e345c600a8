// The norm of a set of gradient tensors, and the tensors scaled to at most a given norm:
//   norm = sqrt(sum over all tensors of sum g^2),   c = min(1, max_norm / (norm + 1e-6)),   out = c g
// The tensors' addresses and sizes travel as kernel arguments (no copy to the device, and a captured
// graph keeps them). Their elements are cut into units of CLIP_UNIT; every block takes a run of units and
// leaves one partial sum, and the scaling kernel's blocks each add the same partial sums in the same
// order, so no block waits for another and the same call gives the same bits.
// Bound by memory: a model's 983 M gradients, 2.5 GB, are read for the norm, read again and written as 2 GB
// in 1071 us, 6.5 TB/s (6.7 is a plain copy), in place in 1149 (6.5 TB/s too); the second reading is what the
// floors of 666 and 744 us do not have, and what lies in L2 (129 MB) is all that can be kept. 32 tensors of
// 8192: 9 us for the two launches.
#pragma once

#include "bulk.cuh"
#include "score.cuh"

namespace fckl {

constexpr int CLIP_THREADS = 256;
constexpr int CLIP_UNIT = 8192;   // elements
constexpr int CLIP_BLOCKS = 1024; // partial sums of one launch at most
constexpr float CLIP_EPS = 1e-6f;

// Tensors of one launch.
template <int CAP>
struct ClipTable {
  int count, units;
  int first[CAP + 1];  // first unit of each tensor
  const void* in[CAP];
  void* out[CAP];
  int64_t n[CAP];
  uint8_t type[CAP];  // fckl_dtype of the input, and of the output << 4
};

template <typename T>
struct alignas(16) Pack16 {
  T v[16 / sizeof(T)];
};

// A tensor seen as 16-byte vectors from the boundary at or below its start: element i is value i + mis.
template <typename T>
__device__ __forceinline__ int misalignment(const void* p) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}

// Sum of squares of one unit's values of this thread. Squares are summed in fp32; where that leaves
// fp32's range (the sum overflows, or its terms are lost below it), or meets a NaN, the same values are
// summed again in fp64.
template <typename T>
__device__ __forceinline__ void unit_squares(const T* x, int64_t n, int mis, int64_t v0, double& sum) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int VECS = CLIP_UNIT / VE / CLIP_THREADS;
  uint4 w[VECS];
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int64_t i = v0 + int64_t(k * CLIP_THREADS + threadIdx.x) * VE - mis;  // first element
    if (i >= 0 && i + VE <= n) {
      w[k] = *reinterpret_cast<const uint4*>(x + i);
    } else {
      Pack16<T> e;
      for (int j = 0; j < VE; ++j) e.v[j] = i + j >= 0 && i + j < n ? x[i + j] : from_f32<T>(0.f);
      w[k] = *reinterpret_cast<const uint4*>(&e);
    }
  }
  float s = 0.f;
  uint32_t some = 0;
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    float f[VE];
    unpack16<T>(w[k], f);
#pragma unroll
    for (int j = 0; j < VE; ++j) s = fmaf(f[j], f[j], s);
    some |= w[k].x | w[k].y | w[k].z | w[k].w;
  }
  if (s >= 0x1p-110f && s < INFINITY) {
    sum += static_cast<double>(s);
  } else if (some) {
#pragma unroll
    for (int k = 0; k < VECS; ++k) {
      float f[VE];
      unpack16<T>(w[k], f);
#pragma unroll
      for (int j = 0; j < VE; ++j) sum = fma(static_cast<double>(f[j]), static_cast<double>(f[j]), sum);
    }
  }
}

__device__ __forceinline__ double block_sum(double v, double* warps) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) warps[threadIdx.x / 32] = v;
  __syncthreads();
  double r = 0.0;
  for (int w = 0; w < CLIP_THREADS / 32; ++w) r += warps[w];
  return r;
}

// The tensor that holds unit u.
template <int CAP>
__device__ __forceinline__ int tensor_of(const ClipTable<CAP>& t, int u) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS)
    squares_kernel(const __grid_constant__ ClipTable<CAP> t, double* partial, unsigned* status) {
  __shared__ double warps[CLIP_THREADS / 32];
  let_next_begin();
  if (status && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  const int per = (t.units + gridDim.x - 1) / gridDim.x;
  const int u0 = static_cast<int>(min(int64_t(blockIdx.x) * per, int64_t(t.units))), u1 = min(u0 + per, t.units);
  double sum = 0.0;
  if (u0 < u1) {
    int k = tensor_of(t, u0);
    for (int u = u0; u < u1; ++u) {
      while (u >= t.first[k + 1]) ++k;
      const int64_t v0 = int64_t(u - t.first[k]) * CLIP_UNIT;
      const int type = t.type[k] & 15;
      if (type == 0) {
        const auto* x = static_cast<const __nv_bfloat16*>(t.in[k]);
        unit_squares(x, t.n[k], misalignment<__nv_bfloat16>(x), v0, sum);
      } else if (type == 2) {
        const auto* x = static_cast<const __half*>(t.in[k]);
        unit_squares(x, t.n[k], misalignment<__half>(x), v0, sum);
      } else {
        const auto* x = static_cast<const float*>(t.in[k]);
        unit_squares(x, t.n[k], misalignment<float>(x), v0, sum);
      }
    }
  }
  const double all = block_sum(sum, warps);
  if (threadIdx.x == 0) partial[blockIdx.x] = all;
}

// The sum of all partial sums, in an order that their number alone sets; every thread gets it.
__device__ __forceinline__ double total_of(const double* partial, int partials, double* warps) {
  double v = 0.0;
  for (int i = threadIdx.x; i < partials; i += CLIP_THREADS) v += partial[i];
  return block_sum(v, warps);
}

__global__ void __launch_bounds__(CLIP_THREADS) norm_kernel(const double* partial, int partials, float* norm) {
  __shared__ double warps[CLIP_THREADS / 32];
  wait_for_previous();
  const double total = total_of(partial, partials, warps);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(total));
}

template <typename T, typename O>
__device__ __forceinline__ void unit_scale(const T* x, O* y, int64_t n, int mis, int64_t v0, float2 c) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int VECS = CLIP_UNIT / VE / CLIP_THREADS;
  struct alignas(VE * sizeof(O) > 16 ? 16 : VE * sizeof(O)) Out {
    O v[VE];
  };
  uint4 w[VECS];
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int64_t i = v0 + int64_t(k * CLIP_THREADS + threadIdx.x) * VE - mis;
    if (i >= 0 && i + VE <= n) {
      w[k] = *reinterpret_cast<const uint4*>(x + i);
    } else {
      Pack16<T> e;
      for (int j = 0; j < VE; ++j) e.v[j] = i + j >= 0 && i + j < n ? x[i + j] : from_f32<T>(0.f);
      w[k] = *reinterpret_cast<const uint4*>(&e);
    }
  }
  // every vector of a tensor has the same alignment in the output
  const bool wide = (reinterpret_cast<uintptr_t>(y) - size_t(mis) * sizeof(O)) % alignof(Out) == 0;
#pragma unroll
  for (int k = 0; k < VECS; ++k) {
    const int64_t i = v0 + int64_t(k * CLIP_THREADS + threadIdx.x) * VE - mis;
    float f[VE];
    unpack16<T>(w[k], f);
    Out o;
#pragma unroll
    for (int j = 0; j < VE; ++j) o.v[j] = from_f32<O>(f[j] * c.x * c.y);
    if (wide && i >= 0 && i + VE <= n) {
      *reinterpret_cast<Out*>(y + i) = o;
    } else {
#pragma unroll
      for (int j = 0; j < VE; ++j)
        if (i + j >= 0 && i + j < n) y[i + j] = o.v[j];
    }
  }
}

template <typename T>
__device__ __forceinline__ void unit_scale_to(const void* in, void* out, int type, int64_t n, int64_t v0, float2 c) {
  const T* x = static_cast<const T*>(in);
  const int mis = misalignment<T>(x);
  if (type == 0) unit_scale(x, static_cast<__nv_bfloat16*>(out), n, mis, v0, c);
  else if (type == 2) unit_scale(x, static_cast<__half*>(out), n, mis, v0, c);
  else unit_scale(x, static_cast<float*>(out), n, mis, v0, c);
}

// Walks its run of units from the end: what the first pass read last may still be in L2 (129 MB). From the
// end / from the start: 192 MB of fp32 in place 92 / 102 us, 96 MB into bf16 43 / 47, 2.5 GB into bf16 1069 / 1075.
template <int CAP>
__global__ void __launch_bounds__(CLIP_THREADS)
    clip_kernel(const __grid_constant__ ClipTable<CAP> t, const double* partial, int partials, float max_norm,
                float* norm) {
  __shared__ double warps[CLIP_THREADS / 32];
  const int per = (t.units + gridDim.x - 1) / gridDim.x;
  const int u0 = static_cast<int>(min(int64_t(blockIdx.x) * per, int64_t(t.units))), u1 = min(u0 + per, t.units);
  int k = u0 < u1 ? tensor_of(t, u1 - 1) : 0;
  wait_for_previous();
  const double total = sqrt(total_of(partial, partials, warps));
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const double ratio = static_cast<double>(max_norm) / (total + static_cast<double>(CLIP_EPS));
  // A NaN stays. A coefficient near or below the smallest normal number, as gradients near the largest
  // have it, is applied in two factors, so that it keeps its digits.
  const double up = ratio < 0x1p-100 ? 0x1p64 : 1.0;
  const float2 c = ratio >= 1.0 ? make_float2(1.f, 1.f)
                                : make_float2(static_cast<float>(ratio * up), static_cast<float>(1.0 / up));
  for (int u = u1 - 1; u >= u0; --u) {
    while (u < t.first[k]) --k;
    if (ratio >= 1.0 && t.in[k] == t.out[k]) continue;
    const int64_t v0 = int64_t(u - t.first[k]) * CLIP_UNIT;
    const int from = t.type[k] & 15, to = t.type[k] >> 4;
    if (from == 0) unit_scale_to<__nv_bfloat16>(t.in[k], t.out[k], to, t.n[k], v0, c);
    else if (from == 2) unit_scale_to<__half>(t.in[k], t.out[k], to, t.n[k], v0, c);
    else unit_scale_to<float>(t.in[k], t.out[k], to, t.n[k], v0, c);
  }
}

}  // namespace fckl
