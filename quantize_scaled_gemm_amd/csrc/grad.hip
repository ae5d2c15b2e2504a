// Global norm of many gradient tensors, and clipping by it.
//
//   S    = sum over tensors and elements of g^2          (binary64)
//   norm = sqrt(S),  k = min(1, max_norm / (norm + 1e-6)),  out = g k
//   (an infinite max_norm: k = 1, whatever the norm)
//
// The tensors are cut into chunks on the host (qsg_grad_plan) and the table
// of chunks lies in device memory, so one launch covers any number of
// tensors.  Squares and sums are binary64: a binary32 square loses gradients
// below 2^-75 and overflows above 2^64, and the conversion and the fma are a
// small part of the time that an element takes to arrive.
//
// Both passes are bound by HBM.  [measured, MI355X, 302 M fp32 gradients] the
// sum reads 1.21 GB in 177 us (6.8 TB/s), the clip reads and writes 2.42 GB in
// 412 us (5.9 TB/s); a 2 GiB device copy moves 4.9-5.1 TB/s.  Chunks of 8192
// elements: 16384 435 us and 32768 439 us for the clip (the last round of
// workgroups is shorter).  Plain instead of non-temporal loads in the sum: 203
// us, and 418 for the clip after them.
#include <float.h>
#include <hip/hip_runtime.h>

#include "qsg.h"
#include "qsg_device.h"
#include "qsg_internal.h"

namespace qsg {

namespace {

constexpr int kSumGroups = QSG_GRAD_WORKSPACE_BYTES / 8;  // workgroups (and partial sums) of a sum, at most

typedef u32x4 u32x4_e __attribute__((aligned(2)));

__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int k = 32; k > 0; k >>= 1) v += __shfl_xor(v, k, 64);
  return v;
}

// sum over a workgroup of 256 threads, in thread 0
__device__ __forceinline__ double block_sum_f64(double v, double* red) {
  v = wave_sum_f64(v);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return ((red[0] + red[1]) + red[2]) + red[3];
}

// 16 bytes of a tensor: 8 bf16 or 4 fp32 values
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float at(u32x4 u, int i) { return (i & 1) ? bf16hi(u[i >> 1]) : bf16lo(u[i >> 1]); }
  static __device__ __forceinline__ u32x4 scaled(u32x4 u, float k) {
    return u32x4{pack_bf16x2(bf16lo(u.x) * k, bf16hi(u.x) * k), pack_bf16x2(bf16lo(u.y) * k, bf16hi(u.y) * k),
                 pack_bf16x2(bf16lo(u.z) * k, bf16hi(u.z) * k), pack_bf16x2(bf16lo(u.w) * k, bf16hi(u.w) * k)};
  }
  static __device__ __forceinline__ float one(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t rounded(float v) { return (uint16_t)pack_bf16x2(v, 0.0f); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float at(u32x4 u, int i) { return __uint_as_float(u[i]); }
  static __device__ __forceinline__ u32x4 scaled(u32x4 u, float k) {
    return u32x4{__float_as_uint(__uint_as_float(u.x) * k), __float_as_uint(__uint_as_float(u.y) * k),
                 __float_as_uint(__uint_as_float(u.z) * k), __float_as_uint(__uint_as_float(u.w) * k)};
  }
  static __device__ __forceinline__ float one(float v) { return v; }
  static __device__ __forceinline__ float rounded(float v) { return v; }
};

constexpr int kFlight = 8;  // 16-byte loads of a thread in flight

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int n) {
  typedef Vec<T> V;
  double s = 0.0;
  const int whole = n / V::N;  // 16-byte pieces
  for (int i0 = threadIdx.x; i0 < whole; i0 += 256 * kFlight) {
    u32x4 u[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      u[k] = u32x4{0, 0, 0, 0};
      if (i0 + k * 256 < whole)
        u[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + (i0 + k * 256) * V::N));
    }
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
#pragma unroll
      for (int i = 0; i < V::N; ++i) {
        const double v = V::at(u[k], i);
        s = fma(v, v, s);
      }
  }
  for (int i = whole * V::N + threadIdx.x; i < n; i += 256) {
    const double v = V::one(g[i]);
    s = fma(v, v, s);
  }
  return s;
}

__global__ __launch_bounds__(256) void grad_sumsq_kernel(const qsg_grad* table, int64_t n, double* partial) {
  __shared__ double red[4];
  double s = 0.0;
  for (int64_t k = blockIdx.x; k < n; k += gridDim.x) {
    const qsg_grad t = table[k];
    s += t.dtype == QSG_BF16 ? chunk_squares(reinterpret_cast<const uint16_t*>(t.g), (int)t.n)
                             : chunk_squares(reinterpret_cast<const float*>(t.g), (int)t.n);
  }
  s = block_sum_f64(s, red);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void grad_sum_kernel(const double* partial, int n, double* sumsq) {
  __shared__ double red[4];
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += 256) s += partial[i];
  s = block_sum_f64(s, red);
  if (threadIdx.x == 0) *sumsq = s;
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* o, int n, float c) {
  typedef Vec<T> V;
  const int whole = n / V::N;
  for (int i0 = threadIdx.x; i0 < whole; i0 += 256 * kFlight) {
    u32x4 u[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i0 + k * 256 < whole)
        u[k] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + (i0 + k * 256) * V::N));
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i0 + k * 256 < whole)
        __builtin_nontemporal_store(V::scaled(u[k], c), reinterpret_cast<u32x4_e*>(o + (i0 + k * 256) * V::N));
  }
  for (int i = whole * V::N + threadIdx.x; i < n; i += 256) o[i] = V::rounded(V::one(g[i]) * c);
}

__global__ __launch_bounds__(256) void grad_clip_kernel(const qsg_grad* table, int64_t n, const double* sumsq,
                                                        float max_norm, float* norm_out) {
  const float norm = (float)sqrt(*sumsq);
  float k = __fdiv_rn(max_norm, norm + 1e-6f);
  if (k > 1.0f || max_norm > FLT_MAX) k = 1.0f;  // a NaN stays under a finite limit
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = norm;
  for (int64_t c = blockIdx.x; c < n; c += gridDim.x) {
    const qsg_grad t = table[n - 1 - c];  // last chunks first: the sum has read them last
    if (!t.out) continue;                     // a tensor of the sum alone
    if (k == 1.0f && t.out == t.g) continue;  // every product is the value itself
    if (t.dtype == QSG_BF16)
      chunk_scale(reinterpret_cast<const uint16_t*>(t.g), reinterpret_cast<uint16_t*>(t.out), (int)t.n, k);
    else
      chunk_scale(reinterpret_cast<const float*>(t.g), reinterpret_cast<float*>(t.out), (int)t.n, k);
  }
}

}  // namespace

void launch_grad_sumsq(const qsg_grad* table, int64_t n, double* sumsq, double* partial, hipStream_t st) {
  const int64_t grid = n < kSumGroups ? n : kSumGroups;
  if (grid > 0) hipLaunchKernelGGL(grad_sumsq_kernel, dim3((unsigned)grid), dim3(256), 0, st, table, n, partial);
  hipLaunchKernelGGL(grad_sum_kernel, dim3(1), dim3(256), 0, st, partial, (int)grid, sumsq);
}

void launch_grad_clip(const qsg_grad* table, int64_t n, const double* sumsq, float max_norm, float* norm_out,
                      hipStream_t st) {
  int64_t grid = n < 65536 ? n : 65536;
  if (grid < 1) grid = 1;  // the norm is written without a tensor too
  hipLaunchKernelGGL(grad_clip_kernel, dim3((unsigned)grid), dim3(256), 0, st, table, n, sumsq, max_norm, norm_out);
}

}  // namespace qsg
