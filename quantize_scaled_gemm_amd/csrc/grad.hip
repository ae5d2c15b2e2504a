// Global norm of many gradient tensors, and clipping by it.
//
//   S    = sum over tensors and elements of g^2          (binary64)
//   norm = sqrt(S),  k = min(1, max_norm / (norm + 1e-6)),  out = g k
//
// The tensors are cut into chunks on the host (qsg_grad_plan) and the table
// of chunks lies in device memory, so one launch covers any number of
// tensors.  Squares and sums are binary64: a binary32 square loses gradients
// below 2^-75 and overflows above 2^64.
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

__device__ __forceinline__ void add_squares_bf16(double& s, u32x4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double lo = bf16lo(w[k]), hi = bf16hi(w[k]);
    s = fma(lo, lo, s);
    s = fma(hi, hi, s);
  }
}

__device__ __forceinline__ void add_squares_f32(double& s, u32x4 u) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const double v = __uint_as_float(w[k]);
    s = fma(v, v, s);
  }
}

__global__ __launch_bounds__(256) void grad_sumsq_kernel(const qsg_grad* table, int64_t n, double* partial) {
  __shared__ double red[4];
  double s = 0.0;
  for (int64_t k = blockIdx.x; k < n; k += gridDim.x) {
    const qsg_grad t = table[k];
    if (t.dtype == QSG_BF16) {
      const uint16_t* g = reinterpret_cast<const uint16_t*>(t.g);
      const int whole = (int)(t.n / 8) * 8;
      for (int i = threadIdx.x * 8; i < whole; i += 256 * 8)
        add_squares_bf16(s, __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + i)));
      for (int i = whole + threadIdx.x; i < (int)t.n; i += 256) {
        const double v = __uint_as_float((uint32_t)g[i] << 16);
        s = fma(v, v, s);
      }
    } else {
      const float* g = reinterpret_cast<const float*>(t.g);
      const int whole = (int)(t.n / 4) * 4;
      for (int i = threadIdx.x * 4; i < whole; i += 256 * 4)
        add_squares_f32(s, __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + i)));
      for (int i = whole + threadIdx.x; i < (int)t.n; i += 256) {
        const double v = g[i];
        s = fma(v, v, s);
      }
    }
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

__global__ __launch_bounds__(256) void grad_clip_kernel(const qsg_grad* table, int64_t n, const double* sumsq,
                                                        float max_norm, float* norm_out) {
  const float norm = (float)sqrt(*sumsq);
  float k = __fdiv_rn(max_norm, norm + 1e-6f);
  if (k > 1.0f) k = 1.0f;  // a NaN stays
  if (blockIdx.x == 0 && threadIdx.x == 0 && norm_out) *norm_out = norm;
  for (int64_t c = blockIdx.x; c < n; c += gridDim.x) {
    const qsg_grad t = table[c];
    if (k == 1.0f && t.out == t.g) continue;  // every product is the value itself
    if (t.dtype == QSG_BF16) {
      const uint16_t* g = reinterpret_cast<const uint16_t*>(t.g);
      uint16_t* o = reinterpret_cast<uint16_t*>(t.out);
      const int whole = (int)(t.n / 8) * 8;
      for (int i = threadIdx.x * 8; i < whole; i += 256 * 8) {
        const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + i));
        const u32x4 v = {pack_bf16x2(bf16lo(u.x) * k, bf16hi(u.x) * k), pack_bf16x2(bf16lo(u.y) * k, bf16hi(u.y) * k),
                         pack_bf16x2(bf16lo(u.z) * k, bf16hi(u.z) * k), pack_bf16x2(bf16lo(u.w) * k, bf16hi(u.w) * k)};
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_e*>(o + i));
      }
      for (int i = whole + threadIdx.x; i < (int)t.n; i += 256)
        o[i] = (uint16_t)pack_bf16x2(__uint_as_float((uint32_t)g[i] << 16) * k, 0.0f);
    } else {
      const float* g = reinterpret_cast<const float*>(t.g);
      float* o = reinterpret_cast<float*>(t.out);
      const int whole = (int)(t.n / 4) * 4;
      for (int i = threadIdx.x * 4; i < whole; i += 256 * 4) {
        const u32x4 u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(g + i));
        const u32x4 v = {__float_as_uint(__uint_as_float(u.x) * k), __float_as_uint(__uint_as_float(u.y) * k),
                         __float_as_uint(__uint_as_float(u.z) * k), __float_as_uint(__uint_as_float(u.w) * k)};
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4_e*>(o + i));
      }
      for (int i = whole + threadIdx.x; i < (int)t.n; i += 256) o[i] = g[i] * k;
    }
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
