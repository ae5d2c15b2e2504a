// Product of two INT8 matrices with a scale for each row of both:
//   C[m,n] = (sum_k A[m,k] B[n,k]) sa[m] sb[n] (+ bias[n]),  both K-contiguous.
// Sums are 32-bit integers and exact, so they may be split and joined in any
// order; only their scaling is rounded.
//
// Three kernels.  The 256 x 256 kernel of the FP8 products serves the large
// ones (gemm_fast.hip); here are
//   * few rows (a decode batch): bound by reading B once.  A workgroup owns 16
//     columns (rows of B), its waves split K, and the operands go from memory
//     straight into the registers of v_mfma_i32_16x16x64_i8, since no wave
//     uses another's;
//   * everything else: 128 x 128 tiles through LDS.
#include <hip/hip_runtime.h>

#include "qsg_device.h"
#include "qsg_internal.h"

namespace qsg {

namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));
// 16 bytes and 4 outputs at any address (gfx950 loads and stores them there)
typedef int v4i_u __attribute__((ext_vector_type(4), aligned(1)));
typedef float f32x4_e __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_e __attribute__((ext_vector_type(2), aligned(2)));

struct Int8Args {
  const int8_t* a;
  const int8_t* b;
  const float* sa;
  const float* sb;
  const void* bias;
  int bias_bf16;
  int64_t M, N, K, lda, ldb, ldc;
  void* c;
  int64_t tiles_m;
};

// 16 bytes of a row of K bytes at k; what lies past its end is 0
__device__ __forceinline__ v4i load_chunk(const int8_t* row, int64_t k, int64_t K) {
  if (k + 16 <= K) return *reinterpret_cast<const v4i_u*>(row + k);
  v4i r = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 15; ++i)
    if (k + i < K) r[i >> 2] |= (int)((uint32_t)(uint8_t)row[k + i] << (8 * (i & 3)));
  return r;
}

__device__ __forceinline__ float bias_at(const Int8Args& g, int64_t n) {
  if (!g.bias) return 0.0f;
  return g.bias_bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(g.bias)[n] << 16)
                     : reinterpret_cast<const float*>(g.bias)[n];
}

// 4 consecutive outputs of row m from their sums
template <bool OUT_BF16>
__device__ __forceinline__ void store4(const Int8Args& g, int64_t m, int64_t n, const int (&sum)[4], float sa) {
  if (m >= g.M || n >= g.N) return;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t at = n + i < g.N ? n + i : n;
    v[i] = fmaf((float)sum[i] * sa, g.sb[at], bias_at(g, at));
  }
  if constexpr (OUT_BF16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(g.c) + m * g.ldc + n;
    const uint32_t lo = pack_bf16x2(v[0], v[1]), hi = pack_bf16x2(v[2], v[3]);
    if (n + 4 <= g.N) {
      *reinterpret_cast<u32x2_e*>(p) = u32x2_e{lo, hi};
    } else {
      p[0] = (uint16_t)lo;
      if (n + 1 < g.N) p[1] = (uint16_t)(lo >> 16);
      if (n + 2 < g.N) p[2] = (uint16_t)hi;
    }
  } else {
    float* p = reinterpret_cast<float*>(g.c) + m * g.ldc + n;
    if (n + 4 <= g.N) {
      *reinterpret_cast<f32x4_e*>(p) = f32x4_e{v[0], v[1], v[2], v[3]};
    } else {
      p[0] = v[0];
      if (n + 1 < g.N) p[1] = v[1];
      if (n + 2 < g.N) p[2] = v[2];
    }
  }
}

// ---------------------------------------------------------------------------
// few rows
// ---------------------------------------------------------------------------
// MT x 16 rows of A against 16 rows of B.  Lane l holds row l % 16 of either
// operand and, of a step of 128 K, bytes 32 (l / 16) .. +31 as two chunks of
// two instructions: both operands split K between lanes alike, so every
// product is made once.  The instruction takes (B, A), and lane l then holds
// row l % 16 of A and columns 4 (l / 16) .. +3.
template <int MT, int WAVES, bool OUT_BF16>
__global__ __launch_bounds__(WAVES * 64) void gemm_int8_few_kernel(Int8Args g) {
  __shared__ v4i red[WAVES][MT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tm = blockIdx.x % g.tiles_m, tn = blockIdx.x / g.tiles_m;
  const int64_t m0 = tm * (16 * MT), n0 = tn * 16;
  // rows past the end read the last one; their results are not stored
  const int64_t bn = n0 + (lane & 15) < g.N ? n0 + (lane & 15) : g.N - 1;
  const int8_t* b = g.b + bn * g.ldb;
  const int8_t* a[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t m = m0 + i * 16 + (lane & 15);
    a[i] = g.a + (m < g.M ? m : g.M - 1) * g.lda;
  }
  const int at = (lane >> 4) * 32;
  v4i acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = v4i{0, 0, 0, 0};
  const int64_t whole = g.K / 128;
#pragma unroll 4
  for (int64_t s = wave; s < whole; s += WAVES) {
    const int64_t k = s * 128 + at;
    const v4i b0 = *reinterpret_cast<const v4i_u*>(b + k), b1 = *reinterpret_cast<const v4i_u*>(b + k + 16);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const v4i a0 = *reinterpret_cast<const v4i_u*>(a[i] + k), a1 = *reinterpret_cast<const v4i_u*>(a[i] + k + 16);
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1, acc[i], 0, 0, 0);
    }
  }
  if (g.K % 128 && whole % WAVES == wave) {
    const int64_t k = whole * 128 + at;
    const v4i b0 = load_chunk(b, k, g.K), b1 = load_chunk(b, k + 16, g.K);
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const v4i a0 = load_chunk(a[i], k, g.K), a1 = load_chunk(a[i], k + 16, g.K);
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0, acc[i], 0, 0, 0);
      acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1, acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < MT; i += WAVES) {
    v4i t = red[0][i][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) t += red[w][i][lane];
    const int64_t m = m0 + i * 16 + (lane & 15);
    const int sum[4] = {t[0], t[1], t[2], t[3]};
    store4<OUT_BF16>(g, m, n0 + 4 * (lane >> 4), sum, m < g.M ? g.sa[m] : 0.0f);
  }
}

// ---------------------------------------------------------------------------
// 128 x 128 tiles
// ---------------------------------------------------------------------------
constexpr int TB = 128;  // rows of either operand, and bytes of K, of a tile

// 16-byte chunk c of LDS row r is at position c ^ swz(r): the lanes that the
// LDS serves together read 8 rows at two neighbouring chunks, which this puts
// on distinct banks
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

template <bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_int8_kernel(Int8Args g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][2][TB * TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (blockIdx.x % g.tiles_m) * TB, n0 = (blockIdx.x / g.tiles_m) * TB;
  // thread: chunk tid % 8 of rows tid / 8 + 32 i of both operands
  const int ch = tid & 7, r0 = tid >> 3;
  const int8_t* pa[4];
  const int8_t* pb[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + r0 + 32 * i, n = n0 + r0 + 32 * i;
    pa[i] = g.a + (m < g.M ? m : g.M - 1) * g.lda;
    pb[i] = g.b + (n < g.N ? n : g.N - 1) * g.ldb;
  }
  const int64_t nk = (g.K + TB - 1) / TB;
  v4i ra[4], rb[4];
  auto fetch = [&](int64_t kt) {
    const int64_t k = kt * TB + ch * 16;
    if ((kt + 1) * TB <= g.K) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ra[i] = *reinterpret_cast<const v4i_u*>(pa[i] + k);
        rb[i] = *reinterpret_cast<const v4i_u*>(pb[i] + k);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ra[i] = load_chunk(pa[i], k, g.K);
        rb[i] = load_chunk(pb[i], k, g.K);
      }
    }
  };
  auto put = [&](int st) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 32 * i, p = r * TB + ((ch ^ swz(r)) * 16);
      *reinterpret_cast<v4i*>(lds[st][0] + p) = ra[i];
      *reinterpret_cast<v4i*>(lds[st][1] + p) = rb[i];
    }
  };
  v16i acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  if (nk > 0) {
    fetch(0);
    put(0);
  }
  __syncthreads();
  for (int64_t kt = 0; kt < nk; ++kt) {
    const int st = (int)(kt & 1);
    if (kt + 1 < nk) fetch(kt + 1);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      v4i fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = 2 * s + (lane >> 5);
        const int ar = wm * 64 + i * 32 + (lane & 31), br = wn * 64 + i * 32 + (lane & 31);
        fa[i] = *reinterpret_cast<const v4i*>(lds[st][0] + ar * TB + ((c ^ swz(ar)) * 16));
        fb[i] = *reinterpret_cast<const v4i*>(lds[st][1] + br * TB + ((c ^ swz(br)) * 16));
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
    if (kt + 1 < nk) put(st ^ 1);
    __syncthreads();
  }
  // lane l holds row l % 32 and, of group q, columns 8 q + 4 (l / 32) .. +3
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + wm * 64 + i * 32 + (lane & 31);
    const float sa = m < g.M ? g.sa[m] : 0.0f;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int sum[4] = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        store4<OUT_BF16>(g, m, n0 + wn * 64 + j * 32 + 8 * q + 4 * (lane >> 5), sum, sa);
      }
  }
}

template <int MT, int WAVES>
void launch_few(Int8Args g, bool bf16, hipStream_t st) {
  g.tiles_m = (g.M + 16 * MT - 1) / (16 * MT);
  const dim3 grid((unsigned)(g.tiles_m * ((g.N + 15) / 16))), block(WAVES * 64);
  if (bf16) hipLaunchKernelGGL((gemm_int8_few_kernel<MT, WAVES, true>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((gemm_int8_few_kernel<MT, WAVES, false>), grid, block, 0, st, g);
}

}  // namespace

void launch_gemm_int8(const int8_t* a, const float* sa, const int8_t* b, const float* sb, int64_t M, int64_t N,
                      int64_t K, int64_t lda, int64_t ldb, const void* bias, int bias_dtype, void* c, int c_dtype,
                      int64_t ldc, hipStream_t st) {
  Int8Args g{};
  g.a = a; g.b = b; g.sa = sa; g.sb = sb;
  g.bias = bias;
  g.bias_bf16 = bias_dtype == QSG_BF16;
  g.M = M; g.N = N; g.K = K; g.lda = lda; g.ldb = ldb; g.ldc = ldc; g.c = c;
  const bool bf16 = c_dtype == QSG_BF16;
  if (M > 64 && launch_gemm_int8_fast(a, sa, b, sb, M, N, K, lda, ldb, bias, g.bias_bf16, c, c_dtype, ldc, st)) return;
  if (M <= 16) launch_few<1, 8>(g, bf16, st);
  else if (M <= 32) launch_few<2, 8>(g, bf16, st);
  else if (M <= 64) launch_few<4, 8>(g, bf16, st);
  else {
    g.tiles_m = (M + TB - 1) / TB;
    const dim3 grid((unsigned)(g.tiles_m * ((N + TB - 1) / TB)));
    if (bf16) hipLaunchKernelGGL(gemm_int8_kernel<true>, grid, dim3(256), 0, st, g);
    else hipLaunchKernelGGL(gemm_int8_kernel<false>, grid, dim3(256), 0, st, g);
  }
}

}  // namespace qsg
