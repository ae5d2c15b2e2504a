// Residual addition + RMS norm with an FP8 output, and its backward pass.
//
// Forward, for each row:
//   h    = x + r            rounded once to the data type: h is the residual
//                           stream that the next layer adds to, and the norm
//                           reads the rounded h because backward does
//   rstd = 1 / sqrt(sum h^2 / cols + eps)
//   y    = fp32(fp32(h rstd) gamma), quantized from binary32
// Backward, with n = h rstd and dn = dy gamma:
//   dx     = rstd (dn - n sum(dn n) / cols) + dres
//   dgamma = sum over rows of dy n
//
// All sums are binary32.  8 consecutive elements of a row (16 bytes of bf16,
// 32 of fp32) are one chunk; a lane takes whole chunks, so a 1 x 32 block is
// 4 lanes and a 1 x 128 block 16.  The cols % 8 elements after the last whole
// chunk go one to a lane.  Chunks are loaded and stored with vector accesses
// that ask only for the element's alignment (gfx950 takes global accesses at
// any byte address), so odd leading dimensions and offsets use the same
// instructions.
#include <hip/hip_runtime.h>

#include "qsg_device.h"
#include "qsg_internal.h"

namespace qsg {

namespace {

// vector accesses at any element's address
typedef u32x4 u32x4_e __attribute__((aligned(2)));
typedef u32x2 u32x2_e __attribute__((aligned(1)));

// ---------------------------------------------------------------------------
// chunks of 8 elements, and single ones
// ---------------------------------------------------------------------------
template <typename In>
struct Chunk;

template <>
struct Chunk<uint16_t> {  // bf16 bit patterns
  uint32_t w[4];
  __device__ __forceinline__ float at(int i) const { return (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]); }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
  }
  __device__ __forceinline__ void load(const uint16_t* p, bool valid) {
    u32x4 u = {0, 0, 0, 0};
    if (valid) u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  __device__ __forceinline__ void store(uint16_t* p) const {
    const u32x4 u = {w[0], w[1], w[2], w[3]};
    *reinterpret_cast<u32x4_e*>(p) = u;
  }
};

template <>
struct Chunk<float> {
  uint32_t w[8];
  __device__ __forceinline__ float at(int i) const { return __uint_as_float(w[i]); }
  __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[i]);
  }
  __device__ __forceinline__ void load(const float* p, bool valid) {
    u32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (valid) {
      u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p));
      v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p + 4));
    }
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  }
  __device__ __forceinline__ void store(float* p) const {
    const u32x4 u = {w[0], w[1], w[2], w[3]}, v = {w[4], w[5], w[6], w[7]};
    *reinterpret_cast<u32x4_e*>(p) = u;
    *reinterpret_cast<u32x4_e*>(p + 4) = v;
  }
};

__device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
// v rounded to the type, as binary32
__device__ __forceinline__ float round1(const uint16_t*, float v) { return bf16lo(pack_bf16x2(v, 0.0f)); }
__device__ __forceinline__ float round1(const float*, float v) { return v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// 8 weights as binary32 (read by every row: an ordinary, cached load)
__device__ __forceinline__ void load_gamma(float (&g)[8], const void* gamma, bool bf16, int64_t c, bool valid) {
  u32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
  if (bf16) {
    if (valid) u = *reinterpret_cast<const u32x4_e*>(reinterpret_cast<const uint16_t*>(gamma) + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
  } else {
    if (valid) {
      const float* p = reinterpret_cast<const float*>(gamma) + c;
      u = *reinterpret_cast<const u32x4_e*>(p);
      v = *reinterpret_cast<const u32x4_e*>(p + 4);
    }
    g[0] = __uint_as_float(u.x); g[1] = __uint_as_float(u.y); g[2] = __uint_as_float(u.z); g[3] = __uint_as_float(u.w);
    g[4] = __uint_as_float(v.x); g[5] = __uint_as_float(v.y); g[6] = __uint_as_float(v.z); g[7] = __uint_as_float(v.w);
  }
}

__device__ __forceinline__ float load_gamma1(const void* gamma, bool bf16, int64_t c) {
  return bf16 ? load1(reinterpret_cast<const uint16_t*>(gamma) + c) : load1(reinterpret_cast<const float*>(gamma) + c);
}

// ---------------------------------------------------------------------------
// sums
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}

// Sum of a wavefront's 64 values, the same in every lane (the rotates add in
// another order in each lane, so one lane's sum is taken for all).
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  v = dpp_add<kDppRor4>(v);
  v = dpp_add<kDppRor8>(v);
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t t = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(v)));
}

// Sum over the TPR threads that share a row.  For TPR > 64 they are a whole
// workgroup, `red` is one of two LDS buffers used in turn, and one barrier
// suffices: a wave writes a buffer again only after the barrier of the call
// between, which every wave passes after its reads.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int i = 1; i < W; ++i) v += red[i];
  }
  return v;
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
enum { Q_NONE = 0, Q_TENSOR = 1, Q_MX = 2, Q_BLOCK = 3 };

struct NormArgs {
  const void* x;
  const void* r;       // residual or null
  int64_t rows, cols, ldx, ldr, ldh;
  const void* gamma;
  bool gamma_bf16;
  float eps;
  void* h;             // or null
  float* rstd;         // or null
  void* y;             // dense, or null
  int quant, fmt, margin;
  bool mx_ceil;
  const float* scale;  // Q_TENSOR
  uint8_t* q;          // dense, or null
  void* s;
  uint32_t* amax_out;  // max |y| bits, or null
};

template <int FMT>
__device__ __forceinline__ u32x2 enc8(const float (&y)[8], float s) {
  const u32x2 v = {enc4<FMT>(y[0] * s, y[1] * s, y[2] * s, y[3] * s),
                   enc4<FMT>(y[4] * s, y[5] * s, y[6] * s, y[7] * s)};
  return v;
}

// Outputs of one chunk of normalised values at row `row`, column c.  A block
// is made of whole chunks of neighbouring lanes, all of them inside the row
// (valid) or all outside.
template <typename In>
__device__ __forceinline__ void emit(const NormArgs& a, int64_t row, int64_t c, bool valid, const float (&y)[8],
                                     float tscale, uint32_t& amax) {
  if (a.y && valid) {
    Chunk<In> o;
    o.set(y);
    o.store(reinterpret_cast<In*>(a.y) + row * a.cols + c);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax_u32(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  amax = umax_u32(amax, m);
  if (a.quant == Q_NONE) return;
  float s = tscale;
  if (a.quant == Q_MX) {
    m = group_max_u32<0x3>(m);
    m = m > 0x7F800000u ? 0x7FC00000u : m;
    const int e = mx_exponent(m, a.fmt == kE4M3 ? Fp8Traits<kE4M3>::kEmaxElem : Fp8Traits<kE5M2>::kEmaxElem,
                              a.mx_ceil, a.margin);
    s = pow2_neg(e);
    if ((threadIdx.x & 3) == 0 && valid)
      reinterpret_cast<uint8_t*>(a.s)[row * (a.cols / 32) + (c >> 5)] = (uint8_t)(e + 127);
  } else if (a.quant == Q_BLOCK) {
    m = group_max_u32<0xF>(m);
    m = m > 0x7F800000u ? 0x7FC00000u : m;
    s = scale_from_amax(__uint_as_float(m), fp8_max(a.fmt), a.margin);
    if ((threadIdx.x & 15) == 0 && valid)
      reinterpret_cast<float*>(a.s)[row * (a.cols / 128) + (c >> 7)] = __fdiv_rn(1.0f, s);
  }
  const u32x2 v = a.fmt == kE4M3 ? enc8<kE4M3>(y, s) : enc8<kE5M2>(y, s);
  if (valid) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_e*>(a.q + row * a.cols + c));
}

// Outputs of one element after the last whole chunk (never in a block).
template <typename In>
__device__ __forceinline__ void emit1(const NormArgs& a, int64_t row, int64_t c, float y, float tscale,
                                      uint32_t& amax) {
  if (a.y) store1(reinterpret_cast<In*>(a.y) + row * a.cols + c, y);
  amax = umax_u32(amax, __float_as_uint(y) & 0x7FFFFFFFu);
  if (a.quant == Q_NONE) return;
  const float v = y * tscale;
  a.q[row * a.cols + c] = (uint8_t)(a.fmt == kE4M3 ? enc4<kE4M3>(v, 0, 0, 0) : enc4<kE5M2>(v, 0, 0, 0));
}

__device__ __forceinline__ float rstd_of(float ss, int64_t cols, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)cols) + eps));
}

// One pass: TPR threads hold a row in registers, NCH chunks each.
template <typename In, int TPR, int NCH>
__global__ __launch_bounds__(256) void norm_row_kernel(NormArgs a) {
  constexpr int RPW = 256 / TPR;
  __shared__ float red[2][4];
  const int t = threadIdx.x % TPR;
  const int sub = TPR == 256 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);  // uniform in a wave
  const int chunks = (int)(a.cols / 8), rest = (int)(a.cols % 8);
  const float tscale = a.quant == Q_TENSOR ? *a.scale : 1.0f;
  uint32_t amax = 0;
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * RPW + sub; row < a.rows; row += (int64_t)gridDim.x * RPW, turn ^= 1) {
    const In* x = reinterpret_cast<const In*>(a.x) + row * a.ldx;
    const In* r = reinterpret_cast<const In*>(a.r) + row * a.ldr;
    In* ho = reinterpret_cast<In*>(a.h) + row * a.ldh;
    Chunk<In> h[NCH];
    float h1 = 0.0f;  // the element after the last whole chunk
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      h[j].load(x + k * 8, k < (uint32_t)chunks);
    }
    if (t < rest) h1 = load1(x + chunks * 8 + t);
    if (a.r) {
      Chunk<In> d[NCH];
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        d[j].load(r + k * 8, k < (uint32_t)chunks);
      }
      if (t < rest) h1 = round1(x, h1 + load1(r + chunks * 8 + t));
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h[j].at(i) + d[j].at(i);
        h[j].set(v);
      }
    }
    if (a.h) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        if (k < (uint32_t)chunks) h[j].store(ho + k * 8);
      }
      if (t < rest) store1(ho + chunks * 8 + t, h1);
    }
    float ss = h1 * h1;
#pragma unroll
    for (int j = 0; j < NCH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h[j].at(i), h[j].at(i), ss);
    ss = row_sum<TPR>(ss, red[turn]);
    const float rstd = rstd_of(ss, a.cols, a.eps);
    if (a.rstd && t == 0) a.rstd[row] = rstd;
    if (a.quant == Q_NONE && !a.y && !a.amax_out) continue;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      const bool valid = k < (uint32_t)chunks;
      float g[8], y[8];
      load_gamma(g, a.gamma, a.gamma_bf16, k * 8, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[j].at(i) * rstd * g[i];
      emit<In>(a, row, k * 8, valid, y, tscale, amax);
    }
    if (t < rest) {
      const int64_t c = chunks * 8 + t;
      emit1<In>(a, row, c, h1 * rstd * load_gamma1(a.gamma, a.gamma_bf16, c), tscale, amax);
    }
  }
  if (a.amax_out) {
    __shared__ uint32_t ured[4];
    block_max_to_global<256>(amax, a.amax_out, ured);
  }
}

// Rows longer than the registers hold: a workgroup reads its row twice (the
// second time h, from the caches).
template <typename In>
__global__ __launch_bounds__(256) void norm_long_kernel(NormArgs a) {
  __shared__ float red[2][4];
  const float tscale = a.quant == Q_TENSOR ? *a.scale : 1.0f;
  uint32_t amax = 0;
  int turn = 0;
  const int64_t chunks = a.cols / 8, padded = (chunks + 255) / 256 * 256;
  const int64_t c1 = chunks * 8 + threadIdx.x;  // this thread's element after the last whole chunk
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const In* x = reinterpret_cast<const In*>(a.x) + row * a.ldx;
    const In* r = reinterpret_cast<const In*>(a.r) + row * a.ldr;
    In* ho = reinterpret_cast<In*>(a.h) + row * a.ldh;
    float ss = 0.0f, h1 = 0.0f;
    for (int64_t k = threadIdx.x; k < chunks; k += 256) {
      Chunk<In> h;
      h.load(x + k * 8, true);
      if (a.r) {
        Chunk<In> d;
        d.load(r + k * 8, true);
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h.at(i) + d.at(i);
        h.set(v);
      }
      if (a.h) h.store(ho + k * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(h.at(i), h.at(i), ss);
    }
    if (c1 < a.cols) {
      h1 = load1(x + c1);
      if (a.r) h1 = round1(x, h1 + load1(r + c1));
      if (a.h) store1(ho + c1, h1);
      ss = fmaf(h1, h1, ss);
    }
    ss = row_sum<256>(ss, red[turn]);
    const float rstd = rstd_of(ss, a.cols, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
    if (a.quant == Q_NONE && !a.y && !a.amax_out) continue;
    const In* hi = a.h ? ho : x;
    // every lane takes part in the block maxima, so the count is padded; each
    // thread reads back the chunks that it wrote itself
    for (int64_t k = threadIdx.x; k < padded; k += 256) {
      const bool valid = k < chunks;
      Chunk<In> h;
      float g[8], y[8];
      h.load(hi + k * 8, valid);
      load_gamma(g, a.gamma, a.gamma_bf16, k * 8, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h.at(i) * rstd * g[i];
      emit<In>(a, row, k * 8, valid, y, tscale, amax);
    }
    if (c1 < a.cols) emit1<In>(a, row, c1, h1 * rstd * load_gamma1(a.gamma, a.gamma_bf16, c1), tscale, amax);
  }
  if (a.amax_out) {
    __shared__ uint32_t ured[4];
    block_max_to_global<256>(amax, a.amax_out, ured);
  }
}

template <typename In>
void launch_row(const NormArgs& a, hipStream_t st) {
  const int64_t chunks = a.cols / 8;
  // one wave per row where it holds the row and there are rows enough to fill
  // the card with waves, else a workgroup per row
  const bool wave = chunks <= 64 || (chunks <= 64 * 16 && a.rows >= 1024 && sizeof(In) == 2);
  int64_t grid = wave ? (a.rows + 3) / 4 : a.rows;
  // an amax output ends in one atomic per workgroup on one address, which the
  // memory side performs one at a time: a persistent grid then
  const int64_t cap = a.amax_out ? 1024 : 1 << 20;
  if (grid > cap) grid = cap;
  const dim3 g((unsigned)grid), b(256);
#define QSG_ROW(TPR, NCH) hipLaunchKernelGGL((norm_row_kernel<In, TPR, NCH>), g, b, 0, st, a)
  if (wave) {
    if (chunks <= 64) QSG_ROW(64, 1);
    else if constexpr (sizeof(In) == 2) {
      if (chunks <= 64 * 2) QSG_ROW(64, 2);
      else if (chunks <= 64 * 4) QSG_ROW(64, 4);
      else if (chunks <= 64 * 8) QSG_ROW(64, 8);
      else QSG_ROW(64, 16);
    }
  } else if (chunks <= 256) QSG_ROW(256, 1);
  else if (chunks <= 256 * 2) QSG_ROW(256, 2);
  else if (chunks <= 256 * 4) QSG_ROW(256, 4);
  else if (chunks <= 256 * 8) QSG_ROW(256, 8);
  else hipLaunchKernelGGL(norm_long_kernel<In>, g, b, 0, st, a);
#undef QSG_ROW
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
struct NormBwdArgs {
  const void* dy;
  const void* h;
  const void* dres;  // or null
  int64_t rows, cols, lddy, ldh, lddres, lddx;
  const void* gamma;
  bool gamma_bf16;
  const float* rstd;
  void* dx;
  float* partial;    // groups x cols, or null (no dgamma)
  float* dots;       // rows: sum(dn h), wide rows only
};

// A group of TPR threads takes rows group, group + groups, ... and holds a
// row in registers, NCH chunks per thread; its share of dgamma stays in
// registers until the end.  WIDE: the rows' dots are read from a.dots, and
// blockIdx.y is the piece of 8 TPR NCH columns.
template <typename In, int TPR, int NCH, bool WIDE>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int THREADS = TPR < 256 ? 256 : TPR, RPW = THREADS / TPR;
  __shared__ float red[2][16];
  const int t = threadIdx.x % TPR;
  const int sub = RPW == 1 ? 0 : __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR);
  const int64_t group = (int64_t)blockIdx.x * RPW + sub, groups = (int64_t)gridDim.x * RPW;
  const int64_t c0 = WIDE ? (int64_t)blockIdx.y * (8 * TPR * NCH) : 0;
  const int64_t here = WIDE && a.cols - c0 > 8 * TPR * NCH ? 8 * TPR * NCH : a.cols - c0;  // columns of this piece
  const int chunks = (int)(here / 8), rest = (int)(here % 8);
  float g[NCH][8], acc[NCH][8], g1 = 0.0f, acc1 = 0.0f;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const uint32_t k = j * TPR + t;
    load_gamma(g[j], a.gamma, a.gamma_bf16, c0 + k * 8, k < (uint32_t)chunks);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  }
  if (t < rest) g1 = load_gamma1(a.gamma, a.gamma_bf16, c0 + chunks * 8 + t);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups, turn ^= 1) {
    const In* pdy = reinterpret_cast<const In*>(a.dy) + row * a.lddy + c0;
    const In* ph = reinterpret_cast<const In*>(a.h) + row * a.ldh + c0;
    const In* pdr = reinterpret_cast<const In*>(a.dres) + row * a.lddres + c0;
    In* pdx = reinterpret_cast<In*>(a.dx) + row * a.lddx + c0;
    Chunk<In> dy[NCH], h[NCH], dr[NCH];
    float dy1 = 0.0f, h1 = 0.0f, dr1 = 0.0f;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      dy[j].load(pdy + k * 8, k < (uint32_t)chunks);
      h[j].load(ph + k * 8, k < (uint32_t)chunks);
    }
    if (t < rest) {
      dy1 = load1(pdy + chunks * 8 + t);
      h1 = load1(ph + chunks * 8 + t);
    }
    if (a.dres) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        dr[j].load(pdr + k * 8, k < (uint32_t)chunks);
      }
      if (t < rest) dr1 = load1(pdr + chunks * 8 + t);
    }
    const float rstd = a.rstd[row];
    float dot;
    if constexpr (WIDE) {
      dot = a.dots[row];
    } else {
      dot = dy1 * g1 * (h1 * rstd);
#pragma unroll
      for (int j = 0; j < NCH; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) dot = fmaf(dy[j].at(i) * g[j][i], h[j].at(i) * rstd, dot);
      dot = row_sum<TPR>(dot, red[turn]);
    }
    const float m = __fdiv_rn(dot, (float)a.cols);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = h[j].at(i) * rstd;
        acc[j][i] = fmaf(dy[j].at(i), n, acc[j][i]);
        v[i] = rstd * fmaf(-n, m, dy[j].at(i) * g[j][i]);
        if (a.dres) v[i] += dr[j].at(i);
      }
      if (k < (uint32_t)chunks) {
        Chunk<In> o;
        o.set(v);
        o.store(pdx + k * 8);
      }
    }
    if (t < rest) {
      const float n = h1 * rstd;
      acc1 = fmaf(dy1, n, acc1);
      store1(pdx + chunks * 8 + t, fmaf(rstd, fmaf(-n, m, dy1 * g1), dr1));
    }
  }
  if (a.partial) {
    float* p = a.partial + group * a.cols + c0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      if (k < (uint32_t)chunks) {
        Chunk<float> o;
        o.set(acc[j]);
        o.store(p + k * 8);
      }
    }
    if (t < rest) p[chunks * 8 + t] = acc1;
  }
}

// dots[row] = sum(dn n) of rows too long for the registers
template <typename In>
__global__ __launch_bounds__(256) void norm_bwd_dot_kernel(NormBwdArgs a) {
  __shared__ float red[2][4];
  int turn = 0;
  const int64_t chunks = a.cols / 8, c1 = chunks * 8 + threadIdx.x;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const In* pdy = reinterpret_cast<const In*>(a.dy) + row * a.lddy;
    const In* ph = reinterpret_cast<const In*>(a.h) + row * a.ldh;
    const float rstd = a.rstd[row];
    float dot = 0.0f;
    for (int64_t k = threadIdx.x; k < chunks; k += 256) {
      Chunk<In> dy, h;
      float g[8];
      dy.load(pdy + k * 8, true);
      h.load(ph + k * 8, true);
      load_gamma(g, a.gamma, a.gamma_bf16, k * 8, true);
#pragma unroll
      for (int i = 0; i < 8; ++i) dot = fmaf(dy.at(i) * g[i], h.at(i) * rstd, dot);
    }
    if (c1 < a.cols) dot = fmaf(load1(pdy + c1) * load_gamma1(a.gamma, a.gamma_bf16, c1), load1(ph + c1) * rstd, dot);
    dot = row_sum<256>(dot, red[turn]);
    if (threadIdx.x == 0) a.dots[row] = dot;
  }
}

// dgamma[c] (+)= sum over groups of partial[group][c], in a fixed order: a
// workgroup takes 32 columns, 8 lanes of 4 columns by 32 rows of groups.
__global__ __launch_bounds__(256) void norm_dgamma_kernel(const float* partial, int64_t groups, int64_t cols,
                                                          float* dgamma, bool accumulate) {
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane * 4;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k = part; k < groups; k += 32) {
    const float* p = partial + k * cols + c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i < cols) v[i] += p[i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[part][lane * 4 + i] = v[i];
  __syncthreads();
  if (threadIdx.x < 32) {
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    if (col < cols) {
      float s = sum[0][threadIdx.x];
      for (int k = 1; k < 32; ++k) s += sum[k][threadIdx.x];
      dgamma[col] = accumulate ? dgamma[col] + s : s;
    }
  }
}

constexpr int64_t kBwdGroups = 1024;     // groups that share the rows of a backward pass, at most
constexpr int64_t kBwdMostCols = 16391; // of a row held in registers: 2048 chunks and 7 elements
constexpr int64_t kBwdPiece = 2048;      // columns of a workgroup beyond that

template <typename In>
void launch_bwd(const NormBwdArgs& a, int64_t groups, hipStream_t st) {
  const int64_t chunks = a.cols / 8;
#define QSG_BWD(TPR, NCH)                                                                          \
  hipLaunchKernelGGL((norm_bwd_kernel<In, TPR, NCH, false>),                                       \
                     dim3((unsigned)(groups / (TPR < 256 ? 256 / TPR : 1))), dim3(TPR < 256 ? 256 : TPR), 0, st, a)
  if (chunks <= 64) QSG_BWD(64, 1);
  else if (chunks <= 256) QSG_BWD(256, 1);
  else if (chunks <= 512) QSG_BWD(256, 2);
  else if (chunks <= 1024) QSG_BWD(256, 4);
  else if (chunks <= 2048) QSG_BWD(1024, 2);
  else {
    int64_t g = a.rows < 4096 ? a.rows : 4096;
    hipLaunchKernelGGL(norm_bwd_dot_kernel<In>, dim3((unsigned)g), dim3(256), 0, st, a);
    const int64_t pieces = (a.cols + kBwdPiece - 1) / kBwdPiece;
    hipLaunchKernelGGL((norm_bwd_kernel<In, 256, 1, true>), dim3((unsigned)groups, (unsigned)pieces), dim3(256), 0, st,
                       a);
  }
#undef QSG_BWD
}

// groups of a backward pass: a multiple of 4 where a workgroup holds 4 rows
int64_t bwd_groups(int64_t rows, int64_t cols) {
  int64_t g = rows < kBwdGroups ? rows : kBwdGroups;
  if (cols < 65 * 8) g = (g + 3) / 4 * 4;
  return g;
}

}  // namespace

void launch_rmsnorm_quantize(const void* x, const void* r, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                             int64_t ldr, const void* gamma, int gamma_dtype, float eps, int scaling, int fmt,
                             int margin, bool mx_ceil, const float* scale, void* h, int64_t ldh, float* rstd, void* y,
                             uint8_t* q, void* s, uint8_t* qt, void* st_, float* amax_out, hipStream_t st) {
  const bool tensorwise = scaling == 0, quantized = q || qt;
  float* three = reinterpret_cast<float*>(s);
  float* amax = tensorwise ? three : amax_out;
  if (amax) launch_fill_u32(reinterpret_cast<uint32_t*>(amax), 0u, 1, st);
  if (rows == 0 || cols == 0) {
    if (tensorwise) launch_compute_scale(three, fmt, margin, three + 1, three + 2, st);
    return;
  }
  // The transposed copy takes tiles of 128 rows, and the current scaling the
  // whole tensor's amax, before the first code can be written: a second
  // kernel reads h (or x) back then.
  const bool two = quantized && (tensorwise || qt);
  NormArgs a{};
  a.x = x; a.r = r;
  a.rows = rows; a.cols = cols; a.ldx = ldx; a.ldr = ldr; a.ldh = ldh;
  a.gamma = gamma; a.gamma_bf16 = gamma_dtype == 1;
  a.eps = eps;
  a.h = h; a.rstd = rstd; a.y = y;
  a.fmt = fmt; a.margin = margin; a.mx_ceil = mx_ceil;
  if (!two && q) {
    a.quant = scaling == 1 ? Q_TENSOR : scaling == 2 ? Q_MX : Q_BLOCK;
    a.scale = scale;
    a.q = q; a.s = s;
  }
  if (tensorwise || !two) a.amax_out = reinterpret_cast<uint32_t*>(amax);
  if (dtype == 1)
    launch_row<uint16_t>(a, st);
  else
    launch_row<float>(a, st);
  if (!two) return;
  if (tensorwise) launch_compute_scale(three, fmt, margin, three + 1, three + 2, st);
  launch_quantize_normed(h ? h : x, dtype, rows, cols, h ? ldh : ldx, rstd, gamma, gamma_dtype, scaling, fmt, margin,
                         mx_ceil, tensorwise ? three + 1 : scale, q, s, qt, st_, tensorwise ? nullptr : amax_out, st);
}

int64_t rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  return (bwd_groups(rows, cols) * cols + (cols > kBwdMostCols ? rows : 0)) * 4;
}

void launch_rmsnorm_bwd(const void* dy, const void* h, const void* dres, int dtype, int64_t rows, int64_t cols,
                        int64_t lddy, int64_t ldh, int64_t lddres, const void* gamma, int gamma_dtype,
                        const float* rstd, void* dx, int64_t lddx, float* dgamma, bool accumulate, void* workspace,
                        hipStream_t st) {
  if (rows == 0) {
    for (int64_t c = 0; c < cols; c += 1 << 30) {  // dgamma = 0
      const int64_t n = cols - c < (1 << 30) ? cols - c : (1 << 30);
      launch_fill_u32(reinterpret_cast<uint32_t*>(dgamma + c), 0u, (int)n, st);
    }
    return;
  }
  const int64_t groups = bwd_groups(rows, cols);
  float* ws = reinterpret_cast<float*>(workspace);
  NormBwdArgs a{};
  a.dy = dy; a.h = h; a.dres = dres;
  a.rows = rows; a.cols = cols; a.lddy = lddy; a.ldh = ldh; a.lddres = lddres; a.lddx = lddx;
  a.gamma = gamma; a.gamma_bf16 = gamma_dtype == 1;
  a.rstd = rstd; a.dx = dx;
  a.partial = dgamma ? ws : nullptr;
  a.dots = ws + groups * cols;
  if (dtype == 1)
    launch_bwd<uint16_t>(a, groups, st);
  else
    launch_bwd<float>(a, groups, st);
  if (dgamma)
    hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, st, ws, groups, cols,
                       dgamma, accumulate);
}

}  // namespace qsg
