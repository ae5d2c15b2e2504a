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
// Sums along rows and each group's share of dgamma are binary32, the sum of the
// shares binary64.  8 consecutive elements of a row (16 bytes of bf16,
// 32 of fp32) are one chunk; a lane takes whole chunks, so a 1 x 32 block is
// 4 lanes and a 1 x 128 block 16.  The cols % 8 elements after the last whole
// chunk go one to a lane.  Chunks are loaded and stored with vector accesses
// that ask only for the element's alignment (gfx950 takes global accesses at
// any byte address), so odd leading dimensions and offsets use the same
// instructions.
//
// Every kernel here is bound by HBM (a few rows by latency).  [measured,
// MI355X] A 2 GiB device copy moves 4.9-5.1 TB/s; the row kernel moves 6.2
// (32768 x 4096, MXFP8 row-wise: 939 MB in 150 us), the column kernel 6.1
// counting what it reads from the caches (268 MB of h and 134 MB of codes in
// 66 us), the backward kernel 5.8 (16384 x 7168 with a residual gradient: 940
// MB in 160 us).  One launch that kept 128 rows of h on the chip for both
// copies would save the second reading of h (2 of 10 bytes an element), but
// 128 rows of 4096 columns are 1 MB, twice a CU's registers and LDS.  32 rows
// fit, and write qt in runs of 32 bytes: a kernel that only moved those bytes
// (32768 x 4096, neighbouring rows on one XCD, no arithmetic) took 206 us, the
// two passes with all of theirs 209.
#include <float.h>
#include <hip/hip_runtime.h>

#include "qsg_device.h"
#include "qsg_internal.h"

namespace qsg {

namespace {

// vector accesses at any element's address
typedef u32x4 u32x4_e __attribute__((aligned(2)));
typedef u32x4 u32x4_b __attribute__((aligned(1)));
typedef u32x2 u32x2_e __attribute__((aligned(1)));
typedef uint32_t u32_b __attribute__((aligned(1)));

// ---------------------------------------------------------------------------
// chunks of 8 elements, and single ones
// ---------------------------------------------------------------------------
// STREAM: a non-temporal store, for what the call does not read back.  What
// the second pass reads (h, or q) is stored plainly and stays in the caches as
// far as they reach.
template <bool STREAM>
__device__ __forceinline__ void keep_apart() {
  // a comment before and after each store: the compiler otherwise merges a
  // plain and a streaming store in two branches into one plain store
  asm volatile("; streaming %0" : : "n"(STREAM));
}
template <bool STREAM>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
  keep_apart<STREAM>();
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_b*>(p));
  else
    *reinterpret_cast<u32x4_b*>(p) = v;
  keep_apart<STREAM>();
}
template <bool STREAM>
__device__ __forceinline__ void put8(void* p, u32x2 v) {
  keep_apart<STREAM>();
  if constexpr (STREAM)
    __builtin_nontemporal_store(v, reinterpret_cast<u32x2_e*>(p));
  else
    *reinterpret_cast<u32x2_e*>(p) = v;
  keep_apart<STREAM>();
}

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
  // the words become new values to the compiler, which would otherwise keep
  // the 8 widened values of an earlier use in registers beside them
  __device__ __forceinline__ void forget_wide() {
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("" : "+v"(w[k]));
  }
  __device__ __forceinline__ void load(const uint16_t* p, bool valid) {
    u32x4 u = {0, 0, 0, 0};
    if (valid) u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p));
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(uint16_t* p) const {
    const u32x4 u = {w[0], w[1], w[2], w[3]};
    put16<STREAM>(p, u);
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
  __device__ __forceinline__ void forget_wide() {}
  __device__ __forceinline__ void load(const float* p, bool valid) {
    u32x4 u = {0, 0, 0, 0}, v = {0, 0, 0, 0};
    if (valid) {
      // plain loads: each takes every other 16 bytes of its cache lines, and a
      // streaming line may be gone when the other comes (22715 x 2944: 240 us
      // a call, plain 219)
      u = *reinterpret_cast<const u32x4_e*>(p);
      v = *reinterpret_cast<const u32x4_e*>(p + 4);
    }
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    w[4] = v.x; w[5] = v.y; w[6] = v.z; w[7] = v.w;
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(float* p) const {
    const u32x4 u = {w[0], w[1], w[2], w[3]}, v = {w[4], w[5], w[6], w[7]};
    put16<STREAM>(p, u);
    put16<STREAM>(p + 4, v);
  }
};

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
// The same for an element that was loaded under a branch.  The compiler moves
// a plain widen() into that branch, and so waits for the element there,
// before it issues the loads that follow (backward 32768 x 1001: 85 us).
__device__ __forceinline__ float widen_here(uint16_t v) {
  uint32_t u = v;
  asm("" : "+v"(u));
  return __uint_as_float(u << 16);
}
__device__ __forceinline__ float widen_here(float v) { return v; }
template <typename In>
__device__ __forceinline__ float load1(const In* p) { return widen(*p); }
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
constexpr int kHalfMirror = 0x141, kMirror = 0x140;  // lane i gets 7 - i of its 8, 15 - i of its 16

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(dpp_u32<CTRL>(__float_as_uint(v)));
}

// Sum over groups of 16 or 64 lanes, the same in every lane of a group: each
// step adds two values that its two lanes hold in either order (quads by
// exchanges, 16 lanes by mirrors, rows by swaps).
template <int LANES>
__device__ __forceinline__ float lane_sum(float v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  v = dpp_add<kHalfMirror>(v);
  v = dpp_add<kMirror>(v);
  if constexpr (LANES == 64) {
    const uint32_t u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const uint32_t t = __float_as_uint(v);
    const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
    v = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  }
  return v;
}

// Sum over the TPR threads (consecutive ones of the workgroup) that share a
// row.  For TPR > 64 every thread of the workgroup calls this together, `red`
// is one of two LDS buffers used in turn, and one barrier suffices: a wave
// writes a buffer again only after the barrier of the call between, which
// every wave passes after its reads.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = lane_sum<TPR < 64 ? TPR : 64>(v);
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    red += threadIdx.x / TPR * W;
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
  bool second, again;  // the second pass reads h, or q, back
};

template <int FMT>
__device__ __forceinline__ u32x2 enc8(const float (&y)[8], float s) {
  const u32x2 v = {enc4<FMT>(y[0] * s, y[1] * s, y[2] * s, y[3] * s),
                   enc4<FMT>(y[4] * s, y[5] * s, y[6] * s, y[7] * s)};
  return v;
}

// Where a row's outputs begin.  Uniform in a wave: the address of a chunk is a
// scalar base and a 32-bit offset.
template <typename In>
struct RowOut {
  In* y;
  uint8_t* q;
  void* s;
  __device__ __forceinline__ RowOut(const NormArgs& a, int64_t row) {
    y = reinterpret_cast<In*>(a.y) + (a.y ? row * a.cols : 0);
    q = a.q + (a.q ? row * a.cols : 0);
    s = nullptr;
    if (a.quant == Q_MX) s = reinterpret_cast<uint8_t*>(a.s) + row * (a.cols / 32);
    if (a.quant == Q_BLOCK) s = reinterpret_cast<float*>(a.s) + row * (a.cols / 128);
  }
};

// Outputs of one chunk of normalised values at column c.  A block is made of
// whole chunks of neighbouring lanes, all of them inside the row (valid) or
// all outside.
template <typename In>
__device__ __forceinline__ void emit(const NormArgs& a, const RowOut<In>& out, uint32_t c, bool valid,
                                     const float (&y)[8], float tscale, uint32_t& amax) {
  if (a.y && valid) {
    Chunk<In> o;
    o.set(y);
    o.template store<true>(out.y + c);
  }
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax_u32(m, __float_as_uint(y[i]) & 0x7FFFFFFFu);
  if (valid) amax = umax_u32(amax, m);
  if (a.quant == Q_NONE) return;
  float s = tscale;
  if (a.quant == Q_MX) {
    m = group_max_u32<0x3>(m);
    m = m > 0x7F800000u ? 0x7FC00000u : m;
    const int e = mx_exponent(m, a.fmt == kE4M3 ? Fp8Traits<kE4M3>::kEmaxElem : Fp8Traits<kE5M2>::kEmaxElem,
                              a.mx_ceil, a.margin);
    s = pow2_neg(e);
    if ((threadIdx.x & 3) == 0 && valid) reinterpret_cast<uint8_t*>(out.s)[c >> 5] = (uint8_t)(e + 127);
  } else if (a.quant == Q_BLOCK) {
    m = group_max_u32<0xF>(m);
    m = m > 0x7F800000u ? 0x7FC00000u : m;
    s = scale_from_amax(__uint_as_float(m), fp8_max(a.fmt), a.margin);
    if ((threadIdx.x & 15) == 0 && valid) reinterpret_cast<float*>(out.s)[c >> 7] = __fdiv_rn(1.0f, s);
  }
  const u32x2 v = a.fmt == kE4M3 ? enc8<kE4M3>(y, s) : enc8<kE5M2>(y, s);
  if (valid) {
    if (a.again)
      put8<false>(out.q + c, v);
    else
      put8<true>(out.q + c, v);
  }
}

// Outputs of one element after the last whole chunk (never in a block).
template <typename In>
__device__ __forceinline__ void emit1(const NormArgs& a, const RowOut<In>& out, uint32_t c, float y, float tscale,
                                      uint32_t& amax) {
  if (a.y) store1(out.y + c, y);
  amax = umax_u32(amax, __float_as_uint(y) & 0x7FFFFFFFu);
  if (a.quant == Q_NONE) return;
  const float v = y * tscale;
  out.q[c] = (uint8_t)(a.fmt == kE4M3 ? enc4<kE4M3>(v, 0, 0, 0) : enc4<kE5M2>(v, 0, 0, 0));
}

// The launch's maximum: stored by a launch's only workgroup (nothing is
// cleared before); by one atomic of each of up to 512, which wait for nothing;
// of more only by those that read a smaller one there, since all of this is
// done one at a time on the memory side (1021 x 4096, 256 workgroups: 12.4 us a
// call, with a read first 14.4; 4096 x 8192, 1024 workgroups: 49.1 and 48.1).
template <int NTHREADS>
__device__ __forceinline__ void finish_amax(uint32_t m, uint32_t* out, uint32_t* lds) {
  if (gridDim.x > 512) return block_max_to_global<NTHREADS>(m, out, lds);
  m = wave_max_u32(m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < NTHREADS / 64; ++i) m = umax_u32(m, lds[i]);
    if (m > 0x7F800000u) m = 0x7FC00000u;
    if (gridDim.x == 1)
      *out = m;
    else
      atomicMax(out, m);
  }
}

__device__ __forceinline__ float rstd_of(float ss, int64_t cols, float eps) {
  return __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(ss, (float)cols) + eps));
}

// One pass: TPR threads hold a row in registers, NCH chunks each; a workgroup
// of BLK threads takes BLK / TPR rows at a time.
template <typename In, int TPR, int NCH, int BLK>
__global__ __launch_bounds__(BLK) void norm_row_kernel(NormArgs a) {
  constexpr int RPW = BLK / TPR;
  constexpr bool EARLY = NCH <= 2;  // the weights fit beside the row: loaded once, before the first row arrives
  __shared__ float red[2][16];
  const int t = threadIdx.x % TPR;
  int sub = threadIdx.x / TPR;
  if constexpr (TPR >= 64) sub = __builtin_amdgcn_readfirstlane(sub);  // uniform in a wave
  const int all_chunks = (int)(a.cols / 8), all_rest = (int)(a.cols % 8);
  const float tscale = a.quant == Q_TENSOR ? *a.scale : 1.0f;
  uint32_t amax = 0;
  int turn = 0;
  const bool outputs = a.quant != Q_NONE || a.y || a.amax_out;
  float ge[EARLY ? NCH : 1][8], g1 = 0.0f;
  if (EARLY && outputs) {
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      load_gamma(ge[j], a.gamma, a.gamma_bf16, k * 8, k < (uint32_t)all_chunks);
    }
  }
  if (t < all_rest && outputs) g1 = load_gamma1(a.gamma, a.gamma_bf16, all_chunks * 8 + t);
  for (int64_t row0 = (int64_t)blockIdx.x * RPW; row0 < a.rows; row0 += (int64_t)gridDim.x * RPW, turn ^= 1) {
    // with barriers in the loop the last workgroup's spare threads stay in it, on a row that is not there
    const int64_t row = row0 + sub;
    const bool there = RPW == 1 || row < a.rows;
    if (TPR <= 64 && !there) break;
    const int chunks = there ? all_chunks : 0, rest = there ? all_rest : 0;
    const In* x = reinterpret_cast<const In*>(a.x) + row * a.ldx;
    const In* r = reinterpret_cast<const In*>(a.r) + row * a.ldr;
    In* ho = reinterpret_cast<In*>(a.h) + row * a.ldh;
    Chunk<In> h[NCH];
    In x1 = 0, r1 = 0;  // the element after the last whole chunk
    if (t < rest) x1 = x[chunks * 8 + t];
    if (t < rest && a.r) r1 = r[chunks * 8 + t];
    if (!a.r) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        h[j].load(x + k * 8, k < (uint32_t)chunks);
      }
    } else {
      Chunk<In> d[NCH];
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        h[j].load(x + k * 8, k < (uint32_t)chunks);
        d[j].load(r + k * 8, k < (uint32_t)chunks);
      }
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = h[j].at(i) + d[j].at(i);
        h[j].set(v);
      }
    }
    float h1 = widen_here(x1);
    if (a.r) h1 = round1(x, h1 + widen_here(r1));
    if (a.h) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        if (k < (uint32_t)chunks) {
          if (a.second)
            h[j].template store<false>(ho + k * 8);
          else
            h[j].template store<true>(ho + k * 8);
        }
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
    if (a.rstd && t == 0 && there) a.rstd[row] = rstd;
    if (!outputs || !there) continue;
    const RowOut<In> out(a, row);
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      const bool valid = k < (uint32_t)chunks;
      float g[8], y[8];
      h[j].forget_wide();
      if constexpr (EARLY) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = ge[j][i];
      } else {
        load_gamma(g, a.gamma, a.gamma_bf16, k * 8, valid);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[j].at(i) * rstd * g[i];
      emit<In>(a, out, k * 8, valid, y, tscale, amax);
      __builtin_amdgcn_sched_barrier(0);  // one chunk's binary32 values at a time in registers
    }
    if (t < rest) emit1<In>(a, out, chunks * 8 + t, h1 * rstd * g1, tscale, amax);
  }
  if (a.amax_out) {
    __shared__ uint32_t ured[16];
    finish_amax<BLK>(amax, a.amax_out, ured);
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
  const int chunks = (int)(a.cols / 8), padded = (chunks + 255) / 256 * 256;
  const int c1 = chunks * 8 + threadIdx.x;  // this thread's element after the last whole chunk
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
    const In* x = reinterpret_cast<const In*>(a.x) + row * a.ldx;
    const In* r = reinterpret_cast<const In*>(a.r) + row * a.ldr;
    In* ho = reinterpret_cast<In*>(a.h) + row * a.ldh;
    float ss = 0.0f, h1 = 0.0f;
    for (int k = threadIdx.x; k < chunks; k += 256) {
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
      if (a.h) h.template store<false>(ho + k * 8);
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
    const RowOut<In> out(a, row);
    // every lane takes part in the block maxima, so the count is padded; each
    // thread reads back the chunks that it wrote itself
    for (int k = threadIdx.x; k < padded; k += 256) {
      const bool valid = k < chunks;
      Chunk<In> h;
      float g[8], y[8];
      h.load(hi + k * 8, valid);
      load_gamma(g, a.gamma, a.gamma_bf16, k * 8, valid);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h.at(i) * rstd * g[i];
      emit<In>(a, out, k * 8, valid, y, tscale, amax);
    }
    if (c1 < a.cols) emit1<In>(a, out, c1, h1 * rstd * load_gamma1(a.gamma, a.gamma_bf16, c1), tscale, amax);
  }
  if (a.amax_out) {
    __shared__ uint32_t ured[4];
    finish_amax<256>(amax, a.amax_out, ured);
  }
}

// How a row is held, by its length [measured, us per call, MXFP8 row-wise with a
// residual unless said otherwise]:
//   16 lanes up to 263 columns      32768 x 128 10.2, a wave a row 23.6
//   a wave up to 1031               32768 x 1024 42, a workgroup of 256 78
//   256 threads up to 8199          32768 x 4096 150 (6.2 TB/s), a wave 187, 1024 threads 368
//   512 threads up to 16391         8192 x 12288 133, 256 threads 139
// and longer rows are read twice.  With at most one row a CU a row's own
// latency is all, and 1024 threads take it (64 x 7168: 6.0, 256 threads 7.6;
// at 512 x 4096 256 threads are ahead, 7.1 to 9.0).
// An amax output ends in one atomic per workgroup on one address, which the
// memory side performs one at a time, so its grid is persistent, with 1024
// threads a workgroup up to 4103 columns (32768 x 512 with a given scale: 25.9,
// 256 threads 32.2; 4096 x 8192: 49.7 and 47.3), or twice as many of 512 where
// many long rows keep both busy (16384 x 4096 with both copies: 104, 1024
// threads 109; 1021 x 4096: 14.5 and 12.4); a single workgroup needs no launch
// that clears it first.
template <typename In>
void launch_row(const NormArgs& a, hipStream_t st) {
  const int64_t chunks = a.cols / 8;
  const int tpr = chunks <= 32 ? 16 : chunks <= 128 ? 64 : chunks <= 1024 ? 256 : 512;  // threads a row
  const bool wide = chunks > 256 && a.rows <= 256 && !(a.amax_out && chunks <= 512 && a.rows <= 4);
  const bool large = a.amax_out && !wide && chunks <= 512;
  const int blk = !large ? 256 : tpr == 256 && a.rows > 2048 ? 512 : 1024;
  const int64_t rpw = wide || tpr == 512 ? 1 : blk / tpr;
  int64_t grid = (a.rows + rpw - 1) / rpw;
  const int64_t cap = !a.amax_out ? 1 << 20 : !large ? 1024 : blk == 512 ? 512 : 256;
  if (grid > cap) grid = cap;
  const dim3 g((unsigned)grid);
  if (a.amax_out && grid > 1) launch_fill_u32(a.amax_out, 0u, 1, st);  // one workgroup stores its maximum
#define QSG_ROW(TPR, NCH, BLK) hipLaunchKernelGGL((norm_row_kernel<In, TPR, NCH, BLK>), g, dim3(BLK), 0, st, a)
#define QSG_ROWS(TPR, NCH)                   \
  do {                                       \
    if (blk == 1024) QSG_ROW(TPR, NCH, 1024); \
    else QSG_ROW(TPR, NCH, 256);             \
  } while (0)
  if (chunks <= 16) QSG_ROWS(16, 1);
  else if (chunks <= 32) QSG_ROWS(16, 2);
  else if (chunks <= 64) QSG_ROWS(64, 1);
  else if (chunks <= 128) QSG_ROWS(64, 2);
  else if (chunks <= 256 && blk == 512) QSG_ROW(256, 1, 512);
  else if (chunks <= 256) QSG_ROWS(256, 1);
  else if (wide && chunks <= 1024) QSG_ROW(1024, 1, 1024);
  else if (wide && chunks <= 2048) QSG_ROW(1024, 2, 1024);
  else if (chunks <= 512 && blk == 512) QSG_ROW(256, 2, 512);
  else if (chunks <= 512) QSG_ROWS(256, 2);
  else if (chunks <= 1024) QSG_ROW(256, 4, 256);
  else if (chunks <= 2048) QSG_ROW(512, 4, 512);
  else hipLaunchKernelGGL(norm_long_kernel<In>, g, dim3(256), 0, st, a);  // one row a workgroup, as counted above
#undef QSG_ROWS
#undef QSG_ROW
}

// ---------------------------------------------------------------------------
// second pass: column-wise copies
// ---------------------------------------------------------------------------
// 4 x 4 byte transpose: a..d are four rows of four bytes (byte k = column
// k); o0..o3 are the four columns (byte k = row k).
__device__ __forceinline__ void transpose4x4(uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t (&o)[4]) {
  // v_perm_b32(hi, lo, sel): selector byte values 0-3 pick bytes of lo, 4-7 of hi
  const uint32_t ab01 = __builtin_amdgcn_perm(b, a, 0x05010400u);  // a0 b0 a1 b1
  const uint32_t ab23 = __builtin_amdgcn_perm(b, a, 0x07030602u);  // a2 b2 a3 b3
  const uint32_t cd01 = __builtin_amdgcn_perm(d, c, 0x05010400u);
  const uint32_t cd23 = __builtin_amdgcn_perm(d, c, 0x07030602u);
  o[0] = __builtin_amdgcn_perm(cd01, ab01, 0x05040100u);           // a0 b0 c0 d0
  o[1] = __builtin_amdgcn_perm(cd01, ab01, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(cd23, ab23, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(cd23, ab23, 0x07060302u);
}

// Where tile k of `tile` rows (or columns) begins: the last tile of a matrix
// that is no multiple of it begins earlier and does some of its neighbour's
// work again, with the same result, so that no tile has an edge inside (the
// only tile of a smaller matrix has).
__device__ __forceinline__ int64_t tile_start(int64_t k, int64_t tile, int64_t n) {
  const int64_t at = k * tile;
  return at + tile > n && n > tile ? n - tile : at;
}

constexpr int CT_ROWS = 128;  // rows of a tile: a column's run in qt is 128 bytes, a cache line

// LDS tile of codes: [column][row / 4], one word holds 4 rows; the stride of 33
// words puts the 64 words that a wave writes at once on 64 banks.
constexpr int CT_STRIDE = CT_ROWS / 4 + 1;

// Codes of COLS columns from LDS to qt: 16 rows (16 bytes) a lane, 8 lanes a
// run.  Runs that are whole cache lines stream out; others stay in L2, where
// the run of the tile below completes their lines (rows = 10000: 44 -> 26 us
// for 10000 x 5008; whole lines: streaming is 3-5 % faster).
template <int COLS>
__device__ __forceinline__ void store_columns(const uint32_t* codes, uint8_t* qt, int64_t rows, int64_t cols,
                                              int64_t r0, int64_t c0) {
  const bool lines = rows % 128 == 0 && (uintptr_t)qt % 128 == 0;
#pragma unroll
  for (int k = 0; k < COLS * 8 / 256; ++k) {
    const int id = k * 256 + threadIdx.x, col = id >> 3, r = (id & 7) * 16;
    const uint32_t* w = codes + col * CT_STRIDE + (r >> 2);
    const u32x4 v = {w[0], w[1], w[2], w[3]};
    uint8_t* p = qt + (c0 + col) * rows + r0 + r;
    if (c0 + col < cols) {
      if (r0 + r + 16 <= rows) {
        if (lines)
          put16<true>(p, v);
        else
          put16<false>(p, v);
      } else {
        for (int b = 0; b < 16; ++b)
          if (r0 + r + b < rows) p[b] = (uint8_t)(codes[col * CT_STRIDE + ((r + b) >> 2)] >> (8 * (b & 3)));
      }
    }
  }
}

struct ColArgs {
  const void* h;
  int64_t rows, cols, ld;
  const float* rstd;
  const void* gamma;
  bool gamma_bf16;
  int quant, fmt, margin;
  bool mx_ceil;
  float* three;        // Q_TENSOR, current scaling: {amax, scale, scale_inv}, or null
  const float* scale;  // Q_TENSOR otherwise
  uint8_t* q;          // Q_TENSOR: rows x cols, or null
  uint8_t* qt;         // cols x rows, or null (Q_TENSOR only)
  void* st;
  int64_t tiles_c, tiles, tile0;
};

constexpr int CT_COLS = 64;

// Between a wave's writes to LDS and its lanes' reads of each other's: the
// memory model's order, and no instruction, since a wave's LDS accesses are
// performed in theirs.
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// max(|a|, |b|, |c|, |d|) of values that are not NaN (written out: the compiler
// puts an instruction before each operand to quiet a NaN)
__device__ __forceinline__ float max4_abs(float a, float b, float c, float d) {
  float m;
  asm("v_max3_f32 %0, |%1|, |%2|, |%3|" : "=v"(m) : "v"(a), "v"(b), "v"(c));
  asm("v_max_f32 %0, %1, |%2|" : "=v"(m) : "v"(m), "v"(d));
  return m;
}

// A workgroup makes the column-wise copy of a 128 x 64 tile of y (and, with a
// per-tensor scale, the row-wise one): thread t holds rows 4 (t / 8) .. + 3 of
// chunk t % 8, so that a wave is 32 rows, the rows of an MXFP8 column block.
//
// A column's maximum: each lane's of its 4 rows go through LDS to the lane of
// that column (64 columns, 64 lanes), which alone makes the scale; no barrier
// where the block is the wave's.  The largest |h rstd| is found first and
// multiplied by |gamma| then: rounding keeps order.  Ordinary values skip what only the others
// need (the wave decides): a row whose rstd is positive and finite has finite
// h, so with finite weights y has no NaN; a block whose maximum is finite is
// scaled to at most the format's maximum, up to a rounding that the encode
// takes back, so nothing is clamped; and an MXFP8 scale (a power of two) is
// put into the weight, which changes no bit of a code: with |gamma| <= 2^60
// and a block maximum of 2^-50 at least, gamma 2^-e is neither too large nor
// subnormal (|h rstd| <= sqrt(cols) <= 2^12), and an element of y that is
// subnormal has the code of zero.
//
// What bounds it: the order of its accesses.  It reads 128-byte pieces of rows
// and writes 128-byte pieces of columns; 32768 x 4096 takes 66-71 us, a copy of
// the kernel without its stores 51, without its loads 57, and the vector
// instructions of the waves are 44 % of the cycles.  Tried without gain: 256 or
// 512 rows a tile (81 and 87 us), 2-16 tiles a workgroup with the next one's
// loads in flight (66-76), a tile order by XCD (the whole call 217 -> 221-225),
// 6-8 waves a SIMD.
template <typename In, int QUANT>
__global__ __launch_bounds__(256) void norm_col_kernel(ColArgs a) {
  __shared__ uint32_t codes[CT_COLS * CT_STRIDE];
  __shared__ __attribute__((aligned(16))) uint32_t lane_max[4][8][CT_COLS];
  __shared__ uint32_t part[4][CT_COLS];  // MXFP8: scale bytes [column][wave]; 1 x 128: maxima of the waves
  __shared__ __attribute__((aligned(16))) float cscale[4][CT_COLS];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3, lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  // last rows first: they are the ones that the first pass has left in the caches
  const int64_t tile = a.tiles - 1 - (a.tile0 + blockIdx.x);
  const int64_t r0 = tile_start(tile / a.tiles_c, CT_ROWS, a.rows), c0 = tile_start(tile % a.tiles_c, CT_COLS, a.cols);
  const int64_t r = r0 + ty * 4, c = c0 + tx * 8;
  const bool whole = a.cols >= CT_COLS, full = whole && a.rows >= CT_ROWS;  // no edge in the columns; none at all
  const In* h = reinterpret_cast<const In*>(a.h);
  Chunk<In> v[4];
  float rs[4], g[8];
  if (full) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j].load(h + (r + j) * a.ld + c, true);
#pragma unroll
    for (int j = 0; j < 4; ++j) rs[j] = a.rstd[r + j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rs[j] = 1.0f;
      if (r + j < a.rows) rs[j] = a.rstd[r + j];
    }
    if (whole) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j].load(h + (r + j) * a.ld + c, r + j < a.rows);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = r + j < a.rows && c + i < a.cols ? load1(h + (r + j) * a.ld + c + i) : 0.0f;
        v[j].set(e);
      }
    }
  }
  if (whole) {
    load_gamma(g, a.gamma, a.gamma_bf16, c, true);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = c + i < a.cols ? load_gamma1(a.gamma, a.gamma_bf16, c + i) : 0.0f;
  }
  float smallest = fminf(fminf(rs[0], rs[1]), fminf(rs[2], rs[3])), largest = fmaxf(fmaxf(rs[0], rs[1]), fmaxf(rs[2], rs[3]));
  bool nan = __builtin_isnan(rs[0]) | __builtin_isnan(rs[1]) | __builtin_isnan(rs[2]) | __builtin_isnan(rs[3]);
#pragma unroll
  for (int i = 0; i < 8; ++i) nan |= !(fabsf(g[i]) <= 0x1p60f);
  const bool plain = __all(!nan && smallest > 0.0f && largest <= FLT_MAX);  // no NaN anywhere in the wave's y
  float n[4][8];  // h rstd
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) n[j][i] = v[j].at(i) * rs[j];

  uint32_t cq[8];  // column i: the codes of rows r .. r + 3
  if constexpr (QUANT == Q_TENSOR) {
    float s;
    if (a.three) {
      s = scale_from_amax(a.three[0], fp8_max(a.fmt), a.margin);
      if (a.tile0 + blockIdx.x == 0 && threadIdx.x == 0) {
        a.three[1] = s;
        a.three[2] = __fdiv_rn(1.0f, s);
      }
    } else {
      s = *a.scale;
    }
    u32x2 rq[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = n[j][i] * g[i];
      rq[j] = a.fmt == kE4M3 ? enc8<kE4M3>(y, s) : enc8<kE5M2>(y, s);
      if (a.q) {
        uint8_t* p = a.q + (r + j) * a.cols + c;
        if (whole) {
          if (r + j < a.rows) put8<false>(p, rq[j]);  // half a line: the next tile completes it in L2
        } else if (r + j < a.rows) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < a.cols) p[i] = (uint8_t)(rq[j][i >> 2] >> (8 * (i & 3)));
        }
      }
    }
    if (!a.qt) return;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t o[4];
      transpose4x4(rq[0][k], rq[1][k], rq[2][k], rq[3][k], o);
#pragma unroll
      for (int i = 0; i < 4; ++i) cq[k * 4 + i] = o[i];
    }
  } else {
    uint32_t cm[8];
    if (plain) {
      // rounding keeps order: the largest product is the product of the largest
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cm[i] = __float_as_uint(max4_abs(n[0][i], n[1][i], n[2][i], n[3][i]) * fabsf(g[i]));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cm[i] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) cm[i] = umax_u32(cm[i], abs_bits_canon(__float_as_uint(n[j][i] * g[i])));
      }
    }
    *reinterpret_cast<u32x4*>(&lane_max[wave][ty & 7][tx * 8]) = u32x4{cm[0], cm[1], cm[2], cm[3]};
    *reinterpret_cast<u32x4*>(&lane_max[wave][ty & 7][tx * 8 + 4]) = u32x4{cm[4], cm[5], cm[6], cm[7]};
    wave_lds_order();
    uint32_t m = lane_max[wave][0][lane];
#pragma unroll
    for (int k = 1; k < 8; ++k) m = umax_u32(m, lane_max[wave][k][lane]);
    // m: the maximum of column c0 + lane over the wave's rows
    bool easy;
    if constexpr (QUANT == Q_MX) {
      const int e = mx_exponent(m, a.fmt == kE4M3 ? Fp8Traits<kE4M3>::kEmaxElem : Fp8Traits<kE5M2>::kEmaxElem,
                                a.mx_ceil, a.margin);
      reinterpret_cast<uint8_t*>(&part[0][0])[lane * 4 + wave] = (uint8_t)(e + 127);
      cscale[wave][lane] = pow2_neg(e);
      easy = plain && __all(m >= 0x26800000u && m < 0x7F800000u) && a.mx_ceil;  // 2^-50 <= m < inf
    } else {
      part[wave][lane] = m;
      __syncthreads();
      m = umax_u32(umax_u32(part[0][lane], part[1][lane]), umax_u32(part[2][lane], part[3][lane]));
      const float s = scale_from_amax(__uint_as_float(m), fp8_max(a.fmt), a.margin);
      cscale[wave][lane] = s;
      if (wave == 0 && c0 + lane < a.cols)
        reinterpret_cast<float*>(a.st)[(c0 + lane) * (a.rows / 128) + r0 / 128] = __fdiv_rn(1.0f, s);
      easy = plain && __all(m < 0x7F800000u);
    }
    wave_lds_order();
    float cs[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cs[i] = cscale[wave][tx * 8 + i];
    if (easy) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = QUANT == Q_MX ? n[j][i] * (g[i] * cs[i]) : n[j][i] * g[i] * cs[i];
        cq[i] = a.fmt == kE4M3 ? enc4_inrange<kE4M3>(z[0], z[1], z[2], z[3]) : enc4_inrange<kE5M2>(z[0], z[1], z[2], z[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) z[j] = n[j][i] * g[i] * cs[i];
        cq[i] = a.fmt == kE4M3 ? enc4<kE4M3>(z[0], z[1], z[2], z[3]) : enc4<kE5M2>(z[0], z[1], z[2], z[3]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) codes[(tx * 8 + i) * CT_STRIDE + ty] = cq[i];
  __syncthreads();
  if constexpr (QUANT == Q_MX) {
    if (threadIdx.x < CT_COLS && c0 + threadIdx.x < a.cols) {
      const uint32_t w = part[threadIdx.x >> 6][threadIdx.x & 63];
      uint8_t* p = reinterpret_cast<uint8_t*>(a.st) + (c0 + threadIdx.x) * (a.rows / 32) + r0 / 32;
      if (full) {
        *reinterpret_cast<u32_b*>(p) = w;
      } else {
        for (int k = 0; k < 4; ++k)
          if (r0 + k * 32 < a.rows) p[k] = (uint8_t)(w >> (8 * k));
      }
    }
  }
  store_columns<CT_COLS>(codes, a.qt, a.rows, a.cols, r0, c0);
}

constexpr int TT_COLS = 128;

// qt = q transposed (bytes), 128 x 128 tiles: with a per-tensor scale the
// column-wise copy has the row-wise one's codes, and reading those back costs
// half of reading h.  Thread t holds rows 4 (t / 8) .. + 3 of 16 columns.
__global__ __launch_bounds__(256) void transpose_bytes_kernel(const uint8_t* q, uint8_t* qt, int64_t rows, int64_t cols,
                                                              int64_t tiles_c, int64_t tiles, int64_t tile0) {
  __shared__ uint32_t codes[TT_COLS * CT_STRIDE];
  const int tx = threadIdx.x & 7, ty = threadIdx.x >> 3;
  const int64_t tile = tiles - 1 - (tile0 + blockIdx.x);  // last rows first, as above
  const int64_t r0 = tile_start(tile / tiles_c, CT_ROWS, rows), c0 = tile_start(tile % tiles_c, TT_COLS, cols);
  const int64_t r = r0 + ty * 4, c = c0 + tx * 16;
  u32x4 v[4];
  if (cols >= TT_COLS) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = u32x4{0, 0, 0, 0};
      if (r + j < rows) v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_b*>(q + (r + j) * cols + c));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w = 0;
        for (int b = 0; b < 4; ++b)
          if (r + j < rows && c + k * 4 + b < cols) w |= (uint32_t)q[(r + j) * cols + c + k * 4 + b] << (8 * b);
        v[j][k] = w;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t o[4];
    transpose4x4(v[0][k], v[1][k], v[2][k], v[3][k], o);
#pragma unroll
    for (int i = 0; i < 4; ++i) codes[(tx * 16 + k * 4 + i) * CT_STRIDE + ty] = o[i];
  }
  __syncthreads();
  store_columns<TT_COLS>(codes, qt, rows, cols, r0, c0);
}

constexpr int64_t kMostTiles = 1 << 23;  // of a launch, whose threads are counted in 32 bits

template <typename In>
void launch_col(ColArgs a, hipStream_t st) {
  a.tiles_c = (a.cols + CT_COLS - 1) / CT_COLS;
  a.tiles = (a.rows + CT_ROWS - 1) / CT_ROWS * a.tiles_c;
  for (a.tile0 = 0; a.tile0 < a.tiles; a.tile0 += kMostTiles) {
    const dim3 g((unsigned)(a.tiles - a.tile0 < kMostTiles ? a.tiles - a.tile0 : kMostTiles));
    if (a.quant == Q_TENSOR) hipLaunchKernelGGL((norm_col_kernel<In, Q_TENSOR>), g, dim3(256), 0, st, a);
    else if (a.quant == Q_MX) hipLaunchKernelGGL((norm_col_kernel<In, Q_MX>), g, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((norm_col_kernel<In, Q_BLOCK>), g, dim3(256), 0, st, a);
  }
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

// Sum over the 4 rows of 16 lanes of a wave, lane by lane.
__device__ __forceinline__ float add_groups(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const uint32_t t = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(t, t, false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// [measured, us per call with dgamma] 16384 x 7168 with a residual gradient 165,
// 8192 x 4096 without 41; the sum of the partials takes 4-5 of them.
//
// A group of TPR threads takes rows group, group + groups, ... and holds a
// row in registers, NCH chunks per thread; its share of dgamma stays in
// registers until the end.  WIDE: the rows' dots are read from a.dots, and
// blockIdx.x is the piece of 8 TPR NCH columns (blockIdx.y the group).
template <typename In, int TPR, int NCH, int BLK, bool WIDE>
__global__ __launch_bounds__(BLK) void norm_bwd_kernel(NormBwdArgs a) {
  constexpr int RPW = BLK / TPR;
  constexpr bool JOIN = TPR > 64 && RPW > 1;  // the groups of a workgroup leave one partial
  __shared__ float red[2][16];
  __shared__ float joined[JOIN ? (RPW - 1) * TPR * 8 : 1];
  const int t = threadIdx.x % TPR;
  int sub = threadIdx.x / TPR;
  if constexpr (TPR >= 64) sub = __builtin_amdgcn_readfirstlane(sub);
  const int64_t group = (int64_t)(WIDE ? blockIdx.y : blockIdx.x) * RPW + sub;
  const int64_t groups = (int64_t)(WIDE ? gridDim.y : gridDim.x) * RPW;
  const int64_t c0 = WIDE ? (int64_t)blockIdx.x * (8 * TPR * NCH) : 0;
  const int64_t here = WIDE && a.cols - c0 > 8 * TPR * NCH ? 8 * TPR * NCH : a.cols - c0;  // columns of this piece
  const int all_chunks = (int)(here / 8), all_rest = (int)(here % 8);
  float g[NCH][8], acc[NCH][8], g1 = 0.0f, acc1 = 0.0f;
#pragma unroll
  for (int j = 0; j < NCH; ++j) {
    const uint32_t k = j * TPR + t;
    load_gamma(g[j], a.gamma, a.gamma_bf16, c0 + k * 8, k < (uint32_t)all_chunks);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[j][i] = 0.0f;
  }
  if (t < all_rest) g1 = load_gamma1(a.gamma, a.gamma_bf16, c0 + all_chunks * 8 + t);
  int turn = 0;
  for (int64_t row = group; row - sub < a.rows; row += groups, turn ^= 1) {
    // with barriers in the loop spare threads stay in it, on a row that is not there
    const bool there = RPW == 1 || row < a.rows;
    if (TPR <= 64 && !there) break;
    const int chunks = there ? all_chunks : 0, rest = there ? all_rest : 0;
    const In* pdy = reinterpret_cast<const In*>(a.dy) + row * a.lddy + c0;
    const In* ph = reinterpret_cast<const In*>(a.h) + row * a.ldh + c0;
    const In* pdr = reinterpret_cast<const In*>(a.dres) + row * a.lddres + c0;
    In* pdx = reinterpret_cast<In*>(a.dx) + row * a.lddx + c0;
    Chunk<In> dy[NCH], h[NCH], dr[NCH];
    In dy1r = 0, h1r = 0, dr1r = 0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      dy[j].load(pdy + k * 8, k < (uint32_t)chunks);
      h[j].load(ph + k * 8, k < (uint32_t)chunks);
    }
    if (t < rest) {
      dy1r = pdy[chunks * 8 + t];
      h1r = ph[chunks * 8 + t];
    }
    if (a.dres) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        const uint32_t k = j * TPR + t;
        dr[j].load(pdr + k * 8, k < (uint32_t)chunks);
      }
      if (t < rest) dr1r = pdr[chunks * 8 + t];
    }
    const float rstd = there ? a.rstd[row] : 0.0f;
    const float dy1 = widen_here(dy1r), h1 = widen_here(h1r), dr1 = widen_here(dr1r);
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
      dy[j].forget_wide();
      h[j].forget_wide();
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
        o.template store<true>(pdx + k * 8);
      }
    }
    if (t < rest) {
      const float n = h1 * rstd;
      acc1 = fmaf(dy1, n, acc1);
      store1(pdx + chunks * 8 + t, fmaf(rstd, fmaf(-n, m, dy1 * g1), dr1));
    }
  }
  if (a.partial) {
    int64_t slot = group;
    if constexpr (TPR == 16) {
      // the 4 groups of a wave leave one partial
#pragma unroll
      for (int j = 0; j < NCH; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[j][i] = add_groups(acc[j][i]);
      acc1 = add_groups(acc1);
      if ((threadIdx.x & 63) >= 16) return;
      slot = group / 4;
    }
    if constexpr (JOIN) {
#pragma unroll
      for (int j = 0; j < NCH; ++j) {
        if (sub > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) joined[((sub - 1) * 8 + i) * TPR + t] = acc[j][i];
        }
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int k = 0; k < RPW - 1; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[j][i] += joined[(k * 8 + i) * TPR + t];
        }
        __syncthreads();
      }
      if (sub > 0) joined[(sub - 1) * TPR + t] = acc1;
      __syncthreads();
      if (sub > 0) return;
#pragma unroll
      for (int k = 0; k < RPW - 1; ++k) acc1 += joined[k * TPR + t];
      slot = blockIdx.x;
    }
    const int chunks = all_chunks, rest = all_rest;
    float* p = a.partial + slot * a.cols + c0;
#pragma unroll
    for (int j = 0; j < NCH; ++j) {
      const uint32_t k = j * TPR + t;
      if (k < (uint32_t)chunks) {
        Chunk<float> o;
        o.set(acc[j]);
        o.template store<false>(p + k * 8);
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

template <int CTRL>
__device__ __forceinline__ double dpp_add(double v) {
  return v + __hiloint2double((int)dpp_u32<CTRL>((uint32_t)__double2hiint(v)), (int)dpp_u32<CTRL>((uint32_t)__double2loint(v)));
}

// Sum over 32 lanes, the same in each, by the steps of lane_sum (shuffles, which
// pass through LDS: dgamma of 333 rows by 1111 columns 5.4 us).
__device__ __forceinline__ double half_wave_sum(double v) {
  v = dpp_add<kDppXor1>(v);
  v = dpp_add<kDppXor2>(v);
  v = dpp_add<kHalfMirror>(v);
  v = dpp_add<kMirror>(v);
  const uint32_t lo = (uint32_t)__double2loint(v), hi = (uint32_t)__double2hiint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto b = __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  return __hiloint2double((int)b[0], (int)a[0]) + __hiloint2double((int)b[1], (int)a[1]);
}

// dgamma[c] (+)= sum over groups of partial[group][c], in a fixed order: a
// workgroup takes 32 columns, 8 lanes of 4 columns by 128 parts of the groups;
// then a half wave takes a column, 4 parts a lane, and adds its lanes pairwise.
// All of it is binary64, rounded once: there are up to 4096 partials, and of
// small ones beside a large one a binary32 chain keeps none.
__global__ __launch_bounds__(1024) void norm_dgamma_kernel(const float* partial, int64_t groups, int64_t cols,
                                                          float* dgamma, bool accumulate) {
  constexpr int PARTS = 128;
  __shared__ double sum[PARTS][33];
  const int lane = threadIdx.x & 7, part = threadIdx.x >> 3;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane * 4;
  double v[4] = {0.0, 0.0, 0.0, 0.0};
  if (c + 4 <= cols) {
#pragma unroll 8
    for (int64_t k = part; k < groups; k += PARTS) {
      const u32x4 u = *reinterpret_cast<const u32x4_e*>(partial + k * cols + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += __uint_as_float(u[i]);
    }
  } else {
    for (int64_t k = part; k < groups; k += PARTS)
      for (int i = 0; i < 4; ++i)
        if (c + i < cols) v[i] += partial[k * cols + c + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[part][lane * 4 + i] = v[i];
  __syncthreads();
  const int p = threadIdx.x & 31, col = threadIdx.x >> 5;
  double s = (sum[p][col] + sum[p + 32][col]) + (sum[p + 64][col] + sum[p + 96][col]);
  s = half_wave_sum(s);
  const int64_t at = (int64_t)blockIdx.x * 32 + col;
  if (p == 0 && at < cols) dgamma[at] = (float)(accumulate ? dgamma[at] + s : s);
}

constexpr int64_t kBwdMostCols = 16391;  // of a row held in registers: 2048 chunks and 7 elements
constexpr int64_t kBwdPiece = 2048;      // columns of a workgroup beyond that

// How a backward pass shares its rows: a workgroup of `blk` threads takes
// blk / tpr rows at a time, and `partials` sums of dgamma are left (4 bytes a
// column each, written and read again): one per workgroup, or per wave where
// rows are a wave's or less.
struct BwdPlan {
  int tpr, blk;
  int64_t grid, partials;
};

// The last shapes of each kind stand in rmsnorm_bwd_workspace too.
BwdPlan bwd_plan(int64_t rows, int64_t cols) {
  const int64_t chunks = cols / 8;
  BwdPlan p;
  p.tpr = chunks <= 32 ? 16 : chunks <= 64 ? 64 : chunks <= 1024 ? 256 : chunks <= 2048 ? 1024 : 256;
  p.blk = p.tpr == 1024 ? 1024 : 256;
  // about as many workgroups as the card holds at once
  int64_t most = chunks <= 32 ? 512 : chunks <= 512 ? 1024 : chunks <= 1024 ? 512 : chunks <= 2048 ? 256 : 128;
  // Two or four rows to a workgroup, which adds their shares of dgamma in LDS:
  // less to write and read again, for a barrier that the rows share.
  // [measured, us a call in a graph with a residual gradient, one / two / four
  // rows]
  //   rows   1024 columns          2048                  4096                  7168
  //    256    6.1 /  6.2 /  6.7     7.2 /  7.0 /  7.3     8.6 /  8.6 /  9.5    12.6 / 11.7
  //    384    7.1 /  6.8 /  7.2     8.6 /  7.4 /  7.6    11.2 /  9.8 / 10.0    16.0 / 13.4
  //    640    8.4 /  7.6 /  7.6    10.2 /  8.7 /  8.2    15.0 / 12.0 / 11.0
  //   1024    9.4 /  8.8 /  8.1    13.1 / 10.3 /  8.9    20.7 / 15.1 / 13.0    23.5 / 21.0
  //   1280   10.2 /  9.3 / 11.0    13.3 / 11.2 / 12.5    21.9 / 17.3 / 19.1    25.6 / 24.8
  //   2048   11.5 / 10.2 / 12.3    15.5 / 13.2 / 15.1    25.6 / 20.6 / 23.1    31.8 / 31.6
  //   8192   20.7 / 20.5 / 23.7    31.4 / 28.8 / 32.7
  //  32768   56.0 / 59.7 / 66.7    96.7 / 94.0 / 97.8
  // Around 160 chunks, one / two rows: 1280 columns 16384 rows 36.6 / 36.5,
  // 20000 42.1 / 42.4, 32768 64.5 / 64.6; 1288 columns 38.7 / 37.0, 44.7 / 43.0,
  // 68.2 / 65.5.  The borders are coarse: four rows stay up to 1280 where two
  // are ahead from 1025 on, and one row beyond 1280 at 7168 columns where two
  // are ahead by 4 % up to 1536.
  if (p.tpr == 256 && rows >= 384) {
    if (chunks <= 512 && rows <= 1280) {
      p.blk = 1024;
      most = 512;
    } else if (chunks <= 512 && (chunks > 160 || rows <= 16384)) {
      p.blk = 512;
      most = 512;
    } else if (chunks > 512 && chunks <= 1024 && rows <= 1280) {
      p.blk = 512;
      most = 256;
    }
  }
  const int64_t rpw = p.blk / p.tpr;
  p.grid = (rows + rpw - 1) / rpw;
  if (p.grid > most) p.grid = most;
  p.partials = p.tpr <= 64 ? p.grid * 4 : p.grid;
  return p;
}

template <typename In>
void launch_bwd(const NormBwdArgs& a, const BwdPlan& p, hipStream_t st) {
  const int64_t chunks = a.cols / 8;
  const dim3 g((unsigned)p.grid);
#define QSG_BWD(TPR, NCH, BLK) hipLaunchKernelGGL((norm_bwd_kernel<In, TPR, NCH, BLK, false>), g, dim3(BLK), 0, st, a)
  if (chunks <= 16) QSG_BWD(16, 1, 256);
  else if (chunks <= 32) QSG_BWD(16, 2, 256);
  else if (chunks <= 64) QSG_BWD(64, 1, 256);
  else if (chunks <= 256 && p.blk == 1024) QSG_BWD(256, 1, 1024);
  else if (chunks <= 256 && p.blk == 512) QSG_BWD(256, 1, 512);
  else if (chunks <= 256) QSG_BWD(256, 1, 256);
  else if (chunks <= 512 && p.blk == 1024) QSG_BWD(256, 2, 1024);
  else if (chunks <= 512 && p.blk == 512) QSG_BWD(256, 2, 512);
  else if (chunks <= 512) QSG_BWD(256, 2, 256);
  else if (chunks <= 1024 && p.blk == 512) QSG_BWD(256, 4, 512);
  else if (chunks <= 1024) QSG_BWD(256, 4, 256);
  else if (chunks <= 2048) QSG_BWD(1024, 2, 1024);
  else {
    const int64_t n = a.rows < 4096 ? a.rows : 4096;
    hipLaunchKernelGGL(norm_bwd_dot_kernel<In>, dim3((unsigned)n), dim3(256), 0, st, a);
    const int64_t pieces = (a.cols + kBwdPiece - 1) / kBwdPiece;
    hipLaunchKernelGGL((norm_bwd_kernel<In, 256, 1, 256, true>), dim3((unsigned)pieces, (unsigned)p.grid), dim3(256), 0,
                       st, a);
  }
#undef QSG_BWD
}

}  // namespace

void launch_rmsnorm_quantize(const void* x, const void* r, int dtype, int64_t rows, int64_t cols, int64_t ldx,
                             int64_t ldr, const void* gamma, int gamma_dtype, float eps, int scaling, int fmt,
                             int margin, bool mx_ceil, const float* scale, void* h, int64_t ldh, float* rstd, void* y,
                             uint8_t* q, void* s, uint8_t* qt, void* st_, float* amax_out, hipStream_t st) {
  const bool tensorwise = scaling == 0;
  float* three = reinterpret_cast<float*>(s);
  float* amax = tensorwise ? three : amax_out;
  if (rows == 0 || cols == 0) {
    if (amax) launch_fill_u32(reinterpret_cast<uint32_t*>(amax), 0u, 1, st);
    if (tensorwise) launch_compute_scale(three, fmt, margin, three + 1, three + 2, st);
    return;
  }
  // The first pass has whole rows: h, rstd, y, and the row-wise copy except
  // under the current scaling, whose scale needs the whole tensor's amax.  The
  // second has tiles: the column-wise copy from h, or from q where both copies
  // share one given scale.
  const int quant = scaling < 0 ? Q_NONE : scaling < 2 ? Q_TENSOR : scaling == 2 ? Q_MX : Q_BLOCK;
  NormArgs a{};
  a.x = x; a.r = r;
  a.rows = rows; a.cols = cols; a.ldx = ldx; a.ldr = ldr; a.ldh = ldh;
  a.gamma = gamma; a.gamma_bf16 = gamma_dtype == 1;
  a.eps = eps;
  a.h = h; a.rstd = rstd; a.y = y;
  a.fmt = fmt; a.margin = margin; a.mx_ceil = mx_ceil;
  a.scale = scale; a.s = s;
  if (q && !tensorwise) {
    a.quant = quant;
    a.q = q;
  }
  a.amax_out = reinterpret_cast<uint32_t*>(amax);
  a.again = scaling == 1 && q && qt;
  a.second = (qt || tensorwise) && !a.again;
  if (dtype == 1)
    launch_row<uint16_t>(a, st);
  else
    launch_row<float>(a, st);
  if (!qt && !tensorwise) return;
  if (a.again) {
    const int64_t tc = (cols + TT_COLS - 1) / TT_COLS, tiles = (rows + CT_ROWS - 1) / CT_ROWS * tc;
    for (int64_t at = 0; at < tiles; at += kMostTiles)
      hipLaunchKernelGGL(transpose_bytes_kernel, dim3((unsigned)(tiles - at < kMostTiles ? tiles - at : kMostTiles)),
                         dim3(256), 0, st, q, qt, rows, cols, tc, tiles, at);
    return;
  }
  ColArgs k{};
  k.h = h ? h : x; k.ld = h ? ldh : ldx;
  k.rows = rows; k.cols = cols;
  k.rstd = rstd; k.gamma = gamma; k.gamma_bf16 = a.gamma_bf16;
  k.quant = quant; k.fmt = fmt; k.margin = margin; k.mx_ceil = mx_ceil;
  k.three = tensorwise ? three : nullptr; k.scale = scale;
  k.q = tensorwise ? q : nullptr;
  k.qt = qt; k.st = st_;
  if (dtype == 1)
    launch_col<uint16_t>(k, st);
  else
    launch_col<float>(k, st);
}

// A workspace serves every shape with no more rows and no more columns, while a
// plan may leave fewer partials of a larger shape (rows joined, fewer groups of
// longer rows): the most that any such shape needs.  The need grows within each
// kind of plan, so its value at the kinds' last shapes and at this one is all.
int64_t rmsnorm_bwd_workspace(int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return 0;
  const int64_t row_ends[] = {383, 1280, 16384, rows};
  const int64_t col_ends[] = {263, 519, 1287, 4103, 8199, kBwdMostCols, cols};
  int64_t most = 0;
  for (const int64_t c : col_ends) {
    if (c > cols) continue;
    for (const int64_t r : row_ends) {
      if (r > rows) continue;
      const int64_t need = bwd_plan(r, c).partials * c + (c > kBwdMostCols ? r : 0);
      if (need > most) most = need;
    }
  }
  return most * 4;
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
  const BwdPlan p = bwd_plan(rows, cols);
  float* ws = reinterpret_cast<float*>(workspace);
  NormBwdArgs a{};
  a.dy = dy; a.h = h; a.dres = dres;
  a.rows = rows; a.cols = cols; a.lddy = lddy; a.ldh = ldh; a.lddres = lddres; a.lddx = lddx;
  a.gamma = gamma; a.gamma_bf16 = gamma_dtype == 1;
  a.rstd = rstd; a.dx = dx;
  a.partial = dgamma ? ws : nullptr;
  a.dots = ws + p.partials * cols;
  if (dtype == 1)
    launch_bwd<uint16_t>(a, p, st);
  else
    launch_bwd<float>(a, p, st);
  if (dgamma)
    hipLaunchKernelGGL(norm_dgamma_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, st, ws, p.partials, cols,
                       dgamma, accumulate);
}

}  // namespace qsg
