// INT8 copies of a matrix and the gated activation that keeps its input in
// INT8 for the backward pass.
//
// Values whose largest magnitude is amax share a scale:
//   s = max(fp32(amax / 127), 2^-126)   (1 for amax 0, NaN for one not finite)
//   code = rint(fp32(v * fp32(1 / s))), and a code stands for code * s.
// A row (a token) shares one, a column (a channel) of the transposed copy, or
// a block of 128 neighbours of the kept activations.
#include <hip/hip_runtime.h>

#include "qsg_device.h"
#include "qsg_internal.h"

namespace qsg {

namespace {

// Vectors that ask for the alignment of an element only: gfx950 loads and
// stores them at any address, so odd leading dimensions take the same path.
typedef uint32_t u32x4_e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_b __attribute__((ext_vector_type(4), aligned(1)));
typedef uint32_t u32x2_b __attribute__((ext_vector_type(2), aligned(1)));

constexpr int kBlock = 128;  // neighbours that share a scale of the kept activations

__device__ __forceinline__ float widen(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16x2(v, 0.0f); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }

// 8 consecutive values, of which the first n (0..8) are there; the rest are 0.
// ONCE: nothing reads them again.
template <bool ONCE = true>
__device__ __forceinline__ void load8(float (&v)[8], const uint16_t* p, int n) {
  if (n >= 8) {
    const u32x4 u = ONCE ? __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p))
                         : *reinterpret_cast<const u32x4_e*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? widen(p[i]) : 0.0f;
  }
}
template <bool ONCE = true>
__device__ __forceinline__ void load8(float (&v)[8], const float* p, int n) {
  if (n >= 8) {
    const u32x4 a = *reinterpret_cast<const u32x4_e*>(p), b = *reinterpret_cast<const u32x4_e*>(p + 4);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8], int n) {
  const u32x4 u = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
  if (n >= 8) {
    __builtin_nontemporal_store(u, reinterpret_cast<u32x4_e*>(p));
  } else {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8], int n) {
  if (n >= 8) {
    const u32x4 a = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    const u32x4 b = {__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
    *reinterpret_cast<u32x4_e*>(p) = a;
    *reinterpret_cast<u32x4_e*>(p + 4) = b;
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8(int8_t* p, u32x2 c, int n) {
  if (n >= 8) {
    __builtin_nontemporal_store(c, reinterpret_cast<u32x2_b*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (int8_t)(c[i >> 2] >> (8 * (i & 3)));
  }
}

// 8 consecutive values as they lie in memory.
template <typename In>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 w;
  __device__ __forceinline__ void load(const uint16_t* p, bool there) {
    w = u32x4{0, 0, 0, 0};
    if (there) w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_e*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (i & 1) ? bf16hi(w[i >> 1]) : bf16lo(w[i >> 1]);
  }
  // new values to the compiler, which would otherwise keep the 8 widened ones
  // of an earlier use beside them (56 -> 88 registers; 8192 x 14336: 61 -> 76 us)
  __device__ __forceinline__ void forget() { asm("" : "+v"(w)); }
};
template <>
struct Raw<float> {
  float v_[8];
  __device__ __forceinline__ void load(const float* p, bool there) { load8(v_, p, there ? 8 : 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v_[i];
  }
  __device__ __forceinline__ void forget() {}
};

// how many of the 8 values from c on are inside a row
__device__ __forceinline__ int left8(int64_t cols, int64_t c) {
  const int64_t n = cols - c;
  return n < 0 ? 0 : (n < 8 ? (int)n : 8);
}

// largest magnitude as a bit pattern: infinity and every NaN are larger than
// any finite one
__device__ __forceinline__ uint32_t amax8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax_u32(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return m;
}

struct Scale {
  float s, inv;
  uint32_t keep;  // 0 where the codes are 0 because the maximum is not finite
};
__device__ __forceinline__ Scale scale_of(uint32_t amax) {
  Scale r;
  r.keep = amax < 0x7F800000u ? ~0u : 0u;
  const float q = __fdiv_rn(__uint_as_float(amax), 127.0f);
  r.s = amax == 0 ? 1.0f : fmaxf(q, 0x1p-126f);
  r.inv = __fdiv_rn(1.0f, r.s);
  if (!r.keep) {
    r.s = __uint_as_float(0x7FC00000u);
    r.inv = 0.0f;
  }
  return r;
}
// the same of a scale that is in memory
__device__ __forceinline__ Scale scale_again(float s) {
  Scale r;
  r.s = s;
  r.keep = s == s ? ~0u : 0u;
  r.inv = r.keep ? __fdiv_rn(1.0f, s) : 0.0f;
  return r;
}

// rint(fp32(v * inv)) in the low byte: adding 1.5 * 2^23 rounds to a whole
// number, ties to even, whose two's complement is the sum's lowest bits (the
// product and the sum are rounded apart, so they may not become one fma)
__device__ __forceinline__ uint32_t code_of(float v, float inv) {
#pragma clang fp contract(off)
  const float p = v * inv;
  return __float_as_uint(p + 12582912.0f);
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, const Scale& s) {
  const uint32_t lo = __builtin_amdgcn_perm(code_of(b, s.inv), code_of(a, s.inv), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(code_of(d, s.inv), code_of(c, s.inv), 0x04000c0cu);
  return (lo | hi) & s.keep;
}
__device__ __forceinline__ u32x2 codes8(const float (&v)[8], const Scale& s) {
  return u32x2{codes4(v[0], v[1], v[2], v[3], s), codes4(v[4], v[5], v[6], v[7], s)};
}

// Maximum over the TPR threads (consecutive ones of the workgroup) that share
// a row.  For TPR > 64 every thread of the workgroup calls it together.
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
  if constexpr (TPR < 64) {
    static_assert(TPR == 16, "groups of a row of lanes");
    return group_max_u32<0xF>(m);
  } else {
    m = wave_max_u32(m);
    if constexpr (TPR > 64) {
      constexpr int W = TPR / 64;
      if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
      __syncthreads();
      red += threadIdx.x / TPR * W;
      m = red[0];
#pragma unroll
      for (int i = 1; i < W; ++i) m = umax_u32(m, red[i]);
    }
    return m;
  }
}

// ---------------------------------------------------------------------------
// row-wise copy
// ---------------------------------------------------------------------------
struct QuantArgs {
  const void* x;
  int64_t rows, cols, ld;
  int8_t* q;   // or null
  float* s;
  int8_t* qt;  // or null
  float* st;
  float* part;  // column maxima of groups of rows
  int parts;
  int64_t tile0;  // first tile of a launch of int8_col_kernel, group of 64 columns of int8_colscale_kernel
};

// A row in the registers of TPR threads, CH chunks of 8 values each; the up to
// 7 values behind the last whole chunk go one to a thread.  Bound by memory, x
// read once and its codes written: 32768 x 4096 bf16 in 62-64 us (6.4 TB/s), 32768
// x 1111 in 22, one row of 4096 in 2.8.
template <typename In, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void int8_row_kernel(QuantArgs a) {
  constexpr int NT = TPR < 256 ? 256 : TPR;
  __shared__ uint32_t red[NT / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (NT / TPR) + threadIdx.x / TPR;
  const bool there = row < a.rows;
  const In* x = reinterpret_cast<const In*>(a.x) + (there ? row * a.ld : 0);
  const int cols = there ? (int)a.cols : 0, whole = cols & ~7;
  Raw<In> raw[CH];
  float v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i) raw[i].load(x + (i * TPR + t) * 8, (i * TPR + t) * 8 < whole);
  const float tail = whole + t < cols ? widen(x[whole + t]) : 0.0f;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    raw[i].get(v);
    m = amax8(v, m);
    raw[i].forget();
  }
  m = umax_u32(m, __float_as_uint(tail) & 0x7FFFFFFFu);
  const Scale s = scale_of(row_max<TPR>(m, red));
  if (!there) return;
  int8_t* q = a.q + row * a.cols;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    raw[i].get(v);
    if ((i * TPR + t) * 8 < whole) store8(q + (i * TPR + t) * 8, codes8(v, s), 8);
  }
  if (whole + t < cols) q[whole + t] = (int8_t)(code_of(tail, s.inv) & s.keep);
  if (t == 0) a.s[row] = s.s;
}

// Rows that are too long for registers are read twice (4096 x 28672 bf16 in 95
// us this way, in 58 from registers; rows of 40000 have no other).
template <typename In>
__global__ __launch_bounds__(1024) void int8_long_row_kernel(QuantArgs a) {
  __shared__ uint32_t red[16];
  const In* x = reinterpret_cast<const In*>(a.x) + (int64_t)blockIdx.x * a.ld;
  int8_t* q = a.q + (int64_t)blockIdx.x * a.cols;
  float v[8];
  uint32_t m = 0;
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
    load8(v, x + c, left8(a.cols, c));
    m = amax8(v, m);
  }
  const Scale s = scale_of(row_max<1024>(m, red));
  for (int64_t c = threadIdx.x * 8; c < a.cols; c += 8192) {
    const int n = left8(a.cols, c);
    load8(v, x + c, n);
    store8(q + c, codes8(v, s), n);
  }
  if (threadIdx.x == 0) a.s[blockIdx.x] = s.s;
}

// The row-wise copy with the columns' maxima of the transposed one: the TPR
// threads of a row (a wave each, or the workgroup) take rows in turn, keep the
// maxima of a thread's columns in registers, and leave the workgroup's as one
// part.  The next row is loaded while a row is worked on.  Plain loads: the
// second pass reads x again, and what is still in the cache then comes from
// there.  Both copies of 14336 x 4096 fp32 in 111 us, against 168 with a pass of
// its own for the maxima; of 32768 x 1024 fp32 in 67 against 87, of 32768 x 2048
// bf16 in 110 against 113.
template <typename In, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void int8_row_col_kernel(QuantArgs a) {
  constexpr int NT = TPR < 256 ? 256 : TPR, PER = NT / TPR;
  static_assert(PER == 1 || TPR == 64, "a wave, or all of the workgroup");
  __shared__ uint32_t red[2][TPR > 64 ? TPR / 64 : 1];
  __shared__ uint32_t join[PER > 1 ? PER - 1 : 1][PER > 1 ? CH * TPR * 8 : 1];
  const int t = threadIdx.x % TPR, at = threadIdx.x / TPR, cols = (int)a.cols;
  uint32_t m[CH][8] = {};
  float v[CH][8], w[CH][8];
  auto load = [&](float (&d)[CH][8], int64_t row) {
    const In* x = reinterpret_cast<const In*>(a.x) + row * a.ld;
#pragma unroll
    for (int i = 0; i < CH; ++i) load8<false>(d[i], x + (i * TPR + t) * 8, row < a.rows ? cols - (i * TPR + t) * 8 : 0);
  };
  int turn = 0;
  auto work = [&](const float (&d)[CH][8], int64_t row) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t b = __float_as_uint(d[i][k]) & 0x7FFFFFFFu;
        m[i][k] = umax_u32(m[i][k], b);
        top = umax_u32(top, b);
      }
    const Scale s = scale_of(row_max<TPR>(top, red[turn]));
    turn ^= 1;
    int8_t* q = a.q + row * a.cols;
#pragma unroll
    for (int i = 0; i < CH; ++i) store8(q + (i * TPR + t) * 8, codes8(d[i], s), cols - (i * TPR + t) * 8);
    if (t == 0) a.s[row] = s.s;
  };
  const int64_t stride = (int64_t)a.parts * PER;
  int64_t row = (int64_t)blockIdx.x * PER + at;
  load(v, row);
  for (; row < a.rows; row += 2 * stride) {
    load(w, row + stride);
    work(v, row);
    if (row + stride >= a.rows) break;
    load(v, row + 2 * stride);
    work(w, row + stride);
  }
  if constexpr (PER > 1) {
    if (at > 0) {
#pragma unroll
      for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) join[at - 1][(i * 8 + k) * TPR + t] = m[i][k];
    }
    __syncthreads();
    if (at > 0) return;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int o = 0; o < PER - 1; ++o) m[i][k] = umax_u32(m[i][k], join[o][(i * 8 + k) * TPR + t]);
  }
  uint32_t* part = reinterpret_cast<uint32_t*>(a.part) + blockIdx.x * a.cols;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if ((i * TPR + t) * 8 + k < cols) part[(i * TPR + t) * 8 + k] = m[i][k];
}

// ---------------------------------------------------------------------------
// transposed copy: the columns' maxima, their scales, the codes
// ---------------------------------------------------------------------------
constexpr int kMostParts = 512;

// Maxima of 512 columns over a part of the rows: a wave reads a row's 512
// columns at a time, the waves take rows in turn.
template <typename In>
__global__ __launch_bounds__(256) void int8_colmax_kernel(QuantArgs a) {
  __shared__ uint32_t red[4][512];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 512 + lane * 8;
  const int n = left8(a.cols, c);
  uint32_t m[8] = {};
  for (int64_t r = (int64_t)blockIdx.y * 4 + wave; r < a.rows; r += (int64_t)a.parts * 4) {
    float v[8];
    load8(v, reinterpret_cast<const In*>(a.x) + r * a.ld + c, n);
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = umax_u32(m[i], __float_as_uint(v[i]) & 0x7FFFFFFFu);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[wave][lane * 8 + i] = m[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int64_t col = (int64_t)blockIdx.x * 512 + i;
    if (col < a.cols)
      reinterpret_cast<uint32_t*>(a.part)[(int64_t)blockIdx.y * a.cols + col] =
          umax_u32(umax_u32(red[0][i], red[1][i]), umax_u32(red[2][i], red[3][i]));
  }
}

// 64 columns a workgroup, 16 waves over the parts, 8 loads of a wave in flight
__global__ __launch_bounds__(1024) void int8_colscale_kernel(QuantArgs a) {
  __shared__ uint32_t red[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = (a.tile0 + blockIdx.x) * 64 + lane;
  const uint32_t* p = reinterpret_cast<const uint32_t*>(a.part) + (col < a.cols ? col : a.cols - 1);
  uint32_t m = 0;
  for (int k = wave; k < a.parts; k += 128) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = p[(int64_t)(k + 16 * i < a.parts ? k + 16 * i : k) * a.cols];
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax_u32(m, v[i]);
  }
  red[wave][lane] = m;
  __syncthreads();
  if (wave == 0 && col < a.cols) {
#pragma unroll
    for (int w = 1; w < 16; ++w) m = umax_u32(m, red[w][lane]);
    a.st[col] = scale_of(m).s;
  }
}

// A tile of 128 rows x 64 columns: a thread encodes 4 rows x 8 columns and
// puts each column's 4 codes into LDS as one word; a column's 128 codes then
// leave as one run of 8 lanes.  Bound by reading x a second time: of the 111 us
// of both copies of 14336 x 4096 fp32 this pass takes half.
constexpr int kColRow = 33;  // words of an LDS column: 32, and one that spreads the banks
template <typename In>
__global__ __launch_bounds__(256) void int8_col_kernel(QuantArgs a) {
  __shared__ uint32_t tile[64 * kColRow];
  const int64_t tile_rows = (a.rows + 127) / 128, tile_cols = (a.cols + 63) / 64;
  // the last rows first: the pass before read them last
  const int64_t at = tile_rows * tile_cols - 1 - (a.tile0 + blockIdx.x);
  const int64_t r0 = at / tile_cols * 128, c0 = at % tile_cols * 64;
  const int ch = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int64_t c = c0 + ch * 8;
  const int n = left8(a.cols, c);
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + rg * 4 + i;
    load8(v[i], reinterpret_cast<const In*>(a.x) + (r < a.rows ? r * a.ld : 0) + c, r < a.rows ? n : 0);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k < n) {
      const Scale s = scale_again(a.st[c + k]);
      tile[(ch * 8 + k) * kColRow + rg] = codes4(v[0][k], v[1][k], v[2][k], v[3][k], s);
    }
  }
  __syncthreads();
  const int64_t r = r0 + (threadIdx.x & 7) * 16;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int col = (threadIdx.x >> 3) + k * 32;
    if (c0 + col >= a.cols || r >= a.rows) continue;
    const uint32_t* w = tile + col * kColRow + (threadIdx.x & 7) * 4;
    int8_t* p = a.qt + (c0 + col) * a.rows + r;
    if (r + 16 <= a.rows) {
      const u32x4 u = {w[0], w[1], w[2], w[3]};
      *reinterpret_cast<u32x4_b*>(p) = u;
    } else {
      const int left = (int)(a.rows - r);
      for (int i = 0; i < left; ++i) p[i] = (int8_t)(w[i >> 2] >> (8 * (i & 3)));
    }
  }
}

// The threads of a launch are counted in 32 bits: what has more workgroups than
// this is launched in pieces.
constexpr int64_t kMostGroups = 1 << 21;

// f(first row, rows of the launch), with `per` rows to a workgroup
template <typename F>
void in_pieces(int64_t rows, int64_t per, F f) {
  for (int64_t r = 0; r < rows; r += kMostGroups * per) f(r, rows - r < kMostGroups * per ? rows - r : kMostGroups * per);
}

template <typename In, int TPR, int CH>
void launch_rows(const QuantArgs& all, hipStream_t st) {
  constexpr int NT = TPR < 256 ? 256 : TPR, PER = NT / TPR;
  in_pieces(all.rows, PER, [&](int64_t r, int64_t n) {
    QuantArgs a = all;
    a.x = reinterpret_cast<const In*>(all.x) + r * all.ld;
    a.q += r * all.cols;
    a.s += r;
    a.rows = n;
    if constexpr (CH > 0)
      hipLaunchKernelGGL((int8_row_kernel<In, TPR, CH>), dim3((unsigned)((n + PER - 1) / PER)), dim3(NT), 0, st, a);
    else
      hipLaunchKernelGGL(int8_long_row_kernel<In>, dim3((unsigned)n), dim3(NT), 0, st, a);
  });
}

template <typename In>
void launch_quantize(const QuantArgs& a, hipStream_t st) {
  // both copies of rows that fit registers: one pass for the rows and the
  // columns' maxima
  const bool fused = a.q && a.qt && a.rows > 0 && a.cols <= 16384;
  if (fused) {
    auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, dim3(a.parts), dim3(threads), 0, st, a); };
    if (a.cols <= 512) go(int8_row_col_kernel<In, 64, 1>, 256);
    else if (a.cols <= 1024) go(int8_row_col_kernel<In, 64, 2>, 256);
    else if (a.cols <= 2048) go(int8_row_col_kernel<In, 64, 4>, 256);
    else if (a.cols <= 4096) go(int8_row_col_kernel<In, 512, 1>, 512);
    else if (a.cols <= 8192) go(int8_row_col_kernel<In, 512, 2>, 512);
    else go(int8_row_col_kernel<In, 1024, 2>, 1024);
  } else if (a.s) {  // by the scales: an empty copy may have no address
    // as few threads as hold a row with 4 chunks each (32768 x 4096 bf16: 64 us,
    // with one chunk 75; 8192 x 12000: 50 and, with two, 55; 4096 x 28672: 58 and,
    // read twice, 95); narrow rows fewer of them, which chunks past the end cost
    // more than they hide (32768 x 700: 15 us with two, 16.5 with four; 100000 x
    // 300: 26 with one, 34; 32768 x 256: 6.2 with 16 threads a row, 9.1 with 64)
    if (a.cols <= 256) launch_rows<In, 16, 2>(a, st);
    else if (a.cols <= 512) launch_rows<In, 64, 1>(a, st);
    else if (a.cols <= 1024) launch_rows<In, 64, 2>(a, st);
    else if (a.cols <= 2048) launch_rows<In, 64, 4>(a, st);
    else if (a.cols <= 8192) launch_rows<In, 256, 4>(a, st);
    else if (a.cols <= 16384) launch_rows<In, 512, 4>(a, st);
    else if (a.cols <= 32768) launch_rows<In, 1024, 4>(a, st);
    else launch_rows<In, 1024, 0>(a, st);
  }
  if (a.st && a.cols > 0) {
    if (a.rows > 0 && !fused)
      hipLaunchKernelGGL(int8_colmax_kernel<In>, dim3((unsigned)((a.cols + 511) / 512), a.parts), dim3(256), 0, st, a);
    in_pieces((a.cols + 63) / 64, 1, [&](int64_t c, int64_t n) {
      QuantArgs b = a;
      b.tile0 = c;
      hipLaunchKernelGGL(int8_colscale_kernel, dim3((unsigned)n), dim3(1024), 0, st, b);
    });
    in_pieces((a.rows + 127) / 128 * ((a.cols + 63) / 64), 1, [&](int64_t t, int64_t n) {
      QuantArgs b = a;
      b.tile0 = t;
      hipLaunchKernelGGL(int8_col_kernel<In>, dim3((unsigned)n), dim3(256), 0, st, b);
    });
  }
}

// Groups of rows whose column maxima are joined by a kernel of their own: what
// fills the chip, as far as each has 16 rows to spread the join's traffic over
// (4096 x 14336 fp32: 256 groups 117 us, 512 131; 14336 x 4096: 111 either
// way; 16384 x 7168 bf16: 256 groups 210, 512 168).
int quantize_parts(int64_t rows) {
  const int64_t some = rows < 256 ? rows : 256;
  return (int)(rows / 16 < some ? some : rows / 16 < kMostParts ? rows / 16 : kMostParts);
}

// ---------------------------------------------------------------------------
// gated activation
// ---------------------------------------------------------------------------
struct GluArgs {
  const void* x;  // forward: gu; backward: da
  int64_t rows, cols, ld;
  int64_t nb;     // blocks of 128 in a row of g
  void* a;        // dense, or null
  int8_t* aq;     // forward
  float* sa;
  int8_t* ck;     // forward: out or null; backward: in
  float* cs;
  void* dgu;      // backward
  int64_t lddgu;
};

// 1 + exp(-g), and silu(g) = g / (1 + exp(-g)) and 1 / (1 + exp(-g)) from it.
// g log2(e) rounded to binary32 is off by up to 2^-24 |g log2(e)|, an error
// that the exponential turns into a relative one.  bf16 results do not show it;
// for fp32 data whole number and fraction of the exponent are formed apart, the
// fraction from both halves of log2(e), and the division is correctly rounded
// (silu against 64 bits at g = -20: 1.7e-7, without either 1.0e-6; at -87
// 1.2e-7 and 3.9e-6).  fp32 hides this behind its memory traffic (8192 x 14336
// with everything kept in 306 us either way, backward 440; 333 x 1111 in 4.8,
// without 4.7), bf16 does not: 16384 x 14336 367 us, without 341.
constexpr float kLog2e = 1.44269504088896340736f, kLog2eLow = 1.92596299e-8f;
__device__ __forceinline__ float one_plus_exp(float g) {
  // (beyond 128 the exponential is infinite or lost in the sum)
  const float x = __builtin_amdgcn_fmed3f(g, -128.0f, 128.0f);
  const float n = __builtin_rintf(x * -kLog2e);
  const float f = fmaf(x, -kLog2eLow, fmaf(x, -kLog2e, -n));
  return 1.0f + __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), (int)n);
}
template <typename In>
__device__ __forceinline__ float sigmoid(float g) {
  if constexpr (sizeof(In) == 4) return __fdiv_rn(1.0f, one_plus_exp(g));
  else return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -kLog2e));
}
template <typename In>
__device__ __forceinline__ float silu(float g) {
  if constexpr (sizeof(In) == 4) return __fdiv_rn(g, one_plus_exp(g));
  else return g * sigmoid<In>(g);
}

// Where a group of 16 lanes is in a matrix of blocks of 128: its lanes take
// the block's whole chunks of 8, and of a row's last block the up to 7 values
// behind its last whole chunk, one to a lane (each in its own loads, they cost
// a wave 7 of every kind).
struct BlockAt {
  int64_t row, b, c;  // block b; this lane's chunk begins at c
  bool whole, one;    // the chunk is there; so is a value at `e`
  int64_t e;
  __device__ __forceinline__ BlockAt(const GluArgs& a, int64_t row_, int64_t b_, int t) : row(row_), b(b_) {
    c = b * kBlock + t * 8;
    whole = c + 8 <= a.cols;
    e = (a.cols & ~(int64_t)7) + t;
    one = b == a.nb - 1 && e < a.cols;
  }
};

// What a group of 16 lanes keeps of one block of one row of g and u; ck and cs
// are the row's.
__device__ __forceinline__ void keep_block(const GluArgs& a, const BlockAt& at, const float (&g)[8],
                                           const float (&u)[8], float g1, float u1, int8_t* ck, float* cs, bool first) {
  const Scale sg = scale_of(group_max_u32<0xF>(amax8(g, __float_as_uint(g1) & 0x7FFFFFFFu)));
  const Scale su = scale_of(group_max_u32<0xF>(amax8(u, __float_as_uint(u1) & 0x7FFFFFFFu)));
  if (at.whole) {
    store8(ck + at.c, codes8(g, sg), 8);
    store8(ck + a.cols + at.c, codes8(u, su), 8);
  }
  if (at.one) {
    ck[at.e] = (int8_t)(code_of(g1, sg.inv) & sg.keep);
    ck[a.cols + at.e] = (int8_t)(code_of(u1, su.inv) & su.keep);
  }
  if (first) {
    cs[at.b] = sg.s;
    cs[a.nb + at.b] = su.s;
  }
}

// One block of 128 of g and of u to 16 neighbouring lanes; groups of lanes take
// the blocks of the matrix in turn.  Bound by memory: 16384 x 14336 bf16 in 339
// us (5.5 TB/s: gu read, a and the codes written), 333 x 1111 fp32 in 4.8.
template <typename In>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(GluArgs a) {
  const int t = threadIdx.x & 15;
  const int64_t units = a.rows * a.nb, stride = (int64_t)gridDim.x * 16;
  for (int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); unit < units; unit += stride) {
    const int64_t row = unit / a.nb;
    const BlockAt at(a, row, unit - row * a.nb, t);
    const In* x = reinterpret_cast<const In*>(a.x) + at.row * a.ld;
    float g[8], u[8], g1 = 0.0f, u1 = 0.0f;
    load8(g, x + at.c, at.whole ? 8 : 0);
    load8(u, x + a.cols + at.c, at.whole ? 8 : 0);
    if (at.one) {
      g1 = widen(x[at.e]);
      u1 = widen(x[a.cols + at.e]);
    }
    if (a.ck) keep_block(a, at, g, u, g1, u1, a.ck + at.row * 2 * a.cols, a.cs + at.row * 2 * a.nb, t == 0);
    if (a.a) {
      In* o = reinterpret_cast<In*>(a.a) + at.row * a.cols;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = silu<In>(g[i]) * u[i];
      if (at.whole) store8(o + at.c, g, 8);
      if (at.one) store1(o + at.e, silu<In>(g1) * u1);
    }
  }
}

// With an INT8 copy of a: a row to a workgroup, which holds a in registers (CH
// > 0, CH chunks of 8 a thread) or computes it twice (CH == 0).  8192 x 14336
// bf16 with gu kept in 147-151 us (5.5 TB/s), without in 104; 61 x 14336 without
// in 5.6.
template <typename In, int NT, int CH>
__global__ __launch_bounds__(NT) void swiglu_row_kernel(GluArgs a) {
  __shared__ uint32_t red[NT / 64];
  const int64_t row = blockIdx.x;
  const In* x = reinterpret_cast<const In*>(a.x) + row * a.ld;
  float h[CH ? CH : 1][8], h1 = 0.0f;
  uint32_t m = 0;
  // chunk k of the row (16 chunks a block): a, and on the first time what is
  // kept, a's copy in dtype and its maximum
  auto chunk = [&](int64_t k, float (&o)[8], bool first_time) {
    const BlockAt at(a, row, k / 16, (int)(k & 15));
    float g[8], u[8], g1 = 0.0f, u1 = 0.0f;
    load8(g, x + at.c, at.whole ? 8 : 0);
    load8(u, x + a.cols + at.c, at.whole ? 8 : 0);
    if (at.one) {
      g1 = widen(x[at.e]);
      u1 = widen(x[a.cols + at.e]);
    }
    if (first_time && a.ck && at.b < a.nb)
      keep_block(a, at, g, u, g1, u1, a.ck + row * 2 * a.cols, a.cs + row * 2 * a.nb, (k & 15) == 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = silu<In>(g[i]) * u[i];
    if (at.one) h1 = silu<In>(g1) * u1;  // (of one chunk of a thread at most)
    if (first_time) {
      m = amax8(o, m);
      if (a.a) {
        In* out = reinterpret_cast<In*>(a.a) + row * a.cols;
        if (at.whole) store8(out + at.c, o, 8);
        if (at.one) store1(out + at.e, h1);
      }
    }
  };
  // chunks of the row, those of its last block's end included
  const int64_t chunks = a.nb * 16;
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) chunk(i * NT + threadIdx.x, h[i], true);
  } else {
    for (int64_t k = threadIdx.x; k < chunks; k += NT) chunk(k, h[0], true);
  }
  m = umax_u32(m, __float_as_uint(h1) & 0x7FFFFFFFu);
  const Scale s = scale_of(row_max<NT>(m, red));
  int8_t* aq = a.aq + row * a.cols;
  auto put = [&](int64_t k, const float (&o)[8]) {
    if (k * 8 + 8 <= a.cols) store8(aq + k * 8, codes8(o, s), 8);
    const BlockAt at(a, row, k / 16, (int)(k & 15));
    if (at.one) aq[at.e] = (int8_t)(code_of(h1, s.inv) & s.keep);
  };
  if constexpr (CH > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) put((int64_t)i * NT + threadIdx.x, h[i]);
  } else {
    for (int64_t k = threadIdx.x; k < chunks; k += NT) {
      chunk(k, h[0], false);
      put(k, h[0]);
    }
  }
  if (threadIdx.x == 0) a.sa[row] = s.s;
}

// 8 codes times their scale, or 0
__device__ __forceinline__ void load_codes(float (&v)[8], const int8_t* p, float s, bool there) {
  u32x2 w = {0, 0};
  if (there) w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_b*>(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)(int8_t)(w[i >> 2] >> (8 * (i & 3))) * s;
}

// Gradients of g and u, and a, from one value of each.
template <typename In>
__device__ __forceinline__ void swiglu_grad(float d, float g, float u, float& dg, float& du, float& act) {
  const float p = sigmoid<In>(g), w = g * p;  // silu(g)
  dg = d * u * (p * (1.0f + g * (1.0f - p)));
  du = d * w;
  act = w * u;
}

// Blocks of 128 as the forward pass takes them; bound by memory: 16384 x 14336
// bf16 with a in 422 us, without 329 (5.6 and 5.7 TB/s), 333 x 1111 fp32 in 4.9.
template <typename In>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(GluArgs a) {
  const int t = threadIdx.x & 15;
  const int64_t units = a.rows * a.nb, stride = (int64_t)gridDim.x * 16;
  for (int64_t unit = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); unit < units; unit += stride) {
    const int64_t row = unit / a.nb;
    const BlockAt at(a, row, unit - row * a.nb, t);
    const float* cs = a.cs + at.row * 2 * a.nb + at.b;
    const int8_t* ck = a.ck + at.row * 2 * a.cols;
    const In* da = reinterpret_cast<const In*>(a.x) + at.row * a.ld;
    const float sg = cs[0], su = cs[a.nb];
    float d[8], g[8], u[8], d1 = 0.0f, g1 = 0.0f, u1 = 0.0f;
    load8(d, da + at.c, at.whole ? 8 : 0);
    load_codes(g, ck + at.c, sg, at.whole);
    load_codes(u, ck + a.cols + at.c, su, at.whole);
    if (at.one) {
      d1 = widen(da[at.e]);
      g1 = (float)ck[at.e] * sg;
      u1 = (float)ck[a.cols + at.e] * su;
    }
    float h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) swiglu_grad<In>(d[i], g[i], u[i], g[i], u[i], h[i]);
    In* o = reinterpret_cast<In*>(a.dgu) + at.row * a.lddgu;
    In* act = reinterpret_cast<In*>(a.a) + (a.a ? at.row * a.cols : 0);
    if (at.whole) {
      store8(o + at.c, g, 8);
      store8(o + a.cols + at.c, u, 8);
      if (a.a) store8(act + at.c, h, 8);
    }
    if (at.one) {
      swiglu_grad<In>(d1, g1, u1, g1, u1, h[0]);
      store1(o + at.e, g1);
      store1(o + a.cols + at.e, u1);
      if (a.a) store1(act + at.e, h[0]);
    }
  }
}

unsigned glu_grid(const GluArgs& a) {
  const int64_t need = (a.rows * a.nb + 15) / 16, most = (int64_t)256 * 32;
  return (unsigned)(need < most ? need : most);
}

template <typename In, int NT, int CH>
void launch_glu_row(const GluArgs& all, hipStream_t st) {
  in_pieces(all.rows, 1, [&](int64_t r, int64_t n) {
    GluArgs a = all;
    a.x = reinterpret_cast<const In*>(all.x) + r * all.ld;
    if (all.a) a.a = reinterpret_cast<In*>(all.a) + r * all.cols;
    a.aq += r * all.cols;
    a.sa += r;
    if (all.ck) {
      a.ck += r * 2 * all.cols;
      a.cs += r * 2 * all.nb;
    }
    hipLaunchKernelGGL((swiglu_row_kernel<In, NT, CH>), dim3((unsigned)n), dim3(NT), 0, st, a);
  });
}

template <typename In>
void launch_glu_fwd(const GluArgs& a, hipStream_t st) {
  if (a.sa) {  // an empty copy may have no address
    // few rows: more threads a row, for the latency of its loads (aq alone of 61 x
    // 14336: 7.5 us with 512 threads, 5.6 with 1024); many rows: more chunks a
    // thread (16384 x 8192: 157 us with 512 threads of two, 164 with 1024 of one;
    // 32768 x 2048: 86 with 256, 111 with 512; 4096 x 28672: 170, and 217 without
    // registers)
    const bool few = a.rows <= 256;
    if (few && a.cols > 8192 && a.cols <= 16384) launch_glu_row<In, 1024, 2>(a, st);
    else if (few && a.cols > 2048 && a.cols <= 8192) launch_glu_row<In, 1024, 1>(a, st);
    else if (a.cols <= 2048) launch_glu_row<In, 256, 1>(a, st);
    else if (a.cols <= 8192) launch_glu_row<In, 512, 2>(a, st);
    else if (a.cols <= 16384) launch_glu_row<In, 512, 4>(a, st);
    else if (a.cols <= 32768) launch_glu_row<In, 1024, 4>(a, st);
    else launch_glu_row<In, 1024, 0>(a, st);
  } else if (a.rows > 0 && a.cols > 0) {
    hipLaunchKernelGGL(swiglu_fwd_kernel<In>, dim3(glu_grid(a)), dim3(256), 0, st, a);
  }
}

}  // namespace

int64_t quantize_int8_workspace(int64_t rows, int64_t cols) { return 4 * cols * quantize_parts(rows); }

void launch_quantize_int8(const void* x, int dtype, int64_t rows, int64_t cols, int64_t ld, int8_t* q, float* s,
                          int8_t* qt, float* st_, void* workspace, hipStream_t st) {
  QuantArgs a{};
  a.x = x; a.rows = rows; a.cols = cols; a.ld = ld;
  a.q = q; a.s = s; a.qt = qt; a.st = st_;
  a.part = reinterpret_cast<float*>(workspace);
  a.parts = quantize_parts(rows);
  if (dtype == QSG_BF16) launch_quantize<uint16_t>(a, st);
  else launch_quantize<float>(a, st);
}

void launch_swiglu_int8_fwd(const void* gu, int dtype, int64_t rows, int64_t cols, int64_t ld, void* out, int8_t* aq,
                            float* sa, int8_t* ck, float* cs, hipStream_t st) {
  GluArgs a{};
  a.x = gu; a.rows = rows; a.cols = cols; a.ld = ld;
  a.nb = (cols + kBlock - 1) / kBlock;
  a.a = out; a.aq = aq; a.sa = sa; a.ck = ck; a.cs = cs;
  if (dtype == QSG_BF16) launch_glu_fwd<uint16_t>(a, st);
  else launch_glu_fwd<float>(a, st);
}

void launch_swiglu_int8_bwd(const void* da, int dtype, int64_t rows, int64_t cols, int64_t ldda, const int8_t* ck,
                            const float* cs, void* dgu, int64_t lddgu, void* out, hipStream_t st) {
  if (rows == 0 || cols == 0) return;
  GluArgs a{};
  a.x = da; a.rows = rows; a.cols = cols; a.ld = ldda;
  a.nb = (cols + kBlock - 1) / kBlock;
  a.a = out; a.ck = const_cast<int8_t*>(ck); a.cs = const_cast<float*>(cs);
  a.dgu = dgu; a.lddgu = lddgu;
  if (dtype == QSG_BF16) hipLaunchKernelGGL(swiglu_bwd_kernel<uint16_t>, dim3(glu_grid(a)), dim3(256), 0, st, a);
  else hipLaunchKernelGGL(swiglu_bwd_kernel<float>, dim3(glu_grid(a)), dim3(256), 0, st, a);
}

}  // namespace qsg
