// Product of two INT8 matrices with a scale for each row of both:
//   C[m,n] = (sum_k A[m,k] B[n,k]) sa[m] sb[n] (+ bias[n]),  both K-contiguous.
// Sums are 32-bit integers and exact, so they may be split and joined in any
// order; only their scaling is rounded.
//
// What bounds it depends on the rows of A: a decode batch reads B once (16 rows
// through 28672 x 4096: 25 us, 4.7 TB/s), a training batch is matrix
// instructions (32768 x 4096 x 4096: 422 to 460 us, 2.4 to 2.6 POP/s).  Five kernels:
//   * 256 x 256 persistent tiles (gemm_fast.hip, the FP8 products' loop);
//   * tiles of 64 and 128 by direct loads into a ring of LDS stages;
//   * 16 to 32 rows of A by 16 to 64 of B, K split over a workgroup's waves, each
//     with a ring of its own;
//   * the same without LDS for 16 x 16, and tiles through registers: operands of
//     any alignment.
// launch_gemm_int8 says which serves what, with both sides' times.
#include <hip/hip_runtime.h>

#include <type_traits>

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
typedef uint32_t u32x4_e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_b __attribute__((ext_vector_type(4), aligned(1)));

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
  // Rows of B a multiple of 4096 bytes apart begin in the same few memory
  // channels, and workgroups that read B in step meet there: each group of 8
  // neighbours then begins at another K step (a sum has no order) and goes
  // round (16 x 28672 x 4096: 27.2 -> 25.0 us, 32 x 16384 x 8192: 31.7 -> 27.8;
  // other row lengths, and more rows than 64, gain nothing, and the kernels that
  // serve those are without it: 1021 x 4096 x 4096 22 us, with it 24).
  int turn;
};

// 16 bytes of a row of K bytes at k; what lies past its end is 0.  One load
// without a branch where a row has 16 bytes: the last 16 of them, shifted.
__device__ __forceinline__ v4i load_chunk(const int8_t* row, int64_t k, int64_t K) {
  if (K >= 16) {
    const int64_t at = k < K - 16 ? k : K - 16;
    return __builtin_bit_cast(v4i, shift_down(*reinterpret_cast<const u32x4_b*>(row + at), (int)(k - at < 16 ? k - at : 16)));
  }
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

// Scales and biases of 4 consecutive columns (past the last one: the last one's)
struct Cols {
  float s[4], c[4];
  __device__ __forceinline__ void read(const Int8Args& g, int64_t n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = n + i < g.N ? n + i : g.N - 1;
      s[i] = g.sb[at];
      c[i] = bias_at(g, at);
    }
  }
};

// 4 consecutive outputs of row m from their sums
template <bool OUT_BF16>
__device__ __forceinline__ void store4(const Int8Args& g, int64_t m, int64_t n, const int (&sum)[4], float sa,
                                       const Cols& col) {
  if (m >= g.M || n >= g.N) return;
  float v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = fmaf((float)sum[i] * sa, col.s[i], col.c[i]);
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
// 16 rows of A against 16 rows of B to a workgroup, any alignment.  Lane l holds row l % 16
// of either operand and, of a step of 128 K, bytes 32 (l / 16) .. +31 as two
// chunks of two instructions: both operands split K between lanes alike, so
// every product is made once.  The instruction takes (B, A), and lane l then
// holds row l % 16 of A and columns 4 (l / 16) .. +3.  The workgroup's waves
// split K; a wave takes 8 steps at a time, all of their loads first.  Bound by
// the loads: one row through 28672 x 4096 in 22.3 us (5.3 TB/s), 16 rows in 34
// (a lane's chunk of A costs the vector-memory path a clock as one of B does).
constexpr int kFewWaves = 4, kFewSteps = 8;

template <bool OUT_BF16>
__global__ __launch_bounds__(kFewWaves * 64) void gemm_int8_few_kernel(Int8Args g) {
  __shared__ v4i red[kFewWaves][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.y * 16, n0 = (int64_t)blockIdx.x * 16;
  const int at = (lane >> 4) * 32;
  // rows past the end read the last one; their results are not stored
  const int64_t m = m0 + (lane & 15) < g.M ? m0 + (lane & 15) : g.M - 1;
  const int64_t n = n0 + (lane & 15) < g.N ? n0 + (lane & 15) : g.N - 1;
  const int8_t* a = g.a + m * g.lda;
  const int8_t* b = g.b + n * g.ldb;
  // read before the sums, so that a workgroup waits for memory once
  const float sa = g.sa[m];
  Cols cols;
  cols.read(g, n0 + 4 * (lane >> 4));
  v4i acc = {0, 0, 0, 0};
  // C steps from s on
  auto steps = [&](int64_t s, auto count) {
    constexpr int C = decltype(count)::value;
    v4i fb[C][2], fa[C][2];
#pragma unroll
    for (int u = 0; u < C; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) fb[u][h] = *reinterpret_cast<const v4i_u*>(b + (s + u) * 128 + at + 16 * h);
#pragma unroll
    for (int u = 0; u < C; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) fa[u][h] = *reinterpret_cast<const v4i_u*>(a + (s + u) * 128 + at + 16 * h);
#pragma unroll
    for (int u = 0; u < C; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[u][h], fa[u][h], acc, 0, 0, 0);
  };
  const int64_t whole = g.K / 128, grouped = whole / kFewSteps * kFewSteps;
  for (int64_t s = wave * kFewSteps; s < grouped; s += kFewWaves * kFewSteps)
    steps(s, std::integral_constant<int, kFewSteps>{});
  for (int64_t s = grouped + wave; s < whole; s += kFewWaves) steps(s, std::integral_constant<int, 1>{});
  if (g.K % 128 && whole % kFewWaves == wave) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t k = whole * 128 + at + 16 * h;
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(load_chunk(b, k, g.K), load_chunk(a, k, g.K), acc, 0, 0, 0);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    v4i v = red[0][lane];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += red[w][lane];
    const int sum[4] = {v[0], v[1], v[2], v[3]};
    store4<OUT_BF16>(g, m0 + (lane & 15), n0 + 4 * (lane >> 4), sum, sa, cols);
  }
}

typedef __attribute__((address_space(3))) void* lds_ptr_t;
constexpr uint32_t OUT_OF_RANGE = 0x80000000u;  // past any resource below

// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N < 64, "vmcnt field");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}
// Workgroup barrier without a memory fence (a fence would also wait for the
// loads in flight); the waits it needs are explicit.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// the same behind this wave's own LDS accesses
__device__ __forceinline__ void lds_barrier_lgkm() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// `most` rows from row0 on, as far as there are so many
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const int8_t* p, int64_t row0, int64_t rows, int64_t ld,
                                                            int most) {
  int64_t n = rows - row0;
  n = n < most ? n : most;
  return __builtin_amdgcn_make_buffer_rsrc((void*)(p + row0 * ld), 0, (int)(n * ld), 0x00020000);
}

// The same with operands of whole 16 bytes.  Lanes that are neighbours load
// different rows above, 16 bytes each, which the vector-memory path takes one
// lane a clock; here a wave's loads cover whole 128-byte row segments and go to
// LDS directly, into a ring of R steps that is the wave's own, so it waits for
// its own loads only.  16-byte chunk c of row r is at position c ^ ring_swz(r):
// of a fragment read (lane l: row l % 16, chunk l / 16 or 4 + l / 16) the lanes
// that the LDS serves together (8p .. 8p+7 with 8p+32 .. 8p+39) then meet
// distinct banks.  61 rows through 4096 x 14336 in 21 us, against 39 from
// registers; through 28672 x 4096 in 32 against 65.
__device__ __forceinline__ int ring_swz(int r) { return ((r >> 1) & 1) | ((r >> 3) & 1) << 1 | ((r >> 2) & 1) << 2; }

template <int MT, int NT, int WAVES, int R, bool OUT_BF16>
__global__ __launch_bounds__(WAVES * 64) void gemm_int8_ring_kernel(Int8Args g) {
  constexpr int ROWS = 16 * (MT + NT), STEP = ROWS * 128, LOADS = STEP / 1024;
  static_assert(MT * NT * 1024 <= STEP, "a wave's sums fit its part of a stage");
  // distinct objects: reads of one stage wait for no load into another
  __shared__ __attribute__((aligned(1024))) uint8_t st0[WAVES * STEP];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[WAVES * STEP];
  __shared__ __attribute__((aligned(1024))) uint8_t st2[R > 2 ? WAVES * STEP : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t st3[R > 3 ? WAVES * STEP : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Workgroups go to the 8 XCDs in turn, each with an L2 of its own: those that
  // read the same rows of B follow each other on one XCD
  const int64_t turn = blockIdx.x / 8, tm = turn % g.tiles_m, tn = turn / g.tiles_m * 8 + blockIdx.x % 8;
  if (tn * (16 * NT) >= g.N) return;
  const int64_t m0 = tm * (16 * MT), n0 = tn * (16 * NT);
  // load i of a step fills 1 KB: rows 8 i + lane / 8 (B's rows, then A's),
  // position lane % 8
  const int pr = lane >> 3;
  const __amdgpu_buffer_rsrc_t ra = rows_rsrc(g.a, m0, g.M, g.lda, 16 * MT), rb = rows_rsrc(g.b, n0, g.N, g.ldb, 16 * NT);
  int ch[2];
  uint32_t va[2], vb[2];  // of rows 0..7 and 8..15; 16 rows further are 16 ld more
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    ch[i] = (lane & 7) ^ ring_swz(8 * i + pr);
    va[i] = (8 * i + pr) * (uint32_t)g.lda + ch[i] * 16;
    vb[i] = (8 * i + pr) * (uint32_t)g.ldb + ch[i] * 16;
  }
  const int K = (int)g.K, nk = (K + 127) / 128, rounds = (nk + WAVES - 1) / WAVES;
  constexpr bool TURN = NT < 4;  // up to 64 rows take no wider one
  const int first = TURN && g.turn ? (int)(tn / 8 * WAVES % nk) : 0;  // the step to begin with
  uint32_t mine = wave * STEP;
  auto issue = [&](uint8_t* st, int round) {
    const int at = round * WAVES + wave, turned = !TURN || at + first < nk ? at + first : at + first - nk;
    const int k = !TURN || at < nk ? turned * 128 : K;
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const uint32_t off = k + ch[i & 1] * 16 < K ? vb[i & 1] + (uint32_t)(i >> 1) * 16 * (uint32_t)g.ldb + k : OUT_OF_RANGE;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(st + mine + i * 1024), 16, off, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
      const uint32_t off = k + ch[i & 1] * 16 < K ? va[i & 1] + (uint32_t)(i >> 1) * 16 * (uint32_t)g.lda + k : OUT_OF_RANGE;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(st + mine + (2 * NT + i) * 1024), 16, off, 0, 0, 0);
    }
  };
  // scales of the tiles that this wave joins in the end
  constexpr int PER = (MT * NT + WAVES - 1) / WAVES;
  Cols cols[PER];
  float sa[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int t = wave + k * WAVES;
    const int64_t m = m0 + t / NT * 16 + (lane & 15);
    sa[k] = g.sa[m < g.M ? m : g.M - 1];
    cols[k].read(g, n0 + t % NT * 16 + 4 * (lane >> 4));
  }
  v4i acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  int fo[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) fo[h] = (lane & 15) * 128 + (((4 * h + (lane >> 4)) ^ ring_swz(lane & 15)) * 16);
  auto step = [&](uint8_t* st, int round) {
    wait_vm<(R - 1) * LOADS>();
    asm volatile("" ::: "memory");
    v4i fb[NT][2], fa[MT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < NT; ++j) fb[j][h] = *reinterpret_cast<const v4i*>(st + mine + j * 2048 + fo[h]);
#pragma unroll
      for (int i = 0; i < MT; ++i) fa[i][h] = *reinterpret_cast<const v4i*>(st + mine + (NT + i) * 2048 + fo[h]);
    }
    // the reads have returned before the loads that replace what they read
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    issue(st, round + R);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[j][h], fa[i][h], acc[i][j], 0, 0, 0);
  };
  issue(st0, 0);
  issue(st1, 1);
  if constexpr (R > 2) issue(st2, 2);
  if constexpr (R > 3) issue(st3, 3);
  int r = 0;
  for (; r + R <= rounds; r += R) {
    step(st0, r);
    step(st1, r + 1);
    if constexpr (R > 2) step(st2, r + 2);
    if constexpr (R > 3) step(st3, r + 3);
  }
  if (r < rounds) step(st0, r++);
  if (R > 2 && r < rounds) step(st1, r++);
  if constexpr (R > 3) {
    if (r < rounds) step(st2, r++);
  }
  wait_vm<0>();  // the loads past the last step have landed, in this wave's part alone
  asm volatile("" ::: "memory");
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) *reinterpret_cast<v4i*>(st0 + mine + (i * NT + j) * 1024 + lane * 16) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    const int t = wave + k * WAVES;
    if (t < MT * NT) {
      v4i v = *reinterpret_cast<const v4i*>(st0 + t * 1024 + lane * 16);
#pragma unroll
      for (int w = 1; w < WAVES; ++w) v += *reinterpret_cast<const v4i*>(st0 + w * STEP + t * 1024 + lane * 16);
      const int sum[4] = {v[0], v[1], v[2], v[3]};
      store4<OUT_BF16>(g, m0 + t / NT * 16 + (lane & 15), n0 + t % NT * 16 + 4 * (lane >> 4), sum, sa[k], cols[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// tiles
// ---------------------------------------------------------------------------
constexpr int TB = 128;  // rows of either operand, and bytes of K, of a tile

// 16-byte chunk c of LDS row r is at position c ^ swz(r): the lanes that the
// LDS serves together read 8 rows at two neighbouring chunks, which this puts
// on distinct banks
__device__ __forceinline__ int swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

// Scales of a wave's 32 NI x 32 NJ outputs from row m0 and column n0 on (read
// before the K loop, which hides their latency): lane l holds row l % 32 and,
// of group q, columns 8 q + 4 (l / 32) .. +3.
template <int NI, int NJ>
struct TileScales {
  float sa[NI];
  Cols col[NJ][4];
  __device__ __forceinline__ TileScales(const Int8Args& g, int64_t m0, int64_t n0, int lane) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int64_t m = m0 + i * 32 + (lane & 31);
      sa[i] = g.sa[m < g.M ? m : g.M - 1];
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) col[j][q].read(g, n0 + j * 32 + 8 * q + 4 * (lane >> 5));
  }
};

// The outputs, 32 rows at a time through the wave's own part of LDS, from which
// they leave in whole row segments of 32 NJ outputs (straight from the
// registers a store would write 8 bytes of each of 32 rows).
template <bool OUT_BF16, int NJ>
constexpr int kTilePitch = 32 * NJ * (OUT_BF16 ? 2 : 4) + 16;
template <bool OUT_BF16, int NI, int NJ>
__device__ __forceinline__ void store_tile(const Int8Args& g, const v16i (&acc)[NI][NJ], const TileScales<NI, NJ>& sc,
                                           int64_t m0, int64_t n0, int lane, uint8_t* lds) {
  constexpr int ESZ = OUT_BF16 ? 2 : 4, PITCH = kTilePitch<OUT_BF16, NJ>;
  constexpr int LPR = 32 * NJ * ESZ / 16, RPI = 64 / LPR;  // lanes of a row, rows of a store
  const int64_t n = n0 + lane % LPR * (16 / ESZ);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf((float)acc[i][j][4 * q + e] * sc.sa[i], sc.col[j][q].s[e], sc.col[j][q].c[e]);
        uint8_t* p = lds + (lane & 31) * PITCH + (j * 32 + 8 * q + 4 * (lane >> 5)) * ESZ;
        if constexpr (OUT_BF16) *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        else *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // other lanes' writes
#pragma unroll
    for (int k = 0; k < 32 / RPI; ++k) {
      const int r = k * RPI + lane / LPR;
      const u32x4 w = *reinterpret_cast<const u32x4*>(lds + r * PITCH + lane % LPR * 16);
      const int64_t m = m0 + i * 32 + r;
      if (m < g.M) {
        uint8_t* p = reinterpret_cast<uint8_t*>(g.c) + (m * g.ldc + n) * ESZ;
        if (n + 16 / ESZ <= g.N) {
          *reinterpret_cast<u32x4_e*>(p) = w;
        } else {
#pragma unroll
          for (int e = 0; e < 16 / ESZ; ++e)
            if (n + e < g.N) {
              if constexpr (OUT_BF16) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
              else reinterpret_cast<uint32_t*>(p)[e] = w[e];
            }
        }
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the reads, before the next rows' writes
  }
}

// Any alignment: through registers, two K tiles ahead.  A K tile is four phases
// of 32 K, and a phase's fragments are read during the phase before; the
// barrier behind which the next K tile is there lies before the last phase,
// whose instructions cover the first reads from it.  1021 x 4095 x 4095 in 41
// us: loads of 16 bytes at any address are what bounds it (aligned, through
// the kernel below, 22).
template <int TM, int TN, bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_int8_kernel(Int8Args g) {
  constexpr int NI = TM / 64, NJ = TN / 64, LA = TM / 32, LB = TN / 32;
  __shared__ __attribute__((aligned(16))) uint8_t st0[(TM + TN) * TB];
  __shared__ __attribute__((aligned(16))) uint8_t st1[(TM + TN) * TB];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave >> 1, wn = wave & 1;
  const int64_t m0 = (blockIdx.x % g.tiles_m) * TM, n0 = (blockIdx.x / g.tiles_m) * TN;
  // thread: chunk tid % 8 of rows tid / 8 + 32 i of both operands
  const int ch = tid & 7, r0 = tid >> 3;
  const int8_t* pa[LA];
  const int8_t* pb[LB];
#pragma unroll
  for (int i = 0; i < LA; ++i) pa[i] = g.a + (m0 + r0 + 32 * i < g.M ? m0 + r0 + 32 * i : g.M - 1) * g.lda;
#pragma unroll
  for (int i = 0; i < LB; ++i) pb[i] = g.b + (n0 + r0 + 32 * i < g.N ? n0 + r0 + 32 * i : g.N - 1) * g.ldb;
  const TileScales<NI, NJ> scales(g, m0 + wm * (TM / 2), n0 + wn * (TN / 2), lane);
  const int K = (int)g.K, nk = (K + TB - 1) / TB;
  struct Regs {
    v4i a[LA], b[LB];
  };
  Regs x0, x1;
  const int plain = K / TB;  // whole K tiles; the loop over them has no branch,
                             // behind which the compiler waits for every load in flight
  auto fetch_plain = [&](Regs& x, int kt) {
    const int k = kt * TB + ch * 16;
#pragma unroll
    for (int i = 0; i < LA; ++i) x.a[i] = *reinterpret_cast<const v4i_u*>(pa[i] + k);
#pragma unroll
    for (int i = 0; i < LB; ++i) x.b[i] = *reinterpret_cast<const v4i_u*>(pb[i] + k);
  };
  auto fetch = [&](Regs& x, int kt) {
    const int k = kt * TB + ch * 16;
    if (kt < plain) {
      fetch_plain(x, kt);
    } else if (kt < nk) {
#pragma unroll
      for (int i = 0; i < LA; ++i) x.a[i] = load_chunk(pa[i], k, K);
#pragma unroll
      for (int i = 0; i < LB; ++i) x.b[i] = load_chunk(pb[i], k, K);
    }
  };
  auto put = [&](uint8_t* st, const Regs& x) {
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      const int r = r0 + 32 * i;
      *reinterpret_cast<v4i*>(st + r * TB + ((ch ^ swz(r)) * 16)) = x.a[i];
    }
#pragma unroll
    for (int i = 0; i < LB; ++i) {
      const int r = r0 + 32 * i;
      *reinterpret_cast<v4i*>(st + (TM + r) * TB + ((ch ^ swz(r)) * 16)) = x.b[i];
    }
  };
  int fo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) fo[s] = (lane & 31) * TB + (((2 * s + (lane >> 5)) ^ swz(lane & 31)) * 16);
  v16i acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  v4i fa[2][NI], fb[2][NJ];
  auto read = [&](const uint8_t* st, int s) {
#pragma unroll
    for (int i = 0; i < NI; ++i) fa[s & 1][i] = *reinterpret_cast<const v4i*>(st + (wm * (TM / 2) + i * 32) * TB + fo[s]);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      fb[s & 1][j] = *reinterpret_cast<const v4i*>(st + TM * TB + (wn * (TN / 2) + j * 32) * TB + fo[s]);
  };
  // K tile kt in `cur`; kt + 1 goes from `ready` to `next`, kt + 2 is fetched into `other`
  auto step = [&](const uint8_t* cur, uint8_t* next, const Regs& ready, Regs& other, int kt, auto all_plain) {
    if constexpr (decltype(all_plain)::value) {
      fetch_plain(other, kt + 2);
      __builtin_amdgcn_sched_barrier(0);  // the loads first, not where their registers are needed
    } else {
      fetch(other, kt + 2);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read(cur, s + 1);
      } else {
        lds_barrier_lgkm();
        read(next, 0);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[s & 1][j], fa[s & 1][i], acc[i][j], 0, 0, 0);
      if (s == 1) put(next, ready);
    }
  };
  fetch(x0, 0);
  fetch(x1, 1);
  put(st0, x0);
  lds_barrier_lgkm();
  read(st0, 0);
  int kt = 0;
  for (; kt + 4 <= plain; kt += 2) {
    step(st0, st1, x1, x0, kt, std::true_type{});
    step(st1, st0, x0, x1, kt + 1, std::true_type{});
  }
  for (; kt + 2 <= nk; kt += 2) {
    step(st0, st1, x1, x0, kt, std::false_type{});
    step(st1, st0, x0, x1, kt + 1, std::false_type{});
  }
  if (kt < nk) step(st0, st1, x1, x0, kt, std::false_type{});
  lds_barrier_lgkm();  // no wave reads a stage any more
  constexpr int PART = 32 * kTilePitch<OUT_BF16, NJ>;
  static_assert(2 * PART <= sizeof(st0), "two waves' rows fit a stage");
  store_tile<OUT_BF16, NI, NJ>(g, acc, scales, m0 + wm * (TM / 2), n0 + wn * (TN / 2), lane,
                               (wave < 2 ? st0 : st1) + (wave & 1) * PART);
}

// TM x TN tiles of operands of whole 16 bytes: the loads go to LDS directly, 3
// K tiles ahead in a ring of 4 stages.  (Through registers and fewer tiles
// ahead, as above, a workgroup a CU waits for each tile's loads: 1021 x 4096 x
// 4096 with 128 x 128 tiles 37 us, 22 here.)  Phases as above.
template <int TM, int TN, bool TURN, bool OUT_BF16>
__global__ __launch_bounds__(256) void gemm_int8_tile_kernel(Int8Args g) {
  constexpr int NI = TM / 64, NJ = TN / 64;   // 32 x 32 tiles of a wave
  constexpr int LA = TM / 32, LB = TN / 32;   // loads of a wave and K tile
  constexpr int STAGE = (TM + TN) * TB, AHEAD = 3, WAIT = (AHEAD - 1) * (LA + LB);
  // distinct objects: reads of one stage wait for no load into another; A's
  // rows of 128 bytes, then B's
  __shared__ __attribute__((aligned(1024))) uint8_t st0[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st1[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st2[STAGE];
  __shared__ __attribute__((aligned(1024))) uint8_t st3[STAGE];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  // Workgroups go to the 8 XCDs in turn: each XCD gets a contiguous part of an
  // order that walks groups of 8 tile-rows column by column
  const uint32_t T = gridDim.x, tiles_m = (uint32_t)g.tiles_m, tiles_n = T / tiles_m;
  const uint32_t at = T % 8 == 0 ? blockIdx.x % 8 * (T / 8) + blockIdx.x / 8 : blockIdx.x;
  const uint32_t y0 = at / (8 * tiles_n) * 8, high = tiles_m - y0 < 8 ? tiles_m - y0 : 8;
  const uint32_t in = at - y0 * tiles_n;
  const int64_t m0 = (int64_t)(y0 + in % high) * TM, n0 = (int64_t)(in / high) * TN;

  // load i of a wave fills the 1 KB block i * 4 + wave of an operand: rows
  // 8 (i * 4 + wave) + lane / 8, position lane % 8
  const int pr = lane >> 3, ch = (lane & 7) ^ pr ^ (wave & 1);  // swz(row), the same for every i
  const uint32_t va = (wave * 8 + pr) * (uint32_t)g.lda + ch * 16, vb = (wave * 8 + pr) * (uint32_t)g.ldb + ch * 16;
  const __amdgpu_buffer_rsrc_t ra = rows_rsrc(g.a, m0, g.M, g.lda, TM), rb = rows_rsrc(g.b, n0, g.N, g.ldb, TN);
  const TileScales<NI, NJ> scales(g, m0 + wm * (TM / 2), n0 + wn * (TN / 2), lane);
  const int K = (int)g.K, nk = (K + TB - 1) / TB;
  const int first = TURN ? (int)(in / high / 8 % nk) : 0;  // the K tile to begin with
  // load i (of A's and then B's) of K tile kt; past the last row, or the
  // last 16 bytes of a row, 0 is read
  auto issue1 = [&](uint8_t* dst, int kt, int i) {
    const bool is_a = i < LA;
    const int j = is_a ? i : i - LA;
    const int kr = !TURN || kt + first < nk ? kt + first : kt + first - nk;
    const uint32_t off = (!TURN || kt < nk) && kr * TB + ch * 16 < K ? kr * TB : OUT_OF_RANGE;
    const uint32_t v = is_a ? va + j * 32 * (uint32_t)g.lda : vb + j * 32 * (uint32_t)g.ldb;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(is_a ? ra : rb,
                                             (lds_ptr_t)(dst + (is_a ? 0 : TM * TB) + (j * 4 + wave) * 1024), 16, v + off,
                                             0, 0, 0);
  };
  auto issue = [&](uint8_t* dst, int kt) {
#pragma unroll
    for (int i = 0; i < LA + LB; ++i) issue1(dst, kt, i);
  };
  int fo[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) fo[s] = (lane & 31) * TB + (((2 * s + (lane >> 5)) ^ swz(lane & 31)) * 16);
  v16i acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  v4i fa[2][NI], fb[2][NJ];
  auto read = [&](const uint8_t* st, int s) {
#pragma unroll
    for (int i = 0; i < NI; ++i) fa[s & 1][i] = *reinterpret_cast<const v4i*>(st + (wm * (TM / 2) + i * 32) * TB + fo[s]);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      fb[s & 1][j] = *reinterpret_cast<const v4i*>(st + TM * TB + (wn * (TN / 2) + j * 32) * TB + fo[s]);
  };
  // K tile kt in `cur`, the next one in `next`; `dst` held the one before
  auto step = [&](const uint8_t* cur, const uint8_t* next, uint8_t* dst, int kt) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (s < 3) {
        read(cur, s + 1);
      } else {
        wait_vm<WAIT>();
        lds_barrier();
        read(next, 0);
      }
      // a third of the loads in each of the first three phases
      constexpr int L3 = (LA + LB + 2) / 3;
      if (s < 3) {
#pragma unroll
        for (int i = s * L3; i < (s + 1) * L3 && i < LA + LB; ++i) issue1(dst, kt + AHEAD, i);
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[s & 1][j], fa[s & 1][i], acc[i][j], 0, 0, 0);
#pragma unroll
      for (int q = 0; q < NI * NJ; ++q) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, (NI + NJ + NI * NJ - 1) / (NI * NJ), 0);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  issue(st0, 0);
  issue(st1, 1);
  issue(st2, 2);
  wait_vm<WAIT>();
  lds_barrier();
  read(st0, 0);
  int kt = 0;
  for (; kt + 4 <= nk; kt += 4) {
    step(st0, st1, st3, kt);
    step(st1, st2, st0, kt + 1);
    step(st2, st3, st1, kt + 2);
    step(st3, st0, st2, kt + 3);
  }
  if (kt < nk) step(st0, st1, st3, kt++);
  if (kt < nk) step(st1, st2, st0, kt++);
  if (kt < nk) step(st2, st3, st1, kt++);
  wait_vm<0>();  // the loads past the last K tile have landed, and
  lds_barrier();  // no wave reads a stage any more
  constexpr int PART = 32 * kTilePitch<OUT_BF16, NJ>;
  static_assert(2 * PART <= STAGE, "two waves' rows fit a stage");
  store_tile<OUT_BF16, NI, NJ>(g, acc, scales, m0 + wm * (TM / 2), n0 + wn * (TN / 2), lane,
                               (wave < 2 ? st0 : st1) + (wave & 1) * PART);
}

void launch_few(const Int8Args& g, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)((g.M + 15) / 16)), block(kFewWaves * 64);
  if (bf16) hipLaunchKernelGGL(gemm_int8_few_kernel<true>, grid, block, 0, st, g);
  else hipLaunchKernelGGL(gemm_int8_few_kernel<false>, grid, block, 0, st, g);
}

template <int MT, int NT, int WAVES, int R>
void launch_ring(Int8Args g, bool bf16, hipStream_t st) {
  g.tiles_m = (g.M + 16 * MT - 1) / (16 * MT);
  const dim3 grid((unsigned)(g.tiles_m * ((g.N + 128 * NT - 1) / (128 * NT)) * 8)), block(WAVES * 64);
  if (bf16) hipLaunchKernelGGL((gemm_int8_ring_kernel<MT, NT, WAVES, R, true>), grid, block, 0, st, g);
  else hipLaunchKernelGGL((gemm_int8_ring_kernel<MT, NT, WAVES, R, false>), grid, block, 0, st, g);
}

template <int TM, int TN>
void launch_any(Int8Args g, bool bf16, hipStream_t st) {
  g.tiles_m = (g.M + TM - 1) / TM;
  const dim3 grid((unsigned)(g.tiles_m * ((g.N + TN - 1) / TN)));
  if (bf16) hipLaunchKernelGGL((gemm_int8_kernel<TM, TN, true>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((gemm_int8_kernel<TM, TN, false>), grid, dim3(256), 0, st, g);
}

template <int TM, int TN, bool TURN = false>
void launch_tile(Int8Args g, bool bf16, hipStream_t st) {
  g.tiles_m = (g.M + TM - 1) / TM;
  const dim3 grid((unsigned)(g.tiles_m * ((g.N + TN - 1) / TN)));
  if (bf16) hipLaunchKernelGGL((gemm_int8_tile_kernel<TM, TN, TURN, true>), grid, dim3(256), 0, st, g);
  else hipLaunchKernelGGL((gemm_int8_tile_kernel<TM, TN, TURN, false>), grid, dim3(256), 0, st, g);
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
  // 256 x 256 tiles where there are 128 of them, for half of the CUs (us with
  // them, and with the kernels below):
  //   2048 x 4096 x 4096 (128 tiles)     46    49
  //   4096 x 4096 x 4096 (256)           64    97
  //   32768 x 256 x 4096 (128)           57    58
  //   257 x 28672 x 4096 (224)           52    61
  // The number says nothing of how full they are; where less than 100 full ones
  // would do, the smaller tiles are the faster:
  //   32768 x 192 x 4096 (128, 96 full ones' work)   56    53
  //   32768 x 128 x 4096 (128, 64)                   58    40
  //   130 x 32768 x 4096 (128, 65)                   52    49
  //   65 x 32768 x 4096 (128, 33)                    50    38
  if (M > 64 && launch_gemm_int8_fast(a, sa, b, sb, M, N, K, lda, ldb, bias, g.bias_bf16, c, c_dtype, ldc, st)) return;
  // direct loads: whole chunks, 31-bit offsets in 128 rows
  const bool dma = (uintptr_t)a % 16 == 0 && (uintptr_t)b % 16 == 0 && lda % 16 == 0 && ldb % 16 == 0 && K % 16 == 0 &&
                   K > 0 && lda < (1 << 24) && ldb < (1 << 24);
  g.turn = M <= 64 && ldb % 4096 == 0;
  auto tiles = [&](int64_t tm, int64_t tn) { return ((M + tm - 1) / tm) * ((N + tn - 1) / tn); };
  if (!dma) {
    // Bound by loads of 16 bytes at any address, a lane a clock: codes realigned
    // once would need a workspace, which this call does not take.
    // 128 x 128 tiles where they occupy the chip (1021 x 4095 x 4095: 41 us, with
    // 64 x 64 58).  K split over waves instead where that needs no more workgroups
    // than CUs (53 x 608 x 12275: 33 us, with 64 x 64 43; 130 x 130 x 333: 3.9 and
    // 5.8; beyond, 64 x 2000 x 4095: 31 and 18), or for one row of blocks that 64 x
    // 64 would fill to a quarter (16 x 4095 x 4095: 17 and 20; one row of 14001 x
    // 4095: 33 and 22)
    if (M > 64 && tiles(128, 128) >= 192) launch_any<128, 128>(g, bf16, st);
    else if (tiles(16, 16) <= 256 || (M <= 16 && tiles(64, 64) < 100)) launch_few(g, bf16, st);
    else launch_any<64, 64>(g, bf16, st);
    return;
  }
  // The largest tiles that still occupy most of the chip (us with tiles of 128 x
  // 128, 64 x 128 and 64 x 64):
  //   256 x 28672 x 4096 (448 tiles of 128 x 128)   55   74   73
  //   1021 x 4096 x 4096 (256)                      22   27   29
  //   512 x 4096 x 4096 (256 of 64 x 128)           18   15   16
  //   1021 x 1024 x 4096 (256 of 64 x 64)           18   13   10
  //   256 x 4096 x 4096 (256)                       17   13   11
  if (M > 64 && tiles(128, 128) >= 192) launch_tile<128, 128>(g, bf16, st);
  else if (M > 64 && tiles(64, 128) >= 224) launch_tile<64, 128>(g, bf16, st);
  else if (M > 32 && tiles(64, 64) >= 160) {
    if (g.turn) launch_tile<64, 64, true>(g, bf16, st);
    else launch_tile<64, 64>(g, bf16, st);
  }
  // fewer tiles: K split over the waves.  (These and the next times are of the
  // forms without g.turn, which takes 1 to 3 us off both sides.)  Tiles of 64 x
  // 64, rings of 32 x 64 and of 32 x 32:
  //   61 x 14336 x 4096 (224 tiles of 64 x 64)      18    -   23
  //   256 x 4096 x 14336 (256)                      37   48    -
  //   128 x 4096 x 14336 (128; 256 of 32 x 64)      37   27   33
  //   61 x 4096 x 14336 (64; 128)                   38    -   21
  else if (M > 64 && tiles(32, 64) >= 200) launch_ring<2, 4, 4, 2>(g, bf16, st);
  // rings of 32 x 32 or 32 x 16, 16 x 32 or 16 x 16: enough workgroups, then
  // fewer reads of A.  32 columns a workgroup from 384 workgroups on, one and a
  // half a CU (us with 32 and with 16 columns; from 256 workgroups to there
  // either may win):
  //                         N = 4096     8192        10240       12288       14336       28672
  //   16 x N x 4096      6.2   6.1    8.7  9.3   12.9 12.7   13.6 14.9   14.1 16.7   25.3 28.5
  //   32 x N x 4096      6.7   6.4    9.4 11.0   14.8 15.4   15.5 17.6   16.4 20.3   28.6 33.9
  //   16 x N x 14336    18.3  14.7   22.9 26.1      -         38.9 37.9      -           -
  //   32 x N x 14336    22.1  18.1   25.6 33.0      -         44.2 48.2      -           -
  else if (M > 32 || (M > 16 && N >= 12288)) launch_ring<2, 2, 4, 2>(g, bf16, st);
  else if (M > 16) launch_ring<2, 1, 4, 3>(g, bf16, st);
  // up to 4 rows read A's lines so seldom that LDS does not pay, from the same
  // number of columns on (us without it and with the ring of 16, K = 4096: one row
  // through 8192 columns 8.3 and 8.8, 12288 11.7 and 13.6, 28672 22 and 26; 4 rows
  // 8.8 and 8.9, 12.3 and 13.8, 24 and 26; 8 rows through 28672 28 and 26; K =
  // 14336, where the ring is the faster: 4 rows through 12288 36 and 33)
  else if (M <= 4 && N >= 12288) launch_few(g, bf16, st);
  else if (N >= 12288) launch_ring<1, 2, 4, 2>(g, bf16, st);
  else launch_ring<1, 1, 4, 4>(g, bf16, st);
}

}  // namespace qsg
