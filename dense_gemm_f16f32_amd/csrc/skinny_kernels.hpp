// Device code of the linear layer for few rows (at most 16: the tokens of a decode step).  The
// product is then a pass over the weights b, which are read once, straight into registers; the
// k range is divided among the waves of a workgroup, whose sums meet in LDS.  A result of at most
// 16 columns (a sliver past the last whole tile, a narrow layer) is the same with the operands
// exchanged: a pass over a.
#pragma once

#include "linear_kernels.hpp"

namespace lk {

template <int TY>
__device__ __forceinline__ void mma16x16(float4v& acc, const int4v& a, const int4v& b) {
  if constexpr (TY == kI8)
    acc = __builtin_bit_cast(
        float4v, __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, __builtin_bit_cast(int4v, acc), 0, 0,
                                                       0));
  else if constexpr (TY == kF16)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                 __builtin_bit_cast(half8, b), acc, 0, 0, 0);
  else
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}

__device__ __forceinline__ int4v load16(const uint16_t* p) {
  return __builtin_bit_cast(int4v, *(const u32x4_any*)p);
}
// 16 bytes of a k-contiguous row of K elements, from element k on; past the row's end they are 0
// and not read.  chunk_load takes the row's last 16 bytes there, and chunk_shift moves them.  No
// branch stands before a load or between loads: after one, the compiler waits for them.  Rows
// below 16 bytes (SHORT) are read element by element.  k is unsigned: past the end of the longest
// row it does not fit 31 bits.
template <int TY, bool SHORT>
__device__ __forceinline__ u32x4 chunk_load(const uint16_t* row, uint32_t k, uint32_t K) {
  constexpr int E = kBytes<TY> ? 16 : 8, B = 16 / E;
  if constexpr (!SHORT) {
    typedef u32x4 any __attribute__((aligned(1)));
    const uint32_t at = k + E <= K ? k : K - E;
    return *(const any*)((const char*)row + (int64_t)at * B);
  }
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < E - 1; ++e) {
    if (k + e < K) {
      if (kBytes<TY>)
        v[e / 4] |= (uint32_t)((const uint8_t*)row)[k + e] << (8 * (e % 4));
      else
        v[e / 2] |= (uint32_t)row[k + e] << (16 * (e % 2));
    }
  }
  return v;
}
// `live`: whether the chunk counts at all (else 0).
template <int TY, bool SHORT>
__device__ __forceinline__ int4v chunk_shift(u32x4 v, uint32_t k, uint32_t K, bool live) {
  constexpr int E = kBytes<TY> ? 16 : 8, B = 16 / E;
  if (!live) v = u32x4{0u, 0u, 0u, 0u};
  if (!SHORT && k + E > K) v = shift_down(v, (int)(8 * B * (k + E - K)));
  return __builtin_bit_cast(int4v, v);
}

// The waves' sums of a 16 x NC block, acc(c)[v] of lane l being row 4 (l / 16) + v, column
// col_of(c, l % 16), added in wave order, then the epilogue (or the split's partial sums).  FLIP: the
// block's rows are columns of the result, its columns rows from n0 on.
template <int TY, int NW, int NC, int MORE, bool FLIP, int NB, class ColOf>
__device__ __forceinline__ void join_waves(const LinArgs& p, const float4v (&acc)[NB],
                                           float GK_LDS* s, int n0, float* W, ColOf col_of) {
  constexpr int LDC = NC + 4;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
#pragma unroll
  for (int c = 0; c < NB; ++c)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      s[(w * 16 + 4 * (lane >> 4) + v) * LDC + col_of(c, lane & 15)] = acc[c][v];
  __syncthreads();
  if constexpr (FLIP) {
    // 8 columns of one row a thread, with the other 16 of a packed block
    constexpr int Q = MORE == kPack ? 4 : 2;
    for (int t = tid; t < NC * Q; t += NW * 64) {
      const int i = t / Q, col = t % Q * 8, row = n0 + i;
      if (!takes_part<MORE>(p, row, col)) continue;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = 0.f;
      if (col < 16) {
#pragma unroll
        for (int u = 0; u < NW; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = sum_add<TY>(f[e], s[(u * 16 + col + e) * LDC + i]);
      }
      finish8<TY, MORE>(p, row, col, f, load_columns<TY>(p, col));
    }
    return;
  }
  // 8 columns of one row a thread; each output element is one thread's sum in wave order
  for (int t = tid; t < 16 * NC / 8; t += NW * 64) {
    const int row = t / (NC / 8), cc = t % (NC / 8) * 8, col = n0 + cc;
    if (!takes_part<MORE>(p, row, col)) continue;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
    for (int u = 0; u < NW; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = sum_add<TY>(f[e], s[(u * 16 + row) * LDC + cc + e]);
    if (W != nullptr) {
      float* const o = W + row * NC + cc;
      *(float4v*)o = float4v{f[0], f[1], f[2], f[3]};
      *(float4v*)(o + 4) = float4v{f[4], f[5], f[6], f[7]};
    } else {
      finish8<TY, MORE>(p, row, col, f, load_columns<TY>(p, col));
    }
  }
}

// b stored k-contiguous (column-major): 16 NB columns a workgroup.  One unit is 128 bytes of
// every row: lane l takes the 16-byte chunks l / 16 and 4 + l / 16 of row l % 16, of a and of b
// alike, so the order of k inside the unit is the same for both.  The loads of U units are in
// flight at once.  HBM bounds it.  With other weights in between (2 GiB of them in turn): 1 x 16384
// x 4096 bf16 26.9 us (5.0 TB/s), 16 x 16384 x 4096 30.1 us (4.5 TB/s), 16 x 8192 x 8192 e4m3 17.0
// us (3.9 TB/s) and 4.3 for its two slices' join.  The same weights again and again stay partly in
// the last-level cache: 24.7, 23.4 and 13.7 us.  int8 with bias and
// gelu_tanh, from memory / the same weights: 1 x 16384 x 4096 16.2 / 15.5 us (4.1 TB/s), 8 rows 18.9 /
// 17.8, 16 rows 17.5 / 15.1, 16 x 8192 x 8192 20.2 / 17.4 with its join.  FLIP: the rows of the product
// are b's (at most 16 columns of the result) and what streams is a: 4096 x 1 x 4096 bf16 10.5 us from
// memory (3.2 TB/s), 6.4 with a partly in the last-level cache; int8 6.3 from memory.
template <int TY, int NB, int NW, bool SHORT, int MORE, bool FLIP>
__global__ void __launch_bounds__(64 * NW) lin_skinny_k(LinArgs p) {
  constexpr int UE = kBytes<TY> ? 128 : 64, CE = UE / 8;   // elements of a unit, of a chunk
  constexpr int NC = 16 * NB, U = 4;
  __shared__ float s[NW * 16 * (NC + 4)];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Work wk = work_of<16, NC>(p, blockIdx.x);
  int m0, n0;
  corner_of<16, NC>(p, wk.tile, m0, n0);
  const int x = lane & 15, g = lane >> 4;
  // rows and columns that do not exist repeat the last one; their sums are not stored
  const uint16_t* const A = FLIP ? p.B : p.A;
  const uint16_t* const B = FLIP ? p.A : p.B;
  const int64_t lda = FLIP ? p.ldb : p.lda, ldb = FLIP ? p.lda : p.ldb;
  const int M = FLIP ? p.N : p.M, N = FLIP ? p.M : p.N;
  const uint16_t* const pa = A + (int64_t)(x < M ? x : M - 1) * lda;
  const uint16_t* pb[NB];
  float4v acc[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int col = n0 + 16 * c + x;
    pb[c] = B + (int64_t)(col < N ? col : N - 1) * ldb;
    acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
  }
  auto mul = [&](int c, const int4v (&a)[2], const int4v (&b)[2]) __attribute__((always_inline)) {
    if constexpr (TY == kE4M3) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int d = 0; d < 4; d += 2)
          mma16x16<kF16>(acc[c], halves(a[h][d], a[h][d + 1]), halves(b[h][d], b[h][d + 1]));
    } else {
      mma16x16<TY>(acc[c], a[0], b[0]);
      mma16x16<TY>(acc[c], a[1], b[1]);
    }
  };
  const int whole = p.K / UE, units = whole + (p.K % UE != 0);
  const int u0 = wk.z < 0 ? 0 : wk.z * p.per_split;
  const int u1 = wk.z >= 0 && u0 + p.per_split < units ? u0 + p.per_split : units;
  const int uw = u1 < whole ? u1 : whole;
  int u = u0 + w;
  for (; u + (U - 1) * NW < uw; u += U * NW) {
    int4v a[U][2], b[U][NB][2];
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t k = (int64_t)(u + i * NW) * 64 + (h * 4 + g) * 8;   // in 16-bit slots
#pragma unroll
        for (int c = 0; c < NB; ++c) b[i][c][h] = load16(pb[c] + k);
        a[i][h] = load16(pa + k);
      }
    // Every load is on its way before the first is used.  With one block of 16-bit columns the
    // waves are many and small, and do without (weights partly in the last-level cache: 16 rows of
    // e4m3, 8192 x 8192: 18.9 -> 16.7 us; one of bf16, 16384 x 4096: 23.1 without, 24.0 with).
    if constexpr (NB > 1 || kBytes<TY>) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int c = 0; c < NB; ++c) mul(c, a[i], b[i][c]);
  }
  for (; u < u1; u += NW) {   // this wave's last units, the matrix's ragged one among them
    u32x4 a[2], b[NB][2];
    uint32_t k[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      k[h] = (uint32_t)u * UE + (h * 4 + g) * CE;
#pragma unroll
      for (int c = 0; c < NB; ++c) b[c][h] = chunk_load<TY, SHORT>(pb[c], k[h], p.K);
      a[h] = chunk_load<TY, SHORT>(pa, k[h], p.K);
    }
    int4v av[2], bv[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) av[h] = chunk_shift<TY, SHORT>(a[h], k[h], p.K, true);
#pragma unroll
    for (int c = 0; c < NB; ++c) {
#pragma unroll
      for (int h = 0; h < 2; ++h) bv[h] = chunk_shift<TY, SHORT>(b[c][h], k[h], p.K, true);
      mul(c, av, bv);
    }
  }
  join_waves<TY, NW, NC, MORE, FLIP>(p, acc, (float GK_LDS*)s, n0, wk.w,
                                     [](int c, int i) { return c * 16 + i; });
}

// b stored n-contiguous (row-major): 16 CP columns a workgroup.  Lane l takes CP consecutive
// columns, from CP (l % 16) on, of the 8 k rows 8 (l / 16) .. + 7 of a 32-deep unit; pairs of
// rows are interleaved by byte permutes into k-runs, one MFMA operand per column.  64 columns a
// workgroup: a wave's load covers 128 bytes of four k rows.  HBM bounds it: 1 x 16384 x 4096 bf16
// 25.7 us (5.2 TB/s) with other weights in between, 21.5 with these partly in the last-level cache.
// Rows of b at any 2-byte address: a k row's 128 bytes touch two lines, 1 x 8191 x 8191 38.8 us
// (3.5 TB/s) either way.
template <int TY, int CP, int NW, int MORE>
__global__ void __launch_bounds__(64 * NW) lin_skinny_n(LinArgs p) {
  constexpr int NC = 16 * CP;
  typedef uint32_t vec __attribute__((ext_vector_type(CP / 2)));
  typedef vec vec_any __attribute__((aligned(2)));
  __shared__ float s[NW * 16 * (NC + 4)];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Work wk = work_of<16, NC>(p, blockIdx.x);
  int m0, n0;
  corner_of<16, NC>(p, wk.tile, m0, n0);
  const int x = lane & 15, g = lane >> 4;
  const uint16_t* const pa = p.A + (int64_t)(x < p.M ? x : p.M - 1) * p.lda + 8 * g;
  const int col = n0 + x * CP;
  const int have = p.N - col;          // this lane's columns that exist
  // a lane without CP columns reads the row's last CP and shifts (rows have at least CP)
  const int over = have >= CP ? 0 : CP - have;
  const uint16_t* const pb = p.B + (int64_t)(8 * g) * p.ldb + col - over;
  float4v acc[CP];
#pragma unroll
  for (int c = 0; c < CP; ++c) acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
  auto row = [&](const uint16_t* q) __attribute__((always_inline)) {
    return (vec)*(const vec_any*)q;
  };
  auto shift = [&](vec v) __attribute__((always_inline)) {
    static_assert(CP == 4, "64 bits");
    if (over > 0) {
      const uint64_t b = over >= 4 ? 0 : __builtin_bit_cast(uint64_t, v) >> (16 * over);
      v = __builtin_bit_cast(vec, b);
    }
    return v;
  };
  auto mul = [&](const int4v& a, const vec (&b)[8]) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      u32x4 o;
      // low or high halves of two rows' words side by side
#pragma unroll
      for (int d = 0; d < 4; ++d)
        o[d] = __builtin_amdgcn_perm(b[2 * d + 1][c / 2], b[2 * d][c / 2],
                                     (c & 1) ? 0x07060302u : 0x05040100u);
      mma16x16<TY>(acc[c], a, __builtin_bit_cast(int4v, o));
    }
  };
  const int whole = p.K / 32, units = whole + (p.K % 32 != 0);
  const int u0 = wk.z < 0 ? 0 : wk.z * p.per_split;
  const int u1 = wk.z >= 0 && u0 + p.per_split < units ? u0 + p.per_split : units;
  const int uw = u1 < whole ? u1 : whole;
  constexpr int U = 2;
  int u = u0 + w;
  for (; u + (U - 1) * NW < uw; u += U * NW) {
    int4v a[U];
    vec b[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t k = (int64_t)(u + i * NW) * 32;
#pragma unroll
      for (int r = 0; r < 8; ++r) b[i][r] = row(pb + (k + r) * p.ldb);
      a[i] = load16(pa + k);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
#pragma unroll
      for (int r = 0; r < 8; ++r) b[i][r] = shift(b[i][r]);
      mul(a[i], b[i]);
    }
  }
  if (u < u1) {   // this wave's last units, at most U, the matrix's ragged one among them
    u32x4 a[U];
    vec b[U][8];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = (u + i * NW < u1 ? u + i * NW : u1 - 1) * 32 + 8 * g;
#pragma unroll
      for (int r = 0; r < 8; ++r) {   // k rows past the last: the last one, not counted
        const int kr = k + r < p.K ? k + r : p.K - 1;
        b[i][r] = row(pb + (int64_t)(kr - 8 * g) * p.ldb);
      }
      a[i] = chunk_load<TY, false>(pa - 8 * g, k, p.K);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool live = u + i * NW < u1;
      const int k = (live ? u + i * NW : u1 - 1) * 32 + 8 * g;
#pragma unroll
      for (int r = 0; r < 8; ++r) b[i][r] = live && k + r < p.K ? shift(b[i][r]) : vec(0u);
      mul(chunk_shift<TY, false>(a[i], k, p.K, live), b[i]);
    }
  }
  join_waves<TY, NW, NC, MORE, false>(p, acc, (float GK_LDS*)s, n0, wk.w,
                                      [](int c, int i) { return i * CP + c; });
}

}  // namespace lk
