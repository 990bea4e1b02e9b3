// Device code of the linear layer for few rows (at most 16: the tokens of a decode step).  The
// product is then a pass over the weights b, which are read once, straight into registers; the
// k range is divided among the waves of a workgroup, whose sums meet in LDS.
#pragma once

#include "linear_kernels.hpp"

namespace lk {

template <int TY>
__device__ __forceinline__ void mma16x16(float4v& acc, const int4v& a, const int4v& b) {
  if constexpr (TY == kF16)
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a),
                                                 __builtin_bit_cast(half8, b), acc, 0, 0, 0);
  else
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), acc, 0, 0, 0);
}

__device__ __forceinline__ int4v load16(const uint16_t* p) {
  return __builtin_bit_cast(int4v, *(const u32x4_any*)p);
}
// 16 bytes of a k-contiguous row from k element k on; elements past K are 0 and not read.
template <int TY>
__device__ __forceinline__ int4v load16_tail(const uint16_t* row, int k, int K) {
  constexpr int E = TY == kE4M3 ? 16 : 8;
  if (k + E <= K) return load16(row + (TY == kE4M3 ? k / 2 : k));
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if (k + e < K) {
      if (TY == kE4M3)
        v[e / 4] |= (uint32_t)((const uint8_t*)row)[k + e] << (8 * (e % 4));
      else
        v[e / 2] |= (uint32_t)row[k + e] << (16 * (e % 2));
    }
  }
  return __builtin_bit_cast(int4v, v);
}

// The waves' sums of a 16 x NC block, acc(c)[v] of lane l being row 4 (l / 16) + v, column
// col_of(c, l % 16), added in wave order, then the epilogue (or the split's partial sums).
template <int TY, int NW, int NC, int NB, class ColOf>
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
  // 8 columns of one row a thread; each output element is one thread's sum in wave order
  for (int t = tid; t < 16 * NC / 8; t += NW * 64) {
    const int row = t / (NC / 8), cc = t % (NC / 8) * 8, col = n0 + cc;
    if (row >= p.M || col >= p.N) continue;
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = 0.f;
#pragma unroll
    for (int u = 0; u < NW; ++u)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] += s[(u * 16 + row) * LDC + cc + e];
    if (W != nullptr) {
      float* const o = W + row * NC + cc;
      *(float4v*)o = float4v{f[0], f[1], f[2], f[3]};
      *(float4v*)(o + 4) = float4v{f[4], f[5], f[6], f[7]};
    } else {
      finish8<TY>(p, row, col, f, load_columns<TY>(p, col));
    }
  }
}

// b stored k-contiguous (column-major): 16 NB columns a workgroup.  One unit is 128 bytes of
// every row: lane l takes the 16-byte chunks l / 16 and 4 + l / 16 of row l % 16, of a and of b
// alike, so the order of k inside the unit is the same for both.  The loads of U units are in
// flight at once.
template <int TY, int NB, int NW>
__global__ void __launch_bounds__(64 * NW) lin_skinny_k(LinArgs p) {
  constexpr int UE = TY == kE4M3 ? 128 : 64, CE = UE / 8;   // elements of a unit, of a chunk
  constexpr int NC = 16 * NB, U = NB == 1 ? 4 : 2;
  __shared__ float s[NW * 16 * (NC + 4)];
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Work wk = work_of<16, NC>(p, blockIdx.x);
  int m0, n0;
  corner_of<16, NC>(p, wk.tile, m0, n0);
  const int x = lane & 15, g = lane >> 4;
  // rows and columns that do not exist repeat the last one; their sums are not stored
  const uint16_t* const pa = p.A + (int64_t)(x < p.M ? x : p.M - 1) * p.lda;
  const uint16_t* pb[NB];
  float4v acc[NB];
#pragma unroll
  for (int c = 0; c < NB; ++c) {
    const int col = n0 + 16 * c + x;
    pb[c] = p.B + (int64_t)(col < p.N ? col : p.N - 1) * p.ldb;
    acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
  }
  auto mul = [&](int c, const int4v (&a)[2], const int4v (&b)[2]) __attribute__((always_inline)) {
    if constexpr (TY == kE4M3) {
      acc[c] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
          __builtin_shufflevector(a[0], a[1], 0, 1, 2, 3, 4, 5, 6, 7),
          __builtin_shufflevector(b[0], b[1], 0, 1, 2, 3, 4, 5, 6, 7), acc[c], 0, 0, 0, 0, 0, 0);
    } else {
      mma16x16<TY>(acc[c], a[0], b[0]);
      mma16x16<TY>(acc[c], a[1], b[1]);
    }
  };
  const int units = (p.K + UE - 1) / UE, whole = p.K / UE;
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
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int c = 0; c < NB; ++c) mul(c, a[i], b[i][c]);
  }
  for (; u < u1; u += NW) {
    int4v a[2], b[NB][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = u * UE + (h * 4 + g) * CE;
#pragma unroll
      for (int c = 0; c < NB; ++c) b[c][h] = load16_tail<TY>(pb[c], k, p.K);
      a[h] = load16_tail<TY>(pa, k, p.K);
    }
#pragma unroll
    for (int c = 0; c < NB; ++c) mul(c, a, b[c]);
  }
  join_waves<TY, NW, NC>(p, acc, (float GK_LDS*)s, n0, wk.w,
                         [](int c, int i) { return c * 16 + i; });
}

// b stored n-contiguous (row-major): 16 CP columns a workgroup.  Lane l takes CP consecutive
// columns, from CP (l % 16) on, of the 8 k rows 8 (l / 16) .. + 7 of a 32-deep unit; pairs of
// rows are interleaved by byte permutes into k-runs, one MFMA operand per column.
template <int TY, int CP, int NW>
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
  // a lane without whole columns reads whole ones further left and shifts; see `row`
  const uint16_t* const pb = p.B + (int64_t)(8 * g) * p.ldb + col;
  float4v acc[CP];
#pragma unroll
  for (int c = 0; c < CP; ++c) acc[c] = float4v{0.f, 0.f, 0.f, 0.f};
  auto row = [&](const uint16_t* q) __attribute__((always_inline)) {
    if (have >= CP) return (vec)*(const vec_any*)q;
    vec v;
#pragma unroll
    for (int d = 0; d < CP / 2; ++d)
      v[d] = (2 * d < have ? (uint32_t)q[2 * d] : 0u) |
             (2 * d + 1 < have ? (uint32_t)q[2 * d + 1] << 16 : 0u);
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
  const int units = (p.K + 31) / 32, whole = p.K / 32;
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
    for (int i = 0; i < U; ++i) mul(a[i], b[i]);
  }
  for (; u < u1; u += NW) {
    const int k = u * 32;
    vec b[8];
#pragma unroll
    for (int r = 0; r < 8; ++r)
      b[r] = k + 8 * g + r < p.K ? row(pb + ((int64_t)k + r) * p.ldb) : vec(0u);
    mul(load16_tail<TY>(pa - 8 * g, k + 8 * g, p.K), b);
  }
  join_waves<TY, NW, NC>(p, acc, (float GK_LDS*)s, n0, wk.w,
                         [](int c, int i) { return i * CP + c; });
}

}  // namespace lk
