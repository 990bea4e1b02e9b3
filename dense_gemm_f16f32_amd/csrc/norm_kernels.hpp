// Device code of the root-mean-square norm and the layer norm, their backward passes, rows in 8 bits,
// and the element-wise part of the linear layer's backward pass.  All of them move each element
// once; HBM bounds them.
#pragma once

#include "linear_kernels.hpp"

namespace nk {

using namespace lk;

// Sum over the NW waves of a workgroup, given to every thread; `s` holds NW floats.
template <int NW>
__device__ __forceinline__ float group_sum(float v, float* s) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NW; ++i) v += s[i];
  }
  return v;
}
// Sum over a wave, all of whose lanes are active, by moves between lanes inside the vector unit: a
// step takes some ten cycles, and one through LDS (__shfl_xor) about a hundred.
template <int CTRL>
__device__ __forceinline__ float lane_move(float v) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int lane = 0) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float row_sum16(float v) {   // over each 16 lanes, in all of them
  v += lane_move<0xB1>(v);    // quads: 1 0 3 2
  v += lane_move<0x4E>(v);    // 2 3 0 1
  v += lane_move<0x141>(v);   // 8 lanes mirrored
  v += lane_move<0x140>(v);   // 16 lanes mirrored
  return v;
}
__device__ __forceinline__ float row_sum(float v) { return lane_value(row_sum16(v)); }
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum16(v);
  return (lane_value(v) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}
// Two sums at once; `s` holds 2 NW floats.
template <int NW>
__device__ __forceinline__ float2v group_sum2(float2v v, float* s) {
  v = float2v{wave_sum(v[0]), wave_sum(v[1])};
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) {
      s[2 * (threadIdx.x >> 6)] = v[0];
      s[2 * (threadIdx.x >> 6) + 1] = v[1];
    }
    __syncthreads();
    v = float2v{0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      v[0] += s[2 * i];
      v[1] += s[2 * i + 1];
    }
  }
  return v;
}
template <int NW>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* s) {
  v = quad_max(v);
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true);
  v = v > o ? v : o;
  uint32_t r = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = (uint32_t)__builtin_amdgcn_readlane((int)v, 16 * i);
    r = r > x ? r : x;
  }
  v = r;
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0u;
#pragma unroll
    for (int i = 0; i < NW; ++i) v = v > s[i] ? v : s[i];
  }
  return v;
}

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;
  const uint16_t* weight;
  const uint16_t* bias;   // layer norm only; may be null
  void* y;
  float* scale;
  uint16_t* h;
  float* mean;   // layer norm only
  float* rstd;
  int64_t x_row, res_row, y_row, h_row;
  int32_t rows, dim;
  float eps, inv_dim;
};

// scale of a row in e4m3 from the bits of its largest magnitude (NaN sorts above infinity).  A
// row of zeros, or one that holds a NaN, takes 1.  The lower bound keeps 1 / scale finite for
// rows below 448 2^-126.
__device__ __forceinline__ float e4m3_scale(uint32_t amax_bits) {
  const float amax = __builtin_bit_cast(float, amax_bits);
  return amax > 0.f ? fmaxf(amax / 448.f, 1.17549435e-38f) : 1.f;
}
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}
// A row's 8-bit scale, with what a division by it takes: the rounded reciprocal, and the scale
// again for the remainder (0 for an infinite scale, whose quotients are 0, or NaN).
struct Divisor {
  float inv, scale;
};
__device__ __forceinline__ Divisor divisor(float scale) {
  return {1.f / scale, scale <= 3.40282347e38f ? scale : 0.f};
}
// v / scale: the product with the rounded reciprocal, and the remainder that it leaves (exact in
// one fma) divided the same way.  Without that step the quotient is off by up to 2^-23 of itself
// and crosses a tie of the 8-bit rounding once in about 2^20 values.
__device__ __forceinline__ float quotient(float v, Divisor d) {
  const float q = v * d.inv;
  return __builtin_fmaf(__builtin_fmaf(-q, d.scale, v), d.inv, q);
}
// 8 quotients to e4m3, nearest, ties to even (at most 448 up to the rounding of the scale)
__device__ __forceinline__ uint2 to_e4m3x8(const float (&v)[8], Divisor d) {
  float q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) q[e] = quotient(v[e], d);
  uint2 o;
  int lo = 0, hi = 0;
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], lo, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], hi, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
  o.x = (uint32_t)lo;
  o.y = (uint32_t)hi;
  return o;
}
// scale of a row in int8: the largest magnitude over 127 (1 for a row of zeros), the quotient in
// fp32.  The integers cannot hold a NaN: a row with one, or with an infinity, has a scale that
// makes every product with it NaN.
__device__ __forceinline__ float int8_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7F800000u) return __builtin_nanf("");
  const float amax = __builtin_bit_cast(float, amax_bits);
  return amax > 0.f ? fmaxf(amax / 127.f, 1.17549435e-38f) : 1.f;
}
// 8 quotients to integers, nearest, ties to even (the addition rounds, and leaves the integer in the
// low bits).  The clamp catches the scale's own rounding, and turns NaN into a number.
__device__ __forceinline__ uint2 to_int8x8(const float (&v)[8], Divisor d) {
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    q[e] = __builtin_bit_cast(
        uint32_t, __builtin_amdgcn_fmed3f(quotient(v[e], d), -127.f, 127.f) + 12582912.f);
  auto bytes = [&](int i) __attribute__((always_inline)) {
    const uint32_t x = __builtin_amdgcn_perm(q[i + 1], q[i], 0x0C0C0400u);
    const uint32_t y = __builtin_amdgcn_perm(q[i + 3], q[i + 2], 0x0C0C0400u);
    return x | (y << 16);
  };
  return uint2{bytes(0), bytes(4)};
}

// What rows are stored as: their own 16-bit type, or 8 bits with a scale a row.
enum { kOut16, kOutE4M3, kOutI8 };
template <int OUT>
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  return OUT == kOutI8 ? int8_scale(amax_bits) : e4m3_scale(amax_bits);
}
template <int OUT>
__device__ __forceinline__ void store_row8(uint8_t* p, const float (&v)[8], Divisor d, int n) {
  const uint2 q = OUT == kOutI8 ? to_int8x8(v, d) : to_e4m3x8(v, d);
  store_bytes8(p, q.x, q.y, n);
}
__device__ __forceinline__ uint32_t max_bits8(const float (&v)[8], uint32_t m) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = abs_bits(v[e]);
    m = m > b ? m : b;
  }
  return m;
}

// One pass: the row's statistics, the 8-bit scale and y come from the row in registers.  HBM bounds
// it: 8192 x 8192 bf16 with residual to e4m3 88 us (5.3 TB/s), 4095 x 4093 f16 29 us (4.6 TB/s; 24.5
// where the rows are partly in the last-level cache); the layer norm 8192 x 8192 bf16 100 - 107 us (5.0 -
// 5.4 TB/s; with three barriers and sums through LDS 106 where this takes 100), to int8 or e4m3 96, 4096 x
// 16384 105, one row of 4096 to e4m3 3.6.  Rows above 16384 are read three times, four to 8 bits: 4096 x
// 32768 362 us, to int8 402.
// One row a workgroup of 64 NW threads, 8 columns a thread at a time.  C > 0: rows of at most
// 512 NW C columns, held in registers.  C == 0: longer rows, read again for each step that
// needs them.
//
// LN (the layer norm): each wave takes the mean of its own columns, m_w, and the sums of the
// differences c from it and of their squares, s_w and q_w (s_w would be 0 but for the mean's
// rounding).  They meet once: with n_w columns a wave and e_w = m_w - m_0,
//   d = sum(n_w e_w + s_w) / n;  mean = m_0 + d
//   var = sum(q_w + 2 (e_w - d) s_w + n_w (e_w - d)^2) / n
// all in differences, so that rows far from 0 keep their deviation's bits (a mean of squares less
// the mean's square would lose them), and with one barrier (with the row's mean first it took
// three).
template <int TY, int OUT, bool LN, int NW, int C>
__global__ void __launch_bounds__(64 * NW) norm_fwd(NormArgs p) {
  const bool back = p.dim >= 8;
  __shared__ float ssum[LN ? 1 : NW];
  __shared__ float4v swave[LN ? 2 : 1][LN ? NW : 1];
  __shared__ uint32_t smax[NW];
  constexpr int STEP = 512 * NW, CR = C > 0 ? C : 1;
  const int64_t row = blockIdx.x;
  const uint16_t* const x = p.x + row * p.x_row;
  const uint16_t* const res = p.res ? p.res + row * p.res_row : nullptr;
  uint16_t* const h = p.h ? p.h + row * p.h_row : nullptr;
  const uint32_t c0 = threadIdx.x * 8, dim = p.dim;   // col and dim + STEP fit 32 bits
  const auto left = [&](uint32_t col) { return (int)(dim - col); };   // columns from col on
  const int steps = C > 0 ? C : (p.dim - 1) / STEP + 1;   // dim > 0
  float hv[CR][8], wv[CR][8], bv[CR][8];
  float own = 0.f, mean = 0.f, shift = 0.f;   // layer norm: the wave's mean, the row's, d - e_w
  auto load_h = [&](uint32_t col, float (&v)[8]) __attribute__((always_inline)) {
    load8(v, x + col, left(col), TY, back);
    if (res) {
      float r[8];
      load8(r, res + col, left(col), TY, back);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
  };
  auto load_bias = [&](uint32_t col, float (&v)[8]) __attribute__((always_inline)) {
    if (LN && p.bias) {
      load8(v, p.bias + col, left(col), TY, back);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
  };
  // differences from the wave's mean; columns past dim stay 0
  auto centre = [&](uint32_t col, float (&v)[8]) __attribute__((always_inline)) {
    if constexpr (LN) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = e < left(col) ? v[e] - own : 0.f;
    }
  };
  float2v sum = {0.f, 0.f};   // of the values or differences (layer norm), of their squares
  auto add = [&](const float (&v)[8], float unit) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = v[e] * unit;
      if constexpr (LN) sum[0] += u;
      sum[1] += u * u;
    }
  };
  // columns of wave w
  auto columns = [&](int w) __attribute__((always_inline)) {
    const int rest = p.dim % STEP - 512 * w;
    return (float)(p.dim / STEP * 512 + (rest < 0 ? 0 : rest < 512 ? rest : 512));
  };
  // mean of the squares (layer norm: about the mean) and eps, in units of 1 / unit^2
  auto moments = [&](float unit, int turn) __attribute__((always_inline)) {
    if constexpr (LN) {
      const float s1 = wave_sum(sum[0]), q = wave_sum(sum[1]);
      float var;
      if constexpr (NW == 1) {
        const float d = s1 * p.inv_dim;
        var = q * p.inv_dim - d * d;
        shift = d / unit;
        mean = own + shift;
      } else {
        float4v(&sw)[NW] = swave[turn];
        if ((threadIdx.x & 63) == 0) sw[threadIdx.x >> 6] = float4v{own, s1, q, 0.f};
        __syncthreads();
        // lane w mod 16 takes wave w's part
        const int w = threadIdx.x & 15;
        const float n = w < NW ? columns(w) : 0.f;
        const float4v t = sw[w < NW ? w : 0];
        const float m0 = lane_value(t[0]);
        const float e = n > 0.f ? (t[0] - m0) * unit : 0.f;
        const float d = row_sum(n > 0.f ? (n * e + t[1]) * p.inv_dim : 0.f);
        const float f = e - d;
        var = row_sum(n > 0.f ? (t[2] + 2.f * f * t[1] + n * f * f) * p.inv_dim : 0.f);
        mean = m0 + d / unit;
        shift = d / unit - (own - m0);
      }
      return (var < 0.f ? 0.f : var) + p.eps * unit * unit;   // NaN stays
    } else {
      return group_sum<NW>(sum[1], ssum) * p.inv_dim + p.eps * unit * unit;
    }
  };
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) load_h(c0 + i * STEP, hv[i]);
#pragma unroll
    for (int i = 0; i < C; ++i) load8(wv[i], p.weight + c0 + i * STEP, left(c0 + i * STEP), TY, back);
    if constexpr (LN) {
#pragma unroll
      for (int i = 0; i < C; ++i) load_bias(c0 + i * STEP, bv[i]);
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const uint32_t col = c0 + (uint32_t)i * STEP;
      if (h && col < dim) store8(h + col, hv[i], left(col), TY);
    }
  }
  if constexpr (LN) {
    // terms of the mean, not of the sum: it cannot leave fp32's range where the values have not
    const float n = columns(threadIdx.x >> 6), inv = n > 0.f ? 1.f / n : 0.f;
#pragma unroll CR
    for (int i = 0; i < steps; ++i) {
      if constexpr (C == 0) load_h(c0 + i * STEP, hv[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) own += hv[C > 0 ? i : 0][e] * inv;
    }
    own = wave_sum(own);
  }
#pragma unroll CR
  for (int i = 0; i < steps; ++i) {
    if constexpr (C == 0) load_h(c0 + i * STEP, hv[0]);
    centre(c0 + i * STEP, hv[C > 0 ? i : 0]);
    add(hv[C > 0 ? i : 0], 1.f);
  }
  float square = moments(1.f, 0), unit = 1.f;
  // Squares outside fp32's range (bf16 rows above 1e19, or below 1e-9 with a tiny eps) are summed
  // again in units that bring them into it; every thread of the row holds the same sum.  (The layer
  // norm's infinite sum less its infinite correction is NaN.)
  if (square < 0x1p-60f || square == __builtin_inff() || (LN && square != square)) {
    unit = square < 1.f ? 0x1p64f : 0x1p-96f;
    if constexpr (NW > 1 && !LN) __syncthreads();   // the first sum has been read
    sum = float2v{0.f, 0.f};
#pragma unroll CR
    for (int i = 0; i < steps; ++i) {
      if constexpr (C == 0) {
        load_h(c0 + i * STEP, hv[0]);
        centre(c0 + i * STEP, hv[0]);
      }
      add(hv[C > 0 ? i : 0], unit);
    }
    square = moments(unit, 1);
  }
  const float rstd = unit / sqrtf(square);
  if (threadIdx.x == 0) {
    if (p.rstd) p.rstd[row] = rstd;
    if (LN && p.mean) p.mean[row] = mean;
  }
  // y of step i
  auto norm = [&](int i, float (&v)[8]) __attribute__((always_inline)) {
    const uint32_t col = c0 + (uint32_t)i * STEP;
    float w[8], b[8];
    if constexpr (C == 0) {
      load_h(col, v);
      centre(col, v);
      load8(w, p.weight + col, left(col), TY, back);
      if constexpr (LN) load_bias(col, b);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float u = C > 0 ? hv[i][e] : v[e], g = C > 0 ? wv[i][e] : w[e];
      if constexpr (LN)
        v[e] = (u - shift) * rstd * g + (C > 0 ? bv[i][e] : b[e]);
      else
        v[e] = u * rstd * g;
    }
  };
  Divisor by = {1.f, 1.f};
  if constexpr (OUT != kOut16) {
    uint32_t m = 0u;
#pragma unroll CR
    for (int i = 0; i < steps; ++i) {
      float v[8];
      norm(i, v);
      m = max_bits8(v, m);   // columns past dim are 0 (their weight and bias read as 0)
    }
    const float scale = row_scale<OUT>(group_max<NW>(m, smax));
    if (threadIdx.x == 0) p.scale[row] = scale;
    by = divisor(scale);
  }
#pragma unroll CR
  for (int i = 0; i < steps; ++i) {
    const uint32_t col = c0 + (uint32_t)i * STEP;
    if (col >= dim) break;
    float v[8];
    norm(i, v);
    if constexpr (OUT != kOut16)
      store_row8<OUT>((uint8_t*)p.y + row * p.y_row + col, v, by, left(col));
    else
      store8((uint16_t*)p.y + row * p.y_row + col, v, left(col), TY);
    // h may be x's or the residual's memory: without registers it is written last
    if constexpr (C == 0) {
      if (h) {
        load_h(col, v);
        store8(h + col, v, left(col), TY);
      }
    }
  }
}

// Rows in 8 bits with a scale a row, as the norm's: one row a workgroup, held in registers.  HBM bounds
// it: 8192 x 8192 bf16 to int8 38 us from and to memory (5.3 TB/s; e4m3 the same), 4095 x 4093 f16 14.3
// (3.5 TB/s), 10.6 on the same matrices, partly in the last-level cache.
struct QuantizeArgs {
  const uint16_t* x;
  uint8_t* y;
  float* scale;
  int64_t x_row, y_row;
  int32_t dim;
};
template <int TY, int OUT, int NW, int C>
__global__ void __launch_bounds__(64 * NW) quantize_rows(QuantizeArgs p) {
  const bool back = p.dim >= 8;
  __shared__ uint32_t smax[NW];
  constexpr int STEP = 512 * NW, CR = C > 0 ? C : 1;
  const int64_t row = blockIdx.x;
  const uint16_t* const x = p.x + row * p.x_row;
  const uint32_t c0 = threadIdx.x * 8, dim = p.dim;   // col and dim + STEP fit 32 bits
  const auto left = [&](uint32_t col) { return (int)(dim - col); };   // columns from col on
  const int steps = C > 0 ? C : (p.dim - 1) / STEP + 1;
  float xv[CR][8];
  uint32_t m = 0u;
#pragma unroll CR
  for (int i = 0; i < steps; ++i) {
    const uint32_t col = c0 + (uint32_t)i * STEP;
    load8(xv[C > 0 ? i : 0], x + col, left(col), TY, back);
    if constexpr (C == 0) m = max_bits8(xv[0], m);
  }
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) m = max_bits8(xv[i], m);
  }
  const float scale = row_scale<OUT>(group_max<NW>(m, smax));
  if (threadIdx.x == 0) p.scale[row] = scale;
  const Divisor by = divisor(scale);
#pragma unroll CR
  for (int i = 0; i < steps; ++i) {
    const uint32_t col = c0 + (uint32_t)i * STEP;
    if (col >= dim) break;
    if constexpr (C == 0) load8(xv[0], x + col, left(col), TY, back);
    store_row8<OUT>(p.y + row * p.y_row + col, xv[C > 0 ? i : 0], by, left(col));
  }
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const float* mean;   // layer norm only
  const float* rstd;
  const uint16_t* dh;
  uint16_t* dx;
  uint16_t* dweight;
  uint16_t* dbias;   // layer norm only
  // partial sums of every workgroup; null: dweight and dbias themselves, or nothing
  float* part;
  float* part_bias;
  int64_t dy_row, h_row, dh_row, dx_row;
  int32_t rows, dim;
  float inv_dim;
};

// Partial column sums: `groups` workgroups each leave one float a column, stored as blocks of 32
// columns by `groups` rows, so that the workgroup that adds a block's rows reads one contiguous
// piece.
__device__ __forceinline__ float* partial(float* part, int groups, int group, int col) {
  return part + ((int64_t)(col >> 5) * groups + group) * 32 + (col & 31);
}
__device__ __forceinline__ void store_partial8(float* part, int groups, int group, int col,
                                               const float (&v)[8]) {   // col: a multiple of 8
  float* const o = partial(part, groups, group, col);
  *(float4v*)o = float4v{v[0], v[1], v[2], v[3]};
  *(float4v*)(o + 4) = float4v{v[4], v[5], v[6], v[7]};
}

// RW rows of at most 512 NW C columns at a time, NW waves each: workgroup b takes rows b RW ..,
// (b + grid) RW .., ...; where registers allow, the next row's values are loaded before the
// current row is worked on.  Each thread keeps its columns' dweight sums in registers; the
// workgroup adds and writes them once (LN, the layer norm: dbias' sums too).  Short rows (one wave
// each) go four to a workgroup.  HBM bounds it: 8192 x 4096 bf16 50 us (5.4 TB/s of dy, h, dh and dx),
// and 5 for sum_partials; with the rows partly in the last-level cache 41 us, and there without the
// loads ahead 70.  The layer norm: 43 - 52 us, its two gradients' partial sums being twice as many (with
// their sum 57 - 63 from and to memory, 8192 x 8192 114).  Above 8192 columns, without loads ahead: 4096 x
// 12288 107 us with the sums (3.8 TB/s), 4096 x 16384 139 (3.9); the RMS norm 93 and 120.
// Without SUMS dx alone.
// (The arguments by value: by reference the RMS norm's kernels took up to 7 % longer, 9 x 2365 f16 3.53
// against 3.24 us.)
template <int TY, bool LN, int NW, int C, int RW, bool SUMS>
__device__ __forceinline__ void norm_bwd_rows(NormBwdArgs p, int group, int groups) {
  static_assert(NW == 1 || RW == 1, "rows of several waves share the workgroup's barrier");
  const bool back = p.dim >= 8;
  __shared__ float ssum[2][2 * NW];
  constexpr int STEP = 512 * NW, CB = LN ? C : 1;
  const int c0 = (RW > 1 ? threadIdx.x & 63 : threadIdx.x) * 8;
  const int rw = RW > 1 ? threadIdx.x >> 6 : 0;
  // With four steps of a row the layer norm's second set of sums leaves no registers for the
  // weights in fp32, nor for the row's values across the sum: both are unpacked twice.
  constexpr bool kTight = LN && C > 2;
  float wv[kTight ? 1 : C][8], dw[C][8], db[CB][8];
  u32x4 wr[kTight ? C : 1];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    if constexpr (kTight)
      wr[i] = raw8(p.weight + c0 + i * STEP, p.dim - c0 - i * STEP, back);
    else
      load8(wv[i], p.weight + c0 + i * STEP, p.dim - c0 - i * STEP, TY, back);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    if constexpr (LN) {
#pragma unroll
      for (int e = 0; e < 8; ++e) db[i][e] = 0.f;
    }
  }
  struct Row {
    u32x4 d[C], h[C], r[C];   // dy, h, dh
    float4v s;                // rstd, mean; a lone float's padding would be copied through memory
  };
  auto load = [&](Row& q, int64_t row) __attribute__((always_inline)) {
    q.s[0] = p.rstd[row];
    if constexpr (LN) q.s[1] = p.mean[row];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = c0 + i * STEP, n = p.dim - col;
      q.d[i] = raw8_load(p.dy + row * p.dy_row + col, n, back);
      q.h[i] = raw8_load(p.h + row * p.h_row + col, n, back);
      q.r[i] = p.dh ? raw8_load(p.dh + row * p.dh_row + col, n, back) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  constexpr bool kAhead = C <= 2;
  const int64_t first = (int64_t)group * RW + rw, step = (int64_t)groups * RW;
  Row cur, nxt;
  if (kAhead && first < p.rows) load(cur, first);
  int turn = 0;
  for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
    if (!kAhead) load(cur, row);
    nxt = cur;
    if (kAhead && row + step < p.rows) load(nxt, row + step);
    const float rstd = cur.s[0], mean = LN ? cur.s[1] : 0.f;
    float2v sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float d[8], x[8];
      const int n = p.dim - c0 - i * STEP;
      if constexpr (kTight) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(wr[i]));
        unpack8(wv[0], wr[i], TY);
      }
      cur.d[i] = raw8_shift(cur.d[i], n, back);
      cur.h[i] = raw8_shift(cur.h[i], n, back);
      cur.r[i] = raw8_shift(cur.r[i], n, back);
      unpack8(d, cur.d[i], TY);
      unpack8(x, cur.h[i], TY);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = LN ? (x[e] - mean) * rstd : x[e] * rstd;
        if constexpr (SUMS) dw[i][e] += d[e] * x[e];
        if constexpr (LN) {
          if constexpr (SUMS) db[i][e] += d[e];
          sum[1] += d[e] * wv[kTight ? 0 : i][e];
        }
        sum[0] += d[e] * wv[kTight ? 0 : i][e] * x[e];
      }
    }
    // two sets of sums in turn, so that one barrier a row is enough
    if constexpr (LN)
      sum = group_sum2<NW>(sum, ssum[turn]);
    else
      sum[0] = group_sum<NW>(sum[0], ssum[turn]);
    const float along = sum[0] * p.inv_dim, level = sum[1] * p.inv_dim;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = c0 + i * STEP;
      float d[8], x[8], r[8];
      if constexpr (kTight) {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("" : "+v"(cur.d[i]), "+v"(cur.h[i]), "+v"(wr[i]));
        unpack8(wv[0], wr[i], TY);
      }
      unpack8(d, cur.d[i], TY);
      unpack8(x, cur.h[i], TY);
      unpack8(r, cur.r[i], TY);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (LN)
          r[e] += rstd * (d[e] * wv[kTight ? 0 : i][e] - level - (x[e] - mean) * rstd * along);
        else
          r[e] += rstd * (d[e] * wv[kTight ? 0 : i][e] - x[e] * rstd * along);
      }
      if (col < p.dim) store8(p.dx + row * p.dx_row + col, r, p.dim - col, TY);
    }
    cur = nxt;
  }
  if constexpr (!SUMS) return;
  if (p.part == nullptr && p.dweight == nullptr &&
      (!LN || (p.part_bias == nullptr && p.dbias == nullptr)))
    return;
  if constexpr (RW > 1) {   // the other rows' sums, in their order
    __shared__ float sdw[RW - 1][(C + (LN ? C : 0)) * 512];
    if (rw > 0) {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sdw[rw - 1][(i * 8 + e) * 64 + (threadIdx.x & 63)] = dw[i][e];
      if constexpr (LN) {
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            sdw[rw - 1][((C + i) * 8 + e) * 64 + (threadIdx.x & 63)] = db[i][e];
      }
    }
    __syncthreads();
    if (rw > 0) return;
#pragma unroll
    for (int r = 0; r < RW - 1; ++r)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dw[i][e] += sdw[r][(i * 8 + e) * 64 + threadIdx.x];
          if constexpr (LN) db[i][e] += sdw[r][((C + i) * 8 + e) * 64 + threadIdx.x];
        }
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int col = c0 + i * STEP;
    if (col >= p.dim) continue;
    if (p.part != nullptr)
      store_partial8(p.part, groups, group, col, dw[i]);
    else if (p.dweight != nullptr)   // the only workgroup
      store8(p.dweight + col, dw[i], p.dim - col, TY);
    if constexpr (LN) {
      if (p.part_bias != nullptr)
        store_partial8(p.part_bias, groups, group, col, db[i]);
      else if (p.dbias != nullptr)
        store8(p.dbias + col, db[i], p.dim - col, TY);
    }
  }
}
template <int TY, bool LN, int NW, int C, int RW>
__global__ void __launch_bounds__(64 * NW * RW) norm_bwd(NormBwdArgs p) {
  norm_bwd_rows<TY, LN, NW, C, RW, true>(p, blockIdx.x, gridDim.x);
}

// The layer norm's weight and bias gradients of COLS columns over all rows, by a workgroup of T
// threads: 8 columns a thread, T / LANES rows at once.
template <int TY, int T, int COLS>
__device__ __forceinline__ void norm_columns(const NormBwdArgs& p, int block) {
  constexpr int R = 8, LANES = COLS / 8, STEP = T / LANES;   // R: rows of a thread in flight
  __shared__ float s[T / 16][2][COLS];
  static_assert(LANES == 2 || LANES == 4, "the moves between lanes");
  const int t = threadIdx.x, c = block * COLS + (t % LANES) * 8, n = p.dim - c;
  const bool back = p.dim >= 8;
  float dw[8], db[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dw[e] = db[e] = 0.f;
  for (int row = t / LANES; row < p.rows; row += R * STEP) {
    u32x4 d[R], h[R];
    float mean[R], rstd[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {   // past the last row: that one again, not counted
      const int64_t r = row + i * STEP < p.rows ? row + i * STEP : p.rows - 1;
      d[i] = raw8_load(p.dy + r * p.dy_row + c, n, back);
      h[i] = raw8_load(p.h + r * p.h_row + c, n, back);
      mean[i] = p.mean[r];
      rstd[i] = p.rstd[r];
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (row + i * STEP >= p.rows) break;
      float g[8], x[8];
      unpack8(g, raw8_shift(d[i], n, back), TY);
      unpack8(x, raw8_shift(h[i], n, back), TY);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[e] += g[e] * ((x[e] - mean[i]) * rstd[i]);
        db[e] += g[e];
      }
    }
  }
  // lanes LANES apart hold the same columns: over each 16 lanes, then over these in order
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float& v = k ? db[e] : dw[e];
      v += lane_move<0x128>(v);                             // 16 lanes rotated by 8
      v += lane_move<0x124>(v);                             // by 4
      if constexpr (LANES == 2) v += lane_move<0x4E>(v);    // quads: 2 3 0 1
      if ((t & 15) < LANES) s[t >> 4][k][(t & 15) * 8 + e] = v;
    }
  }
  __syncthreads();
  if (t < 2 * COLS) {   // the columns of dweight, then of dbias
    const int j = t % COLS, col = block * COLS + j;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < T / 16; ++w) v += s[w][t / COLS][j];
    uint16_t* const out = t < COLS ? p.dweight : p.dbias;
    if (out != nullptr && col < p.dim) out[col] = to_16(v, TY);
  }
}
// Columns of a workgroup: 32 of them fill a cache line's half, 16 leave fewer rows to a thread; rows of
// up to 1024 columns have the workgroups to spare for that.
constexpr int small_columns(int row_columns) { return row_columns <= 1024 ? 16 : 32; }
// A small backward pass in one launch: `columns` workgroups for some columns each of the weight's and
// the bias' gradients, which read dy and h a second time, from a cache, and the others for dx.
template <int TY, int NW, int C, int RW>
__global__ void __launch_bounds__(64 * NW * RW) layer_norm_bwd_small(NormBwdArgs p, int columns) {
  if ((int)blockIdx.x < columns) {
    norm_columns<TY, 64 * NW * RW, small_columns(512 * NW * C)>(p, blockIdx.x);
    return;
  }
  norm_bwd_rows<TY, true, NW, C, RW, false>(p, blockIdx.x - columns, gridDim.x - columns);
}

// Rows too long for registers: read twice, the dweight and dbias sums kept in the workgroup's
// part of the workspace, read and written again for every row, which is most of its time: 4096 x 32768
// bf16 1135 us, the RMS norm 736 (16384 columns, in registers, 139 and 120).
template <int TY, bool LN, int NW>
__global__ void __launch_bounds__(64 * NW) norm_bwd_long(NormBwdArgs p) {
  const bool back = p.dim >= 8;
  __shared__ float ssum[2][2 * NW];
  constexpr int STEP = 512 * NW;
  const int c0 = threadIdx.x * 8;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const float rstd = p.rstd[row], mean = LN ? p.mean[row] : 0.f;
    auto load = [&](int col, float (&g)[8], float (&x)[8], float (&d)[8])
                    __attribute__((always_inline)) {
      const int n = p.dim - col;
      float w[8];
      load8(d, p.dy + row * p.dy_row + col, n, TY, back);
      load8(x, p.h + row * p.h_row + col, n, TY, back);
      load8(w, p.weight + col, n, TY, back);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = LN ? (x[e] - mean) * rstd : x[e] * rstd;
        g[e] = d[e] * w[e];
      }
    };
    float g[8], x[8], d[8];
    float2v sum = {0.f, 0.f};
    for (uint32_t col = c0; col < (uint32_t)p.dim; col += STEP) {
      load(col, g, x, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] += g[e] * x[e];
        if constexpr (LN) sum[1] += g[e];
      }
    }
    if constexpr (LN)
      sum = group_sum2<NW>(sum, ssum[turn]);
    else
      sum[0] = group_sum<NW>(sum[0], ssum[turn]);
    const float along = sum[0] * p.inv_dim, level = sum[1] * p.inv_dim;
    for (uint32_t col = c0; col < (uint32_t)p.dim; col += STEP) {
      float v[8];
      load(col, g, x, d);
      if (p.dh)
        load8(v, p.dh + row * p.dh_row + col, p.dim - col, TY, back);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] += rstd * (LN ? g[e] - level - x[e] * along : g[e] - x[e] * along);
      if (p.part) {
        float* const o = partial(p.part, gridDim.x, blockIdx.x, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (row == blockIdx.x ? 0.f : o[e]) + d[e] * x[e];
      }
      if (LN && p.part_bias) {
        float* const o = partial(p.part_bias, gridDim.x, blockIdx.x, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (row == blockIdx.x ? 0.f : o[e]) + d[e];
      }
      store8(p.dx + row * p.dx_row + col, v, p.dim - col, TY);
    }
  }
}

// out[j] = the sum of n partial sums; one block of 32 columns a workgroup, from block `first` on.
// Blocks past out's `blocks` are those of `more`, whose partial sums follow.
template <int TY>
__global__ void __launch_bounds__(256) sum_partials(const float* part, int n, int first, int cols,
                                                    int blocks, uint16_t* out, uint16_t* more) {
  __shared__ SumLds s;
  const int b = first + blockIdx.x;
  if (b < blocks)
    sum_block<TY>(part, n, b, cols, out, s);
  else
    sum_block<TY>(part + (int64_t)blocks * n * 32, n, b - blocks, cols, more, s);
}

struct DactArgs {
  const uint16_t* dc;
  const uint16_t* pre;   // null (and pre8 too): dpre is dc
  const uint8_t* pre8;   // pre in 8 bits, in its place
  const uint8_t* pre8_scale;
  uint16_t* dpre;        // null: not stored (without pre)
  float* part;           // partial column sums of every row block, or null
  uint16_t* sum;         // the column sums themselves (one row block), or null
  int64_t dc_row, pre_row, dpre_row, pre8_row, ps_row;
  int32_t m, n, act;
  int32_t row_blocks, rows_per_block;   // at most 2^30
};

// dpre = dc act'(pre) and its column sums over a block of rows: 512 columns a workgroup, 4 rows
// at a time.  HBM bounds it: 4096 x 4096 bf16 with gelu_tanh 27 us (3.7 TB/s), 24.5 where dc and pre
// are partly in the last-level cache.
//
// dpre is rounded to the operands' type, once: the matrix instructions take both operands in one
// 16-bit type.  In fp32 it would have to go through the products as two 16-bit halves, which
// doubles their work (at 4096^3 from 216 us to 432) to take a gradient's error, relative in the
// norm, from 0.0023 to the 0.0017 of its own rounding in bf16 (f16: from 0.00029 to 0.00021).  The
// column sums take the unrounded values.
// WHOLE: the workgroup's 512 columns all exist, and nothing is spent on a row's end.  R: rows of a
// thread whose loads are in flight at once.
constexpr int kPre16 = 1, kPre8 = 2;
template <int TY, int PRE, bool WHOLE, int R>
__device__ __forceinline__ void dact_rows(const DactArgs& p, int64_t r0, int rows, int g, int col,
                                          float (&sum)[8]) {
  const int n = WHOLE ? 8 : p.n - col;
  const bool back = WHOLE || p.n >= 8;
  const uint16_t* const dc = p.dc + r0 * p.dc_row + col;
  const uint16_t* const pre = p.pre + r0 * p.pre_row + col;
  const uint8_t* const pre8 = p.pre8 + r0 * p.pre8_row + col;
  const uint8_t* const ps = p.pre8_scale + r0 * p.ps_row + (col >> 5);
  uint16_t* const dpre = p.dpre + r0 * p.dpre_row + col;
  for (int row = g; row < rows; row += 4 * R) {
    u32x4 d[R], u[PRE == kPre16 ? R : 1];
    uint2 q[PRE == kPre8 ? R : 1];
    uint32_t b[PRE == kPre8 ? R : 1];
#pragma unroll
    for (int i = 0; i < R; ++i) {   // past the last row: that one again, not counted
      const int64_t r = row + 4 * i < rows ? row + 4 * i : rows - 1;
      d[i] = raw8_load(dc + r * p.dc_row, n, back);
      if constexpr (PRE == kPre16) u[i] = raw8_load(pre + r * p.pre_row, n, back);
      if constexpr (PRE == kPre8) {
        q[i] = load_bytes8(pre8 + r * p.pre8_row, n, back);
        b[i] = ps[r * p.ps_row];
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = row + 4 * i;
      if (r >= rows) break;
      float v[8];
      unpack8(v, raw8_shift(d[i], n, back), TY);
      if (PRE == 0 && p.dpre != nullptr) store8(dpre + r * p.dpre_row, v, n, TY);
      if constexpr (PRE != 0) {
        float x[8];
        if constexpr (PRE == kPre8)
          unpack_block8(x, q[i].x, q[i].y, b[i]);
        else
          unpack8(x, raw8_shift(u[i], n, back), TY);
        slope8(v, x, p.act);
        if constexpr (PRE == kPre8) {
          // a lost block's slopes are not known: relu's of NaN is 0
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = b[i] == 255u ? __builtin_nanf("") : v[e];
        }
        store8(dpre + r * p.dpre_row, v, n, TY);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
  }
}
// The sums of a workgroup's four waves joined and stored.
template <int TY>
__device__ __forceinline__ void dact_sums(const DactArgs& p, int rb, int t, int g, int col,
                                          float (&sum)[8], float (&s)[3][512]) {
  if (p.part == nullptr && p.sum == nullptr) return;
  const int n = p.n - col;
  if (g > 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s[g - 1][t * 8 + e] = sum[e];
  }
  __syncthreads();
  if (g == 0 && n > 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += s[i][t * 8 + e];
    if (p.sum != nullptr)
      store8(p.sum + col, sum, n, TY);
    else
      store_partial8(p.part, p.row_blocks, rb, col, sum);
  }
}
// Without checkpoints, nor a copy of dc: a kernel of its own, not longer for them.  In us, so / as the
// other's 16-bit rows: 8192 x 8192 bf16 with relu 82 / 90, 4095 x 4097 with silu 26 / 31, 2704 x 3654
// with relu 16.4 / 17.7, 4544 x 6 5.9 / 8.5, 256 x 256 2.9 / 3.1.
template <int TY>
__global__ void __launch_bounds__(256) lin_dact(DactArgs p) {
  __shared__ float s[3][512];
  const int cb = blockIdx.x / p.row_blocks, rb = blockIdx.x - cb * p.row_blocks;
  const int t = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int col = cb * 512 + t * 8, n = p.n - col;
  // rows counted from the block's first: numbers past the last row need not fit 31 bits
  const int64_t r0 = (int64_t)rb * p.rows_per_block;
  const int rows = p.m - r0 < p.rows_per_block ? (int)(p.m - r0) : p.rows_per_block;
  const uint16_t* const dc = p.dc + r0 * p.dc_row + col;
  const uint16_t* const pre = p.pre + r0 * p.pre_row + col;
  uint16_t* const dpre = p.dpre + r0 * p.dpre_row + col;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  if (n > 0) {
#pragma unroll 4
    for (int row = g; row < rows; row += 4) {
      float v[8];
      load8(v, dc + row * p.dc_row, n, TY, p.n >= 8);
      if (p.pre) {
        float u[8];
        load8(u, pre + row * p.pre_row, n, TY, p.n >= 8);
        slope8(v, u, p.act);
        store8(dpre + row * p.dpre_row, v, n, TY);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
  }
  dact_sums<TY>(p, rb, t, g, col, sum, s);
}
// With checkpoints or a copy.
template <int TY>
__device__ __forceinline__ void dact_block(const DactArgs& p, int block, float (&s)[3][512]) {
  const int cb = block / p.row_blocks, rb = block - cb * p.row_blocks;
  const int t = threadIdx.x & 63, g = threadIdx.x >> 6;
  const int col = cb * 512 + t * 8, n = p.n - col;
  // rows counted from the block's first: numbers past the last row need not fit 31 bits
  const int64_t r0 = (int64_t)rb * p.rows_per_block;
  const int rows = p.m - r0 < p.rows_per_block ? (int)(p.m - r0) : p.rows_per_block;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  auto work = [&](auto whole, auto r) __attribute__((always_inline)) {
    constexpr bool WHOLE = decltype(whole)::value;
    constexpr int R = decltype(r)::value;
    if (p.pre8)
      dact_rows<TY, kPre8, WHOLE, R>(p, r0, rows, g, col, sum);
    else if (p.pre)
      dact_rows<TY, kPre16, WHOLE, R>(p, r0, rows, g, col, sum);
    else
      dact_rows<TY, 0, WHOLE, R>(p, r0, rows, g, col, sum);
  };
  if (p.rows_per_block == 4) {   // a row a thread
    if (n > 0) work(std::false_type{}, std::integral_constant<int, 1>{});
  } else if (p.n - cb * 512 >= 512) {
    work(std::true_type{}, std::integral_constant<int, 4>{});
  } else if (n > 0) {
    work(std::false_type{}, std::integral_constant<int, 4>{});
  }
  dact_sums<TY>(p, rb, t, g, col, sum, s);
}

// ---- checkpoints in 8 bits (see pack_block8) -----------------------------------------------
// A wave takes 8 << `lanes` columns of 64 >> lanes rows at once, 8 columns a lane; segs such pieces
// cover a row: one wave's columns are contiguous, and a row of 4097 columns wastes part of a wave, not
// of a workgroup.  kPackRows pieces of rows a wave one below the other, all of their loads in flight.
// HBM bounds both.  bf16, from memory and to memory / on the same matrices, partly in the last-level
// cache: pack8 8192 x 8190 43 us (4.7 TB/s) / 35, unpack8 8192 x 8192 38 us (5.3 TB/s) / 34, through
// gelu_tanh 46 / 38 (47 where every lane provides for a row's end), 8192 x 8190 50, through gelu_tanh 56.
struct PackArgs {
  const uint16_t* x;      // packing; null: unpacking
  uint16_t* y;            // unpacking: act(values), in 16 bits
  uint8_t* q;
  uint8_t* scale;
  int64_t x_row, y_row, q_row, s_row;
  int32_t rows, dim, lanes, segs, act;
};
constexpr int kPackRows = 4;
struct PackPlace {
  int64_t row, col;   // of the lane's first piece; the others are 64 >> lanes rows apart
  int n;              // columns that exist from col on
  bool whole;         // all columns of the workgroup's piece of a row exist
};
__device__ __forceinline__ PackPlace pack_place(const PackArgs& p, uint32_t workgroup) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint32_t seg = workgroup % (uint32_t)p.segs, block = workgroup / (uint32_t)p.segs;
  const int per = 64 >> p.lanes;
  PackPlace t;
  t.row = ((int64_t)block * 4 + w) * (per * kPackRows) + (lane >> p.lanes);
  t.col = (int64_t)seg * (8 << p.lanes) + (lane & ((1 << p.lanes) - 1)) * 8;
  t.n = (int)(p.dim - t.col);
  t.whole = p.dim - (int64_t)seg * (8 << p.lanes) >= (8 << p.lanes);
  return t;
}
template <int TY, bool WHOLE>
__device__ __forceinline__ void pack8_piece(const PackArgs& p, const PackPlace& t) {
  const int per = 64 >> p.lanes, n = WHOLE ? 8 : t.n;
  const bool back = WHOLE || p.dim >= 8;
  u32x4 v[kPackRows];
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {   // rows past the last: that one again, not stored
    const int64_t r = t.row + i * per < p.rows ? t.row + i * per : p.rows - 1;
    v[i] = raw8_load(p.x + r * p.x_row + t.col, n, back);
  }
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {
    float x[8];
    unpack8(x, raw8_shift(v[i], n, back), TY);
    const Block8 b = pack_block8(x, TY);   // quads are whole: every lane is here
    const int64_t r = t.row + i * per;
    if (r >= p.rows || n <= 0) continue;
    store_bytes8(p.q + r * p.q_row + t.col, b.lo, b.hi, n);
    if ((t.col & 31) == 0) p.scale[r * p.s_row + (t.col >> 5)] = (uint8_t)b.scale;
  }
}
template <int TY>
__global__ void __launch_bounds__(256) pack8(PackArgs p) {
  const PackPlace t = pack_place(p, blockIdx.x);
  if (t.whole)
    pack8_piece<TY, true>(p, t);
  else
    pack8_piece<TY, false>(p, t);
}
template <int TY, bool WHOLE>
__device__ __forceinline__ void unpack8_piece(const PackArgs& p, const PackPlace& t) {
  const int per = 64 >> p.lanes, n = WHOLE ? 8 : t.n;
  const bool back = WHOLE || p.dim >= 8;
  uint2 q[kPackRows];
  uint32_t b[kPackRows];
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {
    const int64_t r = t.row + i * per < p.rows ? t.row + i * per : p.rows - 1;
    q[i] = load_bytes8(p.q + r * p.q_row + t.col, n, back);
    b[i] = p.scale[r * p.s_row + (t.col >> 5)];
  }
#pragma unroll
  for (int i = 0; i < kPackRows; ++i) {
    const int64_t r = t.row + i * per;
    if (r >= p.rows) continue;
    float v[8];
    unpack_block8(v, q[i].x, q[i].y, b[i]);
    act_n(v, p.act);
    store8(p.y + r * p.y_row + t.col, v, n, TY);
  }
}
template <int TY>
__device__ __forceinline__ void unpack8_block(const PackArgs& p, uint32_t workgroup) {
  const PackPlace t = pack_place(p, workgroup);
  if (t.whole)
    unpack8_piece<TY, true>(p, t);
  else if (t.n > 0)
    unpack8_piece<TY, false>(p, t);
}
template <int TY>
__global__ void __launch_bounds__(256) unpack8_rows(PackArgs p) {
  unpack8_block<TY>(p, blockIdx.x);
}

// What stands before the products of a backward pass, in one launch: dpre and the column sums in the
// first dact_blocks workgroups, a restored from 8 bits in the others.  HBM bounds it: 4096^3 bf16 with
// both in 8 bits 29 - 33 us (134 MB, 4.4 TB/s); as two launches 26 + 11.
template <int TY>
__global__ void __launch_bounds__(256) lin_prepare(DactArgs d, PackArgs u, int dact_blocks) {
  __shared__ float s[3][512];
  if ((int)blockIdx.x < dact_blocks)
    dact_block<TY>(d, blockIdx.x, s);
  else
    unpack8_block<TY>(u, blockIdx.x - dact_blocks);
}

}  // namespace nk
