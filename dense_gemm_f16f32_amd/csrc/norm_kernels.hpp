// Device code of the root-mean-square norm, its backward pass, and the element-wise part of the
// linear layer's backward pass.  All of them move each element once; HBM bounds them.
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
template <int NW>
__device__ __forceinline__ uint32_t group_max(uint32_t v, uint32_t* s) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d);
    v = v > o ? v : o;
  }
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
  void* y;
  float* scale;
  uint16_t* h;
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
struct __attribute__((packed)) Bytes8 {
  uint32_t x, y;
};
__device__ __forceinline__ void store_e4m3x8(uint8_t* p, const float (&v)[8], Divisor d, int n) {
  const uint2 q = to_e4m3x8(v, d);
  if (n >= 8) {
    *(Bytes8*)p = Bytes8{q.x, q.y};
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = (uint8_t)((e < 4 ? q.x : q.y) >> (8 * (e & 3)));
  }
}

// One pass: the sum of squares, the 8-bit scale and y come from the row in registers.  HBM bounds
// it: 8192 x 8192 bf16 with residual to e4m3 88 us (5.3 TB/s), 4095 x 4093 f16 29 us (4.6 TB/s; 24.5
// where the rows are partly in the last-level cache).
// One row a workgroup of 64 NW threads, 8 columns a thread at a time.  C > 0: rows of at most
// 512 NW C columns, held in registers.  C == 0: longer rows, read again for each step that
// needs them.
template <int TY, bool Q8, int NW, int C>
__global__ void __launch_bounds__(64 * NW) rms_norm_fwd(NormArgs p) {
  const bool back = p.dim >= 8;
  __shared__ float ssum[NW];
  __shared__ uint32_t smax[NW];
  constexpr int STEP = 512 * NW, CR = C > 0 ? C : 1;
  const int64_t row = blockIdx.x;
  const uint16_t* const x = p.x + row * p.x_row;
  const uint16_t* const res = p.res ? p.res + row * p.res_row : nullptr;
  uint16_t* const h = p.h ? p.h + row * p.h_row : nullptr;
  const int c0 = threadIdx.x * 8;
  const int steps = C > 0 ? C : (p.dim - 1) / STEP + 1;   // dim > 0; dim + STEP need not fit
  float hv[CR][8], wv[CR][8];
  auto load_h = [&](int col, float (&v)[8]) __attribute__((always_inline)) {
    load8(v, x + col, p.dim - col, TY, back);
    if (res) {
      float r[8];
      load8(r, res + col, p.dim - col, TY, back);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += r[e];
    }
  };
  float sum = 0.f;
  if constexpr (C > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) load_h(c0 + i * STEP, hv[i]);
#pragma unroll
    for (int i = 0; i < C; ++i) load8(wv[i], p.weight + c0 + i * STEP, p.dim - c0 - i * STEP, TY, back);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = c0 + i * STEP;
      if (h && col < p.dim) store8(h + col, hv[i], p.dim - col, TY);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += hv[i][e] * hv[i][e];
    }
  } else {
    for (int i = 0; i < steps; ++i) {
      load_h(c0 + i * STEP, hv[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += hv[0][e] * hv[0][e];
    }
  }
  float square = group_sum<NW>(sum, ssum) * p.inv_dim + p.eps, unit = 1.f;
  // Squares outside fp32's range (bf16 rows above 1e19, or below 1e-9 with a tiny eps) are summed
  // again in units that bring them into it; every thread of the row holds the same sum.
  if (square < 0x1p-60f || square == __builtin_inff()) {
    unit = square < 1.f ? 0x1p64f : 0x1p-96f;
    if constexpr (NW > 1) __syncthreads();   // the first sum has been read
    sum = 0.f;
#pragma unroll CR
    for (int i = 0; i < steps; ++i) {
      if constexpr (C == 0) load_h(c0 + i * STEP, hv[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float v = hv[C > 0 ? i : 0][e] * unit;
        sum += v * v;
      }
    }
    square = group_sum<NW>(sum, ssum) * p.inv_dim + p.eps * unit * unit;
  }
  const float rstd = unit / sqrtf(square);
  if (p.rstd && threadIdx.x == 0) p.rstd[row] = rstd;
  // y of step i
  auto norm = [&](int i, float (&v)[8]) __attribute__((always_inline)) {
    const int col = c0 + i * STEP;
    float w[8];
    if constexpr (C == 0) {
      load_h(col, v);
      load8(w, p.weight + col, p.dim - col, TY, back);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (C > 0)
        v[e] = hv[i][e] * rstd * wv[i][e];
      else
        v[e] = v[e] * rstd * w[e];
    }
  };
  Divisor by = {1.f, 1.f};
  if constexpr (Q8) {
    uint32_t m = 0u;
#pragma unroll CR
    for (int i = 0; i < steps; ++i) {
      float v[8];
      norm(i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t b = abs_bits(v[e]);   // columns past dim are 0 (their weight reads as 0)
        m = m > b ? m : b;
      }
    }
    const float scale = e4m3_scale(group_max<NW>(m, smax));
    if (threadIdx.x == 0) p.scale[row] = scale;
    by = divisor(scale);
  }
#pragma unroll CR
  for (int i = 0; i < steps; ++i) {
    const int col = c0 + i * STEP;
    if (col >= p.dim) break;
    float v[8];
    norm(i, v);
    if constexpr (Q8)
      store_e4m3x8((uint8_t*)p.y + row * p.y_row + col, v, by, p.dim - col);
    else
      store8((uint16_t*)p.y + row * p.y_row + col, v, p.dim - col, TY);
    // h may be x's or the residual's memory: without registers it is written last
    if constexpr (C == 0) {
      if (h) {
        load_h(col, v);
        store8(h + col, v, p.dim - col, TY);
      }
    }
  }
}

struct NormBwdArgs {
  const uint16_t* dy;
  const uint16_t* h;
  const uint16_t* weight;
  const float* rstd;
  const uint16_t* dh;
  uint16_t* dx;
  uint16_t* dweight;
  float* part;   // partial dweight sums of every workgroup; null: dweight itself, or nothing
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
// workgroup adds and writes them once.  Short rows (one wave each) go four to a workgroup.  HBM
// bounds it: 8192 x 4096 bf16 50 us (5.4 TB/s of dy, h, dh and dx), and 5 for sum_partials; with the
// rows partly in the last-level cache 41 us, and there without the loads ahead 70.
template <int TY, int NW, int C, int RW>
__global__ void __launch_bounds__(64 * NW * RW) rms_norm_bwd(NormBwdArgs p) {
  static_assert(NW == 1 || RW == 1, "rows of several waves share the workgroup's barrier");
  const bool back = p.dim >= 8;
  __shared__ float ssum[2][NW];
  constexpr int STEP = 512 * NW;
  const int c0 = (RW > 1 ? threadIdx.x & 63 : threadIdx.x) * 8;
  const int rw = RW > 1 ? threadIdx.x >> 6 : 0;
  float wv[C][8], dw[C][8];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    load8(wv[i], p.weight + c0 + i * STEP, p.dim - c0 - i * STEP, TY, back);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  struct Row {
    u32x4 d[C], h[C], r[C];   // dy, h, dh
    float4v s;                // rstd first; a lone float's padding would be copied through memory
  };
  auto load = [&](Row& q, int64_t row) __attribute__((always_inline)) {
    q.s[0] = p.rstd[row];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = c0 + i * STEP, n = p.dim - col;
      q.d[i] = raw8_load(p.dy + row * p.dy_row + col, n, back);
      q.h[i] = raw8_load(p.h + row * p.h_row + col, n, back);
      q.r[i] = p.dh ? raw8_load(p.dh + row * p.dh_row + col, n, back) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  constexpr bool kAhead = C <= 2;
  const int64_t first = (int64_t)blockIdx.x * RW + rw, step = (int64_t)gridDim.x * RW;
  Row cur, nxt;
  if (kAhead && first < p.rows) load(cur, first);
  int turn = 0;
  for (int64_t row = first; row < p.rows; row += step, turn ^= 1) {
    if (!kAhead) load(cur, row);
    nxt = cur;
    if (kAhead && row + step < p.rows) load(nxt, row + step);
    const float rstd = cur.s[0];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float d[8], x[8];
      const int n = p.dim - c0 - i * STEP;
      cur.d[i] = raw8_shift(cur.d[i], n, back);
      cur.h[i] = raw8_shift(cur.h[i], n, back);
      cur.r[i] = raw8_shift(cur.r[i], n, back);
      unpack8(d, cur.d[i], TY);
      unpack8(x, cur.h[i], TY);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= rstd;
        dw[i][e] += d[e] * x[e];
        sum += d[e] * wv[i][e] * x[e];
      }
    }
    // two sets of sums in turn, so that one barrier a row is enough
    const float mean = group_sum<NW>(sum, ssum[turn]) * p.inv_dim;
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int col = c0 + i * STEP;
      float d[8], x[8], r[8];
      unpack8(d, cur.d[i], TY);
      unpack8(x, cur.h[i], TY);
      unpack8(r, cur.r[i], TY);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        r[e] += rstd * (d[e] * wv[i][e] - x[e] * rstd * mean);
      if (col < p.dim) store8(p.dx + row * p.dx_row + col, r, p.dim - col, TY);
    }
    cur = nxt;
  }
  if (p.part == nullptr && p.dweight == nullptr) return;
  if constexpr (RW > 1) {   // the other rows' sums, in their order
    __shared__ float sdw[RW - 1][C * 512];
    if (rw > 0) {
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sdw[rw - 1][(i * 8 + e) * 64 + (threadIdx.x & 63)] = dw[i][e];
    }
    __syncthreads();
    if (rw > 0) return;
#pragma unroll
    for (int r = 0; r < RW - 1; ++r)
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] += sdw[r][(i * 8 + e) * 64 + threadIdx.x];
  }
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const int col = c0 + i * STEP;
    if (col >= p.dim) continue;
    if (p.part != nullptr)
      store_partial8(p.part, gridDim.x, blockIdx.x, col, dw[i]);
    else   // the only workgroup
      store8(p.dweight + col, dw[i], p.dim - col, TY);
  }
}

// Rows too long for registers: read twice, the dweight sums kept in the workgroup's
// part of the workspace.
template <int TY, int NW>
__global__ void __launch_bounds__(64 * NW) rms_norm_bwd_long(NormBwdArgs p) {
  const bool back = p.dim >= 8;
  __shared__ float ssum[2][NW];
  constexpr int STEP = 512 * NW;
  const int c0 = threadIdx.x * 8;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x, turn ^= 1) {
    const float rstd = p.rstd[row];
    auto load = [&](int col, float (&g)[8], float (&x)[8], float (&d)[8])
                    __attribute__((always_inline)) {
      const int n = p.dim - col;
      float w[8];
      load8(d, p.dy + row * p.dy_row + col, n, TY, back);
      load8(x, p.h + row * p.h_row + col, n, TY, back);
      load8(w, p.weight + col, n, TY, back);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= rstd;
        g[e] = d[e] * w[e];
      }
    };
    float g[8], x[8], d[8], sum = 0.f;
    for (uint32_t col = c0; col < (uint32_t)p.dim; col += STEP) {
      load(col, g, x, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum += g[e] * x[e];
    }
    const float mean = group_sum<NW>(sum, ssum[turn]) * p.inv_dim;
    for (uint32_t col = c0; col < (uint32_t)p.dim; col += STEP) {
      float v[8];
      load(col, g, x, d);
      if (p.dh)
        load8(v, p.dh + row * p.dh_row + col, p.dim - col, TY, back);
      else
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += rstd * (g[e] - x[e] * mean);
      if (p.part) {
        float* const o = partial(p.part, gridDim.x, blockIdx.x, col);
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (row == blockIdx.x ? 0.f : o[e]) + d[e] * x[e];
      }
      store8(p.dx + row * p.dx_row + col, v, p.dim - col, TY);
    }
  }
}

// out[j] = the sum of n partial sums; one block of 32 columns a workgroup, from block `first` on.
template <int TY>
__global__ void __launch_bounds__(256) sum_partials(const float* part, int n, int first, int cols,
                                                    uint16_t* out) {
  sum_block<TY>(part, n, first + blockIdx.x, cols, out);
}

struct DactArgs {
  const uint16_t* dc;
  const uint16_t* pre;   // null: dpre is dc
  uint16_t* dpre;
  float* part;           // partial column sums of every row block, or null
  uint16_t* sum;         // the column sums themselves (one row block), or null
  int64_t dc_row, pre_row, dpre_row;
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
  if (p.part == nullptr && p.sum == nullptr) return;
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

}  // namespace nk
