// Device code of the linear layer on gfx950: tiled matrix products on 16-bit, e4m3 or int8 operands
// with the layer's epilogue, out = act(a b scale + bias) + residual.
//
// The operand side (panels in LDS, swizzles, buffer->LDS loads, transposing reads, the program
// map) is the fp16 product's, from gemm_kernels.hpp; it moves 16-byte chunks and does not look
// inside them.  What differs here:
//  * the element type: fp16, bf16, e4m3 or int8.  Two 8-bit values ride in each 16-bit slot, so an
//    8-bit operand of K values is a k-major matrix of K/2 slots, and one 64-byte piece of an e4m3
//    row feeds v_mfma_f32_32x32x64_f8f6f4, twice the work of the 16-bit instruction on the same
//    bytes (the unscaled form: scales are applied to the sum, in the epilogue).  Its inner sums
//    are rounded to fewer bits than fp32 (see kHalvesK).  The int8 instructions
//    (v_mfma_i32_16x16x64_i8, 32x32x32) take and leave their registers as the 16-bit ones do; the
//    accumulators hold 32-bit integers, exact up to K = 131071 (2^31 / 128^2), which travel as the
//    bits of floats to the epilogue and are converted there.
//  * the ragged panel: when the panel depth does not divide K, the panel that holds the last
//    K mod BK values is multiplied first, so that every other panel starts at a multiple of BK
//    and keeps the alignment of its rows.
//  * the epilogue: a wave's block of sums goes through LDS to a layout in which a lane holds 8
//    consecutive columns of one row, so that bias, residual, pre-activation and result move in
//    16-byte accesses.
#pragma once

#include "gemm_kernels.hpp"
#include "linear_norm.h"

namespace lk {

using gk::dma_panel;
using gk::elem_off;
using gk::extent;
using gk::float16v;
using gk::float4v;
using gk::half8;
using gk::lds_barrier;
using gk::u32x4;
using gk::wait_vmcnt;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float2v __attribute__((ext_vector_type(2)));
typedef int int8v __attribute__((ext_vector_type(8)));
typedef int int16v __attribute__((ext_vector_type(16)));
typedef int int4v __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));   // 16 bytes at any 16-bit element

constexpr int kF16 = LINEAR_NORM_F16, kBF16 = LINEAR_NORM_BF16, kE4M3 = LINEAR_NORM_E4M3;
constexpr int kI8 = LINEAR_NORM_I8;
template <int TY>
constexpr bool kBytes = TY == kE4M3 || TY == kI8;   // 8-bit operands

struct LinArgs {
  const uint16_t* A;      // 16-bit slots: elements, or pairs of 8-bit values
  const uint16_t* B;
  int64_t lda, ldb;       // slots
  int32_t M, N, K;        // K in elements
  int32_t num_pid_m, num_pid_n, group_m, num_programs, xcd_remap;
  // epilogue; the pointers may be null, except out
  uint16_t* out;
  uint16_t* pre;
  const uint16_t* res;
  const uint16_t* bias;
  const float* scale_a;
  const float* scale_b;
  int64_t ldo, ldp, ldr;
  int32_t act, out_type;
  // the value before the activation in 8 bits (see pack_block8), or null; not with `pre`
  uint8_t* pre8;
  uint8_t* pre8_scale;
  int64_t ldp8, ldps;
  // Split K: the tiles from `first_split` on (all, some or none) are computed in `splits` slices
  // of k, `per_split` panels each, the last one the rest.  Slice z of the i-th of them leaves
  // its sums in W, a BM x BN block at (i splits + z) BM BN; lin_reduce adds the slices.
  float* W;
  int32_t first_split, splits, per_split;
  // Column sums that are to be had of partial sums (see sum_block), by the workgroups behind the
  // product's: a launch less.  Null: none.
  const float* sum_part;
  uint16_t* sum_out;
  int32_t sum_n, sum_cols, sum_first;   // sum_first: workgroups of the product
};

// A workgroup's tile and k slice: the whole tiles first, then the slices, all tiles of slice 0,
// all of slice 1 ...
struct Work {
  int tile, z;       // z < 0: the whole k range
  float* w;          // the slice's block of W
};
template <int BM, int BN>
__device__ __forceinline__ Work work_of(const LinArgs& p, int h) {
  if (h < p.first_split) return {h, -1, nullptr};
  const int r = p.num_programs - p.first_split, u = h - p.first_split;
  const int z = u / r, i = u - z * r;
  return {p.first_split + i, z, p.W + ((int64_t)i * p.splits + z) * (BM * BN)};
}

// ---- 16-bit values ---------------------------------------------------------------------
__device__ __forceinline__ float to_f32(uint16_t v, int type) {
  return type == kF16 ? (float)__builtin_bit_cast(_Float16, v)
                      : __builtin_bit_cast(float, (uint32_t)v << 16);
}
__device__ __forceinline__ uint16_t to_16(float v, int type) {   // nearest, ties to even
  return type == kF16 ? __builtin_bit_cast(uint16_t, (_Float16)v)
                      : __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ void unpack8(float (&f)[8], u32x4 v, int type) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = to_f32((uint16_t)(v[e / 2] >> (16 * (e & 1))), type);
}
__device__ __forceinline__ u32x4 pack8(const float (&f)[8], int type) {
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const float2v x = {f[2 * d], f[2 * d + 1]};
    v[d] = type == kF16 ? __builtin_bit_cast(uint32_t, __builtin_convertvector(x, half2v))
                        : __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
  }
  return v;
}
// 8 16-bit values at p, of which the first n exist (n >= 8: all, n <= 0: none); the others are 0
// and not read.  p is n values before its row's end.  `back`: the row has 8 values at least;
// then a lane at its end reads the row's last 8 and shifts, one load like every other lane's
// (value by value, the lanes at a row's end cost a norm of 4092 columns half as much again).
// In two steps, so that a load can be in flight before its lane's shift has to wait for it.
__device__ __forceinline__ u32x4 raw8_load(const uint16_t* p, int n, bool back) {
  if (back) return *(const u32x4_any*)(p - (n >= 8 ? 0 : 8 - n));
  u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) v[e / 2] |= (uint32_t)p[e] << (16 * (e & 1));
  return v;
}
// The 128 bits of v moved down by `bits` > 0 (128 and more: 0).
__device__ __forceinline__ u32x4 shift_down(u32x4 v, int bits) {
  const uint64_t lo = (uint64_t)v[0] | ((uint64_t)v[1] << 32);
  const uint64_t hi = (uint64_t)v[2] | ((uint64_t)v[3] << 32);
  const uint64_t l = bits >= 128  ? 0
                     : bits >= 64 ? hi >> (bits - 64)
                                  : (lo >> bits) | (hi << (64 - bits));
  const uint64_t h = bits >= 64 ? 0 : hi >> bits;
  return u32x4{(uint32_t)l, (uint32_t)(l >> 32), (uint32_t)h, (uint32_t)(h >> 32)};
}
__device__ __forceinline__ u32x4 raw8_shift(u32x4 v, int n, bool back) {
  return n >= 8 || !back ? v : shift_down(v, 16 * (8 - n));
}
__device__ __forceinline__ u32x4 raw8(const uint16_t* p, int n, bool back) {
  return raw8_shift(raw8_load(p, n, back), n, back);
}
__device__ __forceinline__ void load8(float (&f)[8], const uint16_t* p, int n, int type,
                                      bool back) {
  unpack8(f, raw8(p, n, back), type);
}
struct __attribute__((packed, aligned(2))) Half4 {
  uint32_t x, y;
};
struct __attribute__((packed, aligned(2))) Half2 {
  uint32_t x;
};
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8], int n, int type) {
  u32x4 v = pack8(f, type);
  if (n >= 8) {
    *(u32x4_any*)p = v;
  } else {   // in pieces of 4, 2 and 1
    if (n & 4) {
      *(Half4*)p = Half4{v[0], v[1]};
      p += 4;
      v[0] = v[2];
      v[1] = v[3];
    }
    if (n & 2) {
      *(Half2*)p = Half2{v[0]};
      p += 2;
      v[0] = v[1];
    }
    if (n & 1) *p = (uint16_t)v[0];
  }
}

// ---- checkpoints in 8 bits ---------------------------------------------------------------
// 32 neighbouring values of a row share a scale, a power of two 2^(b - 127) held as the byte b: the
// largest magnitude lies in [64, 128) scales.  Values are integers, rounded to nearest (ties to
// even) and at most 127.  Not below 2^-24 (f16) or 2^-120 (bf16), a scale times an integer is a
// value of its 16-bit type, so what is restored enters the matrix instructions unrounded; with the
// largest magnitude divided by 127 instead (a step of up to half the size) it would be rounded
// again there.  A block that holds an infinity or a NaN has scale NaN (b = 255), and so do all its
// values.
__device__ __forceinline__ int lowest_scale(int type) { return type == kF16 ? 127 - 24 : 127 - 120; }

// Largest of the 4 lanes of a quad, all of which are active.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);   // 1 0 3 2
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);            // 2 3 0 1
  return v > o ? v : o;
}
struct Block8 {
  uint32_t lo, hi;   // 8 integers
  uint32_t scale;    // the block's byte
};
// 8 values of a block, whose others the quad's other lanes hold (0 where there are none).  `least`:
// what a positive value is stored as at least, where its sign has to stay (relu's slope goes by
// it), or -127.
__device__ __forceinline__ Block8 pack_block8(const float (&v)[8], int type, float least = -127.f) {
  uint32_t m = 0u;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v[e]) & 0x7FFFFFFFu;
    m = m > b ? m : b;
  }
  const int exponent = (int)(quad_max(m) >> 23), low = lowest_scale(type);
  const int b = exponent - 6 < low ? low : exponent - 6;
  const float inv = __builtin_bit_cast(float, (uint32_t)(254 - b) << 23);   // 2^(127 - b)
  uint32_t q[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)   // the addition rounds, and leaves the integer in the low bits
    q[e] = __builtin_bit_cast(
        uint32_t,
        __builtin_amdgcn_fmed3f(v[e] * inv, v[e] > 0.f ? least : -127.f, 127.f) + 12582912.f);
  auto bytes = [&](int i) __attribute__((always_inline)) {
    const uint32_t x = __builtin_amdgcn_perm(q[i + 1], q[i], 0x0C0C0400u);
    const uint32_t y = __builtin_amdgcn_perm(q[i + 3], q[i + 2], 0x0C0C0400u);
    return x | (y << 16);
  };
  if (exponent == 255) return {0u, 0u, 255u};
  return {bytes(0), bytes(4), (uint32_t)b};
}
// 8 values back, exact: bytes as (128 + q) - 128, times the scale.
__device__ __forceinline__ void unpack_block8(float (&v)[8], uint32_t lo, uint32_t hi,
                                              uint32_t b) {
  // byte 0 is 2^-127, below the normal numbers, and 255 NaN
  const float scale = b == 255u ? __builtin_nanf("")
                                : __builtin_bit_cast(float, b == 0u ? 0x400000u : b << 23);
  const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = ((float)((w[e / 4] >> (8 * (e & 3))) & 0xFFu) - 128.f) * scale;
}
struct __attribute__((packed)) Bytes8 {
  uint32_t x, y;
};
struct __attribute__((packed)) Bytes4 {
  uint32_t x;
};
struct __attribute__((packed)) Bytes2 {
  uint16_t x;
};
// 8 bytes to p, of which the first n > 0 exist, in pieces of 8, 4, 2 and 1.
__device__ __forceinline__ void store_bytes8(uint8_t* p, uint32_t lo, uint32_t hi, int n) {
  if (n >= 8) {
    *(Bytes8*)p = Bytes8{lo, hi};
    return;
  }
  if (n & 4) {
    *(Bytes4*)p = Bytes4{lo};
    p += 4;
    lo = hi;
  }
  if (n & 2) {
    *(Bytes2*)p = Bytes2{(uint16_t)lo};
    p += 2;
    lo >>= 16;
  }
  if (n & 1) *p = (uint8_t)lo;
}
// 8 bytes from p, of which the first n exist (n >= 8: all, n <= 0: none); the others are 0 and not
// read.  p is n bytes before its row's end; `back`: the row has 8 bytes at least (see raw8_load).
__device__ __forceinline__ uint2 load_bytes8(const uint8_t* p, int n, bool back) {
  uint2 v = {0u, 0u};
  if (back) {
    const Bytes8 q = *(const Bytes8*)(p - (n >= 8 ? 0 : 8 - n));
    uint64_t w = (uint64_t)q.x | ((uint64_t)q.y << 32);
    w = n >= 8 ? w : n <= 0 ? 0u : w >> (8 * (8 - n));
    v.x = (uint32_t)w;
    v.y = (uint32_t)(w >> 32);
    return v;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) (e < 4 ? v.x : v.y) |= (uint32_t)p[e] << (8 * (e & 3));
  return v;
}

// ---- activations -------------------------------------------------------------------------
// exp through the hardware's 2^x (1 ulp).  The argument x log2 e is rounded, which moves the
// result by up to |x| 2^-23 of itself: 2^-22 near 1, 2^-16.5 at |x| = 88, where the result leaves
// fp32's range.  Below 2^-126 it is 0.
__device__ __forceinline__ float fast_exp(float x) {
  return __builtin_amdgcn_exp2f(x * 1.44269504088896f);
}
__device__ __forceinline__ float sigmoid(float x) {   // exp(-x) = inf gives 1 / inf = 0
  return __builtin_amdgcn_rcpf(1.f + fast_exp(-x));
}
// The normal distribution's cumulative function Phi(v); `e` returns exp(-v^2 / 2).  The tail
// Phi(-x) exp(x^2 / 2), x >= 0, falls from 1/2 like 1 / (x sqrt(2 pi)); as t P(t), t = 1 / (1 +
// 0.3 x), a polynomial P of degree 7 holds it to 2^-21 of its value up to x = 14, where exp(-x^2 /
// 2) has left fp32's range (coefficients: least squares on the relative error, weighted until the
// largest errors are equal; evaluated in fp32).  An approximation bounded in absolute error, as
// formula 7.1.26 of Abramowitz and Stegun, is off by 1 % of the tail at v = -8 and 3 % at -12,
// several bf16 steps.
__device__ __forceinline__ float normal_cdf(float v, float& e) {
  e = fast_exp(-0.5f * v * v);
  const float t = __builtin_amdgcn_rcpf(1.f + 0.3f * fabsf(v));
  float q = 0.035674773f;
  q = q * t - 0.15720308f;
  q = q * t + 0.20635349f;
  q = q * t - 0.053683631f;
  q = q * t + 0.12856162f;
  q = q * t + 0.099913493f;
  q = q * t + 0.12075395f;
  q = q * t + 0.1196293f;
  const float tail = q * t * e;
  return v < 0.f ? tail : 1.f - tail;
}

constexpr float kTanhC = 0.79788456080286536f;   // sqrt(2 / pi)

// v * Phi(v) and v * sigmoid(v) with v = -inf are 0 * -inf; their limit is 0 but the formula
// gives NaN, here as in any evaluation of it.
__device__ __forceinline__ float act_value(float v, int act) {
  float e;
  switch (act) {
    case LINEAR_ACT_RELU: return v < 0.f ? 0.f : v;   // NaN stays
    case LINEAR_ACT_GELU: return v * normal_cdf(v, e);
    // tanh u = 2 sigmoid(2u) - 1
    case LINEAR_ACT_GELU_TANH: return v * sigmoid(2.f * kTanhC * (v + 0.044715f * v * v * v));
    case LINEAR_ACT_SILU: return v * sigmoid(v);
    default: return v;
  }
}
__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case LINEAR_ACT_RELU: return v > 0.f ? 1.f : 0.f;
    case LINEAR_ACT_GELU: {
      float e;
      const float c = normal_cdf(v, e);
      return c + v * e * 0.39894228040143268f;   // 1 / sqrt(2 pi)
    }
    case LINEAR_ACT_GELU_TANH: {
      // v p(2u): p + v p (1 - p) 2u'.  p (1 - p) is 0 long before v^2 overflows, and then the
      // slope is p: the product would be 0 times infinity from |v| = 1.8e19 on.
      const float p = sigmoid(2.f * kTanhC * (v + 0.044715f * v * v * v));
      const float d = p * (1.f - p);
      return d == 0.f ? p : p + v * d * (2.f * kTanhC) * (1.f + 0.134145f * v * v);
    }
    case LINEAR_ACT_SILU: {
      const float p = sigmoid(v);
      return p * (1.f + v * (1.f - p));
    }
    default: return 1.f;
  }
}

// The choice is made once for several values: made for each, its branches cost more than the values.
template <int N>
__device__ __forceinline__ void act_n(float (&v)[N], int act) {
#define LK_ACT(A)                                              \
  case A:                                                       \
    _Pragma("unroll") for (int e = 0; e < N; ++e) v[e] = act_value(v[e], A); \
    break;
  switch (act) {
    LK_ACT(LINEAR_ACT_RELU)
    LK_ACT(LINEAR_ACT_GELU)
    LK_ACT(LINEAR_ACT_GELU_TANH)
    LK_ACT(LINEAR_ACT_SILU)
    default: break;
  }
#undef LK_ACT
}
__device__ __forceinline__ void slope8(float (&v)[8], const float (&u)[8], int act) {
#define LK_SLOPE8(A)                                                 \
  case A:                                                            \
    _Pragma("unroll") for (int e = 0; e < 8; ++e) v[e] *= act_slope(u[e], A); \
    break;
  switch (act) {
    LK_SLOPE8(LINEAR_ACT_RELU)
    LK_SLOPE8(LINEAR_ACT_GELU)
    LK_SLOPE8(LINEAR_ACT_GELU_TANH)
    LK_SLOPE8(LINEAR_ACT_SILU)
    default: break;
  }
#undef LK_SLOPE8
}

// ---- epilogue ------------------------------------------------------------------------------
// 8 consecutive columns of one row: v holds the sums.  `bias8` and `sb8` are the columns' bias
// and scales (0 and 1 where there are none).
struct Columns {
  float bias[8], sb[8];
  int n;   // columns that exist, from the first
};
template <int TY>
__device__ __forceinline__ Columns load_columns(const LinArgs& p, int col) {
  const int ot = kBytes<TY> ? p.out_type : TY;
  Columns c;
  c.n = p.N - col;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    c.bias[e] = 0.f;
    c.sb[e] = 1.f;
  }
  if (c.n > 0) {
    if (p.bias) load8(c.bias, p.bias + col, c.n, ot, p.N >= 8);
    if (kBytes<TY> && p.scale_b) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < c.n) c.sb[e] = p.scale_b[col + e];
    }
  }
  return c;
}
// A sum as the matrix instructions leave it.
template <int TY>
__device__ __forceinline__ float sum_value(float v) {
  return TY == kI8 ? (float)__builtin_bit_cast(int, v) : v;
}
// Partial sums added.
template <int TY>
__device__ __forceinline__ float sum_add(float v, float w) {
  if constexpr (TY == kI8)
    return __builtin_bit_cast(float, __builtin_bit_cast(int, v) + __builtin_bit_cast(int, w));
  else
    return v + w;
}
// What a product's launch does besides the product; kernels of their own, so that a plain one is not
// longer for it: nothing, pack what stands before the activation (pre8), or add up column sums (in a
// backward pass, whose products have nothing else in their epilogue).
enum { kPlain, kPack, kSums };
// Whether a lane takes part in what finish8 does: columns that do not exist still belong to a
// block of the checkpoint.
template <int MORE>
__device__ __forceinline__ bool takes_part(const LinArgs& p, int row, int col) {
  return row < p.M && (col < p.N || MORE == kPack);
}
__device__ __forceinline__ void put_pre8(const LinArgs& p, int64_t row, int col, const float (&v)[8],
                                         int n, int ot) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = e < n ? v[e] : 0.f;
  // rounded to 0, a positive value would lose relu's slope of 1
  const Block8 b = pack_block8(x, ot, p.act == LINEAR_ACT_RELU ? 1.f : -127.f);
  if (n <= 0) return;
  store_bytes8(p.pre8 + row * p.ldp8 + col, b.lo, b.hi, n);
  if ((col & 31) == 0) p.pre8_scale[row * p.ldps + (col >> 5)] = (uint8_t)b.scale;
}
template <int TY, int MORE>
__device__ __forceinline__ void finish8(const LinArgs& p, int row, int col, float (&v)[8],
                                        const Columns& c) {
  const int ot = kBytes<TY> ? p.out_type : TY;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = sum_value<TY>(v[e]);
  if (kBytes<TY>) {
    // one scale after the other: their product can leave fp32's range where the result does not
    const float sa = p.scale_a ? p.scale_a[row] : 1.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = v[e] * sa * c.sb[e] + c.bias[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += c.bias[e];
  }
  if (p.pre) store8(p.pre + (int64_t)row * p.ldp + col, v, c.n, ot);
  if constexpr (MORE == kPack) {
    put_pre8(p, row, col, v, c.n, ot);
    if (c.n <= 0) return;
  }
  act_n(v, p.act);
  if (p.res) {
    float r[8];
    load8(r, p.res + (int64_t)row * p.ldr + col, c.n, ot, p.N >= 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += r[e];
  }
  store8(p.out + (int64_t)row * p.ldo + col, v, c.n, ot);
}

// ---- tiles -----------------------------------------------------------------------------------
// A BM x BN tile by WM x WN waves, panels of BK slots.  XB is the MFMA block: 32, or 16 (16-bit
// types only).  One k step covers KD slots of both operands.
template <int TY_, int BM_, int BN_, int BK_, bool AKM, bool BKM, int WM_, int WN_, int XB_,
          bool HALVES_ = false>
struct Tile {
  static constexpr bool HALVES = HALVES_;   // e4m3 values multiplied as f16 (see kHalvesK)
  static constexpr int TY = TY_, BM = BM_, BN = BN_, BK = BK_, WM = WM_, WN = WN_, XB = XB_;
  static constexpr int NW = WM * WN;
  using OA = gk::Opnd<BM, BK, AKM, WM, NW, XB>;
  using OB = gk::Opnd<BN, BK, BKM, WN, NW, XB>;
  static constexpr int R = TY == kE4M3 ? 2 : 1;          // 16-byte LDS chunks per fragment
  static constexpr int KD = OA::KD * R, KS = BK / KD;
  static constexpr int WTM = BM / WM, WTN = BN / WN, TM = OA::T, TN = OB::T;
  static constexpr int VN = XB == 16 ? 4 : 16;
  static constexpr int A_BYTES = OA::BYTES, STAGE = OA::BYTES + OB::BYTES;
  using Acc = std::conditional_t<XB == 16, float4v, float16v>;
  using Frag = std::conditional_t<TY == kE4M3, int8v, int4v>;
  static_assert(!kBytes<TY> || (AKM && BKM), "8-bit operands are k-major");
  static_assert(TY != kE4M3 || XB == 32, "MFMA block of e4m3 operands");
};

template <class T, class O>
__device__ __forceinline__ typename T::Frag read_frag(const char GK_LDS* st,
                                                      const int (&o)[O::NOFF], int t, int kk) {
  if constexpr (T::R == 1) {
    return __builtin_bit_cast(int4v, gk::read_operand<O>(st, o, t, kk));
  } else {
    // any assignment of k to lanes serves, as long as both operands share it
    const int4v lo = __builtin_bit_cast(int4v, gk::read_operand<O>(st, o, t, 2 * kk));
    const int4v hi = __builtin_bit_cast(int4v, gk::read_operand<O>(st, o, t, 2 * kk + 1));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

// 8 e4m3 values as f16, which holds them exactly.  The 8-bit matrix instruction rounds inside:
// its sums are off by up to 2^-13 of the products' magnitudes for K = 7 and 2^-17 for K = 1000
// (f16: 2^-22).  Where the product is bound by memory or by latency -- few rows, or K up to
// kHalvesK -- the f16 instruction, of half the rate, costs little or nothing.
constexpr int kHalvesK = 512;
__device__ __forceinline__ int4v halves(int lo, int hi) {
  int4v v;
  v[0] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, false));
  v[1] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.f, true));
  v[2] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, false));
  v[3] = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.f, true));
  return v;
}

// The blocks are computed transposed (b's columns as the rows of the product): a lane then holds
// 4 consecutive columns of one row of the result -- with XB = 16, row l % 16, columns 4 (l / 16)
// + v; with XB = 32, row l % 32, columns 8 (v / 4) + 4 (l / 32) + v % 4.
template <class T>
__device__ __forceinline__ void mma(typename T::Acc& acc, const typename T::Frag& a,
                                    const typename T::Frag& b) {
  if constexpr (T::TY == kF16)
    acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8, b),
                                                 __builtin_bit_cast(half8, a), acc, 0, 0, 0);
  else if constexpr (T::TY == kBF16)
    acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b),
                                                  __builtin_bit_cast(bf16x8, a), acc, 0, 0, 0);
  else if constexpr (T::TY == kI8)
    acc = __builtin_bit_cast(
        float16v, __builtin_amdgcn_mfma_i32_32x32x32_i8(b, a, __builtin_bit_cast(int16v, acc), 0,
                                                        0, 0));
  else if constexpr (T::HALVES)
#pragma unroll
    for (int d = 0; d < 8; d += 2)
      acc = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          __builtin_bit_cast(half8, halves(b[d], b[d + 1])),
          __builtin_bit_cast(half8, halves(a[d], a[d + 1])), acc, 0, 0, 0);
  else
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b, a, acc, 0, 0, 0, 0, 0, 0);
}

// In place on accumulator registers (see mfma16 in gemm_kernels.hpp, whose wait states and
// their check at build time hold here too).
template <class T>
__device__ __forceinline__ void mma_inplace(typename T::Acc& acc, const typename T::Frag& a,
                                            const typename T::Frag& b) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (T::TY == kF16)
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else if constexpr (T::TY == kBF16)
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else if constexpr (T::TY == kI8)
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
  else
    asm volatile("v_mfma_f32_32x32x64_f8f6f4 %0, %1, %2, %0" : "+a"(acc) : "v"(b), "v"(a));
#else
  (void)acc, (void)a, (void)b;   // the host has no such registers
#endif
}

// ---- operands --------------------------------------------------------------------------------
// Buffer resource over `bytes` (even) from a 2-byte aligned address.  The hardware checks each
// dword of a load against the end; the end is moved up to a whole dword of memory where it cuts
// one (so its first half is still read), never beyond it.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, int64_t bytes) {
  const uint64_t b = ((uintptr_t)base & 2) ? (uint64_t)bytes
                                           : ((uint64_t)bytes + 3) & ~(uint64_t)3;
  const uint32_t hi = (uint32_t)(b >> 32), lo = (uint32_t)b;
  const uint32_t n = (hi & 0x80000000u) ? 0u : (hi ? 0xFFFFFFFCu : lo);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

// Loads of one operand's panels.
template <class O>
struct Loader {
  const uint16_t* ptr;
  int64_t ld, ext;
  int x0;
  uint32_t off[O::LD];
  __device__ __forceinline__ void init(const uint16_t* p, int64_t ld_, int X, int K2, int x0_,
                                       int w, int lane) {
    ptr = p;
    ld = ld_;
    x0 = x0_;
    ext = extent<O::KM>(X, K2, ld_);
    gk::slot_offsets<O>(off, w, lane, ld_);
  }
  // Resource of the whole panel whose first k slot is k0 (empty unless live).
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(int64_t k0, bool live) const {
    const int64_t e0 = elem_off<O::KM>(x0, k0, ld);
    return make_rsrc(ptr + (live ? e0 : 0), live ? 2 * (ext - e0) : 0);
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int i, char GK_LDS* dst,
                                       int w) const {
    gk::buffer_load_lds16(r, (void GK_LDS*)(dst + (i * O::NW + w) * 1024), off[i]);
  }
  __device__ __forceinline__ void panel(int64_t k0, bool live, char GK_LDS* dst, int w) const {
    const __amdgpu_buffer_rsrc_t r = rsrc(k0, live);
#pragma unroll
    for (int i = 0; i < O::LD; ++i) load(r, i, dst, w);
  }
  // The ragged panel: `rem` elements of k from slot k0 on, zeros after them, through registers.
  // Each chunk is put together from aligned dwords, so that none straddles the matrix's end.
  template <int TY>
  __device__ __forceinline__ void ragged(int64_t k0, int rem, char GK_LDS* dst, int w,
                                         int lane) const {
    const int64_t e0 = elem_off<O::KM>(x0, k0, ld);
    const uint32_t lead = (uint32_t)(uintptr_t)(ptr + e0) & 2u;
    const __amdgpu_buffer_rsrc_t r =
        make_rsrc((const char*)(ptr + e0) - lead, 2 * (ext - e0) + lead);
#pragma unroll
    for (int i = 0; i < O::LD; ++i) {
      const int q = (i * O::NW + w) * 64 + lane;
      const int row = q / O::CH, c = (q % O::CH) ^ gk::swz<O>(row);
      u32x4 v = gk::load_chunk<true>(r, off[i] + lead);
      if constexpr (!O::KM) {
        if (row >= rem) v = u32x4{0u, 0u, 0u, 0u};
      } else if constexpr (kBytes<TY>) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const int have = rem - (c * 16 + 4 * d);   // bytes of this dword that exist
          v[d] &= have >= 4 ? ~0u : (have <= 0 ? 0u : (1u << (8 * have)) - 1u);
        }
      } else {
        v = gk::mask_k(v, c * 8, rem);
      }
      *(u32x4 GK_LDS*)(dst + q * 16) = v;
    }
  }
};

// ---- a wave's block of sums, through LDS ---------------------------------------------------
// 32 rows at a time: written in 4-column pieces as the MFMA leaves them, read as 8 columns a
// lane.  A row of the slab is 4 floats longer than the block, which puts the 16 rows that a
// wave writes in one LDS cycle on different banks.
template <class T>
struct Slab {
  static constexpr int LDW = T::WTN + 4, BYTES = 32 * LDW * 4;
  static constexpr int LANES = T::WTN / 8, ROWS = 64 / LANES, ITERS = 32 / ROWS;
  // Rows of a lane in flight: 8 where a product is short for its result (8-bit operands: int8
  // 4095x4097x4093 with residual 94.5 us, 96.7 with 4), else 4 (4096^3 bf16 with all three products
  // of a training step 348.8, with 8 351.0).
  static constexpr int MOST = kBytes<T::TY> ? 8 : 4, U = ITERS < MOST ? ITERS : MOST;
};

template <class T, int MORE>
__device__ __forceinline__ void epilogue(const LinArgs& p, const typename T::Acc (&acc)[T::TM][T::TN],
                                         int m0, int n0, int wm, int wn, int lane,
                                         char GK_LDS* slab, float* W) {   // W: a slice's block, or null
  using S = Slab<T>;
  constexpr int RB = 32 / T::XB;   // MFMA rows of blocks in a slab
  float GK_LDS* const s = (float GK_LDS*)slab;
  const int rr = lane / S::LANES, cc = (lane % S::LANES) * 8;
  const int col = n0 + wn * T::WTN + cc;
  const int row0 = m0 + wm * T::WTM + rr;
  const bool whole = T::BM <= p.M - m0 && T::BN <= p.N - n0;
  const int ot = kBytes<T::TY> ? p.out_type : T::TY;
  Columns c;
  if constexpr (MORE == kSums)
    c.n = p.N - col;
  else
    c = load_columns<T::TY>(p, col);
  const float GK_LDS* const sr = s + rr * S::LDW + cc;
  // block t of the slab's rows
  auto deposit = [&](int t) __attribute__((always_inline)) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the slab's last reads are done
#pragma unroll
    for (int b = 0; b < RB; ++b)
#pragma unroll
      for (int tn = 0; tn < T::TN; ++tn)
#pragma unroll
        for (int v = 0; v < T::VN; v += 4) {
          const int r = b * 16 + (lane & (T::XB - 1));
          const int x = tn * T::XB + (T::XB == 16 ? 4 * (lane >> 4) : 2 * v + 4 * (lane >> 5));
          const typename T::Acc& q = acc[t * RB + b][tn];
          *(float4v GK_LDS*)(s + r * S::LDW + x) = float4v{q[v], q[v + 1], q[v + 2], q[v + 3]};
        }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  };
  if (W != nullptr) {
#pragma unroll
    for (int t = 0; t < T::TM / RB; ++t) {
      deposit(t);
      float* const w = W + (int64_t)(wm * T::WTM + t * 32 + rr) * T::BN + wn * T::WTN + cc;
#pragma unroll
      for (int i = 0; i < S::ITERS; ++i) {
        const float GK_LDS* const q = sr + i * S::ROWS * S::LDW;
        *(float4v*)(w + i * S::ROWS * T::BN) = *(const float4v GK_LDS*)q;
        *(float4v*)(w + i * S::ROWS * T::BN + 4) = *(const float4v GK_LDS*)(q + 4);
      }
    }
    return;
  }
  // U rows of a lane at once, their loads in flight together.  INSIDE: a tile inside the matrix,
  // no bounds; else rows past the last one repeat its loads, and nothing outside is stored.
  auto finish = [&](auto inside) __attribute__((always_inline)) {
    constexpr bool INSIDE = decltype(inside)::value;
    constexpr int U = S::U;
    // one copy of what follows for all t: the accumulators' numbers have to be constants, the rest not
#pragma unroll 1
    for (int t = 0; t < T::TM / RB; ++t) {
#pragma unroll
      for (int x = 0; x < T::TM / RB; ++x)
        if (x == t) deposit(x);
      const int row_t = row0 + t * 32;
#pragma unroll 1
      for (int i = 0; i < S::ITERS; i += U) {
        float f[U * 8];
        u32x4 res[U];
        float sa[U];
        const int row = row_t + i * S::ROWS;
        auto row_of = [&](int u) __attribute__((always_inline)) {
          const int64_t r = row + u * S::ROWS;
          return !INSIDE && r >= p.M ? (int64_t)p.M - 1 : r;
        };
        // one branch for all of a lane's loads: after each the compiler would wait for them
        if (MORE != kSums && p.res) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint16_t* const at = p.res + row_of(u) * p.ldr + col;
            res[u] = INSIDE ? (u32x4)*(const u32x4_any*)at : raw8_load(at, c.n, p.N >= 8);
          }
        }
        if (kBytes<T::TY>) {
#pragma unroll
          for (int u = 0; u < U; ++u) sa[u] = 1.f;
          if (p.scale_a) {
#pragma unroll
            for (int u = 0; u < U; ++u) sa[u] = p.scale_a[row_of(u)];
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const float GK_LDS* const q = sr + (i + u) * S::ROWS * S::LDW;
          const float4v lo = *(const float4v GK_LDS*)q, hi = *(const float4v GK_LDS*)(q + 4);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = sum_value<T::TY>(e < 4 ? lo[e & 3] : hi[e & 3]);
            if constexpr (MORE == kSums)
              f[u * 8 + e] = v;
            else
              f[u * 8 + e] = kBytes<T::TY> ? v * sa[u] * c.sb[e] + c.bias[e] : v + c.bias[e];
          }
        }
        auto values = [&](float (&v)[8], int u) __attribute__((always_inline)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = f[u * 8 + e];
        };
        auto put = [&](uint16_t* base, int64_t ld) __attribute__((always_inline)) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[8];
            values(v, u);
            const int64_t r = row + u * S::ROWS;
            if constexpr (INSIDE)
              *(u32x4_any*)(base + r * ld + col) = pack8(v, ot);
            else if (r < p.M && c.n > 0)
              store8(base + r * ld + col, v, c.n, ot);
          }
        };
        if (MORE != kSums && p.pre) put(p.pre, p.ldp);
        if constexpr (MORE == kPack) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[8];
            values(v, u);
            const int64_t r = row + u * S::ROWS;
            put_pre8(p, r, col, v, INSIDE ? 8 : r < p.M ? c.n : 0, ot);
          }
        }
        if constexpr (MORE != kSums) act_n(f, p.act);
        if (MORE != kSums && p.res) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float r[8];
            unpack8(r, INSIDE ? res[u] : raw8_shift(res[u], c.n, p.N >= 8), ot);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[u * 8 + e] += r[e];
          }
        }
        put(p.out, p.ldo);
      }
    }
  };
  if (whole)
    finish(std::true_type{});
  else
    finish(std::false_type{});
}

// k slots of the matrices, and the ragged panel
struct Panels {
  int np, rem, k2, first;   // panels, elements of the ragged one (0: none), slots, its slot
  // slot where panel s (not the ragged one) starts
  int base;
};
template <int TY, int BK>
__device__ __forceinline__ Panels panels_of(int K) {
  constexpr int E = kBytes<TY> ? 2 : 1;   // elements per slot
  Panels q;
  q.k2 = K / E + K % E;   // E is 1 or 2; K + 1 need not fit
  q.rem = K % (BK * E);
  q.np = K / (BK * E) + (q.rem ? 1 : 0);
  q.first = K / (BK * E) * BK;
  q.base = q.rem ? -BK : 0;
  return q;
}

// Corner of a tile.
template <int BM, int BN>
__device__ __forceinline__ void corner_of(const LinArgs& p, int tile, int& m0, int& n0) {
  int pid, pid_m, pid_n;
  gk::program_tile(tile, p.num_programs, p.num_pid_m, p.num_pid_n, p.group_m,
                   p.xcd_remap, pid, pid_m, pid_n);
  m0 = pid_m * BM;
  n0 = pid_n * BN;
}

// ---------------------------------------------------------------------------------------
// Staged tile: NS LDS stages, operands read RD k steps ahead, one barrier per panel; panels
// past the end are empty (zeros, no memory touched).  64 x 64 with 4 stages for what latency
// bounds (512^3 f16 with bias, gelu and residual 5.8 us; 64 x 8192 x 8192 e4m3 16.8 us, 4.0
// TB/s); 128 x 128 with 2 stages, two workgroups a CU, where 256 x 256 tiles leave CUs idle (2048 x
// 4096 x 4096 bf16: 62 us, 1.11 PFLOP/s; 256 x 256 71 us in two slices of k).
// ---------------------------------------------------------------------------------------
template <class T, int NS, int RD, bool AKM, bool BKM, int MORE = kPlain>
__device__ __forceinline__ void staged_tile(const LinArgs& p, int m0, int n0, const Work& k,
                                            char GK_LDS* const (&S)[NS]) {
  using OA = typename T::OA;
  using OB = typename T::OB;
  constexpr int KS = T::KS, BK = T::BK;
  constexpr int NM = T::TM * T::TN, ND = T::R * (OA::READS + OB::READS), NV = OA::LD + OB::LD;
  static_assert(NS >= 2 && NS * T::STAGE <= 160 * 1024 && (NS - 2) * NV <= 63, "stages");
  static_assert(RD >= 1 && RD < KS && (NS * KS) % (RD + 1) == 0, "read-ahead distance");
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / T::WN, wn = w % T::WN;
  const Panels q = panels_of<T::TY, BK>(p.K);
  const int s0 = k.z < 0 ? 0 : k.z * p.per_split;
  const int s1 = k.z >= 0 && s0 + p.per_split < q.np ? s0 + p.per_split : q.np;
  const int np = s1 - s0;   // this slice's panels (at least one if split)

  Loader<OA> la;
  Loader<OB> lb;
  la.init(p.A, p.lda, p.M, q.k2, m0, w, lane);
  lb.init(p.B, p.ldb, p.N, q.k2, n0, w, lane);
  // Without a ragged panel the matrices' last elements are in the last panel, where the range
  // check can cut them off (see last_element_slot): their owners write them again.
  uint16_t va = 0, vb = 0;
  int pa = -1, pb = -1;
  if (!kBytes<T::TY> && q.rem == 0 && s1 == q.np) {
    pa = gk::last_element_slot<OA>(m0, p.M, p.K, p.A, la.ext, tid, va);
    pb = gk::last_element_slot<OB>(n0, p.N, p.K, p.B, lb.ext, tid, vb);
  }
  auto patch = [&](char GK_LDS* base) __attribute__((always_inline)) {
    if (pa >= 0) *(uint16_t GK_LDS*)(base + pa) = va;
    if (pb >= 0) *(uint16_t GK_LDS*)(base + T::A_BYTES + pb) = vb;
  };
  auto issue = [&](int s, char GK_LDS* base) __attribute__((always_inline)) {
    const int64_t k0 = (int64_t)q.base + (int64_t)(s0 + s) * BK;
    la.panel(k0, s < np, base, w);
    lb.panel(k0, s < np, base + T::A_BYTES, w);
  };
  typename T::Acc acc[T::TM][T::TN];
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) acc[i][j] = typename T::Acc{};
  int oa[OA::NOFF], ob[OB::NOFF];
  gk::operand_offsets<OA>(oa, wm, lane, 0);
  gk::operand_offsets<OB>(ob, wn, lane, T::A_BYTES);
  typename T::Frag fa[RD + 1][T::TM], fb[RD + 1][T::TN];
  auto read = [&](int slot, const char GK_LDS* st, int kk) __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < T::TM; ++t) fa[slot][t] = read_frag<T, OA>(st, oa, t, kk);
#pragma unroll
    for (int t = 0; t < T::TN; ++t) fb[slot][t] = read_frag<T, OB>(st, ob, t, kk);
  };
  // Panel s at position j of the unrolled loop.  NS == 2: its stage is refilled past the
  // barrier in its last steps; NS >= 3: the previous panel's stage at its start.
  auto panel = [&](int s, int j) __attribute__((always_inline)) {
    char GK_LDS* const cur = S[j];
    char GK_LDS* const nxt = S[(j + 1) % NS];
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      if (NS >= 3 && kk == 0) issue(s + NS - 1, S[(j + NS - 1) % NS]);
      if (kk == KS - RD) {
        wait_vmcnt<(NS - 2) * NV>();    // panel s+1 has landed, this wave's part ...
        if (s + 2 == np) patch(nxt);
        lds_barrier();                  // ... and every wave's
        if (NS == 2) issue(s + 2, cur);
      }
      const int ka = kk + RD;
      if (ka < KS)
        read((j * KS + ka) % (RD + 1), cur, ka);
      else
        read((j * KS + ka) % (RD + 1), nxt, ka - KS);
      const int f = (j * KS + kk) % (RD + 1);
#pragma unroll
      for (int tm = 0; tm < T::TM; ++tm)
#pragma unroll
        for (int tn = 0; tn < T::TN; ++tn) mma<T>(acc[tm][tn], fa[f][tm], fb[f][tn]);
      if (NS >= 3 ? kk == 0 : kk == KS - RD)
        gk::sched_step<NM, ND, NV>();
      else
        gk::sched_step<NM, ND, 0>();
    }
  };
  if (np > 0) {
    constexpr int kPre = NS == 2 ? 2 : NS - 1;
    if (q.rem && s0 == 0) {
      la.template ragged<T::TY>(q.first, q.rem, S[0], w, lane);
      lb.template ragged<T::TY>(q.first, q.rem, S[0] + T::A_BYTES, w, lane);
    } else {
      issue(0, S[0]);
    }
#pragma unroll
    for (int j = 1; j < kPre; ++j) issue(j, S[j]);
    wait_vmcnt<(kPre - 1) * NV>();
    if (np == 1) patch(S[0]);
    lds_barrier();
#pragma unroll
    for (int d = 0; d < RD; ++d) read(d, S[0], d);
  }
  for (int s = 0; s < np; s += NS) {
#pragma unroll
    for (int j = 0; j < NS; ++j) panel(s + j, j);
  }
  wait_vmcnt<0>();   // the empty loads past the end, before LDS is used again
  lds_barrier();     // every wave has read its last operands
  constexpr int PER = (T::NW + NS - 1) / NS;   // slabs per stage
  static_assert(PER * Slab<T>::BYTES <= T::STAGE, "slabs fit the stages");
  // The wave's stage, chosen among opaque addresses: recognised as S[w % NS], the compiler puts S
  // itself into LDS and has every workgroup read its dispatch packet from host memory for the
  // workgroup's shape, about 0.5 us a workgroup, one after the other.
  uint32_t slab_at = 0;
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    uint32_t at = (uint32_t)(uintptr_t)S[j];
    asm volatile("" : "+s"(at));
    if (w % NS == j) slab_at = at;
  }
  char GK_LDS* const slab = (char GK_LDS*)(uintptr_t)slab_at + (w / NS) * Slab<T>::BYTES;
  epilogue<T, MORE>(p, acc, m0, n0, wm, wn, lane, slab, k.w);
}

// The NS LDS stages of a staged tile as separate objects (a refill of one is then seen not to
// touch another), their addresses assigned one by one (a list of them would become a table).
#define LK_DECLARE_STAGES(NS, BYTES)                                             \
  __shared__ __attribute__((aligned(16))) char stage0[BYTES];                    \
  __shared__ __attribute__((aligned(16))) char stage1[BYTES];                    \
  __shared__ __attribute__((aligned(16))) char stage2[(NS) > 2 ? (BYTES) : 16];  \
  __shared__ __attribute__((aligned(16))) char stage3[(NS) > 3 ? (BYTES) : 16];  \
  static_assert(NS == 2 || NS == 4, "stages");                                   \
  char GK_LDS* S[NS];                                                            \
  S[0] = (char GK_LDS*)stage0;                                                   \
  S[1] = (char GK_LDS*)stage1;                                                   \
  if constexpr ((NS) > 2) {                                                      \
    S[2] = (char GK_LDS*)stage2;                                                 \
    S[3] = (char GK_LDS*)stage3;                                                 \
  }

// Sum over n partial rows of one block of 32 columns (see store_partial8), in order within a
// thread and then over the 32 threads of a column, 4 columns a thread of 256.
typedef float4v SumLds[32][9];
template <int TY>
__device__ __forceinline__ void sum_block(const float* part, int n, int block, int cols,
                                          uint16_t* out, SumLds& s) {
  const int t = threadIdx.x, c = t & 7, r = t >> 3;
  const float* const q = part + (int64_t)block * n * 32 + c * 4;
  float4v v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int i = r; i < n; i += 32) v += *(const float4v*)(q + i * 32);
  s[r][c] = v;
  __syncthreads();
  if (t < 32 && block * 32 + t < cols) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += s[i][t / 4][t % 4];
    out[block * 32 + t] = to_16(sum, TY);
  }
}

// The workgroups of a product's launch that add partial sums.
template <int TY>
__device__ __forceinline__ bool sums_done(const LinArgs& p, SumLds& s) {
  if (p.sum_part == nullptr || (int)blockIdx.x < p.sum_first) return false;
  sum_block<TY>(p.sum_part, p.sum_n, blockIdx.x - p.sum_first, p.sum_cols, p.sum_out, s);
  return true;
}

template <int TY, int BM, int BN, int BK, int NS, int RD, int WM, int WN, bool AKM, bool BKM,
          bool HALVES, int MORE>
__global__ void __launch_bounds__(64 * WM * WN) lin_staged(LinArgs p) {
  using T = Tile<TY, BM, BN, BK, AKM, BKM, WM, WN, 32, HALVES>;
  LK_DECLARE_STAGES(NS, T::STAGE)
  if constexpr (MORE == kSums) {
    __shared__ SumLds sums;
    if (sums_done<TY>(p, sums)) return;
  }
  int m0, n0;
  const Work k = work_of<BM, BN>(p, blockIdx.x);
  corner_of<BM, BN>(p, k.tile, m0, n0);
  staged_tile<T, NS, RD, AKM, BKM, MORE>(p, m0, n0, k, S);
}

// Both products of a small backward pass and the last step of its bias gradient in one launch:
// workgroups of da's 64 x 64 tiles, then db's, then blocks of 32 columns of dbias.  Latency bounds
// it (1024 x 768 x 128 f16: 7.9 us; as three launches 22 us with the element-wise pass, 13 so).
struct PairArgs {
  LinArgs da, db;
  const float* part;
  uint16_t* dbias;
  int32_t groups, cols;   // of the partial sums
};
template <int TY, bool BKM>
__global__ void __launch_bounds__(256) lin_pair(PairArgs p) {
  using TA = Tile<TY, 64, 64, 64, true, BKM, 2, 2, 32>;
  using TB = Tile<TY, 64, 64, 64, false, false, 2, 2, 32>;
  LK_DECLARE_STAGES(4, TA::STAGE)
  int h = blockIdx.x, m0, n0;
  if (h < p.da.num_programs) {
    corner_of<64, 64>(p.da, h, m0, n0);
    staged_tile<TA, 4, 3, true, BKM>(p.da, m0, n0, Work{h, -1, nullptr}, S);
    return;
  }
  h -= p.da.num_programs;
  if (h < p.db.num_programs) {
    corner_of<64, 64>(p.db, h, m0, n0);
    staged_tile<TB, 4, 3, false, false>(p.db, m0, n0, Work{h, -1, nullptr}, S);
    return;
  }
  __shared__ SumLds sums;
  sum_block<TY>(p.part, p.groups, h - p.db.num_programs, p.cols, p.dbias, sums);
}

// ---------------------------------------------------------------------------------------
// A small backward pass in one launch: both products on 64 x 64 tiles, with dpre = dc act'(pre)
// made on the way into LDS by every workgroup that needs it (a few times over, which costs less
// than a pass of its own and its launch) and rounded there to the operands' type (see dact_rows),
// and its column sums by the workgroups of db's first
// tiles along k.  Panels go through registers, three ahead, and two LDS stages.
// ---------------------------------------------------------------------------------------
struct SmallArgs {
  LinArgs da, db;   // dc in the place of dpre
  const uint16_t* pre;   // without an activation dc again (loaded, not used)
  int64_t ldpre;
  uint16_t* dbias;
  int32_t act;
};

// One operand's panel on its way through registers.  Rows have at least 8 values (see
// raw8_load), and the loads are free of branches: after one, the compiler waits for them.
template <class O, bool DPRE>
struct RegPanel {
  u32x4 v[O::LD], u[DPRE ? O::LD : 1];
  // Loads the panel from k0 on.  Rows past the matrix repeat its last one.
  __device__ __forceinline__ void fetch(const uint16_t* p, int64_t ld, const uint16_t* pre,
                                        int64_t ldpre, int x0, int k0, int X, int K, int t) {
#pragma unroll
    for (int i = 0; i < O::LD; ++i) {
      const int q = i * O::NW * 64 + t, row = q / O::CH, c = (q % O::CH) * 8;
      const int e = (O::KM ? k0 : x0) + c, n = (O::KM ? K : X) - e;
      const int r = (O::KM ? x0 : k0) + row, R = O::KM ? X : K;
      const int64_t at = r < R ? r : R - 1;
      v[i] = raw8_load(p + at * ld + e, n, true);
      if constexpr (DPRE) u[i] = raw8_load(pre + at * ldpre + e, n, true);
    }
  }
  // What lies outside the matrix along k becomes 0 (along x it feeds only results that are not
  // stored).
  __device__ __forceinline__ void settle(int i, int x0, int k0, int X, int K, int t) {
    const int q = i * O::NW * 64 + t, row = q / O::CH, c = (q % O::CH) * 8;
    const int n = O::KM ? K - k0 - c : X - x0 - c;
    v[i] = raw8_shift(v[i], n, true);
    if constexpr (DPRE) u[i] = raw8_shift(u[i], n, true);
    if (!O::KM && k0 + row >= K) v[i] = u32x4{0u, 0u, 0u, 0u};
  }
};

template <class T, bool AKM, bool BKM, int DP, bool SUM>
__device__ __forceinline__ void small_tile(const LinArgs& p, const SmallArgs& a, int tile,
                                           char GK_LDS* smem) {
  using OA = typename T::OA;
  using OB = typename T::OB;
  constexpr int TY = T::TY;
  const int t = threadIdx.x, lane = t & 63;
  const int w = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = w / T::WN, wn = w % T::WN;
  int m0, n0;
  corner_of<64, 64>(p, tile, m0, n0);
  const bool sums = SUM && a.dbias != nullptr && (DP == 1 ? n0 : m0) == 0;
  const int np = (p.K + 63) / 64;
  RegPanel<OA, DP == 1> ra[3];
  RegPanel<OB, DP == 2> rb[3];
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  auto fetch = [&](int j, int s) __attribute__((always_inline)) {
    const int k0 = (s < np ? s : np - 1) * 64;   // past the end: loaded again, not used
    ra[j].fetch(p.A, p.lda, a.pre, a.ldpre, m0, k0, p.M, p.K, t);
    rb[j].fetch(p.B, p.ldb, a.pre, a.ldpre, n0, k0, p.N, p.K, t);
  };
  auto put = [&](auto& r, auto is_dpre, int i, char GK_LDS* at) __attribute__((always_inline)) {
    if constexpr (is_dpre.value) {
      if (a.act != LINEAR_ACT_NONE || (SUM && sums)) {
        float v[8], u[8];
        unpack8(v, r.v[i], TY);
        unpack8(u, r.u[i], TY);
        slope8(v, u, a.act);
        if (SUM && sums) {
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += v[e];
        }
        r.v[i] = pack8(v, TY);
      }
    }
    *(u32x4 GK_LDS*)at = r.v[i];
  };
  auto deposit = [&](int j, int s) __attribute__((always_inline)) {
    if (s >= np) return;
    char GK_LDS* const st = smem + (s & 1) * T::STAGE;
#pragma unroll
    for (int i = 0; i < OA::LD; ++i) {
      const int q = i * 256 + t;
      ra[j].settle(i, m0, s * 64, p.M, p.K, t);
      put(ra[j], std::integral_constant<bool, DP == 1>{}, i,
          st + gk::lds_chunk<OA>(q / OA::CH, q % OA::CH));
    }
#pragma unroll
    for (int i = 0; i < OB::LD; ++i) {
      const int q = i * 256 + t;
      rb[j].settle(i, n0, s * 64, p.N, p.K, t);
      put(rb[j], std::integral_constant<bool, DP == 2>{}, i,
          st + T::A_BYTES + gk::lds_chunk<OB>(q / OB::CH, q % OB::CH));
    }
  };
  int oa[OA::NOFF], ob[OB::NOFF];
  gk::operand_offsets<OA>(oa, wm, lane, 0);
  gk::operand_offsets<OB>(ob, wn, lane, T::A_BYTES);
  typename T::Acc acc[1][1];
  static_assert(T::TM == 1 && T::TN == 1, "one block a wave");
  acc[0][0] = typename T::Acc{};
#pragma unroll
  for (int j = 0; j < 3; ++j) fetch(j, j);
  deposit(0, 0);
  for (int s = 0; s < np; s += 3) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      if (s + j < np) {
        __syncthreads();           // panel s + j is in LDS, panel s + j - 1 has been read
        fetch(j, s + j + 3);
        const char GK_LDS* const st = smem + ((s + j) & 1) * T::STAGE;
#pragma unroll
        for (int kk = 0; kk < T::KS; ++kk)
          mma<T>(acc[0][0], read_frag<T, OA>(st, oa, 0, kk), read_frag<T, OB>(st, ob, 0, kk));
        deposit((j + 1) % 3, s + j + 1);
      }
    }
  }
  __syncthreads();
  if (SUM && sums) {
    // a thread's chunks all lie in the 8 columns from 8 (t % 8) on
    float GK_LDS* const f = (float GK_LDS*)smem;
    const int X = DP == 1 ? p.M : p.N, x0 = DP == 1 ? m0 : n0;
#pragma unroll
    for (int e = 0; e < 8; ++e) f[(t >> 3) * 68 + (t & 7) * 8 + e] = sum[e];
    __syncthreads();
    if (t < 64 && x0 + t < X) {
      float v = 0.f;
#pragma unroll 8
      for (int i = 0; i < 32; ++i) v += f[i * 68 + t];
      a.dbias[x0 + t] = to_16(v, TY);
    }
    __syncthreads();
  }
  epilogue<T, kPlain>(p, acc, m0, n0, wm, wn, lane, smem + w * Slab<T>::BYTES, nullptr);
}

// BKM: b as da's operand is k-contiguous.  COLS: db is column-major (its transpose computed).
template <int TY, bool BKM, bool COLS>
__global__ void __launch_bounds__(256) lin_small_bwd(SmallArgs p) {
  using TA = Tile<TY, 64, 64, 64, true, BKM, 2, 2, 32>;
  using TB = Tile<TY, 64, 64, 64, false, false, 2, 2, 32>;
  static_assert(4 * Slab<TA>::BYTES <= 2 * TA::STAGE && 32 * 68 * 4 <= 2 * TA::STAGE, "LDS");
  __shared__ __attribute__((aligned(16))) char smem[2 * TA::STAGE];
  const int h = blockIdx.x;
  if (h < p.da.num_programs)
    small_tile<TA, true, BKM, 1, false>(p.da, p, h, (char GK_LDS*)smem);
  else
    small_tile<TB, false, false, COLS ? 1 : 2, true>(p.db, p, h - p.da.num_programs,
                                                     (char GK_LDS*)smem);
}

// ---------------------------------------------------------------------------------------
// The 256 x 256 tile (64 slots deep, 4 waves of 128 x 128): the panels in five 32 KiB LDS slots,
// B's in a ring of three and A's in a ring of two, two k steps per panel, each scheduled by
// hand -- see ring_tile in gemm_kernels.hpp, whose order of loads, reads and barriers this is.
// 16-bit types: 64 MFMAs of 16x16x32 a step (int8: of 16x16x64); e4m3: 16 of 32x32x64, the same
// cycles.  Bound by the matrix cores at the chip's power limit: 8192^3 bf16 with bias, gelu and pre-activation 764 - 809
// us (1.36 - 1.44 PFLOP/s, MFMA busy 72 %), e4m3 with bias and silu 390 - 423 us (2.6 - 2.8), int8
// 397 - 418 us (2.6 - 2.8), no LDS bank conflicts.
// ---------------------------------------------------------------------------------------
template <int TY, bool AKM, bool BKM, int MORE>
__device__ __forceinline__ void ring_tile(const LinArgs& p, int m0, int n0, const Work& k,
                                          char GK_LDS* const (&SA)[2],
                                          char GK_LDS* const (&SB)[3]) {
  using T = Tile<TY, 256, 256, 64, AKM, BKM, 2, 2, TY == kE4M3 ? 32 : 16>;
  using OA = typename T::OA;
  using OB = typename T::OB;
  constexpr int BK = 64, NM = T::TM * T::TN, NF = T::TM + T::TN;
  constexpr int LE = NM / 8, RE = NM / NF;   // MFMAs between loads, between fragment reads
  static_assert(T::KS == 2 && OA::LD == 8 && OB::LD == 8 && NM % 8 == 0 && NM % NF == 0, "ring");
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / 2, wn = w % 2;
  const Panels q = panels_of<TY, BK>(p.K);
  const int s0 = k.z < 0 ? 0 : k.z * p.per_split;
  const int s1 = k.z >= 0 && s0 + p.per_split < q.np ? s0 + p.per_split : q.np;
  const int np = s1 - s0;
  Loader<OA> la;
  Loader<OB> lb;
  la.init(p.A, p.lda, p.M, q.k2, m0, w, lane);
  lb.init(p.B, p.ldb, p.N, q.k2, n0, w, lane);
  uint16_t va = 0, vb = 0;
  int pa = -1, pb = -1;
  if (!kBytes<TY> && q.rem == 0 && s1 == q.np) {
    pa = gk::last_element_slot<OA>(m0, p.M, p.K, p.A, la.ext, tid, va);
    pb = gk::last_element_slot<OB>(n0, p.N, p.K, p.B, lb.ext, tid, vb);
  }
  auto patch = [&](char GK_LDS* a, char GK_LDS* b) __attribute__((always_inline)) {
    if (pa >= 0) *(uint16_t GK_LDS*)(a + pa) = va;
    if (pb >= 0) *(uint16_t GK_LDS*)(b + pb) = vb;
  };
  typename T::Acc acc[T::TM][T::TN];
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) acc[i][j] = typename T::Acc{};
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) asm volatile("" : "+a"(acc[i][j]));
  asm volatile("s_nop 7" ::: "memory");

  int oa[OA::NOFF], ob[OB::NOFF];
  gk::operand_offsets<OA>(oa, wm, lane, 0);
  gk::operand_offsets<OB>(ob, wn, lane, 0);
  typename T::Frag fa[2][T::TM], fb[2][T::TN];
  auto k_of = [&](int s) { return (int64_t)q.base + (int64_t)(s0 + s) * BK; };
  // refill resources: B's of the panel loaded in the next first step, A's of the second step's
  __amdgpu_buffer_rsrc_t rb = lb.rsrc(k_of(2), 2 < np), ra = rb;

  if (np > 0) {
    if (q.rem && s0 == 0) {
      la.template ragged<TY>(q.first, q.rem, SA[0], w, lane);
      lb.template ragged<TY>(q.first, q.rem, SB[0], w, lane);
    } else {
      la.panel(k_of(0), true, SA[0], w);
      lb.panel(k_of(0), true, SB[0], w);
    }
    la.panel(k_of(1), 1 < np, SA[1], w);
    lb.panel(k_of(1), 1 < np, SB[1], w);
    wait_vmcnt<OA::LD + OB::LD>();
    if (np == 1) patch(SA[0], SB[0]);
    lds_barrier();
#pragma unroll
    for (int t = 0; t < T::TN; ++t) fb[0][t] = read_frag<T, OB>(SB[0], ob, t, 0);
#pragma unroll
    for (int t = 0; t < T::TM; ++t) fa[0][t] = read_frag<T, OA>(SA[0], oa, t, 0);
  }
  auto panel = [&](int s, int j) __attribute__((always_inline)) {
    char GK_LDS* const a_cur = SA[j % 2];
    char GK_LDS* const b_cur = SB[j % 3];
    char GK_LDS* const a_nxt = SA[(j + 1) % 2];
    char GK_LDS* const b_nxt = SB[(j + 1) % 3];
    char GK_LDS* const b_new = SB[(j + 2) % 3];
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      if (i % LE == LE / 4) lb.load(rb, i / LE, b_new, w);
      mma_inplace<T>(acc[i / T::TN][i % T::TN], fa[0][i / T::TN], fb[0][i % T::TN]);
      if (i == 2 * LE) ra = la.rsrc(k_of(s + 2), s + 2 < np);
      if (i == 3 * LE) asm volatile("" : "+s"(ra));
      if (i % RE == 0) {
        const int r = i / RE;
        if (r < T::TN)
          fb[1][r] = read_frag<T, OB>(b_cur, ob, r, 1);
        else
          fa[1][r - T::TN] = read_frag<T, OA>(a_cur, oa, r - T::TN, 1);
      }
    }
    wait_vmcnt<OB::LD>();      // panel s+1 has landed (this wave's part) ...
    if (s + 2 == np) patch(a_nxt, b_nxt);
    lds_barrier();             // ... every wave's; and every wave has read A of panel s
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      if (i % LE == LE / 4) la.load(ra, i / LE, a_cur, w);
      mma_inplace<T>(acc[i / T::TN][i % T::TN], fa[1][i / T::TN], fb[1][i % T::TN]);
      if (i == 2 * LE) rb = lb.rsrc(k_of(s + 3), s + 3 < np);
      if (i == 3 * LE) asm volatile("" : "+s"(rb));
      if (i % RE == 0) {
        const int r = i / RE;
        if (r < T::TN)
          fb[0][r] = read_frag<T, OB>(b_nxt, ob, r, 0);
        else
          fa[0][r - T::TN] = read_frag<T, OA>(a_nxt, oa, r - T::TN, 0);
      }
    }
  };
  for (int s = 0; s < np; s += 6) {
#pragma unroll
    for (int j = 0; j < 6; ++j) {
      if (s + j >= np) break;
      panel(s + j, j);
    }
  }
  wait_vmcnt<0>();
  asm volatile("s_nop 7\n\ts_nop 7\n\ts_nop 7\n\ts_nop 7" ::: "memory");
#pragma unroll
  for (int i = 0; i < T::TM; ++i)
#pragma unroll
    for (int j = 0; j < T::TN; ++j) asm volatile("" : "+a"(acc[i][j]));
  lds_barrier();   // every wave has read its last operands
  static_assert(Slab<T>::BYTES <= 32768, "a slab fits a slot");
  char GK_LDS* slab = SA[0];
  if (w == 1) slab = SA[1];
  if (w == 2) slab = SB[0];
  if (w == 3) slab = SB[1];
  epilogue<T, MORE>(p, acc, m0, n0, wm, wn, lane, slab, k.w);
}

template <int TY, bool AKM, bool BKM, int MORE>
__device__ __forceinline__ void ring(const LinArgs& p) {
  GK_DECLARE_RING()
  if constexpr (MORE == kSums) {
    if (sums_done<TY>(p, *(SumLds*)slot0)) return;
  }
  int m0, n0;
  const Work k = work_of<256, 256>(p, blockIdx.x);
  corner_of<256, 256>(p, k.tile, m0, n0);
  ring_tile<TY, AKM, BKM, MORE>(p, m0, n0, k, SA, SB);
}
template <int TY, bool AKM, bool BKM>
__global__ void __launch_bounds__(256) lin_ring(LinArgs p) {
  ring<TY, AKM, BKM, kPlain>(p);
}
// The same on int8 operands, or with more to do.
template <int TY, bool AKM, bool BKM, int MORE>
__global__ void __launch_bounds__(256) lin_more_ring(LinArgs p) {
  ring<TY, AKM, BKM, MORE>(p);
}

// The k slices of the split tiles added in order, then the epilogue; a thread per 8 columns, 256
// threads a workgroup, PER workgroups a BM x BN tile (the last one not always full).  Latency
// bounds it: 3 - 5 us.
template <int TY, int BM, int BN, int MORE>
__global__ void __launch_bounds__(256) lin_reduce(LinArgs p) {
  constexpr int Q = BN / 8, PER = (BM * Q + 255) / 256;
  const int i = blockIdx.x / PER, t = (blockIdx.x - i * PER) * 256 + threadIdx.x;
  if (t >= BM * Q) return;
  int m0, n0;
  corner_of<BM, BN>(p, p.first_split + i, m0, n0);
  const int r = t / Q, c = (t - r * Q) * 8, row = m0 + r, col = n0 + c;
  if (!takes_part<MORE>(p, row, col)) return;
  const float* w = p.W + (int64_t)i * p.splits * (BM * BN) + r * BN + c;
  float4v lo = *(const float4v*)w, hi = *(const float4v*)(w + 4);
#pragma unroll 4
  for (int z = 1; z < p.splits; ++z) {
    const float4v l = *(const float4v*)(w + (int64_t)z * (BM * BN));
    const float4v h = *(const float4v*)(w + (int64_t)z * (BM * BN) + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = sum_add<TY>(lo[e], l[e]);
      hi[e] = sum_add<TY>(hi[e], h[e]);
    }
  }
  float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  finish8<TY, MORE>(p, row, col, f, load_columns<TY>(p, col));
}

}  // namespace lk
