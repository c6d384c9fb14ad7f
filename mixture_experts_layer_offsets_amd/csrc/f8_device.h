// Products in 8-bit floating point with a scale for each block of 128: formats and
// layouts shared by the f8_*.hip files.
//
//   rows     x[r][k] ~ s[r][k / 128] E4M3(code), s = max(max|x| / 448, 2^-100)
//   weights  w[n][k] ~ s[n / 128][k / 128] E4M3(code)
//   y[r][n] = sum over blocks b of sx[r][b] sw[n / 128][b] (sum of code products)
//
// The inner sum, 128 products of codes, is one v_mfma_f32_16x16x128_f8f6f4 with a
// zero accumulator; the scales multiply its result in fp32, into accumulators in
// registers.  The two scales are multiplied with each other first, in the forward once for
// a lane's four results: one after the other they would cost an operation more a result.
// Where their product is below 2^-126 it is subnormal, and the block's sum off by up to
// 2^-125 (2^-150 times 128 448^2): half a step of bf16 at 2^-117.
//
// Per instruction (32 cycles of the matrix pipe) that is one
// multiply-add a result value, 4 a lane (16 cycles of the vector pipe): the two
// overlap between the waves of a SIMD.  The instruction keeps fewer bits than fp32 of
// its sum: random codes give 1.33e-5 of the results' norm, the scaled and the
// 32-deep instructions the same (measured), so results are only offered in 16 bits.
//
// The instruction takes the weights as its first operand and the rows as its
// second: lane l holds output (or row) l % 16 and the 16-byte chunks l / 16 and
// l / 16 + 4 of the block, and receives outputs 4 (l / 16) + v of row l % 16.  The
// scale of a row is then one value a lane, and that of the weights one of the wave.
//
// Packed weights: a tile is 16 outputs x 128 contraction values, 2 KB, in the order
// in which one wave's two 16-byte loads take it: chunk c (values 16 c ..) of output
// n at byte ((c / 4) 64 + (c % 4) 16 + n) 16.  In LDS it keeps that order: a wave's
// fragment read is then linear.  Tiles are [group][n / 16][k / 128], so that the
// contraction of one tile row is one contiguous stream; behind them a scale a tile,
// [group][n / 16][k / 128] (8 times the same: 0.2 % more bytes, and found by the
// tile's own number).  Outputs past n and values past k have zero codes.
// Quantised rows are [k / 128][rows][128]: one step of a tile's rows is contiguous.
#pragma once

#include "common.h"
#include "f8.h"
#include "gemm_common.h"

namespace moe {
namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x2_f8 __attribute__((ext_vector_type(2)));
typedef __amdgpu_buffer_rsrc_t f8_rsrc_t;

constexpr int kF8Tile = 2048;            // bytes of a tile
constexpr float kF8Least = 0x1p-100f;    // smallest scale
constexpr float kF8PerMost = 1.0f / 448.0f;

__device__ __forceinline__ int f8_chunk(int c, int n) {  // byte of a chunk in its tile
  return ((c >> 2) * 64 + (c & 3) * 16 + n) * 16;
}

__device__ __forceinline__ f8_rsrc_t f8_buffer(const void *p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, bytes, kBufferDword3);
}

__device__ __forceinline__ float f8_from16(uint32_t u16, bool f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)u16) : bf16_to_f32(u16);
}
__device__ __forceinline__ uint16_t f8_to16(float f, bool f16) {
  return f16 ? __builtin_bit_cast(uint16_t, (_Float16)f) : __builtin_bit_cast(uint16_t, (__bf16)f);
}

// Bits of |v|: as integers they order as the magnitudes do, NaN above infinity, so
// that a block's largest is NaN if one of its values is.
__device__ __forceinline__ uint32_t f8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// A block's scale from the bits of its largest magnitude, and what its values are
// multiplied with.  An infinity gives an infinite scale and NaN a NaN one: no output
// that the block reaches is finite then.
__device__ __forceinline__ float f8_scale(uint32_t top, float *inv) {
  const float a = __uint_as_float(top);
  const float s = top > 0x7F800000u ? a : fmaxf(a * kF8PerMost, kF8Least);
  *inv = 1.0f / s;
  return s;
}

// Four values to four codes: scaled in fp32 and rounded to nearest even.  What is scaled
// is at most 448 (1 + 2^-21): s is off by two roundings and its reciprocal by one; below
// 464 the conversion gives 448.
__device__ __forceinline__ uint32_t f8_codes4(float a, float b, float c, float d, float inv) {
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
}

// 8 values of a 16-bit row from column c on, as loaded; zeros past its k values.
__device__ __forceinline__ u32x4_t f8_load8(const uint16_t *row, int c, int k) {
  if (c + 8 <= k) {
    const u32x4_a2 q = *(const u32x4_a2 *)(row + c);
    return (u32x4_t){q[0], q[1], q[2], q[3]};
  }
  u32x4_t u;
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const uint32_t lo = c + 2 * i < k ? row[c + 2 * i] : 0;
    u[i] = lo | (c + 2 * i + 1 < k ? (uint32_t)row[c + 2 * i + 1] << 16 : 0);
  }
  return u;
}

// 16 lanes hold a block, 8 values each: this lane's 8 codes, and the scale.
template <bool F16>
__device__ __forceinline__ uint2 f8_quantize8(const u32x4_t &u, float *s) {
  // the magnitudes of 16 bits order as those of 32 do
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; i++) top = max(top, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = 8; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 16));
  float inv, v[8];
  *s = f8_scale(f8_mag(f8_from16(top, F16)), &inv);
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = f8_from16((u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu, F16);
  return make_uint2(f8_codes4(v[0], v[1], v[2], v[3], inv), f8_codes4(v[4], v[5], v[6], v[7], inv));
}

// 128 products of codes, summed from zero.
__device__ __forceinline__ f32x4 f8_dot(const i32x8_t &w, const i32x8_t &x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0,
                                                          0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8_t f8_frag(const u32x4_t &a, const u32x4_t &b) {
  return (i32x8_t){(int)a[0], (int)a[1], (int)a[2], (int)a[3],
                   (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// The rows of group g, kept inside [0, rows]: offsets are the caller's.
struct F8Span {
  int begin, end;
};
__device__ __forceinline__ F8Span f8_span(const int32_t *offsets, int g, int rows) {
  if (!offsets) return {0, rows};
  const int b = min(max(offsets[g], 0), rows);
  return {b, max(b, min(max(offsets[g + 1], 0), rows))};
}

// Groups in pieces of P rows, without a scan of their lengths: the pieces of group g
// start at place offsets[g] / P + g, which is no less than where those of group g - 1
// end.  The places in between, at most one a group, and those before group 0's first
// are empty.  Returns the group of place i < rows / P + groups, and its first place.
__device__ __forceinline__ int f8_group_at(const int32_t *offsets, int groups, int rows, int P, int i,
                                           int *first) {
  int lo = 0, hi = groups;
  if (!offsets) hi = 1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (min(max(offsets[mid], 0), rows) / P + mid <= i) lo = mid; else hi = mid;
  }
  *first = offsets ? min(max(offsets[lo], 0), rows) / P + lo : 0;
  return lo;
}

}  // namespace
}  // namespace moe
