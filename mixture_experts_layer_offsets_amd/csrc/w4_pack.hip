// Packing of 4-bit weights: ready-made codes, bf16 weights, and back to values
// (the layout is in w4_device.h).
#include <algorithm>

#include "mx_device.h"
#include "w4_device.h"

namespace moe {

namespace {

// One thread per dword of codes: tile, lane l, dword i hold output
// 16 tile + l % 16 at k = 128 step + 32 i + 8 (l / 16).

// Bit at which value q's code starts in its dword (INT4: the halves' nibbles
// are 3 bits up, where bf16 16.0 takes them; the last one wraps around).
__device__ __forceinline__ int code_bit(int fmt, int q) {
  return fmt == kW4Mx ? 4 * q : (3 + 4 * (q >> 1) + 16 * (q & 1)) & 31;
}
__device__ __forceinline__ uint32_t place_code(uint32_t c, int bit) {
  return bit ? (c << bit) | (c >> (32 - bit)) : c;
}
__device__ __forceinline__ uint32_t take_code(uint32_t d, int bit) {
  return (bit ? (d >> bit) | (d << (32 - bit)) : d) & 15;
}

__global__ __launch_bounds__(256) void w4_pack_kernel(W4Dims d, const uint8_t *__restrict__ codes,
                                                      const void *__restrict__ scales,
                                                      const uint8_t *__restrict__ zeros,
                                                      uint8_t *__restrict__ packed) {
  // a tile a workgroup
  const size_t tile = (size_t)blockIdx.y * gridDim.x + blockIdx.x;
  if (tile >= (size_t)d.groups * d.nt * d.ks) return;
  const size_t id = tile * 256 + threadIdx.x;
  const int i = threadIdx.x & 3, l = threadIdx.x >> 2;
  const int step = (int)(tile % d.ks);
  const size_t gt = tile / d.ks;
  const int n = (int)(gt % d.nt) * 16 + (l & 15);
  const size_t g = gt / d.nt;
  const int k0 = step * 128 + 32 * i + 8 * (l >> 4);
  const size_t row = g * d.n + n;
  uint32_t v = 0;
  if (n < d.n && k0 < d.k) {
    const uint8_t *src = codes + row * (d.k / 2) + k0 / 2;
    for (int q = 0; q < 8; q++)
      v |= place_code((src[q >> 1] >> (4 * (q & 1))) & 15, code_bit(d.fmt, q));
  }
  ((uint32_t *)packed)[id] = v;
  // scales: the lanes l < 16 of dword i own scale i of their output
  if (l >= 16 || i >= d.spg) return;
  const int kg = (step * 128) / d.group + i;
  const bool in = n < d.n && kg < d.k / d.group;
  const size_t from = row * (d.k / d.group) + kg, to = (tile * 16 + l) * d.spg + i;
  uint8_t *ps = packed + d.code_bytes;
  if (d.fmt == kW4Mx) {
    ps[to] = in ? ((const uint8_t *)scales)[from] : 127;
  } else {
    ((uint16_t *)ps)[to] = in ? ((const uint16_t *)scales)[from] : 0;
    if (d.zeros) (ps + d.scale_bytes)[to] = in ? zeros[from] & 15 : 0;
  }
}

// E2M1 code of a value scaled by 2^-s: nearest, ties to the even code,
// saturating; the sign bit is set exactly when v < 0.
__device__ __forceinline__ uint32_t e2m1_code(float v, int s) {
  const float a = fminf(fabsf(ldexpf(v, -s)), 6.0f);
  // quantum 0.5 up to 2, 1 up to 4, 2 up to 6
  uint32_t c;
  if (a <= 2.0f) c = (uint32_t)rintf(a * 2.0f);
  else if (a <= 4.0f) c = 2u + (uint32_t)rintf(a);
  else c = 4u + (uint32_t)rintf(a * 0.5f);
  return c | (v < 0.0f ? 8u : 0u);
}

// One thread per (group of the contraction, output): reads its group of w
// [k][n] (neighbouring threads: neighbouring outputs), writes codes and scale.
__global__ __launch_bounds__(256) void w4_quantize_kernel(W4Dims d, const uint16_t *__restrict__ w,
                                                          uint8_t *__restrict__ packed) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int kg = blockIdx.y;
  const size_t g = blockIdx.z;
  if (n >= d.nt * 16) return;
  const bool in = n < d.n && kg < d.k / d.group;
  const uint16_t *src = w + (g * d.k + (size_t)kg * d.group) * d.n + n;
  float lo = 0.0f, hi = 0.0f;
  for (int q = 0; in && q < d.group; q++) {
    const float v = bf16_to_f32(src[(size_t)q * d.n]);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const int step = kg * d.group / 128, slot = kg % d.spg;
  const size_t tile = (g * d.nt + n / 16) * d.ks + step;
  const size_t to = (tile * 16 + (n & 15)) * d.spg + slot;
  uint8_t *ps = packed + d.code_bytes;
  int sx = 0, z = 8;
  float s = 0.0f;
  if (d.fmt == kW4Mx) {
    const float amax = fmaxf(-lo, hi);
    sx = amax > 0.0f ? min(max(floor_log2(amax) - 2, -127), 127) : -127;
    ps[to] = in ? (uint8_t)(sx + 127) : 127;
  } else {
    const float span = hi - lo;  // past fp32's range only where both ends are near bf16's
    float step = fmaxf(-lo, hi) / 7.0f;
    if (d.zeros) step = isinf(span) ? hi / 15.0f - lo / 15.0f : span / 15.0f;
    uint32_t bits = d.f16_scales ? __builtin_bit_cast(uint16_t, (_Float16)step)
                                 : __builtin_bit_cast(uint16_t, (__bf16)step);
    s = scale_value(bits, d.f16_scales ? ~0u : 0u);
    float for_zero = s;
    // a step past fp16's largest value is held there, and the codes saturate (an
    // infinite weight's step stays infinite)
    if (isinf(s) && !isinf(step)) {
      bits = 0x7BFF;
      s = scale_value(bits, ~0u);
      for_zero = step;
    }
    ((uint16_t *)ps)[to] = in ? bits : 0;
    if (d.zeros) {
      z = s > 0.0f ? (int)fminf(fmaxf(rintf(-lo / for_zero), 0.0f), 15.0f) : 0;
      (ps + d.scale_bytes)[to] = in ? z : 0;
    }
  }
  for (int q0 = 0; q0 < d.group; q0 += 8) {
    uint32_t v = 0;
    for (int q = 0; in && q < 8; q++) {
      const float f = bf16_to_f32(src[(size_t)(q0 + q) * d.n]);
      uint32_t c;
      if (d.fmt == kW4Mx) c = e2m1_code(f, sx);
      else {
        c = s > 0.0f ? (uint32_t)fminf(fmaxf(rintf(f / s) + (float)z, 0.0f), 15.0f) : (uint32_t)z;
        // rounding outwards next to bf16's largest value: one step back into fp32's range
        if (isinf(s * (float)((int)c - z))) c += (int)c < z ? 1 : -1;
      }
      v |= place_code(c, code_bit(d.fmt, q));
    }
    const int k0 = kg * d.group + q0, in128 = k0 & 127;
    const int l = ((in128 & 31) >> 3) * 16 + (n & 15), i = in128 >> 5;
    ((uint32_t *)packed)[(tile * 64 + l) * 4 + i] = v;
  }
}

__global__ __launch_bounds__(256) void w4_unpack_kernel(W4Dims d, const uint8_t *__restrict__ packed,
                                                        float *__restrict__ w) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const size_t g = blockIdx.z;
  if (n >= d.n) return;
  for (int k = blockIdx.y; k < d.k; k += gridDim.y) {
    const size_t tile = (g * d.nt + n / 16) * d.ks + k / 128;
    const int in128 = k & 127, l = ((in128 & 31) >> 3) * 16 + (n & 15), i = in128 >> 5;
    const uint32_t dw = ((const uint32_t *)packed)[(tile * 64 + l) * 4 + i];
    const uint32_t c = take_code(dw, code_bit(d.fmt, k & 7));
    const size_t at = (tile * 16 + (n & 15)) * d.spg + in128 / d.group;
    const uint8_t *ps = packed + d.code_bytes;
    float v;
    if (d.fmt == kW4Mx) {
      const int e = (c >> 1) & 3, man = c & 1;
      const float mag = e ? ldexpf(1.0f + 0.5f * man, e - 1) : 0.5f * man;
      v = ps[at] == 255 ? __uint_as_float(0x7FC00000u)  // E8M0's NaN, as the products have it
                        : ldexpf(c & 8 ? -mag : mag, (int)ps[at] - 127);
    } else {
      const int z = d.zeros ? (ps + d.scale_bytes)[at] : 8;
      v = scale_value(((const uint16_t *)ps)[at], d.f16_scales ? ~0u : 0u) * (float)((int)c - z);
    }
    w[(g * d.k + k) * d.n + n] = v;
  }
}

}  // namespace

void launch_w4_pack(const W4Dims &d, const uint8_t *codes, const void *scales,
                    const uint8_t *zeros, void *packed, hipStream_t s) {
  const size_t n = (size_t)d.groups * d.nt * d.ks, gx = std::min<size_t>(n, 1 << 20);
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)gx, (unsigned)((n + gx - 1) / gx)), dim3(256), 0,
                     s, d, codes, scales, zeros, (uint8_t *)packed);
}

void launch_w4_quantize(const W4Dims &d, const uint16_t *w, void *packed, hipStream_t s) {
  hipLaunchKernelGGL(w4_quantize_kernel, dim3((d.nt * 16 + 255) / 256, d.ks * 128 / d.group, d.groups),
                     dim3(256), 0, s, d, w, (uint8_t *)packed);
}

void launch_w4_unpack(const W4Dims &d, const void *packed, float *w, hipStream_t s) {
  hipLaunchKernelGGL(w4_unpack_kernel, dim3((d.n + 255) / 256, std::min(d.k, 4096), d.groups),
                     dim3(256), 0, s, d, (const uint8_t *)packed, w);
}

}  // namespace moe
