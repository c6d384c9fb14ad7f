// Packing of 8-bit weights with a scale per 128 x 128 block: ready-made codes, 16- or
// 32-bit weights, back to values, and the matrices of the transposed products (the
// layout is in f8_device.h).  Every kernel takes a 128 x 128 block a workgroup.
// Packing and packed back run once for weights that stay, quantising and turning once a
// step in training: bound by memory (6 groups of 7168 x 4096, us and TB/s: packing 70 and
// 5.0, quantising bf16 130 and 4.1 (306 with values loaded one by one), turning 69 and
// 5.1, back to fp32 values 172 and 5.1).
#include <algorithm>

#include "f8_device.h"

namespace moe {

namespace {

constexpr int kPitch = 128 + 4;  // bytes between a block's rows in LDS: columns in other banks

// The block of this workgroup: grid (blocks along k, blocks along n, groups).
struct Block {
  int kb, nb, g, rows, cols;  // rows (outputs) and columns (contraction) of it that exist
};
__device__ __forceinline__ Block block_of(const F8Dims &d) {
  const int kb = blockIdx.x, nb = blockIdx.y;
  return {kb, nb, (int)blockIdx.z, min(kF8Block, d.n - nb * kF8Block), min(kF8Block, d.k - kb * kF8Block)};
}
__device__ __forceinline__ uint8_t *block_tile(const F8Dims &d, void *packed, const Block &b, int j) {
  return (uint8_t *)packed + (((size_t)b.g * d.nt + b.nb * 8 + j) * d.ks + b.kb) * kF8Tile;
}
// the scale of tile j of the block
__device__ __forceinline__ float *tile_scale(const F8Dims &d, void *packed, const Block &b, int j) {
  return (float *)((uint8_t *)packed + d.code_bytes) + ((size_t)b.g * d.nt + b.nb * 8 + j) * d.ks + b.kb;
}
__device__ __forceinline__ void put_scale(const F8Dims &d, void *packed, const Block &b, float s) {
  const int j = threadIdx.x;
  if (j < 8 && b.nb * 8 + j < d.nt) *tile_scale(d, packed, b, j) = s;
}

// The block's codes in LDS, [output][kPitch], to its tiles.
__device__ __forceinline__ void put_tiles(const F8Dims &d, void *packed, const Block &b,
                                          const uint8_t *lds) {
  for (int q = threadIdx.x; q < 1024; q += 256) {  // chunk by chunk, in a tile's order
    const int j = q >> 7, c = ((q >> 6) & 1) * 4 + ((q >> 4) & 3), n = q & 15;
    if (b.nb * 8 + j >= d.nt) break;
    const uint32_t *src = (const uint32_t *)(lds + (16 * j + n) * kPitch + 16 * c);
    *(u32x4_t *)(block_tile(d, packed, b, j) + f8_chunk(c, n)) = (u32x4_t){src[0], src[1], src[2], src[3]};
  }
}
// ... and from its tiles.
__device__ __forceinline__ void get_tiles(const F8Dims &d, const void *packed, const Block &b,
                                          uint8_t *lds) {
  for (int q = threadIdx.x; q < 1024; q += 256) {
    const int j = q >> 7, c = ((q >> 6) & 1) * 4 + ((q >> 4) & 3), n = q & 15;
    u32x4_t v = {0, 0, 0, 0};
    if (b.nb * 8 + j < d.nt) v = *(const u32x4_t *)(block_tile(d, (void *)packed, b, j) + f8_chunk(c, n));
    uint32_t *dst = (uint32_t *)(lds + (16 * j + n) * kPitch + 16 * c);
    dst[0] = v[0]; dst[1] = v[1]; dst[2] = v[2]; dst[3] = v[3];
  }
}

typedef unsigned int u32x4_a1 __attribute__((ext_vector_type(4), aligned(1)));

// A thread moves 16-byte chunks, in a tile's order.
__global__ __launch_bounds__(256) void f8_pack_kernel(F8Dims d, const uint8_t *__restrict__ codes,
                                                      const float *__restrict__ scales, void *packed) {
  const Block b = block_of(d);
  const uint8_t *src = codes + ((size_t)b.g * d.n + b.nb * kF8Block) * d.k + b.kb * kF8Block;
  u32x4_t v[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int q = threadIdx.x + 256 * i, r = (q >> 7) * 16 + (q & 15);
    const int at = 16 * (((q >> 6) & 1) * 4 + ((q >> 4) & 3));
    const uint8_t *p = src + (size_t)r * d.k + at;
    v[i] = (u32x4_t){0, 0, 0, 0};
    if (r < b.rows && at + 16 <= b.cols) {
      const u32x4_a1 u = *(const u32x4_a1 *)p;
      v[i] = (u32x4_t){u[0], u[1], u[2], u[3]};
    } else if (r < b.rows) {
#pragma unroll
      for (int e = 0; e < 16; e++)
        if (at + e < b.cols) v[i][e >> 2] |= (uint32_t)p[e] << (8 * (e & 3));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int q = threadIdx.x + 256 * i, j = q >> 7;
    if (b.nb * 8 + j < d.nt) ((u32x4_t *)block_tile(d, packed, b, j))[q & 127] = v[i];
  }
  put_scale(d, packed, b, scales[((size_t)b.g * d.nb + b.nb) * d.ks + b.kb]);
}

// w [group][k][n]: a thread takes 8 contraction values of 8 outputs, 16 or 32 bytes of
// each row.
template <class T>
__global__ __launch_bounds__(256) void f8_quantize_kernel(F8Dims d, const T *__restrict__ w, int f16,
                                                          void *packed) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kF8Block * kPitch];
  __shared__ uint32_t tops[4];
  const Block b = block_of(d);
  const int n0 = (threadIdx.x & 15) * 8, k0 = (threadIdx.x >> 4) * 8;
  const T *src = w + ((size_t)b.g * d.k + b.kb * kF8Block) * d.n + b.nb * kF8Block;
  T raw[8][8];
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const T *p = src + (size_t)(k0 + i) * d.n;
    if (k0 + i < b.cols && n0 + 8 <= b.rows) {
      if constexpr (sizeof(T) == 4) {
        __builtin_memcpy(raw[i], p + n0, 32);
      } else {
        const u32x4_t u = f8_load8(p, n0, b.rows);
        __builtin_memcpy(raw[i], &u, 16);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; e++) raw[i][e] = k0 + i < b.cols && n0 + e < b.rows ? p[n0 + e] : (T)0;
    }
  }
  auto value = [&](int i, int e) {
    if constexpr (sizeof(T) == 4) return raw[i][e];
    else return f8_from16(raw[i][e], f16);
  };
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; i++)
#pragma unroll
    for (int e = 0; e < 8; e++) top = max(top, f8_mag(value(i, e)));
#pragma unroll
  for (int o = 32; o; o >>= 1) top = max(top, (uint32_t)__shfl_xor((int)top, o, 64));
  if ((threadIdx.x & 63) == 0) tops[threadIdx.x >> 6] = top;
  __syncthreads();
  float inv;
  const float s = f8_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])), &inv);
#pragma unroll
  for (int e = 0; e < 8; e++)
#pragma unroll
    for (int i = 0; i < 8; i += 4)
      *(uint32_t *)(lds + (n0 + e) * kPitch + k0 + i) =
          f8_codes4(value(i, e), value(i + 1, e), value(i + 2, e), value(i + 3, e), inv);
  __syncthreads();
  put_tiles(d, packed, b, lds);
  put_scale(d, packed, b, s);
}

__global__ __launch_bounds__(256) void f8_unpack_kernel(F8Dims d, const void *__restrict__ packed,
                                                        float *__restrict__ w) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kF8Block * kPitch];
  const Block b = block_of(d);
  get_tiles(d, packed, b, lds);
  __syncthreads();
  const float s = *tile_scale(d, (void *)packed, b, 0);
  float *dst = w + ((size_t)b.g * d.k + b.kb * kF8Block) * d.n + b.nb * kF8Block;
  for (int q = threadIdx.x; q < kF8Block * kF8Block; q += 256) {
    const int c = q >> 7, n = q & 127;
    if (n < b.rows && c < b.cols)
      dst[(size_t)c * d.n + n] = s * __builtin_amdgcn_cvt_f32_fp8(lds[n * kPitch + c], 0);
  }
}

// The block's transpose is block (kb, nb) of the matrices [group][n][k] of x*W^T:
// t are their dims, n and k exchanged.
__global__ __launch_bounds__(256) void f8_transpose_kernel(F8Dims d, F8Dims t,
                                                           const void *__restrict__ packed,
                                                           void *__restrict__ turned) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kF8Block * kPitch], out[kF8Block * kPitch];
  const Block b = block_of(d);
  get_tiles(d, packed, b, lds);
  __syncthreads();
  for (int q = threadIdx.x; q < kF8Block * 32; q += 256) {  // 4 outputs of a column
    const int c = q & 127, n = (q >> 7) * 4;
    uint32_t v = 0;
#pragma unroll
    for (int i = 0; i < 4; i++) v |= (uint32_t)lds[(n + i) * kPitch + c] << (8 * i);
    *(uint32_t *)(out + c * kPitch + n) = v;
  }
  __syncthreads();
  const Block to{b.nb, b.kb, b.g, b.cols, b.rows};
  put_tiles(t, turned, to, out);
  put_scale(t, turned, to, *tile_scale(d, (void *)packed, b, 0));
}

dim3 blocks(const F8Dims &d) { return dim3(d.ks, d.nb, d.groups); }

}  // namespace

void launch_f8_pack(const F8Dims &d, const uint8_t *codes, const float *scales, void *packed,
                    hipStream_t s) {
  hipLaunchKernelGGL(f8_pack_kernel, blocks(d), dim3(256), 0, s, d, codes, scales, packed);
}

void launch_f8_quantize(const F8Dims &d, const void *w, int type, void *packed, hipStream_t s) {
  if (type == 2)
    hipLaunchKernelGGL(f8_quantize_kernel<float>, blocks(d), dim3(256), 0, s, d, (const float *)w, 0,
                       packed);
  else
    hipLaunchKernelGGL(f8_quantize_kernel<uint16_t>, blocks(d), dim3(256), 0, s, d,
                       (const uint16_t *)w, type, packed);
}

void launch_f8_unpack(const F8Dims &d, const void *packed, float *w, hipStream_t s) {
  hipLaunchKernelGGL(f8_unpack_kernel, blocks(d), dim3(256), 0, s, d, packed, w);
}

void launch_f8_transpose(const F8Dims &d, const void *packed, void *turned, hipStream_t s) {
  F8Dims t = d;
  t.n = d.k; t.k = d.n;
  t.nt = (t.n + 15) / 16; t.nb = d.ks; t.ks = d.nb;
  t.code_bytes = (size_t)t.groups * t.nt * t.ks * kF8Tile;
  hipLaunchKernelGGL(f8_transpose_kernel, blocks(d), dim3(256), 0, s, d, t, packed, turned);
}

}  // namespace moe
