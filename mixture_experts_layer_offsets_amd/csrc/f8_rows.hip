// Quantisers of 16-bit rows for the 8-bit products: along the rows (forward and data
// gradient) and down the columns of each group's rows (weight gradient).  Both read
// the rows once and write codes and scales, 3 bytes a value: bound by memory (16384 rows of
// 7168: 59 us, 5.9 TB/s; down the columns, with 16384 of 4096 beside them, 118 us, 4.7
// TB/s).
#include <algorithm>

#include "f8_device.h"

namespace moe {

namespace {

// 16 lanes take a block, 8 values each; a workgroup takes 16 rows x kBlocks blocks,
// so that it reads kBlocks 256 bytes of each row and writes 2 KB runs of codes.  Grid
// (blocks / kBlocks, rows / 16), rows past 2^16 workgroups in turn.
constexpr int kBlocks = 4;

template <bool F16>
__global__ __launch_bounds__(256) void f8_quant_rows_kernel(const uint16_t *__restrict__ x, long stride,
                                                            int rows, int k, int ks,
                                                            uint8_t *__restrict__ codes,
                                                            float *__restrict__ scales) {
  const int tid = threadIdx.x, i = tid & 15, kb0 = blockIdx.x * kBlocks;
  for (long r0 = (long)blockIdx.y * 16; r0 < rows; r0 += 16L * gridDim.y) {
    const long r = r0 + (tid >> 4);
    const long rr = r < rows ? r : rows - 1;
    u32x4_t u[kBlocks];
#pragma unroll
    for (int b = 0; b < kBlocks; b++) u[b] = f8_load8(x + rr * stride, (kb0 + b) * kF8Block + 8 * i, k);
#pragma unroll
    for (int b = 0; b < kBlocks; b++) {
      float s;
      const uint2 c = f8_quantize8<F16>(u[b], &s);
      if (r < rows && kb0 + b < ks) {
        const size_t at = (size_t)(kb0 + b) * rows + r;
        *(uint2 *)(codes + at * kF8Block + 8 * i) = c;
        if (i == 0) scales[at] = s;
      }
    }
  }
}

// The columns of one tensor; tiles: its codes go out as packed weights lie.
struct Cols {
  const uint16_t *x;
  long stride;
  int cols, tiles;
  uint8_t *codes;
  float *scales;
};

// A workgroup takes 64 columns of one stage (128 rows of one group): the rows go
// through LDS, then a thread converts 32 values of one column, and the columns' 128
// codes leave through LDS in 16-byte chunks.  Grid (columns of a / 64 + those of b / 64,
// stages), stages past 2^16 in turn.
template <bool F16>
__global__ __launch_bounds__(256) void f8_quant_cols_kernel(Cols a, Cols b, int rows,
                                                            const int32_t *__restrict__ offsets,
                                                            int groups, long stages) {
  __shared__ u32x4_t tile[kF8Block][8];  // 128 rows x 64 values
  // a column's codes at 144 bytes a column: the 16 more put the lanes' writes on
  // different banks
  constexpr int kLine = kF8Block + 16;
  __shared__ __attribute__((aligned(16))) uint8_t lines[64 * kLine];
  __shared__ uint32_t tops[4][64];
  const int ax = (a.cols + 63) / 64;
  const bool first_of = (int)blockIdx.x < ax;
  const Cols m = first_of ? a : b;
  const uint16_t *x = m.x;
  const long stride = m.stride;
  const int cols = m.cols;
  const int tid = threadIdx.x, c0 = (first_of ? blockIdx.x : blockIdx.x - ax) * 64;
  const int cols16 = (cols + 15) & ~15;
  for (long st = blockIdx.y; st < stages; st += gridDim.y) {
    int first;
    const int g = f8_group_at(offsets, groups, rows, kF8Block, (int)st, &first);
    const F8Span sp = f8_span(offsets, g, rows);
    const int r0 = sp.begin + (int)(st - first) * kF8Block;
    if (st < first || r0 >= sp.end) continue;  // an empty place
#pragma unroll
    for (int q = 0; q < 4; q++) {
      const int at = tid + 256 * q, row = at >> 3, c8 = at & 7, c = c0 + 8 * c8;
      u32x4_t v = {0, 0, 0, 0};
      if (r0 + row < sp.end && c < cols) {
        const uint16_t *src = x + (size_t)(r0 + row) * stride + c;
        if (c + 8 <= cols) {
          const u32x4_a2 u = *(const u32x4_a2 *)src;
          v = (u32x4_t){u[0], u[1], u[2], u[3]};
        } else {
#pragma unroll
          for (int e = 0; e < 8; e++)
            if (c + e < cols) v[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
        }
      }
      tile[row][c8] = v;
    }
    __syncthreads();
    const int j = tid & 63, q = tid >> 6;
    const uint16_t *t16 = (const uint16_t *)tile;
    float v[32];
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < 32; e++) {
      v[e] = f8_from16(t16[(32 * q + e) * 64 + j], F16);
      top = max(top, f8_mag(v[e]));
    }
    tops[q][j] = top;
    __syncthreads();
    float inv;
    const float s = f8_scale(max(max(tops[0][j], tops[1][j]), max(tops[2][j], tops[3][j])), &inv);
#pragma unroll
    for (int e = 0; e < 32; e += 16)
      *(u32x4_t *)(lines + j * kLine + 32 * q + e) =
          (u32x4_t){f8_codes4(v[e], v[e + 1], v[e + 2], v[e + 3], inv),
                    f8_codes4(v[e + 4], v[e + 5], v[e + 6], v[e + 7], inv),
                    f8_codes4(v[e + 8], v[e + 9], v[e + 10], v[e + 11], inv),
                    f8_codes4(v[e + 12], v[e + 13], v[e + 14], v[e + 15], inv)};
    if (q == 0 && c0 + j < cols16) m.scales[(size_t)st * cols16 + c0 + j] = s;
    __syncthreads();
#pragma unroll
    for (int p = 0; p < 2; p++) {
      const int at = tid + 256 * p;
      int col, c;
      uint8_t *dst;
      if (m.tiles) {  // chunk by chunk in a tile's order
        col = (at >> 7) * 16 + (at & 15);
        c = ((at >> 6) & 1) * 4 + ((at >> 4) & 3);
        dst = m.codes + ((size_t)((c0 + col) >> 4) * stages + st) * kF8Tile + f8_chunk(c, col & 15);
      } else {
        col = at >> 3;
        c = at & 7;
        dst = m.codes + ((size_t)st * cols + c0 + col) * kF8Block + 16 * c;
      }
      if (c0 + col < (m.tiles ? cols16 : cols))
        *(u32x4_t *)dst = *(const u32x4_t *)(lines + col * kLine + 16 * c);
    }
    __syncthreads();
  }
}

}  // namespace

void launch_f8_quant_rows(const F8Rows &x, int rows, int k, uint8_t *codes, float *scales,
                          hipStream_t s) {
  if (rows <= 0) return;
  const int ks = (k + kF8Block - 1) / kF8Block;
  const dim3 grid((ks + kBlocks - 1) / kBlocks, std::min((rows + 15) / 16, 65535));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, x.p, x.stride, rows, k, ks, codes, scales);
  };
  x.f16 ? go(f8_quant_rows_kernel<true>) : go(f8_quant_rows_kernel<false>);
}

long f8_stages(int rows, int groups) { return rows / kF8Block + groups; }

void launch_f8_quant_cols(const F8Rows &x, const F8Rows &dy, int rows, const F8Dims &d,
                          const int32_t *offsets, uint8_t *xc, float *xs, uint8_t *yc, float *ys,
                          hipStream_t s) {
  if (rows <= 0) return;
  const long stages = f8_stages(rows, d.groups);
  const Cols a{x.p, x.stride, d.k, 0, xc, xs}, b{dy.p, dy.stride, d.n, 1, yc, ys};
  const dim3 grid((d.k + 63) / 64 + (d.n + 63) / 64, (unsigned)std::min(stages, 65535L));
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, b, rows, offsets, d.groups, stages);
  };
  d.f16 ? go(f8_quant_cols_kernel<true>) : go(f8_quant_cols_kernel<false>);
}

}  // namespace moe
