// Quantisers of 16-bit rows for the 8-bit products: along the rows (forward and data
// gradient) and down the columns of each group's rows (weight gradient; a small one is
// computed in the same launch).  Both read
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

// 128 rows x 64 columns of a tensor in LDS, and their codes by T threads, column by column,
// at 144 bytes a column (the 16 more put the lanes' writes on different banks).
constexpr int kLine = kF8Block + 16;
template <int T>
struct ColsLds {
  static constexpr int N = kF8Block * 64 / T;  // values of a thread
  u32x4_t tile[kF8Block][8];
  __attribute__((aligned(16))) uint8_t lines[64 * kLine];
  uint32_t tops[T / 64][64];
};

// Rows r0 .. of those before `end`, columns c0 .. + 63: 8 values a load, zeros outside.
template <int T>
__device__ __forceinline__ void cols_load(const Cols &m, int r0, int end, int c0, u32x4_t (&v)[1024 / T]) {
#pragma unroll
  for (int q = 0; q < 1024 / T; q++) {
    const int at = threadIdx.x + T * q, row = at >> 3, c = c0 + 8 * (at & 7);
    v[q] = (u32x4_t){0, 0, 0, 0};
    if (r0 + row < end && c < m.cols) v[q] = f8_load8(m.x + (size_t)(r0 + row) * m.stride, c, m.cols);
  }
}
template <int T>
__device__ __forceinline__ void cols_put(ColsLds<T> &l, const u32x4_t (&v)[1024 / T]) {
#pragma unroll
  for (int q = 0; q < 1024 / T; q++) {
    const int at = threadIdx.x + T * q;
    l.tile[at >> 3][at & 7] = v[q];
  }
}
// A thread takes N values of column threadIdx.x % 64, the piece that its wave names.
template <bool F16, int T, int N>
__device__ __forceinline__ void cols_top(ColsLds<T> &l, float (&v)[N]) {
  const int j = threadIdx.x & 63, q = threadIdx.x >> 6;
  const uint16_t *t16 = (const uint16_t *)l.tile;
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; e++) {
    v[e] = f8_from16(t16[(N * q + e) * 64 + j], F16);
    top = max(top, f8_mag(v[e]));
  }
  l.tops[q][j] = top;
}
// ... and puts their codes; returns the column's scale.
template <int T, int N>
__device__ __forceinline__ float cols_codes(ColsLds<T> &l, const float (&v)[N]) {
  const int j = threadIdx.x & 63, q = threadIdx.x >> 6;
  uint32_t top = l.tops[0][j];
#pragma unroll
  for (int w = 1; w < T / 64; w++) top = max(top, l.tops[w][j]);
  float inv;
  const float s = f8_scale(top, &inv);
#pragma unroll
  for (int e = 0; e < N; e += 16)
    *(u32x4_t *)(l.lines + j * kLine + N * q + e) =
        (u32x4_t){f8_codes4(v[e], v[e + 1], v[e + 2], v[e + 3], inv),
                  f8_codes4(v[e + 4], v[e + 5], v[e + 6], v[e + 7], inv),
                  f8_codes4(v[e + 8], v[e + 9], v[e + 10], v[e + 11], inv),
                  f8_codes4(v[e + 12], v[e + 13], v[e + 14], v[e + 15], inv)};
  return s;
}

// A workgroup takes 64 columns of one stage (128 rows of one group), which leave in
// 16-byte chunks.  Grid (columns of a / 64 + those of b / 64, stages).
template <bool F16>
__global__ __launch_bounds__(256) void f8_quant_cols_kernel(Cols a, Cols b, int rows,
                                                            const int32_t *__restrict__ offsets,
                                                            int groups, int stages) {
  __shared__ ColsLds<256> lds;
  const int ax = (a.cols + 63) / 64;
  const bool first_of = (int)blockIdx.x < ax;
  const Cols m = first_of ? a : b;
  const int tid = threadIdx.x, c0 = (first_of ? blockIdx.x : blockIdx.x - ax) * 64;
  const int cols16 = (m.cols + 15) & ~15, st = blockIdx.y;
  int first;
  const int g = f8_group_at(offsets, groups, rows, kF8Block, st, &first);
  const F8Span sp = f8_span(offsets, g, rows);
  const int r0 = sp.begin + (st - first) * kF8Block;
  if (st < first || r0 >= sp.end) return;  // an empty place
  u32x4_t u[4];
  cols_load<256>(m, r0, sp.end, c0, u);
  cols_put(lds, u);
  __syncthreads();
  float v[ColsLds<256>::N];
  cols_top<F16>(lds, v);
  __syncthreads();
  const float s = cols_codes(lds, v);
  if (tid < 64 && c0 + tid < cols16) m.scales[(size_t)st * cols16 + c0 + tid] = s;
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
      dst = m.codes + ((size_t)st * m.cols + c0 + col) * kF8Block + 16 * c;
    }
    if (c0 + col < (m.tiles ? cols16 : m.cols))
      *(u32x4_t *)dst = *(const u32x4_t *)(lds.lines + col * kLine + 16 * c);
  }
}

// A small weight gradient in one launch: a workgroup takes 64 x 64 of dw and quantises its
// columns of x and dy stage by stage, the next stage's loads on their way.  Eight waves: one
// holds 16 rows x 32 columns of dw (four waves: 12.2 us for 777 rows in 5 uneven groups of
// 500 x 333, eight 9.1).  Grid (tiles, groups).
constexpr int kFewThreads = 512;

template <bool F16>
__global__ __launch_bounds__(kFewThreads) void f8_wgrad_few_kernel(Cols x, Cols y, int rows,
                                                           const int32_t *__restrict__ offsets,
                                                           uint16_t *__restrict__ dw) {
  constexpr int T = kFewThreads, N = ColsLds<T>::N;
  __shared__ ColsLds<T> xl, yl;
  __shared__ float xs[64], ys[64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, h = lane >> 4;
  const int r16 = 16 * (wave & 3), c32 = 32 * (wave >> 2);  // of the wave, in the tile
  const int nN = (y.cols + 63) / 64, m0 = blockIdx.x / nN * 64, n0 = blockIdx.x % nN * 64;
  const F8Span sp = f8_span(offsets, blockIdx.y, rows);
  f32x4 acc[2];
#pragma unroll
  for (int i = 0; i < 2; i++) acc[i] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  u32x4_t u[1024 / T], w[1024 / T];
  cols_load<T>(x, sp.begin, sp.end, m0, u);
  cols_load<T>(y, sp.begin, sp.end, n0, w);
  for (int r0 = sp.begin; r0 < sp.end; r0 += kF8Block) {
    cols_put(xl, u);
    cols_put(yl, w);
    __syncthreads();
    cols_load<T>(x, r0 + kF8Block, sp.end, m0, u);
    cols_load<T>(y, r0 + kF8Block, sp.end, n0, w);
    float v[N], t[N];
    cols_top<F16>(xl, v);
    cols_top<F16>(yl, t);
    __syncthreads();
    const float sx = cols_codes(xl, v), sy = cols_codes(yl, t);
    if (tid < 64) xs[tid] = sx, ys[tid] = sy;
    __syncthreads();
    auto frag = [&](const uint8_t *lines, int c) {
      const uint8_t *p = lines + (c + l16) * kLine + 16 * h;
      return f8_frag(*(const u32x4_t *)p, *(const u32x4_t *)(p + 64));
    };
    const i32x8_t xf = frag(xl.lines, r16);
    const float s = xs[r16 + l16];
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const f32x4 d = f8_dot(frag(yl.lines, c32 + 16 * i), xf);
#pragma unroll
      for (int e = 0; e < 4; e++) acc[i][e] = fmaf(s * ys[c32 + 16 * i + 4 * h + e], d[e], acc[i][e]);
    }
  }
  const int r = m0 + r16 + l16;
  if (r >= x.cols) return;
  uint16_t *to = dw + ((size_t)blockIdx.y * x.cols + r) * y.cols;
#pragma unroll
  for (int i = 0; i < 2; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const int c = n0 + c32 + 16 * i + 4 * h + e;
      if (c < y.cols) to[c] = f8_to16(acc[i][e], F16);
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
  const int stages = (int)f8_stages(rows, d.groups);
  const Cols a{x.p, x.stride, d.k, 0, xc, xs}, b{dy.p, dy.stride, d.n, 1, yc, ys};
  const dim3 grid((d.k + 63) / 64 + (d.n + 63) / 64, stages);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, b, rows, offsets, d.groups, stages);
  };
  d.f16 ? go(f8_quant_cols_kernel<true>) : go(f8_quant_cols_kernel<false>);
}

// Against two launches: as long as its workgroups, two a CU, take few stages, which are 1.5
// to 2 us each here (1 there).  us here and there: 64 x 64 of 100 rows 6.4 and 11.6; 256 x
// 256 of 300 9.0 and 12.7, of 600 12.2 and 15.1, of 1000 17.3 and 17.2; 1400 x 1400 of 300
// (484 workgroups) 13.5 and 14.6, 2048 x 2048 of 128 (1024) 14.0 and 12.8.  In even groups,
// and in groups that fall off as 1 / g: 5 of 500 x 333, 777 rows 8.2 and 14.0, 12.1 and 14.8;
// 4 of 512 x 512, 2000 rows 13.4 and 16.3, 18.5 and 19.0.
bool f8_wgrad_few(const F8Dims &d, int rows) {
  const long stages = ((long)rows + (long)d.groups * kF8Block - 1) / ((long)d.groups * kF8Block);
  return (long)((d.k + 63) / 64) * ((d.n + 63) / 64) * d.groups <= 512 &&
         stages <= (d.groups == 1 ? 6 : 4);
}

void launch_f8_wgrad_few(const F8Rows &x, const F8Rows &dy, int rows, const F8Dims &d,
                         const int32_t *offsets, uint16_t *dw, hipStream_t s) {
  const Cols a{x.p, x.stride, d.k, 0, nullptr, nullptr}, b{dy.p, dy.stride, d.n, 0, nullptr, nullptr};
  const dim3 grid((unsigned)(((d.k + 63) / 64) * ((d.n + 63) / 64)), d.groups);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kFewThreads), 0, s, a, b, rows, offsets, dw);
  };
  d.f16 ? go(f8_wgrad_few_kernel<true>) : go(f8_wgrad_few_kernel<false>);
}

}  // namespace moe
