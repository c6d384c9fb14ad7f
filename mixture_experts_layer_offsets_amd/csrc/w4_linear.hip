// Products of a few dense or grouped rows with 4-bit weights (w4_device.h).
#include <algorithm>

#include "w4_device.h"

namespace moe {

namespace {

// The rows of group g, kept inside [0, rows]: offsets are the caller's.
struct Span {
  int begin, end;
};
__device__ __forceinline__ Span span_of(const int32_t *offsets, int g, int rows) {
  if (!offsets) return {0, rows};
  return {min(max(offsets[g], 0), rows), min(max(offsets[g + 1], 0), rows)};
}

// 16 rows a pass from memory; the waves of a workgroup split the contraction of
// one tile.  Grid (output tiles, groups).
template <class F, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void w4_linear_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ float red[WAVES * 256];
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Span sp = span_of(offsets, g, rows);
  const W4Row<F> mm[1] = {W4Row<F>(m, (size_t)g * m.nt + blockIdx.x)};
  for (int r0 = sp.begin; r0 < sp.end; r0 += 16) {
    const int nr = min(16, sp.end - r0);
    const RowPtr xr[1] = {{x + (r0 + min(lane & 15, nr - 1)) * xstride}};
    f32x4 acc[1][1];
    zero_acc(acc);
    w4_stream<F, 4>(mm, m.f16, xr, m.k, m.ks * wave / WAVES, m.ks * (wave + 1) / WAVES, acc);
    w4_join<WAVES>(acc, red);
    const int row = 4 * ((tid & 63) >> 4) + (tid >> 6), n = 16 * blockIdx.x + (tid & 15);
    if (tid < 256 && row < nr && n < m.n) out[(r0 + row) * ostride + n] = to_bf16(red[tid]);
    __syncthreads();
  }
}

// Many rows, 16 NB a pass: a workgroup takes 2 kBlockWaves tiles.
template <class F, int NB>
__global__ __launch_bounds__(64 * kBlockWaves * kBlockGroups, 2) void w4_linear_rows_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ __attribute__((aligned(16))) char xs[w4_block_lds<NB>()];
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 63, gt = tid % (64 * kBlockWaves);
  const Span sp = span_of(offsets, g, rows);
  const int j = 2 * (blockIdx.x * kBlockWaves + __builtin_amdgcn_readfirstlane(gt >> 6));
  const size_t base = (size_t)g * m.nt;
  const W4Row<F> mm[2] = {W4Row<F>(m, base + min(j, m.nt - 1)),
                          W4Row<F>(m, base + min(j + 1, m.nt - 1))};
  for (int r0 = sp.begin; r0 < sp.end; r0 += 16 * NB) {
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = x + min(r0 + 16 * p + gt / 16, sp.end - 1) * xstride + 8 * (gt % 16);
    f32x4 acc[2][NB];
    zero_acc(acc);
    w4_block<F>(mm, m.f16, xr, m.k, m.ks, xs, acc);
    if (w4_block_join(acc, xs))
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int p = 0; p < NB; p++)
#pragma unroll
          for (int v = 0; v < 4; v++) {
            const int row = r0 + 16 * p + 4 * (lane >> 4) + v, n = 16 * (j + t) + (lane & 15);
            if (row < sp.end && n < m.n) out[row * ostride + n] = to_bf16(acc[t][p][v]);
          }
    lds_barrier();
  }
}

}  // namespace

void launch_w4_linear(const W4Dims &d, int rows, const uint16_t *x, long xstride,
                      const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                      hipStream_t s) {
  if (rows <= 0) return;
  const W4Mat m = w4_view(d, packed);
  // the rows of a group, if they were spread evenly
  const int avg = (rows + d.groups - 1) / d.groups;
  with_format(d, [&](auto f) {
    using F = decltype(f);
    auto go = [&](auto kernel, int tiles, int waves) {
      hipLaunchKernelGGL(kernel, dim3((d.nt + tiles - 1) / tiles, d.groups), dim3(waves * 64), 0, s,
                         m, x, xstride, offsets, rows, out, ostride);
    };
    constexpr int kBlock = kBlockWaves * kBlockGroups;
    if (avg > 32) go(w4_linear_rows_kernel<F, kLongBlocks<F>>, 2 * kBlockWaves, kBlock);
    else if (avg > 16) go(w4_linear_rows_kernel<F, 2>, 2 * kBlockWaves, kBlock);
    else if ((long)d.nt * d.groups < 512) go(w4_linear_kernel<F, 16>, 1, 16);
    else go(w4_linear_kernel<F, 4>, 1, 4);
  });
}

}  // namespace moe
