// Products of a few dense or grouped rows with 4-bit weights (w4_device.h).
#include <algorithm>

#include "w4_device.h"

namespace moe {

namespace {

// Grid (output tiles, groups).  The waves of a workgroup split the contraction
// of one tile; a group's rows go through in passes of 16 NB.
template <class F, int NB, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void w4_linear_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ float red[WAVES * NB * 256];
  const int g = blockIdx.y, t0 = blockIdx.x;
  // offsets are the caller's: kept inside [0, rows]
  const int rb = offsets ? min(max(offsets[g], 0), rows) : 0;
  const int re = offsets ? min(max(offsets[g + 1], 0), rows) : rows;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const W4Row<F> mm[1] = {W4Row<F>(m, (size_t)g * m.nt + t0)};
  for (int r0 = rb; r0 < re; r0 += 16 * NB) {
    const int nr = min(16 * NB, re - r0);
    RowPtr xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p].p = x + (r0 + min(16 * p + (lane & 15), nr - 1)) * xstride;
    f32x4 acc[1][NB];
    zero_acc(acc);
    w4_stream<F, (NB == 1 ? 4 : (NB == 2 ? 2 : 1))>(mm, m.f16, xr, m.k, m.ks * wave / WAVES, m.ks * (wave + 1) / WAVES, acc);
    w4_join<WAVES>(acc, red);
    for (int i = threadIdx.x; i < NB * 256; i += WAVES * 64) {
      const int l = i & 63, v = (i >> 6) & 3;
      const int row = 16 * (i >> 8) + 4 * (l >> 4) + v, n = 16 * t0 + (l & 15);
      if (row < nr && n < m.n) out[(r0 + row) * ostride + n] = to_bf16(red[i]);
    }
    __syncthreads();
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
    auto go = [&](auto kernel, int waves) {
      hipLaunchKernelGGL(kernel, dim3(d.nt, d.groups), dim3(waves * 64), 0, s, m, x, xstride,
                         offsets, rows, out, ostride);
    };
    const bool few = (long)d.nt * d.groups < 512;
    if (avg <= 16 && few) go(w4_linear_kernel<F, 1, 16>, 16);
    else if (avg <= 16) go(w4_linear_kernel<F, 1, 4>, 4);
    else if (avg <= 32) go(w4_linear_kernel<F, 2, 8>, 8);
    else go(w4_linear_kernel<F, 4, 8>, 8);
  });
}

}  // namespace moe
