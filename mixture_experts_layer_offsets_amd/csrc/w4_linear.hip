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
// one tile.  Grid (output tiles, groups, passes that run side by side).
template <class F, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void w4_linear_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ float red[WAVES * 256];
  const int g = blockIdx.y, tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Span sp = span_of(offsets, g, rows);
  const W4Row<F> mm[1] = {W4Row<F>(m, (size_t)g * m.nt + blockIdx.x)};
  for (int r0 = sp.begin + 16 * blockIdx.z; r0 < sp.end; r0 += 16 * gridDim.z) {
    const int nr = min(16, sp.end - r0);
    const RowPtr xr = {x + (r0 + min(w4_row_of_lane(), nr - 1)) * xstride};
    f32x4 acc[1][1];
    zero_acc(acc);
    w4_stream<F, 4>(mm, m.f16, xr, nr, m.k, m.ks * wave / WAVES, m.ks * (wave + 1) / WAVES, acc);
    w4_join<WAVES>(acc, red, nr);
    const int row = w4_row_of(tid), n = 16 * blockIdx.x + (tid & 15);
    if (tid < 256 && row < nr && n < m.n) out[(r0 + row) * ostride + n] = to_bf16(red[tid]);
    __syncthreads();
  }
}

// Many rows, 16 NB a pass: a workgroup takes NTW kBlockWaves tiles.  Grid (output
// tiles, groups, passes that run side by side).
template <class F, int NTW, int NB>
__global__ __launch_bounds__(64 * kBlockWaves * kBlockGroups, 2) void w4_linear_rows_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ __attribute__((aligned(16))) char xs[w4_block_lds<NB>()];
  const int g = blockIdx.y, tid = threadIdx.x, lane = tid & 63, gt = tid % (64 * kBlockWaves);
  const Span sp = span_of(offsets, g, rows);
  const int j = NTW * (blockIdx.x * kBlockWaves + __builtin_amdgcn_readfirstlane(gt >> 6));
  W4Row<F> mm[NTW];
#pragma unroll
  for (int t = 0; t < NTW; t++) mm[t] = W4Row<F>(m, (size_t)g * m.nt + min(j + t, m.nt - 1));
  for (int r0 = sp.begin + 16 * NB * blockIdx.z; r0 < sp.end; r0 += 16 * NB * gridDim.z) {
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = x + min(r0 + 16 * p + gt / 16, sp.end - 1) * xstride + 8 * (gt % 16);
    f32x4 acc[NTW][NB];
    zero_acc(acc);
    w4_block<F>(mm, m.f16, xr, m.k, m.ks, xs, acc);
    if (w4_block_join(acc, xs))
#pragma unroll
      for (int t = 0; t < NTW; t++)
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
  // The rows of a group, if they were spread evenly: the lengths are on the device.  A
  // group far above the average takes its passes one after the other, its weights
  // read again by each (256 rows over 16 groups of 2048 x 4096 MXFP4: 22 us spread
  // evenly, 141 all in one; as a product of one group 12.6).
  const int avg = (rows + d.groups - 1) / d.groups;
  with_format(d, [&](auto f) {
    using F = decltype(f);
    auto go = [&](auto kernel, int tiles, int waves, int passes) {
      hipLaunchKernelGGL(kernel, dim3((d.nt + tiles - 1) / tiles, d.groups, passes),
                         dim3(waves * 64), 0, s, m, x, xstride, offsets, rows, out, ostride);
    };
    constexpr int kBlock = kBlockWaves * kBlockGroups, kLong = kLongBlocks<F>;
    const long tiles = (long)d.nt * d.groups;
    auto passes = [&](int nb) { return std::min((avg + 16 * nb - 1) / (16 * nb), 65535); };
    auto rows_kernel = [&](auto one, auto two, int nb) {
      const bool wide = tiles * passes(nb) >= 256 * 2 * kBlockWaves;
      if (wide) go(two, 2 * kBlockWaves, kBlock, passes(nb));
      else go(one, kBlockWaves, kBlock, passes(nb));
    };
    // Rows staged through LDS, the more at a time the fewer reads of the weights,
    // as long as the workgroups that are left fill the chip (64 rows, 8192 x 8192
    // MXFP4: 32.4 us in 128 workgroups of 64 rows, 20.0 in 256 of 32; 32 rows: 19.5
    // in 128 of 32, 14.5 in 256 of 16; 16 rows: 14.0 in 128 of 16, 19.0 from
    // memory).  From memory up to 6 rows (8 rows: 13.4 us staged, 14.6; 5: 13.5,
    // 12.2), INT4, whose sums are scaled row by row, up to 8 (8 rows: 17.0, 14.4) ...
    auto blocks = [&](int nb) { return tiles * passes(nb) / kBlockWaves; };
    if (avg > 32 && blocks(kLong) >= 256)
      rows_kernel(w4_linear_rows_kernel<F, 1, kLong>, w4_linear_rows_kernel<F, 2, kLong>, kLong);
    else if (avg > 16 && blocks(2) >= 192)
      rows_kernel(w4_linear_rows_kernel<F, 1, 2>, w4_linear_rows_kernel<F, 2, 2>, 2);
    else if (avg > (F::kGrouped ? 8 : 6) && blocks(1) >= 96)
      rows_kernel(w4_linear_rows_kernel<F, 1, 1>, w4_linear_rows_kernel<F, 2, 1>, 1);
    // ... and where tiles are few (32 rows, 512 outputs of 8192: 10.2 us, staged in 8
    // workgroups 17.9): then more waves split the contraction of one, up to what
    // the CUs hold at once (48 rows, 2048 of 7168: 384 workgroups, 16 waves 19.2 us,
    // 8 waves 18.4)
    else if (tiles * passes(1) <= 256) go(w4_linear_kernel<F, 16>, 1, 16, passes(1));
    else if (tiles * passes(1) <= 512) go(w4_linear_kernel<F, 8>, 1, 8, passes(1));
    else go(w4_linear_kernel<F, 4>, 1, 4, passes(1));
  });
}

}  // namespace moe
