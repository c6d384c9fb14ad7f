// Host-side launchers of the f8_*.hip files (all asynchronous on stream `s`).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kF8Block = 128;  // values that share a scale

// A checked moe_f8_shape and the pieces of its packed buffer: nt = ceil(n / 16)
// tiles of outputs, nb = ceil(n / 128) and ks = ceil(k / 128) blocks.  The layout
// of a tile is in f8_device.h.
struct F8Dims {
  int groups, n, k, f16;
  int nt, nb, ks;
  size_t code_bytes, scale_bytes;  // one scale a tile; rounded up to 256
  size_t bytes() const { return code_bytes + scale_bytes; }
};

// MOE_OK and the dims of a shape, or the error that it is refused with.
int f8_dims(const moe_f8_shape *s, F8Dims *d);

// 16-bit rows of a caller's tensor, `stride` values apart.
struct F8Rows {
  const uint16_t *p;
  long stride;
  int f16;  // fp16, else bf16
};

void launch_f8_pack(const F8Dims &d, const uint8_t *codes, const float *scales, void *packed,
                    hipStream_t s);
void launch_f8_quantize(const F8Dims &d, const void *w, int type, void *packed, hipStream_t s);
void launch_f8_unpack(const F8Dims &d, const void *packed, float *w, hipStream_t s);
void launch_f8_transpose(const F8Dims &d, const void *packed, void *turned, hipStream_t s);

// codes [ceil(k / 128)][rows][128] and scales [ceil(k / 128)][rows] of rows of k
// values.
void launch_f8_quant_rows(const F8Rows &x, int rows, int k, uint8_t *codes, float *scales,
                          hipStream_t s);
// The same down the columns of x [rows][d.k] and dy [rows][d.n]: blocks of 128 rows of
// each group's rows, block b of group g at stage offsets[g] / 128 + g + b of the
// `f8_stages`.  x's codes [stage][k][128], dy's as packed weights [n / 16][stage][tile];
// scales [stage][columns rounded up to 16].
long f8_stages(int rows, int groups);
void launch_f8_quant_cols(const F8Rows &x, const F8Rows &dy, int rows, const F8Dims &d,
                          const int32_t *offsets, uint8_t *xc, float *xs, uint8_t *yc, float *ys,
                          hipStream_t s);

// out[r] = x[r] W_g for the rows r of group g (offsets null: one group, all
// rows), x as launch_f8_quant_rows leaves it.
void launch_f8_gemm(const F8Dims &d, int rows, const uint8_t *codes, const float *scales,
                    const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                    hipStream_t s);
// The same for few rows a group, and from 16-bit rows that are quantised on the way.
void launch_f8_few(const F8Dims &d, int rows, const uint8_t *codes, const float *scales,
                   const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                   hipStream_t s);
void launch_f8_few_rows(const F8Dims &d, int rows, const F8Rows &x, const int32_t *offsets,
                        const void *packed, uint16_t *out, long ostride, hipStream_t s);
// Whether launch_f8_few takes the product, and launch_f8_few_rows.
bool f8_few(const F8Dims &d, int rows);
bool f8_few_staged(const F8Dims &d, int rows);

// dw[g][k][n] = sum over the rows of group g of x[r][k] dy[r][n], from
// launch_f8_quant_cols.
void launch_f8_wgrad(const F8Dims &d, int rows, const uint8_t *xc, const float *xs,
                     const uint8_t *yc, const float *ys, const int32_t *offsets, uint16_t *dw,
                     float *parts, hipStream_t s);
// The same from 16-bit rows, in one launch; whether it takes the product.
void launch_f8_wgrad_few(const F8Rows &x, const F8Rows &dy, int rows, const F8Dims &d,
                         const int32_t *offsets, uint16_t *dw, hipStream_t s);
bool f8_wgrad_few(const F8Dims &d, int rows);
// In how many pieces launch_f8_wgrad takes each group's rows: past one, `parts` holds that
// many fp32 results, columns rounded up to 16.
int f8_splits(const F8Dims &d, int rows);

}  // namespace moe
