// C ABI of the 8-bit products with block scales: argument checks and launches
// (f8_*.hip).
#include "f8.h"

using namespace moe;

namespace {

constexpr int64_t kMostStride = 1L << 32;
constexpr int64_t kMostTiles = 1L << 23;

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

int status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool aligned16(const void *p) { return ((uintptr_t)p & 15) == 0; }

// Whether a value of `rows` rows of na values at a lies on one of rows of nb values at b,
// strides and sizes in 16-bit values.  Rows of one stride may lie between each other's.
bool overlap(const void *a, int64_t sa, int64_t na, const void *b, int64_t sb, int64_t nb,
             int64_t rows) {
  const int64_t d = ((int64_t)(uintptr_t)b - (int64_t)(uintptr_t)a) / 2;
  const int64_t la = (rows - 1) * sa + na, lb = (rows - 1) * sb + nb;  // from first to last
  if (d >= la || -d >= lb) return false;
  if (rows == 1 || sa != sb) return true;
  const int64_t at = ((d % sa) + sa) % sa;
  return at < na || at + nb > sa;
}

// Whether two runs of bytes meet.
bool meet(const void *a, size_t na, const void *b, size_t nb) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return na && nb && x < y + nb && y < x + na;
}

size_t values(const F8Dims &d) { return (size_t)d.groups * d.n * d.k; }

// Bytes from the first to the last value of rows of n values, `size` bytes each.
size_t run_of(int64_t rows, int64_t stride, int64_t n, size_t size) {
  return rows ? ((rows - 1) * stride + n) * size : 0;
}

// Quantised rows in a workspace.
size_t rows_bytes(const F8Dims &d, int32_t rows, size_t *scales) {
  *scales = up256((size_t)d.ks * rows * kF8Block);
  return *scales + up256((size_t)d.ks * rows * 4);
}

// Quantised columns of x and dy in a workspace.
struct Cols {
  size_t xs, yc, ys, parts, bytes;  // where each piece begins; x's codes first
};
Cols cols_of(const F8Dims &d, int32_t rows) {
  const size_t st = f8_stages(rows, d.groups);
  Cols c;
  c.xs = up256(st * d.k * kF8Block);
  c.yc = c.xs + up256(st * ((d.k + 15) & ~15) * 4);
  c.ys = c.yc + up256(st * d.nt * 2048);
  c.parts = c.ys + up256(st * d.nt * 16 * 4);
  const int splits = f8_splits(d, rows);
  c.bytes = c.parts + (splits > 1 ? up256((size_t)splits * d.groups * d.k * d.nt * 16 * 4) : 0);
  return c;
}

int check_rows(const F8Dims &d, int32_t rows, const int32_t *offsets) {
  if (rows < 0 || (!offsets && d.groups != 1)) return MOE_ERR_INVALID_ARG;
  // tiles of 128 rows x 256 outputs take 512 threads each, less than 2^32 in all
  if (rows > (1 << 30) || (rows / 128 + (int64_t)d.groups) * ((d.n + 255) / 256) >= kMostTiles)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_wgrad(const F8Dims &d, int32_t rows) {
  if (rows < 0) return MOE_ERR_INVALID_ARG;
  // stages are a grid's dimension; tiles as in check_rows
  if (f8_stages(rows, d.groups) > 65535 ||
      (int64_t)d.groups * ((d.k + 127) / 128) * ((d.n + 255) / 256) >= kMostTiles)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

namespace moe {

int f8_dims(const moe_f8_shape *s, F8Dims *d) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->groups < 1 || s->n < 1 || s->k < 1) return MOE_ERR_INVALID_ARG;
  if (s->row_type < MOE_ROW_BF16 || s->row_type > MOE_ROW_F32) return MOE_ERR_INVALID_ARG;
  if (s->row_type == MOE_ROW_F32 || s->groups > 1024 || s->n > (1 << 20) || s->k > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  d->groups = s->groups; d->n = s->n; d->k = s->k;
  d->f16 = s->row_type == MOE_ROW_F16;
  d->nt = (s->n + 15) / 16;
  d->nb = (s->n + kF8Block - 1) / kF8Block;
  d->ks = (s->k + kF8Block - 1) / kF8Block;
  const size_t tiles = (size_t)d->groups * d->nt * d->ks;
  d->code_bytes = tiles * 2048;
  d->scale_bytes = up256(tiles * 4);
  return MOE_OK;
}

}  // namespace moe

extern "C" {

size_t moe_f8_bytes(const moe_f8_shape *shape) {
  F8Dims d;
  return f8_dims(shape, &d) ? 0 : d.bytes();
}

int moe_f8_pack(const moe_f8_shape *shape, const uint8_t *codes, const float *scales, void *packed,
                void *stream) {
  F8Dims d;
  const int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (!codes || !scales || !packed || !aligned16(packed)) return MOE_ERR_INVALID_ARG;
  if (meet(packed, d.bytes(), codes, values(d)) ||
      meet(packed, d.bytes(), scales, (size_t)d.groups * d.nb * d.ks * 4))
    return MOE_ERR_INVALID_ARG;
  launch_f8_pack(d, codes, scales, packed, (hipStream_t)stream);
  return status();
}

int moe_f8_quantize(const moe_f8_shape *shape, const void *w, int32_t w_type, void *packed,
                    void *stream) {
  F8Dims d;
  const int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (!w || !packed || !aligned16(packed) || w_type < MOE_ROW_BF16 || w_type > MOE_ROW_F32)
    return MOE_ERR_INVALID_ARG;
  if (meet(packed, d.bytes(), w, values(d) * (w_type == MOE_ROW_F32 ? 4 : 2)))
    return MOE_ERR_INVALID_ARG;
  launch_f8_quantize(d, w, w_type, packed, (hipStream_t)stream);
  return status();
}

int moe_f8_unpack(const moe_f8_shape *shape, const void *packed, float *w, void *stream) {
  F8Dims d;
  const int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (!w || !packed || !aligned16(packed) || meet(w, values(d) * 4, packed, d.bytes()))
    return MOE_ERR_INVALID_ARG;
  launch_f8_unpack(d, packed, w, (hipStream_t)stream);
  return status();
}

int moe_f8_transpose(const moe_f8_shape *shape, const void *packed, void *packed_t, void *stream) {
  F8Dims d;
  const int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (!packed || !packed_t || !aligned16(packed) || !aligned16(packed_t)) return MOE_ERR_INVALID_ARG;
  const moe_f8_shape turned = {d.groups, d.k, d.n, shape->row_type};
  F8Dims t;
  if (f8_dims(&turned, &t) || meet(packed, d.bytes(), packed_t, t.bytes())) return MOE_ERR_INVALID_ARG;
  launch_f8_transpose(d, packed, packed_t, (hipStream_t)stream);
  return status();
}

int moe_f8_quantize_rows(const moe_f8_shape *shape, int32_t rows, const void *x, int64_t x_stride,
                         uint8_t *codes, float *scales, void *stream) {
  F8Dims d;
  const int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (rows < 0 || x_stride < d.k || (rows && (!x || !codes || !scales)) || !aligned16(codes))
    return MOE_ERR_INVALID_ARG;
  if (x_stride > kMostStride || rows > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  const size_t nx = run_of(rows, x_stride, d.k, 2), at = (size_t)d.ks * rows;
  if (meet(codes, at * kF8Block, x, nx) || meet(scales, at * 4, x, nx) ||
      meet(codes, at * kF8Block, scales, at * 4))
    return MOE_ERR_INVALID_ARG;
  launch_f8_quant_rows({(const uint16_t *)x, x_stride, d.f16}, rows, d.k, codes, scales,
                       (hipStream_t)stream);
  return status();
}

size_t moe_f8_linear_workspace_bytes(const moe_f8_shape *shape, int32_t rows) {
  F8Dims d;
  size_t scales;
  if (f8_dims(shape, &d) || check_rows(d, rows, (const int32_t *)1)) return 0;
  return f8_few_staged(d, rows) ? 256 : rows_bytes(d, rows, &scales);
}

int moe_f8_linear(const moe_f8_shape *shape, int32_t rows, const void *x, int64_t x_stride,
                  const int32_t *offsets, const void *packed, void *out, int64_t out_stride,
                  void *ws, size_t ws_bytes, void *stream) {
  F8Dims d;
  int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (x_stride < d.k || out_stride < d.n || !packed || !aligned16(packed) ||
      (rows > 0 && (!x || !out)))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_rows(d, rows, offsets))) return rc;
  if (x_stride > kMostStride || out_stride > kMostStride) return MOE_ERR_UNSUPPORTED;
  if (!rows) return MOE_OK;
  if (overlap(x, x_stride, d.k, out, out_stride, d.n, rows)) return MOE_ERR_INVALID_ARG;
  const F8Rows xr{(const uint16_t *)x, x_stride, d.f16};
  hipStream_t s = (hipStream_t)stream;
  if (f8_few_staged(d, rows)) {
    launch_f8_few_rows(d, rows, xr, offsets, packed, (uint16_t *)out, out_stride, s);
    return status();
  }
  size_t at;
  if (!ws || !aligned16(ws)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < rows_bytes(d, rows, &at)) return MOE_ERR_WORKSPACE;
  uint8_t *codes = (uint8_t *)ws;
  float *scales = (float *)(codes + at);
  launch_f8_quant_rows(xr, rows, d.k, codes, scales, s);
  (f8_few(d, rows) ? launch_f8_few : launch_f8_gemm)(d, rows, codes, scales, offsets, packed,
                                                     (uint16_t *)out, out_stride, s);
  return status();
}

int moe_f8_linear_codes(const moe_f8_shape *shape, int32_t rows, const uint8_t *codes,
                        const float *scales, const int32_t *offsets, const void *packed, void *out,
                        int64_t out_stride, void *stream) {
  F8Dims d;
  int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (out_stride < d.n || !packed || !aligned16(packed) || !aligned16(codes) ||
      (rows > 0 && (!codes || !scales || !out)))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_rows(d, rows, offsets))) return rc;
  if (out_stride > kMostStride) return MOE_ERR_UNSUPPORTED;
  if (!rows) return MOE_OK;
  const size_t no = run_of(rows, out_stride, d.n, 2), at = (size_t)d.ks * rows;
  if (meet(out, no, codes, at * kF8Block) || meet(out, no, scales, at * 4)) return MOE_ERR_INVALID_ARG;
  // sizes that moe_f8_linear takes in one launch go to the kernel that adds in its order
  const bool few = f8_few(d, rows) || f8_few_staged(d, rows);
  (few ? launch_f8_few : launch_f8_gemm)(d, rows, codes, scales, offsets, packed, (uint16_t *)out,
                                         out_stride, (hipStream_t)stream);
  return status();
}

size_t moe_f8_wgrad_workspace_bytes(const moe_f8_shape *shape, int32_t rows) {
  F8Dims d;
  return f8_dims(shape, &d) || check_wgrad(d, rows) ? 0 : cols_of(d, rows).bytes;
}

int moe_f8_wgrad(const moe_f8_shape *shape, int32_t rows, const void *x, int64_t x_stride,
                 const void *dy, int64_t dy_stride, const int32_t *offsets, void *dw, void *ws,
                 size_t ws_bytes, void *stream) {
  F8Dims d;
  int rc = f8_dims(shape, &d);
  if (rc) return rc;
  if (x_stride < d.k || dy_stride < d.n || !dw || !ws || !aligned16(ws) ||
      (rows > 0 && (!x || !dy)) || (!offsets && d.groups != 1))
    return MOE_ERR_INVALID_ARG;
  if ((rc = check_wgrad(d, rows))) return rc;
  if (x_stride > kMostStride || dy_stride > kMostStride) return MOE_ERR_UNSUPPORTED;
  // dw lies in one run; between a tensor's rows it would have to fit into one gap
  if (meet(dw, values(d) * 2, x, run_of(rows, x_stride, d.k, 2)) ||
      meet(dw, values(d) * 2, dy, run_of(rows, dy_stride, d.n, 2)))
    return MOE_ERR_INVALID_ARG;
  const Cols c = cols_of(d, rows);
  if (ws_bytes < c.bytes) return MOE_ERR_WORKSPACE;
  uint8_t *xc = (uint8_t *)ws, *yc = xc + c.yc;
  float *xs = (float *)(xc + c.xs), *ys = (float *)(xc + c.ys);
  hipStream_t s = (hipStream_t)stream;
  const F8Rows xr{(const uint16_t *)x, x_stride, d.f16}, yr{(const uint16_t *)dy, dy_stride, d.f16};
  if (f8_wgrad_few(d, rows)) {
    launch_f8_wgrad_few(xr, yr, rows, d, offsets, (uint16_t *)dw, s);
    return status();
  }
  launch_f8_quant_cols(xr, yr, rows, d, offsets, xc, xs, yc, ys, s);
  launch_f8_wgrad(d, rows, xc, xs, yc, ys, offsets, (uint16_t *)dw, (float *)(xc + c.parts), s);
  return status();
}

}  // extern "C"
