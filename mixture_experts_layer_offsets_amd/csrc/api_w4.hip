// C ABI of the 4-bit expert weights: argument checks and launches (w4_*.hip).
#include <algorithm>

#include "../../include/moe.h"
#include "kernels.h"
#include "w4.h"

using namespace moe;

namespace {

size_t up256(size_t v) { return (v + 255) & ~(size_t)255; }

int status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int check_w4(const moe_w4_shape *s, W4Dims *d) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->groups < 1 || s->n < 1 || s->k < 1 || s->group_size < 1) return MOE_ERR_INVALID_ARG;
  if (s->format != MOE_W4_MXFP4 && s->format != MOE_W4_INT4) return MOE_ERR_INVALID_ARG;
  if (s->zeros < 0 || s->zeros > 1 || s->scale_type < MOE_SCALE_BF16 ||
      s->scale_type > MOE_SCALE_F16)
    return MOE_ERR_INVALID_ARG;
  const bool mx = s->format == MOE_W4_MXFP4;
  if (mx && s->zeros) return MOE_ERR_INVALID_ARG;
  if (s->group_size != 32 && (mx || (s->group_size != 64 && s->group_size != 128)))
    return MOE_ERR_UNSUPPORTED;
  if (s->k % s->group_size || s->groups > 1024 || s->n > (1 << 20) || s->k > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  d->groups = s->groups; d->n = s->n; d->k = s->k;
  d->fmt = mx ? kW4Mx : kW4Int;
  d->group = s->group_size;
  d->f16_scales = s->scale_type == MOE_SCALE_F16;
  d->zeros = s->zeros;
  d->nt = (s->n + 15) / 16;
  d->ks = (s->k + 127) / 128;
  d->spg = 128 / s->group_size;
  const size_t tiles = (size_t)d->groups * d->nt * d->ks;
  d->code_bytes = tiles * 1024;
  d->scale_bytes = up256(tiles * 16 * d->spg * (mx ? 1 : 2));
  d->zero_bytes = d->zeros ? up256(tiles * 16 * d->spg) : 0;
  if (tiles >= (1ull << 31)) return MOE_ERR_UNSUPPORTED;  // 2 TiB of codes
  return MOE_OK;
}

// Workspace of the few-token layer.
struct Work {
  uint16_t *act, *act_s;
  float *y, *y_s, *logits, *w;
  int32_t *plan, *idx, *offsets, *tiles, *order;
};

int check_layer(const moe_shape *s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->tokens < 1 || s->hidden < 1 || s->experts < 1 || s->top_k < 1 || s->inter < 1 ||
      s->shared_inter < 0)
    return MOE_ERR_INVALID_ARG;
  if (s->dtype < MOE_BF16 || s->dtype > MOE_MXFP8_W6E3M2) return MOE_ERR_INVALID_ARG;
  if (s->dtype != MOE_BF16) return MOE_ERR_UNSUPPORTED;
  if (s->hidden % 64 || s->inter % 64 || s->shared_inter % 64) return MOE_ERR_UNSUPPORTED;
  if (s->experts > 1024 || s->top_k > 16 || (int64_t)s->tokens * s->top_k > kW4MaxSlots)
    return MOE_ERR_UNSUPPORTED;
  if ((int64_t)s->hidden * s->experts >= (1L << 31) || s->hidden > (1 << 20))
    return MOE_ERR_UNSUPPORTED;
  // the hidden rows' buffers stay below 2 GiB
  if ((int64_t)s->tokens * s->top_k * s->inter >= (1L << 30) ||
      (int64_t)s->tokens * s->shared_inter >= (1L << 30))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

size_t carve(const moe_shape *s, void *ws, Work *w) {
  char *base = (char *)ws;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    void *p = base ? base + off : nullptr;
    off += up256(bytes);
    return p;
  };
  const size_t T = s->tokens, R = T * s->top_k, H = s->hidden, E = s->experts;
  w->act = (uint16_t *)take(R * s->inter * 2);
  w->act_s = (uint16_t *)take(T * s->shared_inter * 2);
  w->y = (float *)take(R * H * 4);
  w->y_s = (float *)take(s->shared_inter ? T * H * 4 : 0);
  w->plan = (int32_t *)take(w4_plan_words((int)R, (int)E) * 4);
  w->logits = (float *)take(T * E * 4);
  w->idx = (int32_t *)take(R * 4);
  w->w = (float *)take(R * 4);
  w->offsets = (int32_t *)take(2 * 4);
  w->tiles = (int32_t *)take(2 * 4);
  w->order = (int32_t *)take(4);
  return off;
}

}  // namespace

extern "C" {

size_t moe_w4_bytes(const moe_w4_shape *shape) {
  W4Dims d;
  return check_w4(shape, &d) ? 0 : d.bytes();
}

int moe_w4_pack(const moe_w4_shape *shape, const uint8_t *codes, const void *scales,
                const uint8_t *zeros, void *packed, void *stream) {
  W4Dims d;
  const int rc = check_w4(shape, &d);
  if (rc) return rc;
  if (!codes || !scales || !packed || (zeros != nullptr) != (d.zeros != 0))
    return MOE_ERR_INVALID_ARG;
  launch_w4_pack(d, codes, scales, zeros, packed, (hipStream_t)stream);
  return status();
}

int moe_w4_quantize(const moe_w4_shape *shape, const uint16_t *w, void *packed, void *stream) {
  W4Dims d;
  const int rc = check_w4(shape, &d);
  if (rc) return rc;
  if (!w || !packed) return MOE_ERR_INVALID_ARG;
  launch_w4_quantize(d, w, packed, (hipStream_t)stream);
  return status();
}

int moe_w4_unpack(const moe_w4_shape *shape, const void *packed, float *w, void *stream) {
  W4Dims d;
  const int rc = check_w4(shape, &d);
  if (rc) return rc;
  if (!w || !packed) return MOE_ERR_INVALID_ARG;
  launch_w4_unpack(d, packed, w, (hipStream_t)stream);
  return status();
}

int moe_w4_linear(const moe_w4_shape *shape, int32_t rows, const uint16_t *x, int64_t x_stride,
                  const int32_t *offsets, const void *packed, uint16_t *out, int64_t out_stride,
                  void *stream) {
  W4Dims d;
  const int rc = check_w4(shape, &d);
  if (rc) return rc;
  if (rows < 0 || x_stride < d.k || out_stride < d.n || !packed || (rows && (!x || !out)) ||
      (!offsets && d.groups != 1))
    return MOE_ERR_INVALID_ARG;
  // row indices, and a pass past them, take 31 bits
  if (x_stride > (1L << 32) || out_stride > (1L << 32) || rows > (1 << 30))
    return MOE_ERR_UNSUPPORTED;
  if (rows && x == out) return MOE_ERR_INVALID_ARG;
  launch_w4_linear(d, rows, x, x_stride, offsets, packed, out, out_stride, (hipStream_t)stream);
  return status();
}

size_t moe_w4_decode_workspace_bytes(const moe_shape *shape) {
  Work w;
  return check_layer(shape) ? 0 : carve(shape, nullptr, &w);
}

int moe_w4_decode_fwd(const moe_shape *shape, const moe_w4_experts *experts, const uint16_t *x,
                      const uint16_t *w_router, const float *bias, const int32_t *topk_idx_in,
                      const float *topk_w_in, uint16_t *out, void *ws, size_t ws_bytes,
                      void *stream) {
  int rc = check_layer(shape);
  if (rc) return rc;
  if (!experts || !experts->gate || !experts->up || !experts->down || !x || !out || !ws)
    return MOE_ERR_INVALID_ARG;
  const bool router = w_router != nullptr, shared = shape->shared_inter > 0;
  if (router == (topk_idx_in != nullptr) || (topk_idx_in != nullptr) != (topk_w_in != nullptr))
    return MOE_ERR_INVALID_ARG;
  const int T = shape->tokens, H = shape->hidden, E = shape->experts, k = shape->top_k;
  if (router && (k > E || experts->first_expert)) return MOE_ERR_INVALID_ARG;
  if (router && E % 8) return MOE_ERR_UNSUPPORTED;
  if (shared != (experts->shared_gate != nullptr) || shared != (experts->shared_up != nullptr) ||
      shared != (experts->shared_down != nullptr))
    return MOE_ERR_INVALID_ARG;
  // the matrices' own limits (format, group size against H, I and Is)
  auto dims = [&](int groups, int n, int kk, W4Dims *d) {
    const moe_w4_shape s = {groups, n, kk, experts->format, experts->group_size,
                            experts->scale_type, experts->zeros};
    return check_w4(&s, d);
  };
  W4Dims up, down, up_s, down_s;
  if ((rc = dims(E, shape->inter, H, &up)) || (rc = dims(E, H, shape->inter, &down))) return rc;
  if (shared && ((rc = dims(1, shape->shared_inter, H, &up_s)) ||
                 (rc = dims(1, H, shape->shared_inter, &down_s))))
    return rc;
  Work w;
  if (ws_bytes < carve(shape, ws, &w)) return MOE_ERR_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  const int32_t *idx = topk_idx_in;
  const float *wts = topk_w_in;
  int first = experts->first_expert;
  if (router) {
    launch_dense_groups(w.offsets, w.tiles, w.order, T, kTileM, s);
    GemmArgs lg{};
    lg.A = x; lg.lda = H;
    lg.B = w_router; lg.ldb = E;
    lg.C = w.logits; lg.ldc = E;
    lg.bias = bias;
    lg.offsets = w.offsets; lg.tile_start = w.tiles;
    lg.G = 1; lg.N = E; lg.K = H;
    launch_gemm_rows(lg, EPI_F32, false, T, s);
    launch_topk(w.logits, T, E, k, w.idx, w.w, s);
    idx = w.idx;
    wts = w.w;
  }
  W4Layer a{};
  a.up = up; a.down = down;
  a.shared = shared;
  if (shared) { a.up_s = up_s; a.down_s = down_s; }
  a.T = T; a.k = k; a.first = first;
  a.x = x; a.idx = idx; a.w = wts;
  a.w_gate = experts->gate; a.w_up = experts->up; a.w_down = experts->down;
  a.ws_gate = experts->shared_gate; a.ws_up = experts->shared_up; a.ws_down = experts->shared_down;
  a.act = w.act; a.act_s = w.act_s; a.y = w.y; a.y_s = w.y_s; a.plan = w.plan; a.out = out;
  launch_w4_ffn(a, s);
  return status();
}

}  // extern "C"
