// C ABI of the expert-sorted rows: argument checks and launches (sort_rows.hip).
#include "../../include/moe.h"
#include "sort_rows.h"

using namespace moe;

namespace {

int check_sort(const moe_sort_shape *s, SortDims *d) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->tokens < 0 || s->experts < 1 || s->top_k < 1 || s->width < 1 || s->align < 0 ||
      s->token_stride < 0 || s->row_stride < 0)
    return MOE_ERR_INVALID_ARG;
  if (s->row_type < MOE_ROW_BF16 || s->row_type > MOE_ROW_F32) return MOE_ERR_INVALID_ARG;
  d->T = s->tokens; d->E = s->experts; d->k = s->top_k; d->D = s->width;
  d->first = s->first_expert;
  d->align = s->align < 1 ? 1 : s->align;
  d->type = s->row_type;
  d->esize = s->row_type == MOE_ROW_F32 ? 4 : 2;
  d->tstride = s->token_stride ? s->token_stride : d->D;
  d->rstride = s->row_stride ? s->row_stride : d->D;
  if (d->tstride < d->D || d->rstride < d->D) return MOE_ERR_INVALID_ARG;
  if (d->E > 1024 || d->k > 16 || d->align > 1024 || d->T > (1L << 24) || d->D > (1 << 20) ||
      d->tstride > (1L << 32) || d->rstride > (1L << 32))
    return MOE_ERR_UNSUPPORTED;
  d->R = d->T * d->k;
  d->cap = d->R + (d->R < d->E ? d->R : d->E) * (d->align - 1);
  return MOE_OK;
}

int status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

size_t workspace_bytes(const SortDims &d) {
  return ((size_t)(sort_workspace_words(d) + 1) * sizeof(int32_t) + 255) & ~(size_t)255;
}

int check_layout(const SortDims &d, const int32_t *topk_idx, const int32_t *counts,
                 const int32_t *offsets, const int32_t *perm, const int32_t *inv_perm,
                 const void *ws, size_t ws_bytes) {
  if (!counts || !offsets || !ws || (d.R && (!topk_idx || !perm || !inv_perm)))
    return MOE_ERR_INVALID_ARG;
  return ws_bytes < workspace_bytes(d) ? MOE_ERR_WORKSPACE : MOE_OK;
}

}  // namespace

extern "C" {

int64_t moe_sort_max_rows(const moe_sort_shape *shape) {
  SortDims d;
  return check_sort(shape, &d) ? -1 : d.cap;
}

size_t moe_sort_workspace_bytes(const moe_sort_shape *shape) {
  SortDims d;
  return check_sort(shape, &d) ? 0 : workspace_bytes(d);
}

int moe_sort_layout(const moe_sort_shape *shape, const int32_t *topk_idx, int32_t *counts,
                    int32_t *offsets, int32_t *perm, int32_t *inv_perm, void *ws, size_t ws_bytes,
                    void *stream) {
  SortDims d;
  const int rc = check_sort(shape, &d);
  if (rc) return rc;
  if (int bad = check_layout(d, topk_idx, counts, offsets, perm, inv_perm, ws, ws_bytes)) return bad;
  launch_sort_layout(d, topk_idx, counts, offsets, perm, inv_perm, (int32_t *)ws,
                     (hipStream_t)stream);
  return status();
}

int moe_sort_rows(const moe_sort_shape *shape, const void *x, const int32_t *counts,
                  const int32_t *offsets, const int32_t *inv_perm, void *x_sorted, void *stream) {
  SortDims d;
  const int rc = check_sort(shape, &d);
  if (rc) return rc;
  if (!counts || !offsets || (d.R && (!x || !inv_perm || !x_sorted || x == x_sorted)))
    return MOE_ERR_INVALID_ARG;
  launch_sort_rows(d, x, counts, offsets, inv_perm, x_sorted, (hipStream_t)stream);
  return status();
}

int moe_sort_fwd(const moe_sort_shape *shape, const void *x, const int32_t *topk_idx,
                 int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *inv_perm,
                 void *x_sorted, void *ws, size_t ws_bytes, void *stream) {
  SortDims d;
  int rc = check_sort(shape, &d);
  if (rc) return rc;
  rc = check_layout(d, topk_idx, counts, offsets, perm, inv_perm, ws, ws_bytes);
  if (rc) return rc;
  if (d.R && (!x || !x_sorted || x == x_sorted)) return MOE_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (!launch_sort_small(d, x, topk_idx, counts, offsets, perm, inv_perm, x_sorted, s)) {
    launch_sort_layout(d, topk_idx, counts, offsets, perm, inv_perm, (int32_t *)ws, s);
    launch_sort_rows(d, x, counts, offsets, inv_perm, x_sorted, s);
  }
  return status();
}

int moe_sort_bwd(const moe_sort_shape *shape, const void *dx_sorted, const int32_t *inv_perm,
                 void *dx, void *stream) {
  return moe_unsort_fwd(shape, dx_sorted, nullptr, inv_perm, nullptr, dx, stream);
}

int moe_unsort_fwd(const moe_sort_shape *shape, const void *y, const float *topk_w,
                   const int32_t *inv_perm, const void *add, void *out, void *stream) {
  SortDims d;
  const int rc = check_sort(shape, &d);
  if (rc) return rc;
  // the last 16 bytes of a row may be summed twice: not in place
  if (d.R && (!y || !inv_perm || !out || out == y || out == add)) return MOE_ERR_INVALID_ARG;
  launch_unsort(d, y, topk_w, inv_perm, add, out, (hipStream_t)stream);
  return status();
}

int moe_unsort_bwd(const moe_sort_shape *shape, const void *dout, const void *y,
                   const float *topk_w, const int32_t *counts, const int32_t *offsets,
                   const int32_t *inv_perm, void *dy, float *dtopk_w, void *stream) {
  SortDims d;
  const int rc = check_sort(shape, &d);
  if (rc) return rc;
  if (!counts || !offsets ||
      (d.R && (!dout || !topk_w || !inv_perm || !dy || (dtopk_w && !y) || dy == dout || dy == y)))
    return MOE_ERR_INVALID_ARG;
  launch_unsort_bwd(d, dout, y, topk_w, counts, offsets, inv_perm, dy, dtopk_w,
                    (hipStream_t)stream);
  return status();
}

}  // extern "C"
