// C ABI of the gradient norm and clipping: argument checks and launches
// (grad_clip.hip).
#include "grad_clip.h"

using namespace moe;

namespace {

int status() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

size_t bytes_of(const moe_grad_tensor &t) { return (size_t)t.numel * (t.type == MOE_ROW_F32 ? 4 : 2); }

// outs: they are written.
int check(int32_t count, const moe_grad_tensor *t, bool outs) {
  if (count < 0 || (count && !t)) return MOE_ERR_INVALID_ARG;
  if (count > kGradSetMost) return MOE_ERR_UNSUPPORTED;
  for (int i = 0; i < count; i++) {
    if (t[i].numel < 0 || t[i].type < MOE_ROW_BF16 || t[i].type > MOE_ROW_F32)
      return MOE_ERR_INVALID_ARG;
    if (t[i].numel > (1L << 40)) return MOE_ERR_UNSUPPORTED;
    const uintptr_t size = t[i].type == MOE_ROW_F32 ? 4 : 2;
    const uintptr_t x = (uintptr_t)t[i].x, o = (uintptr_t)t[i].out;
    if (t[i].numel && (!x || x % size)) return MOE_ERR_INVALID_ARG;
    if (!outs || !t[i].numel) continue;
    // a tensor over a part of itself is refused
    if (!o || o % size || (x != o && x < o + bytes_of(t[i]) && o < x + bytes_of(t[i])))
      return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

bool known(int32_t norm_type) { return norm_type == MOE_NORM_2 || norm_type == MOE_NORM_INF; }

}  // namespace

extern "C" {

size_t moe_grad_workspace_bytes(int32_t count, const moe_grad_tensor *tensors) {
  return check(count, tensors, false) ? 0 : (grad_partials(count, tensors) * 8 + 255) & ~(size_t)255;
}

int moe_grad_norm(int32_t count, const moe_grad_tensor *tensors, int32_t norm_type, double *total,
                  float *norm, void *ws, size_t ws_bytes, void *stream) {
  const int rc = check(count, tensors, false);
  if (rc) return rc;
  if (!known(norm_type) || (!total && !norm) || !ws || (uintptr_t)ws % 8) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < grad_partials(count, tensors) * 8) return MOE_ERR_WORKSPACE;
  launch_grad_norm(count, tensors, norm_type == MOE_NORM_INF, (double *)ws, total, norm,
                   (hipStream_t)stream);
  return status();
}

int moe_grad_scale(int32_t count, const moe_grad_tensor *tensors, int32_t norm_type,
                   const double *total, float max_norm, float *norm, void *stream) {
  const int rc = check(count, tensors, true);
  if (rc) return rc;
  if (!known(norm_type) || !total || !(max_norm >= 0.0f)) return MOE_ERR_INVALID_ARG;
  launch_grad_scale(count, tensors, norm_type == MOE_NORM_INF, total, 1, max_norm, norm,
                    (hipStream_t)stream);
  return status();
}

int moe_grad_clip(int32_t count, const moe_grad_tensor *tensors, int32_t norm_type, float max_norm,
                  float *norm, void *ws, size_t ws_bytes, void *stream) {
  const int rc = check(count, tensors, true);
  if (rc) return rc;
  if (!known(norm_type) || !(max_norm >= 0.0f) || !ws || (uintptr_t)ws % 8)
    return MOE_ERR_INVALID_ARG;
  if (ws_bytes < grad_partials(count, tensors) * 8) return MOE_ERR_WORKSPACE;
  launch_grad_clip(count, tensors, norm_type == MOE_NORM_INF, (double *)ws, max_norm, norm,
                   (hipStream_t)stream);
  return status();
}

}  // extern "C"
