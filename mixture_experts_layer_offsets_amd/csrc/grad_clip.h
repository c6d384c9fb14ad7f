// Host-side launchers of grad_clip.hip (all asynchronous on stream `s`).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

constexpr int kGradSetMost = 1 << 20;  // tensors of one call, at most

// Partial sums (doubles) of the norm over these tensors: what its workspace holds.
size_t grad_partials(int count, const moe_grad_tensor *t);

// total: the sum of squares, or (inf) the largest magnitude; norm: the norm.
void launch_grad_norm(int count, const moe_grad_tensor *t, bool inf, double *partials, double *total,
                      float *norm, hipStream_t s);
// out = x min(1, max_norm / (norm + 1e-6)), the norm from n partial sums.
void launch_grad_scale(int count, const moe_grad_tensor *t, bool inf, const double *partials, int n,
                       float max_norm, float *norm, hipStream_t s);
// Both, with few launches.
void launch_grad_clip(int count, const moe_grad_tensor *t, bool inf, double *partials,
                      float max_norm, float *norm, hipStream_t s);

}  // namespace moe
