// Host-side launchers of sort_rows.hip (all asynchronous on stream `s`).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kSortChunk = 1024;     // flat rows per histogram, at least
constexpr int kSortMaxChunks = 128;  // histograms of one layout, at most
constexpr int kRowBf16 = 0, kRowF16 = 1, kRowF32 = 2;

// A checked moe_sort_shape: R = T k flat rows, cap rows of a sorted buffer,
// strides in values.
struct SortDims {
  long T, R, cap, tstride, rstride;
  int E, k, D, first, align, type, esize;
};

enum NarrowOp { NARROW_SORT = 0, NARROW_UNSORT = 1, NARROW_UNSORT_BWD = 2 };

long sort_workspace_words(const SortDims &d);
void launch_sort_layout(const SortDims &d, const int32_t *idx, int32_t *counts, int32_t *offsets,
                        int32_t *perm, int32_t *inv, int32_t *ws, hipStream_t s);
void launch_sort_rows(const SortDims &d, const void *x, const int32_t *counts,
                      const int32_t *offsets, const int32_t *inv, void *xs, hipStream_t s);
// Both at once in one launch, where it takes the sizes (else false, nothing done).
bool launch_sort_small(const SortDims &d, const void *x, const int32_t *idx, int32_t *counts,
                       int32_t *offsets, int32_t *perm, int32_t *inv, void *xs, hipStream_t s);
// w and add may be null (weights one, nothing added).
void launch_unsort(const SortDims &d, const void *y, const float *w, const int32_t *inv,
                   const void *add, void *out, hipStream_t s);
// dw null: only dy, and y is not read.
void launch_unsort_bwd(const SortDims &d, const void *dout, const void *y, const float *w,
                       const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *dy,
                       float *dw, hipStream_t s);

}  // namespace moe
