// Tokens sorted by expert and back, with weights applied, and the gradients.
//
// With f = t k + j the flat (token, slot) index and e(f) = idx[f] - first the
// slot's expert here, a slot is kept if 0 <= e(f) < E; the others (experts of
// another GPU, padded tokens) have no row.
//   counts[e]  = kept slots of expert e
//   offsets[e] = sum over e' < e of counts[e'] rounded up to a multiple of A
//   inv[f]     = offsets[e] + #{f' < f : e(f') = e(f)}, or -1; perm its
//                inverse, -1 in the padding and behind offsets[E]
//   sort:    xs[inv[f]] = x[t]                  backward: dx[t] = sum_j dxs[inv]
//   unsort:  out[t] = sum_j w[f] y[inv[f]] (+ add[t])
//            backward: dy[inv[f]] = w[f] dout[t],  dw[f] = <dout[t], y[inv[f]]>
// Sums run in fp32 in ascending j (dw: a fixed tree over the columns), so
// every result is the same from run to run.  A masked slot is never read: its
// weight and whatever lies in rows that no slot owns have no effect.
//
// Every kernel here only moves rows, so the bound is HBM: each row read once,
// each row written once.  A lane moves 16 bytes at a time whatever the row's
// width, stride or alignment: global accesses of 16 bytes need no alignment
// on this GPU, and a row whose bytes are no multiple of 16 ends with a chunk
// that starts 16 bytes before the row's end and overlaps its neighbour (both
// lanes store the same bytes).  Rows narrower than 16 bytes take the
// `narrow` kernels, one lane per token.
#include <algorithm>

#include "common.h"
#include "sort_grid.h"
#include "sort_rows.h"

namespace moe {

namespace {

inline dim3 to_dim3(const GridDims &g) { return dim3(g.x, g.y, g.z); }

typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kSortMaxK = 16;   // top-k bound of the library
// One-launch sort: slots it takes (512: 7.5 us, layout and rows apart 12.8; 1024:
// 13.7 and 13.5), slots if aligned, where every workgroup makes the layout (256 of
// 256 experts to 16 rows: 18.9 and 19.1; 512: 24.3 and 19.5), rows of the sorted
// buffer (one workgroup fills perm's end) and bytes of a row: a wave's worth, which
// is more than it needs (64 slots, rows of 16 to 512 bytes: 12.4 us apart, 5.9 us
// in one launch; to 16 rows 12.7 and 10.4).  Rows that a padding workgroup checks
// one after the other (64 slots of 256 experts to 16 rows of 7168 bf16: 16 rows
// 14.1 us, 32 rows 23.5, 8 rows 9.6).
constexpr int kSortSmallSlots = 512, kSortSmallAligned = 256;
constexpr int kSortSmallRows = 16384, kSortSmallBytes = 1024;
constexpr int kSmallPadRows = 16;
constexpr int kRawBuffer = 0x00020000;  // raw buffer descriptor, gfx9 family
constexpr int kNonTemporal = 2;         // cache policy of a buffer access: nt

// 16 bytes at any alignment, read or written once.
__device__ __forceinline__ u32x4 ld16(const char *p) {
  return __builtin_nontemporal_load((const u32x4u *)p);
}
__device__ __forceinline__ void st16(char *p, const u32x4 &v) { *(u32x4u *)p = v; }
__device__ __forceinline__ void st16_once(char *p, const u32x4 &v) {
  __builtin_nontemporal_store((u32x4u)v, (u32x4u *)p);
}

// A row element type: N values in 16 bytes, and both conversions (to nearest
// even, NaN and infinities kept).
struct Bf16 {
  typedef uint16_t S;
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const u32x4 &v, float *f) {
    const uint4 u = make_uint4(v.x, v.y, v.z, v.w);
    unpack8(u, f);
  }
  static __device__ __forceinline__ u32x4 narrow(const float *f) {
    f32x8 t;
#pragma unroll
    for (int q = 0; q < 8; q++) t[q] = f[q];
    return __builtin_bit_cast(u32x4, __builtin_convertvector(t, bf16x8));
  }
  static __device__ __forceinline__ float get(S s) { return bf16_to_f32(s); }
  static __device__ __forceinline__ S put(float f) { return __builtin_bit_cast(S, (__bf16)f); }
};
struct F16 {
  typedef uint16_t S;
  static constexpr int N = 8;
  static __device__ __forceinline__ void widen(const u32x4 &v, float *f) {
    const f32x8 t = __builtin_convertvector(__builtin_bit_cast(f16x8, v), f32x8);
#pragma unroll
    for (int q = 0; q < 8; q++) f[q] = t[q];
  }
  static __device__ __forceinline__ u32x4 narrow(const float *f) {
    f32x8 t;
#pragma unroll
    for (int q = 0; q < 8; q++) t[q] = f[q];
    return __builtin_bit_cast(u32x4, __builtin_convertvector(t, f16x8));
  }
  static __device__ __forceinline__ float get(S s) { return (float)__builtin_bit_cast(_Float16, s); }
  static __device__ __forceinline__ S put(float f) { return __builtin_bit_cast(S, (_Float16)f); }
};
struct F32 {
  typedef uint32_t S;
  static constexpr int N = 4;
  static __device__ __forceinline__ void widen(const u32x4 &v, float *f) {
#pragma unroll
    for (int q = 0; q < 4; q++) f[q] = __uint_as_float(v[q]);
  }
  static __device__ __forceinline__ u32x4 narrow(const float *f) {
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; q++) v[q] = __float_as_uint(f[q]);
    return v;
  }
  static __device__ __forceinline__ float get(S s) { return __uint_as_float(s); }
  static __device__ __forceinline__ S put(float f) { return __float_as_uint(f); }
};

// Expert of a flat row here, or -1.  The difference is taken in 64 bits: ids
// are the caller's and may be anything.
__device__ __forceinline__ int local_expert(int32_t id, int first, int E) {
  const int64_t e = (int64_t)id - first;
  return e >= 0 && e < E ? (int)e : -1;
}

__device__ __forceinline__ int round_rows(int n, int align) {
  return align > 1 ? (n + align - 1) / align * align : n;
}

// ---------------------------------------------------------------------------
// Layout.  count: per-chunk histograms (kSortChunk flat rows a workgroup), and
// perm filled with -1.  place: every workgroup adds up the histograms of all
// chunks (totals) and of the chunks before its own, scans the totals over the
// experts and ranks its rows: lanes of a wave with the same expert find each
// other by ballots over the bits of the id.  Integers only, no order but f's.

__global__ __launch_bounds__(1024) void sort_count_kernel(const int32_t *__restrict__ idx, int R,
                                                          int first, int E, int chunk,
                                                          int32_t *__restrict__ chunk_counts,
                                                          int32_t *__restrict__ perm, int cap) {
  extern __shared__ int32_t cnt[];
  for (int e = threadIdx.x; e < E; e += 1024) cnt[e] = 0;
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * chunk;
  for (int i = threadIdx.x; i < chunk; i += 1024) {
    const int64_t f = base + i;
    if (f < R) {
      const int e = local_expert(idx[f], first, E);
      if (e >= 0) atomicAdd(&cnt[e], 1);
    }
  }
  for (int64_t r = (int64_t)blockIdx.x * 1024 + threadIdx.x; r < cap; r += (int64_t)gridDim.x * 1024)
    perm[r] = -1;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) chunk_counts[(size_t)blockIdx.x * E + e] = cnt[e];
}

// Exclusive scan over the experts of the padded counts: thread i owns experts
// [i per, (i + 1) per).  cnt and off are LDS; off gets E + 1 entries.
template <int THREADS>
__device__ __forceinline__ void scan_experts(const int32_t *cnt, int32_t *off, int E, int align,
                                             int32_t *wave_sum_lds) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int per = (E + THREADS - 1) / THREADS;
  int sum = 0;
  for (int i = 0; i < per; i++) {
    const int e = tid * per + i;
    if (e < E) sum += round_rows(cnt[e], align);
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  if (lane == 63) wave_sum_lds[wave] = inc;
  __syncthreads();
  int at = inc - sum;
  for (int w = 0; w < wave; w++) at += wave_sum_lds[w];
  for (int i = 0; i < per; i++) {
    const int e = tid * per + i;
    if (e < E) {
      off[e] = at;
      at += round_rows(cnt[e], align);
      if (e == E - 1) off[E] = at;
    }
  }
  __syncthreads();
}

// THREADS: the workgroup's, and the rows it ranks a round.
template <int THREADS>
__global__ __launch_bounds__(THREADS) void sort_place_kernel(
    const int32_t *__restrict__ idx, int R, int first, int E, int align, int chunk, int nchunks,
    const int32_t *__restrict__ chunk_counts, int32_t *__restrict__ counts,
    int32_t *__restrict__ offsets, int32_t *__restrict__ perm, int32_t *__restrict__ inv) {
  constexpr int kWaves = THREADS / 64;
  extern __shared__ int32_t sm[];
  int32_t *tot = sm;             // [E] rows of each expert
  int32_t *run = tot + E;        // [E] next free row of each expert for this chunk
  int32_t *off = run + E;        // [E + 1]
  int32_t *wcnt = off + E + 1;   // [kWaves][E] rows of each expert per wave in this pass
  __shared__ int32_t wsum[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < E; e += THREADS) tot[e] = run[e] = 0;
  for (int i = tid; i < kWaves * E; i += THREADS) wcnt[i] = 0;
  __syncthreads();
  // several threads share an expert's column of the histograms, so that few
  // loads follow one another
  int ep = 1;
  while (ep < E && ep < THREADS) ep <<= 1;
  const int parts = THREADS / ep, part = tid / ep;
  for (int e = tid % ep; e < E; e += ep) {
    int all = 0, before = 0;
#pragma unroll 16
    for (int c = part; c < nchunks; c += parts) {
      const int n = chunk_counts[(size_t)c * E + e];
      all += n;
      before += c < (int)blockIdx.x ? n : 0;
    }
    if (all) atomicAdd(&tot[e], all);
    if (before) atomicAdd(&run[e], before);
  }
  __syncthreads();
  scan_experts<THREADS>(tot, off, E, align, wsum);
  for (int e = tid; e < E; e += THREADS) {
    run[e] += off[e];
    if (blockIdx.x == 0) {
      counts[e] = tot[e];
      offsets[e] = off[e];
      if (e == E - 1) offsets[E] = off[E];
    }
  }
  __syncthreads();
  const int64_t base = (int64_t)blockIdx.x * chunk;
  const int bits = 32 - __clz(E);  // ids -1 .. E - 1, as e + 1 <= E
  for (int round = 0; round < chunk / THREADS; round++) {
    const int64_t f = base + round * THREADS + tid;
    const int e = f < R ? local_expert(idx[f], first, E) : -1;
    uint64_t mine = ~0ull;
    for (int b = 0; b < bits; b++) {
      const bool bit = ((e + 1) >> b) & 1;
      const uint64_t m = __ballot(bit);
      mine &= bit ? m : ~m;
    }
    const uint64_t below = lane ? (~0ull >> (64 - lane)) : 0ull;
    const int rank = __popcll(mine & below), n = __popcll(mine);
    const bool lead = e >= 0 && rank == 0;
    if (lead) wcnt[wave * E + e] = n;
    __syncthreads();
    if (f < R) {
      int pos = -1;
      if (e >= 0) {
        pos = run[e] + rank;
        for (int w = 0; w < wave; w++) pos += wcnt[w * E + e];
        perm[pos] = (int32_t)f;
      }
      inv[f] = pos;
    }
    __syncthreads();
    if (lead) {
      atomicAdd(&run[e], n);
      wcnt[wave * E + e] = 0;
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Rows.

__device__ __forceinline__ int row_block() { return blockIdx.z * gridDim.y + blockIdx.y; }
__device__ __forceinline__ long row_chunk(int lsh) {
  return ((long)blockIdx.x << 6) + (threadIdx.x & ((1 << lsh) - 1));
}

// Zeroes the padding rows [offsets[e] + counts[e], offsets[e + 1]) of one
// expert, this workgroup's share: `sub` of `subs` workgroups, and the wave's
// lanes split over rows and chunks as for tokens.
__device__ __forceinline__ void zero_padding(const int32_t *counts, const int32_t *offsets, int e,
                                             int sub, int subs, int lsh, char *rows, long RB,
                                             long stride) {
  const int lane = threadIdx.x & 63;
  const long c = row_chunk(lsh);
  if (c * 16 >= RB) return;
  const long at = min(c * 16, RB - 16);
  const int end = offsets[e + 1], per = 64 >> lsh;
  for (int r = offsets[e] + counts[e] + sub * per + (lane >> lsh); r < end; r += subs * per)
    st16(rows + r * stride + at, (u32x4){0, 0, 0, 0});
}

// The token of a lane: with WIDE (64 chunks or more) one token a workgroup, so
// its slots' rows come by scalar loads and their addresses stay in scalar
// registers.
template <bool WIDE>
__device__ __forceinline__ int lane_token(const RowGrid &g) {
  if constexpr (WIDE) return row_block();
  return row_block() * (64 >> g.lsh) + ((int)threadIdx.x >> g.lsh);
}

// Row `row` (uniform in the wave) as a buffer of its own: a masked row is an
// empty one, whose loads return zeros without touching memory.  So a token's
// loads need no branches, which would keep them from being in flight together.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const char *rows, int row, long stride,
                                                             long RB) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)(rows + max(row, 0) * stride), (short)0,
                                           row >= 0 ? (int)RB : 0, kRawBuffer);
}
__device__ __forceinline__ u32x4 ld16(__amdgpu_buffer_rsrc_t r, long at) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, 0, kNonTemporal);
}

// xs[inv[t k + j]] = x[t]: each token's row is read once and stored to its
// kept rows.  A token without one is not read (an eighth of 256 experts held,
// 8192 x 8 slots of 7168 bf16: 61 -> 55 us; with every slot kept, where the
// load could go out before the rows are known, 235 -> 236 us).  The sorted rows
// are stored to stay in the caches, for the products that read them next:
// non-temporal stores took 4 us off that sort, but a sort followed by a reader
// of its 235 MB went from 85 to 102 us.
template <int KMAX, bool WIDE>
__global__ __launch_bounds__(kRowBlock) void sort_rows_kernel(
    const char *__restrict__ x, const int32_t *__restrict__ inv, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ offsets, char *__restrict__ xs, int T, int k, int E, long RB,
    long xstride, long rstride, RowGrid g) {
  const int p = row_block() - g.token_blocks;
  if (p >= 0) {
    if (offsets && p < E * kPadSplit)
      zero_padding(counts, offsets, p / kPadSplit, p % kPadSplit, kPadSplit, g.lsh, xs, RB, rstride);
    return;
  }
  const int t = lane_token<WIDE>(g);
  const long c = row_chunk(g.lsh);
  if (t >= T || c * 16 >= RB) return;
  const long at = min(c * 16, RB - 16);
  int row[KMAX];
  int some = -1;
#pragma unroll
  for (int j = 0; j < KMAX; j++) {
    row[j] = inv[(long)t * k + min(j, k - 1)];
    some = max(some, row[j]);
  }
  if (some < 0) return;
  const u32x4 v = ld16(x + t * xstride + at);
#pragma unroll
  for (int j = 0; j < KMAX; j++)
    if (j < k && row[j] >= 0) st16(xs + row[j] * rstride + at, v);
}

// ---------------------------------------------------------------------------
// Layout and rows in one launch, for the few slots of a decode batch: no
// workgroup waits for another, each finds its token's rows itself.  With f's
// expert e, the row of f is the number of slots of lower experts (rounded per
// expert to the alignment) plus those of e before f; every lane holds up to NI
// ids and the wave counts them by ballots.  A token's workgroups write its
// slots' part of the layout, those behind them (align > 1) the padding rows',
// the last one the rest.  7168 bf16, 8 of 256 experts a token: 6.0 us at 8 to
// 256 slots, layout and rows apart 13.6.

// Counts and offsets of up to kSortSmallSlots slots in LDS (cnt [E], off [E+1]).
__device__ __forceinline__ void small_layout(const int32_t *idx, int R, int first, int E, int align,
                                             int32_t *cnt, int32_t *off, int32_t *wsum) {
  for (int e = threadIdx.x; e < E; e += 256) cnt[e] = 0;
  __syncthreads();
  for (int f = threadIdx.x; f < R; f += 256) {
    const int e = local_expert(idx[f], first, E);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  scan_experts<256>(cnt, off, E, align, wsum);
}

template <int NI>
__global__ __launch_bounds__(256) void sort_small_kernel(
    const char *__restrict__ x, const int32_t *__restrict__ idx, int32_t *__restrict__ counts,
    int32_t *__restrict__ offsets, int32_t *__restrict__ perm, int32_t *__restrict__ inv,
    char *__restrict__ xs, int T, int k, int first, int E, int align, int cap, long RB, long xstride,
    long rstride) {
  extern __shared__ int32_t lds[];
  __shared__ int32_t wsum[4];
  int32_t *cnt = lds, *off = lds + E;
  const int tid = threadIdx.x, lane = tid & 63, R = T * k, t = blockIdx.x;
  const long c = (long)blockIdx.y * 256 + tid;
  const long at = min(c * 16, RB - 16);
  if (t < T) {
    const u32x4 v = ld16(x + t * xstride + at);
    int id[NI];
#pragma unroll
    for (int i = 0; i < NI; i++) {
      const int f = lane + 64 * i;
      id[i] = f < R ? local_expert(idx[f], first, E) : -1;
    }
    const int own = lane < k ? local_expert(idx[t * k + lane], first, E) : -1;
    if (align > 1) small_layout(idx, R, first, E, align, cnt, off, wsum);
    for (int j = 0; j < k; j++) {
      const int f = t * k + j, e = __builtin_amdgcn_readlane(own, j);
      const bool writes = blockIdx.y == 0 && tid == 0;
      if (e < 0) {
        if (writes) inv[f] = -1;
        continue;
      }
      int row = align > 1 ? off[e] : 0;
#pragma unroll
      for (int i = 0; i < NI; i++) {
        const bool before = id[i] == e && lane + 64 * i < f;
        row += __popcll(__ballot(before || (align <= 1 && id[i] >= 0 && id[i] < e)));
      }
      if (c * 16 < RB) st16(xs + row * rstride + at, v);
      if (writes) {
        inv[f] = row;
        perm[row] = f;
      }
    }
    return;
  }
  small_layout(idx, R, first, E, align, cnt, off, wsum);
  if (blockIdx.x < gridDim.x - 1) {
    const int r0 = (t - T) * kSmallPadRows;
    for (int r = r0; r < min(r0 + kSmallPadRows, off[E]); r++) {
      int lo = 0, hi = E;  // off[lo] <= r < off[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= r) lo = mid;
        else hi = mid;
      }
      if (r < off[lo] + cnt[lo]) continue;
      if (c * 16 < RB) st16(xs + r * rstride + at, (u32x4){0, 0, 0, 0});
      if (blockIdx.y == 0 && tid == 0) perm[r] = -1;
    }
    return;
  }
  if (blockIdx.y) return;
  for (int e = tid; e <= E; e += 256) {
    offsets[e] = off[e];
    if (e < E) counts[e] = cnt[e];
  }
  for (int r = off[E] + tid; r < cap; r += 256) perm[r] = -1;
}

// out[t] = sum_j (w) y[inv[t k + j]] (+ add[t]).
template <class E, int KMAX, bool WEIGHT, bool ADD, bool WIDE>
__global__ __launch_bounds__(kRowBlock) void unsort_kernel(
    const char *__restrict__ y, const float *__restrict__ w, const int32_t *__restrict__ inv,
    const char *__restrict__ add, char *__restrict__ out, int T, int k, long RB, long tstride,
    long rstride, RowGrid g) {
  const int t = lane_token<WIDE>(g);
  const long c = row_chunk(g.lsh);
  if (t >= T || c * 16 >= RB) return;
  const long at = min(c * 16, RB - 16);
  u32x4 av;
  if constexpr (ADD) av = ld16(add + t * tstride + at);
  int row[KMAX];
  float wt[KMAX];
  int some = -1;
#pragma unroll
  for (int j = 0; j < KMAX; j++) {
    row[j] = inv[(long)t * k + min(j, k - 1)];
    if constexpr (WEIGHT) wt[j] = w[(long)t * k + min(j, k - 1)];
    if (j >= k) row[j] = -1;
    some = max(some, row[j]);
  }
  // All rows' loads go out before the first sum.  WIDE: a masked slot's row is
  // an empty buffer, and its zeros are added with weight zero.  Else its lanes
  // load the token's last row once more and leave the sum alone.
  u32x4 rv[KMAX];
  if constexpr (WIDE) {
#pragma unroll
    for (int j = 0; j < KMAX; j++) rv[j] = ld16(row_buffer(y, row[j], rstride, RB), at);
  } else if (some >= 0) {
#pragma unroll
    for (int j = 0; j < KMAX; j++)
      rv[j] = ld16(y + (row[j] >= 0 ? row[j] : some) * rstride + at);
  }
  float acc[E::N];
#pragma unroll
  for (int q = 0; q < E::N; q++) acc[q] = 0.0f;
#pragma unroll
  for (int j = 0; j < KMAX; j++) {
    float v[E::N];
    E::widen(rv[j], v);
    const float wj = WEIGHT ? (row[j] >= 0 ? wt[j] : 0.0f) : 1.0f;
#pragma unroll
    for (int q = 0; q < E::N; q++) {
      const float sum = WEIGHT ? fmaf(wj, v[q], acc[q]) : acc[q] + v[q];
      acc[q] = WIDE || row[j] >= 0 ? sum : acc[q];
    }
  }
  if constexpr (ADD) {
    float v[E::N];
    E::widen(av, v);
#pragma unroll
    for (int q = 0; q < E::N; q++) acc[q] += v[q];
  }
  st16_once(out + t * tstride + at, E::narrow(acc));
}

// dy[inv[f]] = w[f] dout[t]; dw[f] = <dout[t], y[inv[f]]>.  WPT waves share a
// token: four for rows of more than 128 chunks (one token a workgroup), else
// one (four tokens a workgroup).
template <class E, int KMAX, bool DW, int WPT>
__global__ __launch_bounds__(kBwdBlock) void unsort_bwd_kernel(
    const char *__restrict__ dout, const char *__restrict__ y, const float *__restrict__ w,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets,
    const int32_t *__restrict__ inv, char *__restrict__ dy, float *__restrict__ dw, int T, int k,
    long RB, long tstride, long rstride, int token_blocks, int pad_blocks) {
  __shared__ float red[KMAX][4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int block = blockIdx.y * gridDim.x + blockIdx.x;
  if (block >= token_blocks) {
    const int p = block - token_blocks, e = p / kPadSplit;
    if (p >= pad_blocks) return;  // of the last, partly empty row of the grid
    const int end = offsets[e + 1];
    for (int r = offsets[e] + counts[e] + p % kPadSplit; r < end; r += kPadSplit)
      for (long c = tid; c * 16 < RB; c += 256)
        st16(dy + r * rstride + min(c * 16, RB - 16), (u32x4){0, 0, 0, 0});
    return;
  }
  const int t = WPT == 4 ? block : block * 4 + __builtin_amdgcn_readfirstlane(wave);
  const bool live = t < T;
  int row[KMAX];
  float wt[KMAX], part[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; j++) {  // one token a wave: scalar loads
    part[j] = 0.0f;
    row[j] = live && j < k ? inv[(long)t * k + min(j, k - 1)] : -1;
    wt[j] = live ? w[(long)t * k + min(j, k - 1)] : 0.0f;
  }
  constexpr int kStep = 64 * WPT;
  if (live) {
    for (long c = WPT == 4 ? tid : lane; c * 16 < RB; c += kStep) {
      const long at = min(c * 16, RB - 16);
      const int skip = (int)(c * 16 - at) / (16 / E::N);  // values of an overlapping last chunk
      const u32x4 dv = ld16(dout + t * tstride + at);
      u32x4 yv[KMAX];
      if constexpr (DW) {
#pragma unroll
        for (int j = 0; j < KMAX; j++) yv[j] = ld16(row_buffer(y, row[j], rstride, RB), at);
      }
      float d[E::N];
      E::widen(dv, d);
#pragma unroll
      for (int j = 0; j < KMAX; j++) {
        if (row[j] >= 0) {
          float o[E::N];
#pragma unroll
          for (int q = 0; q < E::N; q++) o[q] = wt[j] * d[q];
          st16(dy + row[j] * rstride + at, E::narrow(o));
          if constexpr (DW) {
            float v[E::N], s = 0.0f;
            E::widen(yv[j], v);
#pragma unroll
            for (int q = 0; q < E::N; q++) s = q >= skip ? fmaf(d[q], v[q], s) : s;
            part[j] += s;
          }
        }
      }
    }
  }
  if constexpr (DW) {
#pragma unroll
    for (int j = 0; j < KMAX; j++) part[j] = j < k ? wave_sum(part[j]) : 0.0f;
    if constexpr (WPT == 4) {
#pragma unroll
      for (int j = 0; j < KMAX; j++)
        if (lane == 0) red[j][wave] = part[j];
      __syncthreads();
      if (tid < k) dw[(long)t * k + tid] = (red[tid][0] + red[tid][1]) + (red[tid][2] + red[tid][3]);
    } else if (live) {
#pragma unroll
      for (int j = 0; j < KMAX; j++)
        if (lane == 0 && j < k) dw[(long)t * k + j] = part[j];
    }
  }
}

// Rows narrower than 16 bytes: one lane per token (and, behind them, one per
// padding-row share of an expert), value by value.
template <class E>
__global__ __launch_bounds__(256) void narrow_kernel(
    NarrowOp op, const typename E::S *__restrict__ a, const typename E::S *__restrict__ b,
    const float *__restrict__ w, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ offsets, const int32_t *__restrict__ inv,
    typename E::S *__restrict__ o, float *__restrict__ dw, int T, int experts, int k, int D,
    long tstride, long rstride) {
  const long id = (long)blockIdx.x * 256 + threadIdx.x;
  if (id >= T) {
    // padding rows of the row outputs (sort, unsort backward)
    if (id >= (long)T + experts || !offsets) return;
    const int e = (int)(id - T);
    for (int r = offsets[e] + counts[e]; r < offsets[e + 1]; r++)
      for (int q = 0; q < D; q++) o[r * rstride + q] = 0;
    return;
  }
  const int t = (int)id;
  for (int q = 0; op == NARROW_UNSORT && q < D; q++) {
    float acc = 0.0f;
    for (int j = 0; j < k; j++) {
      const int r = inv[(long)t * k + j];
      if (r < 0) continue;
      const float v = E::get(a[r * rstride + q]);
      acc = w ? fmaf(w[(long)t * k + j], v, acc) : acc + v;
    }
    if (b) acc += E::get(b[t * tstride + q]);
    o[t * tstride + q] = E::put(acc);
  }
  for (int j = 0; op != NARROW_UNSORT && j < k; j++) {
    const int r = inv[(long)t * k + j];
    float s = 0.0f;
    for (int q = 0; r >= 0 && q < D; q++) {
      const typename E::S v = a[t * tstride + q];
      if (op == NARROW_SORT) {
        o[r * rstride + q] = v;
        continue;
      }
      const float d = E::get(v);
      o[r * rstride + q] = E::put(w[(long)t * k + j] * d);
      if (dw) s = fmaf(d, E::get(b[r * rstride + q]), s);
    }
    if (op == NARROW_UNSORT_BWD && dw) dw[(long)t * k + j] = s;
  }
}

}  // namespace

int sort_chunk(long R) {
  // at most kSortMaxChunks histograms, of whole rounds of 1024 rows
  const long c = (R + kSortMaxChunks - 1) / kSortMaxChunks;
  return (int)std::max<long>(kSortChunk, (c + 1023) / 1024 * 1024);
}

// Histograms of one layout.  No rows: one empty one, so that counts, offsets and
// perm are written.
int sort_chunks(long R) {
  const int chunk = sort_chunk(R);
  return (int)std::max<long>(1, (R + chunk - 1) / chunk);
}

long sort_workspace_words(const SortDims &d) { return (long)sort_chunks(d.R) * d.E; }

void launch_sort_layout(const SortDims &d, const int32_t *idx, int32_t *counts, int32_t *offsets,
                        int32_t *perm, int32_t *inv, int32_t *ws, hipStream_t s) {
  const int chunk = sort_chunk(d.R), n = sort_chunks(d.R), E = d.E;
  hipLaunchKernelGGL(sort_count_kernel, dim3(n), dim3(1024), E * sizeof(int32_t), s, idx, (int)d.R,
                     d.first, E, chunk, ws, perm, (int)d.cap);
  // more experts: fewer waves' counts, which all lie in 64 KB of LDS
  auto place = [&](auto kernel, int threads) {
    hipLaunchKernelGGL(kernel, dim3(n), dim3(threads), ((3 + threads / 64) * E + 1) * sizeof(int32_t),
                       s, idx, (int)d.R, d.first, E, d.align, chunk, n, ws, counts, offsets, perm,
                       inv);
  };
  if (E <= 512) place(sort_place_kernel<1024>, 1024);
  else place(sort_place_kernel<512>, 512);
}

namespace {

template <class E>
void launch_narrow(NarrowOp op, const SortDims &d, const void *a, const void *b, const float *w,
                   const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *o,
                   float *dw, hipStream_t s) {
  typedef typename E::S S;
  const long n = d.T + (offsets ? d.E : 0);
  hipLaunchKernelGGL(narrow_kernel<E>, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, op,
                     (const S *)a, (const S *)b, w, counts, offsets, inv, (S *)o, dw, (int)d.T, d.E,
                     d.k, d.D, d.tstride, d.rstride);
}

void launch_narrow(NarrowOp op, const SortDims &d, const void *a, const void *b, const float *w,
                   const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *o,
                   float *dw, hipStream_t s) {
  if (d.type == kRowBf16) launch_narrow<Bf16>(op, d, a, b, w, counts, offsets, inv, o, dw, s);
  else if (d.type == kRowF16) launch_narrow<F16>(op, d, a, b, w, counts, offsets, inv, o, dw, s);
  else launch_narrow<F32>(op, d, a, b, w, counts, offsets, inv, o, dw, s);
}

}  // namespace

void launch_sort_rows(const SortDims &d, const void *x, const int32_t *counts,
                      const int32_t *offsets, const int32_t *inv, void *xs, hipStream_t s) {
  if (d.T <= 0) return;
  const long RB = (long)d.D * d.esize;
  if (d.align <= 1) offsets = nullptr;  // packed segments have no padding rows
  if (RB < 16) return launch_narrow(NARROW_SORT, d, x, nullptr, nullptr, counts, offsets, inv, xs,
                                    nullptr, s);
  const RowGrid g = row_grid(d.T, RB);
  const dim3 grid = to_dim3(g.dims(g.token_blocks + (offsets ? (long)d.E * kPadSplit : 0)));
  const dim3 b(kRowBlock);
  const long xst = d.tstride * d.esize, rst = d.rstride * d.esize;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, b, 0, s, (const char *)x, inv, counts, offsets, (char *)xs,
                       (int)d.T, d.k, d.E, RB, xst, rst, g);
  };
  if (g.lsh == 6) d.k <= 8 ? go(sort_rows_kernel<8, true>) : go(sort_rows_kernel<kSortMaxK, true>);
  else d.k <= 8 ? go(sort_rows_kernel<8, false>) : go(sort_rows_kernel<kSortMaxK, false>);
}

bool launch_sort_small(const SortDims &d, const void *x, const int32_t *idx, int32_t *counts,
                       int32_t *offsets, int32_t *perm, int32_t *inv, void *xs, hipStream_t s) {
  const long RB = (long)d.D * d.esize;
  if (d.R < 1 || d.R > (d.align > 1 ? kSortSmallAligned : kSortSmallSlots) ||
      d.cap > kSortSmallRows || RB < kSortSmallBytes)
    return false;
  const long pads = d.align > 1 ? (d.cap + kSmallPadRows - 1) / kSmallPadRows : 0;
  const dim3 grid((unsigned)(d.T + pads + 1), (unsigned)((RB + 4095) / 4096)), b(256);
  const size_t lds = (2 * d.E + 1) * sizeof(int32_t);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, b, lds, s, (const char *)x, idx, counts, offsets, perm, inv,
                       (char *)xs, (int)d.T, d.k, d.first, d.E, d.align, (int)d.cap, RB,
                       d.tstride * d.esize, d.rstride * d.esize);
  };
  if (d.R <= 64) go(sort_small_kernel<1>);
  else if (d.R <= 256) go(sort_small_kernel<4>);
  else go(sort_small_kernel<kSortSmallSlots / 64>);
  return true;
}

namespace {

template <class E, int KMAX, bool WEIGHT, bool ADD>
void go_unsort(const SortDims &d, const void *y, const float *w, const int32_t *inv,
               const void *add, void *out, hipStream_t s) {
  const long RB = (long)d.D * d.esize;
  const RowGrid g = row_grid(d.T, RB);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, to_dim3(g.dims(g.token_blocks)), dim3(kRowBlock), 0, s,
                       (const char *)y, w, inv, (const char *)add, (char *)out, (int)d.T, d.k, RB, d.tstride * d.esize,
                       d.rstride * d.esize, g);
  };
  if (g.lsh == 6) go(unsort_kernel<E, KMAX, WEIGHT, ADD, true>);
  else go(unsort_kernel<E, KMAX, WEIGHT, ADD, false>);
}

template <class E>
void pick_unsort(const SortDims &d, const void *y, const float *w, const int32_t *inv,
                 const void *add, void *out, hipStream_t s) {
  if (d.k <= 8) {
    if (w && add) go_unsort<E, 8, true, true>(d, y, w, inv, add, out, s);
    else if (w) go_unsort<E, 8, true, false>(d, y, w, inv, add, out, s);
    else if (add) go_unsort<E, 8, false, true>(d, y, w, inv, add, out, s);
    else go_unsort<E, 8, false, false>(d, y, w, inv, add, out, s);
  } else {
    if (w && add) go_unsort<E, kSortMaxK, true, true>(d, y, w, inv, add, out, s);
    else if (w) go_unsort<E, kSortMaxK, true, false>(d, y, w, inv, add, out, s);
    else if (add) go_unsort<E, kSortMaxK, false, true>(d, y, w, inv, add, out, s);
    else go_unsort<E, kSortMaxK, false, false>(d, y, w, inv, add, out, s);
  }
}

template <class E, int KMAX, bool DW>
void go_unsort_bwd(const SortDims &d, const void *dout, const void *y, const float *w,
                   const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *dy,
                   float *dw, hipStream_t s) {
  const long RB = (long)d.D * d.esize;
  const BwdGrid g = bwd_grid(d.T, RB);
  const int pads = offsets ? d.E * kPadSplit : 0;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, to_dim3(g.dims(pads)), dim3(kBwdBlock), 0, s, (const char *)dout,
                       (const char *)y, w, counts, offsets, inv, (char *)dy, dw, (int)d.T, d.k, RB,
                       d.tstride * d.esize, d.rstride * d.esize, g.token_blocks, pads);
  };
  if (g.wide) go(unsort_bwd_kernel<E, KMAX, DW, 4>);
  else go(unsort_bwd_kernel<E, KMAX, DW, 1>);
}

template <class E>
void pick_unsort_bwd(const SortDims &d, const void *dout, const void *y, const float *w,
                     const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *dy,
                     float *dw, hipStream_t s) {
  if (d.k <= 8 && dw) go_unsort_bwd<E, 8, true>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
  else if (d.k <= 8) go_unsort_bwd<E, 8, false>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
  else if (dw) go_unsort_bwd<E, kSortMaxK, true>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
  else go_unsort_bwd<E, kSortMaxK, false>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
}

}  // namespace

void launch_unsort(const SortDims &d, const void *y, const float *w, const int32_t *inv,
                   const void *add, void *out, hipStream_t s) {
  if (d.T <= 0) return;
  if ((long)d.D * d.esize < 16)
    return launch_narrow(NARROW_UNSORT, d, y, add, w, nullptr, nullptr, inv, out, nullptr, s);
  if (d.type == kRowBf16) pick_unsort<Bf16>(d, y, w, inv, add, out, s);
  else if (d.type == kRowF16) pick_unsort<F16>(d, y, w, inv, add, out, s);
  else pick_unsort<F32>(d, y, w, inv, add, out, s);
}

void launch_unsort_bwd(const SortDims &d, const void *dout, const void *y, const float *w,
                       const int32_t *counts, const int32_t *offsets, const int32_t *inv, void *dy,
                       float *dw, hipStream_t s) {
  if (d.T <= 0) return;
  if (d.align <= 1) offsets = nullptr;
  if ((long)d.D * d.esize < 16)
    return launch_narrow(NARROW_UNSORT_BWD, d, dout, y, w, counts, offsets, inv, dy, dw, s);
  if (d.type == kRowBf16) pick_unsort_bwd<Bf16>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
  else if (d.type == kRowF16) pick_unsort_bwd<F16>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
  else pick_unsort_bwd<F32>(d, dout, y, w, counts, offsets, inv, dy, dw, s);
}

}  // namespace moe
