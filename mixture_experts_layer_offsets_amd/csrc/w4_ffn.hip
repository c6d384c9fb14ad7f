// Few-token FFN of experts with 4-bit weights (w4_device.h).  A row is a (token,
// expert) pair, at the place f of the token's first slot with that expert:
//   gate_up: a[f] = w silu(x Wg) (x Wu), w the routing weight (summed if the token
//            names the expert twice), rounded to bf16;
//   down:    y[f] = a[f] Wd in fp32, and out[t] = the sum of the token's y (+ the
//            shared expert's).  For one token both are one kernel: its hidden
//            rows, one behind the other, times its experts' matrices, one behind
//            the other, is one long contraction.
// No layout is made for up to 256 slots: each workgroup finds its expert's rows
// itself, since a launch costs about 4 us here and the search 1.3 to 2.
//
// Bound by reading the used experts' codes and scales: some 3 us a kernel until
// the first codes are there, then 6 to 7 TB/s until the workgroups end one by one.
// MXFP4, 7168 x 2048, 8 of 48 experts, one token: gate_up 23.4 us (125 MB, which a
// plain read takes 19.5 for), down 17.8 us (62 MB, 10.3).  INT4 in groups of 64
// with fp16 scales, 2048 x 1408, 32 tokens over about 30 of 32 experts: 24.8 us
// (94 MB, 15.0), 13.5 us (47 MB, 8.2), combine 5.0.
//
// Where that does not hold: the kernels are chosen by the routed rows an expert has
// on average.  A shared expert has every token's row and goes through the same
// ones, and so does an expert that the routing favours: its rows beyond a pass read
// its weights again, one pass after the other.  64 tokens x 8 over 256 experts, 64
// of them here, 2048 x 512 MXFP4: 36 us without a shared expert, 60 with one; 7168
// x 2048: 231 and 506.
#include <algorithm>

#include "w4_device.h"

namespace moe {

namespace {

constexpr int kWaves = 8;            // waves of a one-token down workgroup
constexpr int kTokenLds = 64 * 1024;  // most bytes of one token's hidden rows in its LDS

__device__ __forceinline__ uint64_t below(int lane) { return (1ull << lane) - 1; }

__device__ __forceinline__ int local_id(int32_t id, int first, int E) {
  const int64_t e = (int64_t)id - first;
  return e >= 0 && e < E ? (int)e : -1;
}

// Lanes whose e equals this lane's (e >= -1, below E).
__device__ __forceinline__ uint64_t same_expert(int e, int E) {
  uint64_t mine = ~0ull;
  for (int b = 0; b < 32 - __clz(E); b++) {  // the bits of e + 1 <= E
    const bool bit = ((e + 1) >> b) & 1;
    const uint64_t m = __ballot(bit);
    mine &= bit ? m : ~m;
  }
  return mine;
}

// ---------------------------------------------------------------------------
// Plan: one workgroup.  rows[roff[i] .. roff[i + 1]) are the slots of the i-th
// used expert elist[i] (ascending), wrow their weights.

struct Plan {
  int32_t *used, *elist, *roff, *rows;
  float *wrow;
};

constexpr int kPlanThreads = 1024;

__global__ __launch_bounds__(kPlanThreads) void w4_plan_kernel(const int32_t *__restrict__ idx,
                                                               const float *__restrict__ w,
                                                               int slots, int k, int first, int E,
                                                               Plan p) {
  extern __shared__ int32_t lds[];
  int32_t *cnt = lds;                 // [E] rows of each expert, then its next free row
  int32_t *wcnt = cnt + E;            // [16][E] rows per wave in this pass
  int16_t *ids = (int16_t *)(wcnt + 16 * E);  // [slots]
  __shared__ int32_t wsum[16], wused[16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int i = tid; i < 17 * E; i += kPlanThreads) lds[i] = 0;
  for (int f = tid; f < slots; f += kPlanThreads) ids[f] = (int16_t)local_id(idx[f], first, E);
  __syncthreads();
  // slot f is a row if no earlier slot of its token has the same expert
  auto row_expert = [&](int f) {
    if (f >= slots || ids[f] < 0) return -1;
    const int e = ids[f];
    for (int g = f / k * k; g < f; g++)
      if (ids[g] == e) return -1;
    return e;
  };
  for (int f = tid; f < slots; f += kPlanThreads) {
    const int e = row_expert(f);
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  // one thread per expert (E <= 1024): exclusive scans of rows and of use
  const int n = tid < E ? cnt[tid] : 0;
  int inc = n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  const uint64_t use = __ballot(n > 0);
  if (lane == 63) {
    wsum[wave] = inc;
    wused[wave] = __popcll(use);
  }
  __syncthreads();
  int at = inc - n, rank = __popcll(use & below(lane));
  for (int v = 0; v < wave; v++) {
    at += wsum[v];
    rank += wused[v];
  }
  if (n > 0) {
    p.elist[rank] = tid;
    p.roff[rank] = at;
  }
  if (tid == kPlanThreads - 1) {
    p.used[0] = rank + (n > 0);
    p.roff[rank + (n > 0)] = at + n;
  }
  if (tid < E) cnt[tid] = at;
  __syncthreads();
  // stable places, 1024 slots a round
  for (int f0 = 0; f0 < slots; f0 += kPlanThreads) {
    const int f = f0 + tid, e = row_expert(f);
    const uint64_t mine = same_expert(e, E);
    const int before = __popcll(mine & below(lane));
    const bool lead = e >= 0 && before == 0;
    if (lead) wcnt[wave * E + e] = __popcll(mine);
    __syncthreads();
    if (e >= 0) {
      int pos = cnt[e] + before;
      for (int v = 0; v < wave; v++) pos += wcnt[v * E + e];
      float sum = w[f];
      for (int g = f + 1; g < f / k * k + k; g++)
        if (ids[g] == e) sum += w[g];
      p.rows[pos] = f;
      p.wrow[pos] = sum;
    }
    __syncthreads();
    if (lead) {
      atomicAdd(&cnt[e], __popcll(mine));
      wcnt[wave * E + e] = 0;
    }
    __syncthreads();
  }
}

// One token's slots (at most 16), in every wave: its distinct experts in slot
// order, one a lane.
struct Token {
  int used, e, f;  // lane i < used: expert, first slot
};

__device__ __forceinline__ Token one_token(const int32_t *idx, int k, int first, int E) {
  const int lane = threadIdx.x & 63;
  const int e = lane < k ? local_id(idx[lane], first, E) : -1;
  Token t{0, -1, 0};
  for (uint64_t heads = __ballot(e >= 0 && !(same_expert(e, E) & below(lane))); heads;
       heads &= heads - 1) {
    const int at = __ffsll((unsigned long long)heads) - 1;
    const int he = __builtin_amdgcn_readlane(e, at);
    if (lane == t.used) {
      t.e = he;
      t.f = at;
    }
    t.used++;
  }
  return t;
}

// ---------------------------------------------------------------------------
// Rows of one expert.

// One FFN's matrices and slots.  idx null: the shared expert, every token a
// row with weight one (k = 1).
struct Ffn {
  W4Mat gate, up, down;
  const int32_t *idx;
  const float *w;
  int slots, k, first, E;
  uint16_t *act;
  float *y;
};

// n rows, at slots f[r] (f null: 0, 1, ...).
template <bool PLAN>
struct Rows {
  int e, n;
  const int32_t *planned, *idx;
  const float *wrow;
  const uint16_t *list;  // LDS
  const float *wlist;    // LDS
  __device__ __forceinline__ int slot(int r) const {
    if (!idx) return r;
    if constexpr (PLAN) return planned[r];
    return list[r];
  }
  // the routing weight, added up over the token's slots with this expert
  __device__ __forceinline__ float weight(int r) const {
    if (!idx) return 1.0f;
    if constexpr (PLAN) return wrow[r];
    return wlist[r];
  }
};

constexpr int kGuWaves = 4;
constexpr int kBlockThreads = 64 * kBlockWaves * kBlockGroups;
constexpr int kFewSlots = 256;  // slots that a workgroup looks through by itself

// The rows of the u-th used expert (u == used: the shared expert's); n = 0: there
// is none.  Up to kFewSlots slots are looked through here, by each wave for
// itself: the expert's slots by ballots over the ids, four a lane.  With as many
// slots as experts the u-th is expert u; with up to 64 slots the used experts are
// counted by their first slots; else as bits in LDS (which costs two barriers).
// Until the rows are known, at the median workgroup of the kernels above: 1.6 us of
// the one-token gate_up, at 32 tokens 2.0 of gate_up and 1.3 of down.
// WEIGHT: the rows' weights too.
template <bool PLAN, bool WEIGHT>
__device__ __forceinline__ Rows<PLAN> find_rows(const Ffn &q, const Plan &plan, int u) {
  __shared__ uint16_t list[kFewSlots];
  __shared__ float wlist[kFewSlots], ws[kFewSlots];
  Rows<PLAN> r{0, q.slots, nullptr, q.idx, nullptr, list, wlist};
  if (!q.idx) return r;
  r.n = 0;
  if constexpr (PLAN) {
    if (u >= __builtin_amdgcn_readfirstlane(plan.used[0])) return r;
    const int at = __builtin_amdgcn_readfirstlane(plan.roff[u]);
    r.e = __builtin_amdgcn_readfirstlane(plan.elist[u]);
    r.n = __builtin_amdgcn_readfirstlane(plan.roff[u + 1]) - at;
    r.planned = plan.rows + at;
    r.wrow = plan.wrow + at;
    return r;
  }
  constexpr int kIds = kFewSlots / 64;
  const int tid = threadIdx.x, lane = tid & 63;
  int32_t id[kIds];
  float wt[kIds];
#pragma unroll
  for (int i = 0; i < kIds; i++) {
    const int f = min(64 * i + lane, q.slots - 1);
    id[i] = q.idx[f];
    wt[i] = WEIGHT ? q.w[f] : 0.0f;  // of a masked slot: not used
  }
#pragma unroll
  for (int i = 0; i < kIds; i++)
    id[i] = 64 * i + lane < q.slots ? local_id(id[i], q.first, q.E) : -1;
  if (q.E <= q.slots) {
    r.e = u;
  } else if (q.slots <= 64) {
    uint64_t heads = __ballot(id[0] >= 0 && !(same_expert(id[0], q.E) & below(lane)));
    if (u >= __popcll(heads)) return r;
    for (int left = u; left > 0; left--) heads &= heads - 1;
    r.e = __builtin_amdgcn_readlane(id[0], __ffsll((unsigned long long)heads) - 1);
  } else {
    __shared__ uint32_t used[32];
    if (tid < 32) used[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kIds; i++)
      if (tid < 64 && id[i] >= 0) atomicOr(&used[id[i] >> 5], 1u << (id[i] & 31));
    __syncthreads();
    // the u-th set bit, word by word
    const uint32_t word = lane < 32 ? used[lane] : 0;
    uint32_t bits = 0;
    int at = -1, left = u;
    while (++at < (q.E + 31) / 32) {
      bits = __builtin_amdgcn_readlane(word, at);
      if (left < __popc(bits)) break;
      left -= __popc(bits);
    }
    if (at == (q.E + 31) / 32) return r;
    for (; left > 0; left--) bits &= bits - 1;
    r.e = 32 * at + __ffs(bits) - 1;
  }
  // its slots, without those whose token has an earlier one (one of the `back`
  // bits before them), whose weights go to that one; every wave writes, and then
  // reads, the same list
  if (WEIGHT)
#pragma unroll
    for (int i = 0; i < kIds; i++) ws[64 * i + lane] = id[i] == r.e ? wt[i] : 0.0f;
  wave_lds_sync();
  uint64_t prev = 0;
#pragma unroll
  for (int i = 0; i < kIds; i++) {
    const int f = 64 * i + lane, back = f % q.k;
    const uint64_t m = __ballot(id[i] == r.e);
    const uint64_t earlier =
        back <= lane ? m >> (lane - back) & below(back)
                     : (m & below(lane)) | (prev >> (64 - (back - lane)));
    const bool row = id[i] == r.e && !earlier;
    const uint64_t rows = __ballot(row);
    if (row) {
      const int at = r.n + __popcll(rows & below(lane));
      list[at] = (uint16_t)f;
      if (WEIGHT) {
        float sum = wt[i];
        for (int g = f + 1; g < min(f - back + q.k, q.slots); g++) sum += ws[g];
        wlist[at] = sum;
      }
    }
    r.n += __popcll(rows);
    prev = m;
  }
  wave_lds_sync();
  return r;
}

// act[f] of one row and output, from the sums of its gate and up products:
// rounded to bf16 once, weight included, as the matrix operand of down.  That moves
// the outputs by 2.6e-3 of their norm (their own bf16 rounding: 1.7e-3; both, from
// the 64-bit values: 2.4e-3); keeping it out would take a second operand a row.
template <bool PLAN>
__device__ __forceinline__ void put_act(const Ffn &q, const Rows<PLAN> &rows, int r, int n, float g,
                                        float u) {
  if (r < rows.n && n < q.gate.n)
    q.act[(size_t)rows.slot(r) * q.gate.n + n] = to_bf16(rows.weight(r) * silu_f(g) * u);
}

// Waves a SIMD: groups of 32 of INT4 keep more scales than 128 registers hold.
template <class F>
constexpr int kPairWaves = F::kGrouped && F::SPG == 4 ? 3 : 4;

// The product of 16 rows with NP pairs of tiles (lo[i], hi[i]), sums in acc[i] and
// acc[NP + i]; at once where a lane's scaled sums are few, else pair by pair: the
// registers of all at once (more than 128) would take a quarter of the waves.
template <class F, int NP>
__device__ __forceinline__ void stream_pairs(const W4Row<F> (&mm)[2 * NP], uint32_t f16,
                                             const RowPtr &x, int nr, int K, int s0, int s1,
                                             f32x4 (&acc)[2 * NP][1]) {
  if (!F::kGrouped) return w4_batches<F, 1, 4>(mm, f16, x, K, s0, s1, acc);
  if (nr <= 4) return w4_batches<F, 1, 1>(mm, f16, x, K, s0, s1, acc);
#pragma unroll
  for (int i = 0; i < NP; i++) {
    const W4Row<F> pair[2] = {mm[i], mm[NP + i]};
    f32x4 sum[2][1];
    zero_acc(sum);
    w4_batches<F, 1, 4>(pair, f16, x, K, s0, s1, sum);
    acc[i][0] = sum[0][0];
    acc[NP + i][0] = sum[1][0];
  }
}

// gate_up, 16 rows a pass from memory: a workgroup takes tp sets of kGuPairs pairs
// of tiles of one expert, one set after the other; its waves split the contraction.
// Two pairs share a load of the rows: 22.7 us for the 125 MB above when both were
// timed, and 24.3 with one pair and two steps of the contraction loaded together.  Four workgroups fit
// on a CU.  No faster, all at one token / at 32: a ring of steps over all sets
// (25.2 / 31.6 us), four steps together (26.5 / 29.2), rows staged through LDS
// (22.9 / 25.0), five workgroups (24.4 / 25.0); with the rows, the scales and the
// products left out the codes alone take 21.5 / 17.4.  Grid (sets of tile pairs /
// tp, used experts [+ 1: the shared expert]).
constexpr int kGuPairs = 2;

template <class F, bool PLAN>
__global__ __launch_bounds__(kGuWaves * 64, kPairWaves<F>) void w4_gate_up_kernel(
    Ffn routed, Ffn shared, Plan plan, int used, int tp, const uint16_t *x) {
  __shared__ float red[kGuWaves * 2 * kGuPairs * 256];
  const Ffn q = (int)blockIdx.y == used ? shared : routed;
  const int nt = q.gate.nt, j0 = blockIdx.x * tp * kGuPairs;
  if (j0 >= nt) return;
  const Rows<PLAN> rows = find_rows<PLAN, true>(q, plan, blockIdx.y);
  const int tid = threadIdx.x, K = q.gate.k, ks = q.gate.ks;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const size_t base = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * nt;
  for (int r0 = 0; r0 < rows.n; r0 += 16) {
    const int nr = min(16, rows.n - r0);
    const RowPtr xr = {x + (size_t)(rows.slot(r0 + min(w4_row_of_lane(), nr - 1)) / q.k) * K};
    for (int j = j0; j < min(j0 + tp * kGuPairs, nt); j += kGuPairs) {
      W4Row<F> mm[2 * kGuPairs];
#pragma unroll
      for (int i = 0; i < kGuPairs; i++) {
        mm[i] = W4Row<F>(q.gate, base + min(j + i, nt - 1));
        mm[kGuPairs + i] = W4Row<F>(q.up, base + min(j + i, nt - 1));
      }
      f32x4 acc[2 * kGuPairs][1];
      zero_acc(acc);
      stream_pairs<F, kGuPairs>(mm, q.gate.f16, xr, nr, K, ks * wave / kGuWaves,
                                ks * (wave + 1) / kGuWaves, acc);
      w4_join<kGuWaves>(acc, red, nr);
#pragma unroll
      for (int i = 0; i < kGuPairs; i++)
        put_act(q, rows, r0 + w4_row_of(tid), 16 * (j + i) + (tid & 15), red[256 * i + tid],
                red[256 * (kGuPairs + i) + tid]);
      __syncthreads();
    }
  }
}

// gate_up of many rows: a workgroup takes kBlockWaves pairs of tiles.
template <class F, int NB, bool PLAN>
__global__ __launch_bounds__(kBlockThreads, 2) void w4_gate_up_rows_kernel(Ffn routed, Ffn shared,
                                                                           Plan plan, int used,
                                                                           const uint16_t *x) {
  __shared__ __attribute__((aligned(16))) char xs[w4_block_lds<NB>()];
  const Ffn q = (int)blockIdx.y == used ? shared : routed;
  const int nt = q.gate.nt, tid = threadIdx.x, lane = tid & 63, K = q.gate.k;
  if ((int)blockIdx.x * kBlockWaves >= nt) return;
  const Rows<PLAN> rows = find_rows<PLAN, true>(q, plan, blockIdx.y);
  const int gt = tid % (64 * kBlockWaves);
  const int j = blockIdx.x * kBlockWaves + __builtin_amdgcn_readfirstlane(gt >> 6);
  const size_t row = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * nt + min(j, nt - 1);
  const W4Row<F> mm[2] = {W4Row<F>(q.gate, row), W4Row<F>(q.up, row)};
  for (int r0 = 0; r0 < rows.n; r0 += 16 * NB) {
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = x + (size_t)(rows.slot(min(r0 + 16 * p + gt / 16, rows.n - 1)) / q.k) * K + 8 * (gt % 16);
    f32x4 acc[2][NB];
    zero_acc(acc);
    w4_block<F>(mm, q.gate.f16, xr, K, q.gate.ks, xs, acc);
    if (w4_block_join(acc, xs) && j < nt)
#pragma unroll
      for (int p = 0; p < NB; p++)
#pragma unroll
        for (int v = 0; v < 4; v++)
          put_act(q, rows, r0 + 16 * p + 4 * (lane >> 4) + v, 16 * j + (lane & 15), acc[0][p][v],
                  acc[1][p][v]);
    lds_barrier();
  }
}

// ---------------------------------------------------------------------------
// down.

struct Down {
  W4Mat m, shared;  // shared.ks == 0: no shared expert
  const int32_t *idx;
  int k, first, E;
  const uint16_t *act, *act_s;
};

// One token: the hidden rows of its experts (and the shared one) lie in LDS one
// behind the other, and their steps are one sequence, split over the waves, each
// with D steps of codes in flight.  17.8 us for the 62 MB above, of which the
// stream takes about 11; the batches of gate_up here took 18.9 (the rows' loads
// keep registers that the codes need), waves that take every eighth step 18.3.
// A wave's last D refills are of steps that it does not use (16 used, 24 loaded,
// above); most are its neighbour's and come from the caches: 14 % more than the
// codes and scales is read from memory.
// Grid: output tiles.
template <class F, int D>
__global__ __launch_bounds__(kWaves * 64, 4) void w4_down_token_kernel(Down q,
                                                                    uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) char xs[];
  __shared__ float red[kWaves * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Token t = one_token(q.idx, q.k, q.first, q.E);
  f32x4 acc[1][1];
  zero_acc(acc);
  // the steps of `count` matrices, matrix i that of expert (lane i of e), its
  // row at LDS x0 + i rows of K values; put() stages those rows
  auto run = [&](const W4Mat &m, int count, int e, const char *x0, auto put) {
    const int ks = m.ks, K = m.k, total = count * ks;
    const int a = total * wave / kWaves, n = total * (wave + 1) / kWaves - a;
    W4Ring<F, 1, D> ring;
    // the next step to load, and to use: matrix and step in it
    int lu = a / ks, ls = a - lu * ks, cu = lu, cs = ls;
    auto refill = [&](auto d) {
      const size_t row = (size_t)__builtin_amdgcn_readlane(e, lu) * m.nt + blockIdx.x;
      const W4Row<F> mm[1] = {W4Row<F>(m, row)};
      ring.template load<decltype(d)::value>(mm, ls);
      const bool last = ls + 1 == ks;  // at the end: the last step again
      ls = last ? (lu + 1 < count ? 0 : ls) : ls + 1;
      lu += last && lu + 1 < count;
    };
    each<D>([&](auto d) { refill(d); });
    put();
    lds_barrier();
    for (int i0 = 0; i0 < n; i0 += D) {
      each<D>([&](auto d) {
        if (i0 + d < n) {
          const RowLds xr = {x0 + 2 * cu * K};
          bf16x8 x[1][4];
#pragma unroll
          for (int b = 0; b < 4; b++)
            x[0][b] = xr.load(min(128 * cs + 32 * b + 8 * (lane >> 4), K - 8));
          w4_step<F, 1>(m.f16, ring.cw[d], ring.sc[d], x, acc);
          const bool last = cs + 1 == ks;
          cs = last ? 0 : cs + 1;
          cu += last;
        }
        refill(d);
      });
    }
  };
  auto stage = [&](const uint16_t *src, int K, char *dst) {
    for (int c = tid; c < K / 8; c += kWaves * 64) ((w4_u32x4 *)dst)[c] = ((const w4_u32x4 *)src)[c];
  };
  const int I = q.m.k;
  if (t.used > 0)
    run(q.m, t.used, t.e, xs, [&] {
      for (int i = 0; i < t.used; i++)
        stage(q.act + (size_t)__builtin_amdgcn_readlane(t.f, i) * I, I, xs + 2 * i * I);
    });
  if (q.shared.ks) {
    char *x0 = xs + 2 * t.used * I;
    run(q.shared, 1, 0, x0, [&] { stage(q.act_s, q.shared.k, x0); });
  }
  // row 0 of the product: lanes 0..15, first value
  if (lane < 16) red[wave * 16 + lane] = acc[0][0][0];
  lds_barrier();
  const int nn = 16 * blockIdx.x + tid;
  if (tid < 16 && nn < q.m.n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; w++) s += red[w * 16 + tid];
    out[nn] = to_bf16(s);
  }
}

// More tokens: y[f] = act[f] Wd in fp32 at the places of the rows, 16 rows a
// pass, kDownTiles tiles of one expert a workgroup: at the 32 tokens above 13.5 us
// with four tiles; before other steps 14.4, where two took 18.5 and one 28 (the
// search for the rows is the same for all).  Of the 13.5 a workgroup searches 1.3,
// takes its 2.75 steps a wave one memory round trip after the other in 4.9, and
// joins and stores in 2.1; the first ends at 6.3 and the last at 12.7.  With three waves a SIMD a second,
// mostly empty round of workgroups made it 16.5.  Grid (tiles / kDownTiles, used
// experts [+ 1]).
constexpr int kDownTiles = 4;

template <bool PLAN>
__device__ __forceinline__ void put_y(const Ffn &q, const Rows<PLAN> &rows, int r, int n, float v) {
  if (r < rows.n && n < q.down.n) q.y[(size_t)rows.slot(r) * q.down.n + n] = v;
}

template <class F, bool PLAN>
__global__ __launch_bounds__(kGuWaves * 64, kPairWaves<F>) void w4_down_kernel(
    Ffn routed, Ffn shared, Plan plan, int used) {
  __shared__ float red[kGuWaves * kDownTiles * 256];
  const Ffn q = (int)blockIdx.y == used ? shared : routed;
  const int nt = q.down.nt, j0 = blockIdx.x * kDownTiles;
  const Rows<PLAN> rows = find_rows<PLAN, false>(q, plan, blockIdx.y);
  const int tid = threadIdx.x, K = q.down.k, ks = q.down.ks;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const size_t base = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * nt;
  W4Row<F> mm[kDownTiles];
#pragma unroll
  for (int t = 0; t < kDownTiles; t++) mm[t] = W4Row<F>(q.down, base + min(j0 + t, nt - 1));
  for (int r0 = 0; r0 < rows.n; r0 += 16) {
    const int nr = min(16, rows.n - r0);
    const RowPtr xr = {q.act + (size_t)rows.slot(r0 + min(w4_row_of_lane(), nr - 1)) * K};
    f32x4 acc[kDownTiles][1];
    zero_acc(acc);
    stream_pairs<F, kDownTiles / 2>(mm, q.down.f16, xr, nr, K, ks * wave / kGuWaves,
                                    ks * (wave + 1) / kGuWaves, acc);
    w4_join<kGuWaves>(acc, red, nr);
#pragma unroll
    for (int t = 0; t < kDownTiles; t++)
      put_y(q, rows, r0 + w4_row_of(tid), 16 * (j0 + t) + (tid & 15), red[256 * t + tid]);
    __syncthreads();
  }
}

// down of many rows: a workgroup takes 2 kBlockWaves tiles.
template <class F, int NB, bool PLAN>
__global__ __launch_bounds__(kBlockThreads, 2) void w4_down_rows_kernel(Ffn routed, Ffn shared,
                                                                        Plan plan, int used) {
  __shared__ __attribute__((aligned(16))) char xs[w4_block_lds<NB>()];
  const Ffn q = (int)blockIdx.y == used ? shared : routed;
  const int nt = q.down.nt, tid = threadIdx.x, lane = tid & 63, K = q.down.k;
  const Rows<PLAN> rows = find_rows<PLAN, false>(q, plan, blockIdx.y);
  const int gt = tid % (64 * kBlockWaves);
  const int j = 2 * (blockIdx.x * kBlockWaves + __builtin_amdgcn_readfirstlane(gt >> 6));
  const size_t base = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * nt;
  const W4Row<F> mm[2] = {W4Row<F>(q.down, base + min(j, nt - 1)),
                          W4Row<F>(q.down, base + min(j + 1, nt - 1))};
  for (int r0 = 0; r0 < rows.n; r0 += 16 * NB) {
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = q.act + (size_t)rows.slot(min(r0 + 16 * p + gt / 16, rows.n - 1)) * K + 8 * (gt % 16);
    f32x4 acc[2][NB];
    zero_acc(acc);
    w4_block<F>(mm, q.down.f16, xr, K, q.down.ks, xs, acc);
    if (w4_block_join(acc, xs))
#pragma unroll
      for (int t = 0; t < 2; t++)
#pragma unroll
        for (int p = 0; p < NB; p++)
#pragma unroll
          for (int v = 0; v < 4; v++)
            put_y(q, rows, r0 + 16 * p + 4 * (lane >> 4) + v, 16 * (j + t) + (lane & 15),
                  acc[t][p][v]);
    lds_barrier();
  }
}

// out[t] = the sum of the token's rows of y (a token's slots that are its first
// with their expert, ascending), then the shared expert's; rounded once.
__global__ __launch_bounds__(256) void w4_combine_kernel(const float4 *__restrict__ y,
                                                         const int32_t *__restrict__ idx, int first,
                                                         int E, const float4 *__restrict__ ys,
                                                         uint2 *__restrict__ out, int k, int HC) {
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= HC) return;
  float4 v[16];
  bool has[16];
#pragma unroll
  for (int j = 0; j < 16; j++) {
    has[j] = j < k && local_id(idx[t * k + min(j, k - 1)], first, E) >= 0;
    for (int g = 0; g < j && has[j]; g++) has[j] = idx[t * k + g] != idx[t * k + j];
    v[j] = has[j] ? y[(size_t)(t * k + j) * HC + c] : make_float4(0, 0, 0, 0);
  }
  float4 a = make_float4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < 16; j++) {
    a.x += v[j].x; a.y += v[j].y; a.z += v[j].z; a.w += v[j].w;
  }
  if (ys) {
    const float4 s = ys[(size_t)t * HC + c];
    a.x += s.x; a.y += s.y; a.z += s.z; a.w += s.w;
  }
  const bf16x2 lo = {(__bf16)a.x, (__bf16)a.y}, hi = {(__bf16)a.z, (__bf16)a.w};
  out[(size_t)t * HC + c] = make_uint2(__builtin_bit_cast(uint32_t, lo),
                                       __builtin_bit_cast(uint32_t, hi));
}

}  // namespace

size_t w4_plan_words(int slots, int E) { return 64 + 2 * (size_t)E + 64 + 2 * (size_t)slots; }

void launch_w4_ffn(const W4Layer &a, hipStream_t s) {
  const int slots = a.T * a.k, E = a.up.groups, H = a.up.k, I = a.down.k;
  Ffn r{w4_view(a.up, a.w_gate), w4_view(a.up, a.w_up), w4_view(a.down, a.w_down), a.idx, a.w,
        slots, a.k, a.first, E, a.act, a.y};
  Ffn sh = r;
  long token_lds = 2L * a.k * I;
  if (a.shared) {
    sh = {w4_view(a.up_s, a.ws_gate), w4_view(a.up_s, a.ws_up), w4_view(a.down_s, a.ws_down),
          nullptr, nullptr, a.T, 1, 0, 1, a.act_s, a.y_s};
    token_lds += 2L * a.down_s.k;
  }
  Plan p;
  p.used = a.plan;
  p.elist = p.used + 64;
  p.roff = p.elist + E;
  p.rows = p.roff + E + 64;
  p.wrow = (float *)(p.rows + slots);
  const int used = std::min(E, slots), avg = slots / E;
  const unsigned gy = used + (a.shared ? 1 : 0);
  const int nt = a.shared ? std::max(a.up.nt, a.up_s.nt) : a.up.nt;
  const bool plan = slots > kFewSlots, single = a.T == 1 && token_lds <= kTokenLds;
  if (plan)
    hipLaunchKernelGGL(w4_plan_kernel, dim3(1), dim3(kPlanThreads),
                       (17 * E + (slots + 1) / 2) * sizeof(int32_t), s, a.idx, a.w, slots, a.k,
                       a.first, E, p);
  with_format(a.up, [&](auto f) {
    using F = decltype(f);
    const dim3 b(kGuWaves * 64), bb(kBlockThreads);
    // Rows from memory up to an average of 16 an expert, where every tile reads
    // them again; staged from there on, 32 a pass up to an average of 32, then 64
    // (kLongBlocks).  8 experts of 7168 x 2048, MXFP4 / INT4 in groups of 64, us:
    // 16 rows an expert 52.3 / 67.8 from memory, 52.3 / 63.6 staged; 17 rows 82.6 /
    // 100.1 and 53.1 / 64.8; 32 rows 57.5 / 69.9, with 64 a pass 73.5 / 98.0; 40
    // rows 83.3 / 105.7 with 64 a pass, 103.6 / 127.2 with 32.
    auto up = [&](auto kernel) {
      // one set a workgroup up to 1535 sets, then so many that 768 to 1151 workgroups
      // are left.  The 32 tokens above, 1408 sets: one each 24.4 us, two each 28.3
      const int sets = (nt + kGuPairs - 1) / kGuPairs;
      const int tp = std::max(1, (int)((long)sets * gy / 768));
      hipLaunchKernelGGL(kernel, dim3((sets + tp - 1) / tp, gy), b, 0, s, r, sh, p, used, tp, a.x);
    };
    auto up_rows = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((nt + kBlockWaves - 1) / kBlockWaves, gy), bb, 0, s, r, sh, p,
                         used, a.x);
    };
    auto down = [&](auto kernel, int tiles, dim3 block) {
      hipLaunchKernelGGL(kernel, dim3((a.down.nt + tiles - 1) / tiles, gy), block, 0, s, r, sh, p,
                         used);
    };
    if (avg > 32) plan ? up_rows(w4_gate_up_rows_kernel<F, kLongBlocks<F>, true>)
                       : up_rows(w4_gate_up_rows_kernel<F, kLongBlocks<F>, false>);
    else if (avg > 16) plan ? up_rows(w4_gate_up_rows_kernel<F, 2, true>)
                            : up_rows(w4_gate_up_rows_kernel<F, 2, false>);
    else plan ? up(w4_gate_up_kernel<F, true>) : up(w4_gate_up_kernel<F, false>);
    if (single) {
      Down d{r.down, {}, a.idx, a.k, a.first, E, a.act, nullptr};
      if (a.shared) {
        d.shared = sh.down;
        d.act_s = a.act_s;
      }
      hipLaunchKernelGGL((w4_down_token_kernel<F, 8>), dim3(a.down.nt), dim3(kWaves * 64), token_lds,
                         s, d, a.out);
      return;
    }
    if (avg > 32) plan ? down(w4_down_rows_kernel<F, kLongBlocks<F>, true>, 2 * kBlockWaves, bb)
                       : down(w4_down_rows_kernel<F, kLongBlocks<F>, false>, 2 * kBlockWaves, bb);
    else if (avg > 16) plan ? down(w4_down_rows_kernel<F, 2, true>, 2 * kBlockWaves, bb)
                            : down(w4_down_rows_kernel<F, 2, false>, 2 * kBlockWaves, bb);
    else plan ? down(w4_down_kernel<F, true>, kDownTiles, b)
              : down(w4_down_kernel<F, false>, kDownTiles, b);
    const int HC = H / 4;
    hipLaunchKernelGGL(w4_combine_kernel, dim3((HC + 255) / 256, a.T), dim3(256), 0, s,
                       (const float4 *)a.y, a.idx, a.first, E, (const float4 *)(a.shared ? a.y_s : nullptr),
                       (uint2 *)a.out, a.k, HC);
  });
}

}  // namespace moe
