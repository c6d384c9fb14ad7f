// Few-token FFN of experts with 4-bit weights (w4_device.h):
//   plan:    (more than one token) the used experts, and for each the slots
//            that are its tokens' first ones with it, with the routing weight
//            (summed if a token names the expert twice); one token's few slots
//            are looked up by every workgroup itself;
//   gate_up: a[f] = w silu(x Wg) (x Wu) at the place f of such a slot;
//   down:    out[t] = sum over the experts of a Wd (+ the shared expert): the
//            weighted sum of the experts' outputs is the matrix product's own
//            accumulation, and neither expert outputs nor a combine exist.
#include <algorithm>

#include "w4_device.h"

namespace moe {

namespace {

constexpr int kWaves = 8;           // waves of a workgroup
constexpr int kRowLds = 64 * 1024;  // most LDS for staged rows
constexpr int kTokenBlock = 64;     // tokens of one down workgroup

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
  int32_t *wcnt = cnt + E;            // [16][E] rows per wave in this round
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
  float w;         // and weight
};

__device__ __forceinline__ Token one_token(const int32_t *idx, const float *w, int k, int first,
                                           int E) {
  const int lane = threadIdx.x & 63;
  const int e = lane < k ? local_id(idx[lane], first, E) : -1;
  const float own = lane < k ? w[lane] : 0.0f;
  const uint64_t mine = same_expert(e, E);
  const bool head = e >= 0 && !(mine & below(lane));
  float sum = own;
  for (int j = 1; j < k; j++) {  // later slots with the same expert
    const float v = __shfl_down(own, j, 64);
    if (lane + j < k && (mine >> (lane + j) & 1)) sum += v;
  }
  Token t{0, -1, 0, 0.0f};
  for (uint64_t heads = __ballot(head); heads; heads &= heads - 1) {
    const int at = __ffsll((unsigned long long)heads) - 1;
    const int he = __builtin_amdgcn_readlane(e, at);
    const float hw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sum), at));
    if (lane == t.used) {
      t.e = he;
      t.f = at;
      t.w = hw;
    }
    t.used++;
  }
  return t;
}

// ---------------------------------------------------------------------------
// gate_up.

struct Ffn {
  W4Mat gate, up;
  const int32_t *idx;
  const float *w;
  int slots, k, first, E;
  uint16_t *act;
};

// The rows of one expert: n of them, at slots f[r] with weights w[r]; f null: n
// consecutive slots from f1 on, with weight w1.
struct Rows {
  int e, n, f1;
  float w1;
  const int32_t *f;
  const float *w;
  __device__ __forceinline__ int slot(int r) const { return f ? f[r] : f1 + r; }
  __device__ __forceinline__ float weight(int r) const { return f ? w[r] : w1; }
};

// Rows of workgroup row u (u == used: the shared expert's, every token).
template <bool SINGLE>
__device__ __forceinline__ Rows find_rows(const Ffn &q, const Plan &plan, int u, bool shared) {
  if (shared) return {0, q.slots, 0, 1.0f, nullptr, nullptr};
  if constexpr (SINGLE) {
    const Token t = one_token(q.idx, q.w, q.k, q.first, q.E);
    if (u >= t.used) return {0, 0, 0, 0.0f, nullptr, nullptr};
    return {__builtin_amdgcn_readlane(t.e, u), 1, __builtin_amdgcn_readlane(t.f, u),
            __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(t.w), u)), nullptr, nullptr};
  }
  if (u >= __builtin_amdgcn_readfirstlane(plan.used[0])) return {0, 0, 0, 0.0f, nullptr, nullptr};
  const int at = __builtin_amdgcn_readfirstlane(plan.roff[u]);
  return {__builtin_amdgcn_readfirstlane(plan.elist[u]),
          __builtin_amdgcn_readfirstlane(plan.roff[u + 1]) - at, 0, 0.0f, plan.rows + at,
          plan.wrow + at};
}

// a[f] of row r and output n, from the sums of its gate and up products:
// rounded to bf16 once, weight included, as the matrix operand of down.
__device__ __forceinline__ void put_act(const Ffn &q, const Rows &rows, int r, int n, float g,
                                        float u) {
  if (n < q.gate.n)
    q.act[(size_t)rows.slot(r) * q.gate.n + n] = to_bf16(rows.weight(r) * silu_f(g) * u);
}

// Rows in LDS (16 a pass, at most kRowLds).  A workgroup takes `tpw` tile pairs
// of one expert; its waves take their steps in turn.  Grid (tile groups, used
// experts [+ 1: the shared expert]).
template <class F, int D, bool SINGLE>
__global__ __launch_bounds__(kWaves * 64, 4) void w4_gate_up_lds_kernel(Ffn routed, Ffn shared,
                                                                     Plan plan, int used, int tpw,
                                                                     const uint16_t *x) {
  extern __shared__ __attribute__((aligned(16))) char xs[];
  __shared__ float red[kWaves * 2 * 256];
  const bool is_shared = (int)blockIdx.y == used;
  const Ffn q = is_shared ? shared : routed;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = q.gate.k, ks = q.gate.ks, nt = q.gate.nt, KC = K / 8, pitch = w4_pitch(K);
  const int j0 = blockIdx.x * tpw, j1 = min(j0 + tpw, nt);
  if (j0 >= nt) return;
  const Rows rows = find_rows<SINGLE>(q, plan, blockIdx.y, is_shared);
  if (rows.n == 0) return;
  const size_t base = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * nt;
  const int n = wave < ks ? (ks - wave + kWaves - 1) / kWaves : 0;  // steps of this wave
  const int rounds = max((n + D - 1) / D, 1);
  for (int r0 = 0; r0 < rows.n; r0 += 16) {
    const int nr = min(16, rows.n - r0);
    W4Ring<F, 2, D> ring;
    // slot d: step i of this wave
    auto refill = [&](auto d, const W4Row<F>(&m)[2], int i) {
      ring.template load<decltype(d)::value>(m, min(wave + kWaves * i, ks - 1));
    };
    W4Row<F> mm[2] = {W4Row<F>(q.gate, base + j0), W4Row<F>(q.up, base + j0)};
    each<D>([&](auto d) { refill(d, mm, d); });
    for (int c0 = tid; c0 < nr * KC; c0 += kWaves * 64 * 4) {
      w4_u32x4 v[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int c = min(c0 + kWaves * 64 * u, nr * KC - 1), r = c / KC;
        v[u] = *(const w4_u32x4u *)(x + (size_t)(rows.slot(r0 + r) / q.k) * K + (c - r * KC) * 8);
      }
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const int c = c0 + kWaves * 64 * u, r = c / KC;
        if (c < nr * KC) *(w4_u32x4 *)(xs + r * pitch + (c - r * KC) * 16) = v[u];
      }
    }
    lds_barrier();
    const RowLds xr = {xs + min(lane & 15, nr - 1) * pitch};
    for (int j = j0; j < j1; j++) {
      const size_t follow = base + min(j + 1, nt - 1);
      const W4Row<F> after[2] = {W4Row<F>(q.gate, follow), W4Row<F>(q.up, follow)};
      f32x4 acc[2][1];
      zero_acc(acc);
      for (int i0 = 0; i0 < rounds * D; i0 += D) {
        each<D>([&](auto d) {
          const int i = i0 + d;
          if (i < n) {
            bf16x8 a[1][4];
#pragma unroll
            for (int b = 0; b < 4; b++)
              a[0][b] = xr.load(min(128 * (wave + kWaves * i) + 32 * b + 8 * (lane >> 4), K - 8));
            w4_step<F>(q.gate.f16, ring.cw[d], ring.sc[d], a, acc);
          }
          // the next step of this tile, or of the one after it
          const int next = i + D;
          if (next < rounds * D) refill(d, mm, next);
          else refill(d, after, next - rounds * D);
        });
      }
#pragma unroll
      for (int m = 0; m < 2; m++)
#pragma unroll
        for (int v = 0; v < 4; v++) red[(wave * 8 + m * 4 + v) * 64 + lane] = acc[m][0][v];
      lds_barrier();
      const int v = tid >> 6, row = 4 * ((tid & 63) >> 4) + v;
      if (tid < 256 && row < nr) {
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; w++) {
          g += red[(w * 8 + v) * 64 + (tid & 63)];
          u += red[(w * 8 + 4 + v) * 64 + (tid & 63)];
        }
        put_act(q, rows, r0 + row, 16 * j + (tid & 15), g, u);
      }
      lds_barrier();
      mm[0] = after[0];
      mm[1] = after[1];
    }
  }
}

// Rows from memory, 16 NB a pass: wide rows of several tokens.  Grid (tiles,
// used experts [+ 1]).
constexpr int kGuWaves = 4;

template <class F, int NB>
__global__ __launch_bounds__(kGuWaves * 64) void w4_gate_up_kernel(Ffn routed, Ffn shared, Plan plan,
                                                                   int used, const uint16_t *x) {
  __shared__ float red[kGuWaves * 2 * NB * 256];
  const bool is_shared = (int)blockIdx.y == used;
  const Ffn q = is_shared ? shared : routed;
  if ((int)blockIdx.x >= q.gate.nt) return;
  const Rows rows = find_rows<false>(q, plan, blockIdx.y, is_shared);
  const int tid = threadIdx.x, lane = tid & 63, K = q.gate.k, ks = q.gate.ks;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const size_t base = (size_t)__builtin_amdgcn_readfirstlane(rows.e) * q.gate.nt + blockIdx.x;
  const W4Row<F> mm[2] = {W4Row<F>(q.gate, base), W4Row<F>(q.up, base)};
  for (int r0 = 0; r0 < rows.n; r0 += 16 * NB) {
    const int nr = min(16 * NB, rows.n - r0);
    RowPtr xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p].p = x + (size_t)(rows.slot(r0 + min(16 * p + (lane & 15), nr - 1)) / q.k) * K;
    f32x4 acc[2][NB];
    zero_acc(acc);
    w4_stream<F>(mm, q.gate.f16, xr, K, ks * wave / kGuWaves, ks * (wave + 1) / kGuWaves, acc);
    w4_join<kGuWaves>(acc, red);
    for (int i = tid; i < NB * 256; i += kGuWaves * 64) {
      const int row = 16 * (i >> 8) + 4 * ((i & 63) >> 4) + ((i >> 6) & 3);
      if (row < nr) put_act(q, rows, r0 + row, 16 * blockIdx.x + (i & 15), red[i], red[NB * 256 + i]);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// down.

struct Down {
  W4Mat m, shared;  // shared.ks == 0: no shared expert
  const int32_t *idx;
  const float *w;
  int slots, k, first, E, T;
  const uint16_t *act, *act_s;
};

// One token: the hidden rows of its experts (and the shared one) lie in LDS one
// behind the other, and their steps are one sequence, taken in turn by the
// waves.  Grid: output tiles.
template <class F, int D>
__global__ __launch_bounds__(kWaves * 64, 4) void w4_down_token_kernel(Down q,
                                                                    uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) char xs[];
  __shared__ float red[kWaves * 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const Token t = one_token(q.idx, q.w, q.k, q.first, q.E);
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
          w4_step<F>(m.f16, ring.cw[d], ring.sc[d], x, acc);
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

// More tokens, kTokenBlock a workgroup: the steps of all used experts (and the
// shared one) are one sequence, split over the waves; an expert's rows are its
// own tokens, and their sums are added to the wave's [tokens][16] tile in LDS
// at the end of each expert.  Grid (output tiles, token blocks).
template <class F>
__global__ __launch_bounds__(kWaves * 64, 4) void w4_down_kernel(Down q, Plan plan,
                                                              uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) float sums[];  // [waves][tokens][16]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * kTokenBlock, tb = min(q.T - t0, kTokenBlock);
  const int used = plan.used[0], ks = q.m.ks, k = q.k;
  float *mine = sums + wave * tb * 16;
  for (int i = lane; i < tb * 16; i += 64) mine[i] = 0.0f;
  const int total = used * ks + q.shared.ks;
  int a = total * wave / kWaves;
  const int b = total * (wave + 1) / kWaves;
  // rows [0, n) of matrix m's row of tiles at `row`, steps [s0, s1): slot(r) is
  // the place of row r, its token slot(r) / kk
  auto segment = [&](const W4Mat &m, size_t row, const uint16_t *act, int n, auto slot, int kk,
                     int s0, int s1) {
    const W4Row<F> mm[1] = {W4Row<F>(m, row * m.nt + blockIdx.x)};
    for (int r0 = 0; r0 < n; r0 += 16) {
      const int nr = min(16, n - r0);
      const int f = slot(r0 + min(lane & 15, nr - 1));
      const RowPtr xr[1] = {{act + (size_t)f * m.k}};
      f32x4 acc[1][1];
      zero_acc(acc);
      w4_stream<F>(mm, m.f16, xr, m.k, s0, s1, acc);
#pragma unroll
      for (int v = 0; v < 4; v++) {
        const int r = 4 * (lane >> 4) + v, t = __shfl(f, r, 64) / kk - t0;
        if (r < nr) mine[t * 16 + (lane & 15)] += acc[0][0][v];
      }
    }
  };
  for (int u = a / ks; a < b && u < used; u++) {
    const int end = min(b, (u + 1) * ks);
    int r0 = plan.roff[u], r1 = plan.roff[u + 1];
    if (q.T > kTokenBlock) {  // the rows of this block's tokens: slots ascend
      int lo = 0, hi = 0;
      for (int r = r0; r < r1; r += 64) {
        const int f = r + lane < r1 ? plan.rows[r + lane] : 0x7FFFFFFF;
        lo += __popcll(__ballot(f < t0 * k));
        hi += __popcll(__ballot(f < (t0 + tb) * k));
      }
      r1 = r0 + hi;
      r0 += lo;
    }
    const int32_t *rows = plan.rows + r0;
    segment(q.m, __builtin_amdgcn_readfirstlane(plan.elist[u]), q.act, r1 - r0, [&](int r) { return rows[r]; }, k, a - u * ks,
            end - u * ks);
    a = end;
  }
  if (a < b)
    segment(q.shared, 0, q.act_s, tb, [&](int r) { return t0 + r; }, 1, a - used * ks,
            b - used * ks);
  __syncthreads();
  for (int i = tid; i < tb * 16; i += kWaves * 64) {
    float s = 0.0f;
    for (int w = 0; w < kWaves; w++) s += sums[w * tb * 16 + i];
    const int n = 16 * blockIdx.x + (i & 15);
    if (n < q.m.n) out[(size_t)(t0 + (i >> 4)) * q.m.n + n] = to_bf16(s);
  }
}

}  // namespace

size_t w4_plan_words(int slots, int E) { return 64 + 2 * (size_t)E + 64 + 2 * (size_t)slots; }

void launch_w4_ffn(const W4Layer &a, hipStream_t s) {
  const int slots = a.T * a.k, E = a.up.groups, H = a.up.k, I = a.down.k;
  Ffn r{w4_view(a.up, a.w_gate), w4_view(a.up, a.w_up), a.idx, a.w, slots, a.k, a.first, E, a.act};
  Ffn sh = r;
  Down d{w4_view(a.down, a.w_down), {}, a.idx, a.w, slots, a.k, a.first, E, a.T, a.act, nullptr};
  long token_lds = 2L * a.k * I;
  if (a.shared) {
    sh = {w4_view(a.up_s, a.ws_gate), w4_view(a.up_s, a.ws_up), nullptr, nullptr, a.T, 1, 0, 1,
          a.act_s};
    d.shared = w4_view(a.down_s, a.ws_down);
    d.act_s = a.act_s;
    token_lds += 2L * a.down_s.k;
  }
  Plan p;
  p.used = a.plan;
  p.elist = p.used + 64;
  p.roff = p.elist + E;
  p.rows = p.roff + E + 64;
  p.wrow = (float *)(p.rows + slots);
  const int used = std::min(E, slots), avg = slots / E;
  const int nt = a.shared ? std::max(a.up.nt, a.up_s.nt) : a.up.nt;
  const long row_lds = (long)std::min(a.T, 16) * w4_pitch(H);
  const bool staged = row_lds <= kRowLds && avg <= 16;
  const bool single = a.T == 1 && staged && token_lds <= kRowLds;
  if (!single)
    hipLaunchKernelGGL(w4_plan_kernel, dim3(1), dim3(kPlanThreads),
                       (17 * E + (slots + 1) / 2) * sizeof(int32_t), s, a.idx, a.w, slots, a.k,
                       a.first, E, p);
  const unsigned gy = used + (a.shared ? 1 : 0);
  with_format(a.up, [&](auto f) {
    using F = decltype(f);
    if (staged) {
      // about two workgroups a CU
      const int tpw = std::max(1, (int)(((long)nt * gy + 511) / 512));
      auto up = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((nt + tpw - 1) / tpw, gy), dim3(kWaves * 64), row_lds, s, r,
                           sh, p, used, tpw, a.x);
      };
      if (single) up(w4_gate_up_lds_kernel<F, 4, true>);
      else up(w4_gate_up_lds_kernel<F, 4, false>);
    } else {
      auto up = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(nt, gy), dim3(kGuWaves * 64), 0, s, r, sh, p, used, a.x);
      };
      if (avg <= 16) up(w4_gate_up_kernel<F, 1>);
      else if (avg <= 32) up(w4_gate_up_kernel<F, 2>);
      else up(w4_gate_up_kernel<F, 4>);
    }
    if (single)
      hipLaunchKernelGGL((w4_down_token_kernel<F, 8>), dim3(a.down.nt), dim3(kWaves * 64), token_lds,
                         s, d, a.out);
    else
      hipLaunchKernelGGL(w4_down_kernel<F>,
                         dim3(a.down.nt, (a.T + kTokenBlock - 1) / kTokenBlock), dim3(kWaves * 64),
                         kWaves * 64 * std::min(a.T, kTokenBlock), s, d, p, a.out);
  });
}

}  // namespace moe
