// Few-token FFN of experts with 4-bit weights (w4_device.h), in two launches:
//   gate_up: a[f] = w silu(x Wg) (x Wu) for every token and expert it uses, at
//            the place f of its first slot with that expert (w: the routing
//            weight, summed if the token names the expert twice);
//   down:    out[t] = sum over the experts of a Wd (+ the shared expert), one
//            long contraction over all used experts: the weighted sum of the
//            experts' outputs is the matrix product's own accumulation, and
//            neither expert outputs nor a combine exist.
// No layout is made: at a few hundred slots every workgroup finds its expert's
// slots itself (a launch of its own would cost more than the search).
#include <algorithm>

#include "w4_device.h"

namespace moe {

namespace {

__device__ __forceinline__ uint64_t below(int lane) { return (1ull << lane) - 1; }

// Bit u (counted from 0) of the set bits of m, or -1.
__device__ __forceinline__ int nth_bit(uint64_t m, int u) {
  for (; u > 0 && m; u--) m &= m - 1;
  return m ? __ffsll((unsigned long long)m) - 1 : -1;
}

__device__ __forceinline__ int local_id(int32_t id, int first, int E) {
  const int64_t e = (int64_t)id - first;
  return e >= 0 && e < E ? (int)e : -1;
}

// The used experts of a call, found by each workgroup.  Up to 64 slots: one
// slot a lane, in every wave, without LDS or barriers; the u-th expert is that
// of the u-th lane that is its expert's first.  More: ids in LDS, experts in
// ascending order.
struct Few {
  int e;              // this lane's expert, or -1
  uint64_t mine;      // lanes with the same expert
  uint64_t firsts;    // lanes that are the first of their expert
};

__device__ __forceinline__ Few few_slots(const int32_t *idx, int slots, int first, int E) {
  const int lane = threadIdx.x & 63;
  Few s;
  s.e = lane < slots ? local_id(idx[lane], first, E) : -1;
  s.mine = ~0ull;
  const int bits = 32 - __clz(E);  // of e + 1 <= E
  for (int b = 0; b < bits; b++) {
    const bool bit = ((s.e + 1) >> b) & 1;
    const uint64_t m = __ballot(bit);
    s.mine &= bit ? m : ~m;
  }
  s.firsts = __ballot(s.e >= 0 && !(s.mine & below(lane)));
  return s;
}

__device__ __forceinline__ uint64_t read_mask(uint64_t m, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)m, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((uint32_t)(m >> 32), lane);
  return ((uint64_t)hi << 32) | lo;
}

// LDS of the many-slots search.
struct Many {
  int16_t *ids;      // [slots] local expert ids
  uint32_t *used;    // [32] experts that have slots, one bit each
};

template <int THREADS>
__device__ __forceinline__ void many_slots(const int32_t *idx, int slots, int first, int E, Many s) {
  const int tid = threadIdx.x;
  if (tid < 32) s.used[tid] = 0;
  __syncthreads();
  for (int f = tid; f < slots; f += THREADS) {
    const int e = local_id(idx[f], first, E);
    s.ids[f] = (int16_t)e;
    if (e >= 0) atomicOr(&s.used[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
}

// Used experts in the words before this lane's (lanes 0..31 hold the words).
__device__ __forceinline__ int used_before(uint32_t word) {
  const int lane = threadIdx.x & 63, n = __popc(word);
  int inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  return inc - n;
}

// Rows of the u-th used expert: list[r] = f, the first slot of its r-th token
// with it, ascending.  Returns the expert (-1: no u-th one) and the count.
template <int THREADS>
__device__ __forceinline__ int find_rows(const int32_t *idx, int slots, int k, int first, int E,
                                         int u, uint16_t *list, Many ms, int *count) {
  __shared__ int chunk_rows[kW4MaxSlots / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  if (slots <= 64) {
    const Few s = few_slots(idx, slots, first, E);
    const int at = nth_bit(s.firsts, u);
    if (at < 0) return -1;
    const uint64_t members = read_mask(s.mine, at);
    const int t0 = lane / k * k;  // the lane's token's first slot
    const bool row = (members >> lane & 1) && !(members & below(lane) & ~below(t0));
    const uint64_t rows = __ballot(row);
    // every wave writes, and then reads, the same values
    if (row) list[__popcll(rows & below(lane))] = (uint16_t)lane;
    *count = __popcll(rows);
    return __builtin_amdgcn_readlane(s.e, at);
  }
  many_slots<THREADS>(idx, slots, first, E, ms);
  const uint32_t word = lane < 32 ? ms.used[lane] : 0;
  const int before = used_before(word);
  const uint64_t hit = __ballot(before <= u && u < before + __popc(word));
  if (!hit) return -1;
  const int wl = __ffsll((unsigned long long)hit) - 1;
  const int e = 32 * wl + nth_bit(__builtin_amdgcn_readlane(word, wl),
                                  u - __builtin_amdgcn_readlane(before, wl));
  // the first slot of each token with e, 64 slots a wave and turn: counts,
  // then places
  auto is_row = [&](int f) {
    if (f >= slots || ms.ids[f] != e) return false;
    for (int g = f / k * k; g < f; g++)
      if (ms.ids[g] == e) return false;
    return true;
  };
  const int chunks = (slots + 63) / 64, wave = tid >> 6;
  for (int c = wave; c < chunks; c += THREADS / 64) {
    const int n = __popcll(__ballot(is_row(64 * c + lane)));
    if (lane == 0) chunk_rows[c] = n;
  }
  __syncthreads();
  int inc = lane < chunks ? chunk_rows[lane] : 0;
  const int own = inc;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(inc, o, 64);
    if (lane >= o) inc += v;
  }
  *count = __builtin_amdgcn_readlane(inc, 63);
  for (int c = wave; c < chunks; c += THREADS / 64) {
    const bool row = is_row(64 * c + lane);
    const uint64_t rows = __ballot(row);
    const int at = __builtin_amdgcn_readlane(inc - own, c);
    if (row) list[at + __popcll(rows & below(lane))] = (uint16_t)(64 * c + lane);
  }
  __syncthreads();
  return e;
}

// One FFN's matrices and slots.  idx null: the shared expert, every token a
// row with weight one (k = 1).
struct Ffn {
  W4Mat gate, up;
  const int32_t *idx;
  const float *w;
  int slots, k, first, E;
  uint16_t *act;
};

constexpr int kGuWaves = 4;

// Grid (output tiles, used experts [+ 1: the shared expert]).
template <class F, int NB>
__global__ __launch_bounds__(kGuWaves * 64) void w4_gate_up_kernel(Ffn routed, Ffn shared, int used,
                                                                   const uint16_t *x) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ float red[kGuWaves * 2 * NB * 256];
  __shared__ float wrow[16 * NB];
  const bool is_shared = (int)blockIdx.y == used;
  const Ffn &q = is_shared ? shared : routed;
  const W4Mat mm[2] = {q.gate, q.up};
  const int I = q.gate.n, K = q.gate.k, ks = q.gate.ks;
  if ((int)blockIdx.x >= q.gate.nt) return;
  uint16_t *list = (uint16_t *)dyn;
  int expert = 0, count = q.slots;
  if (!is_shared) {
    const Many ms = {(int16_t *)(list + q.slots), (uint32_t *)(dyn + 4 * ((q.slots + 3) & ~3))};
    expert = find_rows<kGuWaves * 64>(q.idx, q.slots, q.k, q.first, q.E, blockIdx.y, list, ms,
                                      &count);
    if (expert < 0) return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const size_t base = ((size_t)expert * q.gate.nt + blockIdx.x) * ks;
  const size_t tile[2] = {base, base};
  for (int r0 = 0; r0 < count; r0 += 16 * NB) {
    const int nr = min(16 * NB, count - r0);
    auto slot = [&](int r) { return is_shared ? r0 + r : (int)list[r0 + r]; };
    RowPtr xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p].p = x + (size_t)(slot(min(16 * p + (lane & 15), nr - 1)) / q.k) * K;
    if (tid < nr) {
      float w = 1.0f;
      if (!is_shared) {
        const int f = slot(tid);
        w = q.w[f];
        for (int g = f + 1; g < f / q.k * q.k + q.k; g++)
          if (local_id(q.idx[g], q.first, q.E) == expert) w += q.w[g];
      }
      wrow[tid] = w;
    }
    f32x4 acc[2][NB];
    zero_acc(acc);
    w4_stream<F>(mm, tile, xr, K, ks * wave / kGuWaves, ks * (wave + 1) / kGuWaves, acc);
    w4_join<kGuWaves>(acc, red);
    for (int i = tid; i < NB * 256; i += kGuWaves * 64) {
      const int l = i & 63, v = (i >> 6) & 3;
      const int row = 16 * (i >> 8) + 4 * (l >> 4) + v, n = 16 * blockIdx.x + (l & 15);
      // rounded to bf16 once, weight included: the matrix operand of down
      if (row < nr && n < I)
        q.act[(size_t)slot(row) * I + n] =
            to_bf16(wrow[row] * silu_f(red[i]) * red[NB * 256 + i]);
    }
    __syncthreads();
  }
}

struct Down {
  W4Mat m, shared;  // shared.ks == 0: no shared expert
  const int32_t *idx;
  int slots, k, first, E, T;
  const uint16_t *act, *act_s;
};

// Grid (output tiles, token blocks of 16 NB).  The steps of all used experts
// and of the shared one are one sequence, split over the waves.
template <class F, int NB, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void w4_down_kernel(Down q, uint16_t *__restrict__ out) {
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  __shared__ float red[WAVES * NB * 256];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int t0 = blockIdx.y * 16 * NB, ks = q.m.ks, k = q.k;
  const bool few = q.slots <= 64;
  const Many ms = {(int16_t *)dyn, (uint32_t *)(dyn + 2 * ((q.slots + 7) & ~7))};
  uint16_t *ulist = (uint16_t *)(ms.used + 32);
  Few s{};
  int used;
  if (few) {
    s = few_slots(q.idx, q.slots, q.first, q.E);
    used = __popcll(s.firsts);
  } else {
    many_slots<WAVES * 64>(q.idx, q.slots, q.first, q.E, ms);
    const uint32_t word = lane < 32 ? ms.used[lane] : 0;
    int at = used_before(word);
    used = __builtin_amdgcn_readlane(at + __popc(word), 31);
    if (wave == 0)
      for (uint32_t b = word; b; b &= b - 1) ulist[at++] = (uint16_t)(32 * lane + __ffs(b) - 1);
    __syncthreads();
  }
  const int total = used * ks + q.shared.ks;
  int a = total * wave / WAVES;
  const int b = total * (wave + 1) / WAVES;
  const __amdgpu_buffer_rsrc_t ra = __builtin_amdgcn_make_buffer_rsrc(
      (void *)q.act, (short)0, (int)((size_t)q.slots * q.m.k * 2), 0x00020000);
  f32x4 acc[1][NB];
  zero_acc(acc);
  int u = a / ks;
  uint64_t firsts = s.firsts;
  for (int i = 0; i < u && firsts; i++) firsts &= firsts - 1;
  RowBuf xr[NB];
  while (a < b && u < used) {
    const int end = min(b, (u + 1) * ks);
    int e;
    uint64_t members = 0;
    if (few) {
      const int at = __ffsll((unsigned long long)firsts) - 1;
      firsts &= firsts - 1;
      e = __builtin_amdgcn_readlane(s.e, at);
      members = read_mask(s.mine, at);
    } else {
      e = ulist[u];
    }
    bool any = false;
#pragma unroll
    for (int p = 0; p < NB; p++) {
      const int t = t0 + 16 * p + (lane & 15);
      int f = -1;
      if (t < q.T) {
        if (few) {
          const uint64_t mt = members >> (t * k) & below(k);
          if (mt) f = t * k + __ffsll((unsigned long long)mt) - 1;
        } else {
          for (int j = k - 1; j >= 0; j--)
            if (ms.ids[t * k + j] == e) f = t * k + j;
        }
      }
      xr[p] = {ra, f >= 0 ? (uint32_t)f * (uint32_t)(q.m.k * 2) : kNoRow};
      any |= f >= 0;
    }
    // an expert that no token of this block uses adds nothing
    if (__ballot(any)) {
      const W4Mat mm[1] = {q.m};
      const size_t tile[1] = {((size_t)__builtin_amdgcn_readfirstlane(e) * q.m.nt + blockIdx.x) * ks};
      w4_stream<F>(mm, tile, xr, q.m.k, a - u * ks, end - u * ks, acc);
    }
    a = end;
    u++;
  }
  if (a < b) {
    const W4Mat mm[1] = {q.shared};
    const size_t tile[1] = {(size_t)blockIdx.x * q.shared.ks};
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void *)q.act_s, (short)0, (int)((size_t)q.T * q.shared.k * 2), 0x00020000);
#pragma unroll
    for (int p = 0; p < NB; p++) {
      const int t = t0 + 16 * p + (lane & 15);
      xr[p] = {rs, t < q.T ? (uint32_t)t * (uint32_t)(q.shared.k * 2) : kNoRow};
    }
    w4_stream<F>(mm, tile, xr, q.shared.k, a - used * ks, b - used * ks, acc);
  }
  w4_join<WAVES>(acc, red);
  for (int i = tid; i < NB * 256; i += WAVES * 64) {
    const int l = i & 63, v = (i >> 6) & 3;
    const int t = t0 + 16 * (i >> 8) + 4 * (l >> 4) + v, n = 16 * blockIdx.x + (l & 15);
    if (t < q.T && n < q.m.n) out[(size_t)t * q.m.n + n] = to_bf16(red[i]);
  }
}

}  // namespace

void launch_w4_ffn(const W4Layer &a, hipStream_t s) {
  Ffn r{w4_view(a.up, a.w_gate), w4_view(a.up, a.w_up), a.idx, a.w, a.T * a.k, a.k, a.first,
        a.up.groups, a.act};
  Ffn sh = r;
  Down d{w4_view(a.down, a.w_down), {}, a.idx, r.slots, a.k, a.first, r.E, a.T, a.act, nullptr};
  if (a.shared) {
    sh = {w4_view(a.up_s, a.ws_gate), w4_view(a.up_s, a.ws_up), nullptr, nullptr, a.T, 1, 0, 1,
          a.act_s};
    d.shared = w4_view(a.down_s, a.ws_down);
    d.act_s = a.act_s;
  }
  const int used = std::min(r.E, r.slots), avg = r.slots / r.E;
  const dim3 gu(a.shared ? std::max(a.up.nt, a.up_s.nt) : a.up.nt, used + (a.shared ? 1 : 0));
  const size_t lds_gu = (size_t)4 * ((r.slots + 3) & ~3) + 128;
  const size_t lds_dn = (size_t)2 * ((r.slots + 7) & ~7) + 128 + 2 * 1024;
  with_format(a.up, [&](auto f) {
    using F = decltype(f);
    auto up = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, gu, dim3(kGuWaves * 64), lds_gu, s, r, sh, used, a.x);
    };
    if (avg <= 16) up(w4_gate_up_kernel<F, 1>);
    else if (avg <= 32) up(w4_gate_up_kernel<F, 2>);
    else up(w4_gate_up_kernel<F, 4>);
    auto down = [&](auto kernel, int nb, int waves) {
      hipLaunchKernelGGL(kernel, dim3(a.down.nt, (a.T + 16 * nb - 1) / (16 * nb)), dim3(waves * 64),
                         lds_dn, s, d, a.out);
    };
    if (a.T <= 16 && a.down.nt >= 256) down(w4_down_kernel<F, 1, 8>, 1, 8);
    else if (a.T <= 16) down(w4_down_kernel<F, 1, 16>, 1, 16);
    else if (a.T <= 32) down(w4_down_kernel<F, 2, 16>, 2, 16);
    else down(w4_down_kernel<F, 4, 8>, 4, 8);
  });
}

}  // namespace moe
