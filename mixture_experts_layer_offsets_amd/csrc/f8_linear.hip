// Products of few rows in 8 bits with a scale per block of 128 (f8_device.h): the
// weights go from memory straight into registers, and the waves of a workgroup split
// the contraction of one tile of 16 outputs, or a few.  Each wave's loads for up to four
// steps are on their way at once; the waves' sums meet in LDS, added in wave order.
//
// Bound by the launch and one or two round trips to memory (1 row, 2048 of 7168: 6.1 us,
// where a launch of a small kernel takes 3.8 and reading the 15 MB of weights 2.5), then by
// reading the weights (64 groups of 2816 x 2048: one row in each 56 us, 369 MB at 6.6 TB/s;
// 64 rows sent at random, which reach 43 of the groups, 41).
#include <algorithm>

#include "f8_device.h"

namespace moe {

namespace {

struct Few {
  const uint8_t *tiles;
  const float *ws;
  const int32_t *offsets;
  uint16_t *out;
  long ostride;
  int rows, n, k, nt, ks, f16;
  int early;  // passes whose first weights need not wait for the offsets
};

// The weights of one tile row, and its scales.
struct TileRow {
  f8_rsrc_t r;
  const float *ws;
  __device__ __forceinline__ TileRow(const Few &p, int g, int t)
      : r(f8_buffer(p.tiles + ((size_t)g * p.nt + t) * p.ks * kF8Tile, p.ks * kF8Tile)),
        ws(p.ws + ((size_t)g * p.nt + t) * p.ks) {}
  __device__ __forceinline__ void load(int st, u32x4_t *w) const {  // read once: not kept in the caches
#pragma unroll
    for (int i = 0; i < 2; i++)
      w[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                             r, (threadIdx.x & 63) * 16 + 1024 * i, st * kF8Tile, 2));
  }
};

__device__ __forceinline__ void add_scaled(f32x4 &acc, const f32x4 &d, float s) {
#pragma unroll
  for (int v = 0; v < 4; v++) acc[v] = fmaf(s, d[v], acc[v]);
}

// The waves' sums of NB blocks of 16 rows from row r0 on, nr of them, with tile t, added
// in wave order and written.
template <int WAVES, int NB>
__device__ __forceinline__ void put(const Few &p, const f32x4 *acc, float *red, int t, long r0, int nr) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int b = 0; b < NB; b++)
#pragma unroll
    for (int v = 0; v < 4; v++) red[((wave * NB + b) * 4 + v) * 64 + lane] = acc[b][v];
  lds_barrier();
  for (int q = tid; q < NB * 256; q += WAVES * 64) {
    float s = red[q];
#pragma unroll
    for (int w = 1; w < WAVES; w++) s += red[w * NB * 256 + q];
    const int row = 16 * (q >> 8) + (q & 15), n = 16 * t + 4 * ((q >> 4) & 3) + ((q >> 6) & 3);
    if (row < nr && n < p.n) p.out[(r0 + row) * p.ostride + n] = f8_to16(s, p.f16);
  }
  lds_barrier();
}

// Quantised rows, up to 16 NB a pass, with TW tiles of outputs, which share the reading
// of the rows; the loads of U steps go out together.  Grid (output tiles / TW, groups,
// passes that run side by side).
template <int WAVES, int TW, int NB, int U>
__global__ __launch_bounds__(WAVES * 64) void f8_few_kernel(Few p, const uint8_t *__restrict__ codes,
                                                            const float *__restrict__ scales) {
  __shared__ float red[WAVES * NB * 256];
  constexpr int kPass = 16 * NB;
  const int g = blockIdx.y, t0 = blockIdx.x * TW, tid = threadIdx.x, lane = tid & 63, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int s0 = p.ks * wave / WAVES, s1 = p.ks * (wave + 1) / WAVES;
  u32x4_t w[U][TW][2];
  float sw[U][TW];
  auto load = [&](int st) {
#pragma unroll
    for (int u = 0; u < U; u++)
#pragma unroll
      for (int t = 0; t < TW; t++) {  // past the end: the last step again, not used
        const TileRow tr(p, g, min(t0 + t, p.nt - 1));
        const int at = min(st + u, p.ks - 1);
        tr.load(at, w[u][t]);
        sw[u][t] = tr.ws[at];
      }
  };
  const bool early = (int)blockIdx.z < p.early;
  if (early) load(s0);
  __builtin_amdgcn_sched_barrier(0);
  const F8Span sp = f8_span(p.offsets, g, p.rows);
  for (long r0 = sp.begin + (long)kPass * blockIdx.z; r0 < sp.end; r0 += (long)kPass * gridDim.z) {
    const int nr = (int)min((long)kPass, sp.end - r0);
    if (!early || r0 >= sp.begin + (long)kPass * gridDim.z) load(s0);
    __builtin_amdgcn_sched_barrier(0);
    long r[NB];
    f32x4 acc[TW][NB];
#pragma unroll
    for (int b = 0; b < NB; b++) {
      r[b] = r0 + min(16 * b + (lane & 15), nr - 1);
#pragma unroll
      for (int t = 0; t < TW; t++) acc[t][b] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    }
    for (int st = s0; st < s1; st += U) {
      u32x4_t x[U][NB][2];
      float sx[U][NB];
#pragma unroll
      for (int u = 0; u < U; u++) {
        const int at = min(st + u, s1 - 1);
#pragma unroll
        for (int b = 0; b < NB; b++) {
          const size_t to = (size_t)at * p.rows + r[b];
          const u32x4_t *c = (const u32x4_t *)(codes + to * kF8Block);
          x[u][b][0] = c[h];
          x[u][b][1] = c[h + 4];
          sx[u][b] = scales[to];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; u++)
        if (st + u < s1)
#pragma unroll
          for (int t = 0; t < TW; t++)
#pragma unroll
            for (int b = 0; b < NB; b++)
              add_scaled(acc[t][b],
                         f8_dot(f8_frag(w[u][t][0], w[u][t][1]), f8_frag(x[u][b][0], x[u][b][1])),
                         sx[u][b] * sw[u][t]);
      if (st + U < s1) load(st + U);
    }
#pragma unroll
    for (int t = 0; t < TW; t++) put<WAVES, NB>(p, acc[t], red, t0 + t, r0, nr);
  }
}

// 16-bit rows, up to kStaged a pass: quantised by every workgroup for its own tile, into
// LDS, while its first weights are on their way.
constexpr int kStaged = 8;
constexpr int staged_lds(int ks) { return kStaged * (ks * (kF8Block + 4) + 16); }
constexpr int kStagedLds = 64 * 1024;

template <bool F16, int WAVES, int U>
__global__ __launch_bounds__(WAVES * 64) void f8_few_rows_kernel(Few p, const uint16_t *__restrict__ x,
                                                                 long stride) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // codes, then scales
  __shared__ float red[WAVES * 256];
  const int g = blockIdx.y, t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int pitch = p.ks * kF8Block + 16;  // rows' chunks in different banks
  float *xs = (float *)(lds + kStaged * pitch);
  const TileRow tr(p, g, t);
  const int s0 = p.ks * wave / WAVES, s1 = p.ks * (wave + 1) / WAVES;
  u32x4_t w[U][2];
  float sw[U];
  auto load = [&](int st) {
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int at = min(st + u, p.ks - 1);
      tr.load(at, w[u]);
      sw[u] = tr.ws[at];
    }
  };
  // one group's first weights need not wait for the offsets; many may be empty
  if (gridDim.y == 1) load(s0);
  const F8Span sp = f8_span(p.offsets, g, p.rows);
  for (long r0 = sp.begin + (long)kStaged * blockIdx.z; r0 < sp.end; r0 += (long)kStaged * gridDim.z) {
    const int nr = (int)min((long)kStaged, sp.end - r0);
    if (gridDim.y > 1 || r0 >= sp.begin + (long)kStaged * gridDim.z) load(s0);
    for (int q = tid >> 4; q < nr * p.ks; q += WAVES * 4) {
      const int row = q / p.ks, kb = q - row * p.ks, i = tid & 15;
      float s;
      const uint2 c = f8_quantize8<F16>(f8_load8(x + (r0 + row) * stride, kb * kF8Block + 8 * i, p.k), &s);
      *(uint2 *)(lds + row * pitch + kb * kF8Block + 8 * i) = c;
      if (i == 0) xs[row * p.ks + kb] = s;
    }
    lds_barrier();
    const int row = min(lane & 15, nr - 1);
    const uint8_t *mine = lds + row * pitch + 16 * h;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int st = s0; st < s1; st += U) {
#pragma unroll
      for (int u = 0; u < U; u++)
        if (st + u < s1) {
          const uint8_t *c = mine + (st + u) * kF8Block;
          add_scaled(acc,
                     f8_dot(f8_frag(w[u][0], w[u][1]),
                            f8_frag(*(const u32x4_t *)c, *(const u32x4_t *)(c + 64))),
                     xs[row * p.ks + st + u] * sw[u]);
        }
      if (st + U < s1) load(st + U);
    }
    put<WAVES, 1>(p, &acc, red, t, r0, nr);
  }
}

Few few_of(const F8Dims &d, int rows, const int32_t *offsets, const void *packed, uint16_t *out,
           long ostride) {
  const uint8_t *tiles = (const uint8_t *)packed;
  return {tiles, (const float *)(tiles + d.code_bytes), offsets, out, ostride,
          rows, d.n, d.k, d.nt, d.ks, d.f16, 0};
}

int average(const F8Dims &d, int rows) { return (rows + d.groups - 1) / d.groups; }

// Workgroups of tw tiles and 16 nb rows.
long blocks(const F8Dims &d, int rows, int tw, int nb) {
  return (long)((d.nt + tw - 1) / tw) * d.groups * ((average(d, rows) + 16 * nb - 1) / (16 * nb));
}

// How a product is split: waves of a workgroup, over the contraction; tiles and blocks of 16
// rows that they take.
struct Split {
  int waves, tw, nb;
};

// The more tiles and rows a workgroup takes, the less often either is read again, as
// long as some 200 workgroups are left (and half of its tiles exist: 16000 rows of 16 x
// 512 in tiles of one 12.7 us, of four 14.2).  One group of 4096 x 4096, us with (tiles,
// blocks of rows) of (4, 4) / (2, 4) / (2, 2) / (1, 2): 256 rows 24 / 30 / 32 / 45, 128
// rows 23 / 17 / 19 / 26, 64 rows 22 / 17 / 13 / 16, 24 rows 19 / 14 / 12 / 11.
// Up to 8 rows a group: one tile, and the more waves the fewer workgroups.
//
// The waves decide the order of addition, and 16-bit rows that launch_f8_few_rows quantises on
// the way get the bits of their codes: both take these.  That many workgroups of one tile and 8
// rows take four waves (1000 rows of 256 x 512, us from rows: 8.6, with eight 11.3; from codes
// 4.3 either way), fewer take eight (16 rows of 2048 x 4096: 8.3, with 16 8.1; from codes 6.0,
// with 16 7.9).
Split split_of(const F8Dims &d, int rows) {
  const int avg = average(d, rows);
  if (avg <= kStaged) {
    const long n = blocks(d, rows, 1, 1);
    return {n <= 256 ? 16 : n <= 512 ? 8 : 4, 1, 1};
  }
  if (f8_few_staged(d, rows) && (long)d.nt * d.groups * ((avg + kStaged - 1) / kStaged) > 512)
    return {4, d.nt > 1 ? 2 : 1, 2};
  auto many = [&](int tw, int nb) {
    return blocks(d, rows, tw, nb) >= 200 && 2 * d.nt > tw;
  };
  if (avg > 32 && many(4, 4)) return {8, 4, 4};
  if (avg > 32 && many(2, 4)) return {8, 2, 4};
  if (many(2, 2)) return {blocks(d, rows, 2, 2) > 512 ? 4 : 8, 2, 2};
  return {8, 1, 2};
}

// Passes of a group: what the average needs, and, for groups longer than it, further ones
// side by side where that takes no more workgroups than the chip runs at once (8 groups of
// 1024 x 2048, 512 rows falling off as 1 / g: 31 us without, 20 so, even ones 18 and 18).
int passes(const F8Dims &d, int rows, int pass, long tiles) {
  const long need = (average(d, rows) + pass - 1) / pass, most = ((long)rows + pass - 1) / pass;
  return (int)std::min(std::max(need, 2048 / (tiles * d.groups)), most);
}

}  // namespace

// Against f8_gemm.hip's tiles of 128 rows x 256 outputs: as long as 64 rows x 64 outputs a
// workgroup take the chip once.  One group, us here and there: 4096 x 4096, 256 rows 21 and
// 35, 300 rows 33 and 34; 1024 x 7168, 1000 rows 30 and 56, 4000 rows 105 and 76; 16 x
// 7168, 4000 rows 29 and 61.  8 groups of 1024 x 2048, even lengths and lengths that fall
// off as 1 / g: 512 rows 18 and 22, 20 and 23; 1024 rows 23 and 24, 25 and 23.  Up to 16
// rows on average the weights are all there is to read: 32 groups of 2816 x 2048, 512 rows
// in even groups 40 here and 54 there, falling off 57 and 55, 1024 even rows 65 and 57.
bool f8_few(const F8Dims &d, int rows) {
  return average(d, rows) <= 16 || blocks(d, rows, 4, 4) <= 256;
}

// Quantising again in every workgroup against a launch of its own (3 us): that is d.nt rows
// d.ks blocks.  Up to 8 rows a group: 8 rows of 2048 x 7168 (57 thousand) 10.6 us against
// 11.5, 32 rows in 32 groups of 2816 x 2048 (90) 21.6 against 23.6; 8 rows of 7168 x 4096
// (115) 12.7 against 11.5, 96 rows in the 32 groups (270) 33.6 against 31.3.  More rows, in
// passes of 8 whose workgroups the chip holds: 16 of 2048 x 4096 (66) 8.3 against 11.0, of
// 4096 x 4096 (131) 12.3 against 11.2; 1000 of 256 x 512 (64, 2000 workgroups) 8.1 against
// 10.2, 4000 of 256 x 128 (64, 8000) 17.5 against 10.8; 16 groups of 1000 x 512, 160 rows
// (40) 8.0 against 10.2, 32 of 512 x 512, 512 rows (66) 11.2 against 10.1.
bool f8_few_staged(const F8Dims &d, int rows) {
  const int avg = average(d, rows);
  const long most = avg <= kStaged ? 100000 : d.groups == 1 ? 66000 : 44000;
  return (long)d.nt * rows * d.ks <= most && staged_lds(d.ks) <= kStagedLds &&
         (avg <= kStaged || (long)d.nt * d.groups * ((avg + kStaged - 1) / kStaged) <= 2048);
}

void launch_f8_few(const F8Dims &d, int rows, const uint8_t *codes, const float *scales,
                   const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                   hipStream_t s) {
  Few p = few_of(d, rows, offsets, packed, out, ostride);
  const int avg = average(d, rows);
  auto go = [&](auto kernel, int waves, int tw, int nb) {
    // Of groups with four rows or more on average few are empty: the first weights need not
    // wait for the offsets.  Weights of empty groups are not read (64 rows, all in one of 64
    // groups of 2816 x 2048: 62 us if they were, 19 so).
    p.early = rows >= 4 * d.groups ? (avg + 16 * nb - 1) / (16 * nb) : 0;
    const int tiles = (d.nt + tw - 1) / tw;
    hipLaunchKernelGGL(kernel, dim3(tiles, d.groups, passes(d, rows, 16 * nb, tiles)), dim3(waves * 64),
                       0, s, p, codes, scales);
  };
  const Split c = split_of(d, rows);
  if (c.tw == 4) go(f8_few_kernel<8, 4, 4, 1>, 8, 4, 4);
  else if (c.nb == 4) go(f8_few_kernel<8, 2, 4, 2>, 8, 2, 4);
  else if (c.tw == 2 && c.waves == 4) go(f8_few_kernel<4, 2, 2, 2>, 4, 2, 2);
  else if (c.tw == 2) go(f8_few_kernel<8, 2, 2, 2>, 8, 2, 2);
  else if (c.nb == 2 && c.waves == 4) go(f8_few_kernel<4, 1, 2, 2>, 4, 1, 2);
  else if (c.nb == 2) go(f8_few_kernel<8, 1, 2, 2>, 8, 1, 2);
  else if (c.waves == 16) go(f8_few_kernel<16, 1, 1, 4>, 16, 1, 1);
  else if (c.waves == 8) go(f8_few_kernel<8, 1, 1, 4>, 8, 1, 1);
  else go(f8_few_kernel<4, 1, 1, 4>, 4, 1, 1);
}

void launch_f8_few_rows(const F8Dims &d, int rows, const F8Rows &x, const int32_t *offsets,
                        const void *packed, uint16_t *out, long ostride, hipStream_t s) {
  const Few p = few_of(d, rows, offsets, packed, out, ostride);
  const int z = passes(d, rows, kStaged, d.nt);
  auto go = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, dim3(d.nt, d.groups, z), dim3(waves * 64), staged_lds(d.ks), s, p,
                       x.p, x.stride);
  };
  const int waves = split_of(d, rows).waves;
  auto pick = [&](auto f16) {
    constexpr bool F16 = decltype(f16)::value;
    if (waves == 16) go(f8_few_rows_kernel<F16, 16, 4>, 16);
    else if (waves == 8) go(f8_few_rows_kernel<F16, 8, 4>, 8);
    else go(f8_few_rows_kernel<F16, 4, 4>, 4);
  };
  x.f16 ? pick(std::true_type{}) : pick(std::false_type{});
}

}  // namespace moe
