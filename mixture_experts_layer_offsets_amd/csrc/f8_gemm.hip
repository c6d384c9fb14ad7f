// Products of many rows in 8 bits with a scale per block of 128 (f8_device.h): the
// forward and data-gradient product of grouped rows, and the weight gradient.
//
//   acc[n][r] += (sx[r][b] sw[n][b]) dot(w codes, x codes)    a block b of 128 a stage
//
// A workgroup of eight waves computes 256 rows (or 128) x 256 outputs, one a CU: its
// waves hold 128 x 64 results each (64 x 64), and two stages lie in LDS (128 KB, or 96;
// with the outputs' scales 136 or 104), which loads fill directly.  The matrix unit
// sums the 128 products of a block from zero, and the scales multiply that sum in fp32.
//
// What bounds it: at 16384 rows x 4096 x 7168 in 6 groups 510 to 524 us with the
// rows' quantising (59), 2.0 PFLOP/s in the product, where the library's 8-bit product with one
// scale a tensor takes 308 us.  Of the cycles in which a CU has work (80 % of the launch: the
// last of five rounds of tiles is a fifth full) the matrix unit is busy in 61 %, and the other
// vector instructions, 5 for each product, take 38: the two hardly overlap, though without
// loads, in registers alone, the instruction reaches 4.7 PFLOP/s, and 4.3 with a multiply-add
// for each of its results.  The weight gradient's scales differ along both sides, two
// operations a result (3.2 PFLOP/s in registers) and 10 vector instructions a product: 572 of
// 672 us (962 GFLOP), 43 % and 54 % of the busy cycles.  Reads of LDS take a quarter of
// them in both, at 4 cycles each, conflicts 2 and 4 % of those.  64 groups of 384 rows x 2816
// x 2048: 221 to 228 us, 39 % and 34 %, the waves waiting 39 % of their time: 27 of a tile's
// 35 us are its loop and the rest its offsets, first loads and results; half-empty last tiles
// cost the rest.
// Tried and not faster: the groups' last tiles last (254 us of 230: their weights are not
// in the cache then), tiles of 64 rows, four waves a SIMD (spills), 128 outputs a tile
// (1024 rows x 4096 x 4096 32 us of 37, but 57 of 46 at 2048 rows).
#include <algorithm>

#include "f8_device.h"
#include "f8_scales.h"

namespace moe {

namespace {

constexpr int kTN = 256;       // outputs of a tile
constexpr int kThreads = 512;  // eight waves, two a SIMD
constexpr int kRing = 4;       // products of a wave in flight (no more than NJ)

// Operands of either product.  "rows" are the instruction's second operand: rows of
// x, or for the weight gradient its columns.
struct Args {
  const uint8_t *xc, *wc;  // codes [step][xpitch][128], tiles [n / 16][wsteps]
  const float *xs, *ws;    // scales [step][spitch]; [n / 16][wsteps], or [step][npitch]
  const int32_t *offsets;
  uint16_t *out;
  float *parts;  // split weight gradient: sums [split][group][xrows][npitch]
  long ostride;
  int rows, groups, n, nt, f16, splits;
  int xrows, xpitch, spitch;  // weight gradient: rows of the result, their pitches
  int wsteps, npitch, nN, MT;
};

template <int TM>
struct Geo {
  static constexpr int WN = TM == 256 ? 2 : 4;  // waves along the outputs
  static constexpr int NI = kTN / WN / 16, NJ = 4;              // 16 x 16 results of a wave
  static constexpr int XB = TM * kF8Block, WB = kTN * kF8Block;  // bytes of a stage
  static constexpr int XQ = XB / 8192;  // loads of a wave and stage, of rows
};

// Tiles of T rows over the groups, one group behind the other, counted by every wave for
// itself, 64 groups at a time.
struct Tiles {
  const int32_t *offsets;
  int groups, rows, T;
  int total;           // tiles of all groups
  int begin, upto, n;  // lane's group of the 64 looked at last: its rows' begin, tiles up to
                       // its end, its own
  int g0;
  __device__ __forceinline__ int count(int at, int before) {  // tiles up to the end of these 64
    const int lane = threadIdx.x & 63;
    g0 = at;
    F8Span sp{0, 0};
    if (at + lane < groups) sp = f8_span(offsets, at + lane, rows);
    begin = sp.begin;
    n = (sp.end - sp.begin + T - 1) / T;
    upto = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int v = __shfl_up(upto, o, 64);
      if (lane >= o) upto += v;
    }
    upto += before;
    return min(__builtin_amdgcn_readlane(upto, 63), 1 << 30);  // spans that overlap add up to more
  }
  __device__ __forceinline__ Tiles(const int32_t *o, int g, int r, int t)
      : offsets(o), groups(g), rows(r), T(t), total(0) {
    for (int at = 0; at < groups; at += 64) total = count(at, total);
    total = min(total, rows / T + groups);  // what ascending offsets reach
  }
  // The group of tile i < total, and the first row of that tile.
  __device__ __forceinline__ int group_of(int i, int *row) {
    if (groups > 64) {
      int before = 0;
      for (int at = 0; at < groups; at += 64) {
        before = count(at, before);
        if (i < before) break;
      }
    }
    const int l = __ffsll((unsigned long long)__ballot(i < upto && i >= upto - n)) - 1;
    const int first = __builtin_amdgcn_readlane(upto - n, l);
    *row = __builtin_amdgcn_readlane(begin, l) + (i - first) * T;
    return g0 + l;
  }
};

// X, A, B: rows, first halves and second halves of the waves' tiles, of two stages: arrays
// of their own, so that the compiler can tell what is read from what is being filled.
template <int TM, bool COLS, bool SPLIT>
__device__ __forceinline__ void f8_tile(const Args &p, uint8_t *X0, uint8_t *X1, uint8_t *A0,
                                        uint8_t *A1, uint8_t *B0, uint8_t *B1) {
  using G = Geo<TM>;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int mt, nt, g, m0, valid, step0, steps;
  size_t xrow;  // first row of the tile, in the operand
  uint16_t *out;
  if constexpr (COLS) {
    const int per = p.MT * p.nN, at = blockIdx.x / per;  // split by split, group by group
    g = SPLIT ? at % p.groups : at;
    tile_of_block(blockIdx.x - at * per, p.MT, p.nN, mt, nt);
    const F8Span sp = f8_span(p.offsets, g, p.rows);
    step0 = sp.begin / kF8Block + g;
    steps = (sp.end - sp.begin + kF8Block - 1) / kF8Block;
    if constexpr (SPLIT) {
      const int z = at / p.groups, from = (int)((long)steps * z / p.splits);
      steps = (int)((long)steps * (z + 1) / p.splits) - from;
      step0 += from;
    }
    m0 = mt * TM;
    valid = min(TM, p.xrows - m0);
    xrow = m0;
    out = p.out + ((size_t)g * p.xrows + m0) * p.ostride;
  } else {
    Tiles tiles(p.offsets, p.groups, p.rows, TM);
    if (blockIdx.x >= (unsigned)(tiles.total * p.nN)) return;
    tile_of_block(blockIdx.x, tiles.total, p.nN, mt, nt);
    g = tiles.group_of(mt, &m0);
    if (g < 0) return;
    const F8Span sp = f8_span(p.offsets, g, p.rows);
    valid = min(TM, sp.end - m0);
    step0 = 0;
    steps = p.wsteps;
    xrow = m0;
    out = p.out + (size_t)m0 * p.ostride;
  }
  const int n0 = nt * kTN, wn0 = (wave % G::WN) * (16 * G::NI), wm0 = (wave / G::WN) * (16 * G::NJ);
  const uint8_t *xc = p.xc + ((size_t)step0 * p.xpitch + xrow) * kF8Block;
  const float *xs = p.xs + (size_t)step0 * p.spitch + xrow;
  // the forward's tiles and scales are a matrix a group
  const size_t wt = (COLS ? 0 : (size_t)g * p.nt) + n0 / 16;
  const uint8_t *wc = p.wc + (wt * p.wsteps + step0) * kF8Tile;
  const float *wsc = COLS ? p.ws + (size_t)step0 * p.npitch + n0
                          : p.ws + ((size_t)g * p.nt + min((n0 + wn0) / 16, p.nt - 1)) * p.wsteps;
  const int tiles = min(kTN / 16, p.nt - n0 / 16);
  const int lane16 = lane * 16;
  // row (lane / 8) of the wave's first 8, its chunks exchanged by the row
  const int ox = wave * G::XQ * 1024 + (lane >> 3) * kF8Block + (((lane & 7) ^ (lane >> 3)) << 4);
  // Stage kt to L, load by load: q < XQ rows, then the outputs' scales (COLS).  Past the
  // end: the last stage again, not used (without a branch, which the scheduler would
  // not move the loop's work across).
  auto dma_x = [&](uint8_t *X, int kt, int q) {
    const int k1 = min(kt, steps - 1);
    const f8_rsrc_t rX = f8_buffer(xc + (size_t)k1 * p.xpitch * kF8Block, valid * kF8Block);
    const lds_ptr_t to = (lds_ptr_t)(X + wave * G::XQ * 1024);
    // the constant offset moves both addresses
    if (q == 0) __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, to, 16, ox, 0, 0, 0);
    if (q == 1) __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, to, 16, ox, 0, 1024, 0);
    if (q == 2) __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, to, 16, ox, 0, 2048, 0);
    if (q == 3) __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, to, 16, ox, 0, 3 * 1024, 0);
  };
  // ... and one tile a wave of the first or second half of each wave's tiles, in two
  auto dma_w = [&](uint8_t *W, int kt, int half, int q) {
    const int k1 = min(kt, steps - 1);
    const int at = wave / (G::NI / 2) * G::NI + wave % (G::NI / 2) + half * (G::NI / 2);
    const int t = min(at, tiles - 1);  // past the last one: that one again
    const f8_rsrc_t rW = f8_buffer(wc + ((size_t)t * p.wsteps + k1) * kF8Tile, kF8Tile);
    const lds_ptr_t to = (lds_ptr_t)(W + wave * kF8Tile);
    if (q == 0) __builtin_amdgcn_raw_ptr_buffer_load_lds(rW, to, 16, lane16, 0, 0, 0);
    if (q == 1) __builtin_amdgcn_raw_ptr_buffer_load_lds(rW, to, 16, lane16, 0, 1024, 0);
  };
  // ... the scales of the first or second half's outputs behind their tiles (COLS), 4
  // bytes a lane, all waves alike: the last six's are zeros
  const int osw[2] = {f8_scale_at(tid, 0, G::NI), f8_scale_at(tid, 1, G::NI)};
  auto dma_s = [&](uint8_t *W, int kt, int half) {
    const int k1 = min(kt, steps - 1);
    const f8_rsrc_t r = f8_buffer(wsc + (size_t)k1 * p.npitch, f8_scale_bytes(wave, p.npitch - n0));
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(W + G::WB / 2 + wave * 256), 4, osw[half],
                                             0, 0, 0);
  };
  // the rows' scales, and behind them that of the wave's outputs (forward)
  constexpr int NS = COLS ? G::NJ : G::NJ + 1;
  const int os = (wm0 + l16) * 4;
  auto scales = [&](int kt, float *s) {
    const int k1 = min(kt, steps - 1);
    const f8_rsrc_t r = f8_buffer(xs + (size_t)k1 * p.spitch, valid * 4);
#pragma unroll
    for (int j = 0; j < G::NJ; j++)
      s[j] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(r, os + 64 * j, 0, 0));
    if constexpr (!COLS)
      s[G::NJ] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(f8_buffer(wsc, p.wsteps * 4), 0, k1 * 4, 0));
  };
  // load n of stage kt's refills: of Bn for the next stage, of Xc and Ac for the one after
  auto refill_load = [&](uint8_t *Xc, uint8_t *Ac, uint8_t *Bn, int kt, int n) {
    if (n >= 0 && n < 2) dma_w(Bn, kt + 1, 1, n);
    else if (n >= 2 && n < 2 + G::XQ) dma_x(Xc, kt + 2, n - 2);
    else if (n >= 2 && n < 4 + G::XQ) dma_w(Ac, kt + 2, 0, n - 2 - G::XQ);
    else if (COLS && n == 4 + G::XQ) dma_s(Ac, kt + 2, 0);
    else if (COLS && n == 5 + G::XQ) dma_s(Bn, kt + 1, 1);
  };
  auto refill = [&](uint8_t *Xc, uint8_t *Ac, uint8_t *Bn, int kt) {
#pragma unroll
    for (int n = 0; n < G::XQ + 6; n++) refill_load(Xc, Ac, Bn, kt, n);
  };
  f32x4 acc[G::NI][G::NJ];
#pragma unroll
  for (int i = 0; i < G::NI; i++)
#pragma unroll
    for (int j = 0; j < G::NJ; j++) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  const int xo = (wm0 + l16) * kF8Block + ((h ^ (l16 & 7)) << 4);  // and, 64 bytes on, h + 4
  const int wo = (wave % G::WN) * (G::NI / 2) * kF8Tile + lane16;  // the wave's tiles, of either half
  const int swo = G::WB / 2 + (wave % G::WN) * (G::NI / 2) * 64 + 16 * h;
  i32x8_t xf[G::NJ], wf[2];
  f32x4 d[kRing], sw[2];
  auto load_x = [&](const uint8_t *X, int j) {
    xf[j] = f8_frag(*(const u32x4_t *)(X + xo + j * 16 * kF8Block),
                         *(const u32x4_t *)(X + (xo ^ 64) + j * 16 * kF8Block));
  };
  auto load_w = [&](const uint8_t *A, const uint8_t *B, int i) {
    const uint8_t *W = (i < G::NI / 2 ? A : B) + wo + i % (G::NI / 2) * kF8Tile;
    wf[i & 1] = f8_frag(*(const u32x4_t *)W, *(const u32x4_t *)(W + 1024));
  };
  auto load_s = [&](const uint8_t *A, const uint8_t *B, int i) {
    if constexpr (COLS)
      sw[i & 1] = *(const f32x4 *)((i < G::NI / 2 ? A : B) + swo + i % (G::NI / 2) * 64);
  };
  // product q = i NJ + j of a stage, whose rows have the scales s
  auto scale = [&](int q, const float *s) {
    const int i = q / G::NJ, j = q % G::NJ;
#pragma unroll
    for (int v = 0; v < 4; v++)
      acc[i][j][v] = fmaf(COLS ? s[j] * sw[i & 1][v] : s[j], d[q % kRing][v], acc[i][j][v]);
  };
  // Xc, Ac, Bc hold stage kt, its rows and first tile read; the last products of the stage
  // before are not scaled yet (so, sc, s1: the rows' scales of stages kt - 1, kt, kt + 1).
  // Before the last tile of the first half the waves meet: what was sent for a stage ago is
  // there then (Bc; Xn and An with stage kt + 1), and Xc, Ac and Bn (stage kt - 1) have been
  // read and are refilled, load by load between the products (in a burst the loads would
  // stall the wave).  The next stage's rows are read as the last tile's products leave
  // theirs.
  float so[G::NJ], sc[NS], s1[NS];
  auto stage = [&](uint8_t *Xc, uint8_t *Ac, uint8_t *Bc, uint8_t *Xn, uint8_t *An, uint8_t *Bn,
                   int kt) {
    constexpr int NQ = G::NI * G::NJ, kLag = kRing - 1, kHalf = G::NI / 2;
    float sn[NS];  // of stage kt + 2: loads that nothing waits for before the next meeting
#pragma unroll
    for (int j = 0; j < G::NJ; j++)
      if constexpr (!COLS) sc[j] *= sc[G::NJ];
#pragma unroll
    for (int i = 0; i < G::NI; i++) {
      if (i == kHalf - 1) {
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
        lds_barrier();
        scales(kt + 2, sn);
      }
      if (i + 1 < G::NI) load_w(Ac, Bc, i + 1);
      else load_w(An, Bn, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < G::NJ; j++) {
        const int q = i * G::NJ + j;
        d[q % kRing] = f8_dot(wf[i & 1], xf[j]);
        if (i == G::NI - 1) load_x(Xn, j);
        if (q >= kLag) scale(q - kLag, sc);
        else scale(NQ - kLag + q, so);
        // the scales of two tiles back have been used
        if (j == kLag - 1) {
          if (i + 1 < G::NI) load_s(Ac, Bc, i + 1);
          else load_s(An, Bn, 0);
        }
        refill_load(Xc, Ac, Bn, kt, q - (kHalf - 1) * G::NJ);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int j = 0; j < NS; j++) {
      if (j < G::NJ) so[j] = sc[j];
      sc[j] = s1[j];
      s1[j] = sn[j];
    }
  };
  if (steps > 0) {
#pragma unroll
    for (int q = 0; q < G::XQ; q++) dma_x(X0, 0, q);
#pragma unroll
    for (int q = 0; q < 2; q++) {
      dma_w(A0, 0, 0, q);
      dma_w(B0, 0, 1, q);
    }
    if constexpr (COLS) {
      dma_s(A0, 0, 0);
      dma_s(B0, 0, 1);
    }
    scales(0, sc);
    // stage 0 is there before the first of stage 1, which the middle of stage 0 waits for:
    // what follows is kLater loads
    constexpr int kLater = G::XQ + 2 + (COLS ? 1 : 0) + NS;
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < G::XQ; q++) dma_x(X1, 1, q);
#pragma unroll
    for (int q = 0; q < 2; q++) dma_w(A1, 1, 0, q);
    if constexpr (COLS) dma_s(A1, 1, 0);
    scales(1, s1);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < G::NJ; j++) so[j] = 0.0f;
#pragma unroll
    for (int q = 0; q < kRing; q++) d[q] = sw[q & 1] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
    __builtin_amdgcn_s_waitcnt(vmcnt_wait(kLater));
    barrier_after_wait();
    if (wm0 < valid) {
#pragma unroll
      for (int j = 0; j < G::NJ; j++) load_x(X0, j);
      load_w(A0, B0, 0);
      load_s(A0, B0, 0);
      int kt = 0;
      for (; kt + 2 <= steps; kt += 2) {
        stage(X0, A0, B0, X1, A1, B1, kt);
        stage(X1, A1, B1, X0, A0, B0, kt + 1);
      }
      if (kt < steps) stage(X0, A0, B0, X1, A1, B1, kt);
#pragma unroll
      for (int q = 0; q < kRing - 1; q++) scale(G::NI * G::NJ - (kRing - 1) + q, so);
    } else {
      // a wave without rows: its loads and the meetings only, which leaves its SIMD to the
      // wave that shares it (waves w and w + 4; their rows lie half a tile apart)
      for (int kt = 0; kt < steps; kt++) {
        __builtin_amdgcn_s_waitcnt(kVmcnt0);
        barrier_after_wait();
        if (kt & 1) refill(X1, A1, B0, kt);
        else refill(X0, A0, B1, kt);
      }
    }
  }
  __builtin_amdgcn_s_waitcnt(kVmcnt0);  // the last loads, not used
  __syncthreads();
  if constexpr (SPLIT) {
    float *to = p.parts + ((size_t)(blockIdx.x / (p.MT * p.nN)) * p.xrows + m0) * p.npitch + n0;
#pragma unroll
    for (int j = 0; j < G::NJ; j++)
#pragma unroll
      for (int i = 0; i < G::NI; i++) {
        const int r = wm0 + 16 * j + l16, c = wn0 + 16 * i + 4 * h;
        if (r < valid && n0 + c < p.npitch) *(f32x4 *)(to + (size_t)r * p.npitch + c) = acc[i][j];
      }
    return;
  }
  // results to LDS, half of the rows a pass, 512 bytes a row with its 16-byte chunks
  // exchanged by the row, then out as whole rows
  constexpr int kRows = TM / 4;  // rows of X0, and of X1
  const int c = tid & 31, cols = p.n - n0 - 8 * c;
  for (int r0 = 0; r0 < TM; r0 += 2 * kRows) {
#pragma unroll
    for (int j = 0; j < G::NJ; j++) {
      const int r = wm0 + 16 * j + l16 - r0;
      if (wm0 + 16 * j < r0 || wm0 + 16 * j >= r0 + 2 * kRows) continue;
#pragma unroll
      for (int i = 0; i < G::NI; i++) {
        const int at = wn0 + 16 * i + 4 * h;
        uint16_t o[4];
#pragma unroll
        for (int v = 0; v < 4; v++) o[v] = f8_to16(acc[i][j][v], p.f16);
        const int b = r % kRows * 512 + ((((at >> 3) ^ r) & 31) << 4) + (at & 4) * 2;
        const uint2 w = make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
        if (wm0 + 16 * j - r0 < kRows) *(uint2 *)(X0 + b) = w;
        else *(uint2 *)(X1 + b) = w;
      }
    }
    __syncthreads();
    for (int r = tid >> 5; r < min(2 * kRows, valid - r0); r += kThreads / 32) {
      const int b = r % kRows * 512 + (((c ^ r) & 31) << 4);
      u32x4_t v;
      if (r < kRows) v = *(const u32x4_t *)(X0 + b);
      else v = *(const u32x4_t *)(X1 + b);
      uint16_t *dst = out + (size_t)(r0 + r) * p.ostride + n0 + 8 * c;
      if (cols >= 8)
        *(u32x4_a2 *)dst = (u32x4_a2){v[0], v[1], v[2], v[3]};
      else
#pragma unroll
        for (int e = 0; e < 8; e++)
          if (e < cols) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
    }
    __syncthreads();
  }
}

template <int TM, bool COLS, bool SPLIT = false>
__global__ __launch_bounds__(kThreads, 2) void f8_gemm_kernel(Args p) {
  using G = Geo<TM>;
  __shared__ __attribute__((aligned(1024))) uint8_t X0[G::XB], X1[G::XB];
  constexpr int kHalf = G::WB / 2 + (COLS ? 2048 : 0);  // and scales
  __shared__ __attribute__((aligned(1024))) uint8_t A0[kHalf], A1[kHalf], B0[kHalf], B1[kHalf];
  f8_tile<TM, COLS, SPLIT>(p, X0, X1, A0, A1, B0, B1);
}

// dw from the splits' sums, added in their order.  A thread takes 4 values of a row.
__global__ __launch_bounds__(256) void f8_join_kernel(const float *__restrict__ parts, int splits,
                                                      long rows, int n, int npitch, int f16,
                                                      uint16_t *__restrict__ out) {
  const int per = (n + 3) / 4;
  const long at = (long)blockIdx.x * 256 + threadIdx.x, r = at / per;
  const int c = (int)(at - r * per) * 4;
  if (r >= rows) return;
  const float *from = parts + r * npitch + c;
  f32x4 s = *(const f32x4 *)from;
#pragma unroll 8
  for (int z = 1; z < splits; z++) {
    const f32x4 v = *(const f32x4 *)(from + (size_t)z * rows * npitch);
#pragma unroll
    for (int e = 0; e < 4; e++) s[e] += v[e];
  }
#pragma unroll
  for (int e = 0; e < 4; e++)
    if (c + e < n) out[r * n + c + e] = f8_to16(s[e], f16);
}

// Tiles of 256 rows read less for the same products; those of 128 take about 0.75 of
// their time, and fill the chip where tiles are few (4096 x 4096, us with 256 / 128: 1024
// rows 53 / 37, 2048 rows 57 / 45, 4096 rows 75 / 83; 64 groups of 384 rows, 2816 x 2048:
// 224 / 273): by the rounds of 256 workgroups that either takes.
bool tall_tiles(long rows, long groups, int nN) {
  auto rounds = [&](int TM) { return ((rows + TM - 1) / TM * groups * nN + 255) / 256; };
  return 4 * rounds(256) <= 3 * rounds(128);
}

}  // namespace

void launch_f8_gemm(const F8Dims &d, int rows, const uint8_t *codes, const float *scales,
                    const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                    hipStream_t s) {
  Args a{};
  a.xc = codes; a.xs = scales;
  a.wc = (const uint8_t *)packed;
  a.ws = (const float *)(a.wc + d.code_bytes);
  a.offsets = offsets;
  a.out = out; a.ostride = ostride;
  a.rows = rows; a.groups = d.groups; a.n = d.n; a.nt = d.nt; a.f16 = d.f16;
  a.xpitch = a.spitch = rows;
  a.wsteps = d.ks;
  a.nN = (d.n + kTN - 1) / kTN;
  auto go = [&](auto kernel, int TM) {
    const long most = d.groups == 1 ? (rows + TM - 1) / TM : rows / TM + d.groups;  // row tiles
    hipLaunchKernelGGL(kernel, dim3((unsigned)(most * a.nN)), dim3(kThreads), 0, s, a);
  };
  const int avg = (rows + d.groups - 1) / d.groups;
  if (tall_tiles(avg, d.groups, a.nN)) go(f8_gemm_kernel<256, false>, 256);
  else go(f8_gemm_kernel<128, false>, 128);
}

// Few results of many rows: a group's stages in pieces of 4 or more on average, as many
// as the chip takes at once, whose sums a second kernel adds.  One group, us without and
// with: 256 x 256 of 1000 rows (7 stages) 17 and 18, so not there, of 4000 39 and 21, of
// 16000 124 and 25 (pieces of 8: 28); 1024 x 1024 of 16000 138 and 60; 2048 x 2048 of 4000
// 48 and 50, of 16000 162 and 135.
int f8_splits(const F8Dims &d, int rows) {
  const long tiles = (long)d.groups * ((d.k + 127) / 128) * ((d.n + 255) / 256);
  const long stages = rows / kF8Block / d.groups;
  if (stages < 12) return 1;
  return (int)std::max(1L, std::min({256 / tiles, stages / 4, 32L}));
}

void launch_f8_wgrad(const F8Dims &d, int rows, const uint8_t *xc, const float *xs,
                     const uint8_t *yc, const float *ys, const int32_t *offsets, uint16_t *dw,
                     float *parts, hipStream_t s) {
  Args a{};
  a.xc = xc; a.xs = xs; a.wc = yc; a.ws = ys;
  a.offsets = offsets;
  a.out = dw; a.ostride = d.n;
  a.rows = rows; a.groups = d.groups; a.n = d.n; a.nt = d.nt; a.f16 = d.f16;
  a.xrows = a.xpitch = d.k;
  a.spitch = (d.k + 15) & ~15;
  a.npitch = (d.n + 15) & ~15;
  a.wsteps = (int)f8_stages(rows, d.groups);
  a.nN = (d.n + kTN - 1) / kTN;
  auto go = [&](auto kernel, int TM) {
    a.MT = (d.k + TM - 1) / TM;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long)d.groups * a.MT * a.nN)), dim3(kThreads), 0, s,
                       a);
  };
  const int splits = f8_splits(d, rows);
  if (splits > 1) {
    a.MT = (d.k + 127) / 128;
    a.splits = splits;
    a.parts = parts;
    hipLaunchKernelGGL((f8_gemm_kernel<128, true, true>),
                       dim3((unsigned)(splits * d.groups * a.MT * a.nN)), dim3(kThreads), 0, s, a);
    const long all = (long)d.groups * d.k * ((d.n + 3) / 4);
    hipLaunchKernelGGL(f8_join_kernel, dim3((unsigned)((all + 255) / 256)), dim3(256), 0, s, parts,
                       splits, (long)d.groups * d.k, d.n, a.npitch, d.f16, dw);
  } else if (tall_tiles(d.k, d.groups, a.nN)) {
    go(f8_gemm_kernel<256, true>, 256);
  } else {
    go(f8_gemm_kernel<128, true>, 128);
  }
}

}  // namespace moe
