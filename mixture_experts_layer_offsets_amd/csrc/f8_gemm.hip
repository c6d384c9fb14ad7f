// Products of many rows in 8 bits with a scale per block of 128 (f8_device.h): the
// forward and data-gradient product of grouped rows, and the weight gradient.
#include <algorithm>

#include "f8_device.h"

namespace moe {

namespace {

constexpr int kTN = 256;       // outputs of a tile
constexpr int kThreads = 512;  // eight waves, two a SIMD

// Operands of either product.  "rows" are the instruction's second operand: rows of
// x, or for the weight gradient its columns.
struct Args {
  const uint8_t *xc, *wc;  // codes [step][xpitch][128], tiles [n / 16][wsteps]
  const float *xs, *ws;    // scales [step][spitch]; [n / 16][wsteps], or [step][npitch]
  const int32_t *offsets;
  uint16_t *out;
  long ostride;
  int rows, groups, n, nt, f16;
  int xrows, xpitch, spitch;  // weight gradient: rows of the result, their pitches
  int wsteps, npitch, nN, MT;
};

template <int TM>
struct Geo {
  static constexpr int WN = TM == 256 ? 2 : TM == 128 ? 4 : 8;  // waves along the outputs
  static constexpr int NI = kTN / WN / 16, NJ = 4;              // 16 x 16 results of a wave
  static constexpr int XB = TM * kF8Block, WB = kTN * kF8Block;  // bytes of a stage
  static constexpr int XQ = XB / 8192, WQ = WB / 8192;           // loads of a wave and stage
  static constexpr int Lds = XB + WB + kThreads * 4;             // and the outputs' scales
};

// One tile of TM rows x 256 outputs.  Operands move from memory straight into LDS, a
// block of 128 contraction values a stage, two stages in turn: while one is used the
// next one arrives.  Rows lie in LDS 128 bytes apart with their chunks exchanged by
// the row's low bits, tiles of weights in the order of the waves' reads.
//   COLS: the weight gradient, whose outputs have scales of their own.
template <int TM, bool COLS>
__device__ __forceinline__ void f8_tile(const Args &p, uint8_t *L0, uint8_t *L1) {
  using G = Geo<TM>;
  const int tid = threadIdx.x, lane = tid & 63, h = lane >> 4, l16 = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int mt, nt, g, first, m0, valid, step0, steps;
  size_t xrow;  // first row of the tile, in the operand
  uint16_t *out;
  if constexpr (COLS) {
    const int per = p.MT * p.nN;
    g = blockIdx.x / per;
    tile_of_block(blockIdx.x - g * per, p.MT, p.nN, mt, nt);
    const F8Span sp = f8_span(p.offsets, g, p.rows);
    step0 = sp.begin / kF8Block + g;
    steps = (sp.end - sp.begin + kF8Block - 1) / kF8Block;
    m0 = mt * TM;
    valid = min(TM, p.xrows - m0);
    xrow = m0;
    out = p.out + ((size_t)g * p.xrows + m0) * p.ostride;
  } else {
    tile_of_block(blockIdx.x, p.MT, p.nN, mt, nt);
    g = f8_group_at(p.offsets, p.groups, p.rows, TM, mt, &first);
    const F8Span sp = f8_span(p.offsets, g, p.rows);
    m0 = sp.begin + (mt - first) * TM;
    if (mt < first || m0 >= sp.end) return;  // an empty place
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
  const int wbytes = (tiles * p.wsteps - (COLS ? step0 : 0)) * kF8Tile;
  uint32_t ox[G::XQ], ow[G::WQ];
#pragma unroll
  for (int q = 0; q < G::XQ; q++) {
    const int row = (wave * G::XQ + q) * 8 + (lane >> 3);
    ox[q] = row * kF8Block + (((lane & 7) ^ (row & 7)) << 4);
  }
#pragma unroll
  for (int q = 0; q < G::WQ; q++) {
    const int piece = wave * G::WQ + q;
    ow[q] = (piece >> 1) * p.wsteps * kF8Tile + (piece & 1) * 1024 + lane * 16;
  }
  // stage kt to L; past the end: zeros, from empty buffers (without a branch, which
  // the scheduler would not move the loop's work across)
  auto dma = [&](uint8_t *L, int kt) {
    const int k1 = min(kt, steps - 1), live = kt < steps ? -1 : 0;
    const f8_rsrc_t rX =
        f8_buffer(xc + (size_t)k1 * p.xpitch * kF8Block, valid * kF8Block & live);
#pragma unroll
    for (int q = 0; q < G::XQ; q++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rX, (lds_ptr_t)(L + (wave * G::XQ + q) * 1024), 16,
                                               ox[q], 0, 0, 0);
    const f8_rsrc_t rW = f8_buffer(wc, wbytes & live);
#pragma unroll
    for (int q = 0; q < G::WQ; q++)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rW,
                                               (lds_ptr_t)(L + G::XB + (wave * G::WQ + q) * 1024), 16,
                                               ow[q], k1 * kF8Tile, 0, 0);
    if constexpr (COLS) {  // 4 bytes a lane, all waves alike: the second half is zeros
      const f8_rsrc_t rS =
          f8_buffer(wsc + (size_t)k1 * p.npitch, min(kTN, p.npitch - n0) * 4 & live);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rS, (lds_ptr_t)(L + G::XB + G::WB + wave * 256), 4,
                                               tid * 4, 0, 0, 0);
    }
  };
  // the scales of this lane's rows, and of the wave's outputs (forward)
  auto scales = [&](int kt, float *s) {
    const int k1 = min(kt, steps - 1);
    const f8_rsrc_t r = f8_buffer(xs + (size_t)k1 * p.spitch, valid * 4);
#pragma unroll
    for (int j = 0; j < G::NJ; j++)
      s[j] = __builtin_bit_cast(
          float, __builtin_amdgcn_raw_buffer_load_b32(r, (wm0 + 16 * j + l16) * 4, 0, 0));
  };
  f32x4 acc[G::NI][G::NJ];
#pragma unroll
  for (int i = 0; i < G::NI; i++)
#pragma unroll
    for (int j = 0; j < G::NJ; j++) acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  auto compute = [&](const uint8_t *L, const float *s) {
    i32x8_t xf[G::NJ];
    const uint8_t *X = L + (wm0 + l16) * kF8Block, *W = L + G::XB + (wn0 / 16) * kF8Tile + lane * 16;
    const int c0 = (h ^ (l16 & 7)) << 4, c1 = ((h + 4) ^ (l16 & 7)) << 4;
#pragma unroll
    for (int j = 0; j < G::NJ; j++)
      xf[j] = f8_frag(*(const u32x4_t *)(X + j * 16 * kF8Block + c0),
                      *(const u32x4_t *)(X + j * 16 * kF8Block + c1));
    // one tile of outputs after the other: its products go out between the scaling of
    // the one before, and the next one's weights are read meanwhile
    i32x8_t wf[2];
    f32x4 d[2][G::NJ], sw[2];
    auto load = [&](int i) {
      wf[i & 1] = f8_frag(*(const u32x4_t *)(W + i * kF8Tile),
                          *(const u32x4_t *)(W + i * kF8Tile + 1024));
      if constexpr (COLS)
        sw[i & 1] = *(const f32x4 *)(L + G::XB + G::WB + (wn0 + 16 * i + 4 * h) * 4);
    };
    f32x4 sp;
    auto scale = [&](int i, int j) {
#pragma unroll
      for (int v = 0; v < 4; v++)
        acc[i][j][v] = fmaf(COLS ? s[j] * sp[v] : s[j], d[i & 1][j][v], acc[i][j][v]);
    };
    load(0);
#pragma unroll
    for (int i = 0; i < G::NI; i++) {
      if constexpr (COLS)
        if (i) sp = sw[(i - 1) & 1];
      if (i + 1 < G::NI) load(i + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < G::NJ; j++) {
        d[i & 1][j] = f8_dot(wf[i & 1], xf[j]);
        if (i) scale(i - 1, j);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (COLS) sp = sw[(G::NI - 1) & 1];
#pragma unroll
    for (int j = 0; j < G::NJ; j++) scale(G::NI - 1, j);
  };
  // Lc holds stage kt (its rows' scales in sc), Ln receives the next one.
  auto stage = [&](uint8_t *Lc, uint8_t *Ln, int kt, float *sc, float *sn) {
    dma(Ln, kt + 1);
    if constexpr (!COLS) {
      const float sw = wsc[kt];
#pragma unroll
      for (int j = 0; j < G::NJ; j++) sc[j] *= sw;
    }
    scales(kt + 1, sn);
    __builtin_amdgcn_sched_barrier(0);
    compute(Lc, sc);
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    barrier_after_wait();
  };
  if (steps > 0) {
    float s0[G::NJ], s1[G::NJ];
    dma(L0, 0);
    scales(0, s0);
    __builtin_amdgcn_s_waitcnt(kVmcnt0);
    barrier_after_wait();
    int kt = 0;
    for (; kt + 2 <= steps; kt += 2) {
      stage(L0, L1, kt, s0, s1);
      stage(L1, L0, kt + 1, s1, s0);
    }
    if (kt < steps) stage(L0, L1, kt, s0, s1);
  }
  __syncthreads();
  // results to LDS, 512 bytes a row with its 16-byte chunks exchanged by the row, then
  // out as whole rows
  constexpr int kRows = TM / 2;  // rows of one buffer
  static_assert(kRows * 512 <= G::Lds, "the tile's results fit");
#pragma unroll
  for (int j = 0; j < G::NJ; j++) {
    const int r = wm0 + 16 * j + l16;
    uint8_t *row = (r < kRows ? L0 : L1) + (r % kRows) * 512;
#pragma unroll
    for (int i = 0; i < G::NI; i++) {
      const int c = wn0 + 16 * i + 4 * h;
      uint16_t o[4];
#pragma unroll
      for (int v = 0; v < 4; v++) o[v] = f8_to16(acc[i][j][v], p.f16);
      *(uint2 *)(row + ((((c >> 3) ^ r) & 31) << 4) + (c & 4) * 2) =
          make_uint2(o[0] | (uint32_t)o[1] << 16, o[2] | (uint32_t)o[3] << 16);
    }
  }
  __syncthreads();
  const int c = tid & 31, cols = p.n - n0 - 8 * c;
  for (int r = tid >> 5; r < valid; r += kThreads / 32) {
    const u32x4_t v =
        *(const u32x4_t *)((r < kRows ? L0 : L1) + (r % kRows) * 512 + (((c ^ r) & 31) << 4));
    uint16_t *dst = out + (size_t)r * p.ostride + n0 + 8 * c;
    if (cols >= 8)
      *(u32x4_a2 *)dst = (u32x4_a2){v[0], v[1], v[2], v[3]};
    else
#pragma unroll
      for (int e = 0; e < 8; e++)
        if (e < cols) dst[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
  }
}

template <int TM, bool COLS>
__global__ __launch_bounds__(kThreads, 2) void f8_gemm_kernel(Args p) {
  __shared__ __attribute__((aligned(1024))) uint8_t L0[Geo<TM>::Lds];
  __shared__ __attribute__((aligned(1024))) uint8_t L1[Geo<TM>::Lds];
  f8_tile<TM, COLS>(p, L0, L1);
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
    a.MT = rows / TM + d.groups;
    hipLaunchKernelGGL(kernel, dim3((unsigned)((long)a.MT * a.nN)), dim3(kThreads), 0, s, a);
  };
  const int avg = (rows + d.groups - 1) / d.groups;
  if (avg > 128) go(f8_gemm_kernel<256, false>, 256);
  else if (avg > 64) go(f8_gemm_kernel<128, false>, 128);
  else go(f8_gemm_kernel<64, false>, 64);
}

void launch_f8_wgrad(const F8Dims &d, int rows, const uint8_t *xc, const float *xs,
                     const uint8_t *yc, const float *ys, const int32_t *offsets, uint16_t *dw,
                     hipStream_t s) {
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
  go(f8_gemm_kernel<256, true>, 256);
}

}  // namespace moe
