// Products of a few rows with 4-bit weights and group scales: formats, packed
// layout and the streaming loop shared by w4_linear.hip and w4_ffn.hip, which takes
// 8-bit weights too (F8Fmt, packed as f8_device.h says).
//
//   y[r][n] = sum_k x[r][k] w[k][n],  x bf16, sums in fp32
//   MXFP4: w = 2^(s - 127) E2M1(code), one E8M0 scale s per 32 along k
//   INT4:  w = s (q - z), one bf16/fp16 scale s (and zero point z, else 8) per
//          32, 64 or 128 along k
//
// With few rows the bound is reading the weights (4.25 bits each for MXFP4):
// 2 M FLOP per weight are nothing for the matrix cores, but unpacking costs
// VALU work per weight, so it has to stay near one operation each.
//
// The products run on v_mfma_f32_16x16x32_bf16 with A = 16 rows of x and B =
// 16 outputs: lane l holds row (or output) l % 16 and the contraction values
// 8 (l / 16) .. + 7 of a 32-wide step, and receives outputs (row 4 (l / 16) +
// v, output l % 16).  MXFP4 codes become scaled bf16 pairs in one conversion
// instruction (exact: E2M1 times a power of two).  INT4 codes become 16 + q:
// the nibble is or-ed into the top mantissa bits of 16.0, two values per
// operation; the offset comes off through the group's sum of x, and the group's
// scale is applied to the fp32 partial sum, so no weight is ever rounded.
//
// Packed layout: a tile is 16 outputs x 128 contraction values, 1 KB, in the
// order in which one wave's 16-byte loads take it: lane l's four dwords are
// the 8 codes of output l % 16 at k = 32 i + 8 (l / 16), i = 0..3.  Tiles are
// [group][n / 16][k / 128], so the K loop of one tile row is one contiguous
// stream.  In a dword the MXFP4 code of value q sits at bits 4 q; INT4 puts
// values 2 p and 2 p + 1 at bits 3 + 4 p and 19 + 4 p (the last one wraps), the
// halves of one bf16 pair.
// Scales follow tile by tile: [group][n / 16][k / 128][16 outputs][spg], spg =
// 4 bytes for MXFP4, 128 / group_size 16-bit scales (and as many zero-point
// bytes) for INT4.  Outputs past n and values past k have zero weights.
#pragma once

#include <type_traits>

#include "common.h"
#include "gemm_common.h"
#include "w4.h"

namespace moe {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef unsigned int w4_u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int w4_u32x4u __attribute__((ext_vector_type(4), aligned(2)));

// Packed pieces of one matrix per group.
struct W4Mat {
  const uint8_t *codes, *scales, *zeros;
  int n, k, nt, ks;
  uint32_t f16;  // mask of scale_value
};

inline W4Mat w4_view(const W4Dims &d, const void *packed) {
  const uint8_t *p = (const uint8_t *)packed;
  return {p, p + d.code_bytes, p + d.code_bytes + d.scale_bytes, d.n, d.k, d.nt, d.ks,
          d.f16_scales ? ~0u : 0u};
}

// f16: all bits, or none.  Both readings are made and one masked in: as a choice it
// becomes a branch at every scale, which no load or product moves past.
__device__ __forceinline__ float scale_value(uint32_t u16, uint32_t f16) {
  const uint32_t h = __float_as_uint((float)__builtin_bit_cast(_Float16, (uint16_t)u16));
  return __uint_as_float((h & f16) | (u16 << 16 & ~f16));
}

typedef __amdgpu_buffer_rsrc_t rsrc_t;

__device__ __forceinline__ rsrc_t w4_buffer(const void *p, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void *)p, (short)0, bytes, kBufferDword3);
}

// Codes: one lane's of a tile, kTile bytes in all; Scales: those that it needs, as loaded.
// col(i, h): first of the 8 contraction values that lanes l / 16 = h hold in the i-th of a
// step's four products.
typedef uint4 W4Codes;
__device__ __forceinline__ int w4_col(int i, int h) { return 32 * i + 8 * h; }

struct MxFmt {
  typedef W4Codes Codes;
  static constexpr int kTile = 1024;
  static __device__ __forceinline__ int col(int i, int h) { return w4_col(i, h); }
  static __device__ __forceinline__ uint32_t part(const Codes &c, int i) {
    const uint32_t d[4] = {c.x, c.y, c.z, c.w};
    return d[i];
  }
  static constexpr bool kBlock = false;
  static constexpr bool kGrouped = false;  // scaled while unpacking
  static constexpr int SPG = 4, kScaleBytes = 64;  // bytes of a tile's scales
  static constexpr bool ZERO = false;
  struct Scales { uint32_t d; };
  static __device__ __forceinline__ Scales load(rsrc_t s, rsrc_t, int step, int n) {
    return {__builtin_amdgcn_raw_buffer_load_b32(s, 4 * n, step * kScaleBytes, 0)};
  }
  static __device__ __forceinline__ bf16x8 unpack(uint32_t d, const Scales &s, int i) {
    const float sc = __uint_as_float(((s.d >> (8 * i)) & 0xFFu) << 23);
    bf16x8 v;
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 0);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 1);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 2);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, sc, 3);
    v[0] = p0[0]; v[1] = p0[1]; v[2] = p1[0]; v[3] = p1[1];
    v[4] = p2[0]; v[5] = p2[1]; v[6] = p3[0]; v[7] = p3[1];
    return v;
  }
};

template <int SPG_, bool ZERO_>
struct IntFmt {
  typedef W4Codes Codes;
  static constexpr int kTile = 1024;
  static __device__ __forceinline__ int col(int i, int h) { return w4_col(i, h); }
  static __device__ __forceinline__ uint32_t part(const Codes &c, int i) { return MxFmt::part(c, i); }
  static constexpr bool kBlock = false;
  static constexpr bool kGrouped = true;
  static constexpr int SPG = SPG_, kScaleBytes = 32 * SPG_;
  static constexpr bool ZERO = ZERO_;
  // as loaded, two scales a register, taken apart at their use
  struct Scales { uint32_t s[(SPG_ + 1) / 2], z; };
  static __device__ __forceinline__ Scales load(rsrc_t ps, rsrc_t pz, int step, int n) {
    Scales s;
    const int at = step * kScaleBytes, az = step * (kScaleBytes / 2);
    if constexpr (SPG_ == 1) s.s[0] = __builtin_amdgcn_raw_buffer_load_b16(ps, 2 * n, at, 0);
    else if constexpr (SPG_ == 2) s.s[0] = __builtin_amdgcn_raw_buffer_load_b32(ps, 4 * n, at, 0);
    else {
      const auto v = __builtin_amdgcn_raw_buffer_load_b64(ps, 8 * n, at, 0);
      s.s[0] = v[0];
      s.s[1] = v[1];
    }
    if constexpr (!ZERO_) s.z = 0;
    else if constexpr (SPG_ == 1) s.z = __builtin_amdgcn_raw_buffer_load_b8(pz, n, az, 0);
    else if constexpr (SPG_ == 2) s.z = __builtin_amdgcn_raw_buffer_load_b16(pz, 2 * n, az, 0);
    else s.z = __builtin_amdgcn_raw_buffer_load_b32(pz, 4 * n, az, 0);
    return s;
  }
  static __device__ __forceinline__ uint32_t scale(const Scales &s, int g) {
    return g & 1 ? s.s[g / 2] >> 16 : s.s[g / 2] & 0xFFFFu;
  }
  static __device__ __forceinline__ float zero(const Scales &s, int g) {
    return (float)((s.z >> (8 * g)) & 0xFFu);
  }
  // 16 + q: the nibble in bits 3..6 of bf16 16.0 (0x4180)
  static __device__ __forceinline__ bf16x8 unpack(uint32_t d, const Scales &, int) {
    uint32_t u[4], mask = 0x00780078u, one = 0x41804180u;
    // in registers, for one and-or each: as literals they take two instructions
    asm("" : "+s"(mask));
    asm("" : "+v"(one));
    u[0] = (d & mask) | one;
    u[1] = ((d >> 4) & mask) | one;
    u[2] = ((d >> 8) & mask) | one;
    u[3] = (__builtin_amdgcn_alignbit(d, d, 12) & mask) | one;
    bf16x8 v;
    __builtin_memcpy(&v, u, 16);
    return v;
  }
};

// E4M3 with an fp32 scale per 128 x 128 block, in f8_device.h's tiles: codes become
// bf16 pairs in one instruction (exact), and the scale multiplies the fp32 sum of a
// step's products.  Lane l's two 16-byte loads are chunks l / 16 and l / 16 + 4.
struct F8Fmt {
  struct Codes { uint4 a, b; };
  static constexpr int kTile = 2048;
  static __device__ __forceinline__ int col(int i, int h) { return 64 * (i >> 1) + 16 * h + 8 * (i & 1); }
  static __device__ __forceinline__ uint2 part(const Codes &c, int i) {
    const uint4 v = i < 2 ? c.a : c.b;
    return i & 1 ? make_uint2(v.z, v.w) : make_uint2(v.x, v.y);
  }
  static constexpr bool kBlock = true;   // one scale a step
  static constexpr bool kGrouped = true;  // scaled sum by sum
  static constexpr int SPG = 1, kScaleBytes = 4;
  static constexpr bool ZERO = false;
  struct Scales { float s; };
  static __device__ __forceinline__ Scales load(rsrc_t s, rsrc_t, int step, int) {
    return {__builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(s, 0, step * kScaleBytes, 0))};
  }
  static __device__ __forceinline__ bf16x8 unpack(uint2 d, const Scales &, int) {
    bf16x8 v;
    const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.x, 1.0f, false);
    const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.x, 1.0f, true);
    const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.y, 1.0f, false);
    const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(d.y, 1.0f, true);
    v[0] = p0[0]; v[1] = p0[1]; v[2] = p1[0]; v[3] = p1[1];
    v[4] = p2[0]; v[5] = p2[1]; v[6] = p3[0]; v[7] = p3[1];
    return v;
  }
};

// The steps of one row of tiles (16 outputs, the whole contraction) as buffers
// of their own: a step's loads then need one scalar offset, and no address
// registers.
template <class F>
struct W4Row {
  rsrc_t c, s, z;
  W4Row() = default;
  __device__ __forceinline__ W4Row(const W4Mat &m, size_t row) {
    c = w4_buffer(m.codes + row * m.ks * F::kTile, m.ks * F::kTile);
    s = w4_buffer(m.scales + row * m.ks * F::kScaleBytes, m.ks * F::kScaleBytes);
    z = F::ZERO ? w4_buffer(m.zeros + row * m.ks * (F::kScaleBytes / 2), m.ks * (F::kScaleBytes / 2))
                : s;
  }
  __device__ __forceinline__ typename F::Codes codes(int step) const {  // read once: not kept in the caches
    auto load = [&](int at) {
      return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(
                                           c, 16 * (threadIdx.x & 63) + at, step * F::kTile, 2));
    };
    if constexpr (F::kTile == 1024) return load(0);
    else return {load(0), load(1024)};
  }
  __device__ __forceinline__ typename F::Scales scales(int step) const {
    return F::load(s, z, step, threadIdx.x & 15);
  }
};

// f(F{}) for the 4-bit format of d.
template <class Fn>
void with_format(const W4Dims &d, Fn &&f) {
  if (d.fmt == kW4Mx) f(MxFmt{});
  else if (d.spg == 1 && !d.zeros) f(IntFmt<1, false>{});
  else if (d.spg == 2 && !d.zeros) f(IntFmt<2, false>{});
  else if (d.spg == 4 && !d.zeros) f(IntFmt<4, false>{});
  else if (d.spg == 1) f(IntFmt<1, true>{});
  else if (d.spg == 2) f(IntFmt<2, true>{});
  else f(IntFmt<4, true>{});
}

__device__ __forceinline__ bf16x8 splat(float f) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = (__bf16)f;
  return v;
}

// A lane's row of x, in memory (a lane past the rows holds the last one again:
// its results are dropped) ...
struct RowPtr {
  const uint16_t *p;
  __device__ __forceinline__ bf16x8 load(int k) const {
    return __builtin_bit_cast(bf16x8, *(const w4_u32x4u *)(p + k));
  }
};
// ... or in LDS.
struct RowLds {
  const char *p;
  __device__ __forceinline__ bf16x8 load(int k) const {
    return __builtin_bit_cast(bf16x8, *(const w4_u32x4 *)(p + 2 * k));
  }
};

// One step: acc[j][p] += a[p] times the codes of tile j, 128 contraction values.
// V: values of a lane's results that are wanted (INT4 scales them one by one).
template <class F, int V, int NTW, int NB>
__device__ __forceinline__ void w4_step(uint32_t f16, const typename F::Codes (&cw)[NTW],
                                        const typename F::Scales (&sc)[NTW],
                                        const bf16x8 (&a)[NB][4], f32x4 (&acc)[NTW][NB]) {
  if constexpr (!F::kGrouped) {
#pragma unroll
    for (int i = 0; i < 4; i++) {  // the tiles' chains of products side by side
#pragma unroll
      for (int j = 0; j < NTW; j++) {
        const bf16x8 b = F::unpack(F::part(cw[j], i), sc[j], i);
#pragma unroll
        for (int p = 0; p < NB; p++)
          acc[j][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][i], b, acc[j][p], 0, 0, 0);
      }
    }
  } else if constexpr (F::kBlock) {
    f32x4 part[NTW][NB];
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int j = 0; j < NTW; j++) {
        const bf16x8 b = F::unpack(F::part(cw[j], i), sc[j], i);
#pragma unroll
        for (int p = 0; p < NB; p++)
          part[j][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a[p][i], b, i ? part[j][p] : (f32x4){0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
      }
    }
#pragma unroll
    for (int j = 0; j < NTW; j++)
#pragma unroll
      for (int p = 0; p < NB; p++)
#pragma unroll
        for (int v = 0; v < V; v++) acc[j][p][v] = fmaf(sc[j].s, part[j][p][v], acc[j][p][v]);
  } else {
    constexpr int kPer = 4 / F::SPG;  // MFMA steps of one scale group
#pragma unroll
    for (int g = 0; g < F::SPG; g++) {
      // the offset: -24 sum x (zero point 8), or sum x for a zero point of each
      // output's own
      f32x4 off[NB];
#pragma unroll
      for (int p = 0; p < NB; p++) {
        off[p] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < kPer; i++)
          off[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              a[p][g * kPer + i], splat(F::ZERO ? 1.0f : -24.0f), off[p], 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < NTW; j++) {
        const float scale = scale_value(F::scale(sc[j], g), f16);
        f32x4 part[NB];
#pragma unroll
        for (int p = 0; p < NB; p++) part[p] = F::ZERO ? (f32x4){0.0f, 0.0f, 0.0f, 0.0f} : off[p];
#pragma unroll
        for (int i = 0; i < kPer; i++) {
          const bf16x8 b = F::unpack(F::part(cw[j], g * kPer + i), sc[j], i);
#pragma unroll
          for (int p = 0; p < NB; p++)
            part[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][g * kPer + i], b, part[p], 0, 0,
                                                              0);
        }
#pragma unroll
        for (int p = 0; p < NB; p++)
#pragma unroll
          for (int v = 0; v < V; v++) {
            float t = part[p][v];
            if constexpr (F::ZERO) t = fmaf(-(16.0f + F::zero(sc[j], g)), off[p][v], t);
            acc[j][p][v] = fmaf(scale, t, acc[j][p][v]);
          }
      }
      // a group at a time: groups side by side would take hundreds of registers
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Up to 16 rows.  Row r is the matrix instruction's row 4 (r % 4) + r / 4, so that
// lane l's v-th result is row l / 16 + 4 v: up to 4 rows need one value of each
// lane only.
__device__ __forceinline__ int w4_row_of_lane() {  // that this lane loads
  return ((threadIdx.x >> 2) & 3) + 4 * (threadIdx.x & 3);
}
__device__ __forceinline__ int w4_row_of(int i) {  // of sum i of w4_join
  return ((i & 63) >> 4) + 4 * ((i >> 6) & 3);
}

// acc[j] += the rows times the row j of tiles over the steps [s0, s1), the rows
// read from memory; x: this lane's row.  The rows, codes and scales of U steps
// are loaded together, one memory round trip; steps past the end load the last
// step again and are not used.  Values of k past K meet zero weights: their
// lanes load the row's last values.
template <class F, int U, int V, int NTW, class Row>
__device__ __forceinline__ void w4_batches(const W4Row<F> (&m)[NTW], uint32_t f16, const Row &x, int K,
                                           int s0, int s1, f32x4 (&acc)[NTW][1]) {
  const int h = (threadIdx.x & 63) >> 4;
  for (int s = s0; s < s1; s += U) {
    typename F::Codes cw[U][NTW];
    typename F::Scales sc[U][NTW];
    bf16x8 a[U][1][4];
#pragma unroll
    for (int u = 0; u < U; u++) {
      const int st = min(s + u, s1 - 1);
#pragma unroll
      for (int i = 0; i < 4; i++) a[u][0][i] = x.load(min(128 * st + F::col(i, h), K - 8));
#pragma unroll
      for (int j = 0; j < NTW; j++) {
        cw[u][j] = m[j].codes(st);
        sc[u][j] = m[j].scales(st);
      }
    }
    // the batch's loads all go out before the first use (else the scheduler
    // saves registers by moving loads to their uses)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < U; u++)
      if (s + u < s1) w4_step<F, V>(f16, cw[u], sc[u], a[u], acc);
  }
}

template <class F, int U, int NTW, class Row>
__device__ __forceinline__ void w4_stream(const W4Row<F> (&m)[NTW], uint32_t f16, const Row &x, int rows,
                                          int K, int s0, int s1, f32x4 (&acc)[NTW][1]) {
  if (F::kGrouped && rows <= 4) w4_batches<F, U, 1>(m, f16, x, K, s0, s1, acc);
  else w4_batches<F, U, 4>(m, f16, x, K, s0, s1, acc);
}

// A ring of D steps whose codes and scales are in flight, refilled step by step
// (the rows lie in LDS).
template <class F, int NTW, int D>
struct W4Ring {
  typename F::Codes cw[D][NTW];
  typename F::Scales sc[D][NTW];

  template <int d>
  __device__ __forceinline__ void load(const W4Row<F> (&m)[NTW], int step) {
#pragma unroll
    for (int j = 0; j < NTW; j++) {
      cw[d][j] = m[j].codes(step);
      sc[d][j] = m[j].scales(step);
    }
  }
};

template <int NTW, int NB>
__device__ __forceinline__ void zero_acc(f32x4 (&acc)[NTW][NB]) {
#pragma unroll
  for (int j = 0; j < NTW; j++)
#pragma unroll
    for (int p = 0; p < NB; p++) acc[j][p] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
}

// The waves' partial sums meet in LDS and are added in wave order.  Afterwards
// red[256 j + i] is output i % 16 of tile j, of row w4_row_of(i), for the first
// `rows` rows.  red: WAVES NTW 256 floats.  The caller synchronises before red is
// written again.
template <int WAVES, int NTW>
__device__ __forceinline__ void w4_join(const f32x4 (&acc)[NTW][1], float *red, int rows) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool few = rows <= 4;  // one value a lane
  constexpr int kQ = NTW * 4;
#pragma unroll
  for (int j = 0; j < NTW; j++)
#pragma unroll
    for (int v = 0; v < 4; v++)
      if (v == 0 || !few) red[(wave * kQ + j * 4 + v) * 64 + lane] = acc[j][0][v];
  lds_barrier();
  for (int q = tid; q < (few ? NTW : kQ) * 64; q += WAVES * 64) {
    const int i = few ? (q & ~63) * 4 + lane : q;
    float t = red[i];
#pragma unroll
    for (int w = 1; w < WAVES; w++) t += red[w * kQ * 64 + i];
    red[i] = t;
  }
  lds_barrier();
}

// f(integral_constant<int, d>) for d = 0 .. N - 1
template <int N, int d = 0, class Fn>
__device__ __forceinline__ void each(Fn &&f) {
  if constexpr (d < N) {
    f(std::integral_constant<int, d>{});
    each<N, d + 1>(f);
  }
}

// ---------------------------------------------------------------------------
// Many rows (16 NB a pass, NB > 1): here every tile would read all the rows
// again, so the rows go through LDS, a step (128 values) at a time, shared by
// the four waves of a group, each with its own NTW tiles.  A workgroup is two
// such groups, which take half of the contraction each.
constexpr int kBlockWaves = 4;    // waves of a group
constexpr int kBlockGroups = 2;
constexpr int kBlockDepth = 4;    // steps in flight
// LDS bytes from one row's step to the next: 16 more than its values, so that 16
// rows' reads of the same columns fall into different banks
constexpr int kBlockPitch = 256 + 16;
// Row blocks of a long pass: groups of 32 keep four scales and offsets a step,
// which leaves registers for two blocks only.
template <class F>
constexpr int kLongBlocks = F::kGrouped && F::SPG == 4 ? 2 : 4;
template <int NB>
constexpr int w4_block_lds() { return kBlockGroups * 2 * 16 * NB * kBlockPitch; }

// acc += rows times tiles m over this group's half of the ks steps.  x[p]:
// address of the 16 bytes that this thread stages of row 16 p + (thread of the
// group) / 16, chunk thread % 16, at step 0.  xs: the workgroup's LDS.  All
// threads of the workgroup call.  A step's rows travel through registers with
// the codes (loads complete in order: rows fetched later than the codes of
// their step would empty the pipeline at every step) into one of two buffers.
template <class F, int NTW, int NB>
__device__ __forceinline__ void w4_block(const W4Row<F> (&m)[NTW], uint32_t f16,
                                         const uint16_t *const (&x)[NB], int K, int ks, char *xs,
                                         f32x4 (&acc)[NTW][NB]) {
  constexpr int D = kBlockDepth;
  const int tid = threadIdx.x, lane = tid & 63;
  const int group = __builtin_amdgcn_readfirstlane(tid / (64 * kBlockWaves));
  const int s0 = ks * group / kBlockGroups, n = ks * (group + 1) / kBlockGroups - s0;
  const int most = (ks + kBlockGroups - 1) / kBlockGroups;  // both groups meet at every barrier
  const int gt = tid % (64 * kBlockWaves), chunk = gt % 16;
  char *mine = xs + group * (2 * 16 * NB * kBlockPitch);
  typename F::Codes cw[D][NTW];
  typename F::Scales sc[D][NTW];
  w4_u32x4 xv[D][NB];
  auto load = [&](auto d, int i) __attribute__((always_inline)) {
    const int st = min(s0 + i, ks - 1), k = min(128 * st, K - 8 - 8 * chunk);
#pragma unroll
    for (int p = 0; p < NB; p++) xv[d][p] = *(const w4_u32x4u *)(x[p] + k);
#pragma unroll
    for (int j = 0; j < NTW; j++) {
      cw[d][j] = m[j].codes(st);
      sc[d][j] = m[j].scales(st);
    }
  };
  auto put = [&](auto d, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < NB; p++)
      *(w4_u32x4 *)(mine + (buf * 16 * NB + 16 * p + gt / 16) * kBlockPitch + 16 * chunk) = xv[d][p];
  };
  each<D>([&](auto d) __attribute__((always_inline)) { load(d, d); });
  put(std::integral_constant<int, 0>{}, 0);
  for (int i0 = 0; i0 < most; i0 += D) {
    each<D>([&](auto d) __attribute__((always_inline)) {
      constexpr int dn = (decltype(d)::value + 1) % D;
      const int i = i0 + d;
      lds_barrier();  // step i's rows are there, and step i - 1's have been read
      if (i + 1 < most) put(std::integral_constant<int, dn>{}, (d + 1) & 1);
      if (i < n) {
        bf16x8 a[NB][4];
#pragma unroll
        for (int p = 0; p < NB; p++)
#pragma unroll
          for (int b = 0; b < 4; b++)
            a[p][b] = __builtin_bit_cast(
                bf16x8, *(const w4_u32x4 *)(mine + ((d & 1) * 16 * NB + 16 * p + (lane & 15)) *
                                                       kBlockPitch + 2 * F::col(b, lane >> 4)));
        w4_step<F, 4>(f16, cw[d], sc[d], a, acc);
      }
      load(d, i + D);
    });
  }
}

// The two groups' sums: group 1 leaves its own in LDS (the rows' buffers are
// free then), group 0 adds them.  Returns whether this wave holds results.
template <int NTW, int NB>
__device__ __forceinline__ bool w4_block_join(f32x4 (&acc)[NTW][NB], char *xs) {
  const int gt = threadIdx.x % (64 * kBlockWaves);
  const bool second = threadIdx.x >= 64 * kBlockWaves;
  float *at = (float *)xs + gt;
  lds_barrier();
#pragma unroll
  for (int q = 0; q < NTW * NB * 4; q++)
    if (second) at[q * 64 * kBlockWaves] = acc[q / (NB * 4)][q / 4 % NB][q % 4];
  lds_barrier();
  if (second) return false;
#pragma unroll
  for (int q = 0; q < NTW * NB * 4; q++)
    acc[q / (NB * 4)][q / 4 % NB][q % 4] += at[q * 64 * kBlockWaves];
  return true;
}

__device__ __forceinline__ uint16_t to_bf16(float f) {
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

}  // namespace
}  // namespace moe
