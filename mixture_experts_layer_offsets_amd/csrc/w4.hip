// Few-row products with 4-bit weights and group scales, and the few-token
// expert FFN on them.
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
// values 2 p and 2 p + 1 at bits 4 p and 16 + 4 p, the halves of one bf16 pair.
// Scales follow tile by tile: [group][n / 16][k / 128][16 outputs][spg], spg =
// 4 bytes for MXFP4, 128 / group_size 16-bit scales (and as many zero-point
// bytes) for INT4.  Outputs past n and values past k have zero weights.
#include <algorithm>

#include "common.h"
#include "mx_device.h"
#include "w4.h"

namespace moe {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kW4Waves = 8;  // waves of a workgroup; they split the contraction
constexpr int kW4Unroll = 4; // steps whose loads a wave has in flight

// Packed pieces of one matrix per group.
struct W4Mat {
  const uint8_t *codes, *scales, *zeros;
  int n, k, nt, ks, f16;
};

W4Mat view(const W4Dims &d, const void *packed) {
  const uint8_t *p = (const uint8_t *)packed;
  return {p, p + d.code_bytes, p + d.code_bytes + d.scale_bytes, d.n, d.k, d.nt, d.ks,
          d.f16_scales};
}

__device__ __forceinline__ float scale_value(uint32_t u16, int f16) {
  return f16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)u16) : bf16_to_f32(u16);
}

// One lane's scales of one tile, as loaded.
struct MxFmt {
  static constexpr bool kGrouped = false;  // scaled while unpacking
  static constexpr int SPG = 4;
  static constexpr bool ZERO = false;
  struct Scales { uint32_t d; };
  static __device__ __forceinline__ Scales load(const W4Mat &m, size_t tile, int n) {
    return {((const uint32_t *)m.scales)[tile * 16 + n]};
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
  static constexpr bool kGrouped = true;
  static constexpr int SPG = SPG_;
  static constexpr bool ZERO = ZERO_;
  struct Scales { uint16_t s[SPG_]; uint8_t z[SPG_]; };
  static __device__ __forceinline__ Scales load(const W4Mat &m, size_t tile, int n) {
    Scales s;
    const size_t at = (tile * 16 + n) * SPG_;
    __builtin_memcpy(s.s, __builtin_assume_aligned(m.scales + at * 2, 2 * SPG_), 2 * SPG_);
    if constexpr (ZERO_)
      __builtin_memcpy(s.z, __builtin_assume_aligned(m.zeros + at, SPG_), SPG_);
    return s;
  }
  // 16 + q: the nibble in bits 3..6 of bf16 16.0 (0x4180)
  static __device__ __forceinline__ bf16x8 unpack(uint32_t d, const Scales &, int) {
    uint32_t u[4];
    u[0] = ((d << 3) & 0x00780078u) | 0x41804180u;
    u[1] = ((d >> 1) & 0x00780078u) | 0x41804180u;
    u[2] = ((d >> 5) & 0x00780078u) | 0x41804180u;
    u[3] = ((d >> 9) & 0x00780078u) | 0x41804180u;
    bf16x8 v;
    __builtin_memcpy(&v, u, 16);
    return v;
  }
};

__device__ __forceinline__ bf16x8 splat(float f) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; i++) v[i] = (__bf16)f;
  return v;
}

// acc[j][p] += rows of block p times output tile j over the steps [s0, s1).
// tile[j]: index of step 0's tile; x[p]: this lane's row of block p.  The
// codes and scales of kW4Unroll steps are loaded together; steps past the end
// load the last step again and are not used.
template <class F, int NTW, int NB>
__device__ __forceinline__ void w4_stream(const W4Mat (&m)[NTW], const size_t (&tile)[NTW],
                                          const uint16_t *const (&x)[NB], int K, int s0, int s1,
                                          f32x4 (&acc)[NTW][NB]) {
  const int lane = threadIdx.x & 63, h8 = 8 * (lane >> 4);
  for (int s = s0; s < s1; s += kW4Unroll) {
    uint4 cw[kW4Unroll][NTW];
    typename F::Scales sc[kW4Unroll][NTW];
#pragma unroll
    for (int u = 0; u < kW4Unroll; u++) {
      const int st = min(s + u, s1 - 1);
#pragma unroll
      for (int j = 0; j < NTW; j++) {
        cw[u][j] = ld_once((const uint4 *)m[j].codes + (tile[j] + st) * 64 + lane);
        sc[u][j] = F::load(m[j], tile[j] + st, lane & 15);
      }
    }
#pragma unroll
    for (int u = 0; u < kW4Unroll; u++) {
      if (s + u >= s1) break;
      const int k0 = (s + u) * 128;
      bf16x8 a[NB][4];
#pragma unroll
      for (int p = 0; p < NB; p++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
          if (k0 + 32 * i < K)  // uniform: k is a multiple of 32
            __builtin_memcpy(&a[p][i], x[p] + k0 + 32 * i + h8, 16);
          else
            a[p][i] = splat(0.0f);
        }
      if constexpr (!F::kGrouped) {
#pragma unroll
        for (int j = 0; j < NTW; j++) {
          const uint32_t d[4] = {cw[u][j].x, cw[u][j].y, cw[u][j].z, cw[u][j].w};
#pragma unroll
          for (int i = 0; i < 4; i++) {
            const bf16x8 b = F::unpack(d[i], sc[u][j], i);
#pragma unroll
            for (int p = 0; p < NB; p++)
              acc[j][p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][i], b, acc[j][p], 0, 0, 0);
          }
        }
      } else {
        constexpr int kPer = 4 / F::SPG;  // MFMA steps of one scale group
#pragma unroll
        for (int g = 0; g < F::SPG; g++) {
          // the offset: -24 sum x (zero point 8), or sum x for a zero point
          // of each output's own
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
            const uint32_t d[4] = {cw[u][j].x, cw[u][j].y, cw[u][j].z, cw[u][j].w};
            const float scale = scale_value(sc[u][j].s[g], m[j].f16);
            f32x4 part[NB];
#pragma unroll
            for (int p = 0; p < NB; p++)
              part[p] = F::ZERO ? (f32x4){0.0f, 0.0f, 0.0f, 0.0f} : off[p];
#pragma unroll
            for (int i = 0; i < kPer; i++) {
              const bf16x8 b = F::unpack(d[g * kPer + i], sc[u][j], i);
#pragma unroll
              for (int p = 0; p < NB; p++)
                part[p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[p][g * kPer + i], b, part[p],
                                                                  0, 0, 0);
            }
#pragma unroll
            for (int p = 0; p < NB; p++)
#pragma unroll
              for (int v = 0; v < 4; v++) {
                float t = part[p][v];
                if constexpr (F::ZERO) t = fmaf(-(16.0f + (float)sc[u][j].z[g]), off[p][v], t);
                acc[j][p][v] = fmaf(scale, t, acc[j][p][v]);
              }
          }
        }
      }
    }
  }
}

// A workgroup's product: its waves split the steps, the partial sums meet in
// LDS and are added in wave order.  Afterwards red[q * 64 + lane] (q = (j NB +
// p) 4 + v) holds output tile j, row 16 p + 4 (lane / 16) + v, output lane %
// 16.  red: kW4Waves NTW NB 256 floats.
template <class F, int NTW, int NB>
__device__ __forceinline__ void w4_product(const W4Mat (&m)[NTW], const size_t (&tile)[NTW],
                                           const uint16_t *const (&x)[NB], int K, int steps,
                                           float *red) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  f32x4 acc[NTW][NB];
#pragma unroll
  for (int j = 0; j < NTW; j++)
#pragma unroll
    for (int p = 0; p < NB; p++) acc[j][p] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
  w4_stream<F, NTW, NB>(m, tile, x, K, steps * wave / kW4Waves, steps * (wave + 1) / kW4Waves, acc);
  constexpr int kQ = NTW * NB * 4;
#pragma unroll
  for (int j = 0; j < NTW; j++)
#pragma unroll
    for (int p = 0; p < NB; p++)
#pragma unroll
      for (int v = 0; v < 4; v++)
        red[(wave * kQ + (j * NB + p) * 4 + v) * 64 + lane] = acc[j][p][v];
  __syncthreads();
  for (int i = tid; i < kQ * 64; i += kW4Waves * 64) {
    float t = red[i];
#pragma unroll
    for (int w = 1; w < kW4Waves; w++) t += red[w * kQ * 64 + i];
    red[i] = t;
  }
  __syncthreads();
}

// ---------------------------------------------------------------------------
// Rows of a dense or grouped operand.  Grid (output tiles / NTW, groups).

template <class F, int NTW, int NB>
__global__ __launch_bounds__(kW4Waves * 64) void w4_linear_kernel(
    W4Mat m, const uint16_t *x, long xstride, const int32_t *__restrict__ offsets, int rows,
    uint16_t *__restrict__ out, long ostride) {
  __shared__ float red[kW4Waves * NTW * NB * 256];
  const int g = blockIdx.y, t0 = blockIdx.x * NTW;
  // offsets are the caller's: kept inside [0, rows]
  const int rb = offsets ? min(max(offsets[g], 0), rows) : 0;
  const int re = offsets ? min(max(offsets[g + 1], 0), rows) : rows;
  const int lane = threadIdx.x & 63;
  W4Mat mm[NTW];
  size_t tile[NTW];
#pragma unroll
  for (int j = 0; j < NTW; j++) {
    mm[j] = m;
    tile[j] = ((size_t)g * m.nt + min(t0 + j, m.nt - 1)) * m.ks;
  }
  for (int r0 = rb; r0 < re; r0 += 16 * NB) {
    const int nr = min(16 * NB, re - r0);
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++) xr[p] = x + (r0 + min(16 * p + (lane & 15), nr - 1)) * xstride;
    w4_product<F, NTW, NB>(mm, tile, xr, m.k, m.ks, red);
    for (int i = threadIdx.x; i < NTW * NB * 256; i += kW4Waves * 64) {
      const int l = i & 63, v = (i >> 6) & 3, jp = i >> 8;
      const int row = 16 * (jp % NB) + 4 * (l >> 4) + v;
      const int n = 16 * (t0 + jp / NB) + (l & 15);
      if (row < nr && n < m.n) out[(r0 + row) * ostride + n] = __builtin_bit_cast(uint16_t, (__bf16)red[i]);
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Few-token FFN.  Grid (output tiles, used experts): workgroup u finds the
// u-th expert that any slot uses (ascending) and the list of its slots.

struct Slots {
  int expert, count;  // expert -1: no u-th expert
};

// list: [slots] LDS; cnt: [E] LDS.  Every thread of the workgroup calls.
__device__ __forceinline__ Slots find_slots(const int32_t *idx, int slots, int first, int E, int u,
                                            int32_t *list, int32_t *cnt) {
  __shared__ int sh[2];
  const int tid = threadIdx.x, lane = tid & 63;
  if (!idx) {  // every token
    for (int f = tid; f < slots; f += kW4Waves * 64) list[f] = f;
    __syncthreads();
    return {0, slots};
  }
  for (int e = tid; e < E; e += kW4Waves * 64) cnt[e] = 0;
  __syncthreads();
  for (int f = tid; f < slots; f += kW4Waves * 64) {
    const int64_t e = (int64_t)idx[f] - first;
    if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
  }
  __syncthreads();
  if (tid < 64) {
    int left = u, expert = -1;
    for (int e0 = 0; e0 < E && expert < 0; e0 += 64) {
      const uint64_t used = __ballot(e0 + lane < E && cnt[min(e0 + lane, E - 1)] > 0);
      const int n = __popcll(used);
      if (left < n) {
        const int before = __popcll(used & ((1ull << lane) - 1));
        const uint64_t hit = __ballot(((used >> lane) & 1) && before == left);
        expert = e0 + __ffsll((unsigned long long)hit) - 1;
      }
      left -= n;
    }
    int at = 0;
    for (int f0 = 0; expert >= 0 && f0 < slots; f0 += 64) {
      const bool mine = f0 + lane < slots && (int64_t)idx[min(f0 + lane, slots - 1)] - first == expert;
      const uint64_t b = __ballot(mine);
      if (mine) list[at + __popcll(b & ((1ull << lane) - 1))] = f0 + lane;
      at += __popcll(b);
    }
    if (lane == 0) {
      sh[0] = expert;
      sh[1] = at;
    }
  }
  __syncthreads();
  return {sh[0], sh[1]};
}

// act[f] = silu(x Wg) (x Wu) for the expert's slots: output tile blockIdx.x of
// the gate and of the up matrix, the same outputs in the same lanes.
template <class F, int NB>
__global__ __launch_bounds__(kW4Waves * 64) void w4_gate_up_kernel(
    W4Mat gate, W4Mat up, const uint16_t *x, const int32_t *__restrict__ idx, int slots, int k,
    int first, int E, uint16_t *__restrict__ act) {
  extern __shared__ int32_t dyn[];
  __shared__ float red[kW4Waves * 2 * NB * 256];
  int32_t *list = dyn, *cnt = dyn + slots;
  const Slots sl = find_slots(idx, slots, first, E, blockIdx.y, list, cnt);
  if (sl.expert < 0) return;
  const int lane = threadIdx.x & 63, I = gate.n;
  const size_t base = ((size_t)sl.expert * gate.nt + blockIdx.x) * gate.ks;
  const W4Mat mm[2] = {gate, up};
  const size_t tile[2] = {base, base};
  for (int r0 = 0; r0 < sl.count; r0 += 16 * NB) {
    const int nr = min(16 * NB, sl.count - r0);
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = x + (size_t)(list[r0 + min(16 * p + (lane & 15), nr - 1)] / k) * gate.k;
    w4_product<F, 2, NB>(mm, tile, xr, gate.k, gate.ks, red);
    for (int i = threadIdx.x; i < NB * 256; i += kW4Waves * 64) {
      const int l = i & 63, v = (i >> 6) & 3, p = i >> 8;
      const int row = 16 * p + 4 * (l >> 4) + v, n = 16 * blockIdx.x + (l & 15);
      // a rounded to bf16, as the layer stores it: the matrix operand of down
      if (row < nr && n < I)
        act[(size_t)list[r0 + row] * I + n] =
            __builtin_bit_cast(uint16_t, (__bf16)(silu_f(red[i]) * red[NB * 256 + i]));
    }
    __syncthreads();
  }
}

// y[f] = act[f] Wd, in fp32.
template <class F, int NTW, int NB>
__global__ __launch_bounds__(kW4Waves * 64) void w4_down_kernel(
    W4Mat m, const uint16_t *act, const int32_t *__restrict__ idx, int slots, int first, int E,
    float *__restrict__ y) {
  extern __shared__ int32_t dyn[];
  __shared__ float red[kW4Waves * NTW * NB * 256];
  int32_t *list = dyn, *cnt = dyn + slots;
  const Slots sl = find_slots(idx, slots, first, E, blockIdx.y, list, cnt);
  if (sl.expert < 0) return;
  const int lane = threadIdx.x & 63, t0 = blockIdx.x * NTW;
  W4Mat mm[NTW];
  size_t tile[NTW];
#pragma unroll
  for (int j = 0; j < NTW; j++) {
    mm[j] = m;
    tile[j] = ((size_t)sl.expert * m.nt + min(t0 + j, m.nt - 1)) * m.ks;
  }
  for (int r0 = 0; r0 < sl.count; r0 += 16 * NB) {
    const int nr = min(16 * NB, sl.count - r0);
    const uint16_t *xr[NB];
#pragma unroll
    for (int p = 0; p < NB; p++)
      xr[p] = act + (size_t)list[r0 + min(16 * p + (lane & 15), nr - 1)] * m.k;
    w4_product<F, NTW, NB>(mm, tile, xr, m.k, m.ks, red);
    for (int i = threadIdx.x; i < NTW * NB * 256; i += kW4Waves * 64) {
      const int l = i & 63, v = (i >> 6) & 3, jp = i >> 8;
      const int row = 16 * (jp % NB) + 4 * (l >> 4) + v;
      const int n = 16 * (t0 + jp / NB) + (l & 15);
      if (row < nr && n < m.n) y[(size_t)list[r0 + row] * m.n + n] = red[i];
    }
    __syncthreads();
  }
}

// out[t] = sum_j w y over the kept slots, ascending j, then the shared
// expert's row; rounded once.
__global__ __launch_bounds__(256) void w4_combine_kernel(
    const float4 *__restrict__ y, const float *__restrict__ w, const int32_t *__restrict__ idx,
    int first, int E, const float4 *__restrict__ ys, uint2 *__restrict__ out, int k, int HC) {
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= HC) return;
  float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int j = 0; j < k; j++) {
    const int64_t e = (int64_t)idx[t * k + j] - first;
    if (e < 0 || e >= E) continue;
    const float4 v = y[(size_t)(t * k + j) * HC + c];
    const float wj = w[t * k + j];
    a[0] = fmaf(wj, v.x, a[0]); a[1] = fmaf(wj, v.y, a[1]);
    a[2] = fmaf(wj, v.z, a[2]); a[3] = fmaf(wj, v.w, a[3]);
  }
  if (ys) {
    const float4 v = ys[(size_t)t * HC + c];
    a[0] += v.x; a[1] += v.y; a[2] += v.z; a[3] += v.w;
  }
  const bf16x2 lo = {(__bf16)a[0], (__bf16)a[1]}, hi = {(__bf16)a[2], (__bf16)a[3]};
  out[(size_t)t * HC + c] = make_uint2(__builtin_bit_cast(uint32_t, lo),
                                       __builtin_bit_cast(uint32_t, hi));
}

// ---------------------------------------------------------------------------
// Packing.  One thread per dword of codes: tile, lane l, dword i hold output
// 16 tile + l % 16 at k = 128 step + 32 i + 8 (l / 16).

// Nibble position of value q in its dword.
__host__ __device__ __forceinline__ int nibble_at(int fmt, int q) {
  return fmt == kW4Mx ? q : (q >> 1) + 4 * (q & 1);
}

__global__ __launch_bounds__(256) void w4_pack_kernel(W4Dims d, const uint8_t *__restrict__ codes,
                                                      const void *__restrict__ scales,
                                                      const uint8_t *__restrict__ zeros,
                                                      uint8_t *__restrict__ packed) {
  const size_t id = (size_t)blockIdx.x * 256 + threadIdx.x;
  const size_t tiles = (size_t)d.groups * d.nt * d.ks;
  if (id >= tiles * 256) return;
  const int i = id & 3, l = (id >> 2) & 63;
  const size_t tile = id >> 8;
  const int step = (int)(tile % d.ks);
  const size_t gt = tile / d.ks;
  const int n = (int)(gt % d.nt) * 16 + (l & 15);
  const size_t g = gt / d.nt;
  const int k0 = step * 128 + 32 * i + 8 * (l >> 4);
  const size_t row = g * d.n + n;
  uint32_t v = 0;
  if (n < d.n && k0 < d.k) {
    const uint8_t *src = codes + row * (d.k / 2) + k0 / 2;
    for (int q = 0; q < 8; q++)
      v |= (uint32_t)((src[q >> 1] >> (4 * (q & 1))) & 15) << (4 * nibble_at(d.fmt, q));
  }
  ((uint32_t *)packed)[id] = v;
  // scales: the lanes l < 16 of dword i own scale i of their output
  if (l >= 16 || i >= d.spg) return;
  const int kg = (step * 128) / d.group + i;
  const bool in = n < d.n && kg < d.k / d.group;
  const size_t from = row * (d.k / d.group) + kg, to = (tile * 16 + l) * d.spg + i;
  uint8_t *ps = packed + d.code_bytes;
  if (d.fmt == kW4Mx) {
    ps[to] = in ? ((const uint8_t *)scales)[from] : 127;
  } else {
    ((uint16_t *)ps)[to] = in ? ((const uint16_t *)scales)[from] : 0;
    if (d.zeros) (ps + d.scale_bytes)[to] = in ? zeros[from] & 15 : 0;
  }
}

// E2M1 code of a value scaled by 2^-s: nearest, ties to the even code,
// saturating; the sign bit is set exactly when v < 0.
__device__ __forceinline__ uint32_t e2m1_code(float v, int s) {
  const float a = fminf(fabsf(ldexpf(v, -s)), 6.0f);
  // quantum 0.5 up to 2, 1 up to 4, 2 up to 6
  uint32_t c;
  if (a <= 2.0f) c = (uint32_t)rintf(a * 2.0f);
  else if (a <= 4.0f) c = 2u + (uint32_t)rintf(a);
  else c = 4u + (uint32_t)rintf(a * 0.5f);
  return c | (v < 0.0f ? 8u : 0u);
}

// One thread per (group of the contraction, output): reads its group of w
// [k][n] (neighbouring threads: neighbouring outputs), writes codes and scale.
__global__ __launch_bounds__(256) void w4_quantize_kernel(W4Dims d, const uint16_t *__restrict__ w,
                                                          uint8_t *__restrict__ packed) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const int kg = blockIdx.y;
  const size_t g = blockIdx.z;
  if (n >= d.nt * 16) return;
  const bool in = n < d.n && kg < d.k / d.group;
  const uint16_t *src = w + (g * d.k + (size_t)kg * d.group) * d.n + n;
  float lo = 0.0f, hi = 0.0f;
  for (int q = 0; in && q < d.group; q++) {
    const float v = bf16_to_f32(src[(size_t)q * d.n]);
    lo = fminf(lo, v);
    hi = fmaxf(hi, v);
  }
  const int step = kg * d.group / 128, slot = kg % d.spg;
  const size_t tile = (g * d.nt + n / 16) * d.ks + step;
  const size_t to = (tile * 16 + (n & 15)) * d.spg + slot;
  uint8_t *ps = packed + d.code_bytes;
  int sx = 0, z = 8;
  float s = 0.0f;
  if (d.fmt == kW4Mx) {
    const float amax = fmaxf(-lo, hi);
    sx = amax > 0.0f ? min(max(floor_log2(amax) - 2, -127), 127) : -127;
    ps[to] = in ? (uint8_t)(sx + 127) : 127;
  } else {
    s = d.zeros ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
    const uint16_t bits = d.f16_scales ? __builtin_bit_cast(uint16_t, (_Float16)s)
                                       : __builtin_bit_cast(uint16_t, (__bf16)s);
    s = scale_value(bits, d.f16_scales);
    ((uint16_t *)ps)[to] = in ? bits : 0;
    if (d.zeros) {
      z = s > 0.0f ? (int)fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 0;
      (ps + d.scale_bytes)[to] = in ? z : 0;
    }
  }
  for (int q0 = 0; q0 < d.group; q0 += 8) {
    uint32_t v = 0;
    for (int q = 0; in && q < 8; q++) {
      const float f = bf16_to_f32(src[(size_t)(q0 + q) * d.n]);
      uint32_t c;
      if (d.fmt == kW4Mx) c = e2m1_code(f, sx);
      else c = s > 0.0f ? (uint32_t)fminf(fmaxf(rintf(f / s) + (float)z, 0.0f), 15.0f) : (uint32_t)z;
      v |= c << (4 * nibble_at(d.fmt, q));
    }
    const int k0 = kg * d.group + q0, in128 = k0 & 127;
    const int l = ((in128 & 31) >> 3) * 16 + (n & 15), i = in128 >> 5;
    ((uint32_t *)packed)[(tile * 64 + l) * 4 + i] = v;
  }
}

__global__ __launch_bounds__(256) void w4_unpack_kernel(W4Dims d, const uint8_t *__restrict__ packed,
                                                        float *__restrict__ w) {
  const int n = blockIdx.x * 256 + threadIdx.x;
  const size_t g = blockIdx.z;
  if (n >= d.n) return;
  for (int k = blockIdx.y; k < d.k; k += gridDim.y) {
    const size_t tile = (g * d.nt + n / 16) * d.ks + k / 128;
    const int in128 = k & 127, l = ((in128 & 31) >> 3) * 16 + (n & 15), i = in128 >> 5;
    const uint32_t dw = ((const uint32_t *)packed)[(tile * 64 + l) * 4 + i];
    const uint32_t c = (dw >> (4 * nibble_at(d.fmt, k & 7))) & 15;
    const size_t at = (tile * 16 + (n & 15)) * d.spg + in128 / d.group;
    const uint8_t *ps = packed + d.code_bytes;
    float v;
    if (d.fmt == kW4Mx) {
      const int e = (c >> 1) & 3, man = c & 1;
      const float mag = e ? ldexpf(1.0f + 0.5f * man, e - 1) : 0.5f * man;
      v = ldexpf(c & 8 ? -mag : mag, (int)ps[at] - 127);
    } else {
      const int z = d.zeros ? (ps + d.scale_bytes)[at] : 8;
      v = scale_value(((const uint16_t *)ps)[at], d.f16_scales) * (float)((int)c - z);
    }
    w[(g * d.k + k) * d.n + n] = v;
  }
}

// f(F{}) for the format of d.
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

}  // namespace

void launch_w4_pack(const W4Dims &d, const uint8_t *codes, const void *scales,
                    const uint8_t *zeros, void *packed, hipStream_t s) {
  const size_t n = (size_t)d.groups * d.nt * d.ks * 256;
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, d, codes,
                     scales, zeros, (uint8_t *)packed);
}

void launch_w4_quantize(const W4Dims &d, const uint16_t *w, void *packed, hipStream_t s) {
  hipLaunchKernelGGL(w4_quantize_kernel, dim3((d.nt * 16 + 255) / 256, d.ks * 128 / d.group, d.groups),
                     dim3(256), 0, s, d, w, (uint8_t *)packed);
}

void launch_w4_unpack(const W4Dims &d, const void *packed, float *w, hipStream_t s) {
  hipLaunchKernelGGL(w4_unpack_kernel, dim3((d.n + 255) / 256, std::min(d.k, 4096), d.groups),
                     dim3(256), 0, s, d, (const uint8_t *)packed, w);
}

void launch_w4_linear(const W4Dims &d, int rows, const uint16_t *x, long xstride,
                      const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                      hipStream_t s) {
  if (rows <= 0) return;
  const W4Mat m = view(d, packed);
  with_format(d, [&](auto f) {
    using F = decltype(f);
    const dim3 grid(d.nt, d.groups), b(kW4Waves * 64);
    if (rows <= 16)
      hipLaunchKernelGGL((w4_linear_kernel<F, 1, 1>), grid, b, 0, s, m, x, xstride, offsets, rows,
                         out, ostride);
    else
      hipLaunchKernelGGL((w4_linear_kernel<F, 1, 4>), grid, b, 0, s, m, x, xstride, offsets, rows,
                         out, ostride);
  });
}

void launch_w4_ffn(const W4Dims &up, const W4Dims &down, const uint16_t *x, const int32_t *idx,
                   int slots, int k, int first, const void *gate, const void *upw,
                   const void *downw, uint16_t *act, float *y, hipStream_t s) {
  const W4Mat mg = view(up, gate), mu = view(up, upw), md = view(down, downw);
  const int E = up.groups, used = std::min(E, slots);
  const size_t lds = (size_t)(slots + E) * sizeof(int32_t);
  with_format(up, [&](auto f) {
    using F = decltype(f);
    const dim3 b(kW4Waves * 64);
    if (slots <= 16) {
      hipLaunchKernelGGL((w4_gate_up_kernel<F, 1>), dim3(up.nt, used), b, lds, s, mg, mu, x, idx,
                         slots, k, first, E, act);
      hipLaunchKernelGGL((w4_down_kernel<F, 1, 1>), dim3(down.nt, used), b, lds, s, md, act, idx,
                         slots, first, E, y);
    } else {
      hipLaunchKernelGGL((w4_gate_up_kernel<F, 2>), dim3(up.nt, used), b, lds, s, mg, mu, x, idx,
                         slots, k, first, E, act);
      hipLaunchKernelGGL((w4_down_kernel<F, 1, 2>), dim3(down.nt, used), b, lds, s, md, act, idx,
                         slots, first, E, y);
    }
  });
}

void launch_w4_combine(const float *y, const float *w, const int32_t *idx, int first, int E,
                       const float *ys, uint16_t *out, int T, int k, int H, hipStream_t s) {
  const int HC = H / 4;
  hipLaunchKernelGGL(w4_combine_kernel, dim3((HC + 255) / 256, T), dim3(256), 0, s,
                     (const float4 *)y, w, idx, first, E, (const float4 *)ys, (uint2 *)out, k, HC);
}

}  // namespace moe
