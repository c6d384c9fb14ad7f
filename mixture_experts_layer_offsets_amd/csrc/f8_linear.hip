// Products of few rows in 8 bits with a scale per block of 128 (f8_device.h): the
// weights go from memory straight into registers, and the waves of a workgroup split
// the contraction of one tile of 16 outputs.
#include <algorithm>

#include "f8_device.h"

namespace moe {

namespace {

// Quantised rows as launch_f8_quant_rows leaves them ...
struct FromCodes {
  const uint8_t *codes;
  const float *scales;
  long rows;
  struct Raw { u32x4_t a, b; float s; };
  __device__ __forceinline__ Raw load(long r, int st, int h) const {
    const size_t at = (size_t)st * rows + r;
    const u32x4_t *p = (const u32x4_t *)(codes + at * kF8Block);
    return {p[h], p[h + 4], scales[at]};
  }
  __device__ __forceinline__ Raw load_end(long r, int st, int h, int) const { return load(r, st, h); }
  static __device__ __forceinline__ i32x8_t codes_of(const Raw &w, float *s) {
    *s = w.s;
    return f8_frag(w.a, w.b);
  }
};

// ... or 16-bit rows, quantised here: every workgroup repeats that for its own tile,
// which takes less than the weights of a step take to arrive.
template <bool F16>
struct FromRows {
  const uint16_t *x;
  long stride;
  struct Raw { u32x4_t v[4]; };
  __device__ __forceinline__ Raw load(long r, int st, int h) const {
    const uint16_t *p = x + r * stride + st * kF8Block + 16 * h;
    Raw w;
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const u32x4_a2 u = *(const u32x4_a2 *)(p + 64 * (i >> 1) + 8 * (i & 1));
      w.v[i] = (u32x4_t){u[0], u[1], u[2], u[3]};
    }
    return w;
  }
  // the step that the row ends in
  __device__ __forceinline__ Raw load_end(long r, int st, int h, int k) const {
    const uint16_t *p = x + r * stride;
    Raw w;
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const int c = st * kF8Block + 64 * (i >> 1) + 16 * h + 8 * (i & 1) + 2 * e;
        const uint32_t lo = c < k ? p[c] : 0;
        w.v[i][e] = lo | (c + 1 < k ? (uint32_t)p[c + 1] << 16 : 0);
      }
    return w;
  }
  static __device__ __forceinline__ i32x8_t codes_of(const Raw &w, float *s) {
    float v[32];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; i++) {
      v[i] = f8_from16((w.v[i >> 3][(i >> 1) & 3] >> (16 * (i & 1))) & 0xFFFFu, F16);
      top = max(top, f8_mag(v[i]));
    }
    // the row's other values of the block: lanes l % 16 + 16 h
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
    float inv;
    *s = f8_scale(top, &inv);
    i32x8_t c;
#pragma unroll
    for (int i = 0; i < 8; i++)
      c[i] = (int)f8_codes4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3], inv);
    return c;
  }
};

struct Few {
  const uint8_t *tiles;
  const float *ws;
  const int32_t *offsets;
  uint16_t *out;
  long ostride;
  int rows, n, k, nt, ks, f16;
};

// Up to 16 rows a pass.  The loads of U steps go out together.  Grid (output tiles,
// groups, passes that run side by side).
template <class Src, int WAVES, int U>
__global__ __launch_bounds__(WAVES * 64) void f8_few_kernel(Few p, Src src) {
  __shared__ float red[WAVES * 256];
  const int g = blockIdx.y, t = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), h = lane >> 4;
  const F8Span sp = f8_span(p.offsets, g, p.rows);
  const f8_rsrc_t rW =
      f8_buffer(p.tiles + ((size_t)g * p.nt + t) * p.ks * kF8Tile, p.ks * kF8Tile);
  const float *ws = p.ws + ((size_t)g * p.nt + t) * p.ks;
  const int s0 = p.ks * wave / WAVES, s1 = p.ks * (wave + 1) / WAVES, full = min(s1, p.k / kF8Block);
  for (long r0 = sp.begin + 16L * blockIdx.z; r0 < sp.end; r0 += 16L * gridDim.z) {
    const int nr = (int)min(16L, sp.end - r0);
    const long r = r0 + min(lane & 15, nr - 1);
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    auto weights = [&](int st, u32x4_t *w) {  // read once: not kept in the caches
#pragma unroll
      for (int i = 0; i < 2; i++)
        w[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                                               rW, lane * 16 + 1024 * i, st * kF8Tile, 2));
    };
    auto step = [&](const u32x4_t *w, const typename Src::Raw &x, float sw) {
      float s;
      const i32x8_t c = Src::codes_of(x, &s);
      const f32x4 d = f8_dot(f8_frag(w[0], w[1]), c);
      s *= sw;
#pragma unroll
      for (int v = 0; v < 4; v++) acc[v] = fmaf(s, d[v], acc[v]);
    };
    for (int st = s0; st < full; st += U) {
      u32x4_t w[U][2];
      typename Src::Raw x[U];
      float sw[U];
#pragma unroll
      for (int u = 0; u < U; u++) {  // past the end: the last step again, not used
        const int at = min(st + u, full - 1);
        weights(at, w[u]);
        x[u] = src.load(r, at, h);
        sw[u] = ws[at];
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < U; u++)
        if (st + u < full) step(w[u], x[u], sw[u]);
    }
    if (full < s1) {  // the contraction ends inside this step
      u32x4_t w[2];
      weights(full, w);
      step(w, src.load_end(r, full, h, p.k), ws[full]);
    }
    // the waves' sums, added in wave order
#pragma unroll
    for (int v = 0; v < 4; v++) red[(wave * 4 + v) * 64 + lane] = acc[v];
    __syncthreads();
    if (tid < 256) {
      float s = red[tid];
#pragma unroll
      for (int w = 1; w < WAVES; w++) s += red[w * 256 + tid];
      const int row = tid & 15, n = 16 * t + 4 * ((tid >> 4) & 3) + (tid >> 6);
      if (row < nr && n < p.n) p.out[(r0 + row) * p.ostride + n] = f8_to16(s, p.f16);
    }
    __syncthreads();
  }
}

template <class Src>
void launch(const F8Dims &d, int rows, const Src &src, const int32_t *offsets, const void *packed,
            uint16_t *out, long ostride, hipStream_t s) {
  if (rows <= 0) return;
  const uint8_t *tiles = (const uint8_t *)packed;
  const Few p{tiles, (const float *)(tiles + d.code_bytes), offsets, out, ostride,
              rows, d.n, d.k, d.nt, d.ks, d.f16};
  const int avg = (rows + d.groups - 1) / d.groups;
  const int passes = std::min((avg + 15) / 16, 65535);
  auto go = [&](auto kernel, int waves) {
    hipLaunchKernelGGL(kernel, dim3(d.nt, d.groups, passes), dim3(waves * 64), 0, s, p, src);
  };
  const long tasks = (long)d.nt * d.groups * passes;
  if (tasks <= 256) go(f8_few_kernel<Src, 16, 2>, 16);
  else if (tasks <= 512) go(f8_few_kernel<Src, 8, 4>, 8);
  else go(f8_few_kernel<Src, 4, 4>, 4);
}

}  // namespace

bool f8_few(const F8Dims &d, int rows) { return rows <= 16L * d.groups; }

void launch_f8_few(const F8Dims &d, int rows, const uint8_t *codes, const float *scales,
                   const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                   hipStream_t s) {
  launch(d, rows, FromCodes{codes, scales, rows}, offsets, packed, out, ostride, s);
}

void launch_f8_few_rows(const F8Dims &d, int rows, const F8Rows &x, const int32_t *offsets,
                        const void *packed, uint16_t *out, long ostride, hipStream_t s) {
  if (x.f16) launch(d, rows, FromRows<true>{x.p, x.stride}, offsets, packed, out, ostride, s);
  else launch(d, rows, FromRows<false>{x.p, x.stride}, offsets, packed, out, ostride, s);
}

}  // namespace moe
