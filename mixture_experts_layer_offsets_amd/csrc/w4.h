// Host-side launchers of the w4_*.hip files (all asynchronous on stream `s`).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kW4Mx = 0, kW4Int = 1;
constexpr int kW4MaxSlots = 4096;  // T*k of one few-token layer call, at most

// A checked moe_w4_shape and the pieces of its packed buffer.  Tiles of 16
// outputs x 128 contraction values: nt = ceil(n / 16), ks = ceil(k / 128);
// spg scales per output and tile.  See
// w4_device.h for the layout of a tile.
struct W4Dims {
  int groups, n, k, fmt, group, f16_scales, zeros;
  int nt, ks, spg;
  size_t code_bytes, scale_bytes, zero_bytes;  // each piece, rounded up to 256
  size_t bytes() const { return code_bytes + scale_bytes + zero_bytes; }
};

void launch_w4_pack(const W4Dims &d, const uint8_t *codes, const void *scales,
                    const uint8_t *zeros, void *packed, hipStream_t s);
void launch_w4_quantize(const W4Dims &d, const uint16_t *w, void *packed, hipStream_t s);
void launch_w4_unpack(const W4Dims &d, const void *packed, float *w, hipStream_t s);

// out[r][:] = x[r] W_g for the rows r in [offsets[g], offsets[g + 1]) (offsets
// null: one group, all rows).
void launch_w4_linear(const W4Dims &d, int rows, const uint16_t *x, long xstride,
                      const int32_t *offsets, const void *packed, uint16_t *out, long ostride,
                      hipStream_t s);

// The few-token expert FFN: gate/up [E][H][I] and down [E][I][H], routing idx
// and w [T][k] (ids less `first`; others are masked), the shared expert's
// matrices if `shared`.  act [T k][I], y [T k][H], act_s [T][Is], y_s [T][H] and
// plan (w4_plan_words) are scratch.
struct W4Layer {
  W4Dims up, down, up_s, down_s;
  bool shared;
  int T, k, first;
  const uint16_t *x;
  const int32_t *idx;
  const float *w;
  const void *w_gate, *w_up, *w_down, *ws_gate, *ws_up, *ws_down;
  uint16_t *act, *act_s, *out;
  float *y, *y_s;
  int32_t *plan;
};
size_t w4_plan_words(int slots, int E);
void launch_w4_ffn(const W4Layer &a, hipStream_t s);

}  // namespace moe
