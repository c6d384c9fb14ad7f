// Which of a stage's output scales a lane of the 8-bit weight gradient loads into LDS
// (f8_gemm.hip).  Plain integer functions, compiled for the device by the kernel and for
// the host by tests/f8_scales_check.cpp.
//
// A tile's 256 outputs lie in 16 tiles of 16; a wave's ni tiles are loaded in two halves,
// ni / 2 of them each.  The scales go the same way: 8 tiles of either half, 4 bytes a lane of
// the first two waves.  The other waves issue the same load (all count the same loads), of
// zeros.
#pragma once

#if defined(__HIPCC__)
#define F8_SCALES_FN __host__ __device__ __forceinline__
#else
#define F8_SCALES_FN inline
#endif

namespace moe {

// Byte of thread tid's scale, from the tile's first output's.  All of it is the load's vector
// offset: a scalar offset need not be part of the buffer's range check, and past the last
// column there is no memory of the stage's own.
F8_SCALES_FN int f8_scale_at(int tid, int half, int ni) {
  const int t = tid >> 4, h = ni / 2;
  return (t / h * ni + t % h + half * h) * 64 + (tid & 15) * 4;
}

// Bytes that the range check lets through, `cols` columns (a multiple of 16) from the tile's
// first output on.
F8_SCALES_FN int f8_scale_bytes(int wave, int cols) {
  return wave < 2 ? (cols < 256 ? cols : 256) * 4 : 0;
}

}  // namespace moe
