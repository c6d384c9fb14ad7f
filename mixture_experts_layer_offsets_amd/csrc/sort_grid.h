// Launch shapes of the expert-sorted rows: workgroups, numbered b = 0, 1, ...,
// spread over grid dimensions that the runtime takes (threads of a dimension
// below 2^32, y and z below 2^16).  Plain integer functions, also compiled for
// the host by tests/sort_grid_check.cpp.
#pragma once

namespace moe {

constexpr int kRowBlock = 64;    // one wave per workgroup for the gathers (see combine_kernel)
constexpr int kBwdBlock = 256;   // threads of a workgroup of the weighted return's gradient
// Workgroups that share one expert's padding rows (65536 rows of 7168 bf16 over 256
// experts to 128 rows: 255 us with 8, 257 to 260 with 2, 4, 16 and 32).
constexpr int kPadSplit = 8;

struct GridDims {
  unsigned x, y, z;
};

// `blocks` (at least 1) as outer x inner, inner at most 65535 and no more than
// `outer` - 1 of the products too many.
inline void split_blocks(long blocks, unsigned &inner, unsigned &outer) {
  outer = (unsigned)((blocks + 65534) / 65535);
  inner = (unsigned)((blocks + outer - 1) / outer);
}

// How a launch maps lanes to rows: 2^lsh lanes share a token (all 64 when its
// row has 64 chunks of 16 bytes or more, then grid x walks the row), 64 >> lsh
// tokens a wave.  Grid y and z count the workgroups that differ in their tokens:
// `token_blocks` of them hold tokens, the ones behind them (E x kPadSplit) zero
// the padding rows.  The row's chunks are the fastest index, so that a row is
// written at one time: with them as the slowest index the sort of 65536 rows of
// 7168 bf16 took 232 us instead of 224, the backward sort of 8192 rows 24.8 us
// instead of 20.4, and the weighted return of 32768 kept rows 55 instead of 48.
struct RowGrid {
  int lsh, token_blocks;
  unsigned x;
  GridDims dims(long blocks) const {  // b = z gridDim.y + y
    GridDims g;
    g.x = x;
    split_blocks(blocks, g.y, g.z);
    return g;
  }
};

inline RowGrid row_grid(long T, long row_bytes) {
  const long nc = (row_bytes + 15) / 16;
  RowGrid g;
  g.lsh = 0;
  while (g.lsh < 6 && (1L << g.lsh) < nc) g.lsh++;
  const int per = 64 >> g.lsh;
  g.token_blocks = (int)((T + per - 1) / per);
  g.x = (unsigned)((nc + 63) >> 6);
  return g;
}

// The gradient of the weighted return: four waves for a token whose row has more
// than 128 chunks, else one.
struct BwdGrid {
  bool wide;
  int token_blocks;
  GridDims dims(long pad_blocks) const {  // b = y gridDim.x + x
    GridDims g;
    g.z = 1;
    split_blocks(token_blocks + pad_blocks, g.x, g.y);
    return g;
  }
};

inline BwdGrid bwd_grid(long T, long row_bytes) {
  BwdGrid g;
  g.wide = row_bytes > 128 * 16;
  g.token_blocks = (int)(g.wide ? T : (T + 3) / 4);
  return g;
}

}  // namespace moe
