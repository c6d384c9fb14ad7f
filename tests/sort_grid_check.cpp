// Launch shapes of the expert-sorted rows on the host: for every size up to the
// documented limits the grid is one that the runtime takes (threads of a
// dimension below 2^32, y and z below 2^16), holds every workgroup, and stays
// inside the 31 bits of the kernels' workgroup and token numbers.
#include <cstdio>

#include "../mixture_experts_layer_offsets_amd/csrc/sort_grid.h"

using namespace moe;

static int bad = 0;

static void check(const char *what, long T, int E, long RB, const GridDims &g, int threads,
                  long rows, long per_row, long blocks) {
  // rows x per_row: the two dimensions that number the workgroups
  const bool ok = (long)g.x * threads < (1L << 32) && g.x > 0 && g.y > 0 && g.z > 0 &&
                  g.y < 65536 && g.z < 65536 && rows * per_row >= blocks &&
                  rows * per_row - blocks < rows && rows * per_row < (1L << 31);
  if (ok) return;
  if (bad++ < 20)
    printf("%s T=%ld E=%d RB=%ld: grid %u x %u x %u for %ld workgroups\n", what, T, E, RB, g.x, g.y,
           g.z, blocks);
}

int main() {
  const long Ts[] = {1, 2, 3, 4, 5, 63, 1000, 8192, 65534, 65535, 65536, 65537, 131070, 131071,
                     1000003, (1L << 24) - 8193, (1L << 24) - 8192, (1L << 24) - 1, 1L << 24};
  const int Es[] = {1, 7, 256, 1024};
  const long RBs[] = {16, 18, 40, 1000, 1024, 2048, 2050, 14336, 1L << 22};
  for (long T : Ts)
    for (int E : Es)
      for (long RB : RBs)
        for (int padded = 0; padded < 2; padded++) {
          const long pads = padded ? (long)E * kPadSplit : 0;
          const RowGrid r = row_grid(T, RB);
          const long tokens = (long)r.token_blocks * (64 >> r.lsh);
          if (tokens < T || tokens >= T + 64 || (r.lsh < 6 && r.x != 1)) {
            printf("row_grid T=%ld RB=%ld\n", T, RB);
            bad++;
          }
          const GridDims g = r.dims(r.token_blocks + pads);
          check("rows", T, E, RB, g, kRowBlock, g.z, g.y, r.token_blocks + pads);
          const BwdGrid b = bwd_grid(T, RB);
          const GridDims h = b.dims(pads);
          if ((long)b.token_blocks * (b.wide ? 1 : 4) < T) {
            printf("bwd_grid T=%ld RB=%ld\n", T, RB);
            bad++;
          }
          check("backward", T, E, RB, h, kBwdBlock, h.y, h.x, b.token_blocks + pads);
        }
  if (!bad) printf("ok\n");
  return bad != 0;
}
