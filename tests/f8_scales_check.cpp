// Host check of the scales' addresses in the 8-bit weight gradient's loop (f8_scales.h,
// compiled here with g++).  For every number of columns: a lane's load either starts past
// what the buffer's range check lets through, or lies whole inside the stage's own scales,
// of which the last stage's end where the workspace's piece may end; and each output's
// scale reaches the place where the wave that owns the output reads it.  Prints one line
// per failure, exit status 1 if any.
#include <cstdio>
#include <vector>

#include "../mixture_experts_layer_offsets_amd/csrc/f8_scales.h"

static int failures = 0;
#define CHECK(c, ...)                   \
  do {                                  \
    if (!(c)) {                         \
      std::printf(__VA_ARGS__);         \
      std::printf("\n");                \
      ++failures;                       \
    }                                   \
  } while (0)

constexpr int kThreads = 512;

static void columns(int n, int ni) {
  const int pitch = (n + 15) / 16 * 16, waves_n = 16 / ni;
  for (int n0 = 0; n0 < n; n0 += 256) {
    const int cols = pitch - n0;
    std::vector<int> lds(2 * 512, -1);  // output (from n0) whose scale a place of either half holds
    for (int half = 0; half < 2; half++)
      for (int tid = 0; tid < kThreads; tid++) {
        const int wave = tid / 64, at = moe::f8_scale_at(tid, half, ni);
        const int bytes = moe::f8_scale_bytes(wave, cols);
        CHECK(at >= 0 && at % 4 == 0, "ni %d tid %d half %d: offset %d", ni, tid, half, at);
        CHECK(bytes <= cols * 4, "n %d ni %d wave %d: %d bytes of %d columns", n, ni, wave, bytes, cols);
        CHECK(at >= bytes || at + 4 <= bytes, "n %d ni %d tid %d half %d: %d straddles %d", n, ni, tid,
              half, at, bytes);
        if (at < bytes) lds[half * 512 + tid] = at / 4;  // a wave's 64 lanes side by side
      }
    for (int c = 0; c < 256 && n0 + c < pitch; c++) {
      const int t = c / 16, wave_n = t / ni, half = t % ni / (ni / 2);
      const int place = half * 512 + (wave_n * (ni / 2) + t % (ni / 2)) * 16 + c % 16;
      CHECK(wave_n < waves_n && lds[place] == c, "n %d ni %d: output %d's place holds %d", n, ni, n0 + c,
            lds[place]);
    }
  }
}

int main() {
  for (int ni : {4, 8})
    for (int n = 1; n <= 2 * 256 + 20; n++) columns(n, ni);
  if (!failures) std::puts("ok");
  return failures ? 1 : 0;
}
