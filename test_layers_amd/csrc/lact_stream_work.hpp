// Whole numbers of the streams of key tiles (stream_kernel), apart from the
// kernels so that a host program can run them: how much work there is, which
// part of it a unit is, and how many parts an item has.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lact {

#define LACT_BOTH __host__ __device__ __forceinline__

// Work is counted in 32 bits.  The host chooses `unit` so that sequences whose
// offsets do not decrease have at most STREAM_MOST units.  Others may have any
// number, since the same rows can be many sequences': their sum is cut there,
// so that sums never decrease and what lies behind is left out.
constexpr int STREAM_MOST = 1 << 30;

// tiles of a unit, for `items` of up to `tiles` each
inline int stream_unit(int64_t items, int64_t tiles) {
  int unit = 1;
  while (items * ((tiles + unit - 1) / unit) > STREAM_MOST && unit < tiles) unit *= 2;
  return unit;
}
LACT_BOTH int stream_work(int rtiles, int units, int heads) {
  const int64_t n = (int64_t)rtiles * units * heads;
  return n < STREAM_MOST ? (int)n : STREAM_MOST;
}
LACT_BOTH int stream_add(int x, int y) {  // of sums, at most 2^31 before it is cut
  const uint32_t sum = (uint32_t)x + (uint32_t)y;
  return sum < (uint32_t)STREAM_MOST ? (int)sum : STREAM_MOST;
}

// The runs of `waves` waves: wave w has the units run w .. run (w + 1) - 1 of `work`.
LACT_BOTH int stream_run(int work, int waves, int share) {
  const int run = (work + waves - 1) / waves;
  return run > share ? run : share;
}

// What a wave at unit t, up to unit t1, does of a sequence whose work begins at
// `before`: units u0 .. u1 - 1 of an item.
struct StreamTake {
  int item, u0, u1;
  LACT_BOTH StreamTake(int t, int t1, int before, int units) {
    const int local = t - before;
    item = local / units;
    u0 = local - item * units;
    u1 = units < u0 + (t1 - t) ? units : u0 + (t1 - t);
  }
};

// An item that a wave enters at unit u0 > 0, the first of its run: whether it
// began in the run before, there as its first item or a later one (the number
// of the first part; two to a wave), and how many runs it lies in.  `left`: work
// from u0 on, which may end inside the item.
struct StreamParts {
  bool begins;
  int part, parts;
  LACT_BOTH StreamParts(int wave, int u0, int units, int run, int left) {
    begins = u0 > 0 && u0 <= run;
    part = 2 * (wave - 1) + (u0 < run ? 1 : 0);
    parts = 2 + ((units - u0 < left ? units - u0 : left) - 1) / run;
  }
};

}  // namespace lact
