// The streams' whole numbers on the host, for offsets in and out of order: every
// item that a wave takes is one of its sequence, every part has its place.
// Prints "N walks, F failures".
#include <stdio.h>
#include <stdlib.h>
#include <vector>

#include "lact_stream_work.hpp"

using namespace lact;

static uint64_t state = 1;
static int64_t below(int64_t n) {  // a linear congruential generator's upper bits
  state = state * 6364136223846793005u + 1442695040888963407u;
  return (int64_t)((state >> 33) % (uint64_t)n);
}
static int failures = 0;
static void want(bool ok, const char* what, int64_t a, int64_t b) {
  if (!ok && failures++ < 10) printf("%s: %lld, %lld\n", what, (long long)a, (long long)b);
}

// the last i < n with upto[i] <= t, as the kernel's search finds it: a step of 64 tries after another
static int find(const std::vector<int>& upto, int n, int t) {
  int lo = 0;
  while (n > 0) {
    const int step = (n + 63) / 64;
    int hits = 0;
    for (int lane = 0; lane < 64; ++lane) hits += lane * step < n && upto[lo + lane * step] <= t;
    if (hits == 0) return lo - 1;
    lo += (hits - 1) * step;
    if (step == 1) return lo;
    n = step < n - (hits - 1) * step ? step : n - (hits - 1) * step;
    lo += 1, n -= 1;
  }
  return lo - 1;
}

// `batch` sequences of up to `few` rows (others have none here) and `keys` keys, G query heads to each of Hk key heads
static void walk(int batch, int Hk, int G, int tokens, int longest, int keys, int waves, bool order, bool full) {
  const int few = longest < (G < 32 ? 32 / G : 1) ? longest : G < 32 ? 32 / G : 1;
  std::vector<int> offsets(batch + 1), klen(batch), rtiles(batch), units(batch), upto(batch + 1);
  for (auto& x : offsets) x = (int)below(tokens + 1);
  if (!order) {  // as many sequences with rows as there can be
    for (int b = 0; b + 1 <= batch; b += 2) {
      offsets[b] = (int)below(tokens);
      offsets[b + 1] = offsets[b] + few < tokens ? offsets[b] + few : tokens;
    }
  } else {
    std::vector<int> rows(batch, 0);
    for (int i = 0; i < tokens; ++i) ++rows[below(batch)];
    offsets[0] = 0;
    for (int b = 0; b < batch; ++b) offsets[b + 1] = offsets[b] + rows[b];
  }
  const int64_t both = (int64_t)batch * ((G * few + 31) / 32), found = (int64_t)tokens * ((G + 31) / 32);
  const int64_t items = (both < found ? both : found) * Hk, tiles = (keys + 31) / 32 + 2;
  const int unit = stream_unit(items, tiles);
  int64_t sum = 0;
  for (int b = 0; b < batch; ++b) {
    const int n = offsets[b + 1] - offsets[b];
    klen[b] = full ? keys : (int)below(keys + 1);
    rtiles[b] = n <= 0 || n > few ? 0 : (G * n + 31) / 32;
    const int t = (klen[b] + 31) / 32;
    units[b] = t == 0 ? 1 : (t + unit - 1) / unit;
    upto[b + 1] = stream_add(upto[b], stream_work(rtiles[b], units[b], Hk));
    sum += (int64_t)rtiles[b] * units[b] * Hk;
    want(upto[b + 1] >= upto[b], "a sum decreases", upto[b], upto[b + 1]);
  }
  if (order) want(sum <= STREAM_MOST && upto[batch] == sum, "a sum of sequences in order", sum, upto[batch]);
  const int work = upto[batch], run = stream_run(work, waves, 2);
  want(work >= 0 && (int64_t)run * waves >= work, "work", work, run);
  for (int w = 0; w < waves && failures < 10; ++w) {
    const int t0 = work < (int64_t)w * run ? work : w * run, t1 = work < (int64_t)t0 + run ? work : t0 + run;
    for (int t = t0; t < t1;) {
      const int b = find(upto, batch, t);
      want(b >= 0 && b < batch, "sequence", b, batch);
      const StreamTake x(t, t1, upto[b], units[b]);
      want(x.item >= 0 && x.item < rtiles[b] * Hk, "item", x.item, rtiles[b] * Hk);
      want(x.u0 >= 0 && x.u0 < x.u1 && x.u1 <= units[b], "unit", x.u0, x.u1);
      if (failures) return;
      if (t == t0 && x.u0 > 0) {
        const StreamParts p(w, x.u0, units[b], run, work - t);
        if (p.begins) {
          want(p.part >= 0 && p.part < 2 * waves, "first part", p.part, 2 * waves);
          want(p.parts >= 2 && (p.part & ~1) + 2 * (p.parts - 1) < 2 * waves, "last part", p.part, p.parts);
        }
      }
      t += x.u1 - x.u0;
    }
  }
}

int main() {
  int n = 0;
  // in order: every unit counts
  for (int i = 0; i < 200; ++i, ++n) {
    const int batch = 1 + (int)below(400), G = 1 << below(7), tokens = 1 + (int)below(600);
    walk(batch, 1 + (int)below(64), G, tokens, 1 + (int)below(tokens), 1 + (int)below(1 << 16), 4 * (1 + (int)below(512)), true, below(2));
  }
  // so many sequences with the same rows that sums pass 2^31 and 2^32
  const int many[][5] = {{10452, 64, 1, 8, 1 << 20}, {1024, 8, 1, 64, 1073676288}, {16384, 8, 4, 8, 1 << 20}, {4096, 1, 1, 32, 1 << 29},
                         {300, 64, 64, 3, 1 << 29}, {100000, 1, 2, 16, 1 << 20}};
  for (auto& c : many)
    for (int i = 0; i < 4; ++i, ++n) walk(c[0], c[1], c[2], c[3], c[3], c[4], i % 2 ? 1024 : 2048, false, i < 2);
  // and short ones
  for (int i = 0; i < 200; ++i, ++n) {
    const int tokens = 1 + (int)below(100);
    walk(1 + (int)below(3000), 1 + (int)below(16), 1 + (int)below(40), tokens, 1 + (int)below(tokens), 1 + (int)below(5000), 4 * (1 + (int)below(512)),
         false, below(2));
  }
  // sums do not depend on how they are grouped
  for (int i = 0; i < 100000; ++i) {
    const int a = (int)below(STREAM_MOST + 1LL), b = (int)below(STREAM_MOST + 1LL), c = (int)below(STREAM_MOST + 1LL);
    want(stream_add(stream_add(a, b), c) == stream_add(a, stream_add(b, c)), "order of a sum", a, b);
    want(stream_add(a, b) >= a && stream_add(a, b) <= STREAM_MOST, "a sum", a, b);
  }
  printf("%d walks, %d failures\n", n, failures);
  return failures != 0;
}
