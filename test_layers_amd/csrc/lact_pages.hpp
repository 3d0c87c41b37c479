// Kernels of a paged cache: where the new tokens of a step go, and their
// copies there.  (Attention over the pages: lact_attention.hpp.)
#pragma once
#include "lact_attention.hpp"

namespace lact {

// ------------------------------------------------------------------ slots
// Request b holds lens[b] tokens and gets counts[b] more.  With c_b the counts
// cut to the step's rows, off the exclusive sum of c, and
//   need_b = ceil((lens_b + c_b) / page) - ceil(lens_b / page),
// request b is served if its tokens fit its row of the table and the inclusive
// sum of need (over requests that fit) is at most what is free; its i-th new
// page is then free[have - 1 - (exclusive sum) - i].  Token i of b stands at
// lens_b + i; a page whose first place is a new token's is a new one, so that
// the thread of that token enters it in the table, and nothing that is read is
// written.
struct SlotArgs {
  const int64_t *lens, *counts;  // [B]
  int32_t* table;                // [B, width]
  const int32_t* free;           // [entries]: free pages, the next one last
  const int64_t* have;           // [1]
  int64_t *offsets, *k_lens;     // [B + 1], [B]
  int64_t *slots, *positions;    // [T]
  int64_t* left;                 // [2]: free pages left, requests not served
  int32_t* base;                 // [B] workspace: place in `free` of a request's first new page; -1: not served
  int32_t B, T, width, entries;
  FastDiv by_page;
};
constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ int64_t slot_len(const SlotArgs& a, int b) {
  const int64_t n = a.lens[b];
  return n < 0 ? 0 : n;
}
__device__ __forceinline__ int pages_of(const SlotArgs& a, int tokens) {
  return (int)a.by_page.div((uint32_t)(tokens + (int)a.by_page.d - 1));
}

// Inclusive sum over the first `waves` waves of the workgroup, cut at `most`
// (x and most at most 2^30: no step leaves 32 bits), and in `total` over all.
__device__ __forceinline__ int cut_sum(int x, int most, int waves, int (&lds)[PLAN_THREADS / WAVE], int& total) {
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  for (int o = 1; o < WAVE; o *= 2) {
    const int y = __shfl_up(x, o, WAVE);
    if (lane >= o) x = min(x + y, most);
  }
  if (lane == WAVE - 1) lds[wave] = x;
  __syncthreads();
  int before = 0;
  total = 0;
  for (int i = 0; i < waves; ++i) {
    if (i == wave) before = total;
    total = min(total + lds[i], most);
  }
  return wave < waves ? min(before + x, most) : total;
}

// A workgroup's sums over all requests: keep(b, first row, rows, length, base,
// whether it is served) for each, and in a.left (where `write`) what is left.
template <class F>
__device__ __forceinline__ void plan_slots(const SlotArgs& a, bool write, F&& keep) {
  __shared__ int lds[2][PLAN_THREADS / WAVE], taken, refused;
  const int have = (int)min(max(a.have[0], (int64_t)0), (int64_t)a.entries), T = a.T, room = a.width * (int)a.by_page.d;
  int rows = 0, wanted = 0;
  if (threadIdx.x == 0) taken = refused = 0;
  for (int b0 = 0; b0 < a.B; b0 += PLAN_THREADS) {
    const int b = b0 + threadIdx.x, waves = min(PLAN_THREADS, a.B - b0 + WAVE - 1) / WAVE;
    const bool live = b < a.B;
    const int64_t len = live ? slot_len(a, b) : 0;
    int count = live ? (int)min(max(a.counts[b], (int64_t)0), (int64_t)T) : 0, sum;
    if (b0) __syncthreads();
    const int end = min(rows + cut_sum(count, T, waves, lds[0], sum), T);
    // the sum before this request, which is not the difference where the sum was cut
    int first = __shfl_up(end, 1, WAVE);
    if (threadIdx.x % WAVE == 0) {
      first = rows;
      for (int i = 0; i < (int)threadIdx.x / WAVE; ++i) first = min(first + lds[0][i], T);
    }
    rows = min(rows + sum, T);
    count = end - first;
    const bool fits = len <= room - count;
    const int need = live && fits ? pages_of(a, (int)len + count) - pages_of(a, (int)len) : 0;
    const int upto = min(wanted + cut_sum(need, have + 1, waves, lds[1], sum), have + 1);
    wanted = min(wanted + sum, have + 1);
    const bool good = fits && (need == 0 || upto <= have);
    if (live) keep(b, first, end, len, !good ? -1 : need ? have - 1 - (upto - need) : 0);
    // what those that are served take is the largest sum that is not too much
    if (write && live) {
      if (good && need) atomicMax(&taken, upto);
      if (!good) atomicAdd(&refused, 1);
    }
  }
  __syncthreads();  // `left` may be what all have read `have` from
  if (write && threadIdx.x == 0) {
    a.offsets[0] = 0;
    a.left[0] = have - taken;
    a.left[1] = refused;
  }
}
__device__ __forceinline__ void plan_write(const SlotArgs& a, int b, int first, int end, int64_t len, int base) {
  a.offsets[b + 1] = end;
  a.k_lens[b] = base >= 0 ? len + (end - first) : len;
}

// Row t, which is request b's (b < 0: none's)
__device__ __forceinline__ void place_row(const SlotArgs& a, int t, int b, int first, int64_t len, int base) {
  int64_t slot = -1, at = 0;
  if (b >= 0) {
    at = len + (t - first);
    if (base >= 0) {
      const int page = (int)a.by_page.d, n = (int)a.by_page.div((uint32_t)at), in = (int)at - n * page;
      const int held = pages_of(a, (int)len);
      int32_t* entry = a.table + (int64_t)b * a.width + n;
      int32_t e;
      if (n < held) {
        e = *entry;
      } else {
        e = a.free[base - (n - held)];
        if (in == 0) *entry = e;
      }
      if (e >= 0) slot = (int64_t)e * page + in;
    }
  }
  a.slots[t] = slot;
  a.positions[t] = at;
}

// Steps of few requests: every workgroup sums them itself and places its rows,
// 1024 or, of a launch of one, all.  All latency: the sums (two loads, two
// barriers a sum), the table's or the free list's entry.  64 requests of one
// token 4.0 us, 1024 requests with 32768 tokens 6.8 us (summed by one workgroup
// and placed by others in a second launch 7.3 and 3.4).  One launch and two, of
// rows as many as requests: 64 5.8 and 7.5 us, 256 6.4 and 8.4, 1000 8.2 and 9.9;
// up to here 16 KB of LDS; with 64, 2000 11.3 and 13.5, 4096 17.8 and 20.0.
constexpr int ONE_GROUP = 1024;  // requests
__global__ __launch_bounds__(PLAN_THREADS) void slots_one_kernel(SlotArgs a) {
  __shared__ int first[ONE_GROUP], base[ONE_GROUP];
  __shared__ int64_t len[ONE_GROUP];
  __shared__ int rows;
  if (threadIdx.x == 0) rows = 0;
  const bool write = blockIdx.x == 0;
  plan_slots(a, write, [&](int b, int f, int e, int64_t l, int x) {
    first[b] = f, len[b] = l, base[b] = x;
    if (b == a.B - 1) rows = e;
    if (write) plan_write(a, b, f, e, l, x);
  });
  for (int t = blockIdx.x * PLAN_THREADS + threadIdx.x; t < a.T; t += gridDim.x * PLAN_THREADS) {
    int lo = 0, hi = a.B;  // the last request that begins at t or before it
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid] <= t) lo = mid;
      else hi = mid;
    }
    if (t < rows) place_row(a, t, lo, first[lo], len[lo], base[lo]);
    else place_row(a, t, -1, 0, 0, 0);
  }
}

// Many requests: one workgroup sums, the others place in a second launch.
__global__ __launch_bounds__(PLAN_THREADS) void slots_plan_kernel(SlotArgs a) {
  plan_slots(a, true, [&](int b, int f, int e, int64_t l, int x) {
    a.base[b] = x;
    plan_write(a, b, f, e, l, x);
  });
}
// A row a thread; a wave finds its first and last rows' requests by 64 tries at
// once, and each lane its own among those.
__global__ __launch_bounds__(256) void slots_fill_kernel(SlotArgs a) {
  const int t = blockIdx.x * 256 + threadIdx.x, lane = threadIdx.x % WAVE, t0 = t - lane;
  if (t0 >= a.T) return;
  auto from = [&](int to) { return find_last(a.B, lane, [&](int i) { return a.offsets[i] <= to; }); };
  int lo = max(0, from(t0)), hi = max(0, from(min(t0 + WAVE, a.T) - 1)) + 1;
  if (t >= a.T) return;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  if (a.B > 0 && t < a.offsets[a.B]) place_row(a, t, lo, (int)a.offsets[lo], slot_len(a, lo), a.base[lo]);
  else place_row(a, t, -1, 0, 0, 0);
}

// ------------------------------------------------------------------ write
// Rows of k and v to their slots, 16 bytes a thread and access.  Bound by
// memory: 32768 tokens of 8 heads of 128 in bf16 45 us, 5.9 TB/s of what it reads
// and writes; 64 tokens 2.4 us.
struct WriteArgs {
  const char* in[2];
  char* out[2];
  AttnStride si[2], so[2];  // of the rows (h, l) and of the pool (b: pages, h, l)
  const int64_t* slots;
  int64_t places;           // pages * page
  int32_t T, tokens;        // rows; rows of a workgroup
  FastDiv by_row, by_head, by_page;  // chunks of a row of all heads, of both tensors; of a head
};
__global__ __launch_bounds__(256) void page_write_kernel(WriteArgs a) {
  const int t0 = blockIdx.x * a.tokens, per = (int)a.by_row.d, items = min(a.tokens, a.T - t0) * per, half = per / 2;
#pragma unroll 4
  for (int i = threadIdx.x; i < items; i += 256) {
    const int r = (int)a.by_row.div((uint32_t)i);
    int c = i - r * per;
    const int w = c >= half ? 1 : 0;
    c -= w * half;
    const int h = (int)a.by_head.div((uint32_t)c), x = (c - h * (int)a.by_head.d) * 16;
    const int64_t slot = a.slots[t0 + r];
    if (slot < 0 || slot >= a.places) continue;
    const int n = (int)a.by_page.div((uint32_t)slot), in = (int)slot - n * (int)a.by_page.d;
    const uint4 v = *reinterpret_cast<const uint4*>(a.in[w] + h * a.si[w].h + (int64_t)(t0 + r) * a.si[w].l + x);
    *reinterpret_cast<uint4*>(a.out[w] + n * a.so[w].b + h * a.so[w].h + in * a.so[w].l + x) = v;
  }
}

}  // namespace lact
