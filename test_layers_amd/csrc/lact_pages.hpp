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
  int64_t* base;                 // [B] workspace: place in `free` of a request's first new page; -1: not served
  int32_t B, T, width, entries;
  FastDiv by_page;
};
constexpr int PLAN_THREADS = 1024;

__device__ __forceinline__ int64_t slot_len(const SlotArgs& a, int b) {
  const int64_t n = a.lens[b];
  return n < 0 ? 0 : n;
}
__device__ __forceinline__ int64_t pages_of(int64_t tokens, int64_t page) { return (tokens + page - 1) / page; }

// inclusive sum over the workgroup's threads, and over all of them
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t (&lds)[PLAN_THREADS / WAVE], int64_t& total) {
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
#pragma unroll
  for (int o = 1; o < WAVE; o *= 2) {
    const int64_t y = __shfl_up(x, o, WAVE);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == WAVE - 1) lds[wave] = x;
  __syncthreads();
  total = 0;
  int64_t before = 0;
#pragma unroll
  for (int i = 0; i < PLAN_THREADS / WAVE; ++i) {
    if (i == wave) before = total;
    total += lds[i];
  }
  return before + x;
}

// One workgroup: offsets, k_lens and left; keep(b, first row, length, base) for each request.
template <class F>
__device__ __forceinline__ void plan_slots(const SlotArgs& a, F&& keep) {
  __shared__ int64_t lds[PLAN_THREADS / WAVE];
  const int64_t page = a.by_page.d, have = min(max(a.have[0], (int64_t)0), (int64_t)a.entries), T = a.T;
  int64_t rows = 0, wanted = 0, taken = 0, refused = 0, sum;
  for (int b0 = 0; b0 < a.B; b0 += PLAN_THREADS) {
    const int b = b0 + threadIdx.x;
    const bool live = b < a.B;
    const int64_t len = live ? slot_len(a, b) : 0;
    int64_t count = live ? min(max(a.counts[b], (int64_t)0), T) : 0;
    const int64_t upto_row = rows + block_sum(count, lds, sum);
    rows += sum;
    const int64_t first = min(upto_row - count, T), end = min(upto_row, T);
    count = end - first;
    const bool fits = len <= a.width * page - count;
    const int64_t need = live && fits ? pages_of(len + count, page) - pages_of(len, page) : 0;
    const int64_t upto = wanted + block_sum(need, lds, sum);
    wanted += sum;
    const bool good = fits && (need == 0 || upto <= have);
    block_sum(good ? need : 0, lds, sum);
    taken += sum;
    block_sum(live && !good ? 1 : 0, lds, sum);
    refused += sum;
    if (live) {
      a.offsets[b + 1] = end;
      a.k_lens[b] = good ? len + count : len;
      keep(b, first, len, !good ? -1 : need ? have - 1 - (upto - need) : 0);
    }
  }
  __syncthreads();  // `left` may be what all have read `have` from
  if (threadIdx.x == 0) {
    a.offsets[0] = 0;
    a.left[0] = have - taken;
    a.left[1] = refused;
  }
}

// Row t, which is request b's (b < 0: none's)
__device__ __forceinline__ void place_row(const SlotArgs& a, int t, int b, int64_t first, int64_t len, int64_t base) {
  int64_t slot = -1, at = 0;
  if (b >= 0) {
    at = len + (t - first);
    if (base >= 0) {
      const int page = (int)a.by_page.d, n = (int)a.by_page.div((uint32_t)at), in = (int)at - n * page;
      const int held = (int)a.by_page.div((uint32_t)(len + page - 1));
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

// Both in one workgroup, for steps of few rows: all latency.
constexpr int ONE_GROUP = 1024;  // requests
__global__ __launch_bounds__(PLAN_THREADS) void slots_one_kernel(SlotArgs a) {
  __shared__ int64_t first[ONE_GROUP], len[ONE_GROUP], base[ONE_GROUP];
  plan_slots(a, [&](int b, int64_t f, int64_t l, int64_t x) { first[b] = f, len[b] = l, base[b] = x; });
  __syncthreads();
  const int64_t rows = a.B > 0 ? a.offsets[a.B] : 0;  // written by this workgroup before the barrier
  for (int t = threadIdx.x; t < a.T; t += PLAN_THREADS) {
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

__global__ __launch_bounds__(PLAN_THREADS) void slots_plan_kernel(SlotArgs a) {
  plan_slots(a, [&](int b, int64_t, int64_t, int64_t x) { a.base[b] = x; });
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
  if (a.B > 0 && t < a.offsets[a.B]) place_row(a, t, lo, a.offsets[lo], slot_len(a, lo), a.base[lo]);
  else place_row(a, t, -1, 0, 0, 0);
}

// ------------------------------------------------------------------ write
// Rows of k and v to their slots, 16 bytes a thread and access.
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
