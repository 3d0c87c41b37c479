// liblact: host side of the operators around the fast-weight layer (window
// attention, rotary positions, add and norm): validation before any HIP call,
// choice of kernel, launches on the caller's stream.  Part of the library's
// one translation unit, after lact.hip.
#pragma once
#include <cmath>
#include <initializer_list>

#include "lact_attention.hpp"
#include "lact_rows.hpp"

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return a / b + (a % b != 0); }

lact_status check_dtype(int32_t t) {
  if (t != LACT_DTYPE_F32 && t != LACT_DTYPE_BF16) return fail(LACT_ERR_INVALID_ARG, "io_dtype = %d", t);
  return LACT_OK;
}
int64_t size_of(int32_t t) { return t == LACT_DTYPE_F32 ? 4 : 2; }

// A [batch, heads, tokens, d] tensor: the pointer, its strides turned to
// bytes (0 for a dimension of at most one), and what an output needs besides.
lact_status check_tensor(const char* name, const void* ptr, const lact_strides* st, int64_t batch, int64_t heads,
                         int64_t tokens, int64_t d, int64_t es, int64_t align, bool output, AttnStride* out) {
  if (!ptr) return fail(LACT_ERR_INVALID_ARG, "%s is NULL", name);
  if (!st) return fail(LACT_ERR_INVALID_ARG, "strides of %s are NULL", name);
  if (!aligned(ptr, align)) return fail(LACT_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)align);
  struct {
    int64_t n, s;
  } dim[3] = {{batch, st->batch}, {heads, st->head}, {tokens, st->token}};
  for (auto& x : dim) {
    if (x.n <= 1) {
      x.s = 0;
      continue;
    }
    // every byte offset of the tensor stays below 2^62
    if (x.s < 0 || x.s > (INT64_C(1) << 60) / x.n / es)
      return fail(LACT_ERR_INVALID_ARG, "%s has a stride of %lld", name, (long long)x.s);
    if (x.s * es % align)
      return fail(LACT_ERR_INVALID_ARG, "%s has a stride of %lld elements: need multiples of %d bytes", name,
                  (long long)x.s, (int)align);
  }
  *out = {dim[0].s * es, dim[1].s * es, dim[2].s * es};
  if (output) {
    // rows are distinct where each dimension steps over all that smaller ones span
    std::sort(dim, dim + 3, [](auto& a, auto& b) { return a.s < b.s; });
    int64_t span = d;
    for (auto& x : dim) {
      if (x.n <= 1) continue;
      if (x.s < span) return fail(LACT_ERR_INVALID_ARG, "%s: output rows overlap", name);
      span += (x.n - 1) * x.s;
    }
  }
  return LACT_OK;
}

// ------------------------------------------------------------------ window attention
constexpr int64_t MOST_TOKENS = INT64_C(1) << 30;
constexpr int64_t MOST_THREADS = (INT64_C(1) << 32) - 1;  // of a launch

lact_status validate(const lact_attention* p) {
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0) return fail(LACT_ERR_INVALID_ARG, "batch = %d < 0", p->batch);
  if (p->kv_heads < 1 || p->heads < 1 || p->heads % p->kv_heads)
    return fail(LACT_ERR_INVALID_ARG, "heads = %d, kv_heads = %d: need a positive multiple", p->heads, p->kv_heads);
  if (p->d < 8 || p->d > 128 || p->d % 8)
    return fail(LACT_ERR_UNSUPPORTED, "d = %d: need a multiple of 8 in [8, 128]", p->d);
  if ((int64_t)p->batch * p->heads > INT32_MAX)
    return fail(LACT_ERR_UNSUPPORTED, "batch * heads = %lld: more than a launch takes", (long long)p->batch * p->heads);
  lact_status r = check_dtype(p->io_dtype);
  if (r) return r;
  if (!(p->scale >= 0x1p-100f) || !(p->scale <= 0x1p100f))
    return fail(LACT_ERR_INVALID_ARG, "scale = %g: need 2^-100 .. 2^100", (double)p->scale);
  if (p->q_len < 0 || p->q_len >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "q_len = %lld", (long long)p->q_len);
  if (p->k_len < 0 || p->k_len >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "k_len = %lld", (long long)p->k_len);
  if (p->window < 0) return fail(LACT_ERR_INVALID_ARG, "window = %lld < 0", (long long)p->window);
  if (p->sinks < 0) return fail(LACT_ERR_INVALID_ARG, "sinks = %lld < 0", (long long)p->sinks);
  return LACT_OK;
}

// calls fn with the element type and the padded head width
template <class F>
lact_status by_tile(const lact_attention& p, F&& fn) {
  if (p.io_dtype == LACT_DTYPE_F32) return p.d <= 64 ? fn(float{}, IC<64>{}) : fn(float{}, IC<128>{});
  return p.d <= 64 ? fn(bf16_t{}, IC<64>{}) : fn(bf16_t{}, IC<128>{});
}

// Whether some row may not see some key before it
bool limited(const lact_attention& p) { return p.window && p.window < p.k_len && p.sinks < p.k_len; }

// keys that the 32 rows of a tile of the few-row kernel can see
int64_t few_keys(const lact_attention& p) {
  const int64_t tokens = std::min(p.q_len, ceil_div(31, p.heads / p.kv_heads) + 1);
  return limited(p) ? std::min(p.k_len, p.window + tokens - 1 + p.sinks) : p.k_len;
}

// workgroups of the few-row kernel that run at once, by its rings in LDS: 64 KB
// (bf16, d <= 64), or 128 (16 heads of 32 in fp32 over 32K keys: in one round
// of splits 65 us, in two 71)
int64_t few_room(const lact_attention& p) {
  int64_t n = 0;
  (void)by_tile(p, [&](auto t, auto dp) {
    n = LDS_MAX / few_lds<decltype(t), decltype(dp)::value>() * NCU;
    return LACT_OK;
  });
  return n;
}

// Row tiles of the few-row kernel, 0 where the other kernel takes the problem.
// A key head's rows in one tile: always.  More of them:
// - where the keys are long and split at least in two, or a few workgroups
//   walk along them while the chip waits (8 heads, 512 tokens over 8192 keys:
//   128 tiles, 81 us in the other kernel and 35 here; 2048 keys: 24 and 20;
//   1024 keys: 16.3 and 18.0; 256 tiles, unsplit at d = 128: 191 and 205);
// - where the other kernel's tiles, rows of one head each, would be empty for
//   the most part (64 heads to a key head, next tokens of a batch of 256, 1024
//   keys: 255 and 52 us; 8 to a key head, 8 tokens: 170 and 164; 16 tokens,
//   half the tiles rather than a quarter: 172 and 310).
int few_tiles(const lact_attention& p) {
  const int64_t G = p.heads / p.kv_heads, tiles = ceil_div(G * p.q_len, 32);
  if (tiles <= 1) return 1;
  const bool split = 2 * tiles * p.batch * p.kv_heads <= few_room(p) && few_keys(p) >= 1536;
  return split || (4 * tiles <= G * ceil_div(p.q_len, 32) && tiles < 65536) ? (int)tiles : 0;
}

// Key splits of the few-row kernel: enough workgroups to fill the chip, none
// with fewer keys than a round of its waves.
int few_splits(const lact_attention& p) {
  const int64_t most = std::max<int64_t>(1, ceil_div(few_keys(p), 256));
  const int64_t want = few_room(p) / std::max<int64_t>(1, (int64_t)p.batch * p.kv_heads * few_tiles(p));
  return (int)std::min<int64_t>(std::min(most, std::max<int64_t>(1, want)), 256);
}

AttnArgs attn_args(const lact_attention& p) {
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.B = p.batch;
  a.H = p.heads;
  a.Hk = p.kv_heads;
  a.G = p.heads / p.kv_heads;
  a.d = p.d;
  a.Lq = (int32_t)p.q_len;
  a.Lk = (int32_t)p.k_len;
  a.window = (int32_t)(limited(p) ? p.window : MOST_TOKENS);
  a.sinks = (int32_t)(limited(p) ? p.sinks : 0);
  a.c = p.scale * LOG2E;
  a.scale = p.scale;
  a.splits = 1;
  a.hg = 1;
  return a;
}

// Row tiles of the forward and dq kernels, `rows` of them a workgroup.  Query
// heads of one key head fill a workgroup's waves as far as they divide: all
// its rows then stand at nearly the same positions, and fewer of its tiles
// are seen in part (32K prompt with four heads to a key head, d = 64: 622 us with
// 128 rows of one head a workgroup, 611 us with 32 rows of four).
void row_tiles(const lact_attention& p, int rows, AttnArgs& a) {
  a.hg = 1;
  while (a.hg < rows / 32 && a.G % (2 * a.hg) == 0) a.hg *= 2;
  a.tiles = (int32_t)ceil_div(p.q_len, rows / a.hg);
}

// Waves that share the rows (keys) of a tile: one wave a 32-row group, or two,
// which make twice as many workgroups of half the work.  fp32 has no pipelined
// order to lose by it (16 heads x 4096: 528 us with one, 471 with two), but
// beyond d = 64 its tiles of 32 keys do not divide.  bf16, by the padded sizes,
// since the host does not know the lengths:
//
// Rows (forward, dq).  d <= 64, two workgroups a compute unit: two waves up to
// one and a half tiles of 128 a unit (1024 tokens, causal, forward: 32 - 128
// tiles 17.7 us with one and 14.4 with two, 288: 23.2 and 21.0, 384: 23.8 and
// 22.0, 448: 23.9 and 25.9; dq of 288 tiles 4 us less, of 512 4 more).  d > 64,
// where one workgroup of dq has a unit: two up to half a tile a unit, beyond
// that they run one after another (128 tiles: 23.2 and 19.0, 160: 23.5 and 25.0;
// dq of 128 tiles 5 us less, of 160 8 more).
int parts_q(const lact_attention& p) {
  const int64_t tiles = (int64_t)p.batch * p.heads * ceil_div(p.q_len, 128);
  if (p.io_dtype == LACT_DTYPE_F32) return p.d <= 64 && tiles <= 4 * NCU ? 2 : 1;
  return 2 * tiles <= (p.d <= 64 ? 3 : 1) * NCU ? 2 : 1;
}
// Keys (dk, dv): two waves up to half a tile a unit (d = 128, 4 heads to a key
// head: 8 - 27 us less; causal, 160 tiles of d = 64, 5 more).  With a window of
// at most half the keys, whose tiles meet equally many rows, up to five quarters,
// where a second round of whole tiles would be short (window 333, 4 heads to a
// key head; the backward with one wave, and what two change.  d = 64: 224 tiles
// of 1024 tokens 122 us, -26; 288: 133, -6, of 2048 tokens 142, +2; 352: 144,
// +3.  d = 128: 256 tiles 216 and 242, -21 and -7; 288: 265 and 277, -12 and
// -14; 352: 297 and 305, -13 and +14; but 160 to 224 tiles, one round, 0 to +6).
// Padded, 280 tiles, window 333, 3 heads to a key head, d = 64 and 128: all
// lengths full 114 and 222, -2 and -8; from a quarter to full 100 and 187, -18
// and -26; half 94 and 137, -20 and +12; a quarter 72 and 110, -5 and -9.
int parts_k(const lact_attention& p) {
  const int64_t tiles = (int64_t)p.batch * p.kv_heads * ceil_div(p.k_len, 128);
  if (p.io_dtype == LACT_DTYPE_F32) return p.d <= 64 && tiles <= 4 * NCU ? 2 : 1;
  if (2 * tiles <= NCU) return 2;
  if (!limited(p) || 2 * p.window > p.k_len || 4 * tiles > 5 * NCU) return 1;
  return p.d <= 64 || 8 * tiles > 7 * NCU ? 2 : 1;
}

// Key tiles of the dk, dv kernel, those of them with sinks, and the splits of
// the rows behind a sink tile's window: parts as long as what a window's tile
// meets, at most 63 of them and no more than make SINK_JOBS of all sink tiles
// together, two a compute unit.  More tiles fill the chip without being split,
// and the workspace for their parts stays below 96 MiB.  Backward, window 128,
// d = 128, as many parts as were allowed before and now (512, 1024 and 2048
// jobs): 8 x 32 heads x 4096 tokens, 4 sinks: 1689 us with 552 MiB, and 1453,
// 1449, 1530 with 104, 168, 296; 8 heads x 32K, 4096 sinks: 3690 us with 2 GiB,
// and 2510, 2357, 2466 with 98, 162, 290 MiB; 1024 sinks: 1225, and 855, 895, 990.
constexpr int64_t SINK_JOBS = 512;
void sink_plan(const lact_attention& p, int64_t BK, AttnArgs& a) {
  a.tiles = (int32_t)ceil_div(p.k_len, BK);
  a.splits = 1;
  a.sink_tiles = 0;
  if (p.sinks == 0 || !limited(p) || p.k_len <= BK) return;
  const int64_t behind = p.k_len - (BK - 1) - p.window;  // rows behind the first sink tile's window
  if (behind <= 0) return;
  const int64_t tiles = ceil_div(p.sinks, BK), most = SINK_JOBS / std::max<int64_t>(1, p.batch * p.kv_heads * tiles);
  if (most < 2) return;
  const int64_t span = std::max(p.window + BK, ceil_div(behind, std::min<int64_t>(63, most)));
  a.sink_tiles = (int32_t)tiles;
  a.span = (int32_t)span;
  a.splits = 1 + (int32_t)ceil_div(behind, span);
}

struct AttnWs {
  size_t part = 0, ml = 0, total = 0;
};
AttnWs attn_ws(const lact_attention& p) {
  AttnWs w;
  if (!few_tiles(p)) return w;
  const int s = few_splits(p);
  if (s == 1) return w;
  const size_t rows = (size_t)p.batch * p.heads * p.q_len;
  w.ml = align256(rows * s * p.d * 4);
  w.total = w.ml + align256(rows * s * 2 * 4);
  return w;
}
AttnWs attn_back_ws(const lact_attention& p) {
  AttnWs w;
  w.part = align256((size_t)p.batch * p.heads * p.q_len * 2 * 4);
  w.total = w.part;
  const int64_t BK = 128 / parts_k(p);
  AttnArgs a = attn_args(p);
  sink_plan(p, BK, a);
  if (a.splits > 1) w.total += align256((size_t)p.batch * p.kv_heads * a.sink_tiles * a.splits * 2 * BK * p.d * 4);
  return w;
}

// Outputs that are an input or each other.  Only whole tensors can be told
// here; that parts do not overlap is the caller's to keep.
lact_status check_apart(std::initializer_list<const void*> outputs, std::initializer_list<const void*> inputs) {
  for (auto o = outputs.begin(); o != outputs.end(); ++o) {
    if (!*o) continue;
    for (const void* i : inputs)
      if (i == *o) return fail(LACT_ERR_INVALID_ARG, "an output is an input");
    for (auto p = outputs.begin(); p != o; ++p)
      if (*p == *o) return fail(LACT_ERR_INVALID_ARG, "two outputs are the same");
  }
  return LACT_OK;
}

#define TRY(expr)                      \
  do {                                 \
    const lact_status s_ = (expr);     \
    if (s_) return s_;                 \
  } while (0)

lact_status check_grid(int64_t n, int threads) {
  if (n > MOST_THREADS / threads)
    return fail(LACT_ERR_UNSUPPORTED, "%lld workgroups of %d: more than a launch takes", (long long)n, threads);
  return LACT_OK;
}
lact_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return LACT_OK;
  NEED(ws, 256);
  if (have < need) return fail(LACT_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", have, need);
  return LACT_OK;
}

// calls fn with the number of waves that share a tile
template <typename T, class DP, class F>
void by_parts(T, DP, int ks, F&& fn) {
  if constexpr (sizeof(T) == 4 && DP::value > 64) fn(IC<1>{});
  else if (ks == 2) fn(IC<2>{});
  else fn(IC<1>{});
}

// check_device for calls that come every few microseconds: the device that
// this thread checked last needs no second look
lact_status check_device_again() {
  static thread_local int last = -1;
  int dev = -1;
  if (last >= 0 && hipGetDevice(&dev) == hipSuccess && dev == last) return LACT_OK;
  TRY(check_device());
  if (hipGetDevice(&dev) == hipSuccess) last = dev;
  return LACT_OK;
}

}  // namespace

extern "C" {

size_t lact_window_attention_workspace_size(const lact_attention* p) {
  g_err.clear();
  if (validate(p)) return 0;
  return attn_ws(*p).total;
}

lact_status lact_window_attention_forward(const lact_attention* p, const void* q, const lact_strides* sq,
                                          const void* k, const lact_strides* sk, const void* v,
                                          const lact_strides* sv, const int64_t* q_lens, const int64_t* k_lens,
                                          void* o, const lact_strides* so, float* lse, void* ws, size_t ws_bytes,
                                          void* stream) {
  g_err.clear();
  TRY(validate(p));
  if (p->batch == 0 || p->q_len == 0) return LACT_OK;
  AttnArgs a = attn_args(*p);
  const int64_t es = size_of(p->io_dtype);
  TRY(check_tensor("q", q, sq, p->batch, p->heads, p->q_len, p->d, es, 16, false, &a.sq));
  if (p->k_len > 0) {
    TRY(check_tensor("k", k, sk, p->batch, p->kv_heads, p->k_len, p->d, es, 16, false, &a.sk));
    TRY(check_tensor("v", v, sv, p->batch, p->kv_heads, p->k_len, p->d, es, 16, false, &a.sv));
  }
  TRY(check_tensor("o", o, so, p->batch, p->heads, p->q_len, p->d, es, 16, true, &a.so));
  if (!aligned(q_lens, 8) || !aligned(k_lens, 8)) return fail(LACT_ERR_INVALID_ARG, "lengths are not 8-byte aligned");
  if (!aligned(lse, 4)) return fail(LACT_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  TRY(check_apart({o, lse}, {q, k, v}));
  const AttnWs w = attn_ws(*p);
  TRY(check_ws(ws, ws_bytes, w.total));
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.out = static_cast<char*>(o);
  a.q_lens = q_lens;
  a.k_lens = k_lens;
  a.lse = lse;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t rows = (int64_t)p->batch * p->heads * p->q_len;
  if ((a.tiles = few_tiles(*p)) > 0) {
    a.splits = few_splits(*p);
    const int64_t grid = (int64_t)p->batch * p->kv_heads * a.tiles * a.splits;
    int threads = 0;
    TRY(by_tile(*p, [&](auto t, auto dp) {
      threads = 64 * few_waves<decltype(t), decltype(dp)::value>();
      return LACT_OK;
    }));
    TRY(check_grid(grid, threads));
    if (a.splits > 1) TRY(check_grid(rows, 256));
    TRY(check_device_again());
    if (a.splits > 1) {
      a.part = static_cast<float*>(ws);
      a.part_ml = reinterpret_cast<float*>(static_cast<char*>(ws) + w.ml);
    }
    return by_tile(*p, [&](auto t, auto dp) -> lact_status {
      using T = decltype(t);
      constexpr int DP = decltype(dp)::value, NW = few_waves<T, DP>();
      {
        KernelTimer kt(LACT_K_ATTN, s);
        LACT_LAUNCH((attn_few_kernel<T, DP>), dim3((unsigned)grid), dim3(64 * NW), s, a);
      }
      KernelTimer kt(LACT_K_ATTN, s);
      if (a.splits > 1) LACT_LAUNCH((attn_join_kernel<T, DP>), dim3((unsigned)rows), dim3(256), s, a);
      HIP_TRY(hipGetLastError());
      return LACT_OK;
    });
  }
  const int ks = parts_q(*p);
  row_tiles(*p, 128 / ks, a);
  const int64_t grid = (int64_t)p->batch * (p->heads / a.hg) * a.tiles;
  TRY(check_grid(grid, 256));
  TRY(check_device_again());
  KernelTimer kt(LACT_K_ATTN, s);
  return by_tile(*p, [&](auto t, auto dp) -> lact_status {
    by_parts(t, dp, ks, [&](auto n) {
      LACT_LAUNCH((attn_fwd_kernel<decltype(t), decltype(dp)::value, decltype(n)::value>), dim3((unsigned)grid), dim3(256), s, a);
    });
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

size_t lact_window_attention_backward_workspace_size(const lact_attention* p) {
  g_err.clear();
  if (validate(p)) return 0;
  return attn_back_ws(*p).total;
}

lact_status lact_window_attention_backward(const lact_attention* p, const void* q, const lact_strides* sq,
                                           const void* k, const lact_strides* sk, const void* v,
                                           const lact_strides* sv, const int64_t* q_lens, const int64_t* k_lens,
                                           const void* o, const lact_strides* so, const float* lse, const void* dO,
                                           const lact_strides* sdo, void* dq, const lact_strides* sdq, void* dk,
                                           const lact_strides* sdk, void* dv, const lact_strides* sdv, void* ws,
                                           size_t ws_bytes, void* stream) {
  g_err.clear();
  TRY(validate(p));
  if (p->batch == 0) return LACT_OK;
  AttnArgs a = attn_args(*p);
  const int64_t es = size_of(p->io_dtype);
  if (p->q_len > 0) {
    TRY(check_tensor("q", q, sq, p->batch, p->heads, p->q_len, p->d, es, 16, false, &a.sq));
    TRY(check_tensor("o", o, so, p->batch, p->heads, p->q_len, p->d, es, 16, false, &a.so));
    TRY(check_tensor("dO", dO, sdo, p->batch, p->heads, p->q_len, p->d, es, 16, false, &a.sdo));
    TRY(check_tensor("dq", dq, sdq, p->batch, p->heads, p->q_len, p->d, es, 16, true, &a.sdq));
    NEED(lse, 4);
  }
  if (p->k_len > 0) {
    TRY(check_tensor("k", k, sk, p->batch, p->kv_heads, p->k_len, p->d, es, 16, false, &a.sk));
    TRY(check_tensor("v", v, sv, p->batch, p->kv_heads, p->k_len, p->d, es, 16, false, &a.sv));
    TRY(check_tensor("dk", dk, sdk, p->batch, p->kv_heads, p->k_len, p->d, es, 16, true, &a.sdk));
    TRY(check_tensor("dv", dv, sdv, p->batch, p->kv_heads, p->k_len, p->d, es, 16, true, &a.sdv));
  }
  if (!aligned(q_lens, 8) || !aligned(k_lens, 8)) return fail(LACT_ERR_INVALID_ARG, "lengths are not 8-byte aligned");
  TRY(check_apart({p->q_len ? dq : nullptr, p->k_len ? dk : nullptr, p->k_len ? dv : nullptr}, {q, k, v, o, dO, lse}));
  const AttnWs w = attn_back_ws(*p);
  TRY(check_ws(ws, ws_bytes, w.total));
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.o = static_cast<const char*>(o);
  a.dO = static_cast<const char*>(dO);
  a.dq = static_cast<char*>(dq);
  a.dk = static_cast<char*>(dk);
  a.dv = static_cast<char*>(dv);
  a.q_lens = q_lens;
  a.k_lens = k_lens;
  a.lse = const_cast<float*>(lse);
  a.stats = static_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + w.part);
  const int ksq = parts_q(*p), ksk = parts_k(*p);
  AttnArgs kv = a;
  sink_plan(*p, 128 / ksk, kv);
  row_tiles(*p, 128 / ksq, a);
  const int64_t heads = (int64_t)p->batch * p->kv_heads, gq = (int64_t)p->batch * (p->heads / a.hg) * a.tiles,
                gk = heads * (kv.tiles + (int64_t)kv.sink_tiles * (kv.splits - 1)),
                gs = kv.splits > 1 ? heads * kv.sink_tiles * 2 * (128 / ksk) : 0;
  TRY(check_grid(std::max(gq, gk), 256));
  TRY(check_grid(gs, 128));
  TRY(check_device_again());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return by_tile(*p, [&](auto t, auto dp) -> lact_status {
    using T = decltype(t);
    constexpr int DP = decltype(dp)::value;
    if (gq > 0) {
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      by_parts(t, dp, ksq, [&](auto n) {
        LACT_LAUNCH((attn_dq_kernel<T, DP, decltype(n)::value>), dim3((unsigned)gq), dim3(256), s, a);
      });
    }
    if (gk > 0) {
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      by_parts(t, dp, ksk, [&](auto n) {
        LACT_LAUNCH((attn_dkv_kernel<T, DP, decltype(n)::value>), dim3((unsigned)gk), dim3(256), s, kv);
      });
    }
    if (gs > 0) {
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      if (ksk == 2) LACT_LAUNCH((attn_sink_sum_kernel<T, 64>), dim3((unsigned)gs), dim3(128), s, kv);
      else LACT_LAUNCH((attn_sink_sum_kernel<T, 128>), dim3((unsigned)gs), dim3(128), s, kv);
    }
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

// ------------------------------------------------------------------ rotary positions
lact_status lact_rotary(const lact_rotary_problem* p, const void* q, const lact_strides* sq, const void* k,
                        const lact_strides* sk, const double* freqs, const int64_t* positions, void* q_out,
                        const lact_strides* sqo, void* k_out, const lact_strides* sko, void* stream) {
  g_err.clear();
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0 || p->heads < 1 || p->kv_heads < 0 || p->heads > 65536 || p->kv_heads > 65536)
    return fail(LACT_ERR_INVALID_ARG, "batch = %d, heads = %d, kv_heads = %d", p->batch, p->heads, p->kv_heads);
  if (p->d < 1 || p->d > 8192) return fail(LACT_ERR_UNSUPPORTED, "d = %d: need 1..8192", p->d);
  if (p->pairs < 0 || 2 * (int64_t)p->pairs > p->d || p->pairs > ROT_TABLE)
    return fail(LACT_ERR_INVALID_ARG, "pairs = %d: need 0 <= 2 pairs <= d, pairs <= %d", p->pairs, ROT_TABLE);
  TRY(check_dtype(p->io_dtype));
  if (p->flags & ~(LACT_ROTARY_INTERLEAVED | LACT_ROTARY_INVERSE))
    return fail(LACT_ERR_INVALID_ARG, "unknown flags 0x%x", p->flags);
  if (!std::isfinite(p->mscale)) return fail(LACT_ERR_INVALID_ARG, "mscale is not finite");
  if (p->tokens < 0 || p->tokens >= MOST_TOKENS)
    return fail(LACT_ERR_INVALID_ARG, "tokens = %lld", (long long)p->tokens);
  if (p->batch == 0 || p->tokens == 0) return LACT_OK;
  const int64_t es = size_of(p->io_dtype);
  RotaryArgs a;
  memset(&a, 0, sizeof(a));
  // widest vectors that every address and the layout allow
  int64_t bits = 0;
  auto tensor = [&](int i, const char* name, const void* in, const lact_strides* si, void* out,
                    const lact_strides* so, int heads) -> lact_status {
    AttnStride bi, bo;
    TRY(check_tensor(name, in, si, p->batch, heads, p->tokens, p->d, es, es, false, &bi));
    TRY(check_tensor(i ? "k_out" : "q_out", out, so, p->batch, heads, p->tokens, p->d, es, es, true, &bo));
    if (in == out && (bi.b != bo.b || bi.h != bo.h || bi.l != bo.l))
      return fail(LACT_ERR_INVALID_ARG, "%s in place with other strides", name);
    a.t[i] = {static_cast<const char*>(in), static_cast<char*>(out), bi.b, bi.h, bi.l, bo.b, bo.h, bo.l, heads};
    bits |= (int64_t)(uintptr_t)in | (int64_t)(uintptr_t)out | bi.b | bi.h | bi.l | bo.b | bo.h | bo.l;
    return LACT_OK;
  };
  TRY(tensor(0, "q", q, sq, q_out, sqo, p->heads));
  if (p->kv_heads > 0) {
    TRY(tensor(1, "k", k, sk, k_out, sko, p->kv_heads));
    // each may be turned in place, not into the other
    TRY(check_apart({q_out, k_out}, {}));
    TRY(check_apart({q_out}, {k}));
    TRY(check_apart({k_out}, {q}));
  }
  if (p->pairs > 0) NEED(freqs, 8);
  if (!aligned(positions, 8)) return fail(LACT_ERR_INVALID_ARG, "positions is not 8-byte aligned");
  const bool il = p->flags & LACT_ROTARY_INTERLEAVED;
  auto fits = [&](int64_t ve) {
    const int64_t part = il ? 2 * p->pairs : p->pairs;
    return bits % (ve * es) == 0 && part % ve == 0 && (p->d - 2 * p->pairs) % ve == 0;
  };
  a.freqs = freqs;
  a.positions = positions;
  a.start = p->start;
  a.B = p->batch;
  a.L = (int32_t)p->tokens;
  a.d = p->d;
  a.pairs = p->pairs;
  a.mscale = p->mscale;
  a.inverse = (p->flags & LACT_ROTARY_INVERSE) != 0;
  // a workgroup's tokens: a table of at most 2048 angles, and at most 8
  // tokens; fewer, and the heads split, where that fills the chip no better
  const int heads = p->heads + p->kv_heads;
  a.tok = (int32_t)std::min<int64_t>(std::min<int64_t>(8, std::max(1, ROT_TABLE / std::max(1, p->pairs))), p->tokens);
  while (a.tok > 1 && p->batch * ceil_div(p->tokens, a.tok) < 8 * NCU) a.tok = (a.tok + 1) / 2;
  int64_t groups = p->batch * ceil_div(p->tokens, a.tok);
  a.head_groups = (int32_t)std::max<int64_t>(1, std::min<int64_t>(heads, 2 * NCU / std::max<int64_t>(1, groups)));
  // and a workgroup's items stay far below 2^31
  a.head_groups = (int32_t)std::max<int64_t>(a.head_groups, ceil_div((int64_t)a.tok * heads * p->d, 1 << 24));
  a.group = (int32_t)ceil_div(heads, a.head_groups);
  a.head_groups = (int32_t)ceil_div(heads, a.group);
  TRY(check_grid(groups * a.head_groups, 256));
  TRY(check_device_again());
  const unsigned grid = (unsigned)(groups * a.head_groups);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  KernelTimer kt(LACT_K_ROTARY, s);
  a.by_pairs = FastDiv((uint32_t)std::max(1, p->pairs));
  a.heads_inner = a.t[0].ih < a.t[0].il;
  a.by_inner = FastDiv((uint32_t)(a.heads_inner ? a.group : a.tok));
  auto launch = [&](auto t, auto ve) -> lact_status {
    using T = decltype(t);
    constexpr int VE = decltype(ve)::value;
    a.by_per = FastDiv((uint32_t)(p->pairs / (il ? (VE > 1 ? VE / 2 : 1) : VE) + (p->d - 2 * p->pairs) / VE));
    if (il) LACT_LAUNCH((rotary_kernel<T, VE, true>), dim3(grid), dim3(256), s, a);
    else LACT_LAUNCH((rotary_kernel<T, VE, false>), dim3(grid), dim3(256), s, a);
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  };
  if (p->io_dtype == LACT_DTYPE_F32)
    return fits(4) ? launch(float{}, IC<4>{}) : fits(2) ? launch(float{}, IC<2>{}) : launch(float{}, IC<1>{});
  return fits(8) ? launch(bf16_t{}, IC<8>{}) : fits(2) ? launch(bf16_t{}, IC<2>{}) : launch(bf16_t{}, IC<1>{});
}

lact_status lact_rotary_frequencies(int32_t pairs, double base, int32_t scaling, double factor, int64_t context,
                                    double slow, double fast, double* freqs, float* mscale) {
  g_err.clear();
  if (pairs < 0 || pairs > ROT_TABLE) return fail(LACT_ERR_INVALID_ARG, "pairs = %d: need 0..%d", pairs, ROT_TABLE);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(LACT_ERR_INVALID_ARG, "base = %g: need a finite value > 1", base);
  if (scaling < LACT_ROTARY_PLAIN || scaling > LACT_ROTARY_YARN)
    return fail(LACT_ERR_INVALID_ARG, "scaling = %d", scaling);
  if (scaling != LACT_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(LACT_ERR_INVALID_ARG, "factor = %g: need a finite value >= 1", factor);
  if (scaling == LACT_ROTARY_YARN && (context < 1 || !(slow >= 0.0) || !(fast > slow) || !std::isfinite(fast)))
    return fail(LACT_ERR_INVALID_ARG, "context = %lld, slow = %g, fast = %g", (long long)context, slow, fast);
  if (pairs > 0) NEED(freqs, 8);
  const double pi2 = 6.283185307179586477;
  if (scaling == LACT_ROTARY_NTK && pairs > 1) base *= std::pow(factor, (double)pairs / (pairs - 1));
  for (int i = 0; i < pairs; ++i) {
    double f = std::pow(base, -(double)i / pairs);
    if (scaling == LACT_ROTARY_LINEAR) f /= factor;
    if (scaling == LACT_ROTARY_YARN) {
      const double turns = (double)context * f / pi2;
      const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    freqs[i] = f;
  }
  if (mscale) *mscale = scaling == LACT_ROTARY_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return LACT_OK;
}

}  // extern "C"

// ------------------------------------------------------------------ add and norm
namespace {

lact_status validate(const lact_norm_problem* p) {
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  if (p->rows < 0) return fail(LACT_ERR_INVALID_ARG, "rows = %lld < 0", (long long)p->rows);
  if (p->cols < 1 || p->cols > 32768) return fail(LACT_ERR_UNSUPPORTED, "cols = %d: need 1..32768", p->cols);
  TRY(check_dtype(p->io_dtype));
  if (!(p->eps >= 0.f) || !std::isfinite(p->eps)) return fail(LACT_ERR_INVALID_ARG, "eps = %g", (double)p->eps);
  return LACT_OK;
}

// A matrix of rows: pointer and row stride in bytes.  `vec` stays set while
// every row starts at a multiple of `width` bytes, a vector's.
lact_status check_rows(const lact_norm_problem& p, const char* name, const void* ptr, int64_t ld, int64_t es,
                       int64_t width, bool output, int64_t* bytes, bool* vec) {
  if (!ptr) return fail(LACT_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(ptr, es)) return fail(LACT_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)es);
  if (p.rows <= 1) ld = 0;  // not looked at
  else if ((ld < p.cols && (output || ld != 0)) || ld > (INT64_C(1) << 60) / p.rows)
    return fail(LACT_ERR_INVALID_ARG, "%s has a row stride of %lld for %d columns", name, (long long)ld, p.cols);
  *bytes = ld * es;
  *vec = *vec && aligned(ptr, width) && *bytes % width == 0;
  return LACT_OK;
}

// in place means the same rows
lact_status check_in_place(const char* name, const void* out, int64_t ldo, const void* in, int64_t ldi) {
  if (out && out == in && ldo != ldi) return fail(LACT_ERR_INVALID_ARG, "%s in place with another row stride", name);
  return LACT_OK;
}

// Threads and 16-byte vectors a thread for a row of `cols` values.  A wave a
// row has no barrier, and four rows share a workgroup, up to two vectors a
// thread (32768 rows of 768 bf16, backward: 40 us, with 256 threads 50; of
// 2048, four vectors: 109 and 101; with 8-bit output 103 and 86).
struct NormPlan {
  int gs, nv;
};
NormPlan norm_plan(const lact_norm_problem& p) {
  const int64_t n = ceil_div(p.cols, 16 / size_of(p.io_dtype));
  const int gs = n <= 128 ? 64 : n <= 1024 ? 256 : 1024;
  const int64_t nv = ceil_div(n, gs);
  return {gs, nv <= 1 && gs < 1024 ? 1 : nv <= 2 ? 2 : nv <= 3 ? 3 : nv <= 4 ? 4 : 8};
}
// Workgroups of the backward, 512 threads or one row's 1024 each: as many as
// run at once, so that few partial sums of dw remain.  One workgroup's rows
// need no second launch to add them up, which takes as long as three more
// rounds of it.
int64_t norm_back_grid(const lact_norm_problem& p, const NormPlan& c) {
  const int64_t at_once = c.gs < 512 ? 512 / c.gs : 1;
  if (p.rows <= 4 * at_once) return std::min<int64_t>(p.rows, 1);
  return std::min<int64_t>(ceil_div(p.rows, c.gs < 512 ? 512 / c.gs : 1), (c.gs == 1024 ? 1 : 2) * NCU);
}

// calls fn with the element type, vectors and threads of the plan, and whether rows are vector-aligned
template <class F>
lact_status by_plan(const lact_norm_problem& p, const NormPlan& c, bool vec, F&& fn) {
  auto with = [&](auto t, auto v) -> lact_status {
    if (c.gs == 64) return c.nv == 1 ? fn(t, IC<1>{}, IC<64>{}, v) : fn(t, IC<2>{}, IC<64>{}, v);
    if (c.gs == 256) return c.nv == 1 ? fn(t, IC<1>{}, IC<256>{}, v) : c.nv == 2 ? fn(t, IC<2>{}, IC<256>{}, v) : c.nv == 3 ? fn(t, IC<3>{}, IC<256>{}, v) : fn(t, IC<4>{}, IC<256>{}, v);
    if (c.nv == 2) return fn(t, IC<2>{}, IC<1024>{}, v);
    if (c.nv == 3) return fn(t, IC<3>{}, IC<1024>{}, v);
    if (c.nv == 4) return fn(t, IC<4>{}, IC<1024>{}, v);
    if constexpr (sizeof(t) == 4) return fn(t, IC<8>{}, IC<1024>{}, v);
    return fail(LACT_ERR_UNSUPPORTED, "internal: %d columns", p.cols);
  };
  if (p.io_dtype == LACT_DTYPE_F32) return vec ? with(float{}, std::true_type{}) : with(float{}, std::false_type{});
  return vec ? with(bf16_t{}, std::true_type{}) : with(bf16_t{}, std::false_type{});
}

}  // namespace

extern "C" {

lact_status lact_add_rmsnorm_forward(const lact_norm_problem* p, const void* x, int64_t ldx, const void* residual,
                                     int64_t ldr, const float* weight, void* h, int64_t ldh, void* y, int64_t ldy,
                                     uint8_t* y8, int64_t ldy8, float* scales, void* stream) {
  g_err.clear();
  TRY(validate(p));
  if (p->rows == 0) return LACT_OK;
  const int64_t es = size_of(p->io_dtype), ve = 16 / es;
  NormArgs a;
  memset(&a, 0, sizeof(a));
  bool vec = p->cols % ve == 0;
  TRY(check_rows(*p, "x", x, ldx, es, 16, false, &a.ldx, &vec));
  if (residual) TRY(check_rows(*p, "residual", residual, ldr, es, 16, false, &a.ldr, &vec));
  NEED(weight, 4);
  if (!y && !y8) return fail(LACT_ERR_INVALID_ARG, "neither y nor y8 is given");
  if (h) TRY(check_rows(*p, "h", h, ldh, es, 16, true, &a.ldh, &vec));
  if (y) TRY(check_rows(*p, "y", y, ldy, es, 16, true, &a.ldy, &vec));
  if (y8) {
    TRY(check_rows(*p, "y8", y8, ldy8, 1, ve, true, &a.ldy8, &vec));
    NEED(scales, 4);
  }
  if (p->rows > 1) {
    TRY(check_in_place("h", h, ldh, x, ldx));
    TRY(check_in_place("h", h, ldh, residual, ldr));
    TRY(check_in_place("y", y, ldy, x, ldx));
    TRY(check_in_place("y", y, ldy, residual, ldr));
  }
  if (y && y == h) return fail(LACT_ERR_INVALID_ARG, "y is h");
  TRY(check_apart({h, y, y8, scales}, {weight}));
  TRY(check_apart({y8, scales}, {x, residual}));
  TRY(check_device_again());
  a.x = static_cast<const char*>(x);
  a.res = static_cast<const char*>(residual);
  a.w = weight;
  a.h = static_cast<char*>(h);
  a.y = static_cast<char*>(y);
  a.y8 = y8;
  a.scales = scales;
  a.rows = p->rows;
  a.cols = p->cols;
  a.eps = p->eps;
  const NormPlan c = norm_plan(*p);
  const int64_t per = c.gs == 64 ? 4 : 1;
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(p->rows, per), (c.gs == 1024 ? 2 : 8) * NCU);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  KernelTimer kt(LACT_K_NORM, s);
  return by_plan(*p, c, vec, [&](auto t, auto nv, auto gs, auto v) -> lact_status {
    using T = decltype(t);
    constexpr int NV = decltype(nv)::value, GS = decltype(gs)::value, NT = GS < 256 ? 256 : GS;
    constexpr bool VEC = decltype(v)::value;
    if (y8) LACT_LAUNCH((norm_kernel<T, NV, GS, VEC, true>), dim3(grid), dim3(NT), s, a);
    else LACT_LAUNCH((norm_kernel<T, NV, GS, VEC, false>), dim3(grid), dim3(NT), s, a);
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

size_t lact_add_rmsnorm_backward_workspace_size(const lact_norm_problem* p) {
  g_err.clear();
  if (validate(p)) return 0;
  const int64_t grid = norm_back_grid(*p, norm_plan(*p));
  return grid > 1 ? align256((size_t)grid * p->cols * 4) : 0;
}

lact_status lact_add_rmsnorm_backward(const lact_norm_problem* p, const void* h, int64_t ldh, const float* weight,
                                      const void* dy, int64_t ldy, const void* dh, int64_t lddh, void* dx,
                                      int64_t lddx, float* dw, void* ws, size_t ws_bytes, void* stream) {
  g_err.clear();
  TRY(validate(p));
  if (p->rows == 0 && !dw) return LACT_OK;
  const int64_t es = size_of(p->io_dtype);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  bool vec = p->cols % (16 / es) == 0;
  const NormPlan c = norm_plan(*p);
  const int64_t grid = norm_back_grid(*p, c);
  if (p->rows > 0) {
    TRY(check_rows(*p, "h", h, ldh, es, 16, false, &a.ldx, &vec));
    TRY(check_rows(*p, "dy", dy, ldy, es, 16, false, &a.ldg, &vec));
    if (dh) TRY(check_rows(*p, "dh", dh, lddh, es, 16, false, &a.lddh, &vec));
    TRY(check_rows(*p, "dx", dx, lddx, es, 16, true, &a.lddx, &vec));
    NEED(weight, 4);
    if (p->rows > 1) {
      TRY(check_in_place("dx", dx, lddx, h, ldh));
      TRY(check_in_place("dx", dx, lddx, dy, ldy));
      TRY(check_in_place("dx", dx, lddx, dh, lddh));
    }
  }
  if (dw) {
    NEED(dw, 4);
    if (grid > 1) TRY(check_ws(ws, ws_bytes, align256((size_t)grid * p->cols * 4)));
  }
  if (p->rows > 0) {
    TRY(check_apart({dx, dw}, {weight}));
    TRY(check_apart({dw}, {h, dy, dh}));
  }
  TRY(check_device_again());
  a.x = static_cast<const char*>(h);
  a.w = weight;
  a.dy = static_cast<const char*>(dy);
  a.dh = static_cast<const char*>(dh);
  a.dx = static_cast<char*>(dx);
  a.part = !dw ? nullptr : grid == 1 ? dw : static_cast<float*>(ws);
  a.rows = p->rows;
  a.cols = p->cols;
  a.eps = p->eps;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (grid > 0) {
    KernelTimer kt(LACT_K_NORM, s);
    TRY(by_plan(*p, c, vec, [&](auto t, auto nv, auto gs, auto v) -> lact_status {
      constexpr int NV = decltype(nv)::value, GS = decltype(gs)::value;
      constexpr bool VEC = decltype(v)::value;
      LACT_LAUNCH((norm_back_kernel<decltype(t), NV, GS, VEC>), dim3((unsigned)grid), dim3(GS < 512 ? 512 : GS), s, a);
      HIP_TRY(hipGetLastError());
      return LACT_OK;
    }));
  }
  if (dw && grid != 1) {
    KernelTimer kt(LACT_K_NORM, s);
    LACT_LAUNCH(norm_dw_kernel, dim3((unsigned)ceil_div(p->cols, 32)), dim3(1024), s, a.part, dw, (int)grid, p->cols);
    HIP_TRY(hipGetLastError());
  }
  return LACT_OK;
}

}  // extern "C"
