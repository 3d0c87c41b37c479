// liblact: host side of the operators on batches of sequences of different
// lengths (packed and paged attention, page slots, page writes).  Part of the
// library's one translation unit, after lact_block.hpp.
#pragma once
#include "lact_pages.hpp"

namespace {

constexpr int32_t MOST_BATCH = 1 << 24;
constexpr int32_t MOST_PAGES = 1 << 28;         // of a pool, by its places
constexpr int64_t MOST_ROW = INT64_C(1) << 27;  // bytes from a token's row to the next in a page

lact_status check_page(int32_t page, int32_t pages, int32_t width) {
  if (page < 8 || page > 65536 || page % 8)
    return fail(LACT_ERR_UNSUPPORTED, "page = %d: need a multiple of 8 in [8, 65536]", page);
  if (pages < 0 || (int64_t)pages * page > INT32_MAX) return fail(LACT_ERR_INVALID_ARG, "pages = %d of %d", pages, page);
  if (width < 0 || (int64_t)width * page >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "width = %d pages of %d", width, page);
  return LACT_OK;
}

// What packed and paged problems share, as a window attention problem of `longest` rows and `k_len` keys
template <class P>
lact_status as_window(const P* p, int64_t k_len, lact_attention* w) {
  *w = {p->batch, p->heads, p->kv_heads, p->d, p->io_dtype, p->scale, p->longest, k_len, p->window, p->sinks};
  if (p->tokens < 0 || p->tokens >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "tokens = %lld", (long long)p->tokens);
  if (p->longest < 0 || p->longest > p->tokens) return fail(LACT_ERR_INVALID_ARG, "longest = %lld", (long long)p->longest);
  if (p->batch > MOST_BATCH) return fail(LACT_ERR_UNSUPPORTED, "batch = %d: more than %d", p->batch, MOST_BATCH);
  if (p->flags & ~LACT_CLEAR_REST) return fail(LACT_ERR_INVALID_ARG, "unknown flags 0x%x", p->flags);
  return validate(w);
}
lact_status validate(const lact_packed* p, lact_attention* w) {
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  return as_window(p, p->longest, w);
}
lact_status validate(const lact_paged* p, lact_attention* w) {
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  TRY(check_page(p->page, p->pages, p->width));
  if (p->k_len < 0 || p->k_len > (int64_t)p->width * p->page)
    return fail(LACT_ERR_INVALID_ARG, "k_len = %lld for %d pages of %d", (long long)p->k_len, p->width, p->page);
  return as_window(p, p->pages > 0 ? p->k_len : 0, w);
}

// Row (or key) tiles of all sequences, `rows` a tile: those of `longest` rows
// for each, or the slots of find_tile, whichever are fewer.
template <class A>
int64_t count_tiles(const lact_attention& w, int64_t tokens, int64_t rows, A& a) {
  a.tiles = (int32_t)ceil_div(w.q_len, rows);
  const int64_t each = (int64_t)w.batch * a.tiles, found = tokens / rows + w.batch;
  a.slots = each <= found ? 0 : (int32_t)found;
  return std::min(each, found);
}

void fill_args(PackedArgs& a, const lact_attention& w, int64_t tokens, const int64_t* offsets) {
  static_cast<AttnArgs&>(a) = attn_args(w);
  a.Lq = (int32_t)tokens;
  a.offsets = offsets;
  a.most = (int32_t)w.q_len;
}
// Workgroups that clear rows of no sequence beside those that compute: the
// host does not know whether there are such rows, and most calls have none.
int rest_groups(int64_t bytes) { return (int)std::min<int64_t>(64, ceil_div(bytes, 1 << 16)); }

lact_status check_offsets(const void* offsets) {
  NEED(offsets, 8);
  return LACT_OK;
}

// ------------------------------------------------------------------ paged attention
// Which kernels take a batch.  The host knows the longest sequence's rows, not
// whether others have as many: sequences of few rows (one 32-row tile of a key
// head, `few`) go to the streams of tiles, longer ones to the forward's kernel,
// in two launches where both may come.  (Sequences of a few 32-row tiles read
// their keys once for each in the streams: 64 and 128 rows of 32 (8) heads over
// 16384 keys 90 and 149 us there.)
struct PagedPlan {
  int64_t few = 0;         // rows of a sequence up to which the streams have it
  int64_t items = 0;       // of the streams, at most
  int64_t few_grid = 0, big_grid = 0;  // workgroups, 0: not launched
  int waves = 0, rows = 0, unit = 1, big_splits = 1, chunk = 1;
  size_t upto = 0, joins = 0, few_part = 0, few_ml = 0, big_part = 0, big_ml = 0, total = 0;  // the workspace
};

// Key splits of the forward's row tiles: `groups` workgroups (as far as the
// host can tell) of `rows` rows a head.
//
// One sequence: all tiles have about as many keys.  A workgroup alone on its
// compute unit takes `alone` us a tile, two take `both`, a join about 6 us, and
// the parts pass memory twice.  Over 16384 keys, 32 (8) heads of 128, us with
// 1, 2, 3, 4, 5, 8 splits: 256 rows (64 workgroups) 319, 177, 127, 102, 107, 87;
// 512 rows 321, 188, 175, 153, 183, 162; 1200 rows 414, 408, 357, 359, 357, 368;
// 2048 rows, one round of two a unit, 493, 522, 527, 533, 543, 584; the model
// chooses 8, 4, 5 and 1.
//
// Several, whose keys only the device knows, while one round holds them: a
// quarter of the most keys a split (less where there are few workgroups), so
// that long ones are split and short ones are not.  40 sequences, 4 of them of
// 512 rows, of up to 12000 keys: with splits of 48 tiles 519 us, of 16 540, none
// 544; one of 512 rows among 64 of one: 352, none 400; 4 of 100: 189, none 493.
// Beyond one round (8 of 1024 rows among 20) none is best: 946, and 1023 with a
// quarter.  The most keys are the caller's bound, and without one the table's
// width: these figures are of tables two pages wider than the longest sequence.
// With tables of 2, 4, 16 times the width and no bound less is split, in the end
// nothing: 40 sequences 547, 540, 538 us (527 with a bound), one chunk among 64
// 546, 636, 618 (508), 4 of 100 360, 490, 493 (196 - 204).
void split_keys(const lact_attention& w, int64_t groups, int64_t rows, int& splits, int& chunk) {
  const bool fp32 = w.io_dtype == LACT_DTYPE_F32, wide = w.d > 64;
  const int64_t room = (fp32 && wide ? 1 : 2) * NCU;
  const int64_t keys = limited(w) ? std::min(w.k_len, w.window + w.sinks + rows) : w.k_len;
  const int64_t tiles = ceil_div(keys, fp32 && wide ? 32 : 64);
  splits = chunk = 1;
  if (w.batch == 1) {
    const double alone = fp32 ? 3.7 : wide ? 1.25 : 0.7, both = fp32 && wide ? alone : fp32 ? 7.4 : wide ? 1.93 : 1.1;
    const double part = (double)groups * 128 * (double)(w.d + 2) * 8 / 4e6;  // us of one split's parts
    double best = 1e30;
    for (int64_t s = 1; s <= 64 && (s == 1 || tiles / s >= 4); ++s) {
      const int64_t full = groups * s / room, left = groups * s % room;
      const double round = (double)full * both + (left == 0 ? 0.0 : left <= NCU ? alone : both);
      const double cost = round * (double)ceil_div(tiles, s) + (s > 1 ? 6.0 + part * (double)s : 0.0);
      if (cost < best) best = cost, splits = (int)s;
    }
    if (splits > 1) chunk = 4;  // of a tile of early rows, which has fewer keys
  } else if (groups <= room) {
    const int64_t s = std::max<int64_t>(4, std::min<int64_t>(32, room / std::max<int64_t>(1, groups)));
    chunk = (int)std::max<int64_t>(8, ceil_div(tiles, s));
    splits = (int)std::max<int64_t>(1, (tiles + chunk / 2) / chunk);
  }
}

// Fewest units of a wave's run: with 1, 2, 4, 8, 16, us with the join, one request
// of 16 heads of 64, window 2048, 15.1, 15.4, 17.2, 21.3, 29.3; 4 of 300 keys, 32 (8)
// heads of 128, 15.9, 20.7, 23.8, 34.4, 51.8; 8 of 4000 keys 34.8, 34.4, 34.3, 36.9, 49.4;
// 400 of 1000, 96 of 8192 and one of 32768 keys the same up to 8 (246, 376, 41).  So
// few units are right; one would do as well as two, and better where all keys
// are few.
constexpr int STREAM_SHARE = 2;

PagedPlan paged_plan(const lact_paged& p, const lact_attention& w) {
  PagedPlan x;
  if (w.batch == 0 || p.tokens == 0 || w.q_len == 0) return x;
  const int64_t G = w.heads / w.kv_heads, small = std::max<int64_t>(1, 32 / G);
  lact_attention f = w;
  if (w.q_len <= small) x.few = w.q_len;
  else if (w.batch > 1) x.few = small;
  f.q_len = x.few;
  int64_t room = 0;  // workgroups of the streams that run at once
  (void)by_tile(w, [&](auto t, auto dp) {
    room = (int64_t)stream_groups<decltype(t), decltype(dp)::value>() * NCU;
    return LACT_OK;
  });
  const size_t rows = (size_t)p.tokens * w.heads;
  auto place = [&](size_t bytes) {
    const size_t at = x.total;
    x.total += align256(bytes);
    return at;
  };
  if (x.few > 0) {
    // no more workgroups than run at once, nor than have a share of the tiles that there can be
    const int64_t items = x.items = std::min((int64_t)w.batch * ceil_div(G * x.few, 32), p.tokens * ceil_div(G, 32)) * w.kv_heads;
    const int64_t tiles = ceil_div(few_keys(f), 32) + 2;  // the sinks' and the window's may be cut anew
    x.unit = stream_unit(items, tiles);
    x.few_grid = std::min(room, ceil_div(items, STREAM_GROUP * STREAM_SHARE) * tiles);
    x.waves = (int)(x.few_grid * STREAM_GROUP);
    x.rows = (int)std::min<int64_t>(32, G * x.few);
    if (w.batch > STREAM_SCAN) x.upto = place((size_t)(w.batch + 1) * 4);
    x.joins = place((size_t)x.waves * sizeof(StreamJoin));
    x.few_part = place((size_t)x.waves * 2 * x.rows * w.d * 4);
    x.few_ml = place((size_t)x.waves * 2 * x.rows * 2 * 4);
  }
  if (x.few < w.q_len) {
    PackedArgs a;
    memset(&a, 0, sizeof(a));
    row_tiles(w, 128, a);
    const int64_t tile = 128 / a.hg, groups = count_tiles(w, p.tokens, tile, a), heads = w.heads / a.hg;
    split_keys(w, std::min(groups, ceil_div(p.tokens, tile)) * heads, tile, x.big_splits, x.chunk);
    x.big_grid = groups * heads * x.big_splits;
  }
  if (x.big_splits > 1) {
    x.big_part = place(rows * x.big_splits * w.d * 4);
    x.big_ml = place(rows * x.big_splits * 2 * 4);
  }
  return x;
}

}  // namespace

extern "C" {

size_t lact_paged_attention_workspace_size(const lact_paged* p) {
  g_err.clear();
  lact_attention w;
  if (validate(p, &w)) return 0;
  return paged_plan(*p, w).total;
}

lact_status lact_paged_attention(const lact_paged* p, const void* q, const lact_strides* sq, const void* k_pages,
                                 const lact_strides* sk, const void* v_pages, const lact_strides* sv,
                                 const int64_t* offsets, const int64_t* k_lens, const int32_t* table, void* o,
                                 const lact_strides* so, float* lse, void* ws, size_t ws_bytes, void* stream) {
  g_err.clear();
  lact_attention w;
  TRY(validate(p, &w));
  if (p->tokens == 0) return LACT_OK;
  PagedArgs a;
  memset(&a, 0, sizeof(a));
  fill_args(a, w, p->tokens, offsets);
  const int64_t es = size_of(w.io_dtype);
  TRY(check_tensor("q", q, sq, 1, w.heads, p->tokens, w.d, es, 16, false, &a.sq));
  TRY(check_tensor("o", o, so, 1, w.heads, p->tokens, w.d, es, 16, true, &a.so));
  if (w.k_len > 0 && w.batch > 0) {
    TRY(check_tensor("k_pages", k_pages, sk, p->pages, w.kv_heads, p->page, w.d, es, 16, false, &a.sk));
    TRY(check_tensor("v_pages", v_pages, sv, p->pages, w.kv_heads, p->page, w.d, es, 16, false, &a.sv));
    if (a.sk.l > MOST_ROW || a.sv.l > MOST_ROW)
      return fail(LACT_ERR_UNSUPPORTED, "a token's stride in a page is more than 2^27 bytes");
    NEED(table, 4);
  }
  TRY(check_offsets(offsets));
  if (w.batch > 0) NEED(k_lens, 8);
  if (!aligned(lse, 4)) return fail(LACT_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  TRY(check_apart({o, lse}, {q, k_pages, v_pages, offsets, k_lens, table}));
  const PagedPlan x = paged_plan(*p, w);
  if (x.items > STREAM_MOST)
    return fail(LACT_ERR_UNSUPPORTED, "%lld sequences and key heads: more than a launch takes", (long long)x.items);
  TRY(check_ws(ws, ws_bytes, x.total));
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k_pages);
  a.v = static_cast<const char*>(v_pages);
  a.out = static_cast<char*>(o);
  a.lse = lse;
  a.k_lens = k_lens;
  a.table = table;
  a.width = p->width;
  a.pages = p->pages;
  a.by_page = FastDiv((uint32_t)p->page);
  a.few = (int32_t)x.few;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int64_t rows = p->tokens * w.heads, clear = p->flags & LACT_CLEAR_REST ? rest_groups(rows * w.d * es) : 0;
  // what is cleared is cleared beside the kernel of the longer sequences, if there is one
  const int64_t few_clear = x.big_grid > 0 ? 0 : clear, big_grid = x.big_grid + (clear - few_clear);
  TRY(check_grid(x.few_grid + few_clear, 64 * STREAM_GROUP));
  TRY(check_grid(big_grid, 256));
  const int64_t joins = ceil_div(p->tokens * ceil_div(w.heads, JOIN_HEADS), 4);
  if (x.big_splits > 1) TRY(check_grid(joins, 256));
  TRY(check_device_again());
  char* const base = static_cast<char*>(ws);
  return by_tile(w, [&](auto t, auto dp) -> lact_status {
    using T = decltype(t);
    constexpr int DP = decltype(dp)::value;
    a.rest = (int32_t)clear;
    PagedArgs f = a;
    if (x.few_grid + few_clear > 0) {
      f.main = (int32_t)x.few_grid;
      f.waves = x.waves;
      f.share = STREAM_SHARE;
      f.unit = x.unit;
      f.rows = x.rows;
      f.upto = w.batch > STREAM_SCAN ? reinterpret_cast<int32_t*>(base + x.upto) : nullptr;
      f.joins = reinterpret_cast<StreamJoin*>(base + x.joins);
      f.part = reinterpret_cast<float*>(base + x.few_part);
      f.part_ml = reinterpret_cast<float*>(base + x.few_ml);
      if (f.upto && x.few_grid > 0) {
        KernelTimer kt(LACT_K_ATTN, s);
        LACT_LAUNCH(stream_plan_kernel, dim3(1), dim3(1024), s, f);
      }
      KernelTimer kt(LACT_K_ATTN, s);
      LACT_LAUNCH((stream_kernel<T, DP>), dim3((unsigned)(x.few_grid + few_clear)), dim3(64 * STREAM_GROUP), s, f);
    }
    if (big_grid > 0) {
      row_tiles(w, 128, a);
      (void)count_tiles(w, p->tokens, 128 / a.hg, a);
      a.splits = x.big_splits;
      a.chunk = x.chunk;
      a.main = (int32_t)x.big_grid;
      a.part = reinterpret_cast<float*>(base + x.big_part);
      a.part_ml = reinterpret_cast<float*>(base + x.big_ml);
      KernelTimer kt(LACT_K_ATTN, s);
      LACT_LAUNCH((attn_fwd_kernel<T, DP, 1, PagedArgs>), dim3((unsigned)big_grid), dim3(256), s, a);
    }
    if (x.waves > 1) {
      KernelTimer kt(LACT_K_ATTN, s);
      LACT_LAUNCH((stream_join_kernel<T>), dim3((unsigned)(x.waves - 1), (unsigned)std::min(x.rows, JOIN_ROWS)), dim3(256), s, f);
    }
    if (x.big_splits > 1) {
      KernelTimer kt(LACT_K_ATTN, s);
      LACT_LAUNCH((split_join_kernel<T, DP>), dim3((unsigned)joins), dim3(256), s, a);
    }
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

// ------------------------------------------------------------------ packed attention
lact_status lact_packed_attention_forward(const lact_packed* p, const void* q, const lact_strides* sq, const void* k,
                                          const lact_strides* sk, const void* v, const lact_strides* sv,
                                          const int64_t* offsets, void* o, const lact_strides* so, float* lse,
                                          void* stream) {
  g_err.clear();
  lact_attention w;
  TRY(validate(p, &w));
  if (p->tokens == 0) return LACT_OK;
  PackedArgs a;
  memset(&a, 0, sizeof(a));
  fill_args(a, w, p->tokens, offsets);
  const int64_t es = size_of(w.io_dtype);
  TRY(check_tensor("q", q, sq, 1, w.heads, p->tokens, w.d, es, 16, false, &a.sq));
  TRY(check_tensor("k", k, sk, 1, w.kv_heads, p->tokens, w.d, es, 16, false, &a.sk));
  TRY(check_tensor("v", v, sv, 1, w.kv_heads, p->tokens, w.d, es, 16, false, &a.sv));
  TRY(check_tensor("o", o, so, 1, w.heads, p->tokens, w.d, es, 16, true, &a.so));
  TRY(check_offsets(offsets));
  if (!aligned(lse, 4)) return fail(LACT_ERR_INVALID_ARG, "lse is not 4-byte aligned");
  TRY(check_apart({o, lse}, {q, k, v, offsets}));
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.out = static_cast<char*>(o);
  a.lse = lse;
  lact_attention all = w;  // for the rules: as many tiles as one sequence of all rows has
  all.batch = 1, all.q_len = all.k_len = p->tokens;
  const int ks = parts_q(all);
  row_tiles(w, 128 / ks, a);
  const int64_t tiles = w.batch == 0 || w.q_len == 0 ? 0 : count_tiles(w, p->tokens, 128 / ks / a.hg, a);
  const int64_t clear = p->flags & LACT_CLEAR_REST ? rest_groups(p->tokens * w.heads * w.d * es) : 0;
  const int64_t main = tiles * (w.heads / a.hg), grid = main + clear;
  TRY(check_grid(grid, 256));
  TRY(check_device_again());
  if (grid == 0) return LACT_OK;
  a.main = (int32_t)main;
  a.rest = (int32_t)clear;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  KernelTimer kt(LACT_K_ATTN, s);
  return by_tile(w, [&](auto t, auto dp) -> lact_status {
    by_parts(t, dp, ks, [&](auto n) {
      LACT_LAUNCH((attn_fwd_kernel<decltype(t), decltype(dp)::value, decltype(n)::value, PackedArgs>), dim3((unsigned)grid),
                  dim3(256), s, a);
    });
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

}  // extern "C"

namespace {

// The backward's workgroups, split sink tiles and workspace
struct PackedBack {
  PackedArgs q, kv;          // tile fields of the two kernels
  int ksq = 1, ksk = 1;
  int64_t gq = 0, gk = 0, gs = 0;  // workgroups: dq; dk, dv; sums of parts
  size_t part = 0, total = 0;
};
// Parts of the rows of a key tile, of `work` tiles a key head (as far as the
// host can tell) and `jobs` workgroups at most: shared work and half of the
// longest workgroup, or all of it, against a launch more and the parts' way
// through memory.  Training steps, us with 1, 2, 3, 5, 8 parts: fp32, 6 texts of
// 4001 tokens, window 333, 12 (4) heads of 96: 721, 680, 598, 583, 584; bf16:
// 135, 141, 145, 169, 203; 4 texts of 8000 tokens, 8 (2) heads of 128, causal:
// 599, 437, 429, 445, 474; 4000 tokens, 32 (8) heads of 128: 413, 351, 355, 381,
// 452; 16 heads of 64: 146, 168, 173, 190, 249.  Of these it takes 5, 1, 5, 3, 1.
int row_splits(const lact_attention& w, int64_t work, int64_t jobs, int64_t BK) {
  const bool fp32 = w.io_dtype == LACT_DTYPE_F32, wide = w.d > 64;
  const int64_t room = (fp32 || wide ? 1 : 2) * NCU, BQ = fp32 && wide ? 32 : 64, G = w.heads / w.kv_heads;
  const int64_t most = G * ceil_div(limited(w) ? std::min(w.k_len, w.window + BK) : w.k_len, BQ);  // row tiles of a key tile
  const double mean = limited(w) ? (double)most : 0.5 * (double)most;
  const double t = (fp32 ? 7.0 : wide ? 3.5 : 1.8) * (BK == 64 ? 0.5 : 1.0);  // us a row tile
  double best = 1e30;
  int parts = 1;
  for (int64_t s = 1; s <= 16 && s <= most && (s == 1 || jobs * w.kv_heads * s <= 8 * NCU); ++s) {
    const double sums = s > 1 ? 8.0 + (double)(jobs * w.kv_heads * s) * (double)(2 * BK * w.d * 8) / 4e6 : 0.0;
    const double longest = (double)most / (double)s, share = (double)(work * w.kv_heads) * mean / (double)room;
    const double cost = std::max(longest, share + 0.5 * longest) * t + sums;
    if (cost < best) best = cost, parts = (int)s;
  }
  return parts;
}

PackedBack packed_back(const lact_packed& p, const lact_attention& w) {
  PackedBack x;
  memset(&x.q, 0, sizeof(x.q));
  memset(&x.kv, 0, sizeof(x.kv));
  x.part = align256((size_t)w.heads * p.tokens * 2 * 4);
  x.total = x.part;
  if (w.batch == 0 || w.q_len == 0) return x;
  lact_attention all = w;
  all.batch = 1, all.q_len = all.k_len = p.tokens;
  x.ksq = parts_q(all);
  x.ksk = parts_k(all);
  row_tiles(w, 128 / x.ksq, x.q);
  x.gq = count_tiles(w, p.tokens, 128 / x.ksq / x.q.hg, x.q) * (w.heads / x.q.hg);
  const int64_t BK = 128 / x.ksk;
  sink_plan(w, BK, x.kv);
  const int64_t tiles = count_tiles(w, p.tokens, BK, x.kv);
  const int64_t split = x.kv.splits > 1 ? (int64_t)w.batch * x.kv.sink_tiles : 0;  // sink tiles in parts, a key head
  const int64_t jobs = tiles + split * x.kv.splits;
  x.kv.rs = row_splits(w, std::min(tiles, ceil_div(p.tokens, BK)) + split, jobs, BK);
  x.gk = jobs * w.kv_heads * x.kv.rs;
  x.gs = (x.kv.rs > 1 ? tiles + split : split) * w.kv_heads * (2 * BK / 8);
  const int64_t parts = x.kv.rs > 1 ? jobs * x.kv.rs : split * x.kv.splits;  // a key head
  x.total += align256((size_t)parts * w.kv_heads * 2 * BK * w.d * 4);
  return x;
}

}  // namespace

extern "C" {

size_t lact_packed_attention_backward_workspace_size(const lact_packed* p) {
  g_err.clear();
  lact_attention w;
  if (validate(p, &w)) return 0;
  return packed_back(*p, w).total;
}

lact_status lact_packed_attention_backward(const lact_packed* p, const void* q, const lact_strides* sq, const void* k,
                                           const lact_strides* sk, const void* v, const lact_strides* sv,
                                           const int64_t* offsets, const void* o, const lact_strides* so,
                                           const float* lse, const void* dO, const lact_strides* sdo, void* dq,
                                           const lact_strides* sdq, void* dk, const lact_strides* sdk, void* dv,
                                           const lact_strides* sdv, void* ws, size_t ws_bytes, void* stream) {
  g_err.clear();
  lact_attention w;
  TRY(validate(p, &w));
  if (p->tokens == 0) return LACT_OK;
  PackedArgs a;
  memset(&a, 0, sizeof(a));
  fill_args(a, w, p->tokens, offsets);
  const int64_t es = size_of(w.io_dtype);
  TRY(check_tensor("q", q, sq, 1, w.heads, p->tokens, w.d, es, 16, false, &a.sq));
  TRY(check_tensor("k", k, sk, 1, w.kv_heads, p->tokens, w.d, es, 16, false, &a.sk));
  TRY(check_tensor("v", v, sv, 1, w.kv_heads, p->tokens, w.d, es, 16, false, &a.sv));
  TRY(check_tensor("o", o, so, 1, w.heads, p->tokens, w.d, es, 16, false, &a.so));
  TRY(check_tensor("dO", dO, sdo, 1, w.heads, p->tokens, w.d, es, 16, false, &a.sdo));
  TRY(check_tensor("dq", dq, sdq, 1, w.heads, p->tokens, w.d, es, 16, true, &a.sdq));
  TRY(check_tensor("dk", dk, sdk, 1, w.kv_heads, p->tokens, w.d, es, 16, true, &a.sdk));
  TRY(check_tensor("dv", dv, sdv, 1, w.kv_heads, p->tokens, w.d, es, 16, true, &a.sdv));
  NEED(lse, 4);
  TRY(check_offsets(offsets));
  TRY(check_apart({dq, dk, dv}, {q, k, v, o, dO, lse, offsets}));
  const PackedBack x = packed_back(*p, w);
  TRY(check_ws(ws, ws_bytes, x.total));
  a.q = static_cast<const char*>(q);
  a.k = static_cast<const char*>(k);
  a.v = static_cast<const char*>(v);
  a.o = static_cast<const char*>(o);
  a.dO = static_cast<const char*>(dO);
  a.dq = static_cast<char*>(dq);
  a.dk = static_cast<char*>(dk);
  a.dv = static_cast<char*>(dv);
  a.lse = const_cast<float*>(lse);
  a.stats = static_cast<float*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + x.part);
  a.rest = rest_groups(p->tokens * w.heads * w.d * es);
  PackedArgs kv = a;
  a.hg = x.q.hg, a.tiles = x.q.tiles, a.slots = x.q.slots, a.main = (int32_t)x.gq;
  kv.tiles = x.kv.tiles, kv.slots = x.kv.slots, kv.main = (int32_t)x.gk;
  kv.rs = std::max(1, x.kv.rs), kv.splits = std::max(1, x.kv.splits), kv.sink_tiles = x.kv.sink_tiles, kv.span = x.kv.span;
  TRY(check_grid(std::max(x.gq, x.gk) + a.rest, 256));
  TRY(check_grid(x.gs, 256));
  TRY(check_device_again());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return by_tile(w, [&](auto t, auto dp) -> lact_status {
    using T = decltype(t);
    constexpr int DP = decltype(dp)::value;
    {
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      by_parts(t, dp, x.ksq, [&](auto n) {
        LACT_LAUNCH((attn_dq_kernel<T, DP, decltype(n)::value, PackedArgs>), dim3((unsigned)(x.gq + a.rest)), dim3(256), s, a);
      });
    }
    {
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      by_parts(t, dp, x.ksk, [&](auto n) {
        LACT_LAUNCH((attn_dkv_kernel<T, DP, decltype(n)::value, PackedArgs>), dim3((unsigned)(x.gk + a.rest)), dim3(256), s, kv);
      });
    }
    if (x.gs > 0) {
      const dim3 grid((unsigned)x.gs);
      KernelTimer kt(LACT_K_ATTN_BWD, s);
      if (x.kv.rs > 1 && x.ksk == 2) LACT_LAUNCH((attn_row_sum_kernel<T, 64>), grid, dim3(256), s, kv);
      else if (x.kv.rs > 1) LACT_LAUNCH((attn_row_sum_kernel<T, 128>), grid, dim3(256), s, kv);
      else if (x.ksk == 2) LACT_LAUNCH((attn_sink_sum_kernel<T, 64, PackedArgs>), grid, dim3(256), s, kv);
      else LACT_LAUNCH((attn_sink_sum_kernel<T, 128, PackedArgs>), grid, dim3(256), s, kv);
    }
    HIP_TRY(hipGetLastError());
    return LACT_OK;
  });
}

}  // extern "C"

// ------------------------------------------------------------------ slots and writes
namespace {

lact_status validate(const lact_slots* p) {
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  if (p->batch < 0 || p->batch > MOST_BATCH) return fail(LACT_ERR_INVALID_ARG, "batch = %d", p->batch);
  TRY(check_page(p->page, 0, p->width));
  if (p->entries < 0 || p->entries >= MOST_PAGES) return fail(LACT_ERR_INVALID_ARG, "entries = %d", p->entries);
  if (p->tokens < 0 || p->tokens >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "tokens = %lld", (long long)p->tokens);
  return LACT_OK;
}

// Whether every workgroup sums the requests itself
bool slots_in_one(const lact_slots& p) { return p.batch <= ONE_GROUP; }

}  // namespace

extern "C" {

size_t lact_page_slots_workspace_size(const lact_slots* p) {
  g_err.clear();
  if (validate(p)) return 0;
  return slots_in_one(*p) ? 0 : align256((size_t)p->batch * 4);
}

lact_status lact_page_slots(const lact_slots* p, const int64_t* lens, const int64_t* counts, int32_t* table,
                            const int32_t* free, const int64_t* have, int64_t* offsets, int64_t* k_lens,
                            int64_t* slots, int64_t* positions, int64_t* left, void* ws, size_t ws_bytes,
                            void* stream) {
  g_err.clear();
  TRY(validate(p));
  if (p->batch > 0) {
    NEED(lens, 8);
    NEED(counts, 8);
    NEED(k_lens, 8);
    if (p->width > 0) NEED(table, 4);
  }
  if (p->entries > 0) NEED(free, 4);
  NEED(have, 8);
  NEED(offsets, 8);
  NEED(left, 8);
  if (p->tokens > 0) {
    NEED(slots, 8);
    NEED(positions, 8);
  }
  TRY(check_apart({offsets, k_lens, slots, positions, left, table}, {lens, counts, free}));
  TRY(check_apart({offsets, k_lens, slots, positions, table}, {have}));
  const bool one = slots_in_one(*p);
  if (!one) TRY(check_ws(ws, ws_bytes, align256((size_t)p->batch * 4)));
  TRY(check_device_again());
  SlotArgs a;
  memset(&a, 0, sizeof(a));
  a.lens = lens, a.counts = counts, a.table = table, a.free = free, a.have = have;
  a.offsets = offsets, a.k_lens = k_lens, a.slots = slots, a.positions = positions, a.left = left;
  a.base = static_cast<int32_t*>(ws);
  a.B = p->batch, a.T = (int32_t)p->tokens, a.width = p->width, a.entries = p->entries;
  a.by_page = FastDiv((uint32_t)p->page);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (one) {
    KernelTimer kt(LACT_K_PAGES, s);
    // `left` in place of `have` is written by the only workgroup that reads it
    // (1024 requests, 32768 tokens: 45 us for 8)
    const unsigned grid = left == have ? 1 : (unsigned)std::max<int64_t>(1, ceil_div(p->tokens, PLAN_THREADS));
    LACT_LAUNCH(slots_one_kernel, dim3(grid), dim3(PLAN_THREADS), s, a);
  } else {
    {
      KernelTimer kt(LACT_K_PAGES, s);
      LACT_LAUNCH(slots_plan_kernel, dim3(1), dim3(PLAN_THREADS), s, a);
    }
    KernelTimer kt(LACT_K_PAGES, s);
    if (p->tokens > 0) LACT_LAUNCH(slots_fill_kernel, dim3((unsigned)ceil_div(p->tokens, 256)), dim3(256), s, a);
  }
  HIP_TRY(hipGetLastError());
  return LACT_OK;
}

lact_status lact_page_write(const lact_write* p, const void* k, const lact_strides* sk, const void* v,
                            const lact_strides* sv, const int64_t* slots, void* k_pages, const lact_strides* skp,
                            void* v_pages, const lact_strides* svp, void* stream) {
  g_err.clear();
  if (!p) return fail(LACT_ERR_INVALID_ARG, "problem is NULL");
  if (p->kv_heads < 1 || p->kv_heads > 65536) return fail(LACT_ERR_INVALID_ARG, "kv_heads = %d", p->kv_heads);
  TRY(check_dtype(p->io_dtype));
  const int64_t es = size_of(p->io_dtype);
  if (p->d < 1 || p->d > 8192 || p->d * es % 16)
    return fail(LACT_ERR_UNSUPPORTED, "d = %d: need a multiple of 16 bytes, at most 8192 elements", p->d);
  TRY(check_page(p->page, p->pages, 0));
  if (p->tokens < 0 || p->tokens >= MOST_TOKENS) return fail(LACT_ERR_INVALID_ARG, "tokens = %lld", (long long)p->tokens);
  if (p->tokens == 0 || p->pages == 0) return LACT_OK;
  WriteArgs a;
  memset(&a, 0, sizeof(a));
  TRY(check_tensor("k", k, sk, 1, p->kv_heads, p->tokens, p->d, es, 16, false, &a.si[0]));
  TRY(check_tensor("v", v, sv, 1, p->kv_heads, p->tokens, p->d, es, 16, false, &a.si[1]));
  TRY(check_tensor("k_pages", k_pages, skp, p->pages, p->kv_heads, p->page, p->d, es, 16, true, &a.so[0]));
  TRY(check_tensor("v_pages", v_pages, svp, p->pages, p->kv_heads, p->page, p->d, es, 16, true, &a.so[1]));
  NEED(slots, 8);
  TRY(check_apart({k_pages, v_pages}, {k, v, slots}));
  a.in[0] = static_cast<const char*>(k);
  a.in[1] = static_cast<const char*>(v);
  a.out[0] = static_cast<char*>(k_pages);
  a.out[1] = static_cast<char*>(v_pages);
  a.slots = slots;
  a.places = (int64_t)p->pages * p->page;
  a.T = (int32_t)p->tokens;
  const int64_t head = p->d * es / 16, row = 2 * p->kv_heads * head;  // at most 2^28
  a.by_head = FastDiv((uint32_t)head);
  a.by_row = FastDiv((uint32_t)row);
  a.by_page = FastDiv((uint32_t)p->page);
  // four accesses a thread where that leaves workgroups enough, one otherwise
  a.tokens = (int32_t)std::max<int64_t>(1, (p->tokens * row >= 4 * 256 * 8 * NCU ? 1024 : 256) / row);
  const int64_t grid = ceil_div(p->tokens, a.tokens);
  TRY(check_grid(grid, 256));
  TRY(check_device_again());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  KernelTimer kt(LACT_K_PAGES, s);
  LACT_LAUNCH(page_write_kernel, dim3((unsigned)grid), dim3(256), s, a);
  HIP_TRY(hipGetLastError());
  return LACT_OK;
}

}  // extern "C"
