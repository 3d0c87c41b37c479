// Sliding-window attention with sinks, forward and backward, on the 32x32
// MFMA tiles of gfx950.
//
// Row r of a sequence stands at p = k_len - q_len + r and sees the keys
// j <= p with j > p - window or j < sinks.  With s = scale q.k:
//   lse = log sum_j exp(s_j),  o = sum_j exp(s_j - lse) v_j
//   P = exp(s - lse), D = dO.o, dS = P (dO.v - D)
//   dq = scale sum_j dS k_j,  dk_j = scale sum_r dS q_r,  dv_j = sum_r P dO_r.
//
// Layout trick all kernels share.  A product runs transposed, so that the
// result's column -- the lane -- is the index that the next product keeps:
// S^T = K Q^T leaves lane n with row n's scores of 16 of a block's 32 keys
// (register r of lane half h holds key 8 (r/4) + 4 h + r%4).  The softmax is
// then lane-local, and since the order of a contraction is free, registers
// 8i .. 8i+7 already are a B operand of O^T = V^T P^T if the A operand reads
// its keys in the same order: V^T comes out of LDS by two transposing 4-row
// reads per fragment, and P never passes through LDS.  The backward's dK and
// dV swap the roles of keys and rows.
//
// Numbers: scores, softmax statistics and all sums are fp32.  For bf16
// tensors P and dS are rounded to bf16 once, as operands of their products
// (half a step, 2^-8 of the value, like the result itself); for fp32 tensors
// every product is an fp32 MFMA and nothing is rounded.
#pragma once
#include "lact_direct.hpp"
#include "lact_stream_work.hpp"

namespace lact {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// Products by which an operand's read from LDS comes before its own: 4 x 32
// cycles of the matrix pipe cover the read (read just before: dk, dv of a 32K
// step of 16 heads, d = 64, 614 us for 575).
constexpr int AHEAD = 4;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// byte strides of a [batch, heads, tokens, d] tensor with d contiguous
struct AttnStride {
  int64_t b, h, l;
};

// How a batch lies in memory.  PADDED: [batch, heads, tokens, d] and lengths.
// PACKED: [heads, tokens, d], with the rows and keys of sequence b at tokens
// offsets[b] .. offsets[b + 1].  PAGED: rows so, keys in pages of a pool
// [pages, heads, page, d] that each sequence's row of a table names.
enum class Lie { PADDED, PACKED, PAGED };

struct AttnArgs {
  static constexpr Lie LIE = Lie::PADDED;
  const char *q, *k, *v, *o, *dO;
  char *out, *dq, *dk, *dv;
  AttnStride sq, sk, sv, so, sdo, sdq, sdk, sdv;
  const int64_t *q_lens, *k_lens;  // device, or null: Lq, Lk
  float* lse;                      // [B, H, Lq], or null (forward)
  float* stats;                    // [2][B, H, Lq]: -lse / scale (fp32: -lse) and -D, D = dO.o
  float* part;                     // partial sums (few-row forward: O; backward: dK, dV of sink tiles)
  float* part_ml;                  // few-row forward: running maximum and sum of each split
  int32_t B, H, Hk, G;             // G = H / Hk query heads share a key head
  int32_t d, Lq, Lk;
  int32_t window, sinks;           // window: 1 << 30 where there is none
  int32_t hg;                      // query heads of a workgroup (forward, dq): its waves share their keys
  int32_t tiles;                   // row tiles (forward, dq; few-row forward: of 32), key tiles (dk, dv), per head
  int32_t splits;                  // few-row forward: key splits; backward: row splits of a sink tile
  int32_t sink_tiles, span;        // backward: key tiles with sinks; rows of one of their splits
  float c;                         // scale * log2(e): exp(scale s) = exp2(c s)
  float scale;
};
struct PackedArgs : AttnArgs {   // Lq: tokens of all sequences, the strides' b unused
  static constexpr Lie LIE = Lie::PACKED;
  const int64_t* offsets;  // [B + 1], device
  int32_t most;            // rows of a sequence (and its keys, packed) that are looked at
  int32_t slots;           // tiles of all sequences together, see find_tile; 0: `tiles` for each
  int32_t main;            // workgroups that compute; those behind them clear rows of no sequence
  int32_t rest;            // how many those are
  int32_t rs;              // dk, dv: parts that the rows of a tile are split in
};
struct PagedArgs : PackedArgs {  // Lk: keys of a sequence that are looked at
  static constexpr Lie LIE = Lie::PAGED;
  const int32_t* table;    // [B, width]
  int32_t width, pages;
  FastDiv by_page;
  int32_t few;             // sequences of up to so many rows are the streams', others the forward's
  int32_t chunk;           // forward: tiles of a key split, of which there are at most `splits`
  int32_t waves, share;    // streams: waves of the launch, fewest units of one
  int32_t unit;            // tiles of a unit of work
  int32_t rows;            // rows of a partial result: of an item, at most 32
  int32_t* upto;           // [B + 1]: work of the sequences before each, null: summed by every workgroup
  struct StreamJoin* joins;  // [waves]
};

// An LDS location's byte offset: the low half of its generic address (a cast to
// the LDS address space would test for null every time).
__device__ __forceinline__ uint32_t lds_at(const void* p) { return (uint32_t)(uintptr_t)p; }

// ------------------------------------------------------------------ tiles
// One LDS tile holds R rows of DP elements (DP = d rounded up to 64 or 128)
// as 16-byte chunks.  Chunk c of row r lies in slot c ^ f(r): the 16-byte
// reads of 16 consecutive rows then fall in 16 different slots, and for bf16
// the transposing reads of 4 rows x 64 bytes in four different 64-byte groups.
template <typename T, int DP>
struct AttnTile {
  static constexpr int CPR = DP * (int)sizeof(T) / 16;  // chunks per row
  static constexpr int STEPS = CPR / 2;                 // chunk pairs: contraction steps of a row product
  static constexpr int DB = DP / 32;                    // 32-wide blocks of d
  __device__ static __forceinline__ int f(int r) {
    if constexpr (sizeof(T) == 4) return r & 15;
    else if constexpr (CPR == 16) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
  }
  __device__ static __forceinline__ int at(int r, int c) { return (r * CPR + (c ^ f(r))) * 16; }

  // Copies rows row0 .. row0 + R - 1 of a matrix (row stride in bytes) to the
  // tile, by NW waves.  Rows outside 0 .. rmax and chunks behind the head's
  // last are read from the nearest one inside: what lies there is masked, or
  // meets a zero, by whoever uses the tile, and no memory outside is touched.
  template <int R, int NW>
  __device__ static __forceinline__ void stage(char* tile, const char* base, int64_t stride, int row0, int rmax,
                                               int cmax, int wave, int lane) {
    constexpr int N = R * CPR / (WAVE * NW);
    static_assert(R * CPR % (WAVE * NW) == 0, "whole copies");
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_at(tile) + (uint32_t)(wave * WAVE * 16));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = (i * NW + wave) * WAVE + lane;
      const int row = s / CPR, c = min((s % CPR) ^ f(row), cmax);
      const int gr = max(0, min(row0 + row, rmax));
      dma16(base + (int64_t)gr * stride + c * 16, m0 + (uint32_t)(i * NW * WAVE * 16));
    }
  }
};

// One direct load of 16 bytes a lane from a uniform base and a lane's offset.
// The base is moved by the scalar unit first: a vector instruction that wrote
// it (a spilled one's v_readlane) has to be five wait states before the load,
// which the compiler does not see here; a scalar move waits for it by itself.
__device__ __forceinline__ void dma16_at(uint32_t off, const char* base, uint32_t m0) {
  const char* at;
  asm volatile("s_mov_b32 m0, %3\n\ts_mov_b64 %0, %2\n\tglobal_load_lds_dwordx4 %1, %0"
               : "=&s"(at)
               : "v"(off), "s"(base), "s"(m0)
               : "memory", "m0");
}

// AttnTile::stage with the lanes' offsets kept: a tile inside the matrix then
// costs no vector arithmetic (formed anew for every tile, offsets were 40 of
// the 143 vector instructions that the forward spends on 32 x 32 scores).
template <typename T, int DP, int R, int NW>
struct Stager {
  using Tile = AttnTile<T, DP>;
  static constexpr int N = R * Tile::CPR / (WAVE * NW);
  static constexpr int64_t FAR = (INT64_C(1) << 31) / R;  // row strides whose offsets need more than 32 bits
  const char* base;
  int64_t stride;
  int rmax, cmax, wave, lane;
  uint32_t off[N];
  __device__ __forceinline__ Stager(const char* base_, int64_t stride_, int rmax_, int cmax_, int wave_, int lane_)
      : base(base_), stride(stride_), rmax(rmax_), cmax(cmax_), wave(wave_), lane(lane_) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int s = (i * NW + wave) * WAVE + lane, row = s / Tile::CPR;
      off[i] = (uint32_t)row * (uint32_t)stride + (uint32_t)min((s % Tile::CPR) ^ Tile::f(row), cmax) * 16u;
    }
  }
  __device__ __forceinline__ void issue(char* tile, int row0) const {
    if (row0 >= 0 && row0 + R - 1 <= rmax && stride < FAR) {
      const char* b = base + (int64_t)row0 * stride;
      const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds_at(tile) + (uint32_t)(wave * WAVE * 16));
#pragma unroll
      for (int i = 0; i < N; ++i) dma16_at(off[i], b, m0 + (uint32_t)(i * NW * WAVE * 16));
    } else {
      Tile::template stage<R, NW>(tile, base, stride, row0, rmax, cmax, wave, lane);
    }
  }
};

// The copies of a K and a V tile, and single rows of both.
template <typename T, int DP, int R, int NW>
struct KeyRows {
  static constexpr int TB = R * AttnTile<T, DP>::CPR * 16;
  Stager<T, DP, R, NW> sk, sv;
  __device__ __forceinline__ KeyRows(const char* kb, int64_t kl, const char* vb, int64_t vl, int rmax, int cmax,
                                     int wave, int lane)
      : sk(kb, kl, rmax, cmax, wave, lane), sv(vb, vl, rmax, cmax, wave, lane) {}
  __device__ __forceinline__ void issue(char* tile, int row0) const {
    sk.issue(tile, row0);
    sv.issue(tile + TB, row0);
  }
  __device__ __forceinline__ const char* k(int j) const { return sk.base + j * sk.stride; }
  __device__ __forceinline__ const char* v(int j) const { return sv.base + j * sv.stride; }
};

// Single rows of dense K and V.
struct TokenRows {
  const char *kb, *vb;
  int64_t kl, vl;
  __device__ __forceinline__ const char* k(int j) const { return kb + j * kl; }
  __device__ __forceinline__ const char* v(int j) const { return vb + j * vl; }
};

// The same out of pages.  The rows that a wave copies at once, 64 / CPR <= 8
// of them at a multiple of as many, lie in one page, since pages are multiples
// of 8 rows: their page is a scalar, and a copy has a scalar base and the
// lanes' kept offsets, as in a dense matrix.  An entry outside the pool is
// taken as the nearest page inside: what it holds is masked (entries before a
// window, say), and no memory outside the pool is touched.
template <typename T, int DP, int R, int NW>
struct PageRows {
  using Tile = AttnTile<T, DP>;
  static constexpr int TB = R * Tile::CPR * 16, N = R * Tile::CPR / (WAVE * NW), GROUP = WAVE / Tile::CPR;
  static_assert(GROUP <= 8, "a group of rows lies in one page");
  typedef const __attribute__((address_space(4))) int32_t* Entries;  // scalar loads: written before the kernel
  const char *kb, *vb;
  AttnStride ks, vs;
  Entries table;
  FastDiv by_page;
  int last, rmax, cmax, wave, lane;
  uint32_t ko[N], vo[N];
  __device__ __forceinline__ PageRows(const PagedArgs& a, int b, int hk, int rmax_, int wave_, int lane_)
      : kb(a.k + hk * a.sk.h), vb(a.v + hk * a.sv.h), ks(a.sk), vs(a.sv),
        table((Entries)(uintptr_t)(a.table + (int64_t)b * a.width)), by_page(a.by_page), last(a.pages - 1), rmax(rmax_),
        cmax(a.d * (int)sizeof(T) / 16 - 1), wave(wave_), lane(lane_) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = (i * NW + wave) * GROUP + lane / Tile::CPR;
      const uint32_t c = (uint32_t)min((lane % Tile::CPR) ^ Tile::f(row), cmax) * 16u;
      ko[i] = (uint32_t)(lane / Tile::CPR) * (uint32_t)ks.l + c;
      vo[i] = (uint32_t)(lane / Tile::CPR) * (uint32_t)vs.l + c;
    }
  }
  __device__ __forceinline__ void issue(char* tile, int row0) const { issue(tile, tile + TB, row0); }
  // (a null tile is left out)
  __device__ __forceinline__ void issue(char* ktile, char* vtile, int row0) const {
    const uint32_t at = (uint32_t)(wave * WAVE * 16);
    const uint32_t mk = __builtin_amdgcn_readfirstlane(lds_at(ktile) + at), mv = __builtin_amdgcn_readfirstlane(lds_at(vtile) + at);
    if (row0 + R - 1 <= rmax) {
      int page[N], in[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = __builtin_amdgcn_readfirstlane(row0 + (i * NW + wave) * GROUP), n = (int)by_page.div((uint32_t)row);
        in[i] = row - n * (int)by_page.d;
        page[i] = table[n];
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int64_t e = max(0, min(page[i], last));
        if (ktile) dma16_at(ko[i], kb + e * ks.b + in[i] * ks.l, mk + (uint32_t)(i * NW * WAVE * 16));
        if (vtile) dma16_at(vo[i], vb + e * vs.b + in[i] * vs.l, mv + (uint32_t)(i * NW * WAVE * 16));
      }
    } else {  // rows behind the last are read from it
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int row = (i * NW + wave) * GROUP + lane / Tile::CPR, gr = min(row0 + row, rmax);
        const int c = min((lane % Tile::CPR) ^ Tile::f(row), cmax) * 16;
        if (ktile) dma16(k(gr) + c, mk + (uint32_t)(i * NW * WAVE * 16));
        if (vtile) dma16(v(gr) + c, mv + (uint32_t)(i * NW * WAVE * 16));
      }
    }
  }
  __device__ __forceinline__ const char* row(const char* base, const AttnStride& s, int j) const {
    const int n = (int)by_page.div((uint32_t)j);
    const int64_t e = max(0, min(table[n], last));
    return base + e * s.b + (int64_t)(j - n * (int)by_page.d) * s.l;
  }
  __device__ __forceinline__ const char* k(int j) const { return row(kb, ks, j); }
  __device__ __forceinline__ const char* v(int j) const { return row(vb, vs, j); }
};

// ------------------------------------------------------------------ products
// A 16-byte chunk per lane is the unit of a row product's operand.  Lane l
// supplies row l % 32 and chunk 2 s + l / 32 of step s, for A and B alike:
// which elements of the contraction that pairs is the same on both sides.
template <typename T> struct AttnFrag;
template <> struct AttnFrag<bf16_t> { using type = bf16x8; };
template <> struct AttnFrag<float> { using type = f32x4; };
template <typename T> using Frag = typename AttnFrag<T>::type;

__device__ __forceinline__ f32x16 mma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 mma32(f32x4 a, f32x4 b, f32x16 c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_32x32x2f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

template <typename T, int DP>
__device__ __forceinline__ Frag<T> row_frag(const char* tile, int row0, int s, int lane) {
  return *reinterpret_cast<const Frag<T>*>(
      tile + AttnTile<T, DP>::at(row0 + (lane & 31), 2 * s + (lane >> 5)));
}

// the same operand straight from a row in memory; chunks behind the last are zero
template <typename F, int STEPS>
__device__ __forceinline__ void load_rows(F (&f)[STEPS], const char* row, int cmax, int lane) {
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const int c = 2 * s + (lane >> 5);
    uint4 x = zero4();
    if (c <= cmax) x = *reinterpret_cast<const uint4*>(row + c * 16);
    f[s] = __builtin_bit_cast(F, x);
  }
}

__device__ __forceinline__ f32x16 zero16() {
  f32x16 z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.f;
  return z;
}

// bf16: A fragment of rows row0 + 16 kb .. + 15 transposed, columns 32 db .. + 31
template <int DP>
__device__ __forceinline__ bf16x8 trans_frag(const char* tile, int row0, int kb, int db, int lane) {
  const int j = lane & 15;
  const int row = row0 + 16 * kb + 4 * (lane >> 5) + (j >> 2);
  const int chunk = 4 * db + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1), half = (j & 1) * 8;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(tile + AttnTile<bf16_t, DP>::at(row, chunk) + half));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) v4s*)(tile + AttnTile<bf16_t, DP>::at(row + 8, chunk) + half));
  typedef short v8s __attribute__((ext_vector_type(8)));
  const v8s v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(bf16x8, v);
}
// fp32: element (row 8 (r/4) + 4 h + r%4, column 32 db + l%32)
template <int DP>
__device__ __forceinline__ float trans_elem(const char* tile, int row0, int r, int db, int lane) {
  const int row = row0 + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3), col = 32 * db + (lane & 31);
  return *reinterpret_cast<const float*>(tile + AttnTile<float, DP>::at(row, col >> 2) + (col & 3) * 4);
}

// A lane's offsets into a bf16 tile, formed once: with the tile's place and a
// block's first row as constants, every read's address is one of these
// registers and an immediate.
typedef const __attribute__((address_space(3))) char* lds_ptr;
template <int DP>
struct AttnAddr {
  using Tile = AttnTile<bf16_t, DP>;
  static constexpr int STEPS = Tile::STEPS, DB = DP / 32, ROW = Tile::CPR * 16;
  int r[STEPS], t[DB][2];
  __device__ __forceinline__ explicit AttnAddr(int lane) {
#pragma unroll
    for (int s = 0; s < STEPS; ++s) r[s] = Tile::at(lane & 31, 2 * s + (lane >> 5));
    const int j = lane & 15, row = 4 * (lane >> 5) + (j >> 2);
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        t[db][i] = Tile::at(row + 8 * i, 4 * db + 2 * ((lane >> 4) & 1) + ((j & 3) >> 1)) + (j & 1) * 8;
  }
  // operand of a row product: rows row0 .. row0 + 31 (row0 a multiple of 32), step s
  __device__ __forceinline__ bf16x8 rows(lds_ptr tile, int row0, int s) const {
    return *reinterpret_cast<const __attribute__((address_space(3))) bf16x8*>(tile + r[s] + row0 * ROW);
  }
  // transposed operand: rows row0 .. row0 + 15 (row0 a multiple of 16), columns 32 db .. 32 db + 31
  __device__ __forceinline__ bf16x8 cols(lds_ptr tile, int row0, int db) const {
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(tile + t[db][0] + row0 * ROW));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)(tile + t[db][1] + row0 * ROW));
    typedef short v8s __attribute__((ext_vector_type(8)));
    const v8s v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    return __builtin_bit_cast(bf16x8, v);
  }
};

// acc^T[d x lane] += sum over the tile's 32 rows from row0 of row^T p, with p
// in the layout a 32x32 product leaves.
template <int DP>
__device__ __forceinline__ void mma_trans(f32x16 (&acc)[DP / 32], const bf16x8 (&b)[2], const char* tile, int row0,
                                          int lane) {
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) acc[db] = mma32(trans_frag<DP>(tile, row0, kb, db, lane), b[kb], acc[db]);
}
// (fp32, see row_steps: blocks of d behind its last are left out)
template <int DP>
__device__ __forceinline__ void mma_trans(f32x16 (&acc)[DP / 32], const f32x16& p, const char* tile, int row0,
                                          int lane, int d) {
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
    if (DP <= 64 || 32 * db < d) {
#pragma unroll
      for (int r = 0; r < 16; ++r)
        acc[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(trans_elem<DP>(tile, row0, r, db, lane), p[r], acc[db], 0, 0, 0);
    }
}
// The steps of a row product, fn(s): fp32 tiles of 128 leave out 32-wide blocks
// behind d (5 texts of up to 1777 tokens, 12 (4) heads of 96: forward 171 -> 141
// us, backward 751 -> 596; at d <= 64 the branch cost 4 % and d <= 32 is rare)
template <typename T, int STEPS, class F>
__device__ __forceinline__ void row_steps(int d, F&& fn) {
  constexpr int N = sizeof(T) == 2 || STEPS <= 8 ? STEPS : 4;
#pragma unroll
  for (int g = 0; g < STEPS; g += N)
    if (N == STEPS || 8 * g < d) {
#pragma unroll
      for (int s = g; s < g + N; ++s) fn(s);
    }
}

// p as the operand of mma_trans: rounded to bf16 (registers 8 i .. 8 i + 7 are
// fragment i), or as it is
struct Pair {
  bf16x8 f[2];
};
__device__ __forceinline__ Pair round_pair(const f32x16& p) {
  Pair b;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    b.f[i] = __builtin_bit_cast(bf16x8, make_uint4(pack_bf16x2(p[8 * i], p[8 * i + 1]), pack_bf16x2(p[8 * i + 2], p[8 * i + 3]),
                                                   pack_bf16x2(p[8 * i + 4], p[8 * i + 5]), pack_bf16x2(p[8 * i + 6], p[8 * i + 7])));
  return b;
}
// the sum of a packed pair of bf16 and c
__device__ __forceinline__ float pair_add(uint32_t x, float c) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, x), bf16x2{(__bf16)1.f, (__bf16)1.f}, c, false);
}

// half a tile of the backward: scores then P, dP - D then dS, and both rounded
// pair by pair
struct Half {
  f32x16 s, ds;
  uint32_t x[8], y[8];
  __device__ __forceinline__ void round(int i) {
    x[i] = pack_bf16x2(ds[2 * i], ds[2 * i + 1]);
    y[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
  }
  __device__ __forceinline__ bf16x8 frag_ds(int i) const {
    return __builtin_bit_cast(bf16x8, make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
  }
  __device__ __forceinline__ bf16x8 frag_s(int i) const {
    return __builtin_bit_cast(bf16x8, make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
  }
};

template <typename T, int DP>
__device__ __forceinline__ void acc_trans(f32x16 (&acc)[DP / 32], const f32x16& p, const char* tile, int row0, int lane,
                                          int d) {
  if constexpr (sizeof(T) == 2) mma_trans<DP>(acc, round_pair(p).f, tile, row0, lane);
  else mma_trans<DP>(acc, p, tile, row0, lane, d);
}

// maximum and sum of a lane and its partner 32 away
__device__ __forceinline__ float pair_max(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float pair_sum(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ __forceinline__ int seq_len(const int64_t* lens, int b, int most) {
  if (!lens) return most;
  const int64_t n = lens[b];
  return (int)(n < 0 ? 0 : n > most ? most : n);
}

// A sequence: its lengths, and in a packed batch the token of its first row.
struct AttnSeq {
  int b, qlen, klen, first;
  __device__ AttnSeq(const AttnArgs& a, int b_)
      : b(b_), qlen(seq_len(a.q_lens, b_, a.Lq)), klen(seq_len(a.k_lens, b_, a.Lk)), first(0) {}
  __device__ AttnSeq(const PackedArgs& a, int b_) : b(b_) {
    first = __builtin_amdgcn_readfirstlane(seq_len(a.offsets, b, a.Lq));
    qlen = __builtin_amdgcn_readfirstlane(min(max(seq_len(a.offsets, b + 1, a.Lq) - first, 0), a.most));
    klen = qlen;
  }
  __device__ AttnSeq(int b_, int qlen_, int klen_, int first_) : b(b_), qlen(qlen_), klen(klen_), first(first_) {}
  __device__ AttnSeq(const PagedArgs& a, int b_) : AttnSeq(static_cast<const PackedArgs&>(a), b_) {
    klen = __builtin_amdgcn_readfirstlane(seq_len(a.k_lens, b, a.Lk));
  }
  // bytes before the sequence's first row, or before its statistics of a head
  template <class A>
  __device__ __forceinline__ int64_t at(const A&, const AttnStride& s) const {
    if constexpr (A::LIE == Lie::PADDED) return b * s.b;
    else return first * s.l;
  }
  template <class A>
  __device__ __forceinline__ int64_t stat(const A& a, int h) const {
    if constexpr (A::LIE == Lie::PADDED) return ((int64_t)b * a.H + h) * a.Lq;
    else return (int64_t)h * a.Lq + first;
  }
};
template <class A>
__device__ __forceinline__ int64_t stats_of(const A& a) {  // statistics of all rows and heads
  return (int64_t)(A::LIE == Lie::PADDED ? a.B : 1) * a.H * a.Lq;
}

// The last of the numbers 0 .. n - 1 for which `upto` holds, which is true of
// none or of the first ones: 64 of them are tried at once.  -1: none.
template <class F>
__device__ __forceinline__ int find_last(int n, int lane, F&& upto) {
  int lo = 0;
  while (n > 0) {
    const int step = (n + WAVE - 1) / WAVE;
    const int i = lane * step;
    const int hits = (int)__popcll(__ballot(i < n && upto(lo + min(i, n - 1))));
    if (hits == 0) return lo - 1;
    lo += (hits - 1) * step;
    if (step == 1) return lo;
    n = min(step, n - (hits - 1) * step);
    lo += 1, n -= 1;  // the first of them is known
  }
  return lo - 1;
}

// The sequence (none: b < 0) and its tile of BM rows that workgroup `id` of a
// packed batch takes.  The host does not know the lengths: it numbers slots,
// of which sequence b has those from offsets[b] / BM + b on.  Rounded down,
// these leave room for its tiles and at most one more, and T / BM + B are
// enough for all.  Where rows have unequal work the long ones go first.  Of up
// to 63 sequences a wave holds all offsets: one trip to memory.
template <class A>
__device__ __forceinline__ AttnSeq find_tile(const A& a, int id, int BM, int lane, bool long_last, int& tile) {
  if (a.slots == 0) {
    tile = long_last ? id / a.B : a.tiles - 1 - id / a.B;
    return AttnSeq(a, id % a.B);
  }
  const int s = long_last ? id : a.slots - 1 - id;
  if (a.B < WAVE) {
    const int at = seq_len(a.offsets, min(lane, a.B), a.Lq);
    const int b = (int)__popcll(__ballot(lane < a.B && at / BM + lane <= s)) - 1;
    if (b < 0) return AttnSeq(b, 0, 0, 0);
    const int first = __builtin_amdgcn_readlane(at, b), rows = __builtin_amdgcn_readlane(at, b + 1) - first;
    tile = s - (first / BM + b);
    if (tile < 0) return AttnSeq(-1, 0, 0, 0);  // offsets that decrease
    const int qlen = min(max(rows, 0), a.most);
    if constexpr (A::LIE == Lie::PACKED) return AttnSeq(b, qlen, qlen, first);
    else return AttnSeq(b, qlen, __builtin_amdgcn_readfirstlane(seq_len(a.k_lens, b, a.Lk)), first);
  }
  auto slot = [&](int i) { return seq_len(a.offsets, i, a.Lq) / BM + i; };
  const int b = __builtin_amdgcn_readfirstlane(find_last(a.B, lane, [&](int i) { return slot(i) <= s; }));
  if (b < 0) return AttnSeq(b, 0, 0, 0);
  tile = __builtin_amdgcn_readfirstlane(s - slot(b));
  if (tile < 0) return AttnSeq(-1, 0, 0, 0);
  return AttnSeq(a, b);
}

// Clears rows of no sequence, those before the first and behind the last, and
// those of a sequence that are not looked at: part `part` of `parts`, by a
// workgroup.  x [heads, tokens, d], lse [heads, tokens]
// (null: none).
template <class A>
__device__ __forceinline__ void clear_rest(const A& a, char* x, const AttnStride& s, int heads, int bytes, float* lse,
                                           int part, int parts) {
  const int before = seq_len(a.offsets, 0, a.Lq), behind = max(before, seq_len(a.offsets, a.B, a.Lq));
  const int64_t rows = before + a.Lq - behind, per = bytes / 16;
  auto token = [&](int64_t r) { return r < before ? r : behind + (r - before); };
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; x && i < rows * heads * per; i += (int64_t)parts * blockDim.x) {
    const int64_t r = i / per / heads, h = i / per % heads;
    *reinterpret_cast<uint4*>(x + h * s.h + token(r) * s.l + i % per * 16) = zero4();
  }
  for (int64_t i = (int64_t)part * blockDim.x + threadIdx.x; lse && i < rows * heads; i += (int64_t)parts * blockDim.x)
    lse[i / rows * a.Lq + token(i % rows)] = 0.f;
  // Rows behind `most`: a wave looks at 64 sequences and clears such rows of one
  // after another; where that leaves waves over, several share them.  (A lane for
  // each sequence, one text of 32768 tokens of which 2048 are looked at, 32 heads
  // of 128: forward 341 ms.)
  if (a.most < a.Lq) {
    const int lane = threadIdx.x % WAVE, per_group = blockDim.x / WAVE, waves = parts * per_group;
    const int me = part * per_group + __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int sets = (a.B + WAVE - 1) / WAVE, share = max(1, waves / max(1, sets));
    for (int set = me / share; set < sets; set += waves / share) {
      const int b = set * WAVE + lane;
      const int first = b < a.B ? seq_len(a.offsets, b, a.Lq) + a.most : 0, end = b < a.B ? seq_len(a.offsets, b + 1, a.Lq) : 0;
      for (uint64_t some = __ballot(first < end); some; some &= some - 1) {
        const int n = __builtin_ctzll(some), from = __builtin_amdgcn_readlane(first, n);
        const int64_t rest = __builtin_amdgcn_readlane(end, n) - from, step = share * WAVE;
        for (int64_t i = me % share * WAVE + lane; x && i < rest * heads * per; i += step) {
          const int64_t r = i / per / heads, h = i / per % heads;
          *reinterpret_cast<uint4*>(x + h * s.h + (from + r) * s.l + i % per * 16) = zero4();
        }
        for (int64_t i = me % share * WAVE + lane; lse && i < rest * heads; i += step)
          lse[i / rest * a.Lq + from + i % rest] = 0.f;
      }
    }
  }
}

// Whether the row at position p sees key k + o, for a run of offsets o
struct Seen {
  int hi, lo, first;
  __device__ __forceinline__ Seen(int p, int k, int window, int sinks)
      : hi(p - k), lo(p - window - k), first(sinks - k) {}
  __device__ __forceinline__ bool operator()(int o) const { return (o <= hi) & ((o > lo) | (o < first)); }
};

// Two waves' parts of a sum, added into part 0's by way of LDS that the whole
// workgroup has done with
template <int RG>
__device__ __forceinline__ float add_parts(float* lds, int rg, int ks, int lane, float x) {
  __syncthreads();
  if (ks == 1) lds[rg * WAVE + lane] = x;
  __syncthreads();
  return ks == 0 ? x + lds[rg * WAVE + lane] : x;
}
template <int RG, int DB>
__device__ __forceinline__ void add_parts(float* lds, int rg, int ks, int lane, f32x16 (&x)[DB]) {
  float* to = lds + rg * DB * 16 * WAVE + lane;
  __syncthreads();
  if (ks == 1) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) to[(db * 16 + r) * WAVE] = x[db][r];
  }
  __syncthreads();
  if (ks == 0) {
#pragma unroll
    for (int db = 0; db < DB; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) x[db][r] += to[(db * 16 + r) * WAVE];
  }
}

// The key tiles of BN keys that rows at positions p_lo .. p_hi can see: the
// `ns` first ones for the sinks, then those from `tl` on for the window.
struct KeyTiles {
  int ns = 0, tl = 0, total = 0;
  __device__ KeyTiles(int p_lo, int p_hi, int window, int sinks, int BN) {
    if (p_hi < 0) return;
    ns = (min(sinks, p_hi + 1) + BN - 1) / BN;
    tl = max(ns, max(0, p_lo - window + 1) / BN);
    total = ns + max(0, p_hi / BN - tl + 1);
  }
  __device__ int at(int i) const { return i < ns ? i : tl + (i - ns); }
  // Indices lo .. hi - 1 of the tiles that all rows at p_lo .. p_hi see whole
  // (lo even: the ring's first place), none where `full` is not set
  __device__ void whole(int p_lo, int p_hi, int window, int BN, bool full, int& lo, int& hi) const {
    lo = min(ns, total), hi = full ? total : 0;
    while (lo < hi && at(lo) * BN <= p_hi - window) ++lo;
    lo += lo & 1;
    while (hi > lo && at(hi - 1) * BN + BN - 1 > p_lo) --hi;
    lo = min(lo, total);
  }
};

// Key splits of a row tile of the forward over pages: of about a chunk's tiles,
// no more than the host allowed.
__device__ __forceinline__ int key_splits(const PagedArgs& a, const KeyTiles& kt) {
  return max(1, min(a.splits, (kt.total + a.chunk / 2) / a.chunk));
}

// the lowest and highest position of a wave's rows
struct AttnWave {
  int lo, hi;
  // some row sees some of the keys k0 .. k1; every row sees all of them
  __device__ __forceinline__ bool some(int k0, int k1, int window, int sinks) const {
    return !(k0 > hi || (k1 <= lo - window && k0 >= sinks));
  }
  __device__ __forceinline__ bool whole(int k0, int k1, int window, int sinks) const {
    return k1 <= lo && (k0 > hi - window || k1 < sinks);
  }
};

// ------------------------------------------------------------------ non-finite tokens
// In the matrix products a masked probability is a zero, and a zero times a
// NaN or infinity of a token that the row does not see is a NaN.  A result
// that is not finite although its row's statistics are is therefore summed
// again, one key (or row) after another and only those that it sees, by its
// wave: lane l holds elements l and l + 64 of a head's row.  Finite inputs
// cost no more than the test of the results.
template <typename T>
struct Lane2 {
  float x[2];
  __device__ __forceinline__ Lane2(const char* row, int d, int lane) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = lane + 64 * j;
      x[j] = 0.f;
      if (c < d) {
        if constexpr (sizeof(T) == 4) x[j] = reinterpret_cast<const float*>(row)[c];
        else x[j] = bf2f(reinterpret_cast<const bf16_t*>(row)[c].x);
      }
    }
  }
  __device__ __forceinline__ float dot(const Lane2& o) const { return wave_sum(x[0] * o.x[0] + x[1] * o.x[1]); }
};
template <typename T>
__device__ __forceinline__ void store_lane2(char* row, const float (&x)[2], int d, int lane) {
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (lane + 64 * j < d) io_traits<T>::store(reinterpret_cast<T*>(row) + lane + 64 * j, x[j]);
}
__device__ __forceinline__ float of_lane(float x, int lane) { return __shfl(x, lane, WAVE); }
__device__ __forceinline__ int of_lane(int x, int lane) { return __shfl(x, lane, WAVE); }

// the columns (of 32) with a value that is not finite, as a mask
template <int DB>
__device__ __forceinline__ uint32_t not_finite(const f32x16 (&a)[DB]) {
  bool bad = false;
#pragma unroll
  for (int db = 0; db < DB; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) bad |= !__builtin_isfinite(a[db][r]);
  const uint64_t b = __ballot(bad);
  return (uint32_t)(b | (b >> 32));
}

// log2 of the sum l relative to m; where nothing was seen every weight is zero
__device__ __forceinline__ float log2_sum(float m, float l) {
  return l == 0.f ? __builtin_huge_valf() : m + log2f(l);
}

// a sum that is NaN in every column stays so
__device__ __forceinline__ bool settled(const float (&x)[2], int d, int lane) {
  return __all((lane >= d || x[0] != x[0]) && (lane + 64 >= d || x[1] != x[1]));
}

// sum of exp2(c q.k - m) v over the visible keys of tiles i0, i0 + di .. < i1.
// m is log2 of the row's whole sum, so that the weights add up to one and no
// value of the type's range leaves fp32 on the way: relative to the lagging
// maximum of the products (see AttnRows::follow) a sum of values from 2^104 on
// may have, which is one way to come here.
template <typename T, class Keys>
__device__ __forceinline__ void slow_o(float (&x)[2], const char* q, const Keys& keys, const AttnArgs& a, int p,
                                       float m, const KeyTiles& kt, int i0, int i1, int di, int bn, int lane) {
  const Lane2<T> qq(q, a.d, lane);
  x[0] = x[1] = 0.f;
#pragma unroll 1
  for (int i = i0; i < i1; i += di)
#pragma unroll 1
    for (int j = kt.at(i) * bn; j < kt.at(i) * bn + bn && j <= p; ++j) {
      if (j <= p - a.window && j >= a.sinks) continue;
      const float pr = __builtin_amdgcn_exp2f(fmaf(qq.dot(Lane2<T>(keys.k(j), a.d, lane)), a.c, -m));
      const Lane2<T> v(keys.v(j), a.d, lane);
#pragma unroll
      for (int e = 0; e < 2; ++e) x[e] = fmaf(pr, v.x[e], x[e]);
      if (settled(x, a.d, lane)) return;
    }
}

// ------------------------------------------------------------------ forward
// A wave's 32 rows: running maximum and sum, and O^T.
template <typename T, int DP>
struct AttnRows {
  static constexpr int STEPS = AttnTile<T, DP>::STEPS, DB = DP / 32;
  Frag<T> q[STEPS];
  f32x16 o[DB];
  float m, l;   // maximum (in units of log2, at most 24 behind), this lane's half of the sum
  float limit;  // the score at which m is 24 behind
  int p;        // position of lane l % 32's row
  AttnWave w;

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int db = 0; db < DB; ++db) o[db] = zero16();
    m = limit = -__builtin_huge_valf();
    l = 0.f;
  }

  // scores of the 32 keys from row `at` of a tile
  __device__ __forceinline__ f32x16 scores(const char* kt, int at, int lane, int d) const {
    f32x16 s = zero16();
    row_steps<T, STEPS>(d, [&](int t) { s = mma32(row_frag<T, DP>(kt, at, t, lane), q[t], s); });
    return s;
  }
  __device__ __forceinline__ void mask(f32x16& s, int k0, int window, int sinks, int lane) const {
    const Seen seen(p, k0 + 4 * (lane >> 5), window, sinks);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = seen(8 * (r >> 2) + (r & 3)) ? s[r] : -__builtin_huge_valf();
  }
  // The sums are taken relative to m, which may lag behind the largest score:
  // exp2 of up to 24 loses nothing in floating point.  A lane then looks only
  // whether one of its own scores is past `limit`; the row's maximum over both
  // of its lanes is formed, and everything rescaled, in the rare block where
  // one is.  `held`: probabilities that are not in o yet.
  __device__ __forceinline__ void follow(const f32x16& s, float c, f32x16* held) {
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    if (__any(top > limit)) {
      const float to = fmaxf(m, pair_max(top) * c);
      const float a = to == m ? 1.f : __builtin_amdgcn_exp2f(m - to);
      m = to;
      limit = (m + 24.f) / c;
      l *= a;
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[db][r] *= a;
      if (held) {
#pragma unroll
        for (int r = 0; r < 16; ++r) (*held)[r] *= a;
      }
    }
  }
  __device__ __forceinline__ void exps(f32x16& s, float c) {
    const float ref = m == -__builtin_huge_valf() ? 0.f : m;  // nothing seen yet: every term is exp2(-inf)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -ref));
      l += s[r];
    }
  }
  // 32 keys, in LDS tiles of as many rows
  __device__ __forceinline__ f32x16 weights(const char* kt, int k0, int window, int sinks, float c, int lane, int d) {
    f32x16 s = scores(kt, 0, lane, d);
    if (!w.whole(k0, k0 + 31, window, sinks)) mask(s, k0, window, sinks, lane);
    follow(s, c, nullptr);
    exps(s, c);
    return s;
  }
  __device__ __forceinline__ void step(const char* kt, const char* vt, int k0, int window, int sinks, float c,
                                       int lane, int d) {
    const f32x16 s = weights(kt, k0, window, sinks, c, lane, d);
    acc_trans<T, DP>(o, s, vt, 0, lane, d);
  }
  // 64 keys that every row sees.  Four runs of products: the scores of one
  // half and of the other, then each half's sums.  The exponentials of a half
  // go between the products of the run behind its own, a few after each, so
  // that one wave keeps matrix and vector pipe busy, and an operand is read
  // from LDS AHEAD products before its own.  The order is spelled out by the
  // scheduling barriers: left to itself the compiler reads an operand just
  // before its product, which then waits for LDS.
  __device__ __forceinline__ void step2(const AttnAddr<DP>& at, lds_ptr kt, lds_ptr vt, float c) {
    static_assert(sizeof(T) == 2, "bf16");
    constexpr int NM = STEPS, E = 16 / NM;  // products of a run; scores behind each
    auto frag = [&](int m) {
      const int run = m / NM, i = m % NM;
      return run < 2 ? at.rows(kt, 32 * run, i) : at.cols(vt, 32 * (run - 2) + 16 * (i / DB), i % DB);
    };
    bf16x8 f[AHEAD];
    auto next = [&](int m) {
      if (m + AHEAD < 4 * NM) f[m % AHEAD] = frag(m + AHEAD);
    };
#pragma unroll
    for (int m = 0; m < AHEAD; ++m) f[m] = frag(m);
    __builtin_amdgcn_sched_barrier(0);
    f32x16 s0 = zero16(), s1 = zero16();
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      s0 = mma32(f[i % AHEAD], q[i], s0);
      next(i);
      __builtin_amdgcn_sched_barrier(0);
    }
    follow(s0, c, nullptr);
    float ref = m == -__builtin_huge_valf() ? 0.f : m;
    auto some = [&](f32x16& s, int i) {
#pragma unroll
      for (int r = i * E; r < i * E + E; ++r) {
        s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], c, -ref));
        l += s[r];
      }
    };
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      s1 = mma32(f[(NM + i) % AHEAD], q[i], s1);
      next(NM + i);
      some(s0, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("" : "+v"(s0));  // the exponentials stay on this side of the branch
    follow(s1, c, &s0);
    ref = m == -__builtin_huge_valf() ? 0.f : m;
    const Pair p0 = round_pair(s0);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      o[i % DB] = mma32(f[(2 * NM + i) % AHEAD], p0.f[i / DB], o[i % DB]);
      next(2 * NM + i);
      some(s1, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    const Pair p1 = round_pair(s1);
#pragma unroll
    for (int i = 0; i < NM; ++i) {
      o[i % DB] = mma32(f[(3 * NM + i) % AHEAD], p1.f[i / DB], o[i % DB]);
      next(3 * NM + i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  // BN keys of which a row may see some or none; of KS waves' parts, part ks
  template <int BN, int KS>
  __device__ __forceinline__ void tile(const char* kt, const char* vt, int ks, int k0, int window, int sinks, float c,
                                       int lane, int d) {
#pragma unroll 1
    for (int i = 32 * ks; i < BN; i += 32 * KS)
      if (w.some(k0 + i, k0 + i + 31, window, sinks))
        step(kt + i * AttnTile<T, DP>::CPR * 16, vt + i * AttnTile<T, DP>::CPR * 16, k0 + i, window, sinks, c, lane, d);
  }
};

template <typename T>
__device__ __forceinline__ void store_row4(char* row, int d, const float (&v)[4]) {
  store4(reinterpret_cast<T*>(row) + d, v);
}

// O^T of a wave to memory: lane l holds row l % 32, 4 consecutive d at a time
template <typename T, int DP>
__device__ __forceinline__ void store_rows(const f32x16 (&o)[DP / 32], float f, char* row, int d, int lane) {
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int c = 32 * db + 8 * g + 4 * (lane >> 5);
      const float v[4] = {o[db][4 * g] * f, o[db][4 * g + 1] * f, o[db][4 * g + 2] * f, o[db][4 * g + 3] * f};
      if (c < d) store_row4<T>(row, c, v);
    }
}

// waves a SIMD: two where 256 registers hold a wave's 32 rows
template <typename T, int DP>
constexpr int attn_waves() { return DP * (int)sizeof(T) > 256 ? 1 : 2; }

// the backward keeps two operands and two sums of 32 rows or keys
template <typename T, int DP>
constexpr int attn_back_waves() { return DP * (int)sizeof(T) >= 256 ? 1 : 2; }

// keys of a tile: 16 KB of K and of V, or 64 keys
template <typename T, int DP>
constexpr int attn_bn() { return DP * (int)sizeof(T) > 256 ? 32 : 64; }

// Where a workgroup works: head and tile.  Query heads that share a key head
// come next to each other, then tiles, so that those reading the same keys
// run together, and (xcd_remap) mostly on one XCD with its L2.
//
// In a packed batch key heads are innermost instead, so that consecutive
// workgroups, which go to the XCDs in turn, put the same ones on an XCD and
// leave each with as many long tiles as the others.  Key splits are outermost:
// an XCD deals its workgroups to its shader engines in turn, too, and with
// every fourth split in use and three empty ones beside it, a quarter of them
// had all the work (eight chunks of 1024 rows among 20 sequences, two of eight
// splits in use: 2.1 ms innermost, 1.0 when all splits are).
struct AttnPlace {
  int b, hk, h, tile, split = 0;
  // of a packed batch: without the sequence (find_tile), whose number is left in b
  __device__ AttnPlace(int id, const PackedArgs& a) {
    const int groups = a.G / a.hg;
    if (a.splits > 1) {
      const int one = a.main / a.splits;
      split = id / one;
      id -= split * one;
    }
    hk = id % a.Hk;
    id /= a.Hk;
    h = hk * a.G + id % groups * a.hg;
    b = id / groups, tile = 0;
  }
  __device__ AttnPlace(int id, const AttnArgs& a) {
    id = xcd_remap(id, gridDim.x);
    const int groups = a.G / a.hg;
    h = id % groups * a.hg;
    id /= groups;
    tile = a.tiles - 1 - id % a.tiles;  // where rows have unequal work the long ones go first
    id /= a.tiles;
    hk = id % a.Hk;
    b = id / a.Hk;
    h += hk * a.G;
  }
};

template <class A>
__device__ __forceinline__ AttnSeq place_seq(const A& a, int BM, int lane, AttnPlace& at) {
  if constexpr (A::LIE == Lie::PADDED) return AttnSeq(a, at.b);
  else return find_tile(a, at.b, BM, lane, false, at.tile);
}

// Four waves x 32 rows; K and V tiles in a two-deep ring of direct loads: a
// tile's 32 KB serve 128 rows, and Q and O never leave the registers.
// KS = 2: two waves share 32 rows, each taking one half of every tile, and
// join at the end: for few rows, which 128 a workgroup would leave on half
// the chip or less.
//
// Bound by the matrix and vector pipes together: per 32 x 32 scores a wave has
// 4 d / 32 products of 32 cycles and, for each score, an fma, an exponential,
// an add to the sum, a share of the maximum and half a conversion, which the
// two waves of a SIMD overlap as far as they can.  32K prompt of 32 heads
// (8 key heads), d = 128, window 2048: 1.08 ms, 990 TFLOP/s, matrix pipes busy
// 55 % of the time; 16 heads, d = 64: 325 us, 820 TFLOP/s, 45 %; no LDS bank
// conflicts.  Packed: 8 prompts of 32768 tokens, causal, the same heads: 1.32 ms,
// 1.05 PFLOP/s; paged: 2048 rows over 32768 keys 1.02 ms, 1.05 PFLOP/s.  Tiles of 32 keys with three waves a SIMD took 1.47 ms for 1.17
// of these at the time: too few products between a tile's waits.
template <typename T, int DP, int KS, class A = AttnArgs>
__global__ __launch_bounds__(256, (attn_waves<T, DP>())) void attn_fwd_kernel(A a) {
  using Tile = AttnTile<T, DP>;
  constexpr bool PAGED = A::LIE == Lie::PAGED;
  constexpr int NW = 4, RG = NW / KS, BN = attn_bn<T, DP>(), TB = BN * Tile::CPR * 16;
  __shared__ __align__(1024) char lds[4 * TB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (A::LIE != Lie::PADDED)
    if ((int)blockIdx.x >= a.main)
      return clear_rest(a, a.out, a.so, a.H, a.d * (int)sizeof(T), a.lse, (int)blockIdx.x - a.main, a.rest);
  const int rg = wave % RG, ks = wave / RG;  // head and rows of the wave; its part of a tile
  const int BM = 32 * RG / a.hg;             // rows of the workgroup
  AttnPlace at(blockIdx.x, a);
  const AttnSeq seq = place_seq(a, BM, lane, at);
  if (A::LIE != Lie::PADDED && seq.b < 0) return;
  const int qlen = seq.qlen, klen = seq.klen;
  if constexpr (PAGED)
    if (qlen <= a.few) return;
  at.h += rg % a.hg;
  const int r0 = at.tile * BM, rw = r0 + 32 * (rg / a.hg), off = klen - qlen;
  if (r0 >= qlen) return;
  const int row = rw + (lane & 31), cmax = a.d * (int)sizeof(T) / 16 - 1;
  const char* qb = a.q + seq.at(a, a.sq) + at.h * a.sq.h;
  AttnRows<T, DP> w;
  w.clear();
  load_rows(w.q, qb + (int64_t)min(row, qlen - 1) * a.sq.l, cmax, lane);
  w.p = off + row;
  w.w = {off + rw, off + min(rw + 31, qlen - 1)};
  const KeyTiles kt(off + r0, off + min(r0 + BM, qlen) - 1, a.window, a.sinks, BN);
  const auto keys = [&] {
    if constexpr (PAGED) return PageRows<T, DP, BN, NW>(a, seq.b, at.hk, klen - 1, wave, lane);
    else return KeyRows<T, DP, BN, NW>(a.k + seq.at(a, a.sk) + at.hk * a.sk.h, a.sk.l, a.v + seq.at(a, a.sv) + at.hk * a.sv.h,
                                       a.sv.l, klen - 1, cmax, wave, lane);
  }();
  const AttnAddr<DP> addr(lane);
  // the workgroup's tiles: all, or a split's (from an even one on: the ring's first place)
  int i0 = 0, i1 = kt.total, splits = 1;
  if constexpr (PAGED) {
    splits = key_splits(a, kt);
    if (at.split >= splits) return;
    i0 = (int)((int64_t)i1 * at.split / splits) & ~1;
    if (at.split + 1 < splits) i1 = (int)((int64_t)i1 * (at.split + 1) / splits) & ~1;
  }
  // ring of two: tile i + 1 is copied while tile i is computed
  auto arrive = [&](int i, char* other) {
    wait_lgkm0();
    wait_vm<0>();
    bar();
    if (i + 1 < i1) keys.issue(other, kt.at(i + 1) * BN);
  };
  auto edge = [&](int i) {
    char* t = lds + (i & 1) * 2 * TB;
    arrive(i, lds + (2 - 2 * (i & 1)) * TB);
    if (w.w.lo <= w.w.hi) w.template tile<BN, KS>(t, t + TB, ks, kt.at(i) * BN, a.window, a.sinks, a.c, lane, a.d);
  };
  if (i0 < i1) keys.issue(lds, kt.at(i0) * BN);
  // Tiles that all rows of the workgroup see whole run in a loop of their own,
  // two a round: with nothing but straight code in it the sums stay in their
  // registers (with the edges' branches inside the loop the compiler copied
  // all 64 twice a tile).
  int i = i0;
  if constexpr (sizeof(T) == 2 && KS == 1) {
    int lo, hi;
    kt.whole(off + r0, off + min(r0 + BM, qlen) - 1, a.window, BN, r0 + BM <= qlen, lo, hi);
    if constexpr (PAGED) lo = min(lo, i1), hi = min(hi, i1);
    for (; i < lo; ++i) edge(i);
    for (; i + 1 < hi; i += 2) {
      arrive(i, lds + 2 * TB);
      w.step2(addr, (lds_ptr)lds, (lds_ptr)lds + TB, a.c);
      arrive(i + 1, lds);
      w.step2(addr, (lds_ptr)lds + 2 * TB, (lds_ptr)lds + 3 * TB, a.c);
    }
  }
#pragma unroll 1
  for (; i < i1; ++i) edge(i);
  float l = pair_sum(w.l);
  if constexpr (KS == 2) {
    static_assert(RG * (32 * DP + 64) * 4 <= 4 * TB, "the join's place");
    float* theirs = reinterpret_cast<float*>(lds) + rg * (32 * DP + 64);  // [d][row], maximum, sum
    __syncthreads();
    if (ks == 1) {
#pragma unroll
      for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) theirs[(16 * db + r) * 64 + lane] = w.o[db][r];
      if (lane < 32) {
        theirs[32 * DP + lane] = w.m;
        theirs[32 * DP + 32 + lane] = l;
      }
    }
    __syncthreads();
    if (ks == 1) return;
    const float m1 = theirs[32 * DP + (lane & 31)], l1 = theirs[32 * DP + 32 + (lane & 31)], m = fmaxf(w.m, m1);
    // a part that saw nothing adds nothing; one whose scores are all NaN has no maximum but a sum
    auto weight = [&](float x, float sum) {
      return sum == 0.f ? 0.f : x == -__builtin_huge_valf() ? 1.f : __builtin_amdgcn_exp2f(x - m);
    };
    const float f0 = weight(w.m, l), f1 = weight(m1, l1);
    l = (l == 0.f ? 0.f : l * f0) + (l1 == 0.f ? 0.f : l1 * f1);
    w.m = m;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const float x = theirs[(16 * db + r) * 64 + lane];
        w.o[db][r] = (f0 == 0.f ? 0.f : f0 * w.o[db][r]) + (f1 == 0.f ? 0.f : f1 * x);
      }
  }
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  char* out = a.out + seq.at(a, a.so) + at.h * a.so.h;
  // a split's result and statistics, by token, head and split
  auto part = [&](int r) { return (((int64_t)(seq.first + r) * a.H + at.h) * a.splits + at.split); };
  if (row < qlen) {
    if (PAGED && splits > 1) {
      store_rows<float, DP>(w.o, inv, reinterpret_cast<char*>(a.part + part(row) * a.d), a.d, lane);
      if (lane < 32) *reinterpret_cast<float2*>(a.part_ml + part(row) * 2) = make_float2(w.m, l);
    } else {
      store_rows<T, DP>(w.o, inv, out + row * a.so.l, a.d, lane);
      if (a.lse && lane < 32)
        a.lse[seq.stat(a, at.h) + row] = l == 0.f ? -__builtin_huge_valf() : w.m * LN2 + logf(l);
    }
  }
  for (uint32_t bad = not_finite(w.o) & (uint32_t)__ballot(row < qlen && l == l); bad; bad &= bad - 1) {
    const int n = __builtin_ctz(bad), r = rw + n;
    float x[2];
    slow_o<T>(x, qb + r * a.sq.l, keys, a, off + r, of_lane(log2_sum(w.m, l), n), kt, i0, i1, 1, BN, lane);
    if (PAGED && splits > 1) store_lane2<float>(reinterpret_cast<char*>(a.part + part(r) * a.d), x, a.d, lane);
    else store_lane2<T>(out + r * a.so.l, x, a.d, lane);
  }
}

// ------------------------------------------------------------------ forward, few rows
// waves of a workgroup, bytes of a tile of 32 keys, and the LDS of a workgroup:
// a wave's ring of two tiles of K and V, where its O^T and statistics fit later
template <typename T, int DP>
constexpr int few_waves() { return DP * (int)sizeof(T) > 256 ? 2 : 4; }
template <typename T, int DP>
constexpr int few_tile() { return 32 * AttnTile<T, DP>::CPR * 16; }
template <typename T, int DP>
constexpr int few_lds() {
  return few_waves<T, DP>() * (4 * few_tile<T, DP>() > 32 * DP * 4 + 256 ? 4 * few_tile<T, DP>() : 32 * DP * 4 + 256);
}

// Few rows a key head, 32 to a workgroup (row r is token r / G's query head r
// % G, so that a workgroup's rows see the same keys): the work is reading
// keys, so the keys are split, over workgroups and again over a workgroup's
// waves.  Bound by memory: next tokens of 96 sequences of up to 8192 keys,
// window 4096, 32 heads (8 key heads) of 128: 265 us, 5.6 TB/s of the 1.48 GB
// that it must read.  Where keys are few, by latency: one sequence of 16
// heads, window 2048: 8.7 us, and 3.0 more for the join.  Each wave runs its
// own ring of 32-key tiles with no barrier; the waves join in LDS, the
// workgroups through `part` in attn_join_kernel.
template <typename T, int DP>
__global__ __launch_bounds__(64 * (few_waves<T, DP>())) void attn_few_kernel(AttnArgs a) {
  using Tile = AttnTile<T, DP>;
  constexpr int NW = few_waves<T, DP>(), TB = few_tile<T, DP>(), WB = few_lds<T, DP>() / NW;
  __shared__ __align__(1024) char lds[few_lds<T, DP>()];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % a.splits, tile = blockIdx.x / a.splits % a.tiles, bk = blockIdx.x / a.splits / a.tiles;
  const int hk = bk % a.Hk, b = bk / a.Hk;
  const int qlen = seq_len(a.q_lens, b, a.Lq), klen = seq_len(a.k_lens, b, a.Lk);
  const int t0 = 32 * tile / a.G;  // the first row's token
  if (t0 >= qlen) return;
  const int off = klen - qlen, rows = a.G * a.Lq, n = lane & 31, at = 32 * tile + n;
  const int row = min(at, rows - 1), tok = row / a.G, cmax = a.d * (int)sizeof(T) / 16 - 1;
  const char* kb = a.k + b * a.sk.b + hk * a.sk.h;
  const char* vb = a.v + b * a.sv.b + hk * a.sv.h;
  AttnRows<T, DP> w;
  w.clear();
  load_rows(w.q, a.q + b * a.sq.b + (int64_t)(hk * a.G + row % a.G) * a.sq.h +
                            (int64_t)min(tok, qlen - 1) * a.sq.l, cmax, lane);
  w.p = off + min(tok, qlen - 1);
  w.w = {off + t0, off + min((32 * tile + 31) / a.G, qlen - 1)};
  const KeyTiles kt(w.w.lo, w.w.hi, a.window, a.sinks, 32);
  const int i0 = (int)((int64_t)kt.total * split / a.splits), i1 = (int)((int64_t)kt.total * (split + 1) / a.splits);
  char* ring = lds + wave * WB;
  auto issue = [&](int i, int buf) {
    char* t = ring + buf * 2 * TB;
    Tile::template stage<32, 1>(t, kb, a.sk.l, kt.at(i) * 32, klen - 1, cmax, 0, lane);
    Tile::template stage<32, 1>(t + TB, vb, a.sv.l, kt.at(i) * 32, klen - 1, cmax, 0, lane);
  };
  if (i0 + wave < i1) issue(i0 + wave, 0);
  int buf = 0;
  for (int i = i0 + wave; i < i1; i += NW, buf ^= 1) {
    wait_lgkm0();  // the tile that the next copies overwrite has been read
    if (i + NW < i1) {
      issue(i + NW, buf ^ 1);
      wait_vm<Tile::CPR>();  // the 2 x CPR / 2 copies of the tile before them have landed
    } else {
      wait_vm<0>();
    }
    asm volatile("" ::: "memory");
    const char* t = ring + buf * 2 * TB;
    w.template tile<32, 1>(t, t + TB, 0, kt.at(i) * 32, a.window, a.sinks, a.c, lane, a.d);
  }
  // join the waves: O as [d][row] and the statistics behind it
  wait_lgkm0();
  float* mine = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) mine[(32 * db + 8 * (r >> 2) + 4 * (lane >> 5) + (r & 3)) * 32 + n] = w.o[db][r];
  float lsum = pair_sum(w.l);
  uint32_t bad = not_finite(w.o) & (uint32_t)__ballot(lsum == lsum);
  if (((bad >> n) & 1) && lsum > 0.f) {  // such a row's part is summed again with weights that add up to one
    w.m = log2_sum(w.m, lsum);
    lsum = 1.f;
  }
  for (; bad; bad &= bad - 1) {
    const int i = __builtin_ctz(bad), r = of_lane(row, i), t = min(r / a.G, qlen - 1);
    float x[2];
    slow_o<T>(x, a.q + b * a.sq.b + (int64_t)(hk * a.G + r % a.G) * a.sq.h + t * a.sq.l, TokenRows{kb, vb, a.sk.l, a.sv.l}, a,
              off + t, of_lane(lsum == 0.f ? __builtin_huge_valf() : w.m, i), kt, i0 + wave, i1, NW, 32, lane);
    mine[lane * 32 + i] = x[0];
    if (lane + 64 < DP) mine[(lane + 64) * 32 + i] = x[1];
  }
  if (lane < 32) {
    mine[DP * 32 + n] = w.m;
    mine[DP * 32 + 32 + n] = lsum;
  }
  __syncthreads();
  auto other = [&](int v) { return reinterpret_cast<const float*>(lds + v * WB); };
  float m = -__builtin_huge_valf(), l = 0.f, f[NW];
#pragma unroll
  for (int v = 0; v < NW; ++v) m = fmaxf(m, other(v)[DP * 32 + n]);
#pragma unroll
  for (int v = 0; v < NW; ++v) {
    const float x = other(v)[DP * 32 + n];
    f[v] = x == -__builtin_huge_valf() ? 0.f : __builtin_amdgcn_exp2f(x - m);
    // a wave that met a NaN has a NaN sum whatever its maximum
    l += other(v)[DP * 32 + 32 + n] == 0.f ? 0.f : other(v)[DP * 32 + 32 + n] * (f[v] == 0.f && x == -__builtin_huge_valf() ? 1.f : f[v]);
  }
  if (at >= rows || tok >= qlen) return;
  constexpr int PER = DP / (2 * NW);  // columns of a thread
  const int c0 = (int)(threadIdx.x >> 5) * PER;
  float* pr = a.part + (((int64_t)bk * rows + at) * a.splits + split) * a.d;
  char* orow = a.out + b * a.so.b + (int64_t)(hk * a.G + row % a.G) * a.so.h + (int64_t)tok * a.so.l;
  // The waves' parts are divided by the sum before they are added, and a split
  // leaves its part so: no larger than the largest value.
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
  for (int v = 0; v < NW; ++v) f[v] *= inv;
#pragma unroll
  for (int j = 0; j < PER; j += 4) {
    if (c0 + j >= a.d) break;
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = l == l ? 0.f : l;
#pragma unroll
      for (int v = 0; v < NW; ++v) x[e] += f[v] == 0.f ? 0.f : f[v] * other(v)[(c0 + j + e) * 32 + n];
    }
    if (a.splits > 1) store4(pr + c0 + j, x);
    else store_row4<T>(orow, c0 + j, x);
  }
  if (threadIdx.x < 32) {
    if (a.splits > 1) {
      float* ml = a.part_ml + (((int64_t)bk * rows + at) * a.splits + split) * 2;
      ml[0] = m;
      ml[1] = l;
    } else if (a.lse) {
      a.lse[((int64_t)b * a.H + hk * a.G + row % a.G) * a.Lq + tok] =
          l == 0.f ? -__builtin_huge_valf() : m * LN2 + logf(l);
    }
  }
}

// One workgroup a row: the splits' results, weighted by their sums relative to
// the common maximum.
// All loads of a thread are independent: the kernel is as long as two trips
// to memory.
template <typename T, int DP>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs a) {
  constexpr int PARTS = 256 / DP;  // threads that share a column
  __shared__ float f[256], red[4], out[PARTS][DP];
  const int rows = a.G * a.Lq, n = blockIdx.x % rows, bk = blockIdx.x / rows, t = threadIdx.x;
  const int hk = bk % a.Hk, b = bk / a.Hk, tok = n / a.G, h = hk * a.G + n % a.G;
  if (tok >= seq_len(a.q_lens, b, a.Lq)) return;
  const float* ml = a.part_ml + ((int64_t)bk * rows + n) * a.splits * 2;
  const float* pr = a.part + ((int64_t)bk * rows + n) * a.splits * a.d;
  constexpr float NONE = -__builtin_huge_valf();
  const float ms = t < a.splits ? ml[2 * t] : NONE, ls = t < a.splits ? ml[2 * t + 1] : 0.f;
  float m = ms;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, WAVE));
  if (t % WAVE == 0) red[t / WAVE] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  // a split without keys counts for nothing; one whose scores are all NaN has no maximum but a sum
  const float w = ls == 0.f ? 0.f : ms == NONE ? ls : ls * __builtin_amdgcn_exp2f(ms - m);
  f[t] = w;
  const float s = wave_sum(w);
  __syncthreads();
  if (t % WAVE == 0) red[t / WAVE] = s;
  __syncthreads();
  const float l = (red[0] + red[1]) + (red[2] + red[3]), inv = l > 0.f || l != l ? 1.f / l : 0.f;
  const int c = t % DP, part = t / DP;
  float x = 0.f;
  if (c < a.d)
#pragma unroll 8
    for (int i = part; i < a.splits; i += PARTS) {
      const float v = pr[(int64_t)i * a.d + c];
      x += f[i] == 0.f ? 0.f : f[i] * inv * v;
    }
  out[part][c] = x;
  __syncthreads();
  if (part == 0 && c < a.d) {
#pragma unroll
    for (int i = 1; i < PARTS; ++i) x += out[i][c];
    io_traits<T>::store(reinterpret_cast<T*>(a.out + b * a.so.b + (int64_t)h * a.so.h + (int64_t)tok * a.so.l) + c, x);
  }
  if (a.lse && t == 0) a.lse[((int64_t)b * a.H + h) * a.Lq + tok] = l == 0.f ? NONE : m * LN2 + logf(l);
}

// The same for the forward's key splits over pages, four heads of a token a
// wave: what it looks up serves all, and their loads are in flight together (36
// next tokens and 4 chunks of 512 rows, 32 heads of 128: a head a wave 31.6 us,
// so 21.9).
constexpr int JOIN_HEADS = 4;
template <typename T, int DP>
__global__ __launch_bounds__(256) void split_join_kernel(PagedArgs a) {
  constexpr float NONE = -__builtin_huge_valf();
  constexpr int BN = attn_bn<T, DP>(), N = JOIN_HEADS;
  const int lane = threadIdx.x % WAVE, c = 2 * lane, quads = (a.H + N - 1) / N, BM = 128 / a.hg;
  const int64_t id = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
  const int h0 = (int)(id % quads) * N, token = (int)(id / quads);
  if (token >= a.Lq) return;
  const int b = __builtin_amdgcn_readfirstlane(find_last(a.B, lane, [&](int i) { return seq_len(a.offsets, i, a.Lq) <= token; }));
  if (b < 0) return;
  const AttnSeq seq(a, b);
  const int row = token - seq.first, r0 = row / BM * BM, off = seq.klen - seq.qlen;
  if (seq.qlen <= a.few || row < 0 || row >= seq.qlen) return;
  const int splits = key_splits(a, KeyTiles(off + r0, off + min(r0 + BM, seq.qlen) - 1, a.window, a.sinks, BN));
  if (splits == 1) return;
  // a head behind the last is the last again: the same is stored twice
  auto place = [&](int i) { return ((int64_t)token * a.H + min(h0 + i, a.H - 1)) * a.splits; };
  float2 s[N];
#pragma unroll
  for (int i = 0; i < N; ++i) s[i] = lane < splits ? *reinterpret_cast<const float2*>(a.part_ml + (place(i) + lane) * 2) : make_float2(NONE, 0.f);
  float f[N], m[N], l[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = s[i].x;
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m[i] = fmaxf(m[i], __shfl_xor(m[i], o, WAVE));
    // a split without keys counts for nothing; one whose scores are all NaN has no maximum but a sum
    f[i] = s[i].y == 0.f ? 0.f : s[i].x == NONE ? s[i].y : s[i].y * __builtin_amdgcn_exp2f(s[i].x - m[i]);
    l[i] = wave_sum(f[i]);
    f[i] *= l[i] > 0.f || l[i] != l[i] ? 1.f / l[i] : 0.f;
  }
  float2 x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = make_float2(0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < splits; ++k) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float g = of_lane(f[i], k);
      float2 v = make_float2(0.f, 0.f);
      if (c < a.d) v = *reinterpret_cast<const float2*>(a.part + (place(i) + k) * a.d + c);
      x[i].x += g == 0.f ? 0.f : g * v.x;
      x[i].y += g == 0.f ? 0.f : g * v.y;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = min(h0 + i, a.H - 1);
    T* out = reinterpret_cast<T*>(a.out + seq.at(a, a.so) + (int64_t)h * a.so.h + (int64_t)row * a.so.l);
    if (c < a.d) io_traits<T>::store(out + c, x[i].x), io_traits<T>::store(out + c + 1, x[i].y);
    if (a.lse && lane == 0) a.lse[seq.stat(a, h) + row] = l[i] == 0.f ? NONE : m[i] * LN2 + logf(l[i]);
  }
}

// ------------------------------------------------------------------ pages, few rows
// Next tokens over pages.  The work is reading keys, of sequences whose lengths
// only the device knows: all tiles of 32 keys that some sequence's rows see,
// one after another -- by sequence, 32 of its rows (ordered by token, as in
// attn_few_kernel) and key head, an item -- are dealt to the launch's waves in
// equal runs.  Each wave goes along its run alone, with its own tiles and no
// barrier: while one begins an item the others read on.  An item that lies in
// one run is finished there; of others each wave leaves its part (at most two
// a wave: its first and its last), which stream_join_kernel adds up.
//
// Bound by memory: 96 requests of 2.1K to 8.2K keys, 32 (8) heads of 128: 367 us,
// 5.5 TB/s of the 2.03 GB (a workgroup for each key head, by attn_few_kernel's
// scheme: 456, two splits of the keys 435 and more of them longer: a workgroup's
// beginning and end took 5 us in which its compute unit read nothing).  Where keys
// are few, by latency: 16 heads of 64, window 2048: 9.9 us, and 4.0 the join.
constexpr int STREAM_SCAN = 256;  // sequences whose work a workgroup sums itself

// The rows of a sequence in tiles of 32, and the units of each, at least one:
// an item that sees no key is written too.
struct StreamItem {
  KeyTiles kt;
  int rtiles, units;
  __device__ __forceinline__ StreamItem(const PagedArgs& a, const AttnSeq& s)
      : kt(s.klen - s.qlen, s.klen - 1, a.window, a.sinks, 32), rtiles(s.qlen > a.few ? 0 : (a.G * s.qlen + 31) / 32),
        units(a.unit == 1 ? max(1, kt.total) : max(1, (kt.total + a.unit - 1) / a.unit)) {}
};
// The sequences that a workgroup has summed the work of
struct StreamScan {
  int upto[STREAM_SCAN + 1], first[STREAM_SCAN], qlen[STREAM_SCAN], klen[STREAM_SCAN];
};
// upto[i]: work of the sequences before i, for i = 0 .. B, by a workgroup of NT threads
template <int NT>
__device__ __forceinline__ void stream_scan(const PagedArgs& a, int* upto, StreamScan* keep) {
  __shared__ int sums[NT / WAVE];
  const int lane = threadIdx.x % WAVE, wave = threadIdx.x / WAVE;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += NT) {
    const int b = b0 + threadIdx.x;
    int x = 0;
    if (b < a.B) {
      const int first = seq_len(a.offsets, b, a.Lq);
      const AttnSeq s(b, min(max(seq_len(a.offsets, b + 1, a.Lq) - first, 0), a.most), seq_len(a.k_lens, b, a.Lk), first);
      const StreamItem it(a, s);
      x = stream_work(it.rtiles, it.units, a.Hk);
      if (keep) keep->first[b] = first, keep->qlen[b] = s.qlen, keep->klen[b] = s.klen;
    }
    for (int o = 1; o < WAVE && o < a.B; o *= 2) {
      const int y = __shfl_up(x, o, WAVE);
      if (lane >= o) x = stream_add(x, y);
    }
    if (b0) __syncthreads();
    if (lane == WAVE - 1) sums[wave] = x;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT / WAVE; ++i)
      if (i < wave) x = stream_add(x, sums[i]);
    if (b < a.B) upto[b + 1] = stream_add(before, x);
#pragma unroll
    for (int i = 0; i < NT / WAVE; ++i) before = stream_add(before, sums[i]);
  }
  if (threadIdx.x == 0) upto[0] = 0;
  __syncthreads();
}
__global__ __launch_bounds__(1024) void stream_plan_kernel(PagedArgs a) { stream_scan<1024>(a, a.upto, nullptr); }

// An item that lies in several runs, noted by the wave of the second of them
// (parts = 0: none begins so): its first row's place, rows and heads, and where
// its first part is.
struct StreamJoin {
  int first, row, rows, head;  // the sequence's first token; rows row .. row + rows - 1, ordered by token; first head
  int part, parts;             // of parts part, part + 2 (or + 1, see below), + 4 ..
};

// A wave keeps one tile of K and one of V: the next K is on its way from the
// scores on, the next V from the sums on, so that each has the other's half of
// the work to land in, and twice as many waves find room as with rings of two
// tiles (fp32, the same requests: 1.94 ms with rings, 1.01 so, 4.0 TB/s; heads of
// 64 580 and 413 us; bf16, one request of 16 heads of 64: 16.4 and 15.5 us with
// the join).  bf16 tiles of 128, whose work is short beside their way, have the
// ring (386 us and 402; one request of 32768 keys 40 and 46).
constexpr int STREAM_GROUP = 4;  // waves of a workgroup
template <typename T, int DP>
constexpr bool stream_ring() { return sizeof(T) == 2 && DP > 64; }
// Workgroups of a compute unit: what its LDS holds, except for bf16 heads of up
// to 64, of which it would hold four and two are fastest.  Two, three, four of
// them, us with the join: 96 requests of 2.1K to 8.2K keys, 32 (8) heads of 64, 219,
// 233, 231; 400 of 1000 keys 144, 150, 159; 8 of 4000 keys 24.5, 25.7, 27.8; one of
// 32768 keys 37.7, 39.8, 45.4, with window 2048 15.4, 15.5, 16.0; 32 requests of 16
// heads with that window 64.8, 63.2, 67.2.
template <typename T, int DP>
constexpr int stream_groups() { return DP <= 64 ? 2 : 1; }
template <typename T, int DP>
__global__ __launch_bounds__(64 * STREAM_GROUP, (stream_groups<T, DP>())) void stream_kernel(PagedArgs a) {
  using Tile = AttnTile<T, DP>;
  constexpr bool RING = stream_ring<T, DP>();
  constexpr int NW = STREAM_GROUP, TB = few_tile<T, DP>(), WB = (RING ? 4 : 2) * TB;
  static_assert(NW * WB * stream_groups<T, DP>() <= 128 * 1024, "LDS of the workgroups of a compute unit");
  __shared__ __align__(1024) char lds[NW * WB];
  __shared__ StreamScan scan;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31;
  if ((int)blockIdx.x >= a.main)
    return clear_rest(a, a.out, a.so, a.H, a.d * (int)sizeof(T), a.lse, (int)blockIdx.x - a.main, a.rest);
  if (!a.upto) stream_scan<64 * NW>(a, scan.upto, &scan);
  const int* upto = a.upto ? a.upto : scan.upto;
  const int work = __builtin_amdgcn_readfirstlane(upto[a.B]), run = stream_run(work, a.waves, a.share);
  const int me = blockIdx.x * NW + wave, cmax = a.d * (int)sizeof(T) / 16 - 1;
  const int t0 = min(work, me * run), t1 = min(work, t0 + run);
  char *const kt_lds = lds + wave * WB, *const vt_lds = kt_lds + TB;
  StreamJoin join = {0, 0, 0, 0, 0, 0};
#pragma unroll 1
  for (int t = t0; t < t1;) {
    const int b = __builtin_amdgcn_readfirstlane(find_last(a.B, lane, [&](int i) { return upto[i] <= t; }));
    auto of = [&](const int(&x)[STREAM_SCAN]) { return __builtin_amdgcn_readfirstlane(x[b]); };
    const AttnSeq seq = a.upto ? AttnSeq(a, b) : AttnSeq(b, of(scan.qlen), of(scan.klen), of(scan.first));
    const int qlen = seq.qlen, klen = seq.klen, off = klen - qlen;
    const StreamItem it(a, seq);
    const KeyTiles& kt = it.kt;
    const StreamTake take(t, t1, __builtin_amdgcn_readfirstlane(upto[b]), it.units);
    const int u0 = take.u0, u1 = take.u1, hk = take.item % a.Hk, r0 = 32 * (take.item / a.Hk);
    const int i0 = u0 * a.unit, i1 = min(kt.total, u1 * a.unit);
    const int rows = a.G * qlen, row = min(r0 + n, rows - 1), tok = row / a.G, h = hk * a.G + row % a.G;
    const char* qb = a.q + seq.at(a, a.sq);
    AttnRows<T, DP> w;
    w.clear();
    const PageRows<T, DP, 32, 1> keys(a, b, hk, klen - 1, 0, lane);
    wait_lgkm0();  // the item before has been read
    if (i0 < i1) keys.issue(kt_lds, vt_lds, kt.at(i0) * 32);
    load_rows(w.q, qb + (int64_t)h * a.sq.h + (int64_t)tok * a.sq.l, cmax, lane);
    w.p = off + tok;
    w.w = {off + r0 / a.G, off + min(r0 + 31, rows - 1) / a.G};
    // a copy of 32 rows is CPR / 2 instructions of a wave
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      const int k0 = kt.at(i) * 32;
      if constexpr (RING) {
        const int at = ((i - i0) & 1) * 2 * TB;
        wait_lgkm0();  // the tile that the next copies overwrite has been read
        if (i + 1 < i1) {
          char* next = kt_lds + 2 * TB - at;
          keys.issue(next, next + TB, kt.at(i + 1) * 32);
          wait_vm<Tile::CPR>();
        } else {
          wait_vm<0>();
        }
        asm volatile("" ::: "memory");
        w.template tile<32, 1>(kt_lds + at, vt_lds + at, 0, k0, a.window, a.sinks, a.c, lane, a.d);
        continue;
      }
      const bool some = w.w.some(k0, k0 + 31, a.window, a.sinks), more = i + 1 < i1;
      if (i == i0) wait_vm<0>();
      else wait_vm<Tile::CPR / 2>();  // K is here, V may not be
      asm volatile("" ::: "memory");
      f32x16 p = zero16();
      if (some) p = w.weights(kt_lds, k0, a.window, a.sinks, a.c, lane, a.d);
      wait_lgkm0();  // K has been read
      if (more) {
        keys.issue(kt_lds, nullptr, kt.at(i + 1) * 32);
        wait_vm<Tile::CPR / 2>();
      } else {
        wait_vm<0>();
      }
      asm volatile("" ::: "memory");
      if (some) acc_trans<T, DP>(w.o, p, vt_lds, 0, lane, a.d);
      wait_lgkm0();  // V has been read
      if (more) keys.issue(nullptr, vt_lds, kt.at(i + 1) * 32);
    }
    const bool whole = u0 == 0 && u1 == it.units;
    const float l = pair_sum(w.l), inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int64_t part = (int64_t)(2 * me + (t == t0 ? 0 : 1)) * a.rows;
    char* out = a.out + seq.at(a, a.so) + (int64_t)h * a.so.h + (int64_t)tok * a.so.l;
    if (r0 + n < rows) {
      if (whole) {
        store_rows<T, DP>(w.o, inv, out, a.d, lane);
        if (a.lse && lane < 32) a.lse[seq.stat(a, h) + tok] = l == 0.f ? -__builtin_huge_valf() : w.m * LN2 + logf(l);
      } else {
        store_rows<float, DP>(w.o, inv, reinterpret_cast<char*>(a.part + (part + n) * a.d), a.d, lane);
        if (lane < 32) *reinterpret_cast<float2*>(a.part_ml + (part + n) * 2) = make_float2(w.m, l);
      }
    }
    for (uint32_t bad = not_finite(w.o) & (uint32_t)__ballot(r0 + n < rows && l == l); bad; bad &= bad - 1) {
      const int i = __builtin_ctz(bad), r = r0 + i;
      float x[2];
      slow_o<T>(x, qb + (int64_t)(hk * a.G + r % a.G) * a.sq.h + (int64_t)(r / a.G) * a.sq.l, keys, a, off + r / a.G,
                of_lane(log2_sum(w.m, l), i), kt, i0, i1, 1, 32, lane);
      if (whole) store_lane2<T>(a.out + seq.at(a, a.so) + (int64_t)(hk * a.G + r % a.G) * a.so.h + (int64_t)(r / a.G) * a.so.l, x, a.d, lane);
      else store_lane2<float>(reinterpret_cast<char*>(a.part + (part + i) * a.d), x, a.d, lane);
    }
    const StreamParts p(me, u0, it.units, run, work - t);
    if (t == t0 && p.begins) join = {seq.first, r0, min(32, rows - r0), hk * a.G, p.part, p.parts};
    t += u1 - u0;
  }
  if (lane == 0) a.joins[me] = join;
}

// Items that lie in several runs: the parts, weighted by their sums relative to
// the common maximum.  Workgroup (w, y) takes rows y, y + 4 .. of the item that
// wave w + 1 noted; its waves share a row's parts.  Its length is that of its
// trips to memory: the note, the statistics, 16 parts at a time of each wave.
constexpr int JOIN_ROWS = 4;
template <typename T>
__global__ __launch_bounds__(256) void stream_join_kernel(PagedArgs a) {
  constexpr float NONE = -__builtin_huge_valf();
  __shared__ float2 other[4][WAVE];
  const StreamJoin j = a.joins[blockIdx.x + 1];
  const int lane = threadIdx.x % WAVE, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE), c = 2 * lane;
  for (int n = blockIdx.y; j.parts > 0 && n < j.rows; n += JOIN_ROWS) {
    // all parts but the first are the first ones of their waves
    auto place = [&](int i) { return (int64_t)(i == 0 ? j.part : (j.part & ~1) + 2 * i) * a.rows + n; };
    auto stat = [&](int i) { return i < j.parts ? *reinterpret_cast<const float2*>(a.part_ml + place(i) * 2) : make_float2(NONE, 0.f); };
    // a part without keys counts for nothing; one whose scores are all NaN has no maximum but a sum
    auto weight = [&](float2 x, float m) { return x.y == 0.f ? 0.f : x.x == NONE ? x.y : x.y * __builtin_amdgcn_exp2f(x.x - m); };
    const float2 head = stat(lane);
    float m = head.x;
    for (int i = lane + WAVE; i < j.parts; i += WAVE) m = fmaxf(m, stat(i).x);
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, WAVE));
    float l = weight(head, m);
    for (int i = lane + WAVE; i < j.parts; i += WAVE) l += weight(stat(i), m);
    l = wave_sum(l);
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    float2 x = make_float2(0.f, 0.f);
    for (int i0 = 0; i0 < j.parts; i0 += WAVE) {
      const float f = weight(i0 == 0 ? head : stat(i0 + lane), m) * inv;
      const int most = min(WAVE, j.parts - i0);
#pragma unroll
      for (int k = 0; k < WAVE / 4; ++k) {  // a wave's 16 of 64 parts: all loads before the first is waited for
        const int i = 4 * k + wave;
        const float g = of_lane(f, i);
        float2 v = make_float2(0.f, 0.f);
        if (i < most && c < a.d) v = *reinterpret_cast<const float2*>(a.part + place(i0 + i) * a.d + c);
        x.x += g == 0.f ? 0.f : g * v.x;
        x.y += g == 0.f ? 0.f : g * v.y;
      }
    }
    __syncthreads();
    other[wave][lane] = x;
    __syncthreads();
    if (wave != 0) continue;
#pragma unroll
    for (int i = 1; i < 4; ++i) x.x += other[i][lane].x, x.y += other[i][lane].y;
    const int tok = (j.row + n) / a.G, h = j.head + (j.row + n) % a.G;
    T* out = reinterpret_cast<T*>(a.out + (int64_t)h * a.so.h + (int64_t)(j.first + tok) * a.so.l);
    if (c < a.d) io_traits<T>::store(out + c, x.x), io_traits<T>::store(out + c + 1, x.y);
    if (a.lse && lane == 0) a.lse[(int64_t)h * a.Lq + j.first + tok] = l == 0.f ? NONE : m * LN2 + logf(l);
  }
}

// ------------------------------------------------------------------ backward: dq
// As the forward, with dP^T = V dO^T beside S^T and dq^T += K^T dS^T.  Lane n
// holds half of its row's dO and o: D = dO.o costs no launch of its own.
//
// bf16: a row's dS sum to zero, sum_j P (dO.v - D) = 0, so that any vector may
// be taken off all keys.  With the rounded dS, and D from a rounded o, they
// do not, and what is left meets the keys' common part, which is larger than
// their spread where a few keys take much of every row.  The kernel takes off
// the row's mean key: with R the sum of the rounded dS,
//   dq = scale (sum_j dS_j k_j - R sum_j P_j k_j),
// for one more product that reads no operand anew; and D + sum_j dS_j, the
// unrounded sum, is the exact D, which is left in `stats` for the dk, dv
// kernel.  Relative error of dq against fp64 where first tokens draw
// attention: 2.2e-3 for 2.8e-3 to 3.8e-3 without (1.7e-3 is the result's own
// rounding).
//
// 32K step of 16 heads, d = 64, window 2048: 585 us, matrix pipes busy 50 % of
// the time with the four products of a score (three are dq's own, one is the
// mean key's); the rest is the vector pipe's share, as in the forward.
template <typename T, int DP, int KS, class A = AttnArgs>
__global__ __launch_bounds__(256, (attn_back_waves<T, DP>())) void attn_dq_kernel(A a) {
  using Tile = AttnTile<T, DP>;
  constexpr int NW = 4, RG = NW / KS, BN = attn_bn<T, DP>(), TB = BN * Tile::CPR * 16, STEPS = Tile::STEPS, DB = DP / 32;
  constexpr bool CENTRE = sizeof(T) == 2;
  __shared__ __align__(1024) char lds[4 * TB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if constexpr (A::LIE != Lie::PADDED)
    if ((int)blockIdx.x >= a.main)
      return clear_rest(a, a.dq, a.sdq, a.H, a.d * (int)sizeof(T), nullptr, (int)blockIdx.x - a.main, a.rest);
  const int rg = wave % RG, ks = wave / RG;  // head and rows of the wave; its part of a tile
  const int BM = 32 * RG / a.hg;             // rows of the workgroup
  AttnPlace at(blockIdx.x, a);
  const AttnSeq seq = place_seq(a, BM, lane, at);
  if (A::LIE != Lie::PADDED && seq.b < 0) return;
  const int qlen = seq.qlen, klen = seq.klen;
  at.h += rg % a.hg;
  const int r0 = at.tile * BM, rw = r0 + 32 * (rg / a.hg), off = klen - qlen, n = lane & 31;
  const int row = rw + n, cmax = a.d * (int)sizeof(T) / 16 - 1;
  const int64_t stat = seq.stat(a, at.h) + row;
  if (A::LIE != Lie::PADDED && r0 >= qlen) return;
  f32x16 dq[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) dq[db] = zero16();
  const char* kb = a.k + seq.at(a, a.sk) + at.hk * a.sk.h;
  const char* vb = a.v + seq.at(a, a.sv) + at.hk * a.sv.h;
  const char* qb = a.q + seq.at(a, a.sq) + at.h * a.sq.h;
  const char* gb = a.dO + seq.at(a, a.sdo) + at.h * a.sdo.h;
  float delta = 0.f, lse = 0.f, lse2 = 0.f;
  const KeyTiles kt(off + r0, off + min(r0 + BM, qlen) - 1, a.window, a.sinks, BN);
  if (r0 < qlen) {
    const int64_t rc = min(row, qlen - 1);
    Frag<T> q[STEPS], g[STEPS];
    {
      Frag<T> o[STEPS];
      load_rows(q, qb + rc * a.sq.l, cmax, lane);
      load_rows(g, gb + rc * a.sdo.l, cmax, lane);
      load_rows(o, a.o + seq.at(a, a.so) + at.h * a.so.h + rc * a.so.l, cmax, lane);
#pragma unroll
      for (int s = 0; s < STEPS; ++s)
#pragma unroll
        for (int e = 0; e < 16 / (int)sizeof(T); ++e) delta = fmaf((float)g[s][e], (float)o[s][e], delta);
    }
    delta = pair_sum(delta);
    lse = row < qlen ? a.lse[stat] : 0.f;
    lse2 = lse * LOG2E;
    f32x16 less;  // -D: what dP's product starts from (bf16)
#pragma unroll
    for (int r = 0; r < 16; ++r) less[r] = sizeof(T) == 4 ? 0.f : -delta;
    float sum = 0.f, rsum = 0.f;  // of dS, exact and rounded
    f32x16 kbar[CENTRE ? DB : 1];
#pragma unroll
    for (auto& x : kbar) x = zero16();
    const int p = off + row;
    const AttnWave w{off + rw, off + min(rw + 31, qlen - 1)};
    const Stager<T, DP, BN, NW> sk(kb, a.sk.l, klen - 1, cmax, wave, lane), sv(vb, a.sv.l, klen - 1, cmax, wave, lane);
    auto arrive = [&](int i, char* other) {
      wait_lgkm0();
      wait_vm<0>();
      bar();
      if (i + 1 < kt.total) {
        sk.issue(other, kt.at(i + 1) * BN);
        sv.issue(other + TB, kt.at(i + 1) * BN);
      }
    };
    // Scores and dP - D to P and dS.  fp32: the exponent is formed in one
    // rounding, log2(e) multiplied last, and D subtracted last: scale log2(e)
    // and lse log2(e) rounded beforehand are a tenth of dk's error budget each.
    auto gradients = [&](f32x16& s, f32x16& ds) {
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if constexpr (sizeof(T) == 4) {
          s[r] = __builtin_amdgcn_exp2f(LOG2E * fmaf(s[r], a.scale, -lse));
          ds[r] = (ds[r] - delta) * s[r];
        } else {
          s[r] = __builtin_amdgcn_exp2f(fmaf(s[r], a.c, -lse2));
          ds[r] *= s[r];
        }
      }
    };
    auto count = [&](const f32x16& ds, const Pair& x) {
#pragma unroll
      for (int r = 0; r < 16; ++r) sum += ds[r];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint4 w = __builtin_bit_cast(uint4, x.f[e]);
        rsum = pair_add(w.x, pair_add(w.y, pair_add(w.z, pair_add(w.w, rsum))));
      }
    };
    if (kt.total > 0) {
      sk.issue(lds, kt.at(0) * BN);
      sv.issue(lds + TB, kt.at(0) * BN);
    }
    int i = 0;
    if constexpr (CENTRE && BN == 64 && KS == 1) {
      const AttnAddr<DP> addr(lane);
      // 64 keys that every row sees, as in AttnRows::step2: runs of scores and
      // dP of one half and the other, then of each half's sums, each of whose
      // operands serves two products
      auto pair = [&](lds_ptr kp, lds_ptr vp, auto masked, int k0) {
        constexpr int NM = 2 * STEPS, E = 16 / NM, NF = 3 * NM;
        const Seen seen(p, k0 + 4 * (lane >> 5), a.window, a.sinks);
        auto frag = [&](int m) {
          const int run = m / NM, i = m % NM;
          if (run < 2) return addr.rows(i & 1 ? vp : kp, 32 * run, i / 2);
          const int v = m - 2 * NM;  // of the sums: half v / STEPS
          return addr.cols(kp, 32 * (v / STEPS) + 16 * (v % STEPS / DB), v % DB);
        };
        bf16x8 f[AHEAD];
        auto next = [&](int m) {
          if (m + AHEAD < NF) f[m % AHEAD] = frag(m + AHEAD);
        };
        Half h0, h1;
        h0.s = h1.s = zero16();
        h0.ds = h1.ds = less;
        auto some = [&](Half& h, int i) {
#pragma unroll
          for (int r = i * E; r < i * E + E; ++r) {
            h.s[r] = __builtin_amdgcn_exp2f(fmaf(h.s[r], a.c, -lse2));
            h.ds[r] *= h.s[r];
            if constexpr (masked.value) {
              const bool see = seen((&h == &h0 ? 0 : 32) + 8 * (r >> 2) + (r & 3));
              h.s[r] = see ? h.s[r] : 0.f;
              h.ds[r] = see ? h.ds[r] : 0.f;
            }
            sum += h.ds[r];
            if (r & 1) {
              h.round(r / 2);
              rsum = pair_add(h.x[r / 2], rsum);
            }
          }
        };
#pragma unroll
        for (int m = 0; m < AHEAD; ++m) f[m] = frag(m);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          if (i & 1) h0.ds = mma32(f[i % AHEAD], g[i / 2], h0.ds);
          else h0.s = mma32(f[i % AHEAD], q[i / 2], h0.s);
          next(i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          if (i & 1) h1.ds = mma32(f[(NM + i) % AHEAD], g[i / 2], h1.ds);
          else h1.s = mma32(f[(NM + i) % AHEAD], q[i / 2], h1.s);
          next(NM + i);
          some(h0, i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const int m = 2 * NM + i / 2, v = i / 2;
          if (i & 1) {
            kbar[v % DB] = mma32(f[m % AHEAD], h0.frag_s(v / DB), kbar[v % DB]);
            next(m);
          } else {
            dq[v % DB] = mma32(f[m % AHEAD], h0.frag_ds(v / DB), dq[v % DB]);
          }
          some(h1, i);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const int m = 2 * NM + STEPS + i / 2, v = i / 2;
          if (i & 1) {
            kbar[v % DB] = mma32(f[m % AHEAD], h1.frag_s(v / DB), kbar[v % DB]);
            next(m);
          } else {
            dq[v % DB] = mma32(f[m % AHEAD], h1.frag_ds(v / DB), dq[v % DB]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      int lo, hi;
      kt.whole(off + r0, off + min(r0 + BM, qlen) - 1, a.window, BN, r0 + BM <= qlen, lo, hi);
      // a tile of which rows may see a part
      auto edge = [&](int i) {
        lds_ptr t = (lds_ptr)lds + (i & 1) * 2 * TB;
        arrive(i, lds + (2 - 2 * (i & 1)) * TB);
        const int k0 = kt.at(i) * BN;
        if (w.lo > w.hi || !w.some(k0, k0 + BN - 1, a.window, a.sinks)) return;
        pair(t, t + TB, std::true_type{}, k0);
      };
#pragma unroll 1
      for (; i < lo; ++i) edge(i);
      for (; i + 1 < hi; i += 2) {
        arrive(i, lds + 2 * TB);
        pair((lds_ptr)lds, (lds_ptr)lds + TB, std::false_type{}, 0);
        arrive(i + 1, lds);
        pair((lds_ptr)lds + 2 * TB, (lds_ptr)lds + 3 * TB, std::false_type{}, 0);
      }
#pragma unroll 1
      for (; i < kt.total; ++i) edge(i);
    } else {
      // a tile of which rows may see a part, 32 keys after another
      auto edge = [&](int i) {
        const char* t = lds + (i & 1) * 2 * TB;
        arrive(i, lds + (2 - 2 * (i & 1)) * TB);
#pragma unroll 1
        for (int sb = 32 * ks; sb < BN; sb += 32 * KS) {
          const int k0 = kt.at(i) * BN + sb;
          if (w.lo > w.hi || !w.some(k0, k0 + 31, a.window, a.sinks)) continue;
          f32x16 s = zero16(), ds = less;
          row_steps<T, STEPS>(a.d, [&](int st) {
            s = mma32(row_frag<T, DP>(t, sb, st, lane), q[st], s);
            ds = mma32(row_frag<T, DP>(t + TB, sb, st, lane), g[st], ds);
          });
          gradients(s, ds);
          if (!w.whole(k0, k0 + 31, a.window, a.sinks)) {
            const Seen seen(p, k0 + 4 * (lane >> 5), a.window, a.sinks);
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const bool see = seen(8 * (r >> 2) + (r & 3));
              s[r] = see ? s[r] : 0.f;
              ds[r] = see ? ds[r] : 0.f;
            }
          }
          if constexpr (CENTRE) {
            const Pair x = round_pair(ds);
            count(ds, x);
            mma_trans<DP>(dq, x.f, t, sb, lane);
            mma_trans<DP>(kbar, round_pair(s).f, t, sb, lane);
          } else {
            mma_trans<DP>(dq, ds, t, sb, lane, a.d);
          }
        }
      };
#pragma unroll 1
      for (; i < kt.total; ++i) edge(i);
    }
    if constexpr (KS == 2) {
      sum = add_parts<RG>(reinterpret_cast<float*>(lds), rg, ks, lane, sum);
      if constexpr (CENTRE) {
        rsum = add_parts<RG>(reinterpret_cast<float*>(lds), rg, ks, lane, rsum);
        add_parts<RG, DB>(reinterpret_cast<float*>(lds), rg, ks, lane, kbar);
      }
      add_parts<RG, DB>(reinterpret_cast<float*>(lds), rg, ks, lane, dq);
    }
    if constexpr (CENTRE) {
      rsum = pair_sum(rsum);
      delta += pair_sum(sum);
#pragma unroll
      for (int db = 0; db < DB; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) dq[db][r] = fmaf(-rsum, kbar[db][r], dq[db][r]);
    }
    // what the dk, dv kernel's products start from: exp2(c (q.k - lse / scale)), dO.v - D
    if (ks == 0 && row < qlen && lane < 32) {
      a.stats[stat] = sizeof(T) == 4 ? -lse : -lse / a.scale;
      a.stats[stats_of(a) + stat] = -delta;
    }
  }
  if (ks != 0) return;
  if (row >= qlen) {  // what a clamped row gathered, finite or not, is nothing
#pragma unroll
    for (int db = 0; db < DB; ++db) dq[db] = zero16();
  }
  char* out = a.dq + seq.at(a, a.sdq) + at.h * a.sdq.h;
  if (row < (A::LIE == Lie::PADDED ? a.Lq : qlen)) store_rows<T, DP>(dq, a.scale, out + (int64_t)row * a.sdq.l, a.d, lane);
  for (uint32_t bad = not_finite(dq) & (uint32_t)__ballot(lse2 == lse2 && delta == delta); bad; bad &= bad - 1) {
    const int i = __builtin_ctz(bad), r = rw + i;
    const float ls = of_lane(lse2, i), de = of_lane(delta, i);
    const Lane2<T> q(qb + r * a.sq.l, a.d, lane), g(gb + r * a.sdo.l, a.d, lane);
    float x[2] = {0.f, 0.f};
#pragma unroll 1
    for (int t = 0; t < kt.total; ++t)
#pragma unroll 1
      for (int j = kt.at(t) * BN; j < kt.at(t) * BN + BN && j <= off + r; ++j) {
        if (j <= off + r - a.window && j >= a.sinks) continue;
        const Lane2<T> k(kb + j * a.sk.l, a.d, lane), v(vb + j * a.sv.l, a.d, lane);
        const float ds = __builtin_amdgcn_exp2f(fmaf(q.dot(k), a.c, -ls)) * (g.dot(v) - de);
#pragma unroll
        for (int e = 0; e < 2; ++e) x[e] = fmaf(ds, k.x[e], x[e]);
        if (settled(x, a.d, lane)) t = kt.total, j = off + r;
      }
    x[0] *= a.scale, x[1] *= a.scale;
    store_lane2<T>(out + r * a.sdq.l, x, a.d, lane);
  }
}

// ------------------------------------------------------------------ backward: dk, dv
// A workgroup owns 128 keys of a key head (64 with KS = 2), a wave 32 of them in registers,
// and meets every row that sees them, over all query heads of the key head
// (their sum needs no atomics).  S = Q K^T and dP = dO V^T have the key in
// the lane and start from the rows' -lse / scale and -D, so that neither is
// subtracted element by element; dv^T += dO^T P and dk^T += Q^T dS.  The same
// 32K step: 560 us, matrix pipes busy 52 % of the time.
//
// Keys below `sinks` are seen by every later row, up to 16 times more than a
// window's; the rows behind the window of a sink tile's last key are split
// over further workgroups of `span` rows each, and the fp32 partial sums of a
// sink tile are added in a fixed order by attn_sink_sum_kernel.
//
// Packed: the rows that a tile meets, over all its query heads, may be split in
// `rs` equal parts, where tiles are few; attn_row_sum_kernel adds them.
//
// The number of a part, of [dk, dv][key][d] each: of a sink tile's splits, and
// behind those of the other tiles by slot.
__device__ __forceinline__ int64_t dkv_part(const PackedArgs& a, int b, int hk, int tile, int split) {
  return ((((int64_t)b * a.Hk + hk) * a.sink_tiles + tile) * a.splits + split) * a.rs;
}
__device__ __forceinline__ int64_t dkv_part(const PackedArgs& a, int slot, int hk) {
  const int64_t sinks = a.splits > 1 ? (int64_t)a.B * a.Hk * a.sink_tiles * a.splits : 0;
  return (sinks + (int64_t)slot * a.Hk + hk) * a.rs;
}

template <typename T, int DP, int KS, class A = AttnArgs>
__global__ __launch_bounds__(256, (attn_back_waves<T, DP>())) void attn_dkv_kernel(A a) {
  constexpr bool PACKED = A::LIE != Lie::PADDED;
  using Tile = AttnTile<T, DP>;
  constexpr int NW = 4, RG = NW / KS, BK = 32 * RG, BQ = attn_bn<T, DP>(), TB = BQ * Tile::CPR * 16, STEPS = Tile::STEPS, DB = DP / 32;
  __shared__ __align__(1024) char lds[4 * TB];
  __shared__ __align__(1024) float stats[2][2][64];  // [ring][-lse / scale, -D][row]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n = lane & 31;
  int tile = 0, split = 0, hk, b, rpart = 0, slot = 0;
  AttnSeq seq(0, 0, 0, 0);
  if constexpr (A::LIE == Lie::PADDED) {
    int id = xcd_remap(blockIdx.x, gridDim.x);
    const int jobs = a.tiles + a.sink_tiles * (a.splits - 1);
    const int job = id % jobs, bk = id / jobs;
    hk = bk % a.Hk, b = bk / a.Hk;
    if (job < a.sink_tiles * a.splits) {
      tile = job / a.splits;
      split = job % a.splits;
    } else {
      tile = job - a.sink_tiles * (a.splits - 1);
    }
    seq = AttnSeq(a, b);
  } else {
    // split sink tiles of all sequences, then the tiles by slots, early keys first: most rows see them
    int id = blockIdx.x;
    if (id >= a.main) {
#pragma unroll 1  // (once in the code: twice, fp32 dk, dv of 12 (4) heads of 96 took 274 us for 263)
      for (int i = 0; i < 2; ++i)
        clear_rest(a, i ? a.dv : a.dk, i ? a.sdv : a.sdk, a.Hk, a.d * (int)sizeof(T), nullptr, id - a.main, a.rest);
      return;
    }
    hk = id % a.Hk, id /= a.Hk;
    if (a.rs > 1) rpart = id % a.rs, id /= a.rs;
    const int jobs = a.splits > 1 ? a.B * a.sink_tiles * a.splits : 0;
    slot = id - jobs;
    if (id < jobs) {
      split = id % a.splits, id /= a.splits;
      tile = id % a.sink_tiles, b = id / a.sink_tiles;
      seq = AttnSeq(a, b);
    } else {
      seq = find_tile(a, slot, BK, lane, true, tile);
      b = seq.b;
      if (b < 0 || (a.splits > 1 && tile < a.sink_tiles)) return;
    }
  }
  const int bk = b * a.Hk + hk;
  const int qlen = seq.qlen, klen = seq.klen, off = klen - qlen;
  if (A::LIE != Lie::PADDED && tile * BK >= klen) return;
  const int k0 = tile * BK, cmax = a.d * (int)sizeof(T) / 16 - 1;
  const int rg = wave % RG, ks = wave / RG;  // keys of the wave; its part of a row tile (see the forward)
  const int key = k0 + 32 * rg + n;
  const char* qh = a.q + seq.at(a, a.sq) + (int64_t)hk * a.G * a.sq.h;
  const char* gh = a.dO + seq.at(a, a.sdo) + (int64_t)hk * a.G * a.sdo.h;
  const char* kh = a.k + seq.at(a, a.sk) + hk * a.sk.h;
  const char* vh = a.v + seq.at(a, a.sv) + hk * a.sv.h;
  const int64_t sh = seq.stat(a, hk * a.G), sn = stats_of(a);
  f32x16 dk[DB], dv[DB];
#pragma unroll
  for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
  // positions of the rows this workgroup meets
  int p_lo = k0, p_hi = klen - 1;
  const int reach = (int)min((int64_t)k0 + BK - 1 + a.window, (int64_t)klen) - 1;  // last that sees k0 + BK - 1 by window
  if (tile < a.sink_tiles && a.splits > 1) {
    if (split == 0) p_hi = reach;
    else {
      p_lo = reach + 1 + (split - 1) * a.span;
      p_hi = min(klen - 1, p_lo + a.span - 1);
    }
  } else if (k0 >= a.sinks) {
    p_hi = reach;
  }
  const int ra = max(0, p_lo - off) / BQ, rz = p_hi - off;  // first row tile, last row
  // of each head's row tiles ra .. rend - 1, those from tile r0 of head h0 to tile r1 - 1 of head h1
  // (PADDED: all, in expressions that leave nothing of the choice in the code: a
  // comparison with head 0 peeled its round off the loop and spilled 100 registers)
  int h0 = 0, h1 = a.G - 1, r0 = ra, rend = rz / BQ + 1, r1 = rend;
  auto from = [&](int h) { return PACKED && h == h0 ? r0 : ra; };
  auto to = [&](int h) { return PACKED && h == h1 ? r1 : rend; };
  if constexpr (PACKED)
    if (a.rs > 1) {
      const int64_t n = max(0, rend - ra), all = n * a.G, s0 = all * rpart / a.rs, s1 = all * (rpart + 1) / a.rs;
      if (s1 > s0) {
        h0 = __builtin_amdgcn_readfirstlane((int)(s0 / n)), h1 = __builtin_amdgcn_readfirstlane((int)((s1 - 1) / n));
        r0 = ra + (int)(s0 - h0 * n), r1 = ra + (int)(s1 - h1 * n);
      } else {
        rend = ra;
      }
    }
  if (k0 < klen && rz >= ra * BQ && p_hi >= p_lo && (!PACKED || rend > ra)) {
    Frag<T> kf[STEPS], vf[STEPS];
    const int64_t kc = min(key, klen - 1);
    load_rows(kf, kh + kc * a.sk.l, cmax, lane);
    load_rows(vf, vh + kc * a.sv.l, cmax, lane);
    const int wk0 = k0 + 32 * rg, wk1 = min(wk0 + 31, klen - 1);
    Stager<T, DP, BQ, NW> sq(qh, a.sq.l, qlen - 1, cmax, wave, lane), sg(gh, a.sdo.l, qlen - 1, cmax, wave, lane);
    auto issue = [&](int h, int rt, char* t, float* st) {
      sq.base = qh + h * a.sq.h;
      sg.base = gh + h * a.sdo.h;
      sq.issue(t, rt * BQ);
      sg.issue(t + TB, rt * BQ);
      if (wave < 2)
        dma4(a.stats + wave * sn + sh + (int64_t)h * a.Lq + min(rt * BQ + lane, qlen - 1),
             __builtin_amdgcn_readfirstlane(lds_at(st) + (uint32_t)wave * 256u));
    };
    auto arrive = [&](int h, int rt, char* other, float* st) {
      wait_lgkm0();
      wait_vm<0>();
      bar();
      if (rt + 1 < to(h)) issue(h, rt + 1, other, st);
      else if (h + 1 < (PACKED ? h1 + 1 : a.G)) issue(h + 1, ra, other, st);
    };
    // -lse / scale or -D of 32 rows, as a product leaves them
    auto start = [&](const float* st, int row0) {
      f32x16 x;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(st + row0 + 8 * g + 4 * (lane >> 5));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * g + e] = v[e];
      }
      return x;
    };
    issue(h0, r0, lds, stats[0][0]);
    int i = 0;  // tiles done: the ring's place
#pragma unroll 1
    for (int h = h0; h < (PACKED ? h1 + 1 : a.G); ++h) {
      int rt = from(h);
      const int re = to(h);
      if constexpr (sizeof(T) == 2 && BQ == 64 && KS == 1) {
        // row tiles that see all keys of the workgroup
        const int last = k0 + BK - 1 < a.sinks ? p_hi : min(p_hi, k0 + a.window - 1);
        const int wa = max(ra, (max(max(k0 + BK - 1, p_lo) - off, 0) + BQ - 1) / BQ);
        const int wz = k0 + BK <= klen && last >= off ? min(re, (last - off + 1) / BQ) : 0;
        const AttnAddr<DP> addr(lane);
        // 64 rows that see every key (see AttnRows::step2)
        auto pair = [&](lds_ptr qp, lds_ptr gp, const float* st, auto masked, int lo, int hi) {
          constexpr int NM = 2 * STEPS, E = 16 / NM;
          auto frag = [&](int m) {
            const int run = m / NM, i = m % NM;
            return run < 2 ? addr.rows(i & 1 ? gp : qp, 32 * run, i / 2)
                           : addr.cols(i & 1 ? qp : gp, 32 * (run - 2) + 16 * (i / 2 / DB), i / 2 % DB);
          };
          bf16x8 f[AHEAD];
          auto next = [&](int m) {
            if (m + AHEAD < 4 * NM) f[m % AHEAD] = frag(m + AHEAD);
          };
          Half h0, h1;
          auto some = [&](Half& h, int i) {
#pragma unroll
            for (int r = i * E; r < i * E + E; ++r) {
              h.s[r] = __builtin_amdgcn_exp2f(h.s[r] * a.c);
              h.ds[r] *= h.s[r];
              if constexpr (masked.value) {
                const int o = (&h == &h0 ? 0 : 32) + 8 * (r >> 2) + (r & 3);
                const bool see = (o >= lo) & (o <= hi);
                h.s[r] = see ? h.s[r] : 0.f;
                h.ds[r] = see ? h.ds[r] : 0.f;
              }
              if (r & 1) h.round(r / 2);
            }
          };
          auto add = [&](const Half& h, int run, int i) {
            const bf16x8 x = f[(run * NM + i) % AHEAD];
            const int v = i / 2;
            if (i & 1) dk[v % DB] = mma32(x, h.frag_ds(v / DB), dk[v % DB]);
            else dv[v % DB] = mma32(x, h.frag_s(v / DB), dv[v % DB]);
            next(run * NM + i);
          };
          h0.s = start(st, 0), h0.ds = start(st + 64, 0);
#pragma unroll
          for (int m = 0; m < AHEAD; ++m) f[m] = frag(m);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            if (i & 1) h0.ds = mma32(f[i % AHEAD], vf[i / 2], h0.ds);
            else h0.s = mma32(f[i % AHEAD], kf[i / 2], h0.s);
            next(i);
            if (i == NM / 2) h1.s = start(st, 32), h1.ds = start(st + 64, 32);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            if (i & 1) h1.ds = mma32(f[(NM + i) % AHEAD], vf[i / 2], h1.ds);
            else h1.s = mma32(f[(NM + i) % AHEAD], kf[i / 2], h1.s);
            next(NM + i);
            some(h0, i);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            add(h0, 2, i);
            some(h1, i);
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            add(h1, 3, i);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        // a tile of which a key may be seen by a part of the rows: those at
        // positions q0 + 4 (lane / 32) + lo .. hi
        auto edge = [&](int h, int rt, int ring) {
          lds_ptr t = (lds_ptr)lds + ring * 2 * TB;
          arrive(h, rt, lds + (2 - 2 * ring) * TB, stats[1 - ring][0]);
          const int q0 = off + rt * BQ, u0 = max(q0, p_lo), u1 = min(q0 + BQ - 1, p_hi);
          if (u0 > u1 || wk0 > wk1 || u1 < wk0 || (wk1 <= u0 - a.window && wk0 >= a.sinks)) return;
          const int base = q0 + 4 * (lane >> 5), lo = max(u0, key) - base,
                    hi = (key < a.sinks ? u1 : min(u1, key + a.window - 1)) - base;
          pair(t, t + TB, stats[ring][0], std::true_type{}, lo, hi);
        };
#pragma unroll 1
        for (; rt < re && (rt < wa || (rt < wz && (i & 1))); ++rt, ++i) edge(h, rt, i & 1);
        for (; rt + 1 < wz; rt += 2, i += 2) {
          arrive(h, rt, lds + 2 * TB, stats[1][0]);
          pair((lds_ptr)lds, (lds_ptr)lds + TB, stats[0][0], std::false_type{}, 0, 0);
          arrive(h, rt + 1, lds, stats[0][0]);
          pair((lds_ptr)lds + 2 * TB, (lds_ptr)lds + 3 * TB, stats[1][0], std::false_type{}, 0, 0);
        }
#pragma unroll 1
        for (; rt < re; ++rt, ++i) edge(h, rt, i & 1);
      } else if constexpr (sizeof(T) == 2) {
        // the wave's 32 rows of a tile in four runs of products, S, dP, dv and
        // dk, with P formed between those of dP and dS between those of dv (5
        // texts of up to 1777 tokens, 12 (4) heads of 96: 100 us one after
        // another, 85 so)
        const AttnAddr<DP> addr(lane);
        auto edge = [&](int h, int rt, int ring) {
          constexpr int NM = STEPS, E = 16 / NM;
          arrive(h, rt, lds + (2 - 2 * ring) * TB, stats[1 - ring][0]);
          const int q0 = off + rt * BQ + 32 * ks, u0 = max(q0, p_lo), u1 = min(q0 + 31, p_hi);
          if (u0 > u1 || wk0 > wk1 || u1 < wk0 || (wk1 <= u0 - a.window && wk0 >= a.sinks)) return;
          const int base = q0 + 4 * (lane >> 5), lo = max(u0, key) - base,
                    hi = (key < a.sinks ? u1 : min(u1, key + a.window - 1)) - base;
          const lds_ptr qp = (lds_ptr)lds + ring * 2 * TB + 32 * ks * AttnAddr<DP>::ROW, gp = qp + TB;
          const float* st = stats[ring][0] + 32 * ks;
          auto frag = [&](int m) {
            const int run = m / NM, i = m % NM;
            return run < 2 ? addr.rows(run ? gp : qp, 0, i) : addr.cols(run == 2 ? gp : qp, 16 * (i / DB), i % DB);
          };
          bf16x8 f[AHEAD];
          auto next = [&](int m) {
            if (m + AHEAD < 4 * NM) f[m % AHEAD] = frag(m + AHEAD);
          };
          Half x;
          x.s = start(st, 0), x.ds = start(st + 64, 0);
#pragma unroll
          for (int m = 0; m < AHEAD; ++m) f[m] = frag(m);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            x.s = mma32(f[i % AHEAD], kf[i], x.s);
            next(i);
            __builtin_amdgcn_sched_barrier(0);
          }
          auto sees = [&](int r) {
            const int o = 8 * (r >> 2) + (r & 3);
            return (o >= lo) & (o <= hi);
          };
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            x.ds = mma32(f[(NM + i) % AHEAD], vf[i], x.ds);
            next(NM + i);
#pragma unroll
            for (int r = i * E; r < i * E + E; ++r) {
              const float e = __builtin_amdgcn_exp2f(x.s[r] * a.c);
              x.s[r] = sees(r) ? e : 0.f;
              if (r & 1) x.y[r / 2] = pack_bf16x2(x.s[r - 1], x.s[r]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            dv[i % DB] = mma32(f[(2 * NM + i) % AHEAD], x.frag_s(i / DB), dv[i % DB]);
            next(2 * NM + i);
#pragma unroll
            for (int r = i * E; r < i * E + E; ++r) {
              x.ds[r] = sees(r) ? x.ds[r] * x.s[r] : 0.f;
              if (r & 1) x.x[r / 2] = pack_bf16x2(x.ds[r - 1], x.ds[r]);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (int i = 0; i < NM; ++i) {
            dk[i % DB] = mma32(f[(3 * NM + i) % AHEAD], x.frag_ds(i / DB), dk[i % DB]);
            next(3 * NM + i);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
#pragma unroll 1
        for (; rt < re; ++rt, ++i) edge(h, rt, i & 1);
      } else {
        // a tile of which rows may see a part, 32 rows after another
        auto edge = [&](int h, int rt, int ring) {
          const char* t = lds + ring * 2 * TB;
          arrive(h, rt, lds + (2 - 2 * ring) * TB, stats[1 - ring][0]);
#pragma unroll 1
          for (int sb = 32 * ks; sb < BQ; sb += 32 * KS) {
            const int q0 = off + rt * BQ + sb, q1 = q0 + 31;  // positions
            const int u0 = max(q0, p_lo), u1 = min(q1, p_hi);
            if (u0 > u1 || wk0 > wk1 || u1 < wk0 || (wk1 <= u0 - a.window && wk0 >= a.sinks)) continue;
            const bool whole = u0 == q0 && u1 == q1 && wk1 <= q0 && wk0 + 31 == wk1 &&
                               (wk0 > q1 - a.window || wk1 < a.sinks);
            const f32x16 less_s = start(stats[ring][0], sb), less_ds = start(stats[ring][1], sb);
            f32x16 s = zero16(), ds = zero16();
            row_steps<T, STEPS>(a.d, [&](int st) {
              s = mma32(row_frag<T, DP>(t, sb, st, lane), kf[st], s);
              ds = mma32(row_frag<T, DP>(t + TB, sb, st, lane), vf[st], ds);
            });
#pragma unroll
            for (int r = 0; r < 16; ++r) {  // fp32: the statistics are added last, see the dq kernel
              s[r] = __builtin_amdgcn_exp2f(LOG2E * fmaf(s[r], a.scale, less_s[r]));
              ds[r] = (ds[r] + less_ds[r]) * s[r];
            }
            if (!whole) {
              // a row's position p = q0 + 4 (lane / 32) + o, against the key's own bounds
              const int base = q0 + 4 * (lane >> 5), lo = max(u0, key) - base,
                        hi = (key < a.sinks ? u1 : min(u1, key + a.window - 1)) - base;
#pragma unroll
              for (int r = 0; r < 16; ++r) {
                const int o = 8 * (r >> 2) + (r & 3);
                const bool see = (o >= lo) & (o <= hi);
                s[r] = see ? s[r] : 0.f;
                ds[r] = see ? ds[r] : 0.f;
              }
            }
            acc_trans<T, DP>(dv, s, t + TB, sb, lane, a.d);
            acc_trans<T, DP>(dk, ds, t, sb, lane, a.d);
          }
        };
#pragma unroll 1
        for (; rt < re; ++rt, ++i) edge(h, rt, i & 1);
      }
    }
  }
  if constexpr (KS == 2) {
    add_parts<RG, DB>(reinterpret_cast<float*>(lds), rg, ks, lane, dk);
    add_parts<RG, DB>(reinterpret_cast<float*>(lds), rg, ks, lane, dv);
    if (ks != 0) return;
  }
  if (key >= klen) {  // masked to zeros, but zero times a NaN of a row that others see is none
#pragma unroll
    for (int db = 0; db < DB; ++db) dk[db] = dv[db] = zero16();
  }
  const bool sink = tile < a.sink_tiles && a.splits > 1;
  bool parts = sink;
  // [batch x key head][sink tile][split][dk, dv][key][d]
  int64_t place = ((int64_t)bk * a.sink_tiles + tile) * a.splits + split;
  if constexpr (PACKED)
    if (a.rs > 1) {
      parts = true;
      place = (sink ? dkv_part(a, b, hk, tile, split) : dkv_part(a, slot, hk)) + rpart;
    }
  float* pk = a.part + place * 2 * BK * a.d;
  char* ok = a.dk + seq.at(a, a.sdk) + hk * a.sdk.h;
  char* ov = a.dv + seq.at(a, a.sdv) + hk * a.sdv.h;
  if (parts) {
    float* to = pk + (32 * rg + n) * a.d;
    store_rows<float, DP>(dk, 1.f, reinterpret_cast<char*>(to), a.d, lane);
    store_rows<float, DP>(dv, 1.f, reinterpret_cast<char*>(to + BK * a.d), a.d, lane);
  } else if (key < (A::LIE == Lie::PADDED ? a.Lk : klen)) {
    store_rows<T, DP>(dk, a.scale, ok + (int64_t)key * a.sdk.l, a.d, lane);
    store_rows<T, DP>(dv, 1.f, ov + (int64_t)key * a.sdv.l, a.d, lane);
  }
  for (uint32_t bad = (not_finite(dk) | not_finite(dv)) & (uint32_t)__ballot(key < klen); bad; bad &= bad - 1) {
    const int i = __builtin_ctz(bad), j = k0 + 32 * rg + i;
    const Lane2<T> k(kh + j * a.sk.l, a.d, lane), v(vh + j * a.sv.l, a.d, lane);
    float x[2] = {0.f, 0.f}, y[2] = {0.f, 0.f};
#pragma unroll 1
    for (int h = h0; h < (PACKED ? h1 + 1 : a.G); ++h)
#pragma unroll 1
      for (int p = max(max(p_lo, j), off + (PACKED ? from(h) * BQ : 0)); p <= (PACKED ? min(p_hi, off + to(h) * BQ - 1) : p_hi); ++p) {
        if (j <= p - a.window && j >= a.sinks) break;
        const int64_t r = p - off, st = sh + (int64_t)h * a.Lq + r;
        const Lane2<T> q(qh + h * a.sq.h + r * a.sq.l, a.d, lane), g(gh + h * a.sdo.h + r * a.sdo.l, a.d, lane);
        const float pr = sizeof(T) == 4 ? __builtin_amdgcn_exp2f(LOG2E * fmaf(q.dot(k), a.scale, a.stats[st]))
                                        : __builtin_amdgcn_exp2f(a.c * (q.dot(k) + a.stats[st]));
        const float ds = pr * (g.dot(v) + a.stats[sn + st]);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[e] = fmaf(ds, q.x[e], x[e]);
          y[e] = fmaf(pr, g.x[e], y[e]);
        }
        if (settled(x, a.d, lane) && settled(y, a.d, lane)) {
          h = a.G;
          break;
        }
      }
    if (parts) {
      float* to = pk + (32 * rg + i) * a.d;
      store_lane2<float>(reinterpret_cast<char*>(to), x, a.d, lane);
      store_lane2<float>(reinterpret_cast<char*>(to + BK * a.d), y, a.d, lane);
    } else {
      x[0] *= a.scale, x[1] *= a.scale;
      store_lane2<T>(ok + j * a.sdk.l, x, a.d, lane);
      store_lane2<T>(ov + j * a.sdv.l, y, a.d, lane);
    }
  }
}

// Four columns of a key's dk or dv: `n` parts, `step` floats apart, in order
__device__ __forceinline__ void sum_parts(float (&sum)[4], const float* pr, int64_t step, int n) {
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(pr + i * step);
    sum[0] += v.x, sum[1] += v.y, sum[2] += v.z, sum[3] += v.w;
  }
}
template <typename T, class A>
__device__ __forceinline__ void store_key(const A& a, const AttnSeq& seq, int hk, int key, int what, int c, float (&sum)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = key >= seq.klen ? 0.f : what ? sum[e] : sum[e] * a.scale;
  char* to = what ? a.dv + seq.at(a, a.sdv) + hk * a.sdv.h + (int64_t)key * a.sdv.l
                  : a.dk + seq.at(a, a.sdk) + hk * a.sdk.h + (int64_t)key * a.sdk.l;
  store4(reinterpret_cast<T*>(to) + c, sum);
}

// dk, dv of the sink tiles, BK keys each: the splits' partial sums, in order
// (behind the first split's rows only sinks are seen: other keys' sums are whole
// with it).  32 threads a key, four columns each.
template <typename T, int BK, class A = AttnArgs>
__global__ __launch_bounds__(256) void attn_sink_sum_kernel(A a) {
  const int keys = a.sink_tiles * BK, place = blockIdx.x * 8 + threadIdx.x / 32;
  const int x = place % (2 * keys), bk = place / (2 * keys), what = x / keys, key = x % keys;
  const int hk = bk % a.Hk, b = bk / a.Hk, c = threadIdx.x % 32 * 4;
  const AttnSeq seq(a, b);
  if (key >= (A::LIE == Lie::PADDED ? a.Lk : seq.klen) || c >= a.d) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  sum_parts(sum, a.part + ((((int64_t)bk * a.sink_tiles + key / BK) * a.splits * 2 + what) * BK + key % BK) * a.d + c,
            (int64_t)2 * BK * a.d, key < a.sinks ? a.splits : 1);
  store_key<T>(a, seq, hk, key, what, c, sum);
}

// dk, dv of a packed batch whose tiles' rows are split: a tile's parts, in
// order.  Workgroups as in the dk, dv kernel, one for eight rows of a tile's dk
// or dv.
template <typename T, int BK>
__global__ __launch_bounds__(256) void attn_row_sum_kernel(PackedArgs a) {
  constexpr int PER = 2 * BK / 8;
  const int lane = threadIdx.x % WAVE, x = blockIdx.x % PER * 8 + threadIdx.x / 32, what = x / BK, c = threadIdx.x % 32 * 4;
  int id = blockIdx.x / PER, tile = 0, n = a.rs;
  const int hk = id % a.Hk, sink = a.splits > 1 ? a.B * a.sink_tiles : 0;
  id /= a.Hk;
  int64_t first;
  AttnSeq seq(0, 0, 0, 0);
  if (id < sink) {
    tile = id % a.sink_tiles;
    seq = AttnSeq(a, id / a.sink_tiles);
    first = dkv_part(a, seq.b, hk, tile, 0);
    if (tile * BK + x % BK < a.sinks) n *= a.splits;
  } else {
    seq = find_tile(a, id - sink, BK, lane, true, tile);
    if (seq.b < 0 || (a.splits > 1 && tile < a.sink_tiles)) return;
    first = dkv_part(a, id - sink, hk);
  }
  const int key = tile * BK + x % BK;
  if (key >= seq.klen || c >= a.d) return;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
  sum_parts(sum, a.part + ((first * 2 + what) * BK + x % BK) * a.d + c, (int64_t)2 * BK * a.d, n);
  store_key<T>(a, seq, hk, key, what, c, sum);
}

}  // namespace lact
