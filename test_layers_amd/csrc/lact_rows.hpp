// Row kernels around the block: rotary positions, and the residual's addition
// with the root-mean-square norm (8-bit output, backward).  All are bound by
// memory: each tensor is read or written once, 16 bytes a lane where the
// addresses allow it.
#pragma once
#include "lact_device.hpp"

namespace lact {

// N consecutive elements at p as floats, N x sizeof(T) a power of two up to
// 16 bytes, p aligned to that
template <typename T, int N>
__device__ __forceinline__ void load_n(const T* p, float (&v)[N]) {
  constexpr int W = N * (int)sizeof(T);
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 4) load4(p, v);
    else if constexpr (N == 2) {
      const float2 x = *reinterpret_cast<const float2*>(p);
      v[0] = x.x, v[1] = x.y;
    } else v[0] = p[0];
  } else if constexpr (W == 16) load_chunk(p, v);
  else if constexpr (N == 2) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(p);
    v[0] = bf2f(x & 0xffffu), v[1] = bf2f(x >> 16);
  } else v[0] = bf2f(p[0].x);
}
template <typename T, int N>
__device__ __forceinline__ void store_n(T* p, const float (&v)[N]) {
  constexpr int W = N * (int)sizeof(T);
  if constexpr (sizeof(T) == 4) {
    if constexpr (N == 4) store4(p, v);
    else if constexpr (N == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else p[0] = v[0];
  } else if constexpr (W == 16) store_chunk(p, v);
  else if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
  else io_traits<bf16_t>::store(p, v[0]);
}

// ------------------------------------------------------------------ rotary positions
struct RotaryTensor {
  const char* in;
  char* out;
  int64_t ib, ih, il, ob, oh, ol;  // byte strides
  int32_t heads;
};

struct RotaryArgs {
  RotaryTensor t[2];         // q and k (k.heads 0: none)
  const double* freqs;       // [pairs] radians a position
  const int64_t* positions;  // [B, L], or null: start + token
  int64_t start;
  int32_t B, L, d, pairs;
  int32_t tok, group, head_groups;  // tokens and heads of a workgroup, groups of heads
  int32_t heads_inner;              // heads are closer in memory than tokens
  FastDiv by_pairs, by_per, by_inner;  // pairs; items of a head's row; group or tok
  float mscale;
  int32_t inverse;
};

constexpr int ROT_TABLE = 2048;  // pairs of one workgroup's table

// (x, y) -> mscale (x cos - y sin, x sin + y cos) for the features (i, i + n)
// or (2 i, 2 i + 1), the rest copied.  A workgroup first fills a table of the
// angles of its tokens, in fp64 turns: a far position times a frequency needs
// all of a double's bits before whole turns are dropped.  All heads of q and
// k then use the table.
//
// Bound by memory: 32768 tokens of 32 + 8 heads of 128, bf16: 131 us, 5.1 TB/s
// of the 671 MB read and written; the table is 1 / 40 of the work.  Short
// calls are bound by the table: two dependent trips to memory around fp64
// sines, 3.4 us for the next tokens of 64 sequences.
template <typename T, int VE, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  __shared__ float cs[ROT_TABLE], sn[ROT_TABLE];
  const int groups = (a.L + a.tok - 1) / a.tok;
  int id = blockIdx.x;
  const int hg = id % a.head_groups;
  id /= a.head_groups;
  const int t0 = (id % groups) * a.tok, b = id / groups;
  const int nt = min(a.tok, a.L - t0), n = a.pairs;
  // items of a head's row: pairs by VE (half layout) or VE / 2, then the copied rest
  constexpr int PV = INTERLEAVED ? (VE > 1 ? VE / 2 : 1) : VE;
  // interleaved vectors hold whole pairs, so an item is one vector; else two
  constexpr bool ONE = INTERLEAVED && VE > 1;
  const int turned = n / PV, per = (int)a.by_per.d;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int h0 = hg * a.group;
  // neighbours in memory go to neighbouring lanes: heads run inside tokens or
  // tokens inside heads; what the last groups lack is skipped
  const int items = a.tok * a.group * per;
  constexpr int U = VE * (int)sizeof(T) >= 16 ? 2 : 4;  // items in flight: all loads of a round before its stores
  float u[U][VE], v[U][VE];
  T* out[U];
  int c[U], tab[U];  // c: -1 nothing to do
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + 256 * k;
      c[k] = -1;
      if (i >= items) continue;
      const int r = (int)a.by_per.div(i), outer = (int)a.by_inner.div(r), inner = r - outer * (int)a.by_inner.d;
      const int t = a.heads_inner ? outer : inner;
      int h = h0 + (a.heads_inner ? inner : outer);
      if (t >= nt || h >= heads) continue;
      const RotaryTensor& x = h < a.t[0].heads ? a.t[0] : a.t[1];
      if (h >= a.t[0].heads) h -= a.t[0].heads;
      const T* in = reinterpret_cast<const T*>(x.in + b * x.ib + h * x.ih + (int64_t)(t0 + t) * x.il);
      out[k] = reinterpret_cast<T*>(x.out + b * x.ob + h * x.oh + (int64_t)(t0 + t) * x.ol);
      const int cc = i - r * per;
      if (cc >= turned && in == out[k]) continue;  // in place, the rest is there
      c[k] = cc;
      tab[k] = t * n + cc * PV;
      const int e0 = cc >= turned ? 2 * n + (cc - turned) * VE : ONE ? cc * VE : INTERLEAVED ? 2 * cc : cc * VE;
      load_n<T, VE>(in + e0, u[k]);
      if (!ONE && cc < turned) load_n<T, VE>(in + e0 + (INTERLEAVED ? 1 : n), v[k]);
      out[k] += e0;
    }
  };
  fetch(threadIdx.x);  // on its way while the table is made
  for (int i = threadIdx.x; i < nt * n; i += 256) {
    const int k = (int)a.by_pairs.div(i), t = t0 + k;
    const double pos = (double)(a.positions ? a.positions[(int64_t)b * a.L + t] : a.start + t);
    double turn = pos * (a.freqs[i - k * n] * 0.15915494309189533577);  // / (2 pi)
    turn -= rint(turn);
    const float near = (float)turn;
    float s, co;
    if constexpr (sizeof(T) == 4) {
      // what rounding the turn cost, up to 2^-23 of angle, is put back to first
      // order (its square is far below fp32): also next to a zero of the sine
      // or cosine the value is then right to a few steps of its own size
      sincospif(2.f * near, &s, &co);
      const float rest = 6.28318530717958648f * (float)(turn - (double)near), s0 = s;
      s = fmaf(rest, co, s);
      co = fmaf(-rest, s0, co);
    } else {
      // the hardware's sine of turns, with the rounding of the turn off by
      // 2^-23.4 at most (measured over 2^17 angles, next to the zeros and far
      // positions among them): below a bf16 step of anything from 2^-14 on
      s = __builtin_amdgcn_sinf(near);
      co = __builtin_amdgcn_cosf(near);
    }
    cs[i] = co * a.mscale;
    sn[i] = (a.inverse ? -s : s) * a.mscale;
  }
  __syncthreads();
  for (int i0 = threadIdx.x; i0 < items; i0 += 256 * U) {
    if (i0 >= 256 * U) fetch(i0);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (c[k] < 0) continue;
      if (c[k] < turned) {
        if constexpr (ONE) {
#pragma unroll
          for (int j = 0; j < VE; j += 2) {
            const float co = cs[tab[k] + j / 2], si = sn[tab[k] + j / 2], x0 = u[k][j], x1 = u[k][j + 1];
            u[k][j] = x0 * co - x1 * si;
            u[k][j + 1] = x0 * si + x1 * co;
          }
        } else {
#pragma unroll
          for (int j = 0; j < VE; ++j) {
            const float co = cs[tab[k] + j], si = sn[tab[k] + j], x0 = u[k][j], x1 = v[k][j];
            u[k][j] = x0 * co - x1 * si;
            v[k][j] = x0 * si + x1 * co;
          }
          store_n<T, VE>(out[k] + (INTERLEAVED ? 1 : n), v[k]);
        }
      }
      store_n<T, VE>(out[k], u[k]);
    }
  }
}

// ------------------------------------------------------------------ add and norm
constexpr int NORM_GROUP = 128;  // columns that share a scale of the 8-bit output
constexpr float E4M3_MAX = 448.f;

struct NormArgs {
  const char *x, *res, *dy, *dh;  // dh: null where no gradient reaches h otherwise
  const float* w;
  char *h, *y, *dx;
  uint8_t* y8;
  float *scales, *part;
  int64_t rows, ldx, ldr, ldh, ldy, ldy8, ldg, lddh, lddx;  // row strides in bytes
  int32_t cols;
  float eps;
};

// One thread's NV vectors of a row: vector j holds columns (j GS + t) VE ..
// Rows that are not vector-aligned take the same 16-byte accesses, which need
// no more than an element's alignment, and single ones in a row's last vector
// (16384 rows of 2047 bf16: 169 us with single ones throughout, 70 so).  The
// weight is read the same way: loaded value by value it took longer than the
// few rows that a workgroup has (the same rows: 70 and 49 us; 8192 of 1000,
// aligned: 21 and 12).
template <typename T, int NV, int GS, bool VEC>
struct NormRow {
  static constexpr int VE = io_traits<T>::VE;
  __device__ static __forceinline__ int col(int j, int t) { return (j * GS + t) * VE; }
  __device__ static __forceinline__ void load(const char* row, int cols, int t, float (&v)[NV][VE]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j, t);
      const T* p = reinterpret_cast<const T*>(row) + c;
#pragma unroll
      for (int e = 0; e < VE; ++e) v[j][e] = 0.f;
      if (VEC ? c < cols : c + VE <= cols) {
        if constexpr (VEC) {
          load_n<T, VE>(p, v[j]);
        } else {
          uint4 u;
          __builtin_memcpy(&u, p, 16);
#pragma unroll
          for (int e = 0; e < VE; ++e) v[j][e] = value(u, e);
        }
      } else if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (c + e < cols) {
            float x[1];
            load_n<T, 1>(p + e, x);
            v[j][e] = x[0];
          }
      }
    }
  }
  // the same vectors as they lie in memory
  __device__ static __forceinline__ void load_raw(const char* row, int cols, int t, uint4 (&v)[NV]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j, t);
      const T* p = reinterpret_cast<const T*>(row) + c;
      v[j] = zero4();
      if (VEC ? c < cols : c + VE <= cols) {
        if constexpr (VEC) v[j] = *reinterpret_cast<const uint4*>(p);
        else __builtin_memcpy(&v[j], p, 16);
      } else if constexpr (!VEC) {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (c + e < cols) {
            if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(p[e]);
            else w[e / 2] |= (uint32_t)p[e].x << (16 * (e % 2));
          }
        v[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  // value e of a vector
  __device__ static __forceinline__ float value(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return e % 2 ? __uint_as_float(w[e / 2] & 0xffff0000u) : __uint_as_float(w[e / 2] << 16);
  }
  __device__ static __forceinline__ void store(char* row, int cols, int t, const float (&v)[NV][VE]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j, t);
      T* p = reinterpret_cast<T*>(row) + c;
      if (VEC ? c < cols : c + VE <= cols) {
        if constexpr (VEC) {
          store_n<T, VE>(p, v[j]);
        } else {
          T u[VE];
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const float x[1] = {v[j][e]};
            store_n<T, 1>(u + e, x);
          }
          __builtin_memcpy(p, u, 16);
        }
      } else if constexpr (!VEC) {
#pragma unroll
        for (int e = 0; e < VE; ++e)
          if (c + e < cols) {
            const float x[1] = {v[j][e]};
            store_n<T, 1>(p + e, x);
          }
      }
    }
  }
  __device__ static __forceinline__ void weights(const float* w, int cols, int t, float (&v)[NV][VE]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j, t);
      if (c + VE <= cols) {
        __builtin_memcpy(v[j], w + c, VE * 4);
      } else {
#pragma unroll
        for (int e = 0; e < VE; ++e) v[j][e] = !VEC && c + e < cols ? w[c + e] : 0.f;
      }
    }
  }
};

// sums of two values over the GS threads of a row; every thread gets them
template <int GS>
__device__ __forceinline__ float2 row_sum2(float a, float b, float2* lds, int t) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (GS > WAVE) {
    __syncthreads();  // the sums of the row before have been read
    if (t % WAVE == 0) lds[t / WAVE] = make_float2(a, b);
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < GS / WAVE; ++i) {
      a += lds[i].x;
      b += lds[i].y;
    }
  }
  return make_float2(a, b);
}

// h = x + residual; y = h w / sqrt(mean h^2 + eps), from the unrounded sum.
// GS threads a row, the row in registers, the weight too over all of the
// workgroup's rows.  The 8-bit output: a 128-column group is 16 (bf16) or 32
// (fp32) neighbouring lanes, so its largest magnitude costs a few lane
// exchanges; y is divided by it before it is rounded, once.
//
// Bound by memory: 32768 rows of 4096 bf16 with a residual to h and 8 bits:
// 181 us, 5.2 TB/s of 943 MB; of 1536 to h and y: 64 us, 6.3 TB/s.
template <typename T, int NV, int GS, bool VEC, bool QUANT>
__global__ __launch_bounds__(GS < 256 ? 256 : GS) void norm_kernel(NormArgs a) {
  using R = NormRow<T, NV, GS, VEC>;
  constexpr int VE = R::VE, NT = GS < 256 ? 256 : GS, RPB = NT / GS;
  __shared__ float2 lds[NT / WAVE];
  const int t = threadIdx.x % GS;
  float w[NV][VE];
  R::weights(a.w, a.cols, t, w);
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / GS; row < a.rows; row += (int64_t)gridDim.x * RPB) {
    float h[NV][VE];
    R::load(a.x + row * a.ldx, a.cols, t, h);
    if (a.res) {
      float r[NV][VE];
      R::load(a.res + row * a.ldr, a.cols, t, r);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) h[j][e] += r[j][e];
    }
    if (a.h) R::store(a.h + row * a.ldh, a.cols, t, h);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) ss = fmaf(h[j][e], h[j][e], ss);
    const float f = rsqrtf(row_sum2<GS>(ss, 0.f, lds, t).x / (float)a.cols + a.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) h[j][e] *= f * w[j][e];
    if (a.y) R::store(a.y + row * a.ldy, a.cols, t, h);
    if constexpr (QUANT) {
      constexpr int LANES = NORM_GROUP / VE;
      const int groups = (a.cols + NORM_GROUP - 1) / NORM_GROUP;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = R::col(j, t);
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < VE; ++e) top = fmaxf(top, fabsf(h[j][e]));
#pragma unroll
        for (int o = LANES / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, WAVE));
        // the floor keeps 1 / scale finite where a group is zero
        top = fmaxf(top, 0x1p-100f);
        const float inv = E4M3_MAX / top;
        if (c >= a.cols) continue;
        if (c % NORM_GROUP == 0) a.scales[row * groups + c / NORM_GROUP] = top / E4M3_MAX;
        uint32_t q[VE / 4];
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
          uint32_t p = __builtin_amdgcn_cvt_pk_fp8_f32(h[j][e] * inv, h[j][e + 1] * inv, 0, false);
          q[e / 4] = __builtin_amdgcn_cvt_pk_fp8_f32(h[j][e + 2] * inv, h[j][e + 3] * inv, p, true);
        }
        uint8_t* to = a.y8 + row * a.ldy8 + c;
        if constexpr (VEC) {
          if constexpr (VE == 8) *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
          else *reinterpret_cast<uint32_t*>(to) = q[0];
        } else if (c + VE <= a.cols) {
          __builtin_memcpy(to, q, VE);
        } else {
#pragma unroll
          for (int e = 0; e < VE; ++e)
            if (c + e < a.cols) to[e] = (uint8_t)(q[e / 4] >> (8 * (e % 4)));
        }
      }
    }
  }
}

// From the stored h, with g = w dy and f = 1 / sqrt(mean h^2 + eps):
//   dx = f g - h f^3 mean(g h) + dh,  dw = sum over rows of dy h f.
// A workgroup takes NT / GS rows at a time, gridDim of them apart, and keeps
// its dw in registers; its threads of a column add up in LDS, and the
// workgroups' partial sums are added in a fixed order by norm_dw_kernel.
// Bound by memory: 32768 rows of 1536 bf16: 82 us, 4.9 TB/s of 403 MB, and
// 4.5 us for the partial sums.
template <typename T, int NV, int GS, bool VEC>
__global__ __launch_bounds__(GS < 512 ? 512 : GS) void norm_back_kernel(NormArgs a) {
  using R = NormRow<T, NV, GS, VEC>;
  constexpr int VE = R::VE, NT = GS < 512 ? 512 : GS, RPB = NT / GS;
  __shared__ float2 lds[NT / WAVE];
  __shared__ float sums[RPB > 1 ? NV * VE * GS : 1];
  const int t = threadIdx.x % GS, group = threadIdx.x / GS;
  float2* mine = lds + group * (GS / WAVE);
  float w[NV][VE], dw[NV][VE];
  R::weights(a.w, a.cols, t, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = 0.f;
  // Rows come as they lie in memory, and the next one's before this one is
  // used: the loads of a row then have a row's arithmetic to arrive.  Every
  // group runs the same number of rounds (a row's sum has barriers where GS > 64).
  uint4 h[NV], g[NV], o[NV];
  auto fetch = [&](int64_t row) {
    const int cols = row < a.rows ? a.cols : 0;
    R::load_raw(a.x + row * a.ldx, cols, t, h);
    R::load_raw(a.dy + row * a.ldg, cols, t, g);
    if (a.dh) R::load_raw(a.dh + row * a.lddh, cols, t, o);
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row0 = (int64_t)blockIdx.x * RPB;
  if (row0 < a.rows) fetch(row0 + group);
  for (; row0 < a.rows; row0 += step) {
    const int64_t row = row0 + group;
    uint4 hc[NV], gc[NV], oc[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) hc[j] = h[j], gc[j] = g[j], oc[j] = a.dh ? o[j] : zero4();
    if (row0 + step < a.rows) fetch(row + step);
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float x = R::value(hc[j], e);
        ss = fmaf(x, x, ss);
        sg = fmaf(R::value(gc[j], e) * w[j][e], x, sg);
      }
    const float2 s = row_sum2<GS>(ss, sg, mine, t);
    const float f = rsqrtf(s.x / (float)a.cols + a.eps), k = f * f * (s.y / (float)a.cols);
    if (row >= a.rows) continue;
    float dx[NV][VE];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        const float x = R::value(hc[j], e), y = R::value(gc[j], e);
        dw[j][e] = fmaf(y, x * f, dw[j][e]);
        dx[j][e] = f * (y * w[j][e] - x * k) + R::value(oc[j], e);
      }
    R::store(a.dx + row * a.lddx, a.cols, t, dx);
  }
  if (!a.part) return;
  if constexpr (RPB > 1) {
    for (int q = 1; q < RPB; ++q) {
      __syncthreads();
      if (group == q) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VE; ++e) sums[(j * VE + e) * GS + t] = dw[j][e];
      }
      __syncthreads();
      if (group == 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < VE; ++e) dw[j][e] += sums[(j * VE + e) * GS + t];
      }
    }
    if (group != 0) return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (R::col(j, t) + e < a.cols) a.part[(int64_t)blockIdx.x * a.cols + R::col(j, t) + e] = dw[j][e];
}

// dw[c] = the sum of part[0 .. n - 1][c]: 32 threads a column, a fixed order
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* part, float* dw, int n, int cols) {
  __shared__ float lds[32][33];
  const int x = threadIdx.x % 32, r = threadIdx.x / 32, c = blockIdx.x * 32 + x;
  float s = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int i = r; i < n; i += 32) s += part[(int64_t)i * cols + c];
  lds[r][x] = s;
  __syncthreads();
  if (r == 0 && c < cols) {
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) y += lds[i][x];
    dw[c] = y;
  }
}

}  // namespace lact
