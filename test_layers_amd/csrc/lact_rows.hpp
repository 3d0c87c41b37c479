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
  int32_t tok, head_groups;  // tokens and head groups of a workgroup
  float mscale;
  int32_t inverse;
};

constexpr int ROT_TABLE = 2048;  // pairs of one workgroup's table

// (x, y) -> mscale (x cos - y sin, x sin + y cos) for the features (i, i + n)
// or (2 i, 2 i + 1), the rest copied.  A workgroup first fills a table of the
// angles of its tokens, in fp64 turns: a far position times a frequency needs
// all of a double's bits before whole turns are dropped.  All heads of q and
// k then use the table.
template <typename T, int VE, bool INTERLEAVED>
__global__ __launch_bounds__(256) void rotary_kernel(RotaryArgs a) {
  __shared__ float cs[ROT_TABLE], sn[ROT_TABLE];
  const int groups = (a.L + a.tok - 1) / a.tok;
  int id = blockIdx.x;
  const int hg = id % a.head_groups;
  id /= a.head_groups;
  const int t0 = (id % groups) * a.tok, b = id / groups;
  const int nt = min(a.tok, a.L - t0), n = a.pairs;
  for (int i = threadIdx.x; i < nt * n; i += 256) {
    const int t = t0 + i / n;
    const double pos = (double)(a.positions ? a.positions[(int64_t)b * a.L + t] : a.start + t);
    double turn = pos * (a.freqs[i % n] * 0.15915494309189533577);  // / (2 pi)
    turn -= rint(turn);
    float s, c;
    if constexpr (sizeof(T) == 4) {
      sincospif(2.f * (float)turn, &s, &c);
    } else {
      // the hardware's sine of turns: off by less than 2^-16, far below a bf16 step
      s = __builtin_amdgcn_sinf((float)turn);
      c = __builtin_amdgcn_cosf((float)turn);
    }
    cs[i] = c * a.mscale;
    sn[i] = (a.inverse ? -s : s) * a.mscale;
  }
  __syncthreads();
  // items of a row: pairs by VE (half layout) or VE / 2, then the copied rest
  constexpr int PV = INTERLEAVED ? (VE > 1 ? VE / 2 : 1) : VE;
  const int turned = n / PV, rest = (a.d - 2 * n) / VE, per = turned + rest;
  const int heads = a.t[0].heads + a.t[1].heads;
  const int h0 = (int)((int64_t)heads * hg / a.head_groups), h1 = (int)((int64_t)heads * (hg + 1) / a.head_groups);
  const int items = nt * (h1 - h0) * per;
  const bool heads_inner = a.t[0].ih < a.t[0].il;  // neighbours in memory go to neighbouring lanes
  for (int i = threadIdx.x; i < items; i += 256) {
    const int c = i % per, r = i / per;
    const int t = heads_inner ? r / (h1 - h0) : r % nt;
    int h = h0 + (heads_inner ? r % (h1 - h0) : r / nt);
    const RotaryTensor& x = h < a.t[0].heads ? a.t[0] : a.t[1];
    if (h >= a.t[0].heads) h -= a.t[0].heads;
    const T* in = reinterpret_cast<const T*>(x.in + b * x.ib + h * x.ih + (int64_t)(t0 + t) * x.il);
    T* out = reinterpret_cast<T*>(x.out + b * x.ob + h * x.oh + (int64_t)(t0 + t) * x.ol);
    if (c >= turned) {
      if (in != out) {
        float v[VE];
        const int e = 2 * n + (c - turned) * VE;
        load_n<T, VE>(in + e, v);
        store_n<T, VE>(out + e, v);
      }
    } else if constexpr (INTERLEAVED && VE > 1) {
      float v[VE];
      load_n<T, VE>(in + c * VE, v);
#pragma unroll
      for (int j = 0; j < VE; j += 2) {
        const float co = cs[t * n + c * PV + j / 2], si = sn[t * n + c * PV + j / 2];
        const float x0 = v[j], x1 = v[j + 1];
        v[j] = x0 * co - x1 * si;
        v[j + 1] = x0 * si + x1 * co;
      }
      store_n<T, VE>(out + c * VE, v);
    } else {
      const int e0 = INTERLEAVED ? 2 * c : c * VE, e1 = INTERLEAVED ? e0 + 1 : e0 + n;
      float u[VE], v[VE];
      load_n<T, VE>(in + e0, u);
      load_n<T, VE>(in + e1, v);
#pragma unroll
      for (int j = 0; j < VE; ++j) {
        const float co = cs[t * n + c * PV + j], si = sn[t * n + c * PV + j];
        const float x0 = u[j], x1 = v[j];
        u[j] = x0 * co - x1 * si;
        v[j] = x0 * si + x1 * co;
      }
      store_n<T, VE>(out + e0, u);
      store_n<T, VE>(out + e1, v);
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

// one thread's NV vectors of a row: vector j holds columns (j GS + t) VE ..
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
      if constexpr (VEC) {
        if (c < cols) load_n<T, VE>(p, v[j]);
      } else {
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
  __device__ static __forceinline__ void store(char* row, int cols, int t, const float (&v)[NV][VE]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = col(j, t);
      T* p = reinterpret_cast<T*>(row) + c;
      if constexpr (VEC) {
        if (c < cols) store_n<T, VE>(p, v[j]);
      } else {
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
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) v[j][e] = col(j, t) + e < cols ? w[col(j, t) + e] : 0.f;
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
// A workgroup takes every gridDim-th row and keeps its dw in registers; the
// workgroups' partial sums are added in a fixed order by norm_dw_kernel.
template <typename T, int NV, int GS, bool VEC>
__global__ __launch_bounds__(GS) void norm_back_kernel(NormArgs a) {
  using R = NormRow<T, NV, GS, VEC>;
  constexpr int VE = R::VE;
  __shared__ float2 lds[GS / WAVE];
  const int t = threadIdx.x;
  float w[NV][VE], dw[NV][VE];
  R::weights(a.w, a.cols, t, w);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e) dw[j][e] = 0.f;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float h[NV][VE], g[NV][VE];
    R::load(a.x + row * a.ldx, a.cols, t, h);
    R::load(a.dy + row * a.ldg, a.cols, t, g);
    float ss = 0.f, sg = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        ss = fmaf(h[j][e], h[j][e], ss);
        sg = fmaf(g[j][e] * w[j][e], h[j][e], sg);
      }
    const float2 s = row_sum2<GS>(ss, sg, lds, t);
    const float f = rsqrtf(s.x / (float)a.cols + a.eps), k = f * f * (s.y / (float)a.cols);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        dw[j][e] = fmaf(g[j][e], h[j][e] * f, dw[j][e]);
        h[j][e] = f * (g[j][e] * w[j][e] - h[j][e] * k);
      }
    if (a.dh) {
      R::load(a.dh + row * a.lddh, a.cols, t, g);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < VE; ++e) h[j][e] += g[j][e];
    }
    R::store(a.dx + row * a.lddx, a.cols, t, h);
  }
  if (!a.part) return;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VE; ++e)
      if (R::col(j, t) + e < a.cols) a.part[(int64_t)blockIdx.x * a.cols + R::col(j, t) + e] = dw[j][e];
}

// dw[c] = the sum of part[0 .. n - 1][c]: 16 threads a column, a fixed order
__global__ __launch_bounds__(1024) void norm_dw_kernel(const float* part, float* dw, int n, int cols) {
  __shared__ float lds[16][64];
  const int c = blockIdx.x * 64 + threadIdx.x % 64, r = threadIdx.x / 64;
  float s = 0.f;
  if (c < cols)
    for (int i = r; i < n; i += 16) s += part[(int64_t)i * cols + c];
  lds[r][threadIdx.x % 64] = s;
  __syncthreads();
  if (r == 0 && c < cols) {
    float x = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) x += lds[i][threadIdx.x];
    dw[c] = x;
  }
}

}  // namespace lact
