// Layer norm of rows, with the residual stream added before it, and its gradients: kernels.
//
//   s = x (+ res),  d = s - mean(s),  y = d rstd weight (+ bias),  rstd = 1 / sqrt(mean(d^2) + eps)
//   gy = d_y weight,  d_s = rstd (gy - mean(gy) - xhat mean(gy xhat)) (+ d_sum),  xhat = d rstd
//   d_weight = sum of d_y xhat over the rows,  d_bias = sum of d_y
//
// A row lies in the registers of NT threads, E elements each, and is read once. Threads take pieces of
// eight neighbouring elements wherever they stand in memory: loads and stores of 16 bytes need no
// alignment here (the compiler is told that there is none), only the last piece of a row whose width
// is not a multiple of eight goes element by element. The mean is taken
// twice: the first, of s, may be off by the rounding of a sum of large values, so the second
// reduction carries sum(d) beside sum(d^2) and what is left of the mean leaves d and the variance.
// The gradients make the statistics again, with their own two sums in that same reduction, so
// nothing is kept from the forward.
//
// Bound by memory: 65536 x 4096 bf16 with a residual, forward 602 us (3.2 GB, 5.3 TB/s), gradients
// 822 us (4.3 GB, 5.2 TB/s) and 8 us for the sums over rows. A row has 8 to 64 threads of eight
// elements up to w = 512 (several rows to a wave: 1e6 x 100 bf16, forward and gradients 667 us, a
// wave to a row 1215), then 16 elements. Streamed loads or stores: forward 655 and 670 us. Threads
// being powers of two, widths just past one leave up to half of them idle (20000 x 8200 bf16,
// forward and gradients 1136 us, 807 at the copy rate), rows below 64 columns more (4e6 x 8, one
// thread of eight: 620 us, 157 at the copy rate).
#pragma once

#include "common.h"

namespace mom {

struct LnGeo {
  int64_t n;
  int w;
  size_t xs;    // elements between rows of x
  float eps, winv;
};

constexpr float kLnScale = 8.271806125530277e-25f;   // 2^-80

// Columns of a thread: 8-element pieces, NT pieces apart.
template <int NT> __device__ __forceinline__ int ln_col(int i, int tid) { return ((i >> 3) * NT + tid) * 8 + (i & 7); }

// Eight elements from an address of theirs on.
struct __attribute__((packed, aligned(2))) LnWord2 { u4 v; };
struct __attribute__((packed, aligned(4))) LnWord4 { f4 v; };
__device__ __forceinline__ void ln_get8(float* v, const bf16* p) {
  const u4 r = reinterpret_cast<const LnWord2*>(p)->v;
#pragma unroll
  for (int j = 0; j < 4; j++) v[2 * j] = bf16_lo(r[j]), v[2 * j + 1] = bf16_hi(r[j]);
}
__device__ __forceinline__ void ln_get8(float* v, const float* p) {
  const f4 r0 = reinterpret_cast<const LnWord4*>(p)->v, r1 = reinterpret_cast<const LnWord4*>(p + 4)->v;
#pragma unroll
  for (int j = 0; j < 4; j++) v[j] = r0[j], v[4 + j] = r1[j];
}
__device__ __forceinline__ void ln_put8(bf16* p, const float* v) {
  u4 r;
#pragma unroll
  for (int j = 0; j < 4; j++) r[j] = pk_bf16(v[2 * j], v[2 * j + 1]);
  reinterpret_cast<LnWord2*>(p)->v = r;
}
__device__ __forceinline__ void ln_put8(float* p, const float* v) {
  f4 r0, r1;
#pragma unroll
  for (int j = 0; j < 4; j++) r0[j] = v[j], r1[j] = v[4 + j];
  reinterpret_cast<LnWord4*>(p)->v = r0;
  reinterpret_cast<LnWord4*>(p + 4)->v = r1;
}

// A thread's elements of a row. `past`: the memory goes on far enough behind the row that its last
// piece can be read whole; what stands there is in v then, past the row's end.
template <typename T, int NT, int E>
__device__ __forceinline__ void ln_load(float (&v)[E], const T* p, int w, int tid, bool past) {
#pragma unroll
  for (int k = 0; k < E / 8; k++) {
    const int c = (k * NT + tid) * 8;
    if (past ? c < w : c + 8 <= w) {
      ln_get8(v + 8 * k, p + c);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++) v[8 * k + j] = 0.0f;
      if (!past)
#pragma unroll
        for (int j = 0; j < 8; j++)
          if (c + j < w) v[8 * k + j] = to_f(p[c + j]);
    }
  }
}
// Whether that is so of a row of a tensor whose rows are `stride` elements apart.
__device__ __forceinline__ bool ln_past(const LnGeo& g, int64_t row, size_t stride) {
  return (size_t)(g.n - 1 - row) * stride + (size_t)g.w >= (size_t)((g.w + 7) & ~7);
}

template <typename T, int NT, int E>
__device__ __forceinline__ void ln_store(T* p, const float (&v)[E], int w, int tid) {
#pragma unroll
  for (int k = 0; k < E / 8; k++) {
    const int c = (k * NT + tid) * 8;
    if (c + 8 <= w) {
      ln_put8(p + c, v + 8 * k);
    } else {
#pragma unroll
      for (int j = 0; j < 8; j++)
        if (c + j < w) p[c + j] = to_t<T>(v[8 * k + j]);
    }
  }
}

// Sums over the NT threads of a row, in a fixed order; every thread gets them. Up to 64 threads are
// neighbours in a wave. Consecutive calls of more alternate between two places in LDS, so one
// barrier each is enough.
template <int NT> struct LnSum {
  float* lds;   // [2][NT / 64][4]
  int buf = 0;
  static __device__ __forceinline__ float lanes(float v) {
    v += dpp<QP_SWAP1>(v);
    v += dpp<QP_X2>(v);
    v += dpp<DPP_ROW_HALF_MIRROR>(v);
    if constexpr (NT >= 16) v += dpp<DPP_ROW_MIRROR>(v);
    if constexpr (NT == 32) {
      const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
      v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    }
    if constexpr (NT >= 64) v = col4_sum(v);
    return v;
  }
  template <int M> __device__ __forceinline__ void operator()(float (&v)[M]) {
#pragma unroll
    for (int i = 0; i < M; i++) v[i] = lanes(v[i]);
    if constexpr (NT > 64) {
      float* at = lds + buf * (NT / 64) * 4;
      buf ^= 1;
      if ((threadIdx.x & 63) == 0)
#pragma unroll
        for (int i = 0; i < M; i++) at[(threadIdx.x >> 6) * 4 + i] = v[i];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < M; i++) v[i] = at[i];
#pragma unroll
      for (int k = 1; k < NT / 64; k++)
#pragma unroll
        for (int i = 0; i < M; i++) v[i] += at[k * 4 + i];
    }
  }
};

// d = scale (s - mean), zero past the row's end, and the row's sums: m[0] of what is left of the
// mean, m[1] of d^2, with GY also m[2] of gy = dy wt and m[3] of gy d. d and the sums are of the
// centred row. The first mean is taken about s0, the row's first value, so that a row of one value
// is centred to exact zeros, however large it is.
template <int NT, int E, bool GY, class Sum>
__device__ __forceinline__ void ln_center(const LnGeo& g, const float (&s)[E], const float (&dy)[E],
                                          const float (&wt)[E], float s0, float scale, float (&d)[E],
                                          float (&m)[GY ? 4 : 2], int tid, Sum& sum) {
  float one[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < E; i++)
    if (ln_col<NT>(i, tid) < g.w) one[0] = fmaf(fmaf(s[i], scale, -s0 * scale), g.winv, one[0]);
  sum(one);
  const float mean = fmaf(s0, scale, one[0]);
#pragma unroll
  for (int i = 0; i < (GY ? 4 : 2); i++) m[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < E; i++) {
    d[i] = ln_col<NT>(i, tid) < g.w ? fmaf(s[i], scale, -mean) : 0.0f;
    m[0] += d[i];
    m[1] = fmaf(d[i], d[i], m[1]);
    if constexpr (GY) {
      const float gy = ln_col<NT>(i, tid) < g.w ? dy[i] * wt[i] : 0.0f;
      m[2] += gy;
      m[3] = fmaf(gy, d[i], m[3]);
    }
  }
  sum(m);
  const float off = m[0] * g.winv;
#pragma unroll
  for (int i = 0; i < E; i++) d[i] = ln_col<NT>(i, tid) < g.w ? d[i] - off : 0.0f;
  m[1] = fmaf(-off, m[0], m[1]);
  if (m[1] < 0.0f) m[1] = 0.0f;   // NaN stays
  if constexpr (GY) m[3] = fmaf(-off, m[2], m[3]);
}

// The row's d and the rstd that goes with it. A row whose squares (or differences) overflow is
// centred again at 2^-80 of its size, where eps is nothing beside them; one that holds an infinity
// or a NaN stays NaN.
template <int NT, int E, bool GY, class Sum>
__device__ __forceinline__ float ln_stats(const LnGeo& g, const float (&s)[E], const float (&dy)[E],
                                          const float (&wt)[E], float s0, float (&d)[E], float (&m)[GY ? 4 : 2],
                                          float& scale, int tid, Sum& sum) {
  scale = 1.0f;
  float eps = g.eps;
  ln_center<NT, E, GY>(g, s, dy, wt, s0, scale, d, m, tid, sum);
  if (!(m[1] < __builtin_inff())) {   // the same for all threads of the row
    scale = kLnScale;
    eps = 0.0f;
    ln_center<NT, E, GY>(g, s, dy, wt, s0, scale, d, m, tid, sum);
  }
  return 1.0f / sqrtf(fmaf(m[1], g.winv, eps));
}

// Rows are dealt to the workgroups, 256 / NT at a time where NT is less, one after the other.
template <typename T, int NT, int E, bool RES>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_ln_fwd(LnGeo g, const T* __restrict__ x, const float* res,
                                                                const float* __restrict__ weight,
                                                                const float* __restrict__ bias, T* __restrict__ y,
                                                                float* total) {
  constexpr int RPB = NT <= 64 ? 256 / NT : 1;
  __shared__ float lds[NT > 64 ? NT / 64 * 8 : 1];
  const int tid = NT <= 64 ? (int)threadIdx.x % NT : (int)threadIdx.x, at = NT <= 64 ? (int)threadIdx.x / NT : 0;
  LnSum<NT> sum{lds};
  float wt[E], bs[E];
  ln_load<float, NT, E>(wt, weight, g.w, tid, false);
  if (bias != nullptr) {
    ln_load<float, NT, E>(bs, bias, g.w, tid, false);
  } else {
#pragma unroll
    for (int i = 0; i < E; i++) bs[i] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t row = (int64_t)blockIdx.x * RPB + at; row < g.n; row += step) {
    float s[E], d[E], m[2], scale, s0 = to_f(x[(size_t)row * g.xs]);
    const bool past = ln_past(g, row, (size_t)g.w);
    ln_load<T, NT, E>(s, x + (size_t)row * g.xs, g.w, tid, ln_past(g, row, g.xs));
    if constexpr (RES) {
      float r[E];
      s0 += res[(size_t)row * g.w];
      ln_load<float, NT, E>(r, res + (size_t)row * g.w, g.w, tid, past);
#pragma unroll
      for (int i = 0; i < E; i++) s[i] += r[i];
    }
    const float rstd = ln_stats<NT, E, false>(g, s, s, s, s0, d, m, scale, tid, sum);
    // behind the row's sums, which need every thread's s0: `total` may be `res`
    if constexpr (RES) ln_store<float, NT, E>(total + (size_t)row * g.w, s, g.w, tid);
#pragma unroll
    for (int i = 0; i < E; i++) d[i] = fmaf(d[i] * rstd, wt[i], bs[i]);
    ln_store<T, NT, E>(y + (size_t)row * g.w, d, g.w, tid);
  }
}

// part: a row of w sums for each workgroup, of d_weight, then of d_bias (NULL: neither is wanted).
// A thread adds its rows' values one after the other in float32, n / 768 of them at w = 4096, n / 24576
// up to w = 64: the sums are off by at most that many times 2^-24 of the values' magnitudes together;
// what the workgroups leave is added in double.
// TS: of the normed rows (float where a residual was added). With E = 32 elements a thread's 2 E
// sums stand in LDS (ln_wide_lds bytes) and the weights are loaded for each row: 16384 x 16384 bf16
// with residual 947 us at 1024 threads of 16 elements, whose 128 registers do not hold them. It
// still spills 28 to 42 registers (116 to 172 bytes of scratch a lane).
template <int NT, int E> constexpr size_t ln_wide_lds = E == 32 ? (size_t)2 * E * NT * 4 : 0;
template <typename T, typename TS, int NT, int E>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_ln_bwd(LnGeo g, const TS* __restrict__ x,
                                                                const float* __restrict__ weight,
                                                                const T* __restrict__ dy, const float* d_sum,
                                                                T* __restrict__ d_x, float* d_res,
                                                                float* __restrict__ part) {
  constexpr int RPB = NT <= 64 ? 256 / NT : 1;
  constexpr bool HOLD = E < 32;
  extern __shared__ float acc[];   // [2][E][NT]
  __shared__ float lds[NT > 64 ? NT / 64 * 8 : 256 * E];
  const int tid = NT <= 64 ? (int)threadIdx.x % NT : (int)threadIdx.x, at = NT <= 64 ? (int)threadIdx.x / NT : 0;
  LnSum<NT> sum{lds};
  float held[HOLD ? E : 1], dw[E], db[E];
  if constexpr (HOLD) ln_load<float, NT, E>(held, weight, g.w, tid, false);
#pragma unroll
  for (int i = 0; i < E; i++) {
    dw[i] = db[i] = 0.0f;
    if constexpr (!HOLD) acc[i * NT + tid] = acc[(E + i) * NT + tid] = 0.0f;
  }
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t row = (int64_t)blockIdx.x * RPB + at; row < g.n; row += step) {
    float s[E], v[E], d[E], wt[E], m[4], scale;
    const bool past = ln_past(g, row, (size_t)g.w);
    const float s0 = to_f(x[(size_t)row * g.xs]);
    ln_load<TS, NT, E>(s, x + (size_t)row * g.xs, g.w, tid, ln_past(g, row, g.xs));
    ln_load<T, NT, E>(v, dy + (size_t)row * g.w, g.w, tid, past);
    if constexpr (HOLD) {
#pragma unroll
      for (int i = 0; i < E; i++) wt[i] = held[i];
    } else {
      ln_load<float, NT, E>(wt, weight, g.w, tid, false);
    }
    const float rstd = ln_stats<NT, E, true>(g, s, v, wt, s0, d, m, scale, tid, sum);
    const float m1 = m[2] * g.winv, m2 = m[3] * g.winv * rstd, rs = rstd * scale;
#pragma unroll
    for (int i = 0; i < E; i++) {
      const float xhat = d[i] * rstd;
      if constexpr (HOLD) {
        db[i] += v[i];
        dw[i] = fmaf(v[i], xhat, dw[i]);
      } else {   // the thread's own places
        acc[(E + i) * NT + tid] += v[i];
        acc[i * NT + tid] = fmaf(v[i], xhat, acc[i * NT + tid]);
      }
      d[i] = rs * (fmaf(v[i], wt[i], -m1) - xhat * m2);
    }
    if (d_sum != nullptr) {
      ln_load<float, NT, E>(s, d_sum + (size_t)row * g.w, g.w, tid, past);
#pragma unroll
      for (int i = 0; i < E; i++) d[i] += s[i];
    }
    if (d_x != nullptr) ln_store<T, NT, E>(d_x + (size_t)row * g.w, d, g.w, tid);
    if (d_res != nullptr) ln_store<float, NT, E>(d_res + (size_t)row * g.w, d, g.w, tid);
  }
  if (part == nullptr) return;
  if constexpr (!HOLD)
#pragma unroll
    for (int i = 0; i < E; i++) dw[i] = acc[i * NT + tid], db[i] = acc[(E + i) * NT + tid];
  float* pw = part + (size_t)blockIdx.x * g.w;
  float* pb = pw + (size_t)gridDim.x * g.w;
  if constexpr (RPB > 1) {   // the rows' places first
    for (int k = 0; k < 2; k++) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < E; i++) lds[(at * E + i) * NT + tid] = k == 0 ? dw[i] : db[i];
      __syncthreads();
      if (at == 0) {
        float v[E];
#pragma unroll
        for (int i = 0; i < E; i++) {
          v[i] = lds[i * NT + tid];
          for (int q = 1; q < RPB; q++) v[i] += lds[(q * E + i) * NT + tid];
        }
        ln_store<float, NT, E>(k == 0 ? pw : pb, v, g.w, tid);
      }
    }
  } else {
    ln_store<float, NT, E>(pw, dw, g.w, tid);
    ln_store<float, NT, E>(pb, db, g.w, tid);
  }
}

// The parameters' gradients from np partial rows each (zeros for none), summed in double: 64
// columns a workgroup, its 16 waves take every 16th row. blockIdx.y: 0 d_weight, 1 d_bias.
__global__ __launch_bounds__(1024) void k_ln_sum(const float* __restrict__ part, int np, int w, float* d_weight,
                                                 float* d_bias) {
  __shared__ double lds[16][64];
  float* out = blockIdx.y == 0 ? d_weight : d_bias;
  if (out == nullptr) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = (int)blockIdx.x * 64 + lane;
  double s = 0.0;
  if (c < w) {
    const float* p = part + (size_t)blockIdx.y * np * w + c;
#pragma unroll 8
    for (int k = wave; k < np; k += 16) s += (double)p[(size_t)k * w];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= w) return;
  for (int k = 1; k < 16; k++) s += lds[k][lane];
  out[c] = (float)s;
}

}  // namespace mom
