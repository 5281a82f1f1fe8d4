// Norms of queries and keys for each head with the position rotation in the same
// pass, and their gradients.
//
//   n = x rstd, rstd = 1 / sqrt(mean x^2 + eps);  u = n w + bias[head];  hat = M^T u
// (M: the de-rotation of the moments path). Gradients, with d = the cotangent of hat:
//   du = M d;  d_bias = sum du;  dn = w sum_{heads of the group} du;  d_w = sum n (..)
//   d_x = rstd (dn - n mean(dn n))
//   d_angle = sum (hat_x d_y - hat_y d_x) over its pair;  d_Q = sum u (x) conj(d)
// over channels and over both q and k (and over all heads where they turn alike).
//
// All of it is streaming: each row of 2 to 128 values is one or a few 16-byte pieces
// per lane, LPR lanes a row and eight values a lane, so that pairs and quaternion
// blocks lie in one lane (half-split rows give a lane four values of each half). A
// wave's 64 / LPR row slots are the heads of one group (HPP of them, HL times) by
// tokens: angles are evaluated once for the 2c rows that share them, the group's raw
// row is read once, and sums over its heads stay in the wave.
#pragma once

#include "common.h"
#include "kernels_rot.h"

#include <type_traits>

namespace mom {

constexpr int QKT = 256;

struct QkGeo {
  int b, s, c, h, g, r;
  size_t qs, ks;    // elements between tokens of q and k
  int rot_h, RW, A, J;
  int hpg, HPP, HL; // heads per group; head slots of a wave; times they are filled
  int nblk;         // workgroups per group (backward)
  float eps, rinv;  // added to the mean square; 1 / r
};

// Column of value e (0..7) of lane l of a row.
template <bool HALF>
__device__ __forceinline__ int qk_col(int l, int e, int r) {
  return HALF ? (e < 4 ? 4 * l + e : (r >> 1) + 4 * l + e - 4) : 8 * l + e;
}
template <bool HALF>
__device__ __forceinline__ bool qk_has(int l, int e, int r) {
  return HALF ? 4 * l + (e & 3) < (r >> 1) : 8 * l + e < r;
}

template <typename T, bool HALF>
__device__ __forceinline__ void ld8(const T* row, int l, int r, bool vec, float (&v)[8]) {
  if (vec) {
    const bool in = HALF ? 4 * l < (r >> 1) : 8 * l < r;
    if (!in) {
      for (int e = 0; e < 8; e++) v[e] = 0.0f;
    } else if constexpr (HALF) {
      const f4 a = ld4(row + 4 * l), b = ld4(row + (r >> 1) + 4 * l);
      for (int e = 0; e < 4; e++) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    } else if constexpr (sizeof(T) == 2) {
      ldv(row + 8 * l, v);
    } else {
      const f4 a = ld4(row + 8 * l), b = ld4(row + 8 * l + 4);
      for (int e = 0; e < 4; e++) {
        v[e] = a[e];
        v[4 + e] = b[e];
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++) v[e] = qk_has<HALF>(l, e, r) ? to_f(row[qk_col<HALF>(l, e, r)]) : 0.0f;
  }
}
template <typename T, bool HALF>
__device__ __forceinline__ void st8(T* row, int l, int r, bool vec, const float (&v)[8]) {
  if (vec) {
    const bool in = HALF ? 4 * l < (r >> 1) : 8 * l < r;
    if (!in) return;
    if constexpr (HALF) {
      st4(row + 4 * l, f4{v[0], v[1], v[2], v[3]});
      st4(row + (r >> 1) + 4 * l, f4{v[4], v[5], v[6], v[7]});
    } else if constexpr (sizeof(T) == 2) {
      stv(row + 8 * l, v);
    } else {
      st4(row + 8 * l, f4{v[0], v[1], v[2], v[3]});
      st4(row + 8 * l + 4, f4{v[4], v[5], v[6], v[7]});
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; e++)
      if (qk_has<HALF>(l, e, r)) row[qk_col<HALF>(l, e, r)] = to_t<T>(v[e]);
  }
}

// A lane's eight values of a row, in flight: as loaded from memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 v;
  template <bool HALF>
  __device__ __forceinline__ void load(const bf16* row, int l, int r, bool vec) {
    if (vec) {
      v = make_uint4(0, 0, 0, 0);
      if (HALF ? 4 * l >= (r >> 1) : 8 * l >= r) return;
      if constexpr (HALF) {
        const uint2 a = *reinterpret_cast<const uint2*>(row + 4 * l);
        const uint2 b = *reinterpret_cast<const uint2*>(row + (r >> 1) + 4 * l);
        v = make_uint4(a.x, a.y, b.x, b.y);
      } else {
        v = *reinterpret_cast<const uint4*>(row + 8 * l);
      }
    } else {
      bf16 e[8];
#pragma unroll
      for (int i = 0; i < 8; i++) e[i] = qk_has<HALF>(l, i, r) ? row[qk_col<HALF>(l, i, r)] : (bf16)0.0f;
      v = __builtin_bit_cast(uint4, e);
    }
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      o[2 * i] = bf16_lo(w[i]);
      o[2 * i + 1] = bf16_hi(w[i]);
    }
  }
};
template <>
struct Raw8<float> {
  float v[8];
  template <bool HALF>
  __device__ __forceinline__ void load(const float* row, int l, int r, bool vec) { ld8<float, HALF>(row, l, r, vec, v); }
  __device__ __forceinline__ void zero() {
    for (int i = 0; i < 8; i++) v[i] = 0.0f;
  }
  __device__ __forceinline__ void get(float (&o)[8]) const {
    for (int i = 0; i < 8; i++) o[i] = v[i];
  }
};

// Sine and cosine. The nearest multiple of pi/2 (FAST: the whole turns) is taken off, below
// 1e5 in three floats, which hold pi/2 to 2^-76 (FAST: in two), else in doubles, which reach
// to 2^50; beyond, neighbouring floats are 2^27 radians apart, and the rest is taken as zero.
// FAST (bf16 results): the rest, up to half a turn (from 1e5 on the quarters are put back, up
// to a whole one), goes through the sine and cosine instructions, whose error of about 2^-20
// is far below the result's rounding of 2^-9; otherwise, at most pi/4, through the Taylor
// series to x^9 and x^10 (the next terms are below 2^-28). Evaluated for bf16 rows the series
// costs 80 more instructions a lane and head.
template <bool FAST, bool BIG>
__device__ __forceinline__ void sincos_f(float x, float& s, float& c) {
  constexpr double kPi2 = 1.5707963267948966, kPi2Lo = 6.123233995736766e-17;   // pi/2: double and remainder
  constexpr float P1 = (float)kPi2, P2 = (float)(kPi2 - (double)P1),
                  P3 = (float)(kPi2 - (double)P1 - (double)P2 + kPi2Lo);
  float t;
  int n = 0;
  if constexpr (!BIG) {
    // FAST takes off whole turns
    const float k = FAST ? 4.0f * rintf(x * 0.159154943091895336f) : rintf(x * 0.636619772367581343f);
    t = fmaf(-k, P2, fmaf(-k, P1, x));
    if constexpr (!FAST) {
      t = fmaf(-k, P3, t);
      n = (int)k;
    }
  } else {
    const double k = rint((double)x * 0.6366197723675814);
    const double d = fma(-k, kPi2Lo, fma(-k, kPi2, (double)x));
    t = fabs(d) <= 1.0 ? (float)d : x - x;   // zero; NaN for infinities and NaN
    n = (int)(k - 4.0 * floor(0.25 * k));
    if constexpr (FAST) t += (float)n * P1;
  }
  if constexpr (FAST) {
    const float turns = t * 0.159154943091895336f;
    s = __builtin_amdgcn_sinf(turns);
    c = __builtin_amdgcn_cosf(turns);
  } else {
    const float t2 = t * t;
    float a = fmaf(t2, 2.75573192e-6f, -1.98412698e-4f);
    a = fmaf(t2, a, 8.33333333e-3f);
    a = fmaf(t2, a, -1.66666667e-1f);
    a = fmaf(t2 * t, a, t);
    float b = fmaf(t2, -2.75573192e-7f, 2.48015873e-5f);
    b = fmaf(t2, b, -1.38888889e-3f);
    b = fmaf(t2, b, 4.16666667e-2f);
    b = fmaf(t2, b, -0.5f);
    b = fmaf(t2, b, 1.0f);
    const float u = (n & 1) ? b : a, v = (n & 1) ? a : b;
    s = (n & 2) ? -u : u;
    c = ((n + 1) & 2) ? -v : v;
  }
}

// The rotation of one (token, head) as a lane needs it: ROT 1, 2: cos and sin of its
// four angles; ROT 3: its two quaternions. Blocks past the rotated width are identity.
template <int ROT>
struct QkRot {
  float v[ROT == 0 ? 1 : 8];
  template <bool VEC, typename T>
  __device__ __forceinline__ void load(const T* row, int l, const QkGeo& g) {
    if constexpr (ROT == 1 || ROT == 2) {
      if (VEC) {
        f4 t = {0.0f, 0.0f, 0.0f, 0.0f};
        if (4 * l < g.A) t = ld4(row + 4 * l);
        for (int i = 0; i < 4; i++) v[i] = t[i];
      } else {
        for (int i = 0; i < 4; i++) v[i] = 4 * l + i < g.A ? to_f(row[4 * l + i]) : 0.0f;
      }
    } else if constexpr (ROT == 3) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        f4 t = {1.0f, 0.0f, 0.0f, 0.0f};
        if (2 * l + i < g.J) t = ld4(row + 4 * (2 * l + i));
        for (int e = 0; e < 4; e++) v[4 * i + e] = t[e];
      }
    }
  }
  // Angles to their cosines and sines.
  template <bool FAST>
  __device__ __forceinline__ void make(int l, const QkGeo& g) {
    if constexpr (ROT == 1 || ROT == 2) {
      // angles past the rotated width were loaded as zero: the identity
      const float big = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
      if (big < 1e5f) {
#pragma unroll
        for (int i = 0; i < 4; i++) sincos_f<FAST, false>(v[i], v[4 + i], v[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; i++) sincos_f<FAST, true>(v[i], v[4 + i], v[i]);
      }
    }
  }
  // TR: M^T u (queries and keys); otherwise M u (their cotangents).
  template <bool TR>
  __device__ __forceinline__ void turn(float (&u)[8]) const {
    if constexpr (ROT == 1 || ROT == 2) {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int ex = ROT == 1 ? 2 * i : i, ey = ROT == 1 ? 2 * i + 1 : i + 4;
        const float c = v[i], s = TR ? v[4 + i] : -v[4 + i], x = u[ex], y = u[ey];
        u[ex] = x * c - y * s;
        u[ey] = x * s + y * c;
      }
    } else if constexpr (ROT == 3) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        const f4 q = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
        const f4 z = qmul(TR ? qconj(q) : q, f4{u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]});
        for (int e = 0; e < 4; e++) u[4 * i + e] = z[e];
      }
    }
  }
};

// Sums over the LPR lanes of a row, and over the first `n` (a power of two) row slots
// of each n in a wave; every lane gets the sum.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<QP_SWAP1>(v);
  v += dpp<QP_X2>(v);
  v += dpp<DPP_ROW_HALF_MIRROR>(v);
  if constexpr (LPR == 16) v += dpp<DPP_ROW_MIRROR>(v);
  return v;
}
template <int LPR>
__device__ __forceinline__ float slot_sum(float v, int n) {
  if constexpr (LPR == 8) {
    if (n > 1) v += dpp<0x128>(v);   // rotate the 16 lanes of a row by 8
    n >>= 1;
  }
  if (n > 1) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  if (n > 2) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  }
  return v;
}

// Sums of N rows over the n head slots of a token, each slot left with its share of the
// rows: after it, v[0 .. N / n - 1] (v[0] where n >= N) are the rows from qk_own_row() on. The swaps
// of gfx950 move two rows at once, so a row costs half a swap and half an add per step
// instead of a full exchange; where slots outnumber rows, several hold the same one.
__host__ __device__ __forceinline__ int qk_own_row(int N, int n, int hs) {
  // head slots split the rows from the widest step down
  int row = 0;
  for (int d = n / 2, m = N; d >= 1 && m > 1; d /= 2, m /= 2)
    if (hs & d) row += m / 2;
  return row;
}
// Whether this slot is the one that writes its rows (the first of those that share them).
__host__ __device__ __forceinline__ bool qk_own_writes(int N, int n, int hs) { return n <= N || (hs & (n / N - 1)) == 0; }
// D: head slots apart in this step; M: rows that the slot holds before it.
template <int LPR, int D, int M, int N>
__device__ __forceinline__ void slot_scatter(float (&v)[N][8], int lane) {
  if constexpr (D >= 1) {
    constexpr int H = M > 1 ? M / 2 : 1;
#pragma unroll
    for (int i = 0; i < H; i++)
#pragma unroll
      for (int e = 0; e < 8; e++) {
        const float a = v[i][e], b = M > 1 ? v[i + M / 2][e] : a;
        if constexpr (D * LPR == 32) {
          const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
          v[i][e] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        } else if constexpr (D * LPR == 16) {
          const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
          v[i][e] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        } else {   // 8 lanes: rotate the 16 lanes of a row by 8
          const bool hi = lane & 8;
          v[i][e] = (hi ? b : a) + dpp<0x128>(hi ? a : b);
        }
      }
    slot_scatter<LPR, D / 2, H, N>(v, lane);
  }
}

// 1 / sqrt(v): the instruction, right to one unit in the last place, which is of the size of
// the sum's and the products' own roundings (float rows use it too). It takes subnormal
// inputs for zero: those are brought into its range by a power of two, and back.
__device__ __forceinline__ float recip_sqrt(float v) {
  const bool small = v < 0x1p-100f;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v) * (small ? 0x1p32f : 1.0f);
}

// C: channels padded to 1, 2 or 4. HB: heads per row slot whose bias stays in registers
// (0: HL is larger, it is read again for each token). VEC: rows, their strides and the
// angles are whole 16-byte pieces (8 bytes, bf16 angles); others go one element at a time.
// A wave takes tokens a grid apart, with the next one's rows already in flight.
// Bound by memory, most of it what it writes: bf16, 8 x 8192 tokens of two channels, 64 heads
// in 8 groups, r = 128: 5.1 GB in 1.15 to 1.31 ms, 1.24 on average (4.1 TB/s; a large copy 4.75).
// float32, 2 x 2048 tokens, 16 heads, r = 64: 24 us.
template <typename T, int LPR, int ROT, int C, int HB, bool VEC>
__global__ __launch_bounds__(QKT) void k_qk_fwd(QkGeo g, const T* __restrict__ q, const T* __restrict__ k,
                                                const float* __restrict__ wq, const float* __restrict__ wk,
                                                const float* __restrict__ bq, const float* __restrict__ bk,
                                                const T* __restrict__ rot, T* __restrict__ qhat,
                                                T* __restrict__ khat) {
  constexpr bool HALF = ROT == 2;
  constexpr int RPW = 64 / LPR, NB = HB > 0 ? HB : 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPR, slot = lane / LPR;
  const int gi = blockIdx.y, TPW = RPW / g.HPP, hs = slot % g.HPP, ts = slot / g.HPP;
  const size_t ntok = (size_t)g.b * g.s, step = (size_t)gridDim.x * (QKT / 64) * TPW;
  float w[2][8], bv[2][NB][8];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    ld8<float, HALF>(x ? wk : wq, l, g.r, VEC, w[x]);
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const int hg = i * g.HPP + hs;
      const float* bias = x ? bk : bq;
      for (int e = 0; e < 8; e++) bv[x][i][e] = 0.0f;
      if (HB > 0 && bias != nullptr && hg < g.hpg)
        ld8<float, HALF>(bias + (size_t)(gi * g.hpg + hg) * g.r, l, g.r, VEC, bv[x][i]);
    }
  }
  Raw8<T> raw[2][C];
  QkRot<ROT> R0[NB];
  auto fetch = [&](size_t tok) {
    const bool live = tok < ntok;
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        raw[x][c].zero();
        if (live && c < g.c)
          raw[x][c].template load<HALF>((x ? k : q) + tok * (x ? g.ks : g.qs) + ((size_t)c * g.g + gi) * g.r, l, g.r,
                                        VEC);
      }
    if constexpr (ROT != 0 && HB > 0) {
#pragma unroll
      for (int i = 0; i < NB; i++) {
        const int hg = i * g.HPP + hs;
        if (live && hg < g.hpg)
          R0[i].template load<VEC>(rot + (tok * g.rot_h + (g.rot_h > 1 ? gi * g.hpg + hg : 0)) * g.RW, l, g);
      }
    }
  };
  size_t t0 = ((size_t)blockIdx.x * (QKT / 64) + wave) * TPW;
  if (t0 < ntok) fetch(t0 + ts);
  for (; t0 < ntok; t0 += step) {
    const size_t tok = t0 + ts;
    float n[2][C][8];
    QkRot<ROT> R[NB];
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) raw[x][c].get(n[x][c]);
#pragma unroll
    for (int i = 0; i < NB; i++) R[i] = R0[i];
    if (t0 + step < ntok) fetch(tok + step);
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (c >= g.c) break;
        float ss = 0.0f;
        for (int e = 0; e < 8; e++) ss += n[x][c][e] * n[x][c][e];
        const float rstd = recip_sqrt(row_sum<LPR>(ss) * g.rinv + g.eps);
        for (int e = 0; e < 8; e++) n[x][c][e] *= rstd * w[x][e];
      }
    auto head = [&](int hg, QkRot<ROT>& Rh, auto bias) {
      const int hi = gi * g.hpg + hg;
      Rh.template make<sizeof(T) == 2>(l, g);
#pragma unroll
      for (int x = 0; x < 2; x++) {
        float b8[8];
        bias(x, hi, b8);
#pragma unroll
        for (int c = 0; c < C; c++) {
          if (c >= g.c) break;
          float u[8];
          for (int e = 0; e < 8; e++) u[e] = n[x][c][e] + b8[e];
          Rh.template turn<true>(u);
          st8<T, HALF>((x ? khat : qhat) + ((tok * g.c + c) * g.h + hi) * g.r, l, g.r, VEC, u);
        }
      }
    };
    if (tok >= ntok) continue;
    if constexpr (HB > 0) {
#pragma unroll
      for (int i = 0; i < NB; i++)
        if (i * g.HPP + hs < g.hpg)
          head(i * g.HPP + hs, R[i], [&](int x, int, float (&b8)[8]) {
            for (int e = 0; e < 8; e++) b8[e] = bv[x][i][e];
          });
    } else {
      for (int i = 0; i < g.HL; i++) {
        const int hg = i * g.HPP + hs;
        if (hg >= g.hpg) break;
        if constexpr (ROT != 0)
          R[0].template load<VEC>(rot + (tok * g.rot_h + (g.rot_h > 1 ? gi * g.hpg + hg : 0)) * g.RW, l, g);
        head(hg, R[0], [&](int x, int hi, float (&b8)[8]) {
          for (int e = 0; e < 8; e++) b8[e] = 0.0f;
          const float* bias = x ? bk : bq;
          if (bias != nullptr) ld8<float, HALF>(bias + (size_t)hi * g.r, l, g.r, VEC, b8);
        });
      }
    }
  }
}

// One row's share of the gradients: d, the cotangent of its hat, becomes du and is added
// to sb (the head's) and ds (the group's); the rotation's goes to dr.
template <int ROT>
__device__ __forceinline__ void qk_row_grad(const QkRot<ROT>& R, const float (&n)[8], const float (&w)[8],
                                            const float (&b)[8], float (&d)[8], float (&dr)[8], float (&sb)[8],
                                            float (&ds)[8]) {
  if constexpr (ROT == 3) {
#pragma unroll
    for (int j = 0; j < 2; j++) {
      f4 u;
      for (int e = 0; e < 4; e++) u[e] = n[4 * j + e] * w[4 * j + e] + b[4 * j + e];
      const f4 z = qmul(u, qconj(f4{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]}));
      for (int e = 0; e < 4; e++) dr[4 * j + e] += z[e];
    }
  }
  R.template turn<false>(d);
  if constexpr (ROT == 1 || ROT == 2) {
    // in the frame before the turn: u_x du_y - u_y du_x (turning both keeps it)
#pragma unroll
    for (int j = 0; j < 4; j++) {
      const int ex = ROT == 1 ? 2 * j : j, ey = ROT == 1 ? 2 * j + 1 : j + 4;
      dr[j] += (n[ex] * w[ex] + b[ex]) * d[ey] - (n[ey] * w[ey] + b[ey]) * d[ex];
    }
  }
  for (int e = 0; e < 8; e++) {
    sb[e] += d[e];
    ds[e] += d[e];
  }
}

// HB: heads per row slot (1, 2) whose sums of du stand in registers; 0: any number, they
// stand in LDS, one place per thread and head. part_b [2][nblk][h][r], part_w
// [2][nblk][g][r]; part_rot [b,s,g][RW] where all heads share a rotation (d_rot is then
// their sum over g). HPP: head slots of a token (all a wave has, with HB = 0 or 2).
// Registers decide: about 230, so two waves per SIMD, whose loads are issued when their token
// starts; neither the vector pipes (64 % busy) nor memory (3.5 TB/s) is at its end. Sizes as at
// k_qk_fwd: 5.9 GB in 1.65 to 1.81 ms, 1.69 on average, and 48 us in float32. Queries and keys
// one after the other need fewer registers but more passes (1.71 ms where this took 1.63); a
// launch bound of three or four waves spills.
template <typename T, int LPR, int ROT, int C, int HB, int HPP, bool VEC>
__global__ __launch_bounds__(QKT) void k_qk_bwd(QkGeo g, const T* __restrict__ q, const T* __restrict__ k,
                                                const float* __restrict__ wq, const float* __restrict__ wk,
                                                const float* __restrict__ bq, const float* __restrict__ bk,
                                                const T* __restrict__ rot, const T* __restrict__ dqh,
                                                const T* __restrict__ dkh, T* __restrict__ d_q, T* __restrict__ d_k,
                                                T* __restrict__ d_rot, float* __restrict__ part_rot,
                                                float* __restrict__ part_w, float* __restrict__ part_b) {
  constexpr bool HALF = ROT == 2, LDSB = HB == 0;
  constexpr int RPW = 64 / LPR, TPW = RPW / HPP, NB = HB > 0 ? HB : 1, NR = ROT == 3 ? 8 : 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  float* acc = reinterpret_cast<float*>(lds);   // LDSB: [HL][16][threads]; then the block's sums
  const int NT = blockDim.x, NWV = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPR, slot = lane / LPR;
  const int gi = blockIdx.y, hs = slot % HPP, ts = slot / HPP;
  const size_t ntok = (size_t)g.b * g.s;
  float w[2][8], dw[2][8], db[2][NB][8];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    ld8<float, HALF>(x ? wk : wq, l, g.r, VEC, w[x]);
    for (int e = 0; e < 8; e++) dw[x][e] = 0.0f;
    for (int i = 0; i < NB; i++)
      for (int e = 0; e < 8; e++) db[x][i][e] = 0.0f;
  }
  if constexpr (LDSB) {
    for (int i = 0; i < g.HL * 16; i++) acc[i * NT + threadIdx.x] = 0.0f;
  }
  auto raw_row = [&](int x, int c, size_t tok) {
    return (x ? k : q) + tok * (x ? g.ks : g.qs) + ((size_t)c * g.g + gi) * g.r;
  };
  auto hat_row = [&](int x, int c, size_t tok, int hi) { return (x ? dkh : dqh) + ((tok * g.c + c) * g.h + hi) * g.r; };
  auto rot_row = [&](size_t tok, int hi) { return (tok * g.rot_h + (g.rot_h > 1 ? hi : 0)) * g.RW; };
  auto ld_bias = [&](int x, int hi, float (&b8)[8]) {
    const float* bias = x ? bk : bq;
    for (int e = 0; e < 8; e++) b8[e] = 0.0f;
    if (bias != nullptr) ld8<float, HALF>(bias + (size_t)hi * g.r, l, g.r, VEC, b8);
  };
  // A row slot without a row (past the last token) has rstd = 0: with eps = 0 its zeros would
  // become 0 * inf = NaN, which the sums of d_w would take up.
  auto norm = [&](float (&n)[8], bool live) {
    float ss = 0.0f;
    for (int e = 0; e < 8; e++) ss += n[e] * n[e];
    const float ms = row_sum<LPR>(ss) * g.rinv + g.eps;
    const float rstd = live ? recip_sqrt(ms) : 0.0f;
    for (int e = 0; e < 8; e++) n[e] *= rstd;
    return rstd;
  };
  // the group's raw rows 0 .. 2C - 1 (q's channels, then k's), from the sums of du over its
  // heads: each head slot finishes its share of them, and sums d_w for q or k by its rows
  constexpr int N = 2 * C;
  constexpr int own = N > HPP ? N / HPP : 1;
  const int orow = qk_own_row(N, HPP, hs);
  const bool writes = qk_own_writes(N, HPP, hs);
  auto finish = [&](size_t tok, bool live, const float (&n)[N][8], const float (&rstd)[N], float (&ds)[N][8]) {
    slot_scatter<LPR, HPP / 2, N, N>(ds, lane);
#pragma unroll
    for (int i = 0; i < own; i++) {
      const int row = orow + i, x = row / C, c = row % C;
      float nn[8], rs = 0.0f, m = 0.0f, wx[8];
#pragma unroll
      for (int j = i; j < N; j += own) {            // row j is this slot's
        const bool is = j == row;
        rs = is ? rstd[j] : rs;
        for (int e = 0; e < 8; e++) nn[e] = j == i || is ? n[j][e] : nn[e];
      }
#pragma unroll
      for (int e = 0; e < 8; e++) {
        wx[e] = x ? w[1][e] : w[0][e];
        const float t = ds[i][e] * nn[e];
        if constexpr (own > C) {                    // one slot for both q and k
          dw[i / C][e] += t;
        } else {
          dw[0][e] += t;
        }
        ds[i][e] *= wx[e];
        m += ds[i][e] * nn[e];
      }
      m = row_sum<LPR>(m) * g.rinv;
      T* out = x ? d_k : d_q;
      if (live && writes && c < g.c && out != nullptr) {
        float o[8];
        for (int e = 0; e < 8; e++) o[e] = (ds[i][e] - nn[e] * m) * rs;
        st8<T, HALF>(out + ((tok * g.c + c) * g.g + gi) * g.r, l, g.r, VEC, o);
      }
    }
  };
  // the rotation's: one head's own, or the group's share of the one for all heads
  auto st_rot = [&](size_t tok, int hi, const float (&dr)[8]) {
    if (d_rot == nullptr) return;
    T* o = d_rot + rot_row(tok, hi);
    if constexpr (ROT == 3) {
      for (int j = 0; j < 2; j++)
        if (2 * l + j < g.J) st4(o + 4 * (2 * l + j), f4{dr[4 * j], dr[4 * j + 1], dr[4 * j + 2], dr[4 * j + 3]});
    } else if (VEC) {
      if (4 * l < g.A) st4(o + 4 * l, f4{dr[0], dr[1], dr[2], dr[3]});
    } else {
      for (int j = 0; j < 4; j++)
        if (4 * l + j < g.A) o[4 * l + j] = to_t<T>(dr[j]);
    }
  };
  auto st_rot1 = [&](size_t tok, bool live, float (&dr)[8]) {
#pragma unroll
    for (int e = 0; e < NR; e++) dr[e] = slot_sum<LPR>(dr[e], HPP);
    if (live && hs == 0) {
      float* o = part_rot + (tok * g.g + gi) * g.RW;
      for (int e = 0; e < NR; e++)
        if (NR * l + e < g.RW) o[NR * l + e] = dr[e];
    }
  };
  for (size_t t0 = ((size_t)blockIdx.x * NWV + wave) * TPW; t0 < ntok; t0 += (size_t)g.nblk * NWV * TPW) {
    const size_t tok = t0 + ts;
    const bool live = tok < ntok;
    if constexpr (!LDSB) {
      // every load of the token first
      Raw8<T> raw[2][C], hat[2][NB][C];
      QkRot<ROT> R[NB];
      float dr[NB][8];
      bool on[NB];
#pragma unroll
      for (int x = 0; x < 2; x++)
#pragma unroll
        for (int c = 0; c < C; c++) {
          raw[x][c].zero();
          if (live && c < g.c) raw[x][c].template load<HALF>(raw_row(x, c, tok), l, g.r, VEC);
        }
#pragma unroll
      for (int i = 0; i < NB; i++) {
        const int hg = i * HPP + hs, hi = gi * g.hpg + hg;
        on[i] = live && hg < g.hpg;
        for (int e = 0; e < 8; e++) dr[i][e] = 0.0f;
        if constexpr (ROT != 0)
          if (on[i]) R[i].template load<VEC>(rot + rot_row(tok, hi), l, g);
#pragma unroll
        for (int x = 0; x < 2; x++)
#pragma unroll
          for (int c = 0; c < C; c++) {
            hat[x][i][c].zero();
            if (on[i] && c < g.c) hat[x][i][c].template load<HALF>(hat_row(x, c, tok, hi), l, g.r, VEC);
          }
      }
#pragma unroll
      for (int i = 0; i < NB; i++)
        if constexpr (ROT != 0)
          if (on[i]) R[i].template make<sizeof(T) == 2>(l, g);
      float n[N][8], ds[N][8], rstd[N];
#pragma unroll
      for (int x = 0; x < 2; x++) {
#pragma unroll
        for (int c = 0; c < C; c++) {
          const int j = x * C + c;
          raw[x][c].get(n[j]);
          rstd[j] = c < g.c ? norm(n[j], live) : 0.0f;
          for (int e = 0; e < 8; e++) ds[j][e] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < NB; i++) {
          if (!on[i]) continue;
          float b8[8];
          if constexpr (ROT != 0) ld_bias(x, gi * g.hpg + i * HPP + hs, b8);
#pragma unroll
          for (int c = 0; c < C; c++) {
            if (c >= g.c) break;
            float d[8];
            hat[x][i][c].get(d);
            qk_row_grad<ROT>(R[i], n[x * C + c], w[x], b8, d, dr[i], db[x][i], ds[x * C + c]);
          }
        }
      }
      finish(tok, live, n, rstd, ds);
      if constexpr (ROT != 0) {
        if (part_rot != nullptr) {
#pragma unroll
          for (int i = 1; i < NB; i++)
            for (int e = 0; e < NR; e++) dr[0][e] += dr[i][e];
          st_rot1(tok, live, dr[0]);
        } else {
#pragma unroll
          for (int i = 0; i < NB; i++)
            if (on[i]) st_rot(tok, gi * g.hpg + i * HPP + hs, dr[i]);
        }
      }
    } else {
      float n[N][8], ds[N][8], rstd[N], dr1[8];
#pragma unroll
      for (int x = 0; x < 2; x++)
#pragma unroll
        for (int c = 0; c < C; c++) {
          const int j = x * C + c;
          for (int e = 0; e < 8; e++) n[j][e] = ds[j][e] = 0.0f;
          if (live && c < g.c) ld8<T, HALF>(raw_row(x, c, tok), l, g.r, VEC, n[j]);
          rstd[j] = c < g.c ? norm(n[j], live) : 0.0f;
        }
      for (int e = 0; e < 8; e++) dr1[e] = 0.0f;
      for (int i = 0; i < g.HL; i++) {
        const int hg = i * HPP + hs, hi = gi * g.hpg + hg;
        if (!live || hg >= g.hpg) continue;
        QkRot<ROT> R;
        if constexpr (ROT != 0) {
          R.template load<VEC>(rot + rot_row(tok, hi), l, g);
          R.template make<sizeof(T) == 2>(l, g);
        }
        float dr[8];
        for (int e = 0; e < 8; e++) dr[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < 2; x++) {
          float b8[8], sb[8];
          ld_bias(x, hi, b8);
          for (int e = 0; e < 8; e++) sb[e] = 0.0f;
#pragma unroll
          for (int c = 0; c < C; c++) {
            if (c >= g.c) break;
            float d[8];
            ld8<T, HALF>(hat_row(x, c, tok, hi), l, g.r, VEC, d);
            qk_row_grad<ROT>(R, n[x * C + c], w[x], b8, d, dr, sb, ds[x * C + c]);
          }
#pragma unroll
          for (int e = 0; e < 8; e++) acc[(i * 16 + 8 * x + e) * NT + threadIdx.x] += sb[e];
        }
        if constexpr (ROT != 0) {
          if (part_rot == nullptr) st_rot(tok, hi, dr);
          for (int e = 0; e < 8; e++) dr1[e] += dr[e];
        }
      }
      if constexpr (ROT != 0)
        if (part_rot != nullptr) st_rot1(tok, live, dr1);
      finish(tok, live, n, rstd, ds);
    }
  }
  // the block's sums, in a fixed order: over the token slots of its waves. src [16][threads];
  // heads hs0 + (head slot) of the group, or (isw) d_w, over the head slots that own rows of
  // q (of k) and write them
  const int NTS = NWV * TPW;
  float* red = acc + (LDSB ? (size_t)g.HL * 16 * NT : 0);
  auto sum_block = [&](const float* src, int hs0, bool isw) {
    float* part = isw ? part_w : part_b;
    if (part == nullptr) return;
    for (int id = threadIdx.x; id < HPP * 16 * LPR; id += NT) {
      const int ll = id % LPR, ve = id / LPR % 16, hh = id / (16 * LPR), x = ve / 8, e = ve % 8;
      if (!qk_has<HALF>(ll, e, g.r) || (isw ? hh > 0 : hs0 + hh >= g.hpg)) continue;
      double s = 0.0;
      for (int t = 0; t < NTS; t++) {
        const int th = (t / TPW) * 64 + (t % TPW) * HPP * LPR + ll;
        if (!isw) {
          s += (double)src[ve * NT + th + hh * LPR];
        } else {
          for (int o = 0; o < HPP; o++) {
            if (!qk_own_writes(N, HPP, o)) continue;
            if (own > C) s += (double)src[ve * NT + th + o * LPR];
            else if (qk_own_row(N, HPP, o) / C == x) s += (double)src[e * NT + th + o * LPR];
          }
        }
      }
      const size_t row = isw ? ((size_t)x * g.nblk + blockIdx.x) * g.g + gi
                             : ((size_t)x * g.nblk + blockIdx.x) * g.h + gi * g.hpg + hs0 + hh;
      part[row * g.r + qk_col<HALF>(ll, e, g.r)] = (float)s;
    }
  };
  auto to_red = [&](const float (&v)[2][8]) {
    __syncthreads();
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int e = 0; e < 8; e++) red[(8 * x + e) * NT + threadIdx.x] = v[x][e];
    __syncthreads();
  };
  if constexpr (LDSB) {
    __syncthreads();
    for (int i = 0; i < g.HL; i++) sum_block(acc + (size_t)i * 16 * NT, i * HPP, false);
  } else {
#pragma unroll
    for (int i = 0; i < NB; i++) {
      float v[2][8];
      for (int x = 0; x < 2; x++)
        for (int e = 0; e < 8; e++) v[x][e] = db[x][i][e];
      to_red(v);
      sum_block(red, i * HPP, false);
    }
  }
  to_red(dw);
  sum_block(red, 0, true);
}

// The sums of the blocks' partials, in double and in a fixed order: d_w over the n_w
// rows of part_w [2][n_w][r], d_b over the n_b rows of part_b [2][n_b][hr]. A workgroup
// takes 16 columns of one of them, 64 threads each. 12 us beside 1.69 ms of k_qk_bwd.
__global__ __launch_bounds__(1024) void k_qk_sum(const float* __restrict__ part_w, int n_w, int r,
                                                 float* __restrict__ d_wq, float* __restrict__ d_wk,
                                                 const float* __restrict__ part_b, int n_b, int hr,
                                                 float* __restrict__ d_bq, float* __restrict__ d_bk, int cols) {
  __shared__ double red[64][17];
  const int wb = (r + 15) / 16, x = blockIdx.y, j = threadIdx.x >> 4;
  for (int cb = blockIdx.x; cb < cols; cb += gridDim.x) {
    const bool isw = cb < wb;
    const float* part = isw ? part_w : part_b;
    const int n = isw ? n_w : n_b, w = isw ? r : hr;
    float* out = isw ? (x ? d_wk : d_wq) : (x ? d_bk : d_bq);
    if (out == nullptr) continue;   // all threads alike
    const int e = (cb - (isw ? 0 : wb)) * 16 + (int)(threadIdx.x & 15);
    double s = 0.0;
    if (e < w) {
      const float* src = part + (size_t)x * n * w + e;
#pragma unroll 8
      for (int i = j; i < n; i += 64) s += (double)src[(size_t)i * w];
    }
    red[j][threadIdx.x & 15] = s;
    __syncthreads();
    if (j == 0 && e < w) {
      for (int i = 1; i < 64; i++) s += red[i][threadIdx.x];
      out[e] = (float)s;
    }
    __syncthreads();   // read before the next columns' sums are written
  }
}

}  // namespace mom
