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

namespace mom {

constexpr int QKT = 256;

struct QkGeo {
  int b, s, c, h, g, r;
  size_t qs, ks;    // elements between tokens of q and k
  int rot_h, RW, A, J;
  int hpg, HPP, HL; // heads per group; head slots of a wave; times they are filled
  int vin, vio, vrot;  // 16-byte pieces: raw rows, hat rows, angles
  int nblk;         // workgroups per group (backward)
  float eps;
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

// Sine and cosine, to fp32 rounding for |x| < 1e5: the nearest multiple of pi/2 is
// taken off with pi/2 in three floats, and the rest, at most pi/4, goes through the
// Taylor series to x^9 and x^10 (the next terms are below 2^-28). Larger angles go
// to the library's functions.
__device__ __forceinline__ void sincos_f(float x, float& s, float& c) {
  if (fabsf(x) < 1e5f) {
    const float k = rintf(x * 0.636619772367581343f);
    constexpr double kPi2 = 1.5707963267948966;
    constexpr float P1 = (float)kPi2, P2 = (float)(kPi2 - (double)P1);
    constexpr float P3 = 6.123233995736766e-17f;   // pi/2 beyond a double
    float t = fmaf(-k, P1, x);
    t = fmaf(-k, P2, t);
    t = fmaf(-k, P3, t);
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
    const int n = (int)k;
    const float u = (n & 1) ? b : a, v = (n & 1) ? a : b;
    s = (n & 2) ? -u : u;
    c = ((n + 1) & 2) ? -v : v;
  } else {
    sincosf(x, &s, &c);
  }
}

// The rotation of one (token, head) as a lane needs it: ROT 1, 2: cos and sin of its
// four angles; ROT 3: its two quaternions. Blocks past the rotated width are identity.
template <typename T, int ROT>
struct QkRot {
  float v[ROT == 0 ? 1 : 8];
  __device__ __forceinline__ void load(const T* row, int l, const QkGeo& g) {
    if constexpr (ROT == 1 || ROT == 2) {
      float a[4];
      if (g.vrot) {
        f4 t = {0.0f, 0.0f, 0.0f, 0.0f};
        if (4 * l < g.A) t = ld4(row + 4 * l);
        for (int i = 0; i < 4; i++) a[i] = t[i];
      } else {
        for (int i = 0; i < 4; i++) a[i] = 4 * l + i < g.A ? to_f(row[4 * l + i]) : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 4; i++) sincos_f(a[i], v[4 + i], v[i]);
    } else if constexpr (ROT == 3) {
#pragma unroll
      for (int i = 0; i < 2; i++) {
        f4 t = {1.0f, 0.0f, 0.0f, 0.0f};
        if (2 * l + i < g.J) t = ld4(row + 4 * (2 * l + i));
        for (int e = 0; e < 4; e++) v[4 * i + e] = t[e];
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

// One row, normed: n = x rstd.
template <typename T, bool HALF, int LPR>
__device__ __forceinline__ float ld_norm(const T* row, int l, const QkGeo& g, bool vec, float (&n)[8]) {
  ld8<T, HALF>(row, l, g.r, vec, n);
  float ss = 0.0f;
  for (int e = 0; e < 8; e++) ss += n[e] * n[e];
  const float rstd = 1.0f / sqrtf(row_sum<LPR>(ss) / (float)g.r + g.eps);
  for (int e = 0; e < 8; e++) n[e] *= rstd;
  return rstd;
}

// C: channels padded to 1, 2 or 4.
template <typename T, int LPR, int ROT, int C>
__global__ __launch_bounds__(QKT) void k_qk_fwd(QkGeo g, const T* __restrict__ q, const T* __restrict__ k,
                                                const float* __restrict__ wq, const float* __restrict__ wk,
                                                const float* __restrict__ bq, const float* __restrict__ bk,
                                                const T* __restrict__ rot, T* __restrict__ qhat,
                                                T* __restrict__ khat) {
  constexpr bool HALF = ROT == 2;
  constexpr int RPW = 64 / LPR;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPR, slot = lane / LPR;
  const int gi = blockIdx.y, TPW = RPW / g.HPP, hs = slot % g.HPP;
  const size_t tok = ((size_t)blockIdx.x * (QKT / 64) + wave) * TPW + slot / g.HPP;
  // whole waves of tokens past the end leave; single slots stay for the sums over lanes
  const bool live = tok < (size_t)g.b * g.s;
  float n[2][C][8], w[2][8];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    ld8<float, HALF>(x ? wk : wq, l, g.r, false, w[x]);
#pragma unroll
    for (int c = 0; c < C; c++) {
      const T* row = (x ? k : q) + tok * (x ? g.ks : g.qs) + ((size_t)c * g.g + gi) * g.r;
      if (live && c < g.c) {
        ld8<T, HALF>(row, l, g.r, g.vin, n[x][c]);
      } else {
        for (int e = 0; e < 8; e++) n[x][c][e] = 0.0f;
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 2; x++)
#pragma unroll
    for (int c = 0; c < C; c++) {
      float ss = 0.0f;
      for (int e = 0; e < 8; e++) ss += n[x][c][e] * n[x][c][e];
      const float rstd = 1.0f / sqrtf(row_sum<LPR>(ss) / (float)g.r + g.eps);
      for (int e = 0; e < 8; e++) n[x][c][e] *= rstd * w[x][e];
    }
  if (!live) return;
  for (int i = 0; i < g.HL; i++) {
    const int hg = i * g.HPP + hs;
    if (hg >= g.hpg) return;
    const int hi = gi * g.hpg + hg;
    QkRot<T, ROT> R;
    if constexpr (ROT != 0) R.load(rot + (tok * g.rot_h + (g.rot_h > 1 ? hi : 0)) * g.RW, l, g);
#pragma unroll
    for (int x = 0; x < 2; x++) {
      const float* bias = x ? bk : bq;
      float bv[8];
      for (int e = 0; e < 8; e++) bv[e] = 0.0f;
      if (bias != nullptr) ld8<float, HALF>(bias + (size_t)hi * g.r, l, g.r, false, bv);
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (c >= g.c) break;
        float u[8];
        for (int e = 0; e < 8; e++) u[e] = n[x][c][e] + bv[e];
        R.template turn<true>(u);
        st8<T, HALF>((x ? khat : qhat) + ((tok * g.c + c) * g.h + hi) * g.r, l, g.r, g.vio, u);
      }
    }
  }
}

// LDSB: the sums of du for each head stand in LDS (HL > 1), one place per thread and
// head; otherwise in registers. part_b [2][nblk][h][r], part_w [2][nblk][g][r]; part_rot
// [b,s,g][RW] where all heads share a rotation (d_rot is then their sum over g).
template <typename T, int LPR, int ROT, int C, bool LDSB>
__global__ __launch_bounds__(QKT) void k_qk_bwd(QkGeo g, const T* __restrict__ q, const T* __restrict__ k,
                                                const float* __restrict__ wq, const float* __restrict__ wk,
                                                const float* __restrict__ bq, const float* __restrict__ bk,
                                                const T* __restrict__ rot, const T* __restrict__ dqh,
                                                const T* __restrict__ dkh, T* __restrict__ d_q, T* __restrict__ d_k,
                                                T* __restrict__ d_rot, float* __restrict__ part_rot,
                                                float* __restrict__ part_w, float* __restrict__ part_b) {
  constexpr bool HALF = ROT == 2;
  constexpr int RPW = 64 / LPR;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  float* acc = reinterpret_cast<float*>(lds);   // LDSB: [HL][16][threads]; then the block's sums
  const int NT = blockDim.x, NWV = NT / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l = lane % LPR, slot = lane / LPR;
  const int gi = blockIdx.y, TPW = RPW / g.HPP, hs = slot % g.HPP, ts = slot / g.HPP;
  const size_t ntok = (size_t)g.b * g.s;
  float w[2][8], bv[2][8], dw[2][8], db[2][8];
#pragma unroll
  for (int x = 0; x < 2; x++) {
    ld8<float, HALF>(x ? wk : wq, l, g.r, false, w[x]);
    for (int e = 0; e < 8; e++) dw[x][e] = db[x][e] = bv[x][e] = 0.0f;
  }
  if constexpr (LDSB) {
    for (int i = 0; i < g.HL * 16; i++) acc[i * NT + threadIdx.x] = 0.0f;
  }
  for (size_t t0 = ((size_t)blockIdx.x * NWV + wave) * TPW; t0 < ntok; t0 += (size_t)g.nblk * NWV * TPW) {
    const size_t tok = t0 + ts;
    const bool live = tok < ntok;
    float n[2][C][8], rstd[2][C], ds[2][C][8];
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        const T* row = (x ? k : q) + tok * (x ? g.ks : g.qs) + ((size_t)c * g.g + gi) * g.r;
        if (live && c < g.c) {
          ld8<T, HALF>(row, l, g.r, g.vin, n[x][c]);
        } else {
          for (int e = 0; e < 8; e++) n[x][c][e] = 0.0f;
        }
        for (int e = 0; e < 8; e++) ds[x][c][e] = 0.0f;
      }
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        float ss = 0.0f;
        for (int e = 0; e < 8; e++) ss += n[x][c][e] * n[x][c][e];
        rstd[x][c] = 1.0f / sqrtf(row_sum<LPR>(ss) / (float)g.r + g.eps);
        for (int e = 0; e < 8; e++) n[x][c][e] *= rstd[x][c];
      }
    float dr1[8];   // d_rot over the heads of the group (rot_h = 1)
    for (int e = 0; e < 8; e++) dr1[e] = 0.0f;
    for (int i = 0; i < g.HL; i++) {
      const int hg = i * g.HPP + hs;
      if (!live || hg >= g.hpg) continue;
      const int hi = gi * g.hpg + hg;
      QkRot<T, ROT> R;
      const size_t rrow = (tok * g.rot_h + (g.rot_h > 1 ? hi : 0)) * g.RW;
      if constexpr (ROT != 0) R.load(rot + rrow, l, g);
      float dr[8];
      for (int e = 0; e < 8; e++) dr[e] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; x++) {
        if constexpr (ROT == 3) {
          const float* bias = x ? bk : bq;
          if (bias != nullptr) ld8<float, HALF>(bias + (size_t)hi * g.r, l, g.r, false, bv[x]);
        }
        float sb[8];
        for (int e = 0; e < 8; e++) sb[e] = 0.0f;
#pragma unroll
        for (int c = 0; c < C; c++) {
          if (c >= g.c) break;
          float d[8];
          ld8<T, HALF>((x ? dkh : dqh) + ((tok * g.c + c) * g.h + hi) * g.r, l, g.r, g.vio, d);
          if constexpr (ROT == 3) {
#pragma unroll
            for (int j = 0; j < 2; j++) {
              f4 u;
              for (int e = 0; e < 4; e++) u[e] = n[x][c][4 * j + e] * w[x][4 * j + e] + bv[x][4 * j + e];
              const f4 z = qmul(u, qconj(f4{d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]}));
              for (int e = 0; e < 4; e++) dr[4 * j + e] += z[e];
            }
          }
          R.template turn<false>(d);
          if constexpr (ROT == 1 || ROT == 2) {
            // in the frame before the turn: u_x du_y - u_y du_x (turning both keeps it)
            const float* bias = x ? bk : bq;
            if (c == 0 && bias != nullptr) ld8<float, HALF>(bias + (size_t)hi * g.r, l, g.r, false, bv[x]);
#pragma unroll
            for (int j = 0; j < 4; j++) {
              const int ex = ROT == 1 ? 2 * j : j, ey = ROT == 1 ? 2 * j + 1 : j + 4;
              const float ux = n[x][c][ex] * w[x][ex] + bv[x][ex], uy = n[x][c][ey] * w[x][ey] + bv[x][ey];
              dr[j] += ux * d[ey] - uy * d[ex];
            }
          }
          for (int e = 0; e < 8; e++) {
            sb[e] += d[e];
            ds[x][c][e] += d[e];
          }
        }
        if constexpr (LDSB) {
#pragma unroll
          for (int e = 0; e < 8; e++) acc[(i * 16 + 8 * x + e) * NT + threadIdx.x] += sb[e];
        } else {
          for (int e = 0; e < 8; e++) db[x][e] += sb[e];
        }
      }
      if constexpr (ROT != 0) {
        if (g.rot_h > 1 || g.h == 1) {
          if (d_rot != nullptr) {
            T* o = d_rot + rrow;
            if constexpr (ROT == 3) {
              for (int j = 0; j < 2; j++)
                if (2 * l + j < g.J) st4(o + 4 * (2 * l + j), f4{dr[4 * j], dr[4 * j + 1], dr[4 * j + 2], dr[4 * j + 3]});
            } else if (g.vrot) {
              if (4 * l < g.A) st4(o + 4 * l, f4{dr[0], dr[1], dr[2], dr[3]});
            } else {
              for (int j = 0; j < 4; j++)
                if (4 * l + j < g.A) o[4 * l + j] = to_t<T>(dr[j]);
            }
          }
        } else {
          for (int e = 0; e < 8; e++) dr1[e] += dr[e];
        }
      }
    }
    if constexpr (ROT != 0) {
      if (part_rot != nullptr) {
#pragma unroll
        for (int e = 0; e < (ROT == 3 ? 8 : 4); e++) dr1[e] = slot_sum<LPR>(dr1[e], g.HPP);
        if (live && hs == 0) {
          float* o = part_rot + (tok * g.g + gi) * g.RW;
          for (int e = 0; e < (ROT == 3 ? 8 : 4); e++) {
            const int at = (ROT == 3 ? 8 : 4) * l + e;
            if (at < g.RW) o[at] = dr1[e];
          }
        }
      }
    }
    // the group's raw rows
#pragma unroll
    for (int x = 0; x < 2; x++)
#pragma unroll
      for (int c = 0; c < C; c++) {
        if (c >= g.c) break;
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) {
          const float s = slot_sum<LPR>(ds[x][c][e], g.HPP);
          dw[x][e] += s * n[x][c][e];
          ds[x][c][e] = s * w[x][e];
          m += ds[x][c][e] * n[x][c][e];
        }
        m = row_sum<LPR>(m) / (float)g.r;
        T* out = x ? d_k : d_q;
        if (live && hs == 0 && out != nullptr) {
          float o[8];
          for (int e = 0; e < 8; e++) o[e] = (ds[x][c][e] - n[x][c][e] * m) * rstd[x][c];
          st8<T, HALF>(out + ((tok * g.c + c) * g.g + gi) * g.r, l, g.r, g.vio, o);
        }
      }
  }
  // the block's sums, in a fixed order: over the token slots of its waves
  __syncthreads();
  const int NTS = NWV * TPW;   // token slots of the block
  float* red = acc + (LDSB ? (size_t)g.HL * 16 * NT : 0);   // [16][threads]
  for (int i = 0; i < (LDSB ? g.HL : 1) + 1; i++) {
    const bool isw = i == (LDSB ? g.HL : 1);   // last: d_w, equal in all head slots
    float* src = LDSB && !isw ? acc + (size_t)i * 16 * NT : red;
    if (!LDSB || isw) {
      __syncthreads();
#pragma unroll
      for (int x = 0; x < 2; x++)
        for (int e = 0; e < 8; e++) red[(8 * x + e) * NT + threadIdx.x] = isw ? dw[x][e] : db[x][e];
      __syncthreads();
    }
    float* part = isw ? part_w : part_b;
    if (part == nullptr) continue;
    // thread -> (head slot, value, lane of the row)
    for (int id = threadIdx.x; id < g.HPP * 16 * LPR; id += NT) {
      const int ll = id % LPR, ve = id / LPR % 16, hh = id / (16 * LPR), x = ve / 8, e = ve % 8;
      const int hg = i * g.HPP + hh;
      if (!qk_has<HALF>(ll, e, g.r) || (isw ? hh > 0 : hg >= g.hpg)) continue;
      double s = 0.0;
      for (int t = 0; t < NTS; t++) {
        const int th = (t / TPW) * 64 + ((t % TPW) * g.HPP + hh) * LPR + ll;
        s += (double)src[ve * NT + th];
      }
      const int col = qk_col<HALF>(ll, e, g.r);
      if (isw)
        part[(((size_t)x * g.nblk + blockIdx.x) * g.g + gi) * g.r + col] = (float)s;
      else
        part[(((size_t)x * g.nblk + blockIdx.x) * g.h + gi * g.hpg + hg) * g.r + col] = (float)s;
    }
  }
}

// out_x[e] = sum over i < n of part[x][i][e] (x = 0: q, 1: k), e < w; in double, one
// workgroup for 64 values: four lanes groups of the sum each, joined in LDS.
__global__ __launch_bounds__(256) void k_qk_sum(const float* __restrict__ part, int n, int w,
                                                float* __restrict__ out_q, float* __restrict__ out_k) {
  __shared__ double red[4][64];
  const int x = blockIdx.y, e = blockIdx.x * 64 + (threadIdx.x & 63), j = threadIdx.x >> 6;
  float* out = x ? out_k : out_q;
  if (out == nullptr) return;
  double s = 0.0;
  if (e < w)
    for (int i = j; i < n; i += 4) s += (double)part[((size_t)x * n + i) * w + e];
  red[j][threadIdx.x & 63] = s;
  __syncthreads();
  if (j == 0 && e < w) out[e] = (float)(red[0][threadIdx.x] + red[1][threadIdx.x] + red[2][threadIdx.x] + red[3][threadIdx.x]);
}

}  // namespace mom
