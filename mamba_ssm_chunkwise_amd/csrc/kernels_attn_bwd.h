// Linear attention with a decay for each head: gradients.
//
// With G the cotangent of the state after a chunk, over the chunk's rows u, j
// (s = (q.k) e^{a_u - a_j} and t = (dy.x) e^{a_u - a_j}, both for j <= u):
//   d_q[u] = sum_j t[u][j] k[j] + e^{a_u} H^T dy[u]
//   d_k[j] = sum_u t[u][j] q[u] + e^{a_end - a_j} G^T x[j]
//   d_x[j] = sum_u s[u][j] dy[u] + e^{a_end - a_j} G k[j]
//   G'     = e^{a_end} G + sum_u e^{a_u} dy[u] (outer) q[u]
// with H the state entering the chunk. The log-decay of token t scales all that
// crosses it, and is summed from just that, so no large terms cancel over a long
// sequence: pairs j < t <= u inside the chunk (row sums of (q.k) t minus its column
// sums, from t on: the pairs on one side drop out exactly), what the rows from t on
// read of H (q.d_q of the second term), what later chunks read of the rows before t
// (k.d_k of the second term), and e^{a_end} <G, H>.
//
// A workgroup walks one chain's chunks in reverse with G in fp32 registers; H
// comes from the copies that the forward (or a walk over k and x) left per chunk.
//
// Rounding. s and t enter the products as two bf16 pieces each (17 bits; s as one where p and r
// are both above 64, for which LDS is too small), so that d_q, d_k and d_x are right to their own
// rounding: with one piece they had 1.4 times its error, 1.65 in sequences of a few tokens. The
// second pieces cost 6 to 8 % of the kernel. The copies of H and G that the outputs and d_da read
// are rounded once: pieces of them would double the 25 % of the forward's bytes that the copies
// of H are, and do not fit LDS.
//
// Eight waves and one workgroup per CU: the operand tiles, both score tiles and the copies
// of G and H take most of the LDS, and with eight waves a wave's share of G is half of what
// it would be with the walk's four.
// Measured, bf16, p = 64, r = 128, 512 chains of 16384 rows: 3.5 to 3.7 ms for 14.0 GB (8.6
// read, the copies of H among them, 5.4 written: 3.8 to 4.0 TB/s; a large copy reaches 4.75),
// vector pipes 41 %, matrix pipes 22 % busy. When it took 3.36 ms, with scores of one piece, it
// took 3.07 without its stores and 3.32 without the copies' loads, so what bounds it is the
// chunk's chain of phases (three barriers, LDS round trips between products), not bytes.
#pragma once

#include <type_traits>

#include "kernels_attn.h"

namespace mom {

constexpr int ABT = 512;  // threads: eight waves
constexpr int ABW = 8;

template <typename T, int RT, int PT>   // PT tiles of 16 state rows p
struct LdsB {
  static constexpr int L = AV<T>::L;
  static constexpr int RC = 16 * RT, PC = 16 * PT;
  static constexpr int RP = AV<T>::pitch(RC), PP = AV<T>::pitch(PC), SP = AV<T>::pitch(L);
  static constexpr size_t E = sizeof(T);
  // pieces of s and of t, a tile for each: bf16 two, but with both widths at their largest, where
  // LDS ends, s has one
  static constexpr int NTP = sizeof(T) == 2 ? 2 : 1, NS = RT == 8 && PT == 8 ? 1 : NTP;
  static constexpr size_t tab = 0;
  static constexpr size_t sums = sizeof(DecayTab);   // rsum, csum, up, vp [4][64], th[8]
  static constexpr size_t k = sums + 16 * 64 * 4 + 32;
  static constexpr size_t q = k + (size_t)L * RP * E, x = q + (size_t)L * RP * E, dy = x + (size_t)L * PP * E,
                          s = dy + (size_t)L * PP * E, t = s + (size_t)NS * L * SP * E,
                          hs = t + (size_t)NTP * L * SP * E, gs = hs + (size_t)16 * PT * RP * E,
                          total = gs + (size_t)16 * PT * RP * E;
};

// The state copies that enter a chunk: tile pairs of two quads a lane (as k_attn_walk
// saves them), in flight to the LDS tile [p][r].
template <typename T, int RT, int PT>
struct StageH {
  static constexpr int PAIRS = PT * RT / 2 * 64, N = (PAIRS + ABT - 1) / ABT;
  using quad = typename AV<T>::quad;
  quad v[N][2];
  __device__ __forceinline__ void load(const T* src) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * ABT + (int)threadIdx.x;
      if (PAIRS % ABT == 0 || e < PAIRS) {
        v[i][0] = *reinterpret_cast<const quad*>(src + (size_t)e * 8);
        v[i][1] = *reinterpret_cast<const quad*>(src + (size_t)e * 8 + 4);
      }
    }
  }
  __device__ __forceinline__ void store(T* t) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * ABT + (int)threadIdx.x, lane = e & 63, tp = e >> 6, m = tp % (RT / 2), pt = tp / (RT / 2);
      if (PAIRS % ABT == 0 || e < PAIRS) {
        st_quad<16 * RT>(t, 16 * pt + (lane & 15), 8 * m + (lane >> 4), v[i][0]);
        st_quad<16 * RT>(t, 16 * pt + (lane & 15), 8 * m + 4 + (lane >> 4), v[i][1]);
      }
    }
  }
};

// PART: d_q and d_k go, in float32, to a slice of their own for each head and p tile
// (heads that share keys, or state rows in several tiles; k_attn_sum adds them), and
// d_da likewise for each p tile; otherwise straight to the caller's tensors. VEC as in
// k_attn_walk.
template <typename T, int RT, int PT, bool PART, bool VEC>
__global__ __launch_bounds__(ABT, 1) void k_attn_bwd(
    AttnGeo g, const T* __restrict__ x, const T* __restrict__ k, const T* __restrict__ q, const T* __restrict__ da,
    const T* __restrict__ save, const T* __restrict__ dy, const float* d_last,
    const float* __restrict__ seg_loc, T* __restrict__ d_x, T* __restrict__ d_k,
    T* __restrict__ d_q, T* __restrict__ d_da, float* d_h0, float* __restrict__ part_k,
    float* __restrict__ part_q, float* __restrict__ part_da) {
  using LD = LdsB<T, RT, PT>;
  using V = AV<T>;
  constexpr int L = V::L, NT = L / 16, NJ = L / 32;
  constexpr int NG = ABW / PT > 0 ? ABW / PT : 1;   // wave groups: each has all p tiles of a share of the r tiles
  constexpr int RW = RT / NG;                       // r tiles of G a wave owns
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  DecayTab* tab = reinterpret_cast<DecayTab*>(lds + LD::tab);
  float* rsum = reinterpret_cast<float*>(lds + LD::sums);   // [jt][u]
  float* csum = rsum + 4 * 64;                              // [ut][j]
  float* up = csum + 4 * 64;                                // [wave along r][u]
  float* vp = up + 4 * 64;                                  // [wave along r][j]
  float* th = vp + 4 * 64;                                  // [wave]
  T* ks = reinterpret_cast<T*>(lds + LD::k);
  T* qs = reinterpret_cast<T*>(lds + LD::q);
  T* xs = reinterpret_cast<T*>(lds + LD::x);
  T* ys = reinterpret_cast<T*>(lds + LD::dy);
  T* ss = reinterpret_cast<T*>(lds + LD::s);
  T* ts = reinterpret_cast<T*>(lds + LD::t);
  T* hs = reinterpret_cast<T*>(lds + LD::hs);
  T* gs = reinterpret_cast<T*>(lds + LD::gs);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lq = lane >> 4;

  const int nch = g.b * g.h;
  const int seg = g.nseg - 1 - (int)blockIdx.x / (nch * g.npt), rem = blockIdx.x % (nch * g.npt);
  const int item = xcd_order(rem, nch * g.npt);
  const int pt = item % g.npt, chain = item / g.npt;
  const int bi = chain / g.h, hi = chain % g.h, gi = hi / g.hpg;
  const int Vb = attn_len(g, bi), nkb = (Vb + g.CT - 1) / g.CT;
  const Segment sg(g, seg, Vb, nkb);
  const int n0 = sg.n0, nlive = sg.n1;
  const int p0 = pt * 16 * PT, pn = min(g.p - p0, 16 * PT);
  const unsigned kst = (unsigned)(g.g * g.r), xst = (unsigned)(g.h * g.p);
  const size_t row0 = (size_t)bi * g.s * g.c;
  const T* kb = k + row0 * kst + (size_t)gi * g.r;
  const T* qb = q + row0 * kst + (size_t)gi * g.r;
  const T* xb = x + row0 * xst + (size_t)hi * g.p + p0;
  const T* yb = dy + row0 * xst + (size_t)hi * g.p + p0;
  const T* dab = da + (size_t)bi * g.s * g.h + hi;
  constexpr size_t TILES = (size_t)PT * RT * 256;
  // slices: rows of h * npt * r values (d_q, d_k) and h * npt values a token (d_da)
  const int slice = hi * g.npt + pt;
  const unsigned pst = (unsigned)(g.h * g.npt * g.r);

  const int mp = wave % PT, mr = (wave / PT) * RW;   // this wave's p tile and first r tile of G
  f4 G[RW];
#pragma unroll
  for (int i = 0; i < RW; i++) {
    G[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    if (g.nseg > 1)   // k_attn_scan left every segment's there (d_h0 may be d_last itself)
      G[i] = *reinterpret_cast<const f4*>(seg_loc + (((size_t)chain * g.nseg + seg) * g.npt + pt) * TILES +
                                          tile_off(RT, mp, mr + i, lane));
    else if (d_last != nullptr)
      G[i] = ld_state4(d_last + (size_t)chain * g.p * g.r, g.p, g.r, p0 + 16 * mp + ln, 16 * (mr + i) + 4 * lq);
  }
  // the next chunk's rows, in flight while this one is worked on
  Stage<T, 16 * RT, ABT> sk, sq;
  Stage<T, 16 * PT, ABT> sx, sy;
  StageH<T, RT, PT> sh;
  sk.setup(kst, g.r);
  sq.setup(kst, g.r);
  sx.setup(xst, pn);
  sy.setup(xst, pn);
  T dnext = (T)0.0f;
  const int ltok = (lane * g.cinv) >> 16;   // the token of row u = lane
  auto fetch = [&](int n) {
    const int t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    if constexpr (VEC) {
      sk.load(row_rsrc(kb + u0 * kst, kst, nrows, g.r));
      sq.load(row_rsrc(qb + u0 * kst, kst, nrows, g.r));
      sx.load(row_rsrc(xb + u0 * xst, xst, nrows, pn));
      sy.load(row_rsrc(yb + u0 * xst, xst, nrows, pn));
    } else if constexpr (sizeof(T) == 4) {
      sk.load_each(row_rsrc(kb + u0 * kst, kst, nrows, g.r), g.r);
      sq.load_each(row_rsrc(qb + u0 * kst, kst, nrows, g.r), g.r);
      sx.load_each(row_rsrc(xb + u0 * xst, xst, nrows, pn), pn);
      sy.load_each(row_rsrc(yb + u0 * xst, xst, nrows, pn), pn);
    }
    sh.load(save + (((size_t)chain * g.NK + n) * g.npt + pt) * TILES);
    dnext = (T)0.0f;
    if (wave == 0 && lane < nrows && ltok * g.c == lane) dnext = dab[(size_t)(t0 + ltok) * g.h];
  };
  // tiles of the scores without pairs j <= u are never written: zeros throughout
  constexpr int STILE = L * LD::SP;
  for (int e = threadIdx.x; e < (LD::NS + LD::NTP) * STILE / 4; e += ABT)   // s, and t behind it
    reinterpret_cast<typename V::quad*>(ss)[e] = typename V::quad{};
  rsum[threadIdx.x] = 0.0f;   // and csum behind it
  const ScoreTiles<NT> tl(g.c);
  if (nlive > n0) fetch(nlive - 1);
  if constexpr (VEC) dropped_stores<T, (2 * RT + PT) * NT / ABW>();
  for (int n = nlive - 1; n >= n0; n--) {
    const int t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    // (the barrier that ended the last chunk covers these writes)
    if constexpr (VEC || sizeof(T) == 4) {
      sk.store(ks);
      sq.store(qs);
      sx.store(xs);
      sy.store(ys);
    } else {
      sk.direct(ks, row_rsrc(kb + u0 * kst, kst, nrows, g.r), g.r);
      sq.direct(qs, row_rsrc(qb + u0 * kst, kst, nrows, g.r), g.r);
      sx.direct(xs, row_rsrc(xb + u0 * xst, xst, nrows, pn), pn);
      sy.direct(ys, row_rsrc(yb + u0 * xst, xst, nrows, pn), pn);
    }
    sh.store(hs);
#pragma unroll
    for (int i = 0; i < RW; i++) st_quad<LD::RC>(gs, 16 * mp + ln, 4 * (mr + i) + lq, to_quad<T>(G[i]));
    if (wave == 0) decay_table(tab, log2_decay(to_f(dnext)), lane);
    __syncthreads();
    if (n > n0) fetch(n - 1);
    const float dec = ex2((float)tab->total);

    // <G, H> of this wave's tiles
    {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < RW; i++) {
        const f4 h = quad_f(ld_quad<LD::RC>(hs, 16 * mp + ln, 4 * (mr + i) + lq));
#pragma unroll
        for (int e = 0; e < 4; e++) v += G[i][e] * h[e];
      }
      v = col4_sum(row16_sum(v));
      if (lane == 0) th[wave] = v;
    }
    // s, t (stored [u][j]) and the sums of (q.k) t over pairs of different tokens
    const int la = fresh<PT == 8 || !VEC>(lane);
#pragma unroll 1
    for (int at = wave; at < tl.pairs; at += ABW) {
      const int code = (int)(tl.lower >> (4 * at)) & 15, ut = 16 * (code >> 2), jt = 16 * (code & 3);
      f4 a = {0.0f, 0.0f, 0.0f, 0.0f}, b = a;
      typename V::frag kf[RT / 2], qf[RT / 2], xf[PT / 2], yf[PT / 2];
#pragma unroll
      for (int m = 0; m < RT / 2; m++) {
        kf[m] = row_frag<LD::RC>(ks, jt, m, la);
        qf[m] = row_frag<LD::RC>(qs, ut, m, la);
      }
#pragma unroll
      for (int m = 0; m < PT / 2; m++) {
        xf[m] = row_frag<LD::PC>(xs, jt, m, la);
        yf[m] = row_frag<LD::PC>(ys, ut, m, la);
      }
      const int u = ut + ln, tok = (u * g.cinv) >> 16;
      const float uh = tab->hi[u], ul = tab->lo[u];
      const f4 jh = *reinterpret_cast<const f4*>(tab->hi + jt + 4 * lq);
      const f4 jl = *reinterpret_cast<const f4*>(tab->lo + jt + 4 * lq);
      issue_fence();
#pragma unroll
      for (int m = 0; m < (RT > PT ? RT : PT) / 2; m++) {
        if (m < RT / 2) a = mma32(kf[m], qf[m], a);
        if (m < PT / 2) b = mma32(xf[m], yf[m], b);
      }
      // j <= u: up to the last row of u's token; another token: below its first row
      const int first = tok * g.c - jt - 4 * lq, last = first + g.c - 1;
      float rs = 0.0f;
      f4 cs;
#pragma unroll
      for (int e = 0; e < 4; e++) {
        const float w = ex2((uh - jh[e]) + (ul - jl[e])), qk = a[e];
        a[e] = keep_if(e <= last, qk * w);
        b[e] = keep_if(e <= last, b[e] * w);
        cs[e] = keep_if(e < first, qk * b[e]);
        rs += cs[e];
      }
#pragma unroll
      for (int i = 0; i < LD::NS; i++) {
        const typename V::quad piece = to_quad<T>(a);
        st_quad<LD::L>(ss + i * STILE, u, jt / 4 + lq, piece);
        a -= quad_f(piece);
      }
#pragma unroll
      for (int i = 0; i < LD::NTP; i++) {
        const typename V::quad piece = to_quad<T>(b);
        st_quad<LD::L>(ts + i * STILE, u, jt / 4 + lq, piece);
        b -= quad_f(piece);
      }
      rs = col4_sum(rs);
      if (lq == 0) rsum[4 * jt + u] = rs;
#pragma unroll
      for (int e = 0; e < 4; e++) cs[e] = row16_sum(cs[e]);
      if (ln == 0) *reinterpret_cast<f4*>(csum + 4 * ut + jt + 4 * lq) = cs;
    }
    __syncthreads();

    using TO = typename std::conditional<PART, float, T>::type;
    auto chunk_rows = [&](T* out, float* part) -> TO* {
      if constexpr (PART) return part + (row0 + u0) * pst + (size_t)slice * g.r;
      else return out == nullptr ? nullptr : out + (row0 + u0) * kst + (size_t)gi * g.r;
    };
    const RowOut<TO, VEC> oq(chunk_rows(d_q, part_q), PART ? pst : kst, nrows, g.r);
    const RowOut<TO, VEC> ok(chunk_rows(d_k, part_k), PART ? pst : kst, nrows, g.r);
    const RowOut<T, VEC> ox(d_x == nullptr ? nullptr : d_x + (row0 + u0) * xst + (size_t)hi * g.p + p0, xst, nrows, pn);
    // d_q and d_k (transposed: columns are rows u of the chunk). A wave takes RB r tiles by
    // UB tiles of rows, and keeps the operands of its r tiles.
    {
      constexpr int RB = RT * NT >= 16 ? 2 : 1, WR = RT / RB, WU = ABW / WR, UB = NT / WU;
      static_assert(WR * WU == ABW && UB * WU == NT && WR <= 4, "tiles and waves");
      const int wr = wave % WR, rt0 = wr * RB, ut0 = wave / WR * UB;
      // row tiles whose operands are in flight together: as registers allow
      constexpr int JB = PT == 4 ? UB : 1;
      // `in`, the operands contracted over p (with the state or its cotangent) and over the
      // rows of the chunk; out: their rows' tiles, and the sums of what the first gives
      auto rows_grad = [&](const T* st, const T* cs, auto first, auto second, const float* w, const T* own, float* sums,
                           const RowOut<TO, VEC>& out, int l) {
        typename V::frag sf[RB][PT / 2], cf[RB][NJ];
#pragma unroll
        for (int i = 0; i < RB; i++) {
#pragma unroll
          for (int m = 0; m < PT / 2; m++) sf[i][m] = col_frag<LD::RC>(st, m, 16 * (rt0 + i), l);
#pragma unroll
          for (int m = 0; m < NJ; m++) cf[i][m] = col_frag<LD::RC>(cs, m, 16 * (rt0 + i), l);
        }
#pragma unroll
        for (int j0 = 0; j0 < UB; j0 += JB) {
          typename V::frag ff[JB][PT / 2], gf[JB][NJ], ge[JB][NJ];   // ge: the larger pieces
          typename V::quad ow[JB][RB];
          float wu[JB];
#pragma unroll
          for (int j = 0; j < JB; j++) {
            const int ut = ut0 + j0 + j;
#pragma unroll
            for (int m = 0; m < PT / 2; m++) ff[j][m] = first(ut, m);
#pragma unroll
            for (int m = 0; m < NJ; m++) gf[j][m] = second(ut, m, ts + (LD::NTP - 1) * STILE);
            wu[j] = w[16 * ut + ln];
#pragma unroll
            for (int i = 0; i < RB; i++) ow[j][i] = ld_quad<LD::RC>(own + 16 * ut * LD::RP, l & 15, 4 * (rt0 + i) + lq);
          }
          issue_fence();
          f4 a[JB][RB];
#pragma unroll
          for (int j = 0; j < JB; j++)
#pragma unroll
            for (int i = 0; i < RB; i++) a[j][i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int m = 0; m < PT / 2; m++)
#pragma unroll
            for (int j = 0; j < JB; j++)
#pragma unroll
              for (int i = 0; i < RB; i++) a[j][i] = mma32(sf[i][m], ff[j][m], a[j][i]);
          if constexpr (LD::NTP > 1) {
            issue_fence();
#pragma unroll
            for (int j = 0; j < JB; j++)
#pragma unroll
              for (int m = 0; m < NJ; m++) ge[j][m] = second(ut0 + j0 + j, m, ts);
          }
#pragma unroll
          for (int j = 0; j < JB; j++) {
            float us = 0.0f;
#pragma unroll
            for (int i = 0; i < RB; i++) {
              a[j][i] *= wu[j];
              const f4 v = quad_f(ow[j][i]);
              us += a[j][i][0] * v[0] + a[j][i][1] * v[1] + a[j][i][2] * v[2] + a[j][i][3] * v[3];
            }
            us = col4_sum(us);
            if (lq == 0) sums[wr * 64 + 16 * (ut0 + j0 + j) + ln] = us;
          }
#pragma unroll
          for (int m = 0; m < NJ; m++)
#pragma unroll
            for (int j = 0; j < JB; j++)
#pragma unroll
              for (int i = 0; i < RB; i++) a[j][i] = mma32(cf[i][m], gf[j][m], a[j][i]);
          if constexpr (LD::NTP > 1) {
#pragma unroll
            for (int m = 0; m < NJ; m++)
#pragma unroll
              for (int j = 0; j < JB; j++)
#pragma unroll
                for (int i = 0; i < RB; i++) a[j][i] = mma32(cf[i][m], ge[j][m], a[j][i]);
          }
#pragma unroll
          for (int j = 0; j < JB; j++)
#pragma unroll
            for (int i = 0; i < RB; i++) out.put(16 * (ut0 + j0 + j) + ln, 16 * (rt0 + i) + 4 * lq, a[j][i]);
        }
      };
      {
        const int lb = fresh<PT == 8 || !VEC>(lane);
        rows_grad(hs, ks, [&](int ut, int m) { return row_frag<LD::PC>(ys, 16 * ut, m, lb); },
                  [&](int ut, int m, const T* t) { return row_frag<LD::L>(t, 16 * ut, m, lb); }, tab->start, qs, up, oq, lb);
      }
      __builtin_amdgcn_sched_barrier(0);
      {
        const int lc = fresh<PT == 8 || !VEC>(lane);
        rows_grad(gs, qs, [&](int ut, int m) { return row_frag<LD::PC>(xs, 16 * ut, m, lc); },
                  [&](int ut, int m, const T* t) { return col_frag<LD::L>(t, m, 16 * ut, lc); }, tab->end, ks, vp, ok, lc);
      }
    }
    // d_x, likewise over PB tiles of rows p
    __builtin_amdgcn_sched_barrier(0);
    {
      constexpr int PB = PT * NT >= 16 ? 2 : 1, WP = PT / PB, WU = ABW / WP, UB = NT / WU > 0 ? NT / WU : 1;
      static_assert(WP * WU == ABW && UB * WU == NT, "tiles and waves");
      const int ld = fresh<PT == 8 || !VEC>(lane);
      const int pj0 = wave % WP * PB, ut0 = wave / WP * UB;
#pragma unroll
      for (int j = 0; j < UB; j++) {
        const int ut = ut0 + j, u = 16 * ut + ln;
        typename V::frag kf[RT / 2], gf[PB][RT / 2], sf[LD::NS][NJ], yf[PB][NJ];
#pragma unroll
        for (int m = 0; m < RT / 2; m++) {
          kf[m] = row_frag<LD::RC>(ks, 16 * ut, m, ld);
#pragma unroll
          for (int i = 0; i < PB; i++) gf[i][m] = row_frag<LD::RC>(gs, 16 * (pj0 + i), m, ld);
        }
#pragma unroll
        for (int m = 0; m < NJ; m++) {
#pragma unroll
          for (int i = 0; i < LD::NS; i++) sf[i][m] = col_frag<LD::L>(ss + i * STILE, m, 16 * ut, ld);
#pragma unroll
          for (int i = 0; i < PB; i++) yf[i][m] = col_frag<LD::PC>(ys, m, 16 * (pj0 + i), ld);
        }
        const float en = tab->end[u];
        issue_fence();
        f4 a[PB];
#pragma unroll
        for (int i = 0; i < PB; i++) a[i] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < RT / 2; m++)
#pragma unroll
          for (int i = 0; i < PB; i++) a[i] = mma32(gf[i][m], kf[m], a[i]);
#pragma unroll
        for (int i = 0; i < PB; i++) a[i] *= en;
#pragma unroll
        for (int k2 = LD::NS - 1; k2 >= 0; k2--)
#pragma unroll
          for (int m = 0; m < NJ; m++)
#pragma unroll
            for (int i = 0; i < PB; i++) a[i] = mma32(yf[i][m], sf[k2][m], a[i]);
#pragma unroll
        for (int i = 0; i < PB; i++) ox.put(u, 16 * (pj0 + i) + 4 * lq, a[i]);
      }
    }
    // G'
    __builtin_amdgcn_sched_barrier(0);
    {
      const int le = fresh<PT == 8 || !VEC>(lane);
      typename V::frag qf[NJ][RW], yr[NJ];
      f4 w0[NJ], w1[NJ];
#pragma unroll
      for (int m = 0; m < NJ; m++) {
        yr[m] = col_frag<LD::PC>(ys, m, 16 * mp, le);
        w0[m] = *reinterpret_cast<const f4*>(tab->start + 32 * m + 4 * lq);
        w1[m] = *reinterpret_cast<const f4*>(tab->start + 32 * m + 16 + 4 * lq);
#pragma unroll
        for (int i = 0; i < RW; i++) qf[m][i] = col_frag<LD::RC>(qs, m, 16 * (mr + i), le);
      }
      issue_fence();
      Scaled<V::NSPLIT> yf[NJ];
#pragma unroll
      for (int m = 0; m < NJ; m++) yf[m].make(yr[m], w0[m], w1[m]);
#pragma unroll
      for (int i = 0; i < RW; i++) G[i] *= dec;
#pragma unroll
      for (int m = 0; m < NJ; m++)
#pragma unroll
        for (int k2 = 0; k2 < V::NSPLIT; k2++)
#pragma unroll
          for (int i = 0; i < RW; i++) G[i] = mma32(qf[m][i], yf[m].piece(k2), G[i]);
    }
    __syncthreads();   // every tile has been read; the sums are complete
    if (wave == 0) {
      // suffix sums over the rows from a token on, prefix sums over the rows before it
      double suf = 0.0, pre = 0.0, thr = 0.0;
      if (lane < L) {
#pragma unroll
        for (int i = 0; i < NT; i++) suf += (double)rsum[i * 64 + lane] - (double)csum[i * 64 + lane];
#pragma unroll
        for (int i = 0; i < (RT * NT >= 16 ? RT / 2 : RT); i++) {
          suf += (double)up[i * 64 + lane];
          pre += (double)vp[i * 64 + lane];
        }
      }
      for (int i = 0; i < ABW; i++) thr += (double)th[i];
      const double si = wave_sum_incl(suf), pi = wave_sum_incl(pre);
      const double v = lane63(si) - si + suf + pi - pre + thr * (double)dec;
      if (lane < nrows && ltok * g.c == lane) {
        if constexpr (PART)
          part_da[((size_t)bi * g.s + t0 + ltok) * g.h * g.npt + slice] = (float)v;
        else if (d_da != nullptr)
          d_da[((size_t)bi * g.s + t0 + ltok) * g.h + hi] = to_t<T>((float)v);
      }
    }
  }

  // rows past the sequence's length are zero
  {
    const int z0 = sg.z0, z1 = sg.z1;
    for (int u = z0 * g.c + wave; u < z1 * g.c; u += ABW) {
      const size_t at = row0 + u;
      for (int e = lane; e < pn && d_x != nullptr; e += 64) d_x[at * xst + (size_t)hi * g.p + p0 + e] = (T)0.0f;
      for (int e = lane; e < g.r; e += 64) {
        if constexpr (PART) {
          part_q[at * pst + (size_t)slice * g.r + e] = 0.0f;
          part_k[at * pst + (size_t)slice * g.r + e] = 0.0f;
        } else {
          if (d_q != nullptr) d_q[at * kst + (size_t)gi * g.r + e] = (T)0.0f;
          if (d_k != nullptr) d_k[at * kst + (size_t)gi * g.r + e] = (T)0.0f;
        }
      }
    }
    for (int t = z0 + (int)threadIdx.x; t < z1; t += ABT) {
      if constexpr (PART)
        part_da[((size_t)bi * g.s + t) * g.h * g.npt + slice] = 0.0f;
      else if (d_da != nullptr)
        d_da[((size_t)bi * g.s + t) * g.h + hi] = (T)0.0f;
    }
  }
  if (d_h0 != nullptr && seg == 0) {
#pragma unroll
    for (int i = 0; i < RW; i++)
      st_state4(d_h0 + (size_t)chain * g.p * g.r, g.p, g.r, p0 + 16 * mp + ln, 16 * (mr + i) + 4 * lq, G[i]);
  }
}

// Jobs of sums: out[row][group][w] = sum of the group's n consecutive slices of
// part[row][groups * n][w], `total` values of out. One launch for all of them.
struct SumJob {
  const float* part;
  void* out;
  size_t total;
  int n, w;
};
struct SumJobs {
  SumJob job[3];
};
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum(SumJobs jobs) {
  const SumJob j = jobs.job[blockIdx.y];
  T* out = reinterpret_cast<T*>(j.out);
  for (size_t e = (size_t)blockIdx.x * 256 + threadIdx.x; e < j.total; e += (size_t)gridDim.x * 256) {
    const size_t grp = e / j.w;
    const float* src = j.part + grp * j.n * j.w + e % j.w;
    float s = 0.0f;
#pragma unroll 4
    for (int i = 0; i < j.n; i++) s += src[(size_t)i * j.w];
    out[e] = to_t<T>(s);
  }
}

}  // namespace mom
