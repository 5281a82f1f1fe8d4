// Linear attention with a decay for each head: shared tile helpers, and the
// walks over a sequence (forward, and the state alone).
//
// Per (b, head) chain the state h~[t] = e^{da_t} h~[t-1] + sum_c x[t,c] (outer) k[t,c]
// is read out as y[t,c] = h~[t] q[t,c]. Over a chunk of tokens whose rows (t, c)
// are folded into one index u, with a_u the inclusive sum of da up to u's token:
//   y[u]  = e^{a_u} H q[u] + sum_{j <= u} (q[u].k[j]) e^{a_u - a_j} x[j]
//   H'    = e^{a_end} H + sum_j e^{a_end - a_j} x[j] (outer) k[j]
// (j <= u: the token of j is not after that of u, so channels of one token see
// each other). A workgroup walks the chunks of one chain with H in fp32
// accumulator registers, so q, k, x are read once and y is written once.
//
// Rounding. Products of bf16 values are exact in fp32. The two operands that the
// walk itself makes are rounded to bf16 for the matrix instructions: the scores
// (q.k) e^{a_u - a_j}, and a copy of H where y reads it. The running H never is:
// the decayed writes e^{a_end - a_j} x[j] enter as the sum of three bf16 pieces
// (24 bits), so the state, which is handed on to later calls, keeps fp32 accuracy.
//
// MFMA fragments here span 32 slots of the contracted index in the order in which
// a pair of accumulator tiles holds its rows: lane group q (= lane / 16) has
// indices 4q..4q+3 of the first 16 and 4q..4q+3 of the second 16 ("two quads").
// With every operand loaded in that order, the accumulator tiles of one product
// are operands of the next without leaving the registers.
#pragma once

#include "common.h"

namespace mom {

constexpr int ATT = 256;  // threads of a walk: four waves, each owning tiles of 16 state rows
constexpr int ATW = 4;

struct AttnGeo {
  int b, s, c, h, g, p, r;
  int V;        // min(valid_len, s)
  int hpg;      // heads per key group
  int CT;       // tokens per chunk: L / c
  int NK;       // chunks over all s tokens
  int nseg;     // segments a chain's walk is split into
  int seg0;     // first segment of this launch
  int SL;       // chunks per segment
  int npt;      // column tiles of the state rows p that separate workgroups take
  int PT;       // rows of p in such a tile
  int cinv;     // ceil(65536 / c): u / c = (u * cinv) >> 16 for a row u of a chunk
  const int* lens;  // per-sequence valid lengths [b] (device), or nullptr
};

__device__ __forceinline__ int attn_len(const AttnGeo& g, int bi) {
  if (g.lens == nullptr) return g.V;
  const int v = g.lens[bi];
  return v < 0 ? 0 : (v < g.V ? v : g.V);
}

// Decays. Sums of da are kept in units of log2 as a float and its remainder
// (from a sum in double), so that differences of long sums keep 24 bits of the
// difference. A decay below e^-110 is zero in fp32; da is clamped there (also
// -inf, a cleared state) so that later differences stay finite. NaN stays NaN.
constexpr double kLog2e = 1.4426950408889634;
__device__ __forceinline__ double log2_decay(float da) { return (double)(da < -110.0f ? -110.0f : da) * kLog2e; }
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- types ------------------------------------------------------------------
template <typename T> struct AV;
template <> struct AV<bf16> {
  static constexpr int L = 64;    // rows per chunk
  static constexpr int PE = 8;    // elements per 16-byte piece
  static constexpr int NSPLIT = 3;
  using quad = uint2;
  using frag = bf8;
  __host__ __device__ static constexpr int pitch(int n) { return n + ((16 - n % 64) + 64) % 64; }
};
template <> struct AV<float> {
  static constexpr int L = 32;
  static constexpr int PE = 4;
  static constexpr int NSPLIT = 1;
  using quad = f4;
  struct frag { f4 v[2]; };
  __host__ __device__ static constexpr int pitch(int n) { return n + 4; }
};

__device__ __forceinline__ f4 mma32(bf8 a, bf8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f4 mma32(const AV<float>::frag& a, const AV<float>::frag& b, f4 c) {
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int i = 0; i < 4; i++) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h][i], b.v[h][i], c, 0, 0, 0);
  return c;
}

template <typename T> __device__ __forceinline__ typename AV<T>::quad to_quad(f4 v);
template <> __device__ __forceinline__ uint2 to_quad<bf16>(f4 v) {
  return make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
}
template <> __device__ __forceinline__ f4 to_quad<float>(f4 v) { return v; }
__device__ __forceinline__ f4 quad_f(uint2 v) { return f4{bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y)}; }
__device__ __forceinline__ f4 quad_f(f4 v) { return v; }
__device__ __forceinline__ bf8 join(uint2 a, uint2 b) { return as_bf8(u4{a.x, a.y, b.x, b.y}); }
__device__ __forceinline__ AV<float>::frag join(f4 a, f4 b) { return AV<float>::frag{{a, b}}; }
template <typename T> __device__ __forceinline__ typename AV<T>::frag acc_frag(f4 a, f4 b) {
  return join(to_quad<T>(a), to_quad<T>(b));
}

// ---- LDS tiles [row][column] ---------------------------------------------------
// Rows of `pitch` elements. In bf16 tiles the 4-element quads of rows 8..15 of
// each 16 are swapped pairwise (quad v sits at v ^ 1): with rows 8 banks apart,
// reads of one quad from 16 rows, and transposing reads of 4 rows, are then both
// free of bank conflicts.
template <typename T> __device__ __forceinline__ int swz(int row);
template <> __device__ __forceinline__ int swz<bf16>(int row) { return (row >> 3) & 1; }
template <> __device__ __forceinline__ int swz<float>(int) { return 0; }

template <typename T>
__device__ __forceinline__ typename AV<T>::quad ld_quad(const T* t, int P, int row, int v) {
  return *reinterpret_cast<const typename AV<T>::quad*>(t + row * P + 4 * (v ^ swz<T>(row)));
}
template <typename T>
__device__ __forceinline__ void st_quad(T* t, int P, int row, int v, typename AV<T>::quad x) {
  *reinterpret_cast<typename AV<T>::quad*>(t + row * P + 4 * (v ^ swz<T>(row))) = x;
}
// One 16-byte piece (column piece * PE) of a row.
__device__ __forceinline__ void st_piece(bf16* t, int P, int row, int piece, uint4 x) {
  if (swz<bf16>(row)) x = make_uint4(x.z, x.w, x.x, x.y);
  *reinterpret_cast<uint4*>(t + row * P + 8 * piece) = x;
}
__device__ __forceinline__ void st_piece(float* t, int P, int row, int piece, uint4 x) {
  *reinterpret_cast<uint4*>(t + row * P + 4 * piece) = x;
}

// Fragment of rows row0 + lane % 16, contracted over columns 32m .. 32m + 31.
template <typename T>
__device__ __forceinline__ typename AV<T>::frag row_frag(const T* t, int P, int row0, int m, int lane) {
  const int row = row0 + (lane & 15), q = lane >> 4;
  return join(ld_quad(t, P, row, 8 * m + q), ld_quad(t, P, row, 8 * m + 4 + q));
}
// Fragment of columns col0 + lane % 16, contracted over rows 32m .. 32m + 31.
// bf16: transposing reads; in each 16-lane group, lane j receives element j % 4
// of the 8-byte pieces that lanes 4r + j / 4 address, r = 0..3.
typedef short as4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ as4 lds_tr16(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) as4*)p);
}
__device__ __forceinline__ bf8 col_frag(const bf16* t, int P, int m, int col0, int lane) {
  const int row = 32 * m + 4 * (lane >> 4) + ((lane >> 2) & 3);
  const bf16* p0 = t + row * P + col0 + 4 * ((lane & 3) ^ swz<bf16>(row));
  const as4 v[2] = {lds_tr16(p0), lds_tr16(p0 + 16 * P)};
  return __builtin_bit_cast(bf8, v);
}
__device__ __forceinline__ AV<float>::frag col_frag(const float* t, int P, int m, int col0, int lane) {
  AV<float>::frag f;
  const float* p0 = t + (32 * m + 4 * (lane >> 4)) * P + col0 + (lane & 15);
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int i = 0; i < 4; i++) f.v[h][i] = p0[(16 * h + i) * P];
  return f;
}

// c + a (B operand x scaled by w per slot), to fp32 accuracy of the scaled values:
// in bf16 the scaled operand is split into three bf16 pieces, each exact in the rest
// of the one before.
template <int N>
struct Scaled;
template <>
struct Scaled<3> {
  bf8 p[3];
  __device__ __forceinline__ void make(bf8 x, f4 w0, f4 w1) {
    u4 o[3];
#pragma unroll
    for (int k = 0; k < 4; k++) {
      float a = (float)x[2 * k] * (k < 2 ? w0[2 * k] : w1[2 * k - 4]);
      float b = (float)x[2 * k + 1] * (k < 2 ? w0[2 * k + 1] : w1[2 * k - 3]);
#pragma unroll
      for (int i = 0; i < 3; i++) {
        o[i][k] = pk_bf16(a, b);
        if (i < 2) {
          a -= bf16_lo(o[i][k]);
          b -= bf16_hi(o[i][k]);
        }
      }
    }
    for (int i = 0; i < 3; i++) p[i] = as_bf8(o[i]);
  }
  __device__ __forceinline__ f4 mma(bf8 a, f4 c) const {
#pragma unroll
    for (int i = 2; i >= 0; i--) c = mma32(a, p[i], c);
    return c;
  }
};
template <>
struct Scaled<1> {
  AV<float>::frag p;
  __device__ __forceinline__ void make(const AV<float>::frag& x, f4 w0, f4 w1) { p = AV<float>::frag{{x.v[0] * w0, x.v[1] * w1}}; }
  __device__ __forceinline__ f4 mma(const AV<float>::frag& a, f4 c) const { return mma32(a, p, c); }
};

// ---- staging ----------------------------------------------------------------
// A [L][COLS] block of rows on its way from global memory to an LDS tile, in 16-byte
// pieces. Rows >= nrows and columns >= n are zeros, whatever the memory there holds.
// Rows that are whole pieces go through registers (load, later store), so that they can
// be in flight while another chunk is worked on; others are fetched one element at a
// time, straight into the tile. Offsets inside a chunk fit 32 bits (the plan refuses
// wider rows), so that addresses are a scalar base and one register.
template <typename T, int COLS, int NT>
struct Stage {
  static constexpr int L = AV<T>::L, PE = AV<T>::PE, PR = COLS / PE, N = (L * PR + NT - 1) / NT;
  uint4 v[N];
  __device__ __forceinline__ void load(const T* base, unsigned stride, int nrows, int n) {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * NT + (int)threadIdx.x, row = e / PR, c0 = e % PR * PE;
      v[i] = make_uint4(0, 0, 0, 0);
      if (row < nrows && c0 < n) v[i] = *reinterpret_cast<const uint4*>(base + ((unsigned)row * stride + (unsigned)c0));
    }
  }
  __device__ __forceinline__ void store(T* t, int P) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * NT + (int)threadIdx.x, row = e / PR, piece = e % PR;
      if (L * PR % NT == 0 || row < L) st_piece(t, P, row, piece, v[i]);
    }
  }
  __device__ __forceinline__ static void direct(T* t, int P, const T* base, unsigned stride, int nrows, int n) {
#pragma unroll 1
    for (int e = (int)threadIdx.x; e < L * PR; e += NT) {
      const int row = e / PR, c0 = e % PR * PE;
      T x[PE];
#pragma unroll
      for (int i = 0; i < PE; i++)
        x[i] = row < nrows && c0 + i < n ? base[(unsigned)row * stride + (unsigned)(c0 + i)] : (T)0.0f;
      st_piece(t, P, row, e % PR, __builtin_bit_cast(uint4, x));
    }
  }
};

// Per-row decay tables of a chunk, written by one wave (lane u = row u).
struct DecayTab {
  float hi[64], lo[64];   // a_u in log2 units: hi + lo
  float start[64];        // e^{a_u}
  float end[64];          // e^{a_end - a_u}
  double total;           // a_end in log2 units
  double pad;             // tiles behind it start at 16 bytes
};
// v: log2 decay of row u = lane (zero where the row does not open a token).
__device__ __forceinline__ double wave_sum_incl(double v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const double o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ void decay_table(DecayTab* t, double v, int lane) {
  const double a = wave_sum_incl(v, lane), e = __shfl(a, 63);
  const float hi = (float)a;
  t->hi[lane] = hi;
  t->lo[lane] = (float)(a - hi);
  t->start[lane] = ex2(hi);
  t->end[lane] = ex2((float)(e - a));
  if (lane == 0) t->total = e;
}

// Work of a block: workgroups are handed out round-robin to the eight XCDs, so
// consecutive chains (heads of one key group read the same rows) are given to one
// XCD and share its L2.
__device__ __forceinline__ int xcd_order(int bid, int n) {
  const int per = n / 8;
  return bid < 8 * per ? (bid % 8) * per + bid / 8 : bid;
}

// State tiles in memory: tile (pt, rt) of 16 state rows p by 16 columns r is 64
// lanes of four values, lane (q, n): p = 16pt + n, r = 16rt + 4q .. 4q + 3.
__device__ __forceinline__ size_t tile_off(int RT, int pt, int rt, int lane) {
  return ((size_t)(pt * RT + rt) * 64 + lane) * 4;
}

// Four consecutive columns of a float32 state row from / to the caller's [p][r].
__device__ __forceinline__ f4 ld_state4(const float* st, int p, int r, int pi, int r0) {
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (pi < p) {
    const float* s = st + (size_t)pi * r + r0;
    if ((r & 3) == 0) {
      if (r0 < r) v = *reinterpret_cast<const f4*>(s);
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++)
        if (r0 + i < r) v[i] = s[i];
    }
  }
  return v;
}
__device__ __forceinline__ void st_state4(float* st, int p, int r, int pi, int r0, f4 v) {
  if (pi >= p) return;
  float* s = st + (size_t)pi * r + r0;
  if ((r & 3) == 0) {
    if (r0 < r) *reinterpret_cast<f4*>(s) = v;
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (r0 + i < r) s[i] = v[i];
  }
}
// Four consecutive columns c0.. of the row of n elements at base[off] (quad-aligned when
// n % 4 == 0).
template <typename T>
__device__ __forceinline__ void st_row4(T* base, unsigned off, int n, int c0, f4 v) {
  off += (unsigned)c0;
  if ((n & 3) == 0) {
    if (c0 < n) *reinterpret_cast<typename AV<T>::quad*>(base + off) = to_quad<T>(v);
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++)
      if (c0 + i < n) base[off + i] = to_t<T>(v[i]);
  }
}

// LDS of the walks.
template <typename T, int RT, int PW>
struct LdsA {
  static constexpr int L = AV<T>::L, RP = AV<T>::pitch(16 * RT), PT = 16 * ATW * PW, PP = AV<T>::pitch(PT),
                       SP = AV<T>::pitch(L);
  static constexpr size_t tab = 0, k = sizeof(DecayTab), x = k + (size_t)L * RP * sizeof(T),
                          state_total = x + (size_t)L * PP * sizeof(T), q = state_total,
                          s = q + (size_t)L * RP * sizeof(T), total = s + (size_t)L * SP * sizeof(T);
  static_assert(sizeof(DecayTab) % 16 == 0, "tiles start at 16 bytes");
};

// H' = e^{a_end} H + sum_j w_j x[j] (outer) k[j] over the rows of the LDS tiles.
// A wave owns state rows 16 (wave * PW + pw) .. + 15 and all columns.
template <typename T, int RT, int PW>
__device__ __forceinline__ void state_update(f4 (&H)[PW][RT], const T* ks, const T* xs, const float* w, float dec,
                                             int wave, int lane) {
  using LD = LdsA<T, RT, PW>;
  constexpr int NJ = AV<T>::L / 32;
  const int q = lane >> 4;
  Scaled<AV<T>::NSPLIT> xf[PW][NJ];
#pragma unroll
  for (int m = 0; m < NJ; m++) {
    const f4 w0 = *reinterpret_cast<const f4*>(w + 32 * m + 4 * q);
    const f4 w1 = *reinterpret_cast<const f4*>(w + 32 * m + 16 + 4 * q);
#pragma unroll
    for (int pw = 0; pw < PW; pw++) xf[pw][m].make(col_frag(xs, LD::PP, m, 16 * (wave * PW + pw), lane), w0, w1);
  }
#pragma unroll
  for (int rt = 0; rt < RT; rt++) {
#pragma unroll
    for (int pw = 0; pw < PW; pw++) H[pw][rt] *= dec;
#pragma unroll
    for (int m = 0; m < NJ; m++) {
      const auto kf = col_frag(ks, LD::RP, m, 16 * rt, lane);
#pragma unroll
      for (int pw = 0; pw < PW; pw++) H[pw][rt] = xf[pw][m].mma(kf, H[pw][rt]);
    }
  }
}

// ---- walks --------------------------------------------------------------------
// MODE 0: the forward, writing y, the last state, and with `save` the state that
//         enters each chunk as an operand copy (T, tile order);
// MODE 1: the state alone (k, x): with seg_loc each segment from zero, leaving its
//         last state and log2 decay there; without, the walk that only saves;
// MODE 2: the cotangent of the state alone, chunks in reverse: k is q, x is d_y,
//         and the weights are e^{a_u}.
// VEC: rows are whole 16-byte pieces; the next chunk's are then in flight while one is
// worked on. A chain split into segments starts each of them from the states that the
// segments before it (after it, MODE 2 users) left in seg_loc.
template <typename T, int RT, int PW, int MODE, bool VEC>
__global__ __launch_bounds__(ATT, 2) void k_attn_walk(AttnGeo g, const T* __restrict__ x, const T* __restrict__ k,
                                                      const T* __restrict__ q, const T* __restrict__ da,
                                                      const float* __restrict__ h0, T* __restrict__ y,
                                                      float* __restrict__ h_last, T* __restrict__ save,
                                                      float* __restrict__ seg_loc, double* __restrict__ seg_dec) {
  using LD = LdsA<T, RT, PW>;
  using V = AV<T>;
  constexpr int L = V::L, NT = L / 16, NJ = L / 32, PT16 = ATW * PW;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  DecayTab* tab = reinterpret_cast<DecayTab*>(lds + LD::tab);
  T* ks = reinterpret_cast<T*>(lds + LD::k);
  T* xs = reinterpret_cast<T*>(lds + LD::x);
  T* qs = reinterpret_cast<T*>(lds + LD::q);
  T* ss = reinterpret_cast<T*>(lds + LD::s);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lq = lane >> 4;

  // block -> (segment, p tile, chain), chains in XCD order within a segment
  const int nch = g.b * g.h;
  const int seg = g.seg0 + blockIdx.x / (nch * g.npt), rem = blockIdx.x % (nch * g.npt);
  const int item = xcd_order(rem, nch * g.npt);
  const int pt = item % g.npt, chain = item / g.npt;
  const int bi = chain / g.h, hi = chain % g.h, gi = hi / g.hpg;
  const int Vb = attn_len(g, bi), nkb = (Vb + g.CT - 1) / g.CT;
  const int n0 = seg * g.SL, n1 = min(n0 + g.SL, g.NK);
  const int p0 = pt * LD::PT, pn = min(g.p - p0, LD::PT);
  const unsigned kst = (unsigned)(g.g * g.r), xst = (unsigned)(g.h * g.p);   // strides of a row u
  const size_t row0 = (size_t)bi * g.s * g.c;
  const T* kb = k + row0 * kst + (size_t)gi * g.r;
  const T* qb = MODE == 0 ? q + row0 * kst + (size_t)gi * g.r : nullptr;
  const T* xb = x + row0 * xst + (size_t)hi * g.p + p0;
  const T* dab = da + (size_t)bi * g.s * g.h + hi;
  constexpr size_t TILES = (size_t)PT16 * RT * 256;   // values of a state in tile order

  f4 H[PW][RT];
#pragma unroll
  for (int pw = 0; pw < PW; pw++)
#pragma unroll
    for (int rt = 0; rt < RT; rt++) H[pw][rt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
  if (MODE == 0 || seg_loc == nullptr || save != nullptr) {
    if (h0 != nullptr) {
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          H[pw][rt] = ld_state4(h0 + (size_t)chain * g.p * g.r, g.p, g.r, p0 + 16 * (wave * PW + pw) + ln,
                                16 * rt + 4 * lq);
    }
    for (int s = 0; s < seg; s++) {   // what the segments before this one leave
      const size_t at = ((size_t)chain * g.nseg + s) * g.npt + pt;
      const float dec = ex2((float)seg_dec[at]);
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          H[pw][rt] = H[pw][rt] * dec +
                      *reinterpret_cast<const f4*>(seg_loc + at * TILES + tile_off(RT, wave * PW + pw, rt, lane));
    }
  }
  double acc_dec = 0.0;

  const int nlive = min(n1, nkb);
  Stage<T, 16 * RT, ATT> sk, sq;
  Stage<T, LD::PT, ATT> sx;
  T dnext = (T)0.0f;                        // da of the token that row u = lane opens
  const int ltok = (lane * g.cinv) >> 16;   // the token of row u = lane
  auto chunk = [&](int i) { return MODE == 2 ? nlive - 1 - (i - n0) : i; };
  auto fetch = [&](int n) {
    const int t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    if constexpr (VEC) {
      sk.load(kb + u0 * kst, kst, nrows, g.r);
      sx.load(xb + u0 * xst, xst, nrows, pn);
      if constexpr (MODE == 0) sq.load(qb + u0 * kst, kst, nrows, g.r);
    }
    dnext = (T)0.0f;
    if (wave == 0 && lane < nrows && ltok * g.c == lane) dnext = dab[(size_t)(t0 + ltok) * g.h];
  };
  if (nlive > n0) fetch(chunk(n0));
  for (int i = n0; i < nlive; i++) {
    const int n = chunk(i), t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    __syncthreads();   // the last chunk's tiles have been read
    if constexpr (VEC) {
      sk.store(ks, LD::RP);
      sx.store(xs, LD::PP);
      if constexpr (MODE == 0) sq.store(qs, LD::RP);
    } else {
      sk.direct(ks, LD::RP, kb + u0 * kst, kst, nrows, g.r);
      sx.direct(xs, LD::PP, xb + u0 * xst, xst, nrows, pn);
      if constexpr (MODE == 0) sq.direct(qs, LD::RP, qb + u0 * kst, kst, nrows, g.r);
    }
    if (wave == 0) decay_table(tab, log2_decay(to_f(dnext)), lane);
    __syncthreads();
    if (i + 1 < nlive) fetch(chunk(i + 1));
    const double total = tab->total;
    acc_dec += total;

    if constexpr (MODE != 2) {
      if (save != nullptr) {
        T* dst = save + (((size_t)chain * g.NK + n) * g.npt + pt) * TILES;
#pragma unroll
        for (int pw = 0; pw < PW; pw++)
#pragma unroll
          for (int rt = 0; rt < RT; rt += 2) {
            // the two quads of a fragment side by side
            T* d = dst + ((size_t)((wave * PW + pw) * RT + rt) * 64 + lane * 2) * 4;
            *reinterpret_cast<typename V::quad*>(d) = to_quad<T>(H[pw][rt]);
            *reinterpret_cast<typename V::quad*>(d + 4) = to_quad<T>(H[pw][rt + 1]);
          }
      }
    }

    if constexpr (MODE == 0) {
      // scores s[u][j] = (q[u].k[j]) e^{a_u - a_j}, one 16x16 tile (columns u) at a time
#pragma unroll
      for (int it = 0; it < (NT * NT + ATW - 1) / ATW; it++) {
        const int id = it * ATW + wave, ut = id % NT, jt = id / NT;
        f4 a = {0.0f, 0.0f, 0.0f, 0.0f};
        // rows of a token never straddle 16 rows unless c = 3 (then up to two rows further)
        if (jt <= ut || (g.c == 3 && jt == ut + 1)) {
#pragma unroll
          for (int m = 0; m < RT / 2; m++)
            a = mma32(row_frag(ks, LD::RP, 16 * jt, m, lane), row_frag(qs, LD::RP, 16 * ut, m, lane), a);
          const int u = 16 * ut + ln, tu = (u * g.cinv) >> 16;
          const float uh = tab->hi[u], ul = tab->lo[u];
          const f4 jh = *reinterpret_cast<const f4*>(tab->hi + 16 * jt + 4 * lq);
          const f4 jl = *reinterpret_cast<const f4*>(tab->lo + 16 * jt + 4 * lq);
#pragma unroll
          for (int e = 0; e < 4; e++) {
            const int tj = ((16 * jt + 4 * lq + e) * g.cinv) >> 16;
            a[e] = tj <= tu ? a[e] * ex2((uh - jh[e]) + (ul - jl[e])) : 0.0f;
          }
        }
        st_quad(ss, LD::SP, 16 * ut + ln, 4 * jt + lq, to_quad<T>(a));
      }
      __syncthreads();
      // y[u] for this wave's rows p
      typename V::frag hf[PW][RT / 2];
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int m = 0; m < RT / 2; m++) hf[pw][m] = acc_frag<T>(H[pw][2 * m], H[pw][2 * m + 1]);
      typename V::frag xf[PW][NJ];
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int m = 0; m < NJ; m++) xf[pw][m] = col_frag(xs, LD::PP, m, 16 * (wave * PW + pw), lane);
#pragma unroll
      for (int ut = 0; ut < NT; ut++) {
        f4 a[PW];
#pragma unroll
        for (int pw = 0; pw < PW; pw++) a[pw] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int m = 0; m < RT / 2; m++) {
          const auto qf = row_frag(qs, LD::RP, 16 * ut, m, lane);
#pragma unroll
          for (int pw = 0; pw < PW; pw++) a[pw] = mma32(hf[pw][m], qf, a[pw]);
        }
        const int u = 16 * ut + ln;
        const float st = tab->start[u];
#pragma unroll
        for (int pw = 0; pw < PW; pw++) a[pw] *= st;
#pragma unroll
        for (int m = 0; m < NJ; m++) {
          if (32 * m < 16 * (ut + 1) || g.c == 3) {
            const auto sf = row_frag(ss, LD::SP, 16 * ut, m, lane);
#pragma unroll
            for (int pw = 0; pw < PW; pw++) a[pw] = mma32(xf[pw][m], sf, a[pw]);
          }
        }
        if (u < nrows) {
#pragma unroll
          for (int pw = 0; pw < PW; pw++)
            st_row4(y + (row0 + u0) * xst + (size_t)hi * g.p, (unsigned)u * xst, g.p,
                    p0 + 16 * (wave * PW + pw) + 4 * lq, a[pw]);
        }
      }
    }
    state_update<T, RT, PW>(H, ks, xs, MODE == 2 ? tab->start : tab->end, ex2((float)total), wave, lane);
  }

  if constexpr (MODE == 0) {
    // rows past the sequence's length are zero
    const int z0 = max(n0 * g.CT, Vb), z1 = min(n1 * g.CT, g.s);
    for (int u = z0 * g.c + (int)(threadIdx.x / 16); u < z1 * g.c; u += ATT / 16) {
      T* yr = y + (row0 + u) * xst + (size_t)hi * g.p + p0;
      for (int e = threadIdx.x % 16; e < pn; e += 16) yr[e] = (T)0.0f;
    }
    if (h_last != nullptr && seg == g.nseg - 1) {
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          st_state4(h_last + (size_t)chain * g.p * g.r, g.p, g.r, p0 + 16 * (wave * PW + pw) + ln, 16 * rt + 4 * lq,
                    H[pw][rt]);
    }
  } else if (seg_loc != nullptr && save == nullptr) {
    const size_t at = ((size_t)chain * g.nseg + seg) * g.npt + pt;
    if (threadIdx.x == 0) seg_dec[at] = acc_dec;
#pragma unroll
    for (int pw = 0; pw < PW; pw++)
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
        *reinterpret_cast<f4*>(seg_loc + at * TILES + tile_off(RT, wave * PW + pw, rt, lane)) = H[pw][rt];
  }
}

// ---- one token per sequence -------------------------------------------------------
// state <- e^{da} state + sum_c x[c] (outer) k[c];  y[c] = state q[c], in fp32.
// LPR lanes share a state row, four columns each (r <= 4 LPR); a wave takes
// 64 / LPR rows at a time and NB such batches, with all their loads in flight first:
// the state is read and written once and is all that counts (2 * 4 p r bytes against
// 2 (2 r + 2 p) for the rest).
template <typename T, int LPR, int NB>
__global__ __launch_bounds__(256) void k_attn_step(AttnGeo g, int nslots, const T* __restrict__ x,
                                                   const T* __restrict__ k, const T* __restrict__ q,
                                                   const T* __restrict__ da, const int* __restrict__ slots,
                                                   float* __restrict__ state, T* __restrict__ y) {
  constexpr int RPW = 64 / LPR;                 // rows per wave and batch
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int chain = blockIdx.x, bi = chain / g.h, hi = chain % g.h, gi = hi / g.hpg;
  const int row0 = ((int)blockIdx.y * 4 + wave) * RPW * NB + lane / LPR, r0 = 4 * (lane % LPR);
  const int slot = slots == nullptr ? bi : slots[bi];
  const bool live = slot >= 0 && slot < nslots && attn_len(g, bi) > 0;
  if (!live) {
    for (int i = 0; i < NB; i++) {
      const int pi = row0 + i * RPW;
      if (lane % LPR == 0 && pi < g.p)
        for (int c = 0; c < g.c; c++) y[(((size_t)bi * g.c + c) * g.h + hi) * g.p + pi] = (T)0.0f;
    }
    return;
  }
  float* st = state + ((size_t)slot * g.h + hi) * g.p * g.r;
  f4 S[NB];
#pragma unroll
  for (int i = 0; i < NB; i++) S[i] = ld_state4(st, g.p, g.r, row0 + i * RPW, r0);
  const float dec = ex2((float)log2_decay(to_f(da[chain])));
#pragma unroll
  for (int i = 0; i < NB; i++) S[i] *= dec;
  for (int c = 0; c < g.c; c++) {
    const T* kr = k + (((size_t)bi * g.c + c) * g.g + gi) * g.r;
    const T* xr = x + (((size_t)bi * g.c + c) * g.h + hi) * g.p;
    f4 kv;
#pragma unroll
    for (int e = 0; e < 4; e++) kv[e] = r0 + e < g.r ? to_f(kr[r0 + e]) : 0.0f;
#pragma unroll
    for (int i = 0; i < NB; i++) {
      const int pi = row0 + i * RPW;
      const float xv = pi < g.p ? to_f(xr[pi]) : 0.0f;
      S[i] += xv * kv;
    }
  }
#pragma unroll
  for (int i = 0; i < NB; i++) st_state4(st, g.p, g.r, row0 + i * RPW, r0, S[i]);
  for (int c = 0; c < g.c; c++) {
    const T* qr = q + (((size_t)bi * g.c + c) * g.g + gi) * g.r;
    T* yr = y + (((size_t)bi * g.c + c) * g.h + hi) * g.p;
    f4 qv;
#pragma unroll
    for (int e = 0; e < 4; e++) qv[e] = r0 + e < g.r ? to_f(qr[r0 + e]) : 0.0f;
#pragma unroll
    for (int i = 0; i < NB; i++) {
      float v = S[i][0] * qv[0] + S[i][1] * qv[1] + S[i][2] * qv[2] + S[i][3] * qv[3];
#pragma unroll
      for (int d = 1; d < LPR; d *= 2) v += __shfl_xor(v, d);
      const int pi = row0 + i * RPW;
      if (lane % LPR == 0 && pi < g.p) yr[pi] = to_t<T>(v);
    }
  }
}

}  // namespace mom
