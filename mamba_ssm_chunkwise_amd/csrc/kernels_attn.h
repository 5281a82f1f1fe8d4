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
// Rounding. Products of bf16 values are exact in fp32. What the walk itself makes for the
// matrix instructions is split into bf16 pieces, each the rounded rest of those before: the
// decayed writes e^{a_end - a_j} x[j] into three (24 bits), so that the state, which is handed
// on to later calls, keeps fp32 accuracy, and the scores (q.k) e^{a_u - a_j} into two (17 bits),
// so that y is right to its own rounding. With scores of one piece y had 1.4 times that error,
// and up to 1.7 times in sequences of a few tokens, where single scores stand out. The second
// piece costs 8 of 105 us in 128 ragged chains of up to 4096 rows, 2 % in 32 of 240000, nothing
// where the chains fill the card (memory bounds them). Only the copy of H that y reads is
// rounded to one piece: e^{a_u} weights it, and two would cost another 7 us and 9 %.
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
  int NK;       // chunks over V tokens
  int nseg;     // segments a chain's walk is split into (each sequence splits its own length)
  int seg0;     // first segment of this launch
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

// Chunks [n0, n1) of a segment of a sequence of nkb chunks, and the share [z0, z1) of the
// tokens past its length whose outputs the segment clears.
struct Segment {
  int n0, n1, z0, z1;
  __device__ __forceinline__ Segment(const AttnGeo& g, int seg, int Vb, int nkb) {
    const int sl = (nkb + g.nseg - 1) / g.nseg, zl = (g.s - Vb + g.nseg - 1) / g.nseg;
    n0 = min(seg * sl, nkb);
    n1 = min(n0 + sl, nkb);
    z0 = min(Vb + seg * zl, g.s);
    z1 = min(z0 + zl, g.s);
  }
};

// Decays. Sums of da are kept in units of log2 as a float and its remainder
// (from a sum in double), so that differences of long sums keep 24 bits of the
// difference. A decay below e^-110 is zero in fp32: a cleared state (da = -inf among it).
// Its place in the sums is taken by kReset, so that later differences stay finite and no
// growth that fp32 can hold makes up for it. NaN stays NaN.
constexpr double kLog2e = 1.4426950408889634;
constexpr float kCleared = -110.0f;
constexpr double kReset = -150000.0;   // in log2 units; a chunk of other decays sums to -1.1e4 at least
constexpr float kGone = -1e5f;         // sums below hold a cleared state
__device__ __forceinline__ double log2_decay(float da) { return da < kCleared ? kReset : (double)da * kLog2e; }
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- types ------------------------------------------------------------------
template <typename T> struct AV;
template <> struct AV<bf16> {
  static constexpr int L = 64;    // rows per chunk
  static constexpr int PE = 8;    // elements per 16-byte piece
  static constexpr int NSPLIT = 3;
  using quad = uint2;
  using frag = bf8;
  __host__ __device__ static constexpr int pitch(int n) { return n; }
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
// COLS is 64 or 128 (32 for the float scores). bf16 rows are not padded: quad v (four
// columns, 8 bytes) of a row sits at v ^ swz(row). What 32 lanes read together, one quad
// and its neighbour of 16 rows, or (transposing reads) four quads of eight rows, then
// touches each of the 64 banks once, and the pairs of quads that 16-byte pieces are stay
// together. Measured: no conflicts in the walk over k and x, whose reads transpose; 28 to 30 %
// of the LDS cycles in the forward and 13 % in the gradients, which read row fragments and
// tables too (which of these, and why, is open). Float rows are padded by one quad instead.
template <typename T, int COLS> __device__ __forceinline__ int swz(int row) {
  if constexpr (sizeof(T) != 2) return 0;
  else if constexpr (COLS >= 128) return ((row & 7) << 2) | (((row >> 3) & 1) << 1);
  else return (((row >> 1) & 3) << 2) | (((row >> 3) & 1) << 1);
}
template <int COLS, typename T>
__device__ __forceinline__ typename AV<T>::quad ld_quad(const T* t, int row, int v) {
  return *reinterpret_cast<const typename AV<T>::quad*>(t + row * AV<T>::pitch(COLS) + 4 * (v ^ swz<T, COLS>(row)));
}
template <int COLS, typename T>
__device__ __forceinline__ void st_quad(T* t, int row, int v, typename AV<T>::quad x) {
  *reinterpret_cast<typename AV<T>::quad*>(t + row * AV<T>::pitch(COLS) + 4 * (v ^ swz<T, COLS>(row))) = x;
}
// One 16-byte piece (columns piece * PE ..) of a row.
template <int COLS, typename T>
__device__ __forceinline__ void st_piece(T* t, int row, int piece, uint4 x) {
  constexpr int PE = AV<T>::PE;
  *reinterpret_cast<uint4*>(t + row * AV<T>::pitch(COLS) + 4 * ((piece * (PE / 4)) ^ swz<T, COLS>(row))) = x;
}

// Fragment of rows row0 + lane % 16, contracted over columns 32m .. 32m + 31.
template <int COLS, typename T>
__device__ __forceinline__ typename AV<T>::frag row_frag(const T* t, int row0, int m, int lane) {
  const int row = lane & 15, q = lane >> 4;
  const T* t0 = t + row0 * AV<T>::pitch(COLS);   // row0 is a multiple of 16: no change of swz
  return join(ld_quad<COLS>(t0, row, 8 * m + q), ld_quad<COLS>(t0, row, 8 * m + 4 + q));
}
// Fragment of columns col0 + lane % 16, contracted over rows 32m .. 32m + 31.
// bf16: transposing reads; in each 16-lane group, lane j receives element j % 4
// of the 8-byte pieces that lanes 4r + j / 4 address, r = 0..3.
typedef short as4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ as4 lds_tr16(const bf16* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) as4*)p);
}
template <int COLS>
__device__ __forceinline__ bf8 col_frag(const bf16* t, int m, int col0, int lane) {
  constexpr int P = AV<bf16>::pitch(COLS);
  const int row = 4 * (lane >> 4) + ((lane >> 2) & 3);
  const bf16* p0 = t + 32 * m * P + row * P + 4 * ((col0 / 4 + (lane & 3)) ^ swz<bf16, COLS>(row));
  const as4 v[2] = {lds_tr16(p0), lds_tr16(p0 + 16 * P)};
  return __builtin_bit_cast(bf8, v);
}
template <int COLS>
__device__ __forceinline__ AV<float>::frag col_frag(const float* t, int m, int col0, int lane) {
  constexpr int P = AV<float>::pitch(COLS);
  AV<float>::frag f;
  const float* p0 = t + (32 * m + 4 * (lane >> 4)) * P + col0 + (lane & 15);
#pragma unroll
  for (int h = 0; h < 2; h++)
#pragma unroll
    for (int i = 0; i < 4; i++) f.v[h][i] = p0[(16 * h + i) * P];
  return f;
}

// An operand scaled by w per slot, to fp32 accuracy of the scaled values: in bf16 it is
// split into three bf16 pieces, each the rounded rest of those before.
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
  __device__ __forceinline__ bf8 piece(int i) const { return p[2 - i]; }   // the smallest first
};
template <>
struct Scaled<1> {
  AV<float>::frag p;
  __device__ __forceinline__ void make(const AV<float>::frag& x, f4 w0, f4 w1) { p = AV<float>::frag{{x.v[0] * w0, x.v[1] * w1}}; }
  __device__ __forceinline__ const AV<float>::frag& piece(int) const { return p; }
};

// Nothing is scheduled across: the loads before it are all issued before the matrix
// instructions behind it, which then wait for them one by one. (Left to itself the compiler
// saves registers by loading one operand pair, waiting out its latency, and so on.)
__device__ __forceinline__ void issue_fence() { __builtin_amdgcn_sched_barrier(0); }

// ---- staging ----------------------------------------------------------------
// Rows of a chunk in global memory through a buffer descriptor that ends with the last
// valid row: loads past it return zeros and stores past it are dropped by the hardware, so
// that neither needs a branch. (With branches the compiler cannot count what is in flight,
// and waiting for a chunk's loads would wait for the last chunk's stores too.) Offsets
// inside a chunk fit 32 bits: the plan refuses wider rows.
constexpr unsigned kPast = 0xFFFFFFF0u;   // an offset past every descriptor's end
using Rsrc = __amdgpu_buffer_rsrc_t;
// Rows of n elements, `stride` elements apart; none where nrows = 0 or base is nullptr.
template <typename T>
__device__ __forceinline__ Rsrc row_rsrc(const T* base, unsigned stride, int nrows, int n) {
  const unsigned bytes = base == nullptr || nrows == 0 ? 0u : ((unsigned)(nrows - 1) * stride + (unsigned)n) * (unsigned)sizeof(T);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, bytes, 0x00027000);
}
__device__ __forceinline__ uint4 buf_load(Rsrc r, unsigned off) {
  return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
}
__device__ __forceinline__ void buf_store(Rsrc r, unsigned off, uint2 v) {
  __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(unsigned __attribute__((ext_vector_type(2))), v), r, off, 0, 0);
}
__device__ __forceinline__ void buf_store(Rsrc r, unsigned off, f4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u4, v), r, off, 0, 0);
}

// A [L][COLS] block of rows on its way from global memory to an LDS tile, in 16-byte
// pieces. Rows >= nrows and columns >= n are zeros, whatever the memory there holds.
// Pieces go through registers (load, later store), so that they can be in flight while
// another chunk is worked on. VEC: rows are whole pieces. Others are fetched one element
// at a time: as many registers for floats; bf16 elements, a register each until they are
// packed, go straight into the tile (direct) instead.
template <typename T, int COLS, int NT>
struct Stage {
  static constexpr int L = AV<T>::L, PE = AV<T>::PE, PR = COLS / PE, N = (L * PR + NT - 1) / NT;
  static_assert(L * PR % NT == 0 && NT % PR == 0, "whole rows of pieces");
  uint4 v[N];
  unsigned off0, step;   // byte offset of the thread's first piece, and from one to the next
  __device__ __forceinline__ void setup(unsigned stride, int n) {
    const int row = (int)threadIdx.x / PR, c0 = (int)threadIdx.x % PR * PE;
    off0 = c0 < n ? ((unsigned)row * stride + (unsigned)c0) * (unsigned)sizeof(T) : kPast;
    step = c0 < n ? (unsigned)(NT / PR) * stride * (unsigned)sizeof(T) : 0u;
  }
  __device__ __forceinline__ void load(Rsrc r) {
#pragma unroll
    for (int i = 0; i < N; i++) v[i] = buf_load(r, off0 + (unsigned)i * step);
  }
  // One element at a time: floats of rows that are not whole pieces.
  __device__ __forceinline__ void load_each(Rsrc r, int n) {
    const int c0 = (int)threadIdx.x % PR * PE;
#pragma unroll
    for (int i = 0; i < N; i++) {
      unsigned x[4];
#pragma unroll
      for (int e = 0; e < 4; e++)
        x[e] = __builtin_amdgcn_raw_buffer_load_b32(r, c0 + e < n ? off0 + (unsigned)i * step + 4u * e : kPast, 0, 0);
      v[i] = make_uint4(x[0], x[1], x[2], x[3]);
    }
  }
  // `drop`: the rows that become zeros, whatever they hold.
  struct NoRow {
    __device__ __forceinline__ bool operator()(int) const { return false; }
  };
  template <typename F = NoRow>
  __device__ __forceinline__ void store(T* t, F drop = F{}) const {
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * NT + (int)threadIdx.x;
      st_piece<COLS>(t, e / PR, e % PR, drop(e / PR) ? make_uint4(0, 0, 0, 0) : v[i]);
    }
  }
  template <typename F = NoRow>
  __device__ __forceinline__ void direct(T* t, Rsrc r, int n, F drop = F{}) const {
    static_assert(sizeof(T) == 2, "bf16 elements");
    const int c0 = (int)threadIdx.x % PR * PE;
    unsigned short x[N][PE];
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
      for (int e = 0; e < PE; e++)
        x[i][e] = __builtin_amdgcn_raw_buffer_load_b16(r, c0 + e < n ? off0 + (unsigned)i * step + 2u * e : kPast, 0, 0);
    issue_fence();
#pragma unroll
    for (int i = 0; i < N; i++) {
      const int e = i * NT + (int)threadIdx.x;
      const uint4 v8 = make_uint4(x[i][0] | (unsigned)x[i][1] << 16, x[i][2] | (unsigned)x[i][3] << 16,
                                  x[i][4] | (unsigned)x[i][5] << 16, x[i][6] | (unsigned)x[i][7] << 16);
      st_piece<COLS>(t, e / PR, e % PR, drop(e / PR) ? make_uint4(0, 0, 0, 0) : v8);
    }
  }
};

// Rows u of a chunk on their way out: four columns c0.. of one row at a time.
template <typename T, bool VEC>
struct RowOut {
  Rsrc r;
  unsigned stride;
  int n;
  __device__ __forceinline__ RowOut(T* b, unsigned st, int nr, int cols) : r(row_rsrc(b, st, nr, cols)), stride(st), n(cols) {}
  __device__ __forceinline__ void put(int u, int c0, f4 v) const {
    const unsigned off = ((unsigned)u * stride + (unsigned)c0) * (unsigned)sizeof(T);
    if constexpr (VEC) {
      buf_store(r, c0 < n ? off : kPast, to_quad<T>(v));
    } else {
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const unsigned o = c0 + i < n ? off + (unsigned)(i * sizeof(T)) : kPast;
        if constexpr (sizeof(T) == 2)
          __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, to_t<T>(v[i])), r, o, 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[i]), r, o, 0, 0);
      }
    }
  }
};

// Per-row decay tables of a chunk, written by one wave (lane u = row u).
struct DecayTab {
  float hi[64], lo[64];   // a_u in log2 units: hi + lo
  float start[64];        // e^{a_u}
  float end[64];          // e^{a_end - a_u}
  float own[64];          // log2 decay of the token that the row opens (kReset: cleared); 0 elsewhere
  double total;           // a_end in log2 units
  double pad;             // tiles behind it start at 16 bytes
};
// Inclusive sum over the 64 lanes, in the vector unit: within rows of 16 by shifts, then
// each row's total into the next one, then the lower half's into the upper.
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double v) {
  const long long b = __builtin_bit_cast(long long, v);
  const int lo = __builtin_amdgcn_update_dpp(0, (int)b, CTRL, ROWS, 0xF, true);
  const int hi = __builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xF, true);
  return v + __builtin_bit_cast(double, ((long long)hi << 32) | (unsigned)lo);
}
__device__ __forceinline__ double wave_sum_incl(double v) {
  v = dpp_add<0x111, 0xF>(v);   // row_shr:1, 2, 4, 8 (zero shifted in)
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);   // row_bcast:15 into rows 1 and 3
  return dpp_add<0x143, 0xC>(v);   // row_bcast:31 into rows 2 and 3
}
__device__ __forceinline__ double lane63(double v) {
  const long long b = __builtin_bit_cast(long long, v);
  const unsigned lo = __builtin_amdgcn_readlane((int)b, 63), hi = __builtin_amdgcn_readlane((int)(b >> 32), 63);
  return __builtin_bit_cast(double, ((long long)hi << 32) | lo);
}
// v: log2 decay of row u = lane (zero where the row does not open a token). FORGET: for what the
// chunk leaves behind it alone: log-decays that are not finite and stand before its last
// cleared state are left out.
template <bool FORGET = false>
__device__ __forceinline__ void decay_table(DecayTab* t, double v, int lane) {
  if constexpr (FORGET) {
    const unsigned long long resets = __ballot(v == kReset);
    if (resets != 0 && lane < 63 - __builtin_clzll(resets) && !(fabs(v) < 1e30)) v = 0.0;
  }
  const double a = wave_sum_incl(v), e = lane63(a);
  const float hi = (float)a;
  t->hi[lane] = hi;
  t->lo[lane] = (float)(a - hi);
  t->start[lane] = ex2(hi);
  t->end[lane] = ex2((float)(e - a));
  t->own[lane] = (float)v;
  if (lane == 0) t->total = e;
}

// The lane number as a value that the compiler takes for a new one: LDS addresses are then
// made again for each phase of a chunk, from a few instructions, instead of being kept in
// dozens of registers over the whole loop.
template <bool ON = true>
__device__ __forceinline__ int fresh(int lane) {
  if constexpr (ON) asm volatile("" : "+v"(lane));
  return lane;
}

// v where keep, else zero, whatever v is; without a branch.
__device__ __forceinline__ float keep_if(bool keep, float v) {
  return __uint_as_float(__float_as_uint(v) & (keep ? 0xFFFFFFFFu : 0u));
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
// N stores that the hardware drops. A walk issues as many behind its first loads as each of
// its chunks has stores behind the next chunk's loads, so that waiting for loads at the top
// of the loop means the same number of younger operations on both ways in.
template <typename T, int N>
__device__ __forceinline__ void dropped_stores() {
  const Rsrc r = __builtin_amdgcn_make_buffer_rsrc(nullptr, 0, 0, 0x00027000);
#pragma unroll
  for (int i = 0; i < N; i++) buf_store(r, kPast, typename AV<T>::quad{});
}

// LDS of the walks.
template <typename T, int RT, int PW>
struct LdsA {
  static constexpr int L = AV<T>::L, RC = 16 * RT, PC = 16 * ATW * PW;   // columns of the tiles
  static constexpr int RP = AV<T>::pitch(RC), PP = AV<T>::pitch(PC), SP = AV<T>::pitch(L);
  static constexpr size_t tab = 0, k = 2 * sizeof(DecayTab), x = k + (size_t)L * RP * sizeof(T),
                          state_total = x + (size_t)L * PP * sizeof(T), q = state_total,
                          s = q + (size_t)L * RP * sizeof(T), sl = s + (size_t)L * SP * sizeof(T),
                          total = sl + (sizeof(T) == 2 ? (size_t)L * SP * sizeof(T) : 0);
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
  // the rows of both halves of the chunk in flight together, as registers allow
  constexpr int MB = PW == 1 ? NJ : 1;
#pragma unroll
  for (int m0 = 0; m0 < NJ; m0 += MB) {
    typename AV<T>::frag kf[MB][RT], xr[MB][PW];
    f4 w0[MB], w1[MB];
#pragma unroll
    for (int m = 0; m < MB; m++) {
      w0[m] = *reinterpret_cast<const f4*>(w + 32 * (m0 + m) + 4 * q);
      w1[m] = *reinterpret_cast<const f4*>(w + 32 * (m0 + m) + 16 + 4 * q);
#pragma unroll
      for (int pw = 0; pw < PW; pw++) xr[m][pw] = col_frag<LD::PC>(xs, m0 + m, 16 * (wave * PW + pw), lane);
    }
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int rt = 0; rt < RT; rt++) kf[m][rt] = col_frag<LD::RC>(ks, m0 + m, 16 * rt, lane);
    issue_fence();
    if (m0 == 0) {
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int pw = 0; pw < PW; pw++) H[pw][rt] *= dec;
    }
    Scaled<AV<T>::NSPLIT> xf[MB][PW];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int pw = 0; pw < PW; pw++) xf[m][pw].make(xr[m][pw], w0[m], w1[m]);
    // tile by tile within each piece of the scaled rows, so that consecutive matrix
    // instructions do not wait for one another's sums
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
      for (int i = 0; i < AV<T>::NSPLIT; i++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
#pragma unroll
          for (int pw = 0; pw < PW; pw++) H[pw][rt] = mma32(kf[m][rt], xf[m][pw].piece(i), H[pw][rt]);
  }
}

// A chunk token by token, for a wave whose values are not all finite: the matrix products
// give every row of a chunk its share of every other one, and a share of zero (a later
// token's, or one from before a cleared state) is NaN where the other holds a NaN or an
// infinity. Here a value meets only what reads it. Leaves y in `a` and the chunk's last state
// in H. Finite values never come here; 128 chains of 4096 rows from states of NaN, every chunk
// of them: 1180 us instead of 104.
template <typename T, int RT, int PW>
__device__ __forceinline__ void walk_tokens(f4 (&H)[PW][RT], f4 (&a)[AV<T>::L / 16][PW], const T* ks, const T* xs,
                                            const T* qs, const float* own, int c, int nrows, int wave, int lane) {
  using LD = LdsA<T, RT, PW>;
  const int ln = lane & 15, lq = lane >> 4;
#pragma unroll 1
  for (int u0 = 0; u0 < nrows; u0 += c) {
    const float log_dec = own[u0], dec = ex2(log_dec);
    const bool cleared = log_dec < kGone;
#pragma unroll
    for (int pw = 0; pw < PW; pw++)
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
#pragma unroll
        for (int e = 0; e < 4; e++) H[pw][rt][e] = cleared ? 0.0f : H[pw][rt][e] * dec;
#pragma unroll 1
    for (int u = u0; u < u0 + c; u++) {
      float x[PW];
#pragma unroll
      for (int pw = 0; pw < PW; pw++) {
        const int col = 16 * (wave * PW + pw) + ln;
        x[pw] = to_f(xs[u * LD::PP + 4 * ((col >> 2) ^ swz<T, LD::PC>(u)) + (col & 3)]);
      }
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
        const f4 kv = quad_f(ld_quad<LD::RC>(ks, u, 4 * rt + lq));
#pragma unroll
        for (int pw = 0; pw < PW; pw++) H[pw][rt] += x[pw] * kv;
      }
    }
#pragma unroll 1
    for (int u = u0; u < u0 + c; u++) {
      float v[PW];
#pragma unroll
      for (int pw = 0; pw < PW; pw++) v[pw] = 0.0f;
#pragma unroll
      for (int rt = 0; rt < RT; rt++) {
        const f4 qv = quad_f(ld_quad<LD::RC>(qs, u, 4 * rt + lq));
#pragma unroll
        for (int pw = 0; pw < PW; pw++)
          v[pw] += H[pw][rt][0] * qv[0] + H[pw][rt][1] * qv[1] + H[pw][rt][2] * qv[2] + H[pw][rt][3] * qv[3];
      }
      // the sums of state rows n stand in lanes n; they go to lane (q, u % 16) for rows 4q + e
#pragma unroll
      for (int pw = 0; pw < PW; pw++) {
        v[pw] = col4_sum(v[pw]);
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float y = __shfl(v[pw], 4 * lq + e);
#pragma unroll
          for (int ut = 0; ut < AV<T>::L / 16; ut++)
            if (ut == (u >> 4) && ln == (u & 15)) a[ut][pw][e] = y;
        }
      }
    }
  }
}

// The 16x16 tiles (ut, jt) of the scores that hold pairs j <= u, four bits each: the lower
// triangle, and, with three channels, whose tokens straddle 16 rows, the tile right of the
// diagonal too. The others stay zero.
template <int NT> struct ScoreTiles;
template <> struct ScoreTiles<4> {
  static constexpr int SB = 3;       // tiles that a wave of four has in work together
  unsigned long long list, lower;    // tile k of wave w of four: entry 4k + w; the last wave (decay tables) has least
  int n, pairs;                      // entries of `list`; of `lower`, each tile once
  __device__ __forceinline__ ScoreTiles(int c)
      : list(c == 3 ? 0xB61FEDCA98540ull : 0x5AE049D0F8Cull), lower(0xB61FEDCA98540ull), n(c == 3 ? 13 : 12),
        pairs(c == 3 ? 13 : 10) {}
};
template <> struct ScoreTiles<2> {
  static constexpr int SB = 1;
  unsigned long long list, lower;
  int n, pairs;
  __device__ __forceinline__ ScoreTiles(int c) : list(0x1540ull), lower(0x1540ull), n(c == 3 ? 4 : 3), pairs(n) {}
};

// ---- walks --------------------------------------------------------------------
// MODE 0: the forward, writing y, the last state, and with `save` the state that
//         enters each chunk as an operand copy (T, tile order);
// MODE 1: the state alone (k, x): each segment from zero, leaving its last state and
//         log2 decay in seg_loc and seg_dec, or (with save) the walk that only saves;
// MODE 2: the cotangent of the state alone, chunks in reverse: k is q, x is d_y,
//         and the weights are e^{a_u}.
// VEC: rows are whole 16-byte pieces; the next chunk's are then in flight while one is
// worked on. A chain split into segments takes three launches: the segments' own states
// (MODE 1 or 2), k_attn_scan, which joins them, and the walk itself.
//
// Why so: scores cost L (r + p) operations a row beside the state's 4 p r, so L is the
// smallest that keeps the matrix instructions in whole tiles for all four waves (64 rows in
// bf16; 32 in float, whose tiles are twice as large). Two workgroups share a CU, one's loads
// under the other's barriers; three measured no faster.
// Bound: memory where the chains fill the card. bf16, r = 128: 512 chains of 16384 rows,
// p = 64, with the saved copies, 8.6 GB in 1.89 ms (4.6 TB/s; a large copy reaches 4.75);
// 32 chains of 240000 rows, p = 128, 8.0 GB in 2.1 to 2.3 ms (3.5 to 3.8 TB/s) behind a MODE 1
// pass of 3.9 GB in 0.83 to 0.91 ms (4.3 to 4.7 TB/s), matrix pipes 32 % and vector pipes 52 %
// busy. Else the latency of a chunk: its phases depend on one another through LDS and three
// barriers (128 chains of 4096 rows, p = 64: 114 to 127 us; of ragged rows, the longest deciding:
// 103 us).
template <typename T, int RT, int PW, int MODE, bool VEC>
__global__ __launch_bounds__(ATT, 2) void k_attn_walk(AttnGeo g, const T* __restrict__ x, const T* __restrict__ k,
                                                      const T* __restrict__ q, const T* __restrict__ da,
                                                      const float* h0, T* __restrict__ y,
                                                      float* h_last, T* __restrict__ save,
                                                      float* __restrict__ seg_loc, double* __restrict__ seg_dec) {
  using LD = LdsA<T, RT, PW>;
  using V = AV<T>;
  constexpr int L = V::L, NT = L / 16, NJ = L / 32, PT16 = ATW * PW;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  DecayTab* tabs = reinterpret_cast<DecayTab*>(lds + LD::tab);   // this chunk's and the next one's
  T* ks = reinterpret_cast<T*>(lds + LD::k);
  T* xs = reinterpret_cast<T*>(lds + LD::x);
  T* qs = reinterpret_cast<T*>(lds + LD::q);
  T* ss = reinterpret_cast<T*>(lds + LD::s);
  constexpr int SP = sizeof(T) == 2 ? 2 : 1;   // pieces of a score, a tile for each
  constexpr int STILE = L * LD::SP;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lq = lane >> 4;

  // block -> (segment, p tile, chain), chains in XCD order within a segment
  const int nch = g.b * g.h;
  const int seg = g.seg0 + blockIdx.x / (nch * g.npt), rem = blockIdx.x % (nch * g.npt);
  const int item = xcd_order(rem, nch * g.npt);
  const int pt = item % g.npt, chain = item / g.npt;
  const int bi = chain / g.h, hi = chain % g.h, gi = hi / g.hpg;
  const int Vb = attn_len(g, bi), nkb = (Vb + g.CT - 1) / g.CT;
  const Segment sg(g, seg, Vb, nkb);
  const int n0 = sg.n0, nlive = sg.n1;
  const int p0 = pt * LD::PC, pn = min(g.p - p0, LD::PC);
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
  if (MODE == 0 || save != nullptr) {
    // Where k_attn_scan ran, it left every segment's there, the first one's too: h_last may be h0
    // itself, and the last segment's workgroup may be done before the first one's has started.
    if (g.nseg > 1) {
      const float* src = seg_loc + (((size_t)chain * g.nseg + seg) * g.npt + pt) * TILES;
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          H[pw][rt] = *reinterpret_cast<const f4*>(src + tile_off(RT, wave * PW + pw, rt, lane));
    } else if (h0 != nullptr) {
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
          H[pw][rt] = ld_state4(h0 + (size_t)chain * g.p * g.r, g.p, g.r, p0 + 16 * (wave * PW + pw) + ln,
                                16 * rt + 4 * lq);
    }
  }
  double acc_dec = 0.0;

  Stage<T, 16 * RT, ATT> sk, sq;
  Stage<T, LD::PC, ATT> sx;
  sk.setup(kst, g.r);
  sq.setup(kst, g.r);
  sx.setup(xst, pn);
  T dnext = (T)0.0f;                        // da of the token that row u = lane opens
  const int ltok = (lane * g.cinv) >> 16;   // the token of row u = lane
  auto chunk = [&](int i) { return MODE == 2 ? nlive - 1 - (i - n0) : i; };
  auto fetch = [&](int n) {
    const int t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    if constexpr (VEC) {
      sk.load(row_rsrc(kb + u0 * kst, kst, nrows, g.r));
      sx.load(row_rsrc(xb + u0 * xst, xst, nrows, pn));
      if constexpr (MODE == 0) sq.load(row_rsrc(qb + u0 * kst, kst, nrows, g.r));
    } else if constexpr (sizeof(T) == 4) {
      sk.load_each(row_rsrc(kb + u0 * kst, kst, nrows, g.r), g.r);
      sx.load_each(row_rsrc(xb + u0 * xst, xst, nrows, pn), pn);
      if constexpr (MODE == 0) sq.load_each(row_rsrc(qb + u0 * kst, kst, nrows, g.r), g.r);
    }
  };
  // the last wave makes each chunk's decay table while the chunk before is worked on
  constexpr int TWAVE = ATW - 1;
  auto fetch_da = [&](int n) {
    const int t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    dnext = (T)0.0f;
    if (lane < nrows && ltok * g.c == lane) dnext = dab[(size_t)(t0 + ltok) * g.h];
  };
  if (nlive > n0) {
    if (wave == TWAVE) {
      fetch_da(chunk(n0));
      decay_table<MODE == 1>(tabs, log2_decay(to_f(dnext)), lane);
      if (n0 + 1 < nlive) fetch_da(chunk(n0 + 1));
    }
    fetch(chunk(n0));
    if constexpr (VEC && MODE == 0) dropped_stores<T, NT * PW>();
  }
  if constexpr (MODE == 0) {
    for (int e = threadIdx.x; e < SP * STILE / 4; e += ATT)
      reinterpret_cast<typename V::quad*>(ss)[e] = typename V::quad{};
  }
  for (int i = n0; i < nlive; i++) {
    const int n = chunk(i), t0 = n * g.CT, nrows = min(g.CT, Vb - t0) * g.c;
    const size_t u0 = (size_t)t0 * g.c;
    const DecayTab* tab = tabs + ((i - n0) & 1);
    __syncthreads();   // the last chunk's tiles have been read
    auto to_lds = [&](auto... drop) {
      if constexpr (VEC || sizeof(T) == 4) {
        sk.store(ks, drop...);
        sx.store(xs, drop...);
        if constexpr (MODE == 0) sq.store(qs);
      } else {
        sk.direct(ks, row_rsrc(kb + u0 * kst, kst, nrows, g.r), g.r, drop...);
        sx.direct(xs, row_rsrc(xb + u0 * xst, xst, nrows, pn), pn, drop...);
        if constexpr (MODE == 0) sq.direct(qs, row_rsrc(qb + u0 * kst, kst, nrows, g.r), g.r);
      }
    };
    // In a chunk that clears the state, what stood before is dropped: weights of zero would not
    // do where it is not finite (MODE 0 sees that in y).
    const float end = (float)tab->total;
    const bool clears = MODE == 1 && end < kGone;
    if (clears) to_lds([&](int u) { return end - tab->hi[u] < kGone; });
    else to_lds();
    __syncthreads();
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

    if (i + 1 < nlive) {
      fetch(chunk(i + 1));
      if (wave == TWAVE) {
        decay_table<MODE == 1>(tabs + ((i + 1 - n0) & 1), log2_decay(to_f(dnext)), lane);
        if (i + 2 < nlive) fetch_da(chunk(i + 2));
      }
    }
    const double total = tab->total;
    acc_dec = clears ? -INFINITY : acc_dec + total;
    bool apart = false;   // this wave's values are not all finite: token by token

    if constexpr (MODE == 0) {
      // scores s[u][j] = (q[u].k[j]) e^{a_u - a_j} in 16x16 tiles (columns u)
      const int la = fresh(lane), ln = la & 15, lq = la >> 4;
      const ScoreTiles<NT> tl(g.c);
      constexpr int SB = ScoreTiles<NT>::SB;
#pragma unroll 1
      for (int b0 = 0; b0 < tl.n; b0 += ATW * SB) {
        constexpr int MB = PW == 1 ? RT / 2 : RT / 4;   // operand pairs in flight: as registers allow
        f4 a[SB];
        int ut[SB], jt[SB];
#pragma unroll
        for (int k2 = 0; k2 < SB; k2++) {
          const int code = (int)(tl.list >> (4 * min(b0 + k2 * ATW + wave, tl.n - 1))) & 15;   // past the end: the last one
          ut[k2] = 16 * (code >> 2);
          jt[k2] = 16 * (code & 3);
          a[k2] = f4{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int m0 = 0; m0 < RT / 2; m0 += MB) {
          typename V::frag kf[SB][MB], qf[SB][MB];
#pragma unroll
          for (int m = 0; m < MB; m++)
#pragma unroll
            for (int k2 = 0; k2 < SB; k2++) {
              kf[k2][m] = row_frag<LD::RC>(ks, jt[k2], m0 + m, la);
              qf[k2][m] = row_frag<LD::RC>(qs, ut[k2], m0 + m, la);
            }
          issue_fence();
#pragma unroll
          for (int m = 0; m < MB; m++)
#pragma unroll
            for (int k2 = 0; k2 < SB; k2++) a[k2] = mma32(kf[k2][m], qf[k2][m], a[k2]);
        }
        f4 jh[SB], jl[SB];
        float uh[SB], ul[SB];
#pragma unroll
        for (int k2 = 0; k2 < SB; k2++) {
          uh[k2] = tab->hi[ut[k2] + ln];
          ul[k2] = tab->lo[ut[k2] + ln];
          jh[k2] = *reinterpret_cast<const f4*>(tab->hi + jt[k2] + 4 * lq);
          jl[k2] = *reinterpret_cast<const f4*>(tab->lo + jt[k2] + 4 * lq);
        }
#pragma unroll
        for (int k2 = 0; k2 < SB; k2++) {
          // j <= u: up to the last row of u's token
          const int u = ut[k2] + ln, last = ((u * g.cinv) >> 16) * g.c + g.c - 1 - jt[k2] - 4 * lq;
#pragma unroll
          for (int e = 0; e < 4; e++)
            a[k2][e] = keep_if(e <= last, a[k2][e] * ex2((uh[k2] - jh[k2][e]) + (ul[k2] - jl[k2][e])));
#pragma unroll
          for (int i = 0; i < SP; i++) {
            const typename V::quad piece = to_quad<T>(a[k2]);
            st_quad<LD::L>(ss + i * STILE, u, jt[k2] / 4 + lq, piece);
            if (i + 1 < SP) a[k2] -= quad_f(piece);
          }
        }
      }
      typename V::frag hf[PW][RT / 2];
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int m = 0; m < RT / 2; m++) hf[pw][m] = acc_frag<T>(H[pw][2 * m], H[pw][2 * m + 1]);
      __syncthreads();
      // y[u] for this wave's rows p, all row tiles together
      constexpr int MB = PW == 1 ? RT / 2 : RT / 4;
      const int lb = fresh(lane);
      f4 a[NT][PW];
#pragma unroll
      for (int ut = 0; ut < NT; ut++)
#pragma unroll
        for (int pw = 0; pw < PW; pw++) a[ut][pw] = f4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int m0 = 0; m0 < RT / 2; m0 += MB) {
        typename V::frag qf[MB][NT];
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
          for (int ut = 0; ut < NT; ut++) qf[m][ut] = row_frag<LD::RC>(qs, 16 * ut, m0 + m, lb);
        issue_fence();
#pragma unroll
        for (int m = 0; m < MB; m++)
#pragma unroll
          for (int ut = 0; ut < NT; ut++)
#pragma unroll
            for (int pw = 0; pw < PW; pw++) a[ut][pw] = mma32(hf[pw][m0 + m], qf[m][ut], a[ut][pw]);
      }
      {
        typename V::frag xf[NJ][PW], sf[NJ][NT];
        float st[NT];
        // scores of the 32 rows j from 32m on that some u of tile ut reads (a token has up to four rows)
        auto reads = [](int ut, int m) { return 32 * m <= 16 * ut + 15 + 3; };
#pragma unroll
        for (int ut = 0; ut < NT; ut++) st[ut] = tab->start[16 * ut + (lb & 15)];
#pragma unroll
        for (int m = 0; m < NJ; m++)
#pragma unroll
          for (int pw = 0; pw < PW; pw++) xf[m][pw] = col_frag<LD::PC>(xs, m, 16 * (wave * PW + pw), lb);
#pragma unroll
        for (int i = SP - 1; i >= 0; i--) {   // the smaller pieces first
#pragma unroll
          for (int m = 0; m < NJ; m++)
#pragma unroll
            for (int ut = 0; ut < NT; ut++)
              if (reads(ut, m)) sf[m][ut] = row_frag<LD::L>(ss + i * STILE, 16 * ut, m, lb);
          issue_fence();
          if (i == SP - 1) {
#pragma unroll
            for (int ut = 0; ut < NT; ut++)
#pragma unroll
              for (int pw = 0; pw < PW; pw++) a[ut][pw] *= st[ut];
          }
#pragma unroll
          for (int m = 0; m < NJ; m++)
#pragma unroll
            for (int ut = 0; ut < NT; ut++)
#pragma unroll
              for (int pw = 0; pw < PW; pw++)
                if (reads(ut, m)) a[ut][pw] = mma32(xf[m][pw], sf[m][ut], a[ut][pw]);
        }
      }
      // Where the state that entered, a row of x or a row of k is not finite, no column of the
      // chunk's last row is (it reads them all, if only with weights of zero): the check of 4 PW
      // values finds them.
      float nan = 0.0f;
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int e = 0; e < 4; e++) nan = fmaf(a[NT - 1][pw][e], 0.0f, nan);
      apart = __any(nan != 0.0f);
      if (__builtin_expect(apart, 0)) walk_tokens<T, RT, PW>(H, a, ks, xs, qs, tab->own, g.c, nrows, wave, lane);
      const RowOut<T, VEC> yo(y + (row0 + u0) * xst + (size_t)hi * g.p + p0, xst, nrows, pn);
#pragma unroll
      for (int ut = 0; ut < NT; ut++)
#pragma unroll
        for (int pw = 0; pw < PW; pw++) yo.put(16 * ut + ln, 16 * (wave * PW + pw) + 4 * lq, a[ut][pw]);
    }
    if (clears) {
#pragma unroll
      for (int pw = 0; pw < PW; pw++)
#pragma unroll
        for (int rt = 0; rt < RT; rt++) H[pw][rt] = f4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    if (!apart)
      state_update<T, RT, PW>(H, ks, xs, MODE == 2 ? tab->start : tab->end, ex2((float)total), wave, fresh(lane));
  }

  if constexpr (MODE == 0) {
    // rows past the sequence's length are zero
    for (int u = sg.z0 * g.c + (int)(threadIdx.x / 16); u < sg.z1 * g.c; u += ATT / 16) {
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
  } else if (save == nullptr) {
    const size_t at = ((size_t)chain * g.nseg + seg) * g.npt + pt;
    if (threadIdx.x == 0) seg_dec[at] = acc_dec;
#pragma unroll
    for (int pw = 0; pw < PW; pw++)
#pragma unroll
      for (int rt = 0; rt < RT; rt++)
        *reinterpret_cast<f4*>(seg_loc + at * TILES + tile_off(RT, wave * PW + pw, rt, lane)) = H[pw][rt];
  }
}

// Joins the segments of each chain: seg_loc[seg], the state that the segment leaves from
// zero, becomes the state that it starts from (from `first`, or zeros; BACK: the segments
// in reverse). One thread for four values of a state. A chain of dependent reads: bound by
// their latency, so eight segments' are in flight together. 32 chains, p = r = 128, 16
// segments: 13 us.
template <bool BACK>
__global__ __launch_bounds__(256) void k_attn_scan(AttnGeo g, int RT, int tiles, const float* __restrict__ first,
                                                   float* __restrict__ seg_loc, const double* __restrict__ seg_dec) {
  const int pt = blockIdx.x % g.npt, chain = blockIdx.x / g.npt, e = blockIdx.y * 256 + threadIdx.x;
  if (4 * e >= tiles) return;
  const int lane = e & 63, tile = e >> 6, rt = tile % RT, pi = pt * g.PT + 16 * (tile / RT) + (lane & 15);
  f4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (first != nullptr)
    v = ld_state4(first + (size_t)chain * g.p * g.r, g.p, g.r, pi, 16 * rt + 4 * (lane >> 4));
  constexpr int U = 8;   // segments whose loads are in flight together
  for (int s0 = 0; s0 < g.nseg; s0 += U) {
    f4 loc[U];
    float dec[U];   // log2; -inf: the segment clears the state
#pragma unroll
    for (int i = 0; i < U; i++) {
      if (s0 + i < g.nseg - 1) {   // the last one's own state is not needed
        const int s = BACK ? g.nseg - 1 - s0 - i : s0 + i;
        const size_t at = ((size_t)chain * g.nseg + s) * g.npt + pt;
        loc[i] = *reinterpret_cast<const f4*>(seg_loc + at * tiles + 4 * e);
        dec[i] = (float)seg_dec[at];
      }
    }
#pragma unroll
    for (int i = 0; i < U; i++) {
      if (s0 + i < g.nseg) {
        const int s = BACK ? g.nseg - 1 - s0 - i : s0 + i;
        *reinterpret_cast<f4*>(seg_loc + (((size_t)chain * g.nseg + s) * g.npt + pt) * tiles + 4 * e) = v;
        if (s0 + i < g.nseg - 1) {
          const float w = ex2(dec[i]);
#pragma unroll
          for (int c = 0; c < 4; c++) v[c] = (dec[i] == -INFINITY ? 0.0f : v[c] * w) + loc[i][c];
        }
      }
    }
  }
}

// ---- one token per sequence -------------------------------------------------------
// state <- e^{da} state + sum_c x[c] (outer) k[c];  y[c] = state q[c], in fp32.
// LPR lanes share a state row, four columns each (r <= 4 LPR); a wave takes
// 64 / LPR rows at a time and NB such batches, with all their loads in flight first:
// the state is read and written once and is all that counts (2 * 4 p r bytes against
// 2 (2 r + 2 p) for the rest). Bound by memory: 256 sequences of 64 heads, p = 64, r = 128
// (1.08 GB): 227 to 233 us, 4.6 to 4.75 TB/s, a large copy's rate. One sequence: the launch's own time (4 us
// of the 11 that the call takes on the host).
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
  // a decay of zero clears the state whatever the slot holds (0 * NaN would not)
  const float log_dec = to_f(da[chain]), dec = ex2((float)log2_decay(log_dec));
  const bool cleared = log_dec < kCleared;
#pragma unroll
  for (int i = 0; i < NB; i++)
#pragma unroll
    for (int e = 0; e < 4; e++) S[i][e] = cleared ? 0.0f : S[i][e] * dec;
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
