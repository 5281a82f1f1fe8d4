// Gated linear recurrence with a decay for each channel: kernels.
//
//   h[t] = a[t] h[t-1] + u[t],  y[t] = h[t] silu(z[t])     (no z: y = h)
//   LOG : a = exp(g), u = x;   MIX : a = s(g), u = (1-a) x;   UNIT: a = s(g), u = sqrt(1-a^2) x
//
// A lane has V neighbouring channels and REC_R tokens that follow each other; the waves of a
// workgroup have the same channels and one run of tokens after the other, so a wave reads whole
// pieces of rows and nothing crosses lanes. A run is the map h -> P h + H of its entering state;
// the waves exchange (P, H) through LDS, once for a tile of all their runs, and every wave
// applies those before its own. The last wave hands on what enters the next tile. The next tile's
// rows are in flight meanwhile.
//
// A decay of exactly zero (one that underflows) clears: what stood before, infinities and NaN too,
// is gone. In a run's map that is a sign bit on P, which no product of decays has by itself, so a
// product that only underflows is told apart from it.
//
// Bound by memory: 8 x 8192 x 4096 bf16 with z, forward 425 us (405 to 441; 2.15 GB, 5.1 TB/s; a
// copy reaches 4.9), gradients 738 us (717 to 784; 3.76 GB, 5.1 TB/s), vector pipes 57 and 52 % busy.
// Where chain groups are too few for the card the sequence is cut into segments, whose maps take a
// second pass over x and g, but for the last segment's: 60000 tokens of 4096 channels, 248 us (213 to
// 271; 0.87 GB, 3.5 TB/s, on 224 of 256 CUs, vector pipes 64 % busy) beside the walk's 430 (2.0 GB,
// 4.7 TB/s). Workgroups that take tiles one by one and hand states on through memory instead were
// slower (553 us and a launch that clears).
#pragma once

#include <type_traits>

#include "common.h"

namespace mom {

constexpr int REC_W = 16;              // waves of a workgroup of the forward walk
template <typename T> constexpr int REC_R = 16 / sizeof(T);   // tokens of a lane there
constexpr int REC_WB = 8;              // waves of a workgroup of the gradients' walk
constexpr int REC_RB = 8;              // tokens of a lane there
constexpr int REC_TILE = REC_W * REC_R<__bf16>;   // segments are whole multiples of any tile (fp32's are 64 tokens)
constexpr int REC_SAVE = REC_WB * REC_RB;   // tokens between saved states: a tile of the gradients' walk
constexpr int REC_SW = 16;             // waves of a workgroup that makes a segment's map
constexpr int REC_SR = 8;              // its lanes' tokens in flight

struct RecGeo {
  int b, s, w;
  int V;               // min(valid_len, s)
  int ncg;             // channel groups (64 * channels of a lane)
  int nseg;            // segments of a sequence
  size_t xs, gs, zs;   // elements between tokens
  size_t xr, gr, zr;   // the same within a sequence: w where it has one token, as the next may be farther than 32 bits
  const int* lens;
};

__device__ __forceinline__ int rec_len(const RecGeo& g, int bi) {
  if (g.lens == nullptr) return g.V;
  const int v = g.lens[bi];
  return v < 0 ? 0 : (v < g.V ? v : g.V);
}

constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int V> struct RecVec { typedef T type __attribute__((ext_vector_type(V))); };
template <typename T> struct RecVec<T, 1> { typedef T type; };
template <typename T, int V> using rvec = typename RecVec<T, V>::type;

template <typename T, int V> __device__ __forceinline__ float rec_get(const rvec<T, V>& v, int i) {
  if constexpr (V == 1) return to_f(v); else return to_f((T)v[i]);
}
template <typename T, int V> __device__ __forceinline__ rvec<T, V> rec_vec(const float (&f)[V]) {
  rvec<T, V> v;
  if constexpr (V == 1) {
    v = to_t<T>(f[0]);
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) v[i] = to_t<T>(f[i]);
  }
  return v;
}
template <typename T, int V> __device__ __forceinline__ void rec_put(T* p, const float (&f)[V]) {
  *reinterpret_cast<rvec<T, V>*>(p) = rec_vec<T, V>(f);
}
template <typename T, int V> __device__ __forceinline__ rvec<T, V> rec_ld(const T* p) {
  return *reinterpret_cast<const rvec<T, V>*>(p);
}

// A wave's rows of a tensor as a buffer that ends with them: rows past the sequence's end read as
// zeros and are not written, without a branch. `n` rows from p on, `cols` columns from p's to the
// tensor's last.
using RecBuf = __amdgpu_buffer_rsrc_t;
template <typename T>
__device__ __forceinline__ RecBuf rec_buf(const T* p, size_t stride, int n, int cols) {
  const unsigned bytes = n <= 0 ? 0u : (unsigned)((n - 1) * stride + cols) * (unsigned)sizeof(T);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(p), 0, bytes, 0x00027000);
}
template <typename T, int V> __device__ __forceinline__ rvec<T, V> rec_bld(RecBuf r, unsigned off, unsigned row) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  if constexpr (sizeof(T) * V == 2) return __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(r, off, row, 0));
  else if constexpr (sizeof(T) * V == 4)
    return __builtin_bit_cast(rvec<T, V>, __builtin_amdgcn_raw_buffer_load_b32(r, off, row, 0));
  else return __builtin_bit_cast(rvec<T, V>, (u2)__builtin_amdgcn_raw_buffer_load_b64(r, off, row, 0));
}
// Stores are streamed past the caches' other lines: 8 x 8192 x 4096 bf16, forward 448 us without that,
// 407 with it, gradients 743 and 731; with a kernel that reads y at once behind it 616 and 604 us, of
// 8 x 1024 x 4096 82 and 79. (Loads likewise slow down where x and g are read twice; single 16-bit
// stores, 8 x 8192 x 4095 gradients, 1198 us without and 1750 with it, so those go without.) These two
// widths are what was measured: rows of 4- and 8-byte stores that are not whole 128-byte lines (8 x
// 8192 x 4094, 1269 us for the gradients) are streamed too, and have not been timed otherwise.
constexpr int kRecStream = 2;   // the instruction's nt bit
template <typename T, int V> __device__ __forceinline__ void rec_bst(RecBuf r, unsigned off, const float (&f)[V]) {
  typedef unsigned u2 __attribute__((ext_vector_type(2)));
  const rvec<T, V> v = rec_vec<T, V>(f);
  if constexpr (sizeof(T) * V == 2) __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, v), r, off, 0, 0);
  else if constexpr (sizeof(T) * V == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, off, 0, kRecStream);
  else __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u2, v), r, off, 0, kRecStream);
}

// Rows t0, t0 + 1, ... of a tensor at a lane's channels (p: the sequence's first row at the
// workgroup's first channel), in flight together; n rows are left. Where all R are there the rows'
// offsets are scalars (no lane is past the buffer's end: `lane_off` of one without channels is 0);
// else they stand in the lanes' own offsets, which is what the buffer's end is compared with.
template <typename T, int V, int R>
__device__ __forceinline__ void rec_rows(rvec<T, V> (&r)[R], const T* p, size_t stride, int t0, int n, int cols,
                                         unsigned lane_off) {
  const RecBuf buf = rec_buf(p + (size_t)t0 * stride, stride, min(n, R), cols);
  const unsigned step = (unsigned)stride * (unsigned)sizeof(T);
  if (n >= R) {
#pragma unroll
    for (int i = 0; i < R; i++) r[i] = rec_bld<T, V>(buf, lane_off, (unsigned)i * step);
  } else {
#pragma unroll
    for (int i = 0; i < R; i++) r[i] = rec_bld<T, V>(buf, lane_off + (unsigned)i * step, 0);
  }
}

// The decay a, and for the logistic gates b = 1 - a and the input's factor f (else 1). The
// logistic of the smaller side is q = e / (1 + e) with e = exp(-|g|); the larger is 1 - q, whose one
// rounding is half that of a reciprocal near 1 and without its bias, which a long memory would
// add up (against 64 bits, gates from 4 to 9: mean 0.065 units of 2^-24 and rms 0.65 by the
// reciprocal). sqrt(1 - a^2) = sqrt(b (1 + a)) takes the root of e as an exponential, exp(-|g| / 2),
// so that it does not vanish where b leaves the range (the instruction has no subnormal results).
template <int GATE> __device__ __forceinline__ void rec_gate(float g, float& a, float& b, float& f) {
  if constexpr (GATE == 0) {
    a = __builtin_amdgcn_exp2f(g * kLog2e);
    b = 0.0f;
    f = 1.0f;
  } else {
    const float h = __builtin_amdgcn_exp2f(-fabsf(g) * (GATE == 1 ? kLog2e : 0.5f * kLog2e));
    const float e = GATE == 1 ? h : h * h;
    const float r = __builtin_amdgcn_rcpf(1.0f + e), q = e * r;
    const float p = 1.0f - q;
    a = g < 0.0f ? q : p;
    b = g < 0.0f ? p : q;
    f = GATE == 1 ? b : __builtin_amdgcn_sqrtf(r * (1.0f + a)) * (g < 0.0f ? 1.0f : h);
  }
}

__device__ __forceinline__ float rec_sigma(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// A map applied to a state; a map after another. A state of zero stays out of it however far the
// product of a growing run's decays went (infinity times zero would be NaN).
__device__ __forceinline__ float rec_apply(float P, float H, float h) {
  return __float_as_int(P) < 0 || h == 0.0f ? H : fmaf(P, h, H);
}
__device__ __forceinline__ float rec_chain(float P, float next) { return __float_as_int(next) < 0 ? next : P * next; }

// One token. A decay of zero (CLEAR: there may be some) forgets what it meets, NaN too; where a
// wave's tokens hold none, as almost everywhere, nothing has to be compared.
template <bool CLEAR> __device__ __forceinline__ float rec_next(float a, float h, float u) {
  return CLEAR && a == 0.0f ? u : fmaf(a, h, u);
}
// The sign of a cleared map outlasts decays of the same run that are not numbers: the gradients'
// map of the run, which starts behind them, still forgets at the clearing token.
template <bool CLEAR> __device__ __forceinline__ float rec_prod(float P, float a) {
  if constexpr (CLEAR) return a == 0.0f ? -1.0f : __builtin_copysignf(P * a, P);
  else return P * a;
}
template <bool CLEAR> __device__ __forceinline__ float rec_back(float a, float d) {
  return CLEAR && a == 0.0f ? 0.0f : a * d;
}
template <int R, int V> __device__ __forceinline__ bool rec_clears(const float (&a)[R][V]) {
  float m = a[0][0];
#pragma unroll
  for (int i = 0; i < R; i++)
#pragma unroll
    for (int j = 0; j < V; j++) m = fminf(m, a[i][j]);
  return __any(m == 0.0f);
}
// Keeps what is computed of v behind this point: the compiler would move what both of rec_either's
// branches share before them, where all tokens' values are live at once.
template <typename R> __device__ __forceinline__ void rec_pin(R& v) {
  if constexpr (sizeof(R) == 2) {
    unsigned w = __builtin_bit_cast(unsigned short, v);
    asm volatile("" : "+v"(w));
    v = __builtin_bit_cast(R, (unsigned short)w);
  } else {
    asm volatile("" : "+v"(v));
  }
}
// Calls f(CLEAR) once.
template <class F> __device__ __forceinline__ void rec_either(bool clears, F&& f) {
  if (clears) f(std::integral_constant<bool, true>{});
  else f(std::integral_constant<bool, false>{});
}

// Where a workgroup stands: its sequence, its lanes' channels and its segment's tokens.
struct RecAt {
  int bi, seg, c0, ch, Vb, t0, t1;   // c0: the workgroup's first channel, ch: the lane's (0 without one)
  bool on;                           // the lane has channels
  __device__ RecAt(const RecGeo& g, int V) {
    const int items = g.b * g.ncg;
    seg = (int)blockIdx.x / items;
    const int it = (int)blockIdx.x % items;
    bi = it / g.ncg;
    c0 = (it % g.ncg) * 64 * V;
    const int c = c0 + (int)(threadIdx.x & 63) * V;
    on = c < g.w;
    ch = on ? c : 0;
    Vb = rec_len(g, bi);
    // each sequence has segments of its own length, whole tiles
    const int per = ((Vb + REC_TILE - 1) / REC_TILE + g.nseg - 1) / g.nseg * REC_TILE;
    t0 = min(seg * per, Vb);
    t1 = min(t0 + per, Vb);
  }
};

// Zeros in a segment's share of the rows past the sequence's length.
template <typename T, int V>
__device__ __forceinline__ void rec_zero_rows(const RecGeo& g, const RecAt& at, T* out, int wave, int waves) {
  if (!at.on || out == nullptr) return;
  const float zero[V] = {};
  T* p = out + ((size_t)at.bi * g.s) * g.w + at.ch;
  const int per = (g.s - at.Vb + g.nseg - 1) / g.nseg, t0 = at.Vb + at.seg * per;
  for (int t = t0 + wave; t < min(t0 + per, g.s); t += waves) rec_put<T, V>(p + (size_t)t * g.w, zero);
}

// The maps of the segments before a workgroup's own (BACK: behind it), in order, on the state that
// enters the first: every wave joins a share of them, then all apply the waves' maps. part:
// [segment][b][w] of P, then of H; first: [b][w]; sp, sh: [waves][64][V] in LDS.
template <int V, int W, bool BACK>
__device__ __forceinline__ void rec_enter(const RecGeo& g, const RecAt& at, const float* part, const float* first,
                                          float (&sp)[W][64][V], float (&sh)[W][64][V], float (&h)[V]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const size_t n = (size_t)g.b * g.w, o = (size_t)at.bi * g.w + at.ch;
  const float* hpart = part + (size_t)g.nseg * n;
  const int many = BACK ? g.nseg - 1 - at.seg : at.seg, per = (many + W - 1) / W;
  float P[V], H[V];
#pragma unroll
  for (int j = 0; j < V; j++) P[j] = 1.0f, H[j] = 0.0f, h[j] = first[o + j];
#pragma unroll 4
  for (int i = wave * per; i < min((wave + 1) * per, many); i++) {
    const size_t k = (size_t)(BACK ? g.nseg - 1 - i : i) * n + o;
#pragma unroll
    for (int j = 0; j < V; j++) {
      const float p = part[k + j];
      H[j] = rec_apply(p, hpart[k + j], H[j]);
      P[j] = rec_chain(P[j], p);
    }
  }
#pragma unroll
  for (int j = 0; j < V; j++) sp[wave][lane][j] = P[j], sh[wave][lane][j] = H[j];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < W; k++)
#pragma unroll
    for (int j = 0; j < V; j++) h[j] = rec_apply(sp[k][lane][j], sh[k][lane][j], h[j]);
  __syncthreads();
}

// The map of a segment: every wave walks a run of its own and the waves' maps are joined at the
// end. BACK: of the cotangent c[t] = a[t] (d_y[t] silu(z[t]) + c[t+1]), from the last token.
// The outermost segment also copies the state that enters it, which the caller's output may
// overwrite before another workgroup has read it.
template <typename T, int GATE, bool Z, int V, bool BACK>
__global__ __launch_bounds__(REC_SW * 64) void k_rec_seg(RecGeo g, const T* __restrict__ x, const T* __restrict__ gg,
                                                   const T* __restrict__ z, const float* __restrict__ h0,
                                                   float* __restrict__ part, float* __restrict__ first) {
  __shared__ float sp[REC_SW][64][V], sh[REC_SW][64][V];
  const RecAt at(g, V);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t n = (size_t)g.b * g.w, o = (size_t)at.bi * g.w + at.ch;
  if (at.seg == (BACK ? g.nseg - 1 : 0) && wave == 0 && at.on)
#pragma unroll
    for (int i = 0; i < V; i++) first[o + i] = h0 ? h0[o + i] : 0.0f;
  const int per = (at.t1 - at.t0 + REC_SW - 1) / REC_SW;
  const int r0 = min(at.t0 + wave * per, at.t1), r1 = min(r0 + per, at.t1);
  const size_t row = (size_t)at.bi * g.s, xst = BACK ? (size_t)g.w : g.xs;
  const T* xp = x + row * xst + at.c0;   // BACK: d_y
  const T* gp = gg + row * g.gs + at.c0;
  const T* zp = Z ? z + row * g.zs + at.c0 : nullptr;
  const int cols = g.w - at.c0;
  const unsigned lo = at.on ? (unsigned)(lane * V * (int)sizeof(T)) : 0u;
  float P[V], H[V];
#pragma unroll
  for (int i = 0; i < V; i++) P[i] = 1.0f, H[i] = 0.0f;
  constexpr int R = REC_SR;
  rvec<T, V> rx[R], rg[R], rz[R];
  const int nr = (r1 - r0 + R - 1) / R;
  auto fetch = [&](int k) {
    const int t = r0 + (BACK ? nr - 1 - k : k) * R;
    rec_rows<T, V, R>(rx, xp, xst, t, r1 - t, cols, lo);
    rec_rows<T, V, R>(rg, gp, g.gs, t, r1 - t, cols, lo);
    if constexpr (Z) rec_rows<T, V, R>(rz, zp, g.zs, t, r1 - t, cols, lo);
  };
  if (nr > 0) fetch(0);
  for (int k = 0; k < nr; k++) {
    const int cnt = r1 - r0 - (BACK ? nr - 1 - k : k) * R;
    float a[R][V], u[R][V];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
      for (int j = 0; j < V; j++) {
        float b, f;
        rec_gate<GATE>(rec_get<T, V>(rg[i], j), a[i][j], b, f);
        u[i][j] = rec_get<T, V>(rx[i], j);
        if constexpr (!BACK && GATE != 0) u[i][j] *= f;
        if constexpr (Z) {
          const float zz = rec_get<T, V>(rz[i], j);
          u[i][j] *= zz * rec_sigma(zz);
        }
        rec_pin(a[i][j]);
        rec_pin(u[i][j]);
      }
    if (k + 1 < nr) fetch(k + 1);
    if (cnt < R)
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) a[i][j] = i < cnt ? a[i][j] : 1.0f;
    rec_either(rec_clears<R, V>(a), [&](auto cl) {
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
          const int q = BACK ? R - 1 - i : i;
          if constexpr (BACK) H[j] = rec_back<cl.value>(a[q][j], u[q][j] + H[j]);
          else H[j] = rec_next<cl.value>(a[q][j], H[j], u[q][j]);
          P[j] = rec_prod<cl.value>(P[j], a[q][j]);
        }
    });
  }
#pragma unroll
  for (int j = 0; j < V; j++) sp[wave][lane][j] = P[j], sh[wave][lane][j] = H[j];
  __syncthreads();
  if (wave != 0 || !at.on) return;
  for (int k = 1; k < REC_SW; k++) {
    const int from = BACK ? REC_SW - 1 - k : k;
    if (k == 1 && BACK)
#pragma unroll
      for (int j = 0; j < V; j++) P[j] = sp[REC_SW - 1][lane][j], H[j] = sh[REC_SW - 1][lane][j];
#pragma unroll
    for (int j = 0; j < V; j++) {
      H[j] = rec_apply(sp[from][lane][j], sh[from][lane][j], H[j]);
      P[j] = rec_chain(P[j], sp[from][lane][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < V; j++) {
    part[(size_t)at.seg * n + o + j] = P[j];
    part[(size_t)(g.nseg + at.seg) * n + o + j] = H[j];
  }
}

// The forward walk of a segment. OUT: with y; else only the states that `save` keeps, the one
// entering every REC_SAVE tokens, [b][ceil(V / REC_SAVE)][w].
template <typename T, int GATE, bool Z, int V, bool OUT>
__global__ __launch_bounds__(REC_W * 64) void k_rec_fwd(RecGeo g, const T* __restrict__ x, const T* __restrict__ gg,
                                                   const T* __restrict__ z, const float* h0,
                                                   const float* __restrict__ part, const float* __restrict__ first,
                                                   T* __restrict__ y, float* h_last, float* __restrict__ save) {
  constexpr int R = REC_R<T>, W = REC_W, TL = W * R;
  __shared__ float sp[2][W][64][V], sh[2][W][64][V], se[2][64][V];
  const RecAt at(g, V);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t row = (size_t)at.bi * g.s, o = (size_t)at.bi * g.w + at.ch;
  const T* xp = x + row * g.xs + at.c0;
  const T* gp = gg + row * g.gs + at.c0;
  const T* zp = Z ? z + row * g.zs + at.c0 : nullptr;
  T* yp = OUT ? y + row * g.w + at.c0 : nullptr;
  const int cols = g.w - at.c0, nsv = (g.V + REC_SAVE - 1) / REC_SAVE;
  const unsigned lo = at.on ? (unsigned)(lane * V * (int)sizeof(T)) : 0u, step = (unsigned)g.w * (unsigned)sizeof(T);
  float h[V], last[V];   // last: past the tile so far, in the last wave
  if (g.nseg > 1) {
    rec_enter<V, W, false>(g, at, part, first, sp[0], sh[0], h);
  } else {
#pragma unroll
    for (int j = 0; j < V; j++) h[j] = h0 ? h0[o + j] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < V; j++) last[j] = h[j];
  rvec<T, V> rx[R], rg[R], rz[R];
  auto fetch = [&](int t) {
    rec_rows<T, V, R>(rx, xp, g.xr, t, at.Vb - t, cols, lo);
    rec_rows<T, V, R>(rg, gp, g.gr, t, at.Vb - t, cols, lo);
    if constexpr (Z && OUT) rec_rows<T, V, R>(rz, zp, g.zr, t, at.Vb - t, cols, lo);
  };
  if (at.t0 < at.t1) fetch(at.t0 + wave * R);
  int buf = 0;
  for (int t = at.t0; t < at.t1; t += TL, buf ^= 1) {
    const int tw = t + wave * R, cnt = at.Vb - tw;   // this wave's tokens
    float a[R][V], u[R][V], P[V], H[V];
    rvec<T, V> cz[R];
#pragma unroll
    for (int i = 0; i < R; i++) {
      if constexpr (Z && OUT) cz[i] = rz[i];
#pragma unroll
      for (int j = 0; j < V; j++) {
        float b, f;
        rec_gate<GATE>(rec_get<T, V>(rg[i], j), a[i][j], b, f);
        const float v = rec_get<T, V>(rx[i], j);
        u[i][j] = GATE == 0 ? v : f * v;
        rec_pin(a[i][j]);
        rec_pin(u[i][j]);
      }
    }
    if (t + TL < at.t1) fetch(tw + TL);
    if (cnt < R)   // padding hands the state on
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) a[i][j] = i < cnt ? a[i][j] : 1.0f;
    const bool clears = rec_clears<R, V>(a);
    rec_either(clears, [&](auto cl) {
#pragma unroll
      for (int j = 0; j < V; j++) P[j] = 1.0f, H[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
          P[j] = rec_prod<cl.value>(P[j], a[i][j]);
          H[j] = rec_next<cl.value>(a[i][j], H[j], u[i][j]);
        }
    });
#pragma unroll
    for (int j = 0; j < V; j++) sp[buf][wave][lane][j] = P[j], sh[buf][wave][lane][j] = H[j];
    __syncthreads();   // each buffer is written again only past the next one
    if (t > at.t0)
#pragma unroll
      for (int j = 0; j < V; j++) h[j] = se[buf ^ 1][lane][j];
#pragma unroll
    for (int k = 0; k < W - 1; k++)
      if (k < wave)
#pragma unroll
        for (int j = 0; j < V; j++) h[j] = rec_apply(sp[buf][k][lane][j], sh[buf][k][lane][j], h[j]);
    if (save != nullptr && (wave * R) % REC_SAVE == 0 && tw < at.Vb && at.on) {
      float* sv = save + ((size_t)at.bi * nsv + tw / REC_SAVE) * g.w + at.ch;
#pragma unroll
      for (int j = 0; j < V; j++) sv[j] = h[j];
    }
    if (wave == W - 1)
#pragma unroll
      for (int j = 0; j < V; j++) se[buf][lane][j] = last[j] = rec_apply(P[j], H[j], h[j]);
    if constexpr (OUT) {
      const RecBuf yb = rec_buf(yp + (size_t)tw * g.w, (size_t)g.w, min(cnt, R), cols);
      if (at.on) rec_either(clears, [&](auto cl) {
#pragma unroll
        for (int i = 0; i < R; i++) {
          float out[V];
          if constexpr (Z) rec_pin(cz[i]);
#pragma unroll
          for (int j = 0; j < V; j++) {
            h[j] = rec_next<cl.value>(a[i][j], h[j], u[i][j]);
            out[j] = h[j];
            if constexpr (Z) {
              const float zz = rec_get<T, V>(cz[i], j);
              out[j] *= zz * rec_sigma(zz);
            }
          }
          rec_bst<T, V>(yb, lo + (unsigned)i * step, out);
        }
      });
    }
  }
  if constexpr (OUT) {
    if (h_last != nullptr && at.seg == g.nseg - 1) {
      __syncthreads();   // h_last may be h0: every wave has read it
      if (wave == W - 1 && at.on)
#pragma unroll
        for (int j = 0; j < V; j++) h_last[o + j] = last[j];
    }
    rec_zero_rows<T, V>(g, at, y, wave, W);
  }
}

// The gradients' walk of a segment, from its last tile to its first: the states of a tile again
// from the saved one that enters it, and the cotangent c[t] = a[t] delta[t] that the tokens hand
// to the left, the waves' maps of both exchanged at once.
template <typename T, int GATE, bool Z, int V>
__global__ __launch_bounds__(REC_WB * 64) void k_rec_bwd(RecGeo g, const T* __restrict__ x, const T* __restrict__ gg,
                                                   const T* __restrict__ z, const float* __restrict__ save,
                                                   const T* __restrict__ dy, const float* d_last,
                                                   const float* __restrict__ part, const float* __restrict__ first,
                                                   T* __restrict__ d_x, T* __restrict__ d_g, T* __restrict__ d_z,
                                                   float* d_h0) {
  constexpr int R = REC_RB, W = REC_WB, TL = REC_SAVE;
  __shared__ float sp[2][W][64][V], sh[2][W][64][V], sc[2][W][64][V], se[2][64][V];
  const RecAt at(g, V);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const size_t row = (size_t)at.bi * g.s, o = (size_t)at.bi * g.w + at.ch;
  const T* xp = x + row * g.xs + at.c0;
  const T* gp = gg + row * g.gs + at.c0;
  const T* zp = Z ? z + row * g.zs + at.c0 : nullptr;
  const T* dp = dy + row * g.w + at.c0;
  const size_t out0 = row * g.w + at.c0;
  const int cols = g.w - at.c0, nsv = (g.V + TL - 1) / TL;
  const unsigned lo = at.on ? (unsigned)(lane * V * (int)sizeof(T)) : 0u, step = (unsigned)g.w * (unsigned)sizeof(T);
  const float* sv = save + (size_t)at.bi * nsv * g.w + at.ch;
  float c[V], last[V];   // from the right; last: before the tile so far, in the first wave
  if (g.nseg > 1) {
    rec_enter<V, W, true>(g, at, part, first, sp[0], sh[0], c);
  } else {
#pragma unroll
    for (int j = 0; j < V; j++) c[j] = d_last ? d_last[o + j] : 0.0f;
  }
#pragma unroll
  for (int j = 0; j < V; j++) last[j] = c[j];
  rvec<T, V> rx[R], rg[R], rz[R], rd[R];
  float hs[V];
  auto fetch = [&](int n) {
    const int t = at.t0 + n * TL + wave * R;
    rec_rows<T, V, R>(rx, xp, g.xr, t, at.Vb - t, cols, lo);
    rec_rows<T, V, R>(rg, gp, g.gr, t, at.Vb - t, cols, lo);
    if constexpr (Z) rec_rows<T, V, R>(rz, zp, g.zr, t, at.Vb - t, cols, lo);
    rec_rows<T, V, R>(rd, dp, (size_t)g.w, t, at.Vb - t, cols, lo);
#pragma unroll
    for (int j = 0; j < V; j++) hs[j] = sv[(size_t)(at.t0 / TL + n) * g.w + j];
  };
  const int nt = (at.t1 - at.t0 + TL - 1) / TL;
  if (nt > 0) fetch(nt - 1);
  int buf = 0;
  for (int n = nt - 1; n >= 0; n--, buf ^= 1) {
    const int tw = at.t0 + n * TL + wave * R, cnt = at.Vb - tw;
    float a[R][V], b[R][V], f[R][V], xx[R][V], s[R][V], dz[R][V], P[V], H[V], C[V], h[V];
#pragma unroll
    for (int j = 0; j < V; j++) h[j] = hs[j];
#pragma unroll
    for (int i = 0; i < R; i++)
#pragma unroll
      for (int j = 0; j < V; j++) {
        rec_gate<GATE>(rec_get<T, V>(rg[i], j), a[i][j], b[i][j], f[i][j]);
        xx[i][j] = rec_get<T, V>(rx[i], j);
        s[i][j] = rec_get<T, V>(rd[i], j);
        if constexpr (Z) {   // d_y silu'(z), for the state, and d_y silu(z)
          const float zz = rec_get<T, V>(rz[i], j), sg = rec_sigma(zz), ds = s[i][j] * sg;
          dz[i][j] = ds * fmaf(zz, 1.0f - sg, 1.0f);
          s[i][j] = ds * zz;
          rec_pin(dz[i][j]);
        }
        rec_pin(a[i][j]);
        rec_pin(f[i][j]);
        rec_pin(s[i][j]);
      }
    if (n > 0) fetch(n - 1);
    if (cnt < R)
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) a[i][j] = i < cnt ? a[i][j] : 1.0f;
    const bool clears = rec_clears<R, V>(a);
    rec_either(clears, [&](auto cl) {
#pragma unroll
      for (int j = 0; j < V; j++) P[j] = 1.0f, H[j] = 0.0f, C[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; i++)
#pragma unroll
        for (int j = 0; j < V; j++) {
          P[j] = rec_prod<cl.value>(P[j], a[i][j]);
          H[j] = rec_next<cl.value>(a[i][j], H[j], GATE == 0 ? xx[i][j] : f[i][j] * xx[i][j]);
          C[j] = rec_back<cl.value>(a[R - 1 - i][j], s[R - 1 - i][j] + C[j]);
        }
    });
#pragma unroll
    for (int j = 0; j < V; j++)
      sp[buf][wave][lane][j] = P[j], sh[buf][wave][lane][j] = H[j], sc[buf][wave][lane][j] = C[j];
    __syncthreads();
    if (n < nt - 1)
#pragma unroll
      for (int j = 0; j < V; j++) c[j] = se[buf ^ 1][lane][j];
#pragma unroll
    for (int k = 0; k < W - 1; k++)
      if (k < wave)
#pragma unroll
        for (int j = 0; j < V; j++) h[j] = rec_apply(sp[buf][k][lane][j], sh[buf][k][lane][j], h[j]);
#pragma unroll
    for (int k = W - 1; k > 0; k--)
      if (k > wave)
#pragma unroll
        for (int j = 0; j < V; j++) c[j] = rec_apply(sp[buf][k][lane][j], sc[buf][k][lane][j], c[j]);
    if (wave == 0)
#pragma unroll
      for (int j = 0; j < V; j++) se[buf][lane][j] = last[j] = rec_apply(P[j], C[j], c[j]);
    const size_t e = out0 + (size_t)tw * g.w;
    const RecBuf zb = rec_buf(d_z + e, (size_t)g.w, Z && d_z ? min(cnt, R) : 0, cols);
    const RecBuf xb = rec_buf(d_x + e, (size_t)g.w, d_x ? min(cnt, R) : 0, cols);
    const RecBuf gb = rec_buf(d_g + e, (size_t)g.w, d_g ? min(cnt, R) : 0, cols);
    if (at.on) rec_either(clears, [&](auto cl) {
#pragma unroll
      for (int i = 0; i < R; i++) {
        float out[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
          const float before = h[j];
          h[j] = rec_next<cl.value>(a[i][j], h[j], GATE == 0 ? xx[i][j] : f[i][j] * xx[i][j]);
          out[j] = dz[i][j] * h[j];
          dz[i][j] = before;   // for d_g
        }
        if constexpr (Z) rec_bst<T, V>(zb, lo + (unsigned)i * step, out);
      }
#pragma unroll
      for (int i = R - 1; i >= 0; i--) {
        float ox[V], og[V];
#pragma unroll
        for (int j = 0; j < V; j++) {
          const float d = s[i][j] + c[j], aa = a[i][j], before = dz[i][j];
          float q;
          if constexpr (GATE == 0) {
            ox[j] = d;
            q = before;
          } else {
            ox[j] = f[i][j] * d;
            if constexpr (GATE == 1) q = b[i][j] * (before - xx[i][j]);
            else q = b[i][j] * before - aa * xx[i][j] * (f[i][j] * __builtin_amdgcn_rcpf(1.0f + aa));
          }
          c[j] = rec_back<cl.value>(aa, d);
          og[j] = rec_back<cl.value>(aa, q * d);
        }
        const unsigned off = lo + (unsigned)i * step;
        rec_bst<T, V>(xb, off, ox);
        rec_bst<T, V>(gb, off, og);
      }
    });
  }
  if (d_h0 != nullptr && at.seg == 0) {
    __syncthreads();   // d_h0 may be d_h_last: every wave has read it
    if (wave == 0 && at.on)
#pragma unroll
      for (int j = 0; j < V; j++) d_h0[o + j] = last[j];
  }
  rec_zero_rows<T, V>(g, at, d_x, wave, W);
  rec_zero_rows<T, V>(g, at, d_g, wave, W);
  if constexpr (Z) rec_zero_rows<T, V>(g, at, d_z, wave, W);
}

// One token of each sequence on a pool of states.
template <typename T, int GATE, bool Z, int V>
__global__ __launch_bounds__(256) void k_rec_step(RecGeo g, const T* __restrict__ x, const T* __restrict__ gg,
                                                  const T* __restrict__ z, const int* __restrict__ slots, int64_t nslots,
                                                  float* __restrict__ state, T* __restrict__ y) {
  const int ch = ((int)blockIdx.x * 256 + (int)threadIdx.x) * V;
  if (ch >= g.w) return;
  for (int bi = blockIdx.y; bi < g.b; bi += gridDim.y) {
    const int64_t slot = slots ? (int64_t)slots[bi] : (int64_t)bi;
    T* yp = y + (size_t)bi * g.w + ch;
    float out[V] = {};
    if (slot >= 0 && slot < nslots && rec_len(g, bi) > 0) {
      float* sp = state + (size_t)slot * g.w + ch;
      const rvec<T, V> vx = rec_ld<T, V>(x + (size_t)bi * g.xs + ch), vg = rec_ld<T, V>(gg + (size_t)bi * g.gs + ch);
      rvec<T, V> vz;
      if constexpr (Z) vz = rec_ld<T, V>(z + (size_t)bi * g.zs + ch);
      rvec<float, V> st = rec_ld<float, V>(sp);
      float h[V];
#pragma unroll
      for (int j = 0; j < V; j++) {
        float a, b, f;
        rec_gate<GATE>(rec_get<T, V>(vg, j), a, b, f);
        const float v = rec_get<T, V>(vx, j);
        h[j] = rec_next<true>(a, rec_get<float, V>(st, j), GATE == 0 ? v : f * v);
        out[j] = h[j];
        if constexpr (Z) {
          const float zz = rec_get<T, V>(vz, j);
          out[j] *= zz * rec_sigma(zz);
        }
      }
      rec_put<float, V>(sp, h);
    }
    rec_put<T, V>(yp, out);
  }
}

}  // namespace mom
