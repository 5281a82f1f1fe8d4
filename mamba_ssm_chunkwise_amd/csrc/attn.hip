// C ABI of linear attention with a decay for each head: validation, planning,
// dispatch. The operation and its conventions are stated in include/moments.h.
#include "moments.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "host.h"
#include "kernels_attn.h"
#include "kernels_attn_bwd.h"

using namespace mom;

namespace {

struct AttnPlan {
  AttnGeo g;    // forward walk
  AttnGeo gb;   // backward walk (segments of its own)
  bool bf, empty;
  bool bwd;     // few enough items for the gradients' launch
  bool vec;     // rows of r and of p are whole 16-byte pieces
  bool part;    // d_q, d_k (and d_da) by slices that k_attn_sum adds
  int RT;       // 16-column tiles of r: 4 or 8
  bool wide;    // 128 rows of p a workgroup (bf16, p > 64), else 64
  int items;    // chains times p tiles
  size_t seg_dec, save, seg_loc_b, seg_dec_b, part_q, part_k, part_da;  // workspace offsets (seg_loc at 0)
  size_t ws_fwd, ws_bwd, flag_bwd, saved;
};

// Segments a chain's walk is split into: one when the chains alone nearly fill the `want`
// places that the chip has for workgroups of the walk, else as many as fill them, of four
// chunks or more (two, up to eight segments). Measured on 32 chains of 8192 tokens, the launches'
// times together: one segment 465 us, 4: 189, 8: 114, 16 (taken): 102, 32: 116; on 8 chains:
// 16: 61, 32 (taken): 46, 64: 51.
void split(AttnGeo& g, int items, long want) {
  long n = 1;
  if ((long)items * 4 < want * 3)
    n = std::min<long>((want + items - 1) / items, std::max(g.NK / 4, std::min(g.NK / 2, 8)));
  g.nseg = (int)std::max<long>(1, n);
  g.seg0 = 0;
}

int make_attn_plan(const moments_attn_desc* d, AttnPlan* P) {
  if (d == nullptr) return MOMENTS_EINVAL;
  if (d->b < 0 || d->s < 0 || d->h < 0 || d->c < 1 || d->g < 1 || d->p < 1 || d->r < 1) return MOMENTS_EINVAL;
  if (d->h % d->g != 0 || d->valid_len < 0) return MOMENTS_EINVAL;
  if (d->dtype != MOMENTS_F32 && d->dtype != MOMENTS_BF16) return MOMENTS_EINVAL;
  if (d->r > 128 || d->c > 4 || d->p > 4096 || d->s > (int64_t)1 << 28) return MOMENTS_ENOTSUP;
  if (d->b > (int64_t)1 << 24 || d->h > (int64_t)1 << 20 || d->b * d->h > (int64_t)1 << 24) return MOMENTS_ENOTSUP;
  // a token row of a tensor: the kernels address the rows of a chunk with 32-bit offsets
  if (d->h * d->p > (int64_t)1 << 23 || d->h * d->r > (int64_t)1 << 23) return MOMENTS_ENOTSUP;
  if (d->g > (int64_t)1 << 20) return MOMENTS_ENOTSUP;   // with h = 0, that is: else g <= h
  P->empty = d->b == 0 || d->h == 0;
  P->bf = d->dtype == MOMENTS_BF16;
  const int tsz = P->bf ? 2 : 4, L = P->bf ? AV<bf16>::L : AV<float>::L;
  AttnGeo& g = P->g;
  g = AttnGeo{};
  g.b = (int)d->b; g.s = (int)d->s; g.c = (int)d->c; g.h = (int)d->h; g.g = (int)d->g; g.p = (int)d->p; g.r = (int)d->r;
  g.V = (int)std::min(d->valid_len, d->s);
  g.hpg = P->empty ? 1 : g.h / g.g;
  g.CT = L / g.c;
  g.NK = (g.V + g.CT - 1) / g.CT;
  g.cinv = (65536 + g.c - 1) / g.c;
  // Rows of whole 16-byte pieces are fetched a chunk ahead; others, which such loads cannot
  // address, element by element. Aligned shapes, either way: float, 32 chains of 3800 rows,
  // forward 49 and 63 us, gradients 97 and 113; bf16, 512 of 16384, 1.87 and 3.99 ms, 3.5 and 8.7 ms.
  P->vec = (g.r * tsz) % 16 == 0 && (g.p * tsz) % 16 == 0;
  g.lens = (const int*)d->valid_lens;
  // Half the columns where they do: r = 64, float, 32 chains of 3800 rows, 4 tiles 45 us for the
  // segments' states both ways, 49 for the walk and 97 for the gradients, 8 tiles 66, 77 and 159.
  P->RT = g.r <= 64 ? 4 : 8;
  // All of up to 128 state rows to a workgroup, so that keys and scores are made once:
  // 32 chains of 240000 rows, p = 128, 0.88 ms for the segments' states and 2.20 for the walk;
  // two workgroups of 64 each 1.04 and 2.87. Float, whose LDS tiles are
  // twice as large, stays at 64.
  P->wide = P->bf && g.p > 64;
  g.PT = P->wide ? 128 : 64;
  g.npt = (g.p + g.PT - 1) / g.PT;
  P->items = g.b * g.h * g.npt;
  // A launch holds fewer than 2^32 threads: the walks take 256 for each item, the gradients 512
  // (attn_bwd and the size of its workspace refuse those that are too many for them alone).
  const int64_t items = (int64_t)g.b * g.h * g.npt;
  if (items >= ((int64_t)1 << 32) / ATT || (int64_t)g.h * g.npt * g.r > (int64_t)1 << 23) return MOMENTS_ENOTSUP;
  P->bwd = items < ((int64_t)1 << 32) / ABT;
  P->gb = g;
  if (!P->empty) {
    split(g, P->items, 2 * kCUs);      // two workgroups of the walk share a CU
    split(P->gb, P->items, kCUs);      // one of the backward
  }
  P->part = g.hpg > 1 || g.npt > 1;
  const size_t tiles = (size_t)(g.PT / 16) * P->RT * 256;
  size_t o = 0;
  if (g.nseg > 1) o = align256(o + (size_t)P->items * g.nseg * tiles * 4);
  P->seg_dec = o;
  if (g.nseg > 1) o = align256(o + (size_t)P->items * g.nseg * 8);
  P->ws_fwd = o;   // nothing with one segment
  P->saved = (size_t)P->items * g.NK * tiles * tsz;
  P->save = o;
  o = align256(o + P->saved);
  P->seg_loc_b = o;
  if (P->gb.nseg > 1) o = align256(o + (size_t)P->items * P->gb.nseg * tiles * 4);
  P->seg_dec_b = o;
  if (P->gb.nseg > 1) o = align256(o + (size_t)P->items * P->gb.nseg * 8);
  const size_t rows = (size_t)g.b * g.s * g.c * g.h * g.npt;
  P->part_q = o;
  if (P->part) o = align256(o + rows * g.r * 4);
  P->part_k = o;
  if (P->part) o = align256(o + rows * g.r * 4);
  P->part_da = o;
  if (P->part) o = align256(o + (size_t)g.b * g.s * g.h * g.npt * 4);
  P->flag_bwd = o;
  P->ws_bwd = o + 256;
  return MOMENTS_OK;
}

// Calls f(TT<T>, IC<RT>, IC<PW>, IC<VEC>) for the compiled variant of the plan.
template <class F>
int with_attn(const AttnPlan& P, F&& f) {
  auto by_vec = [&](auto tt, auto rt, auto pw) -> int {
    return P.vec ? f(tt, rt, pw, IC<1>{}) : f(tt, rt, pw, IC<0>{});
  };
  if (P.bf) {
    if (P.RT == 4) return P.wide ? by_vec(TT<bf16>{}, IC<4>{}, IC<2>{}) : by_vec(TT<bf16>{}, IC<4>{}, IC<1>{});
    return P.wide ? by_vec(TT<bf16>{}, IC<8>{}, IC<2>{}) : by_vec(TT<bf16>{}, IC<8>{}, IC<1>{});
  }
  return P.RT == 4 ? by_vec(TT<float>{}, IC<4>{}, IC<1>{}) : by_vec(TT<float>{}, IC<8>{}, IC<1>{});
}

template <typename T, int RT, int PW, int MODE, bool VEC>
int launch_walk(const AttnGeo& g, int nseg, const T* x, const T* k, const T* q, const T* da, const float* h0, T* y,
                float* h_last, T* save, float* seg_loc, double* seg_dec, hipStream_t st) {
  using LD = LdsA<T, RT, PW>;
  const size_t lds = MODE == 0 ? LD::total : LD::state_total;
  static std::atomic<uint64_t> done{0};
  MOM_TRY(set_lds_once(done, k_attn_walk<T, RT, PW, MODE, VEC>, lds));
  ProfScope ps(MODE == 0 ? KID_ATTN_FWD : KID_ATTN_STATE, st);
  hipLaunchKernelGGL((k_attn_walk<T, RT, PW, MODE, VEC>), dim3((unsigned)((size_t)g.b * g.h * g.npt * nseg)), dim3(ATT),
                     lds, st, g, x, k, q, da, h0, y, h_last, save, seg_loc, seg_dec);
  return check_launch();
}

int launch_scan(const AttnPlan& P, const AttnGeo& g, bool back, const float* first, float* seg_loc,
                const double* seg_dec, hipStream_t st) {
  const int tiles = (g.PT / 16) * P.RT * 256;
  const dim3 grid((unsigned)P.items, (unsigned)((tiles / 4 + 255) / 256));
  ProfScope ps(KID_ATTN_SCAN, st);
  if (back)
    hipLaunchKernelGGL(k_attn_scan<true>, grid, dim3(256), 0, st, g, P.RT, tiles, first, seg_loc, seg_dec);
  else
    hipLaunchKernelGGL(k_attn_scan<false>, grid, dim3(256), 0, st, g, P.RT, tiles, first, seg_loc, seg_dec);
  return check_launch();
}

// The states that the segments of the forward walk start from.
template <typename T, int RT, int PW, bool VEC>
int run_segments(const AttnPlan& P, const T* x, const T* k, const T* da, const float* h0, unsigned char* ws,
                 hipStream_t st) {
  if (P.g.nseg < 2) return 0;
  float* seg = (float*)ws;
  double* dec = (double*)(ws + P.seg_dec);
  MOM_TRY((launch_walk<T, RT, PW, 1, VEC>(P.g, P.g.nseg - 1, x, k, nullptr, da, nullptr, nullptr, nullptr, nullptr,
                                          seg, dec, st)));
  return launch_scan(P, P.g, false, h0, seg, dec, st);
}

int attn_fwd(const moments_attn_desc* desc, const void* x, const void* k, const void* q, const void* da,
             const float* h0, void* y, float* h_last, void* saved, size_t saved_bytes, bool want_saved,
             void* workspace, size_t workspace_bytes, void* stream) {
  AttnPlan P;
  MOM_TRY(make_attn_plan(desc, &P));
  if (P.empty) return 0;
  if (P.g.s > 0 && (!x || !k || !q || !da || !y)) return MOMENTS_EINVAL;
  if (want_saved && P.saved > 0 && saved == nullptr) return MOMENTS_EINVAL;
  if (want_saved && saved_bytes < P.saved) return MOMENTS_EWORKSPACE;
  const void* ptrs[] = {x, k, q, da, h0, y, h_last, saved, workspace};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  if (workspace_bytes < P.ws_fwd || (P.ws_fwd > 0 && workspace == nullptr)) return MOMENTS_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  float* seg = P.g.nseg > 1 ? (float*)ws : nullptr;
  double* sdec = P.g.nseg > 1 ? (double*)(ws + P.seg_dec) : nullptr;
  MOM_TRY(with_attn(P, [&](auto tt, auto rt, auto pw, auto vec) -> int {
    constexpr bool VEC = decltype(vec)::value != 0;
    using T = typename decltype(tt)::type;
    constexpr int RT = decltype(rt)::value, PW = decltype(pw)::value;
    MOM_TRY((run_segments<T, RT, PW, VEC>(P, (const T*)x, (const T*)k, (const T*)da, h0, ws, st)));
    return launch_walk<T, RT, PW, 0, VEC>(P.g, P.g.nseg, (const T*)x, (const T*)k, (const T*)q, (const T*)da, h0, (T*)y,
                                     h_last, want_saved ? (T*)saved : nullptr, seg, sdec, st);
  }));
  if (check_finite_on()) {
    const OutSpan outs[] = {{y, (size_t)P.g.b * P.g.s * P.g.c * P.g.h * P.g.p, !P.bf},
                            {h_last, (size_t)P.g.b * P.g.h * P.g.p * P.g.r, true}};
    return check_finite(outs, 2, nullptr, st);
  }
  return 0;
}

// Gradients where there are no sequences or no heads: those of keys and queries may hold
// values, and are zero (sums of no slices).
int attn_bwd_empty(const AttnPlan& P, void* d_k, void* d_q, hipStream_t st) {
  const AttnGeo& g = P.g;
  const size_t keys = (size_t)g.b * g.s * g.c * g.g * g.r;
  if (keys == 0 || (d_k == nullptr && d_q == nullptr)) return 0;
  const SumJobs jobs = {{{nullptr, d_q, d_q ? keys : 0, 0, g.r}, {nullptr, d_k, d_k ? keys : 0, 0, g.r}, {}}};
  ProfScope ps(KID_ATTN_SUM, st);
  const dim3 grid((unsigned)std::min<size_t>((keys + 255) / 256, 16384), 2);
  if (P.bf)
    hipLaunchKernelGGL((k_attn_sum<bf16>), grid, dim3(256), 0, st, jobs);
  else
    hipLaunchKernelGGL((k_attn_sum<float>), grid, dim3(256), 0, st, jobs);
  return check_launch();
}

int attn_bwd(const moments_attn_desc* desc, const void* x, const void* k, const void* q, const void* da,
             const float* h0, const void* saved, size_t saved_bytes, bool use_saved, const void* d_y,
             const float* d_last, void* d_x, void* d_k, void* d_q, void* d_da, float* d_h0, void* workspace,
             size_t workspace_bytes, void* stream) {
  AttnPlan P;
  MOM_TRY(make_attn_plan(desc, &P));
  if (P.empty) return attn_bwd_empty(P, d_k, d_q, (hipStream_t)stream);
  if (!P.bwd) return MOMENTS_ENOTSUP;
  if (P.g.s > 0 && (!x || !k || !q || !da || !d_y)) return MOMENTS_EINVAL;
  if (use_saved && P.saved > 0 && saved == nullptr) return MOMENTS_EINVAL;
  if (use_saved && saved_bytes < P.saved) return MOMENTS_EWORKSPACE;
  const void* ptrs[] = {x, k, q, da, h0, saved, d_y, d_last, d_x, d_k, d_q, d_da, d_h0, workspace};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  if (workspace == nullptr || workspace_bytes < P.ws_bwd) return MOMENTS_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  MOM_TRY(with_attn(P, [&](auto tt, auto rt, auto pw, auto vec) -> int {
    constexpr bool VEC = decltype(vec)::value != 0;
    using T = typename decltype(tt)::type;
    constexpr int RT = decltype(rt)::value, PW = decltype(pw)::value, PT = 4 * PW;
    const T *xt = (const T*)x, *kt = (const T*)k, *qt = (const T*)q, *dat = (const T*)da, *dyt = (const T*)d_y;
    const T* copies = (const T*)saved;
    if (!use_saved) {   // the states entering the chunks, by a walk over k and x
      T* own = (T*)(ws + P.save);
      MOM_TRY((run_segments<T, RT, PW, VEC>(P, xt, kt, dat, h0, ws, st)));
      MOM_TRY((launch_walk<T, RT, PW, 1, VEC>(P.g, P.g.nseg, xt, kt, nullptr, dat, h0, nullptr, nullptr, own,
                                         P.g.nseg > 1 ? (float*)ws : nullptr,
                                         P.g.nseg > 1 ? (double*)(ws + P.seg_dec) : nullptr, st)));
      copies = own;
    }
    const AttnGeo& g = P.gb;
    float* seg = g.nseg > 1 ? (float*)(ws + P.seg_loc_b) : nullptr;
    double* sdec = g.nseg > 1 ? (double*)(ws + P.seg_dec_b) : nullptr;
    if (g.nseg > 1) {
      AttnGeo g2 = g;
      g2.seg0 = 1;
      MOM_TRY((launch_walk<T, RT, PW, 2, VEC>(g2, g.nseg - 1, dyt, qt, nullptr, dat, nullptr, nullptr, nullptr, nullptr,
                                         seg, sdec, st)));
      MOM_TRY(launch_scan(P, g, true, d_last, seg, sdec, st));
    }
    float* pq = (float*)(ws + P.part_q);
    float* pk = (float*)(ws + P.part_k);
    float* pa = (float*)(ws + P.part_da);
    auto go = [&](auto part) -> int {
      constexpr bool PART = decltype(part)::value != 0;
      const size_t lds = LdsB<T, RT, PT>::total;
      static_assert(LdsB<T, RT, PT>::total <= kLdsLimit, "LDS");
      static std::atomic<uint64_t> done{0};
      MOM_TRY(set_lds_once(done, k_attn_bwd<T, RT, PT, PART, VEC>, lds));
      ProfScope ps(KID_ATTN_BWD, st);
      hipLaunchKernelGGL((k_attn_bwd<T, RT, PT, PART, VEC>), dim3((unsigned)((size_t)P.items * g.nseg)), dim3(ABT), lds, st,
                         g, xt, kt, qt, dat, copies, dyt, d_last, seg, (T*)d_x, (T*)d_k, (T*)d_q, (T*)d_da,
                         d_h0, pk, pq, pa);
      return check_launch();
    };
    if (!P.part) return go(IC<0>{});
    MOM_TRY(go(IC<1>{}));
    const size_t keys = (size_t)g.b * g.s * g.c * g.g * g.r, toks = (size_t)g.b * g.s * g.h;
    const SumJobs jobs = {{{pq, d_q, d_q != nullptr ? keys : 0, g.hpg * g.npt, g.r},
                           {pk, d_k, d_k != nullptr ? keys : 0, g.hpg * g.npt, g.r},
                           {pa, d_da, d_da != nullptr ? toks : 0, g.npt, 1}}};
    const unsigned blocks = (unsigned)std::min<size_t>((std::max(keys, toks) + 255) / 256, 16384);
    if (blocks == 0) return 0;
    ProfScope ps(KID_ATTN_SUM, st);
    hipLaunchKernelGGL((k_attn_sum<T>), dim3(blocks, 3), dim3(256), 0, st, jobs);
    return check_launch();
  }));
  if (check_finite_on()) {
    const AttnGeo& g = P.g;
    const size_t tok = (size_t)g.b * g.s;
    const OutSpan outs[] = {{d_x, tok * g.c * g.h * g.p, !P.bf}, {d_k, tok * g.c * g.g * g.r, !P.bf},
                            {d_q, tok * g.c * g.g * g.r, !P.bf}, {d_da, tok * g.h, !P.bf},
                            {d_h0, (size_t)g.b * g.h * g.p * g.r, true}};
    return check_finite(outs, 5, ws + P.flag_bwd, st);
  }
  return 0;
}

}  // namespace

extern "C" {

int moments_attn_validate(const moments_attn_desc* desc) {
  AttnPlan P;
  return make_attn_plan(desc, &P);
}

int64_t moments_attn_workspace_size(const moments_attn_desc* desc, int is_bwd) {
  AttnPlan P;
  const int rc = make_attn_plan(desc, &P);
  if (rc != 0) return rc;
  if (is_bwd && !P.bwd) return MOMENTS_ENOTSUP;
  return P.empty ? 0 : (int64_t)(is_bwd ? P.ws_bwd : P.ws_fwd);
}

int64_t moments_attn_saved_size(const moments_attn_desc* desc) {
  AttnPlan P;
  const int rc = make_attn_plan(desc, &P);
  if (rc != 0) return rc;
  return P.empty ? 0 : (int64_t)P.saved;
}

int moments_attn_fwd(const moments_attn_desc* desc, const void* xhat, const void* bhat, const void* qhat,
                     const void* da, const float* h0, void* y, float* h_last, void* workspace,
                     size_t workspace_bytes, void* stream) {
  return attn_fwd(desc, xhat, bhat, qhat, da, h0, y, h_last, nullptr, 0, false, workspace, workspace_bytes, stream);
}

int moments_attn_fwd_save(const moments_attn_desc* desc, const void* xhat, const void* bhat, const void* qhat,
                          const void* da, const float* h0, void* y, float* h_last, void* saved, size_t saved_bytes,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return attn_fwd(desc, xhat, bhat, qhat, da, h0, y, h_last, saved, saved_bytes, true, workspace, workspace_bytes,
                  stream);
}

int moments_attn_bwd(const moments_attn_desc* desc, const void* xhat, const void* bhat, const void* qhat,
                     const void* da, const float* h0, const void* d_y, const float* d_h_last, void* d_xhat,
                     void* d_bhat, void* d_qhat, void* d_da, float* d_h0, void* workspace, size_t workspace_bytes,
                     void* stream) {
  return attn_bwd(desc, xhat, bhat, qhat, da, h0, nullptr, 0, false, d_y, d_h_last, d_xhat, d_bhat, d_qhat, d_da,
                  d_h0, workspace, workspace_bytes, stream);
}

int moments_attn_bwd_saved(const moments_attn_desc* desc, const void* xhat, const void* bhat, const void* qhat,
                           const void* da, const float* h0, const void* saved, size_t saved_bytes, const void* d_y,
                           const float* d_h_last, void* d_xhat, void* d_bhat, void* d_qhat, void* d_da, float* d_h0,
                           void* workspace, size_t workspace_bytes, void* stream) {
  return attn_bwd(desc, xhat, bhat, qhat, da, h0, saved, saved_bytes, true, d_y, d_h_last, d_xhat, d_bhat, d_qhat,
                  d_da, d_h0, workspace, workspace_bytes, stream);
}

int moments_attn_step(const moments_attn_desc* desc, const void* xhat, const void* bhat, const void* qhat,
                      const void* da, const int32_t* slots, int64_t nslots, float* state, void* y, void* stream) {
  AttnPlan P;
  MOM_TRY(make_attn_plan(desc, &P));
  if (desc->s != 1 || nslots < 0 || nslots > (int64_t)1 << 30) return MOMENTS_EINVAL;
  if (slots == nullptr && nslots < desc->b) return MOMENTS_EINVAL;
  if (P.empty) return 0;
  if (!xhat || !bhat || !qhat || !da || !y || (!state && nslots > 0)) return MOMENTS_EINVAL;
  const void* ptrs[] = {xhat, bhat, qhat, da, state, y};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  const AttnGeo& g = P.g;
  auto go = [&](auto tt, auto lpr, auto nb) -> int {
    using T = typename decltype(tt)::type;
    constexpr int LPR = decltype(lpr)::value, NB = decltype(nb)::value, rows = 4 * (64 / LPR) * NB;
    ProfScope ps(KID_ATTN_STEP, st);
    hipLaunchKernelGGL((k_attn_step<T, LPR, NB>), dim3((unsigned)(g.b * g.h), (unsigned)((g.p + rows - 1) / rows)),
                       dim3(256), 0, st, g, (int)nslots, (const T*)xhat, (const T*)bhat, (const T*)qhat,
                       (const T*)da, (const int*)slots, state, (T*)y);
    return check_launch();
  };
  auto by_r = [&](auto tt) -> int {
    if (g.r <= 32) return go(tt, IC<8>{}, IC<2>{});
    if (g.r <= 64) return go(tt, IC<16>{}, IC<4>{});
    return go(tt, IC<32>{}, IC<8>{});
  };
  MOM_TRY(P.bf ? by_r(TT<bf16>{}) : by_r(TT<float>{}));
  if (check_finite_on()) {
    // y tells of the states too: a value that is not finite spoils its row's sum
    const OutSpan outs[] = {{y, (size_t)g.b * g.c * g.h * g.p, !P.bf}};
    return check_finite(outs, 1, nullptr, st);
  }
  return 0;
}

}  // extern "C"
