// C ABI of the norms of queries and keys with the position rotation: validation,
// planning, dispatch. The operation and its conventions are stated in include/moments.h.
#include "moments.h"

#include <hip/hip_runtime.h>

#include <algorithm>

#include "host.h"
#include "kernels_attn_bwd.h"
#include "kernels_qk.h"

using namespace mom;

namespace {

struct QkPlan {
  QkGeo g;
  bool bf, empty, vec;
  int HB;               // heads a row slot keeps in registers (0: any number)
  int LPR, C, NT;       // lanes a row; padded channels; threads of the backward
  int nfwd;             // workgroups per group of the forward
  size_t lds;           // of the backward
  size_t part_w, part_b, part_rot, ws, flag;
};

// bases: q and k start at 16 bytes (else their rows cannot be read in whole pieces).
int make_qk_plan(const moments_qk_desc* d, QkPlan* P, bool bases) {
  if (d == nullptr) return MOMENTS_EINVAL;
  if (d->b < 0 || d->s < 0 || d->h < 0 || d->c < 1 || d->g < 1 || d->r < 1 || d->h % d->g != 0) return MOMENTS_EINVAL;
  if (d->dtype != MOMENTS_F32 && d->dtype != MOMENTS_BF16) return MOMENTS_EINVAL;
  if (!(d->eps >= 0.0f)) return MOMENTS_EINVAL;
  int A = 0, J = 0;
  switch (d->rot_kind) {
    case MOMENTS_ROT_NONE:
      break;
    case MOMENTS_ROT_COMPLEX_PAIRWISE:
    case MOMENTS_ROT_COMPLEX_HALF:
      if (d->rope_dim < 2 || d->rope_dim % 2 != 0 || d->rope_dim > d->r) return MOMENTS_EINVAL;
      if (d->rot_kind == MOMENTS_ROT_COMPLEX_HALF && d->r % 2 != 0) return MOMENTS_EINVAL;
      A = (int)(d->rope_dim / 2);
      break;
    case MOMENTS_ROT_QUATERNION:
      if (d->quat_blocks < 1 || d->quat_blocks > d->r / 4) return MOMENTS_EINVAL;
      J = (int)d->quat_blocks;
      break;
    default:
      return MOMENTS_EINVAL;
  }
  if (d->rot_kind != MOMENTS_ROT_NONE && d->rot_h != 1 && d->rot_h != d->h) return MOMENTS_EINVAL;
  if (d->r > 128 || d->c > 4 || d->g > 65535 || d->h / d->g > 128 || d->s > (int64_t)1 << 28 ||
      d->b > (int64_t)1 << 24 || d->b * d->s > (int64_t)1 << 30)
    return MOMENTS_ENOTSUP;
  const int64_t row = d->c * d->g * d->r;
  const int64_t qs = d->q_stride == 0 ? row : d->q_stride, ks = d->k_stride == 0 ? row : d->k_stride;
  if (qs < row || ks < row) return MOMENTS_EINVAL;
  P->empty = d->b == 0 || d->h == 0;
  P->bf = d->dtype == MOMENTS_BF16;
  const int tsz = P->bf ? 2 : 4;
  QkGeo& g = P->g;
  g = QkGeo{};
  g.b = (int)d->b; g.s = (int)d->s; g.c = (int)d->c; g.h = (int)d->h; g.g = (int)d->g; g.r = (int)d->r;
  g.qs = (size_t)qs; g.ks = (size_t)ks;
  g.rot_h = (int)d->rot_h; g.A = A; g.J = J; g.RW = J > 0 ? 4 * J : A;
  g.eps = d->eps;
  g.rinv = 1.0f / (float)d->r;
  // The rules below on 8 x 8192 tokens of two channels, 64 heads in 8 groups, r = 128, bf16
  // ("large"), and 2 x 2048 of two, 16 heads, r = 64, float ("small"), forward and backward.
  // Whole pieces, or, where alignment does not allow them, element by element: large 1.24 and
  // 1.69 ms against 4.4 and 10.1, small 24 and 48 us against 148 and 543.
  P->vec = bases && g.r % 8 == 0 && qs * tsz % 16 == 0 && ks * tsz % 16 == 0 && A % 4 == 0;
  // 16 lanes for rows that 8 would do: small 29 and 58 us.
  P->LPR = g.r <= 64 && P->vec ? 8 : 16;
  // Channels are held in registers; four places for two: large 2.1 and 5.5 ms, small 28 and 71 us.
  P->C = g.c <= 1 ? 1 : g.c <= 2 ? 2 : 4;
  if (P->empty) return MOMENTS_OK;
  g.hpg = g.h / g.g;
  const int rpw = 64 / P->LPR;
  g.HPP = P->vec ? 1 : rpw;
  while (g.HPP < g.hpg && g.HPP < rpw) g.HPP *= 2;
  g.HL = (g.hpg + g.HPP - 1) / g.HPP;
  // sums for each head in registers while a head slot serves one or two heads, else in LDS:
  // 64 bytes a thread and head, so fewer threads where there are many. LDS always: large 1.6
  // and 2.8 ms, small 27 and 213 us.
  P->HB = P->vec && g.HL <= (P->C == 4 ? 1 : 2) ? g.HL : 0;
  P->NT = QKT;
  while (P->HB == 0 && P->NT > 64 && (size_t)(g.HL + 1) * 64 * P->NT > kLdsLimit) P->NT /= 2;
  P->lds = (size_t)(P->HB == 0 ? g.HL + 1 : 1) * 64 * P->NT;
  const int64_t per = (int64_t)(P->NT / 64) * (rpw / g.HPP);   // tokens a workgroup has at once
  const int64_t most = std::max<int64_t>(1, ((int64_t)g.b * g.s + per - 1) / per);
  g.nblk = (int)std::min<int64_t>(most, std::max<int64_t>(1, 2048 / g.g));
  const int64_t perf = QKT / 64 * (rpw / g.HPP);
  P->nfwd = (int)std::min<int64_t>(((int64_t)g.b * g.s + perf - 1) / perf, std::max<int64_t>(1, 4096 / g.g));
  size_t o = 0;
  P->part_w = o; o = align256(o + (size_t)2 * g.nblk * g.g * g.r * 4);
  P->part_b = o; o = align256(o + (size_t)2 * g.nblk * g.h * g.r * 4);
  P->part_rot = o;
  if (g.RW > 0 && g.rot_h == 1 && g.h > 1) o = align256(o + (size_t)g.b * g.s * g.g * g.RW * 4);
  P->flag = o;
  P->ws = o + 256;
  return MOMENTS_OK;
}

// Calls f(TT<T>, IC<LPR>, IC<ROT>, IC<C>, IC<HB>, IC<HPP>, IC<VEC>) for the compiled variant of the
// plan. Rows that are not whole pieces have one variant for all widths, channels and heads.
template <class F>
int with_qk(const QkPlan& P, int rot_kind, F&& f) {
  auto by_hb = [&](auto tt, auto lpr, auto rot, auto cc) -> int {
    constexpr int RPW = 64 / decltype(lpr)::value;
    switch (P.HB) {
      case 0: return f(tt, lpr, rot, cc, IC<0>{}, IC<RPW>{}, IC<1>{});
      case 2:
        if constexpr (decltype(cc)::value < 4) return f(tt, lpr, rot, cc, IC<2>{}, IC<RPW>{}, IC<1>{});
        break;
      case 1:
        switch (P.g.HPP) {
          case 1: return f(tt, lpr, rot, cc, IC<1>{}, IC<1>{}, IC<1>{});
          case 2: return f(tt, lpr, rot, cc, IC<1>{}, IC<2>{}, IC<1>{});
          case 4: return f(tt, lpr, rot, cc, IC<1>{}, IC<4>{}, IC<1>{});
          case 8:
            if constexpr (RPW == 8) return f(tt, lpr, rot, cc, IC<1>{}, IC<8>{}, IC<1>{});
        }
    }
    return MOMENTS_ENOTSUP;   // no plan has another combination
  };
  auto by_c = [&](auto tt, auto lpr, auto rot) -> int {
    switch (P.C) {
      case 1: return by_hb(tt, lpr, rot, IC<1>{});
      case 2: return by_hb(tt, lpr, rot, IC<2>{});
    }
    return by_hb(tt, lpr, rot, IC<4>{});
  };
  auto by_lpr = [&](auto tt, auto rot) -> int {
    if (!P.vec) return f(tt, IC<16>{}, rot, IC<4>{}, IC<0>{}, IC<4>{}, IC<0>{});
    return P.LPR == 8 ? by_c(tt, IC<8>{}, rot) : by_c(tt, IC<16>{}, rot);
  };
  auto by_rot = [&](auto tt) -> int {
    switch (rot_kind) {
      case MOMENTS_ROT_NONE: return by_lpr(tt, IC<0>{});
      case MOMENTS_ROT_COMPLEX_PAIRWISE: return by_lpr(tt, IC<1>{});
      case MOMENTS_ROT_COMPLEX_HALF: return by_lpr(tt, IC<2>{});
    }
    return by_lpr(tt, IC<3>{});
  };
  return P.bf ? by_rot(TT<bf16>{}) : by_rot(TT<float>{});
}

bool at_element(const void* p, bool bf) { return ((uintptr_t)p & (bf ? 1 : 3)) == 0; }

// The parameters' gradients from the partials of nblk workgroups a group (zeros for none).
int launch_qk_sum(const QkGeo& g, const float* pw, const float* pb, int nblk, float* d_wq, float* d_wk, float* d_bq,
                  float* d_bk, hipStream_t st) {
  if (!d_wq && !d_wk && !d_bq && !d_bk) return 0;
  ProfScope ps(KID_QK_SUM, st);
  const int cols = (g.r + 15) / 16 + (d_bq || d_bk ? (int)(((int64_t)g.h * g.r + 15) / 16) : 0);
  // a launch holds fewer than 2^32 threads
  hipLaunchKernelGGL(k_qk_sum, dim3((unsigned)std::min(cols, 1 << 20), 2), dim3(1024), 0, st, pw, nblk * g.g, g.r,
                     d_wq, d_wk, pb, nblk, g.h * g.r, d_bq, d_bk, cols);
  return check_launch();
}

// Gradients where there are no sequences or no heads: those that hold values are zero (sums
// of no slices).
int qk_bwd_empty(const QkPlan& P, void* d_q, void* d_k, float* d_wq, float* d_wk, float* d_bq, float* d_bk,
                 void* d_rot, hipStream_t st) {
  const QkGeo& g = P.g;
  const size_t tok = (size_t)g.b * g.s, raw = tok * g.c * g.g * g.r, rot = tok * g.rot_h * g.RW;
  const SumJobs jobs = {{{nullptr, d_q, d_q ? raw : 0, 0, g.r},
                         {nullptr, d_k, d_k ? raw : 0, 0, g.r},
                         {nullptr, d_rot, d_rot ? rot : 0, 0, std::max(g.RW, 1)}}};
  const size_t most = std::max({jobs.job[0].total, jobs.job[1].total, jobs.job[2].total});
  if (most > 0) {
    ProfScope ps(KID_QK_SUM, st);
    const dim3 grid((unsigned)std::min<size_t>((most + 255) / 256, 16384), 3);
    if (P.bf)
      hipLaunchKernelGGL((k_attn_sum<bf16>), grid, dim3(256), 0, st, jobs);
    else
      hipLaunchKernelGGL((k_attn_sum<float>), grid, dim3(256), 0, st, jobs);
    MOM_TRY(check_launch());
  }
  return launch_qk_sum(g, nullptr, nullptr, 0, d_wq, d_wk, d_bq, d_bk, st);
}

}  // namespace

extern "C" {

int64_t moments_qk_workspace_size(const moments_qk_desc* desc) {
  QkPlan P, U;   // where q and k start is not known here
  const int rc = make_qk_plan(desc, &P, true);
  if (rc != 0) return rc;
  MOM_TRY(make_qk_plan(desc, &U, false));
  return P.empty ? 0 : (int64_t)std::max(P.ws, U.ws);
}

int moments_qk_fwd(const moments_qk_desc* desc, const void* q, const void* k, const float* wq, const float* wk,
                   const float* bq, const float* bk, const void* rot, void* qhat, void* khat, void* stream) {
  QkPlan P;
  MOM_TRY(make_qk_plan(desc, &P, aligned16(q) && aligned16(k)));
  const QkGeo& g = P.g;
  if (P.empty || g.s == 0) return 0;
  if (!q || !k || !wq || !wk || !qhat || !khat) return MOMENTS_EINVAL;
  if ((desc->rot_kind == MOMENTS_ROT_NONE) != (rot == nullptr)) return MOMENTS_EINVAL;
  if (!at_element(q, P.bf) || !at_element(k, P.bf)) return MOMENTS_EINVAL;
  const void* ptrs[] = {wq, wk, bq, bk, rot, qhat, khat};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  MOM_TRY(with_qk(P, desc->rot_kind, [&](auto tt, auto lpr, auto rk, auto cc, auto hb, auto hpp, auto vec) -> int {
    using T = typename decltype(tt)::type;
    constexpr int LPR = decltype(lpr)::value, ROT = decltype(rk)::value, C = decltype(cc)::value;
    ProfScope ps(KID_QK_FWD, st);
    hipLaunchKernelGGL((k_qk_fwd<T, LPR, ROT, C, decltype(hb)::value, decltype(vec)::value != 0>),
                       dim3((unsigned)P.nfwd, (unsigned)g.g), dim3(QKT), 0, st, g, (const T*)q, (const T*)k, wq, wk,
                       bq, bk, (const T*)rot, (T*)qhat, (T*)khat);
    return check_launch();
  }));
  if (check_finite_on()) {
    const size_t n = (size_t)g.b * g.s * g.c * g.h * g.r;
    const OutSpan outs[] = {{qhat, n, !P.bf}, {khat, n, !P.bf}};
    return check_finite(outs, 2, nullptr, st);
  }
  return 0;
}

int moments_qk_bwd(const moments_qk_desc* desc, const void* q, const void* k, const float* wq, const float* wk,
                   const float* bq, const float* bk, const void* rot, const void* d_qhat, const void* d_khat,
                   void* d_q, void* d_k, float* d_wq, float* d_wk, float* d_bq, float* d_bk, void* d_rot,
                   void* workspace, size_t workspace_bytes, void* stream) {
  QkPlan P;
  MOM_TRY(make_qk_plan(desc, &P, aligned16(q) && aligned16(k)));
  const QkGeo& g = P.g;
  if (P.empty) return qk_bwd_empty(P, d_q, d_k, d_wq, d_wk, d_bq, d_bk, d_rot, (hipStream_t)stream);
  if (g.s > 0 && (!q || !k || !wq || !wk || !d_qhat || !d_khat)) return MOMENTS_EINVAL;
  if (g.s > 0 && (desc->rot_kind == MOMENTS_ROT_NONE) != (rot == nullptr)) return MOMENTS_EINVAL;
  if (desc->rot_kind == MOMENTS_ROT_NONE && d_rot != nullptr) return MOMENTS_EINVAL;
  if ((bq == nullptr && d_bq != nullptr) || (bk == nullptr && d_bk != nullptr)) return MOMENTS_EINVAL;
  if (!at_element(q, P.bf) || !at_element(k, P.bf)) return MOMENTS_EINVAL;
  const void* ptrs[] = {wq, wk, bq, bk, rot, d_qhat, d_khat, d_q, d_k, d_wq, d_wk, d_bq, d_bk, d_rot, workspace};
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  if (workspace == nullptr || workspace_bytes < P.ws) return MOMENTS_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const bool rot1 = g.RW > 0 && g.rot_h == 1 && g.h > 1;
  float* pw = d_wq || d_wk ? (float*)(ws + P.part_w) : nullptr;
  float* pb = d_bq || d_bk ? (float*)(ws + P.part_b) : nullptr;
  float* pr = rot1 && d_rot ? (float*)(ws + P.part_rot) : nullptr;
  // Without tokens there is nothing to read (q, k, the weights and rot may be NULL): the sums
  // over tokens, of no partials, are all that is left.
  const int nblk = g.s > 0 ? g.nblk : 0;
  auto rows = [&](auto tt, auto lpr, auto rk, auto cc, auto hb, auto hpp, auto vec) -> int {
    using T = typename decltype(tt)::type;
    constexpr int LPR = decltype(lpr)::value, ROT = decltype(rk)::value, C = decltype(cc)::value;
    {
      auto kernel = k_qk_bwd<T, LPR, ROT, C, decltype(hb)::value, decltype(hpp)::value, decltype(vec)::value != 0>;
      if (P.lds > 64 * 1024) MOM_TRY(set_lds(kernel, P.lds));
      ProfScope ps(KID_QK_BWD, st);
      hipLaunchKernelGGL(kernel, dim3((unsigned)g.nblk, (unsigned)g.g), dim3(P.NT), P.lds, st, g, (const T*)q,
                         (const T*)k, wq, wk, bq, bk, (const T*)rot, (const T*)d_qhat, (const T*)d_khat, (T*)d_q,
                         (T*)d_k, (T*)(rot1 ? nullptr : d_rot), pr, pw, pb);
      MOM_TRY(check_launch());
    }
    if (pr != nullptr) {
      const size_t total = (size_t)g.b * g.s * g.RW;
      ProfScope ps(KID_QK_SUM, st);
      const SumJobs jobs = {{{pr, d_rot, total, g.g, g.RW}, {}, {}}};
      hipLaunchKernelGGL((k_attn_sum<T>), dim3((unsigned)std::min<size_t>((total + 255) / 256, 16384)), dim3(256), 0,
                         st, jobs);
      MOM_TRY(check_launch());
    }
    return 0;
  };
  if (nblk > 0) MOM_TRY(with_qk(P, desc->rot_kind, rows));
  MOM_TRY(launch_qk_sum(g, pw, pb, nblk, d_wq, d_wk, d_bq, d_bk, st));
  if (check_finite_on()) {
    const size_t raw = (size_t)g.b * g.s * g.c * g.g * g.r;
    const OutSpan outs[] = {{d_q, raw, !P.bf}, {d_k, raw, !P.bf}, {d_rot, (size_t)g.b * g.s * g.rot_h * g.RW, !P.bf},
                            {d_wq, (size_t)g.r, true}, {d_wk, (size_t)g.r, true},
                            {d_bq, (size_t)g.h * g.r, true}, {d_bk, (size_t)g.h * g.r, true}};
    return check_finite(outs, 7, ws + P.flag, st);
  }
  return 0;
}

}  // extern "C"
