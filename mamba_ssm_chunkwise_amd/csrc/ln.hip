// C ABI of layer norm with the residual stream: validation, planning, dispatch. The operation and
// its conventions are stated in include/moments.h.
#include "moments.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "host.h"
#include "kernels_ln.h"

using namespace mom;

namespace {

struct LnPlan {
  LnGeo g;
  bool bf, res, empty;
  int NT, E;          // threads of a row, elements of a thread
  int nblk, nfwd;     // workgroups of the gradients and of the forward
  size_t part, flag, ws;
};

int make_ln_plan(const moments_ln_desc* d, LnPlan* P) {
  if (d == nullptr) return MOMENTS_EINVAL;
  if (d->n < 0 || d->w < 1 || (d->residual != 0 && d->residual != 1) || d->reserved != 0) return MOMENTS_EINVAL;
  if (d->dtype != MOMENTS_F32 && d->dtype != MOMENTS_BF16) return MOMENTS_EINVAL;
  if (!(d->eps >= 1e-30f) || !std::isfinite(d->eps)) return MOMENTS_EINVAL;
  const int64_t xs = d->x_stride == 0 ? d->w : d->x_stride;
  if (xs < d->w) return MOMENTS_EINVAL;
  if (d->w > 16384 || d->n > (int64_t)1 << 40 || xs > (int64_t)1 << 40 || d->n * d->w > (int64_t)1 << 50)
    return MOMENTS_ENOTSUP;
  P->empty = d->n == 0;
  P->bf = d->dtype == MOMENTS_BF16;
  P->res = d->residual != 0;
  LnGeo& g = P->g;
  g = LnGeo{};
  g.n = d->n; g.w = (int)d->w; g.xs = (size_t)xs;
  g.eps = d->eps;
  g.winv = 1.0f / (float)d->w;
  P->E = g.w <= 512 ? 8 : 16;
  P->NT = 8;
  while (P->NT * P->E < g.w) P->NT *= 2;
  const int rows = P->NT <= 64 ? 256 / P->NT : 1, nb = std::max(P->NT, P->NT <= 64 ? 256 : 128);
  const int64_t all = (d->n + rows - 1) / rows;
  P->nfwd = (int)std::min<int64_t>(all, kCUs * 4096 / nb);
  P->nblk = (int)std::min<int64_t>(all, kCUs * std::max(768 / nb, 1));
  P->part = 0;
  P->flag = align256((size_t)2 * P->nblk * g.w * 4);
  P->ws = P->flag + 256;
  return MOMENTS_OK;
}

// Calls f(TT<T>, IC<NT>, IC<E>) for the compiled variant of the plan.
template <class F>
int with_ln(const LnPlan& P, F&& f) {
  auto by_w = [&](auto tt) -> int {
    switch (P.NT) {
      case 8: return f(tt, IC<8>{}, IC<8>{});
      case 16: return f(tt, IC<16>{}, IC<8>{});
      case 32: return f(tt, IC<32>{}, IC<8>{});
      case 64: return P.E == 8 ? f(tt, IC<64>{}, IC<8>{}) : f(tt, IC<64>{}, IC<16>{});
      case 128: return f(tt, IC<128>{}, IC<16>{});
      case 256: return f(tt, IC<256>{}, IC<16>{});
      case 512: return f(tt, IC<512>{}, IC<16>{});
    }
    return f(tt, IC<1024>{}, IC<16>{});
  };
  return P.bf ? by_w(TT<bf16>{}) : by_w(TT<float>{});
}

bool at_element(const void* p, bool bf) { return ((uintptr_t)p & (bf ? 1 : 3)) == 0; }

int all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  return 0;
}

int launch_ln_sum(const float* part, int np, int w, float* d_weight, float* d_bias, hipStream_t st) {
  if (!d_weight && !d_bias) return 0;
  ProfScope ps(KID_LN_SUM, st);
  hipLaunchKernelGGL(k_ln_sum, dim3((unsigned)((w + 63) / 64), 2), dim3(1024), 0, st, part, np, w, d_weight, d_bias);
  return check_launch();
}

}  // namespace

extern "C" {

int64_t moments_ln_workspace_size(const moments_ln_desc* desc) {
  LnPlan P;
  MOM_TRY(make_ln_plan(desc, &P));
  return P.empty ? 0 : (int64_t)P.ws;
}

int moments_ln_fwd(const moments_ln_desc* desc, const void* x, const float* res, const float* weight,
                   const float* bias, void* y, float* sum, void* stream) {
  LnPlan P;
  MOM_TRY(make_ln_plan(desc, &P));
  if (P.empty) return 0;
  if (!x || !weight || !y) return MOMENTS_EINVAL;
  if (P.res ? !res || !sum : res != nullptr || sum != nullptr) return MOMENTS_EINVAL;
  if (!at_element(x, P.bf)) return MOMENTS_EINVAL;
  MOM_TRY(all_aligned({res, weight, bias, y, sum}));
  hipStream_t st = (hipStream_t)stream;
  MOM_TRY(with_ln(P, [&](auto tt, auto nt, auto ee) -> int {
    using T = typename decltype(tt)::type;
    constexpr int NT = decltype(nt)::value, E = decltype(ee)::value;
    ProfScope ps(KID_LN_FWD, st);
    const dim3 grid((unsigned)P.nfwd), block(NT <= 64 ? 256 : NT);
    if (P.res)
      hipLaunchKernelGGL((k_ln_fwd<T, NT, E, true>), grid, block, 0, st, P.g, (const T*)x, res, weight, bias,
                         (T*)y, sum);
    else
      hipLaunchKernelGGL((k_ln_fwd<T, NT, E, false>), grid, block, 0, st, P.g, (const T*)x, res, weight, bias,
                         (T*)y, sum);
    return check_launch();
  }));
  if (check_finite_on()) {
    const size_t n = (size_t)P.g.n * P.g.w;
    const OutSpan outs[] = {{y, n, !P.bf}, {sum, n, true}};
    return check_finite(outs, 2, nullptr, st);
  }
  return 0;
}

int moments_ln_bwd(const moments_ln_desc* desc, const void* x, const float* weight, const void* d_y,
                   const float* d_sum, void* d_x, float* d_res, float* d_weight, float* d_bias, void* workspace,
                   size_t workspace_bytes, void* stream) {
  LnPlan P;
  MOM_TRY(make_ln_plan(desc, &P));
  if (P.res) P.g.xs = (size_t)P.g.w;   // x is the sum: float32 rows, one after the other
  hipStream_t st = (hipStream_t)stream;
  if (!P.res && (d_sum != nullptr || d_res != nullptr)) return MOMENTS_EINVAL;
  MOM_TRY(all_aligned({weight, d_y, d_sum, d_x, d_res, d_weight, d_bias, workspace}));
  if (P.empty) return launch_ln_sum(nullptr, 0, P.g.w, d_weight, d_bias, st);
  if (!x || !weight || !d_y) return MOMENTS_EINVAL;
  if (!at_element(x, P.bf && !P.res)) return MOMENTS_EINVAL;
  if (workspace == nullptr || workspace_bytes < P.ws) return MOMENTS_EWORKSPACE;
  unsigned char* ws = (unsigned char*)workspace;
  float* part = d_weight || d_bias ? (float*)(ws + P.part) : nullptr;
  MOM_TRY(with_ln(P, [&](auto tt, auto nt, auto ee) -> int {
    using T = typename decltype(tt)::type;
    // as many threads as a row of the plan has, or half of 1024 with twice the elements
    constexpr bool WIDE = decltype(nt)::value == 1024;
    constexpr int NT = WIDE ? 512 : decltype(nt)::value, E = WIDE ? 32 : decltype(ee)::value;
    const auto go = [&](auto ts) -> int {
      using TS = typename decltype(ts)::type;
      constexpr size_t lds = ln_wide_lds<NT, E>;
      if constexpr (lds > 0) {
        static std::atomic<uint64_t> done{0};
        MOM_TRY(set_lds_once(done, k_ln_bwd<T, TS, NT, E>, lds));
      }
      ProfScope ps(KID_LN_BWD, st);
      hipLaunchKernelGGL((k_ln_bwd<T, TS, NT, E>), dim3((unsigned)P.nblk), dim3(NT <= 64 ? 256 : NT), lds, st, P.g,
                         (const TS*)x, weight, (const T*)d_y, d_sum, (T*)d_x, d_res, part);
      return check_launch();
    };
    return P.res ? go(TT<float>{}) : go(TT<T>{});
  }));
  MOM_TRY(launch_ln_sum(part, P.nblk, P.g.w, d_weight, d_bias, st));
  if (check_finite_on()) {
    const size_t n = (size_t)P.g.n * P.g.w, w = (size_t)P.g.w;
    const OutSpan outs[] = {{d_x, n, !P.bf}, {d_res, n, true}, {d_weight, w, true}, {d_bias, w, true}};
    return check_finite(outs, 4, ws + P.flag, st);
  }
  return 0;
}

}  // extern "C"
