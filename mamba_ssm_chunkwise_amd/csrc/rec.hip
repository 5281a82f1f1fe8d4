// C ABI of the gated linear recurrence: validation, planning, dispatch. The operation and its
// conventions are stated in include/moments.h.
#include "moments.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <initializer_list>

#include "host.h"
#include "kernels_rec.h"

using namespace mom;

namespace {

struct RecPlan {
  RecGeo g;
  bool bf, z, empty;
  int VC;                                // channels of a lane
  size_t part, first, save, flag_bwd;    // workspace offsets; part and first at the start for both directions
  size_t ws_fwd, ws_bwd, saved;
};

// A launch holds fewer than 2^32 threads, up to 1024 of them to a workgroup.
constexpr int64_t kMostItems = ((int64_t)1 << 22) - 1;

// bases: x, g and z start where a lane's two channels can be read as one piece.
int make_rec_plan(const moments_rec_desc* d, RecPlan* P, bool bases) {
  if (d == nullptr) return MOMENTS_EINVAL;
  if (d->b < 0 || d->s < 0 || d->w < 1 || d->valid_len < 0 || d->reserved != 0) return MOMENTS_EINVAL;
  if (d->dtype != MOMENTS_F32 && d->dtype != MOMENTS_BF16) return MOMENTS_EINVAL;
  if (d->gate != MOMENTS_GATE_LOG && d->gate != MOMENTS_GATE_MIX && d->gate != MOMENTS_GATE_UNIT) return MOMENTS_EINVAL;
  if (d->has_z != 0 && d->has_z != 1) return MOMENTS_EINVAL;
  if (d->w > (int64_t)1 << 24 || d->s > (int64_t)1 << 28 || d->b > (int64_t)1 << 24) return MOMENTS_ENOTSUP;
  const int64_t xs = d->x_stride == 0 ? d->w : d->x_stride, gs = d->g_stride == 0 ? d->w : d->g_stride;
  const int64_t zs = d->z_stride == 0 ? d->w : d->z_stride;
  if (xs < d->w || gs < d->w || (d->has_z && zs < d->w)) return MOMENTS_EINVAL;
  // A lane's tokens are addressed with 32-bit offsets; where a sequence has one token, the next
  // sequence's may be as far as the card's memory goes.
  const int64_t far = (int64_t)1 << (d->s > 1 ? 25 : 37);
  if (xs > far || gs > far || (d->has_z && zs > far)) return MOMENTS_ENOTSUP;
  P->empty = d->b == 0;
  P->bf = d->dtype == MOMENTS_BF16;
  P->z = d->has_z != 0;
  RecGeo& g = P->g;
  g = RecGeo{};
  g.b = (int)d->b; g.s = (int)d->s; g.w = (int)d->w;
  g.V = (int)std::min(d->valid_len, d->s);
  g.xs = (size_t)xs; g.gs = (size_t)gs; g.zs = (size_t)zs;
  g.xr = d->s > 1 ? g.xs : (size_t)d->w; g.gr = d->s > 1 ? g.gs : (size_t)d->w; g.zr = d->s > 1 ? g.zs : (size_t)d->w;
  g.lens = (const int*)d->valid_lens;
  P->VC = bases && d->w % 2 == 0 && xs % 2 == 0 && gs % 2 == 0 && (!P->z || zs % 2 == 0) ? 2 : 1;
  const int64_t ncg = (d->w + 64 * P->VC - 1) / (64 * P->VC);
  if (d->b * ncg > kMostItems) return MOMENTS_ENOTSUP;
  g.ncg = (int)ncg;
  const int64_t items = d->b * ncg, tiles = (g.V + REC_TILE - 1) / REC_TILE;
  // Segments where the chain groups alone leave half the CUs without one: as many as fill them once
  // (a second round of workgroups costs as much as the first: 8 x 8192 x 2050 bf16, 136 groups, one
  // segment 982 us for forward and gradients, two 1514), of a tile or more, from four tiles on
  // (600 x 512: a tile each 54 us, two 69, one segment 75; 2 x 300 x 4096, three tiles: one segment
  // 47 us, three 53). From 129 to 255 groups that is one segment, and the CUs past the groups have no
  // work; of these only 136 groups were measured. A ragged batch has the same number for each sequence,
  // so the longest one's segments take longest.
  const int64_t n = tiles < 4 ? 1 : std::max<int64_t>(1, std::min(kCUs / std::max<int64_t>(items, 1), tiles));
  const int64_t per = std::max<int64_t>((tiles + n - 1) / n, 1);
  g.nseg = (int)std::max<int64_t>((tiles + per - 1) / per, 1);
  const size_t states = (size_t)g.b * g.w * 4, nsv = (size_t)((g.V + REC_SAVE - 1) / REC_SAVE);
  size_t o = 0;
  P->part = o;
  if (g.nseg > 1) o = align256(o + 2 * states * g.nseg);
  P->first = o;
  if (g.nseg > 1) o = align256(o + states);
  P->ws_fwd = o;
  P->saved = states * nsv;
  P->save = o;
  o = align256(o + P->saved);
  P->flag_bwd = o;
  P->ws_bwd = o + 256;
  return MOMENTS_OK;
}

// Calls f(TT<T>, IC<GATE>, IC<Z>, IC<V>) for the compiled variant of the plan.
template <class F>
int with_rec(const RecPlan& P, int gate, F&& f) {
  auto by_v = [&](auto tt, auto gk, auto zk) -> int {
    return P.VC == 2 ? f(tt, gk, zk, IC<2>{}) : f(tt, gk, zk, IC<1>{});
  };
  auto by_z = [&](auto tt, auto gk) -> int { return P.z ? by_v(tt, gk, IC<1>{}) : by_v(tt, gk, IC<0>{}); };
  auto by_gate = [&](auto tt) -> int {
    switch (gate) {
      case MOMENTS_GATE_LOG: return by_z(tt, IC<0>{});
      case MOMENTS_GATE_MIX: return by_z(tt, IC<1>{});
    }
    return by_z(tt, IC<2>{});
  };
  return P.bf ? by_gate(TT<bf16>{}) : by_gate(TT<float>{});
}

bool at_element(const void* p, bool bf) { return ((uintptr_t)p & (bf ? 1 : 3)) == 0; }
bool pairs(const void* x, const void* gg, const void* z, bool bf) {
  return (((uintptr_t)x | (uintptr_t)gg | (uintptr_t)z) & (bf ? 3 : 7)) == 0;
}

int make_call_plan(const moments_rec_desc* d, const void* x, const void* gg, const void* z, RecPlan* P) {
  MOM_TRY(make_rec_plan(d, P, pairs(x, gg, z, d != nullptr && d->dtype == MOMENTS_BF16)));
  if (!at_element(x, P->bf) || !at_element(gg, P->bf) || !at_element(z, P->bf)) return MOMENTS_EINVAL;
  return 0;
}

int all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p != nullptr && !aligned16(p)) return MOMENTS_EINVAL;
  return 0;
}

// The forward's launches: y and h_last (y NULL: only the saved states).
int launch_rec_fwd(const RecPlan& P, int gate, const void* x, const void* gg, const void* z, const float* h0, void* y,
                   float* h_last, float* save, unsigned char* ws, hipStream_t st) {
  const RecGeo& g = P.g;
  float *part = (float*)(ws + P.part), *first = (float*)(ws + P.first);
  return with_rec(P, gate, [&](auto tt, auto gk, auto zk, auto vk) -> int {
    using T = typename decltype(tt)::type;
    constexpr int G = decltype(gk)::value, V = decltype(vk)::value;
    constexpr bool Z = decltype(zk)::value != 0;
    const unsigned items = (unsigned)g.b * g.ncg;
    if (g.nseg > 1) {
      ProfScope ps(KID_REC_SEG, st);
      hipLaunchKernelGGL((k_rec_seg<T, G, false, V, false>), dim3(items * (g.nseg - 1)), dim3(REC_SW * 64), 0, st, g,
                         (const T*)x, (const T*)gg, (const T*)z, h0, part, first);
      MOM_TRY(check_launch());
    }
    if (y != nullptr) {
      ProfScope ps(KID_REC_FWD, st);
      hipLaunchKernelGGL((k_rec_fwd<T, G, Z, V, true>), dim3(items * g.nseg), dim3(REC_W * 64), 0, st, g, (const T*)x,
                         (const T*)gg, (const T*)z, h0, part, first, (T*)y, h_last, save);
    } else {
      ProfScope ps(KID_REC_FWD, st);
      hipLaunchKernelGGL((k_rec_fwd<T, G, false, V, false>), dim3(items * g.nseg), dim3(REC_W * 64), 0, st, g, (const T*)x,
                         (const T*)gg, (const T*)nullptr, h0, part, first, (T*)nullptr, (float*)nullptr, save);
    }
    return check_launch();
  });
}

int rec_forward(const moments_rec_desc* desc, const void* x, const void* gg, const void* z, const float* h0, void* y,
                float* h_last, void* saved, size_t saved_bytes, bool want_saved, void* workspace,
                size_t workspace_bytes, void* stream) {
  RecPlan P;
  MOM_TRY(make_call_plan(desc, x, gg, z, &P));
  const RecGeo& g = P.g;
  if (P.empty) return 0;
  if (g.s > 0 && (!x || !gg || !y)) return MOMENTS_EINVAL;
  if (P.z ? g.s > 0 && !z : z != nullptr) return MOMENTS_EINVAL;
  MOM_TRY(all_aligned({h0, y, h_last, saved, workspace}));
  if (want_saved && P.saved > 0) {
    if (saved == nullptr) return MOMENTS_EINVAL;
    if (saved_bytes < P.saved) return MOMENTS_EWORKSPACE;
  }
  if (P.ws_fwd > 0 && (workspace == nullptr || workspace_bytes < P.ws_fwd)) return MOMENTS_EWORKSPACE;
  if (g.s == 0 && h_last == nullptr) return 0;
  hipStream_t st = (hipStream_t)stream;
  void* out = g.s > 0 ? y : (void*)h_last;   // with no tokens y is not written
  MOM_TRY(launch_rec_fwd(P, desc->gate, x, gg, z, h0, out, h_last, want_saved && P.saved > 0 ? (float*)saved : nullptr,
                         (unsigned char*)workspace, st));
  if (check_finite_on()) {
    const OutSpan outs[] = {{y, (size_t)g.b * g.s * g.w, !P.bf}, {h_last, (size_t)g.b * g.w, true}};
    return check_finite(outs, 2, nullptr, st);
  }
  return 0;
}

int rec_backward(const moments_rec_desc* desc, const void* x, const void* gg, const void* z, const float* h0,
                 const void* saved, size_t saved_bytes, bool have_saved, const void* d_y, const float* d_h_last,
                 void* d_x, void* d_g, void* d_z, float* d_h0, void* workspace, size_t workspace_bytes, void* stream) {
  RecPlan P;
  MOM_TRY(make_call_plan(desc, x, gg, z, &P));
  const RecGeo& g = P.g;
  if (P.empty) return 0;
  if (g.s > 0 && (!x || !gg || !d_y)) return MOMENTS_EINVAL;
  if (P.z ? g.s > 0 && !z : z != nullptr || d_z != nullptr) return MOMENTS_EINVAL;
  MOM_TRY(all_aligned({h0, saved, d_y, d_h_last, d_x, d_g, d_z, d_h0, workspace}));
  if (have_saved && P.saved > 0) {
    if (saved == nullptr) return MOMENTS_EINVAL;
    if (saved_bytes < P.saved) return MOMENTS_EWORKSPACE;
  }
  if (workspace == nullptr || workspace_bytes < P.ws_bwd) return MOMENTS_EWORKSPACE;
  if (!d_x && !d_g && !d_z && !d_h0) return 0;
  hipStream_t st = (hipStream_t)stream;
  unsigned char* ws = (unsigned char*)workspace;
  const float* save = (const float*)saved;
  if (!have_saved) {
    save = (const float*)(ws + P.save);
    if (P.saved > 0)
      MOM_TRY(launch_rec_fwd(P, desc->gate, x, gg, z, h0, nullptr, nullptr, (float*)(ws + P.save), ws, st));
  }
  float *part = (float*)(ws + P.part), *first = (float*)(ws + P.first);
  MOM_TRY(with_rec(P, desc->gate, [&](auto tt, auto gk, auto zk, auto vk) -> int {
    using T = typename decltype(tt)::type;
    constexpr int G = decltype(gk)::value, V = decltype(vk)::value;
    constexpr bool Z = decltype(zk)::value != 0;
    const unsigned items = (unsigned)g.b * g.ncg;
    if (g.nseg > 1) {
      ProfScope ps(KID_REC_SEG, st);
      hipLaunchKernelGGL((k_rec_seg<T, G, Z, V, true>), dim3(items * g.nseg), dim3(REC_SW * 64), 0, st, g, (const T*)d_y,
                         (const T*)gg, (const T*)z, d_h_last, part, first);
      MOM_TRY(check_launch());
    }
    ProfScope ps(KID_REC_BWD, st);
    hipLaunchKernelGGL((k_rec_bwd<T, G, Z, V>), dim3(items * g.nseg), dim3(REC_WB * 64), 0, st, g, (const T*)x,
                       (const T*)gg, (const T*)z, save, (const T*)d_y, d_h_last, part, first, (T*)d_x, (T*)d_g,
                       (T*)d_z, d_h0);
    return check_launch();
  }));
  if (check_finite_on()) {
    const size_t n = (size_t)g.b * g.s * g.w;
    const OutSpan outs[] = {{d_x, n, !P.bf}, {d_g, n, !P.bf}, {d_z, n, !P.bf}, {d_h0, (size_t)g.b * g.w, true}};
    return check_finite(outs, 4, ws + P.flag_bwd, st);
  }
  return 0;
}

}  // namespace

extern "C" {

int moments_rec_validate(const moments_rec_desc* desc) {
  RecPlan P;   // with a lane to each channel there are the most workgroups
  MOM_TRY(make_rec_plan(desc, &P, true));
  return make_rec_plan(desc, &P, false);
}

int64_t moments_rec_workspace_size(const moments_rec_desc* desc, int is_bwd) {
  RecPlan P, U;   // where x, g and z start is not known here
  MOM_TRY(make_rec_plan(desc, &P, true));
  MOM_TRY(make_rec_plan(desc, &U, false));
  if (P.empty) return 0;
  return (int64_t)(is_bwd ? std::max(P.ws_bwd, U.ws_bwd) : std::max(P.ws_fwd, U.ws_fwd));
}

int64_t moments_rec_saved_size(const moments_rec_desc* desc) {
  RecPlan P;
  MOM_TRY(make_rec_plan(desc, &P, true));
  return P.empty ? 0 : (int64_t)P.saved;
}

int moments_rec_fwd(const moments_rec_desc* desc, const void* x, const void* g, const void* z, const float* h0,
                    void* y, float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
  return rec_forward(desc, x, g, z, h0, y, h_last, nullptr, 0, false, workspace, workspace_bytes, stream);
}

int moments_rec_fwd_save(const moments_rec_desc* desc, const void* x, const void* g, const void* z, const float* h0,
                         void* y, float* h_last, void* saved, size_t saved_bytes, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return rec_forward(desc, x, g, z, h0, y, h_last, saved, saved_bytes, true, workspace, workspace_bytes, stream);
}

int moments_rec_bwd(const moments_rec_desc* desc, const void* x, const void* g, const void* z, const float* h0,
                    const void* d_y, const float* d_h_last, void* d_x, void* d_g, void* d_z, float* d_h0,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return rec_backward(desc, x, g, z, h0, nullptr, 0, false, d_y, d_h_last, d_x, d_g, d_z, d_h0, workspace,
                      workspace_bytes, stream);
}

int moments_rec_bwd_saved(const moments_rec_desc* desc, const void* x, const void* g, const void* z, const float* h0,
                          const void* saved, size_t saved_bytes, const void* d_y, const float* d_h_last, void* d_x,
                          void* d_g, void* d_z, float* d_h0, void* workspace, size_t workspace_bytes, void* stream) {
  return rec_backward(desc, x, g, z, h0, saved, saved_bytes, true, d_y, d_h_last, d_x, d_g, d_z, d_h0, workspace,
                      workspace_bytes, stream);
}

int moments_rec_step(const moments_rec_desc* desc, const void* x, const void* g, const void* z, const int32_t* slots,
                     int64_t nslots, float* state, void* y, void* stream) {
  RecPlan P;
  MOM_TRY(make_call_plan(desc, x, g, z, &P));
  if (desc->s != 1 || nslots < 0 || nslots > (int64_t)1 << 30 || (slots == nullptr && nslots < desc->b)) return MOMENTS_EINVAL;
  if (P.empty) return 0;
  const RecGeo& q = P.g;
  if (!x || !g || !y || (nslots > 0 && !state) || P.z != (z != nullptr)) return MOMENTS_EINVAL;
  MOM_TRY(all_aligned({state, y}));
  if (((uintptr_t)slots & 3) != 0) return MOMENTS_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  MOM_TRY(with_rec(P, desc->gate, [&](auto tt, auto gk, auto zk, auto vk) -> int {
    using T = typename decltype(tt)::type;
    constexpr int V = decltype(vk)::value;
    ProfScope ps(KID_REC_STEP, st);
    const int cols = (q.w + 256 * V - 1) / (256 * V);   // a launch holds fewer than 2^32 threads
    hipLaunchKernelGGL((k_rec_step<T, decltype(gk)::value, decltype(zk)::value != 0, V>),
                       dim3((unsigned)cols, (unsigned)std::min(q.b, std::min(65535, (1 << 23) / cols))), dim3(256), 0,
                       st, q, (const T*)x, (const T*)g, (const T*)z, slots, nslots, state, (T*)y);
    return check_launch();
  }));
  if (check_finite_on()) {
    const OutSpan outs[] = {{y, (size_t)q.b * q.w, !P.bf}};
    return check_finite(outs, 1, nullptr, st);
  }
  return 0;
}

}  // extern "C"
