// C ABI of the gradients' norm and clipping: validation, planning, dispatch. The operation and its
// conventions are stated in include/moments.h.
#include "moments.h"

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "host.h"
#include "kernels_grad.h"

using namespace mom;

namespace {

constexpr int64_t kMostSpans = 1 << 20;

unsigned long long pieces_of(const moments_span& s) {
  const unsigned long long bytes = (unsigned long long)s.n * (s.dtype == MOMENTS_F32 ? 4 : 2);
  return (bytes + GRAD_PIECE - 1) / GRAD_PIECE;
}

int check_spans(const moments_span* spans, int64_t count) {
  if (count < 0 || (count > 0 && spans == nullptr)) return MOMENTS_EINVAL;
  if (count > kMostSpans) return MOMENTS_ENOTSUP;
  for (int64_t i = 0; i < count; i++) {
    const moments_span& s = spans[i];
    if (s.n < 0 || s.reserved != 0 || (s.dtype != MOMENTS_F32 && s.dtype != MOMENTS_BF16)) return MOMENTS_EINVAL;
    if (s.n == 0) continue;
    const uintptr_t low = s.dtype == MOMENTS_F32 ? 3 : 1;
    if (s.p == nullptr || ((uintptr_t)s.p & low) != 0 || ((uintptr_t)s.out & low) != 0) return MOMENTS_EINVAL;
    if (s.n > (int64_t)1 << 40) return MOMENTS_ENOTSUP;
  }
  return 0;
}

// Calls f(args, blocks) for the launches that hold the spans: up to GRAD_SPANS tensors each, and
// fewer pieces than 2^31.
template <class F>
int each_launch(const moments_span* spans, int64_t count, F&& f) {
  GradArgs A;
  int64_t i = 0;
  while (i < count) {
    A.count = 0;
    A.pieces = 0;
    for (; i < count && A.count < GRAD_SPANS; i++) {
      if (spans[i].n == 0) continue;
      const unsigned long long n = pieces_of(spans[i]);
      if (A.count > 0 && A.pieces + n >= 1ull << 31) break;
      void* out = spans[i].out ? spans[i].out : const_cast<void*>(spans[i].p);
      A.span[A.count++] = {spans[i].p, out, (unsigned long long)spans[i].n, A.pieces, spans[i].dtype == MOMENTS_F32};
      A.pieces += (unsigned)n;
    }
    if (A.count > 0) MOM_TRY(f(A, (int)std::min<unsigned>(A.pieces, GRAD_BLOCKS)));
  }
  return 0;
}

// The launches' workgroups together: a partial sum each.
int64_t blocks_of(const moments_span* spans, int64_t count) {
  int64_t n = 0;
  (void)each_launch(spans, count, [&](const GradArgs&, int blocks) -> int {
    n += blocks;
    return 0;
  });
  return n;
}

struct Range {
  uintptr_t a, b;
  int64_t span;
  bool out;
};

}  // namespace

extern "C" {

int moments_grad_validate(const moments_span* spans, int64_t count) {
  MOM_TRY(check_spans(spans, count));
  if (count == 0) return 0;
  Range* r = (Range*)malloc(sizeof(Range) * 2 * (size_t)count);
  if (r == nullptr) return MOMENTS_ENOTSUP;
  int64_t n = 0;
  for (int64_t i = 0; i < count; i++) {
    const moments_span& s = spans[i];
    if (s.n == 0) continue;
    const uintptr_t bytes = (uintptr_t)s.n * (s.dtype == MOMENTS_F32 ? 4 : 2);
    r[n++] = {(uintptr_t)s.p, (uintptr_t)s.p + bytes, i, s.out == nullptr || s.out == s.p};
    if (s.out != nullptr && s.out != s.p) r[n++] = {(uintptr_t)s.out, (uintptr_t)s.out + bytes, i, true};
  }
  std::sort(r, r + n, [](const Range& x, const Range& y) { return x.a < y.a; });
  int rc = 0;
  uintptr_t end = 0, end_out = 0;   // of all ranges so far, and of those that are written
  for (int64_t i = 0; i < n && rc == 0; i++) {
    if (r[i].a < end_out || (r[i].out && r[i].a < end)) rc = MOMENTS_EINVAL;
    end = std::max(end, r[i].b);
    if (r[i].out) end_out = std::max(end_out, r[i].b);
  }
  free(r);
  return rc;
}

int64_t moments_grad_workspace_size(const moments_span* spans, int64_t count) {
  MOM_TRY(check_spans(spans, count));
  return (int64_t)align256((size_t)std::max<int64_t>(blocks_of(spans, count), 1) * 8);
}

int moments_grad_norm(const moments_span* spans, int64_t count, float* norm, void* workspace, size_t workspace_bytes,
                      void* stream) {
  MOM_TRY(check_spans(spans, count));
  if (norm == nullptr || ((uintptr_t)norm & 3) != 0 || !aligned16(workspace)) return MOMENTS_EINVAL;
  const int64_t blocks = blocks_of(spans, count);
  if (workspace == nullptr || workspace_bytes < (size_t)std::max<int64_t>(blocks, 1) * 8) return MOMENTS_EWORKSPACE;
  hipStream_t st = (hipStream_t)stream;
  double* part = (double*)workspace;
  int64_t at = 0;
  MOM_TRY(each_launch(spans, count, [&](const GradArgs& A, int n) -> int {
    ProfScope ps(KID_GRAD_NORM, st);
    hipLaunchKernelGGL(k_grad_norm, dim3((unsigned)n), dim3(GRAD_T), 0, st, A, part + at);
    at += n;
    return check_launch();
  }));
  {
    ProfScope ps(KID_GRAD_TOTAL, st);
    hipLaunchKernelGGL(k_grad_total, dim3(1), dim3(1024), 0, st, part, blocks, norm);
    MOM_TRY(check_launch());
  }
  if (check_finite_on()) {
    const OutSpan outs[] = {{norm, 1, true}};
    return check_finite(outs, 1, nullptr, st);
  }
  return 0;
}

int moments_grad_clip(const moments_span* spans, int64_t count, const float* norm, float max_norm, void* stream) {
  MOM_TRY(check_spans(spans, count));
  if (norm == nullptr || ((uintptr_t)norm & 3) != 0 || !(max_norm >= 0.0f)) return MOMENTS_EINVAL;
  hipStream_t st = (hipStream_t)stream;
  return each_launch(spans, count, [&](const GradArgs& A, int n) -> int {
    ProfScope ps(KID_GRAD_CLIP, st);
    hipLaunchKernelGGL(k_grad_clip, dim3((unsigned)n), dim3(GRAD_T), 0, st, A, norm, max_norm);
    return check_launch();
  });
}

}  // extern "C"
