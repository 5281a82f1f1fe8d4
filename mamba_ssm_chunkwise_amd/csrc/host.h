// Host helpers shared by the library's translation units: the last HIP error,
// launch checks, the optional per-kernel event timing (moments_profile_*) and
// the debug finiteness check. Defined in moments.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "moments.h"

namespace mom {

constexpr size_t kLdsLimit = 160 * 1024;
constexpr long kCUs = 256;  // compute units of the part (MI355X)

enum KernelId {
  KID_CARRY, KID_SCAN, KID_FWD, KID_REDUCE, KID_BWD, KID_DSCAN, KID_FIX, KID_ZERO, KID_PREP, KID_GSCAN, KID_GFIX,
  KID_CSCAN, KID_ROTSEG, KID_ROTCARRY, KID_ROTAPPLY, KID_PAIR, KID_GENTRY, KID_CSUM, KID_CGRP,
  KID_ATTN_STATE, KID_ATTN_SCAN, KID_ATTN_FWD, KID_ATTN_BWD, KID_ATTN_SUM, KID_ATTN_STEP, KID_QK_FWD, KID_QK_BWD, KID_QK_SUM,
  KID_REC_SEG, KID_REC_FWD, KID_REC_BWD, KID_REC_STEP, KID_LN_FWD, KID_LN_BWD, KID_LN_SUM,
  KID_GRAD_NORM, KID_GRAD_TOTAL, KID_GRAD_CLIP,
  KID_N
};

// Brackets one launch with events when profiling is on.
struct ProfScope {
  int kid;
  hipStream_t st;
  hipEvent_t a = nullptr;
  ProfScope(int k, hipStream_t s);
  ~ProfScope();
};

// Records the error for moments_last_hip_error(); returns MOMENTS_EHIP.
int hip_fail(hipError_t e);

inline int check_launch() {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? 0 : hip_fail(e);
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

template <typename K>
int set_lds(K kernel, size_t bytes) {
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  return e == hipSuccess ? 0 : hip_fail(e);
}

// set_lds once for each device instead of at every launch: `done` is a static of the
// launch site (one bit a device; devices past 63 are set every time).
template <typename K>
int set_lds_once(std::atomic<uint64_t>& done, K kernel, size_t bytes) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e);
  const uint64_t bit = dev < 64 ? uint64_t{1} << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return 0;
  const int rc = set_lds(kernel, bytes);
  if (rc == 0) done.fetch_or(bit, std::memory_order_relaxed);
  return rc;
}

#define MOM_TRY(x)          \
  do {                      \
    const int _rc = (x);    \
    if (_rc != 0) return _rc; \
  } while (0)

template <int V> using IC = std::integral_constant<int, V>;
template <typename T> struct TT { using type = T; };

// Debug finiteness check, on when the environment variable MOMENTS_CHECK_FINITE
// is set to anything but "" or "0". It waits for the stream and returns
// MOMENTS_ENONFINITE if any listed output holds a NaN or an infinity. flag_mem: 4 bytes of the
// call's workspace, or nullptr where it has none (a flag of the library's own, under a lock).
struct OutSpan {
  const void* p;
  size_t n;
  bool f32;
};
bool check_finite_on();
int check_finite(const OutSpan* outs, int nout, unsigned char* flag_mem, hipStream_t st);

}  // namespace mom
