// Norm of many gradients and their clipping: kernels.
//
//   norm = sqrt(sum over all values of v^2),  v <- v min(1, max_norm / (norm + 1e-6))
//
// A launch takes the addresses of up to GRAD_SPANS tensors as its argument, so nothing is copied to
// the device before it and a captured graph keeps them. The values are dealt to the workgroups in
// pieces of GRAD_PIECE bytes, whichever tensor they are of. Squares are summed in double, so that
// neither large nor small gradients leave the range, and in a fixed order.
//
// Bound by memory: 0.47e9 bf16 values in 56 tensors, norm 185 us (0.94 GB, 5.1 TB/s), clipping into
// other buffers 340 us (1.88 GB, 5.5 TB/s).
#pragma once

#include "common.h"

namespace mom {

constexpr int GRAD_SPANS = 64;
constexpr int GRAD_T = 256;
constexpr int GRAD_U = 8;                                // 16-byte loads of a thread in flight
constexpr int GRAD_PIECE = GRAD_T * GRAD_U * 16;         // bytes
constexpr int GRAD_BLOCKS = 2048;                        // workgroups of a launch, at most

struct GradSpan {
  const void* p;
  void* out;           // where the clipped values go (p: in place)
  unsigned long long n;
  unsigned piece0;     // pieces of the spans before this one
  int f32;
};
struct GradArgs {
  int count;
  unsigned pieces;
  GradSpan span[GRAD_SPANS];
};

// The span that holds a piece: the last whose first piece is not past it.
__device__ __forceinline__ int grad_find(const GradArgs& A, unsigned piece) {
  int lo = 0, hi = A.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (A.span[mid].piece0 <= piece) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A span in whole 16-byte words from its first aligned address on: `head` values before them.
struct GradCut {
  unsigned long long head, words, tail;   // values, words, values past the last word
  __device__ GradCut(const GradSpan& s) {
    const unsigned e = s.f32 ? 4 : 2, per = 16 / e;
    head = ((16 - (unsigned)((uintptr_t)s.p & 15)) & 15) / e;
    if (head > s.n) head = s.n;
    words = (s.n - head) / per;
    tail = s.n - head - words * per;
  }
};

__device__ __forceinline__ void grad_add(double& s, float v) { s = fma((double)v, (double)v, s); }

__global__ __launch_bounds__(GRAD_T) void k_grad_norm(GradArgs A, double* __restrict__ part) {
  __shared__ double lds[GRAD_T / 64];
  double s[4] = {};
  for (unsigned piece = blockIdx.x; piece < A.pieces; piece += gridDim.x) {
    const GradSpan sp = A.span[grad_find(A, piece)];
    const GradCut cut(sp);
    const unsigned long long w0 = (unsigned long long)(piece - sp.piece0) * (GRAD_T * GRAD_U);
    const u4* words = reinterpret_cast<const u4*>(reinterpret_cast<const char*>(sp.p) + cut.head * (sp.f32 ? 4 : 2));
    u4 v[GRAD_U];
#pragma unroll
    for (int i = 0; i < GRAD_U; i++) {
      const unsigned long long k = w0 + i * GRAD_T + threadIdx.x;
      v[i] = k < cut.words ? words[k] : u4{0, 0, 0, 0};
    }
    if (sp.f32) {
#pragma unroll
      for (int i = 0; i < GRAD_U; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) grad_add(s[j], __uint_as_float(v[i][j]));
    } else {
#pragma unroll
      for (int i = 0; i < GRAD_U; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          grad_add(s[j], bf16_lo(v[i][j]));
          grad_add(s[j], bf16_hi(v[i][j]));
        }
    }
    if (piece == sp.piece0) {   // the values outside the words
      const unsigned k = threadIdx.x;
      const unsigned long long at = k < cut.head ? k : cut.head + cut.words * (sp.f32 ? 4 : 8) + (k - cut.head);
      if (k < cut.head + cut.tail)
        grad_add(s[0], sp.f32 ? reinterpret_cast<const float*>(sp.p)[at] : to_f(reinterpret_cast<const bf16*>(sp.p)[at]));
    }
  }
  double t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x == 0) part[blockIdx.x] = (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

__global__ __launch_bounds__(1024) void k_grad_total(const double* __restrict__ part, int64_t n, float* norm) {
  __shared__ double lds[16];
  double t = 0.0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < n; i += 1024) t += part[i];
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) t += __shfl_xor(t, o, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = t;
  __syncthreads();
  if (threadIdx.x != 0) return;
  t = 0.0;
  for (int i = 0; i < 16; i++) t += lds[i];
  *norm = (float)sqrt(t);
}

// A norm that is not finite leaves the values as they are. Pieces are taken from the last one back,
// those that the norm read last first: they are the ones that a cache may still hold.
__global__ __launch_bounds__(GRAD_T) void k_grad_clip(GradArgs A, const float* __restrict__ norm, float max_norm) {
  const float n = *norm;
  float f = max_norm / (n + 1e-6f);
  if (!(n >= 0.0f && n < __builtin_inff()) || !(f < 1.0f)) f = 1.0f;
  for (unsigned i0 = blockIdx.x; i0 < A.pieces; i0 += gridDim.x) {
    const unsigned piece = A.pieces - 1 - i0;
    const GradSpan sp = A.span[grad_find(A, piece)];
    if (f == 1.0f && sp.p == sp.out) continue;
    const GradCut cut(sp);
    const unsigned long long w0 = (unsigned long long)(piece - sp.piece0) * (GRAD_T * GRAD_U);
    const unsigned long long shift = cut.head * (sp.f32 ? 4 : 2);
    const u4* words = reinterpret_cast<const u4*>(reinterpret_cast<const char*>(sp.p) + shift);
    char* out = reinterpret_cast<char*>(sp.out) + shift;
    const bool whole = ((uintptr_t)out & 15) == 0;
    u4 v[GRAD_U];
#pragma unroll
    for (int i = 0; i < GRAD_U; i++) {
      const unsigned long long k = w0 + i * GRAD_T + threadIdx.x;
      v[i] = k < cut.words ? words[k] : u4{0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < GRAD_U; i++) {
      const unsigned long long k = w0 + i * GRAD_T + threadIdx.x;
      if (f != 1.0f) {
#pragma unroll
        for (int j = 0; j < 4; j++)
          v[i][j] = sp.f32 ? __float_as_uint(__uint_as_float(v[i][j]) * f)
                           : pk_bf16(bf16_lo(v[i][j]) * f, bf16_hi(v[i][j]) * f);
      }
      if (k < cut.words) {
        if (whole) {
          reinterpret_cast<u4*>(out)[k] = v[i];
        } else if (sp.f32) {   // the output stands otherwise to 16 bytes than the input
#pragma unroll
          for (int j = 0; j < 4; j++) reinterpret_cast<float*>(out)[4 * k + j] = __uint_as_float(v[i][j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; j++) {
            reinterpret_cast<unsigned short*>(out)[8 * k + 2 * j] = (unsigned short)v[i][j];
            reinterpret_cast<unsigned short*>(out)[8 * k + 2 * j + 1] = (unsigned short)(v[i][j] >> 16);
          }
        }
      }
    }
    if (piece == sp.piece0) {
      const unsigned k = threadIdx.x;
      const unsigned long long at = k < cut.head ? k : cut.head + cut.words * (sp.f32 ? 4 : 8) + (k - cut.head);
      if (k < cut.head + cut.tail) {
        if (sp.f32)
          reinterpret_cast<float*>(sp.out)[at] = reinterpret_cast<const float*>(sp.p)[at] * f;
        else
          reinterpret_cast<bf16*>(sp.out)[at] = to_t<bf16>(to_f(reinterpret_cast<const bf16*>(sp.p)[at]) * f);
      }
    }
  }
}

}  // namespace mom
