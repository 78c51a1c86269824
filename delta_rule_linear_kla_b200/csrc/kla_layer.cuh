// Shared pieces of the layer operators around the recurrence (short causal
// convolution, selective scan, query/key norm): host-side argument checks and
// the element helpers of their kernels.
#pragma once

#include "kla_common.cuh"

namespace kla {
namespace layer {

// ---- host: argument checks (same conventions as kla_api.cu) ----

struct Span {
  uintptr_t lo, hi;
};

// Bytes of `rows` rows of `n` elements, ld elements apart (the last row ends
// after its n elements).
inline Span span(const void* p, long long rows, long long n, long long ld, int es) {
  const uintptr_t a = (uintptr_t)p;
  if (!p || rows <= 0 || n <= 0) return Span{a, a};
  return Span{a, a + (uintptr_t)((rows - 1) * ld + n) * es};
}
inline Span span(const void* p, long long n, int es) { return span(p, 1, n, n, es); }

inline bool overlap(Span a, Span b) {
  return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi;
}

// True when a written span overlaps an input or another written span.
template <int NI, int NO>
inline bool conflicts(const Span (&in)[NI], const Span (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Span& s : in)
      if (overlap(out[i], s)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

template <int NP>
inline bool misaligned(const void* const (&p)[NP]) {
  for (const void* q : p)
    if (((uintptr_t)q & 15u) != 0) return true;
  return false;
}

// Rows of a wider matrix may start anywhere: whether groups of v elements of
// them can be accessed at once (rows of n elements, ld apart).
inline bool rows_aligned(const void* p, long long n, long long ld, int v, int es) {
  return n % v == 0 && ld % v == 0 && (uintptr_t)p % (uintptr_t)(v * es) == 0;
}
inline bool misplaced(const void* p, int es) { return (uintptr_t)p % (uintptr_t)es != 0; }

// Longest sequence: token indices and their roundings up stay inside an int.
constexpr int kMaxTokens = 1 << 30;

inline bool dtype_ok(int dtype) { return dtype == KLA_BF16 || dtype == KLA_FP32; }
inline int elem(int dtype) { return dtype == KLA_BF16 ? 2 : 4; }

// Sizes of an activation [rows][ld]: every offset (in bytes) below 2^46, so
// that no 64-bit index below can wrap.
inline bool size_ok(long long rows, long long ld) {
  return rows >= 0 && ld >= 0 && rows < (1LL << 40) && ld < (1LL << 40) &&
         (rows == 0 || ld <= (1LL << 44) / rows);
}

// ---- device: element helpers ----

__device__ __forceinline__ float sigmoid(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}
// x sigmoid(x): -0 for x far below zero (1 + e^-x = inf), NaN for -inf as the
// formula gives.
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }

// log(1 + e^x) without overflow or cancellation on either side.
__device__ __forceinline__ float softplus(float x) {
  return fmaxf(x, 0.f) + log1pf(__expf(-fabsf(x)));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Up to 4 consecutive elements at p, of which the first n exist; vec says
// that a whole group of 4 is aligned for one vector access.
template <typename T>
__device__ __forceinline__ float4 ld4(const T* p, int n, bool vec) {
  if (vec && n >= 4) return IO<T>::ld4(p);
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n > 0) r.x = IO<T>::ld(p);
  if (n > 1) r.y = IO<T>::ld(p + 1);
  if (n > 2) r.z = IO<T>::ld(p + 2);
  if (n > 3) r.w = IO<T>::ld(p + 3);
  return r;
}
template <typename T>
__device__ __forceinline__ void st4(T* p, float4 v, int n, bool vec) {
  if (vec && n >= 4) {
    IO<T>::st4(p, v);
    return;
  }
  if (n > 0) IO<T>::st(p, v.x);
  if (n > 1) IO<T>::st(p + 1, v.y);
  if (n > 2) IO<T>::st(p + 2, v.z);
  if (n > 3) IO<T>::st(p + 3, v.w);
}

// Tokens of sequence b that exist: lengths[b] clamped to [0, T] (no lengths:
// all T).
__device__ __forceinline__ int live_tokens(const int* lengths, int b, int T) {
  if (!lengths) return T;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

}  // namespace layer
}  // namespace kla
