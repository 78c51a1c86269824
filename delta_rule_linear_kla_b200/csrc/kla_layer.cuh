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

// Longest sequence, and most channels of one: their indices and roundings up
// to blocks stay inside an int.
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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float sigmoid(float x) {
  return rcp(1.f + ex2(x * -1.4426950408889634f));
}
// x sigmoid(x): -0 for x far below zero (1 + e^-x = inf), NaN for -inf as the
// formula gives.
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }

// Two fp32 values in one register pair, and the packed operations on them
// (one issue slot for two results).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pack2(float a, float b) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpack2(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 v) {
  const float2 f = unpack2(v);
  return pack2(ex2(f.x), ex2(f.y));
}

__device__ __forceinline__ f32x2 both(float a) { return pack2(a, a); }

__device__ __forceinline__ f32x2 sigmoid2(f32x2 x) {
  const float2 t = unpack2(mul2(x, both(-1.4426950408889634f)));
  const float2 u = unpack2(add2(pack2(ex2(t.x), ex2(t.y)), both(1.f)));
  return pack2(rcp(u.x), rcp(u.y));
}
__device__ __forceinline__ f32x2 silu2(f32x2 x) { return mul2(x, sigmoid2(x)); }

// log(1 + e^x) = max(x, 0) + log(1 + e), e = e^-|x|, without overflow or
// cancellation on either side: log(1 + e) as e times a polynomial of degree 8
// fitted to log(1 + e) / e on [0, 1] by reweighted least squares (relative
// error 3e-8, 2e-7 evaluated in fp32), as exact for tiny e as for others, with
// one special function a value.
__device__ __forceinline__ f32x2 softplus2(f32x2 x) {
  const float2 t = unpack2(mul2(x, both(1.4426950408889634f))), v = unpack2(x);
  const f32x2 e = pack2(ex2(-fabsf(t.x)), ex2(-fabsf(t.y)));
  f32x2 r = fma2(e, both(0.0052326936f), both(-0.029505236f));
  r = fma2(e, r, both(0.078225948f));
  r = fma2(e, r, both(-0.13663246f));
  r = fma2(e, r, both(0.19106007f));
  r = fma2(e, r, both(-0.24842982f));
  r = fma2(e, r, both(0.33319098f));
  r = fma2(e, r, both(-0.49999493f));
  r = fma2(e, r, both(0.99999994f));
  return fma2(e, r, pack2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return unpack2(softplus2(both(x))).x; }

// Four neighbouring values as two pairs.
struct Quad {
  f32x2 a, b;
};
__device__ __forceinline__ Quad quad(float4 v) { return Quad{pack2(v.x, v.y), pack2(v.z, v.w)}; }
__device__ __forceinline__ float4 flat(Quad v) {
  const float2 a = unpack2(v.a), b = unpack2(v.b);
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ Quad operator+(Quad x, Quad y) {
  return Quad{add2(x.a, y.a), add2(x.b, y.b)};
}
__device__ __forceinline__ Quad operator*(Quad x, Quad y) {
  return Quad{mul2(x.a, y.a), mul2(x.b, y.b)};
}
__device__ __forceinline__ Quad fma4(Quad x, Quad y, Quad z) {
  return Quad{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)};
}
__device__ __forceinline__ Quad all4(float x) { return Quad{both(x), both(x)}; }
__device__ __forceinline__ Quad sigmoid4(Quad x) { return Quad{sigmoid2(x.a), sigmoid2(x.b)}; }
__device__ __forceinline__ Quad silu4(Quad x) { return Quad{silu2(x.a), silu2(x.b)}; }
__device__ __forceinline__ Quad softplus4(Quad x) { return Quad{softplus2(x.a), softplus2(x.b)}; }

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

// Four elements as they lie in memory, to be held between a load and its use.
template <typename T>
struct Raw4;
template <>
struct Raw4<__nv_bfloat16> {
  uint2 r;
  __device__ __forceinline__ float4 get() const {
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
  }
};
template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ float4 get() const { return r; }
};
template <typename T>
__device__ __forceinline__ Raw4<T> ld_raw4(const T* p) {
  Raw4<T> v;
  v.r = *reinterpret_cast<const decltype(v.r)*>(p);
  return v;
}
// The first n of the four at p (ld4's rule), zeros behind.
template <typename T>
__device__ __forceinline__ Raw4<T> ld_raw4(const T* p, int n, bool vec) {
  Raw4<T> v;
  if (vec && n >= 4) {
    v.r = *reinterpret_cast<const decltype(v.r)*>(p);
    return v;
  }
  v.r = {};
  T* o = reinterpret_cast<T*>(&v.r);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) o[i] = p[i];
  return v;
}

// Copies of 16 or 4 bytes to shared memory that hold no register while they are
// in flight; cp_wait waits for all but the last KEEP committed groups of this
// thread.
__device__ __forceinline__ void cp16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void cp4(void* to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(to)),
               "l"(from)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int KEEP>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(KEEP) : "memory");
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
