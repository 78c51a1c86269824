// Short causal depthwise convolution: the mixing of neighbouring tokens in
// front of a linear-attention recurrence, for prompts, their backward pass
// and single tokens.
//
//   p[t][d] = bias[d] + sum_{j<W} w[d][j] x[t-W+1+j][d],   y = p or p sigmoid(p)
//
// with x[-W+1 .. -1] the state s0 (the last W-1 inputs of what came before).
// All arithmetic is fp32; only y (and dx, ds0) are rounded, once, to the
// activations' type.
#include <type_traits>

#include "kla_layer.cuh"

namespace kla {
namespace conv {

using namespace layer;

// V channels of one row as they lie in memory, and as P packed pairs of fp32
// (a single channel leaves the second of its pair 0).
template <int V>
constexpr int kPairs = (V + 1) / 2;

template <typename T, int V>
struct Row {
  static constexpr int P = kPairs<V>;
  static constexpr int B = sizeof(T) * V;  // 2 .. 16 bytes
  using Raw = typename std::conditional<
      B == 16, uint4, typename std::conditional<B == 8, uint2, T>::type>::type;
  Raw r;
  __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const Raw*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<Raw*>(p) = r; }
  __device__ __forceinline__ void zero() { r = Raw{}; }
  __device__ __forceinline__ void get(f32x2 (&f)[P]) const {
    if constexpr (V == 1) {
      f[0] = pack2(IO<T>::ld(reinterpret_cast<const T*>(&r)), 0.f);
    } else {
      const uint32_t* u = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if constexpr (sizeof(T) == 2)
          f[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
        else
          f[i] = pack2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
      }
    }
  }
  __device__ __forceinline__ void set(const f32x2 (&f)[P]) {
    if constexpr (V == 1) {
      IO<T>::st(reinterpret_cast<T*>(&r), unpack2(f[0]).x);
    } else {
      uint32_t* u = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float2 v = unpack2(f[i]);
        if constexpr (sizeof(T) == 2) {
          __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
          u[i] = *reinterpret_cast<uint32_t*>(&h);
        } else {
          u[2 * i] = __float_as_uint(v.x);
          u[2 * i + 1] = __float_as_uint(v.y);
        }
      }
    }
  }
};

// Row i of a sequence's inputs, i in [-(W-1), T): the state before 0.
template <typename T, int V, int W>
__device__ __forceinline__ Row<T, V> input_row(const T* xb, long long ldx, const T* s0b, int D,
                                               int i) {
  Row<T, V> r;
  if (i >= 0)
    r.load(xb + (long long)i * ldx);
  else if (s0b)
    r.load(s0b + (long long)(W - 1 + i) * D);
  else
    r.zero();
  return r;
}

// The W taps and the bias of V channels from c, as pairs; a channel's taps are
// one 16- or 8-byte access for W = 4 or 2.
template <int V, int W>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int c,
                                          f32x2 (&tap)[W][kPairs<V>], f32x2 (&b0)[kPairs<V>]) {
  float f[2][W], q[2];
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool in = 2 * i + k < V;
      const float* p = w + (long long)(c + 2 * i + k) * W;
      if constexpr (W == 4) {
        const float4 v = in ? *reinterpret_cast<const float4*>(p) : make_float4(0, 0, 0, 0);
        f[k][0] = v.x; f[k][1] = v.y; f[k][2] = v.z; f[k][3] = v.w;
      } else if constexpr (W == 2) {
        const float2 v = in ? *reinterpret_cast<const float2*>(p) : make_float2(0, 0);
        f[k][0] = v.x; f[k][1] = v.y;
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) f[k][j] = in ? p[j] : 0.f;
      }
      q[k] = in && bias ? bias[c + 2 * i + k] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < W; ++j) tap[j][i] = pack2(f[0][j], f[1][j]);
    b0[i] = pack2(q[0], q[1]);
  }
}

// p = bias + sum of the taps, oldest first
template <int V, int W>
__device__ __forceinline__ void taps_sum(const f32x2 (&tap)[W][kPairs<V>],
                                         const f32x2 (&b0)[kPairs<V>],
                                         const f32x2 (&win)[W - 1][kPairs<V>],
                                         const f32x2 (&cur)[kPairs<V>], f32x2 (&p)[kPairs<V>]) {
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
    p[i] = b0[i];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) p[i] = fma2(tap[j][i], win[j][i], p[i]);
    p[i] = fma2(tap[W - 1][i], cur[i], p[i]);
  }
}

// SiLU of a pair (value by value: the packed form takes registers that the
// prompt's kernel does not have, 57 us instead of 53 for 8 x 4096 x 2048)
__device__ __forceinline__ f32x2 activate(f32x2 p) {
  const float2 v = unpack2(p);
  return pack2(silu(v.x), silu(v.y));
}

template <int V, int W>
__device__ __forceinline__ void shift(f32x2 (&win)[W - 1][kPairs<V>],
                                      const f32x2 (&cur)[kPairs<V>]) {
#pragma unroll
  for (int i = 0; i < kPairs<V>; ++i) {
#pragma unroll
    for (int j = 0; j + 1 < W - 1; ++j) win[j][i] = win[j + 1][i];
    win[W - 2][i] = cur[i];
  }
}

// ---------------------------------------------------------------- prompt
//
// Bound by HBM: one read of x and one write of y.  A thread walks L tokens of
// V channels with the last W-1 inputs in registers, so that x is read once
// but for W-1 rows at the start of each walk (from L2); neighbouring lanes
// hold neighbouring channels.  Four rows are in flight while the four before
// are computed, on packed pairs of channels.  Blocks of 128 threads at 72
// registers, 28 warps an SM, carry enough loads: 8 x 4096 x 2048 bf16 takes
// 53 us, 5.0 TB/s (64 us with 256 threads at 64 registers, 107 us with eight
// channels a thread).
constexpr int kFT = 128;
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kFT, 7)
conv_fwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ s0,
                const int* __restrict__ lengths, T* __restrict__ y, T* __restrict__ sT,
                int Tn, int D, unsigned CG, unsigned NB, int L, unsigned total) {
  constexpr int P = kPairs<V>;
  const unsigned id = blockIdx.x * kFT + threadIdx.x;
  if (id >= total) return;
  const unsigned rest = id / CG, cg = id - rest * CG, b = rest / NB, tb = rest - b * NB;
  const int c = (int)cg * V;
  const int n = live_tokens(lengths, b, Tn);
  const T* xb = x + (long long)b * Tn * ldx + c;
  const T* s0b = s0 ? s0 + (long long)b * (W - 1) * D + c : nullptr;
  T* yb = y + (long long)b * Tn * D + c;

  const int t0 = (int)tb * L, t1 = min(Tn, t0 + L), tn = min(t1, n);
  Row<T, V> next[4];
  auto fetch = [&](int t) {
    const T* px = xb + (long long)t * ldx;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      next[i].load(px);
      px += ldx;
    }
  };
  if (t0 + 4 <= tn) fetch(t0);
  f32x2 tap[W][P], b0[P], win[W - 1][P];  // win[j] = row t - (W-1) + j
  load_taps<V, W>(w, bias, c, tap, b0);
  if (t0 < tn) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_row<T, V, W>(xb, ldx, s0b, D, t0 - (W - 1) + j).get(win[j]);
  }
  auto one = [&](const Row<T, V>& r, T* to) {
    f32x2 cur[P], p[P];
    r.get(cur);
    taps_sum<V, W>(tap, b0, win, cur, p);
    shift<V, W>(win, cur);
    if (SILU)
#pragma unroll
      for (int i = 0; i < P; ++i) p[i] = activate(p[i]);
    Row<T, V> o;
    o.set(p);
    o.store(to);
  };
  int t = t0;
  T* py = yb + (long long)t * D;
  while (t + 4 <= tn) {
    Row<T, V> r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = next[i];
    t += 4;
    if (t + 4 <= tn) fetch(t);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      one(r[i], py);
      py += D;
    }
  }
  for (; t < tn; ++t) {
    Row<T, V> r;
    r.load(xb + (long long)t * ldx);
    one(r, yb + (long long)t * D);
  }
  Row<T, V> zero;
  zero.zero();
  for (t = max(t0, tn); t < t1; ++t) zero.store(yb + (long long)t * D);

  if (sT && tb == NB - 1) {  // the last W-1 inputs that exist
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
      input_row<T, V, W>(xb, ldx, s0b, D, n - (W - 1) + j)
          .store(sT + ((long long)b * (W - 1) + j) * D + c);
  }
}

// ---------------------------------------------------------------- backward
//
// dp = dy act'(p);  dx[i] = sum_j w[j] dp[i + W-1-j];  dw[j] = sum_t dp[t]
// x[t-W+1+j];  dbias = sum dp; the state's rows take dx at negative i, and
// the final state's gradient goes to the rows that it copied.  Bound by HBM:
// x and dy read, dx written.  A thread walks L + W-1 tokens of V channels
// once, forming p and dp and emitting dx[t-W+1] at token t; the W-1 tokens
// behind its own L are formed twice.  dw and dbias are summed in registers,
// over the block's walks in shared memory, and over blocks by
// conv_reduce_kernel in a fixed order (no atomics).  4 x 8192 x 2048 bf16: 103 us,
// 3.9 TB/s; about 28 instructions a value (54 % of the issue slots at 16 warps
// an SM, the registers' limit) hold it above the 62 us of its bytes.
constexpr int kBX = 32, kBY = 4;  // channel groups x walks of a block

template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(kBX* kBY, 4)
conv_bwd_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w,
                const float* __restrict__ bias, const T* __restrict__ s0,
                const int* __restrict__ lengths, const T* __restrict__ gy,
                const T* __restrict__ gs, T* __restrict__ dx, T* __restrict__ ds0,
                float* __restrict__ part, int Tn, int D, int CB, int NB, int L) {
  constexpr int P = kPairs<V>;
  const int cb = blockIdx.x % CB;
  const int rest = blockIdx.x / CB;
  const int nb = rest % NB, b = rest / NB;  // this block's kBY * L tokens
  const int c = (cb * kBX + threadIdx.x) * V;
  f32x2 dw[W][P], db[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    db[i] = pack2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = db[i];
  }
  const int t0 = (nb * kBY + threadIdx.y) * L;
  if (c < D && t0 < Tn) {
    const int n = live_tokens(lengths, b, Tn);
    const T* xb = x + (long long)b * Tn * ldx + c;
    const T* s0b = s0 ? s0 + (long long)b * (W - 1) * D + c : nullptr;
    const T* gb = gy + (long long)b * Tn * D + c;
    const T* gsb = gs ? gs + (long long)b * (W - 1) * D + c : nullptr;
    T* db_x = dx + (long long)b * Tn * D + c;
    T* db_s = ds0 ? ds0 + (long long)b * (W - 1) * D + c : nullptr;
    const int t1 = min(Tn, t0 + L), tn = min(t1, n);
    Row<T, V> nx[4], ng[4];
    auto fetch = [&](int t) {
      const T *px = xb + (long long)t * ldx, *pg = gb + (long long)t * D;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        nx[i].load(px);
        ng[i].load(pg);
        px += ldx;
        pg += D;
      }
    };
    if (t0 + 4 <= tn) fetch(t0);
    f32x2 tap[W][P], b0[P];
    load_taps<V, W>(w, bias, c, tap, b0);
    f32x2 win[W - 1][P];  // rows t - (W-1) .. t - 1
    f32x2 dpw[W - 1][P];  // dp[t - (W-1)] .. dp[t - 1]
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Row<T, V> r;
      r.zero();  // rows at or past the length are not read
      if (t0 - (W - 1) + j < n) r = input_row<T, V, W>(xb, ldx, s0b, D, t0 - (W - 1) + j);
      r.get(win[j]);
#pragma unroll
      for (int i = 0; i < P; ++i) dpw[j][i] = pack2(0.f, 0.f);
    }
    // dp of token t, whose sums go to dw where it is one of the walk's own
    auto grad = [&](const Row<T, V>& rx, const Row<T, V>& rg, bool own, f32x2 (&dp)[P]) {
      f32x2 cur[P];
      rx.get(cur);
      rg.get(dp);
      if (SILU) {
        f32x2 p[P];
        taps_sum<V, W>(tap, b0, win, cur, p);
#pragma unroll
        for (int i = 0; i < P; ++i) {  // act' = s + p (s - s^2)
          const f32x2 s = sigmoid2(p[i]);
          dp[i] = mul2(dp[i], fma2(p[i], fma2(mul2(s, both(-1.f)), s, s), s));
        }
      }
      if (own) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][i] = fma2(dp[i], win[j][i], dw[j][i]);
          dw[W - 1][i] = fma2(dp[i], cur[i], dw[W - 1][i]);
          db[i] = add2(db[i], dp[i]);
        }
      }
      shift<V, W>(win, cur);
    };
    // dx[t - (W-1)]
    auto back = [&](const f32x2 (&dp)[P], f32x2 (&o)[P]) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        o[i] = mul2(tap[0][i], dp[i]);
#pragma unroll
        for (int j = 1; j < W; ++j) o[i] = fma2(tap[j][i], dpw[W - 1 - j][i], o[i]);
      }
      shift<V, W>(dpw, dp);
    };
    int t = t0;
    while (t + 4 <= tn) {
      Row<T, V> rx[4], rg[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) { rx[i] = nx[i]; rg[i] = ng[i]; }
      if (t + 8 <= tn) fetch(t + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f32x2 dp[P], o[P];
        grad(rx[i], rg[i], true, dp);
        back(dp, o);
        const int at = t + i - (W - 1);
        Row<T, V> ro;
        ro.set(o);
        if (at >= t0)
          ro.store(db_x + (long long)at * D);
        else if (t0 == 0 && db_s)
          ro.store(db_s + (long long)(W - 1 + at) * D);
      }
      t += 4;
    }
    const int emit0 = t0 == 0 ? -(W - 1) : t0;
    for (; t < t1 + W - 1; ++t) {
      f32x2 dp[P], o[P];
      if (t < n) {
        Row<T, V> rx, rg;
        rx.load(xb + (long long)t * ldx);
        rg.load(gb + (long long)t * D);
        grad(rx, rg, t < t1, dp);
      } else {
#pragma unroll
        for (int i = 0; i < P; ++i) dp[i] = pack2(0.f, 0.f);
      }
      back(dp, o);
      const int at = t - (W - 1);
      if (at < emit0 || at >= t1) continue;
      if (at >= n) {  // no such token: zero, whatever the taps are
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = pack2(0.f, 0.f);
      }
      const int r = t - n;  // row of the final state that holds input `at`
      if (gsb && r >= 0 && r < W - 1) {
        Row<T, V> rs;
        f32x2 f[P];
        rs.load(gsb + (long long)r * D);
        rs.get(f);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = add2(o[i], f[i]);
      }
      Row<T, V> ro;
      ro.set(o);
      if (at >= 0)
        ro.store(db_x + (long long)at * D);
      else if (db_s)
        ro.store(db_s + (long long)(W - 1 + at) * D);
    }
  }
  // block sums: [W + 1][kBX * V], one walk after the other
  __shared__ float red[kBY][W + 1][kBX * V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float2 v = unpack2(dw[j][e / 2]);
      red[threadIdx.y][j][threadIdx.x * V + e] = e & 1 ? v.y : v.x;
    }
    const float2 v = unpack2(db[e / 2]);
    red[threadIdx.y][W][threadIdx.x * V + e] = e & 1 ? v.y : v.x;
  }
  __syncthreads();
  float* pb = part + (long long)(b * NB + nb) * (W + 1) * D;
  for (int i = threadIdx.y * kBX + threadIdx.x; i < (W + 1) * kBX * V; i += kBX * kBY) {
    const int j = i / (kBX * V), k = i % (kBX * V);
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < kBY; ++r) s += red[r][j][k];
    const int d = cb * kBX * V + k;
    if (d < D) pb[(long long)j * D + d] = s;
  }
}

// Sums the blocks' parts [P][W + 1][D] in order: dw[d][j], dbias[d].
__global__ void __launch_bounds__(256)
conv_reduce_kernel(const float* __restrict__ part, int P, int W, int D, float* __restrict__ dw,
                   float* __restrict__ dbias) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const long long i = (long long)blockIdx.x * 32 + lane, n = (long long)(W + 1) * D;
  float s = 0.f;
  if (i < n)
    for (int p = row; p < P; p += 8) s += part[(long long)p * n + i];
  red[row][lane] = s;
  __syncthreads();
  if (row == 0 && i < n) {
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += red[r][lane];
    const int j = (int)(i / D), d = (int)(i % D);
    if (j < W)
      dw[(long long)d * W + j] = s;
    else if (dbias)
      dbias[d] = s;
  }
}

// ---------------------------------------------------------------- one token
//
// y of the new token from the state's W-1 inputs, and the state moved on by
// one in place.  A thread owns its channels of one sequence, so no other
// thread reads what it writes.
template <typename T, int V, int W, bool SILU>
__global__ void __launch_bounds__(128)
conv_step_kernel(const T* __restrict__ x, long long ldx, const float* __restrict__ w,
                 const float* __restrict__ bias, T* __restrict__ s, T* __restrict__ y, int D,
                 unsigned CG, unsigned total) {
  const unsigned id = blockIdx.x * 128 + threadIdx.x;
  if (id >= total) return;
  const long long b = id / CG;
  const int c = (int)(id - (unsigned)b * CG) * V;
  T* sb = s + b * (W - 1) * D + c;
  Row<T, V> rows[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].load(sb + (long long)j * D);
  rows[W - 1].load(x + b * ldx + c);
  constexpr int P = kPairs<V>;
  f32x2 tap[W][P], b0[P], win[W - 1][P], cur[P], p[P];
  load_taps<V, W>(w, bias, c, tap, b0);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j].get(win[j]);
  rows[W - 1].get(cur);
  taps_sum<V, W>(tap, b0, win, cur, p);
  if (SILU)
#pragma unroll
    for (int i = 0; i < P; ++i) p[i] = activate(p[i]);
  Row<T, V> o;
  o.set(p);
  o.store(y + b * D + c);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) rows[j + 1].store(sb + (long long)j * D);
}

// ---------------------------------------------------------------- host side

// Tokens that one thread walks.  Long walks read fewer rows twice and load
// their taps for more tokens; short prompts need the threads more.  32 tokens
// where that still gives every SM 1024 threads (8 x 4096 x 2048 bf16, with
// 256-thread blocks: 66 us with 32 and 64, 68 with 16), then 16, then 4.
static int fwd_walk(long long B, int T, int CG) {
  for (int L = 32; L > 4; L /= 2)
    if (B * ((T + L - 1) / L) * CG >= 148LL * 1024) return L;
  return 4;
}

// Tokens of one backward walk (a block runs kBY of them side by side): the
// longest that gives every SM the four blocks that it holds (4 x 8192 x 2048
// bf16: 103 us with 64, 112 with 32; 2 x 8192: 56 and 61), 16 where that gives
// two, and 8 for less.
static int bwd_walk(long long B, int T, int D, int V) {
  const long long cb = (D + kBX * V - 1) / (kBX * V);
  auto blocks = [&](int L) { return B * cb * ((T + L * kBY - 1) / (L * kBY)); };
  return blocks(64) >= 4 * 148 ? 64 : blocks(32) >= 4 * 148 ? 32 : blocks(16) >= 2 * 148 ? 16 : 8;
}

static long long bwd_parts(int B, int T, int D, int V) {
  const int L = bwd_walk(B, T, D, V);
  return (long long)B * ((T + kBY * L - 1) / (kBY * L));
}

// Sequences of one launch with this many threads each: kernels count their
// threads in 32 bits, and single channels of short prompts or tokens can be more
// (2^32 of them take 17 GB).  A sequence alone is not: D <= 2^30, and four walks
// of 32 tokens of that many channels do not fit the memory.
static int launch_batch(int B, long long threads) {
  const long long most = 0xffffff00LL / threads;
  return (int)(B < most ? B : most);
}

template <typename T, int V, int W>
static cudaError_t launch_fwd(const void* x, long long ldx, const float* w, const float* bias,
                              const void* s0, const int* lengths, void* y, void* sT, int B,
                              int Tn, int D, bool silu, cudaStream_t st) {
  const int CG = D / V, L = fwd_walk(B, Tn, CG), NB = (Tn + L - 1) / L;
  const int per = launch_batch(B, (long long)NB * CG);
  if (per < 1) return cudaErrorInvalidValue;
  auto k = silu ? conv_fwd_kernel<T, V, W, true> : conv_fwd_kernel<T, V, W, false>;
  for (int b = 0; b < B; b += per) {
    const long long rows = (long long)b * Tn, st_at = (long long)b * (W - 1) * D;
    const unsigned total = (unsigned)((long long)(B - b < per ? B - b : per) * NB * CG);
    k<<<(total - 1) / kFT + 1, kFT, 0, st>>>(
        (const T*)x + rows * ldx, ldx, w, bias, s0 ? (const T*)s0 + st_at : nullptr,
        lengths ? lengths + b : nullptr, (T*)y + rows * D, sT ? (T*)sT + st_at : nullptr, Tn, D,
        CG, NB, L, total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || B - b <= per) return e;
  }
  return cudaSuccess;
}

template <typename T, int V, int W>
static cudaError_t launch_bwd(const void* x, long long ldx, const float* w, const float* bias,
                              const void* s0, const int* lengths, const void* gy,
                              const void* gs, void* dx, float* dw, float* dbias, void* ds0,
                              int B, int Tn, int D, bool silu, float* part, cudaStream_t st) {
  const int CB = (D + kBX * V - 1) / (kBX * V), L = bwd_walk(B, Tn, D, V);
  const int NB = (Tn + kBY * L - 1) / (kBY * L);
  const long long blocks = (long long)CB * NB * B;
  if (blocks > 0x7fffffffLL || (long long)NB * B > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto k = silu ? conv_bwd_kernel<T, V, W, true> : conv_bwd_kernel<T, V, W, false>;
  k<<<(unsigned)blocks, dim3(kBX, kBY), 0, st>>>((const T*)x, ldx, w, bias, (const T*)s0,
                                                 lengths, (const T*)gy, (const T*)gs, (T*)dx,
                                                 (T*)ds0, part, Tn, D, CB, NB, L);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long n = (long long)(W + 1) * D;
  conv_reduce_kernel<<<(unsigned)((n + 31) / 32), 256, 0, st>>>(part, B * NB, W, D, dw, dbias);
  return cudaGetLastError();
}

template <typename T, int V, int W>
static cudaError_t launch_step(const void* x, long long ldx, const float* w, const float* bias,
                               void* s, void* y, int B, int D, bool silu, cudaStream_t st) {
  const int CG = D / V;
  const int per = launch_batch(B, CG);
  auto k = silu ? conv_step_kernel<T, V, W, true> : conv_step_kernel<T, V, W, false>;
  for (int b = 0; b < B; b += per) {
    const unsigned total = (unsigned)((long long)(B - b < per ? B - b : per) * CG);
    k<<<(total - 1) / 128 + 1, 128, 0, st>>>((const T*)x + b * ldx, ldx, w, bias,
                                             (T*)s + (long long)b * (W - 1) * D,
                                             (T*)y + (long long)b * D, D, CG, total);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || B - b <= per) return e;
  }
  return cudaSuccess;
}

// The checks that all three calls share.
static kla_status check(int B, int T, int D, int W, int dtype, long long ldx) {
  if (B < 1 || T < 0 || D < 1 || W < 1 || !dtype_ok(dtype)) return KLA_ERR_INVALID_ARG;
  if (ldx < D || !size_ok((long long)B * (T > W ? T : W), ldx)) return KLA_ERR_INVALID_ARG;
  if (T > kMaxTokens || D > kMaxTokens || W < 2 || W > 4) return KLA_ERR_UNSUPPORTED;
  return KLA_OK;
}

#define KLA_CONV_WIDTH(W, CALL)          \
  switch (W) {                           \
    case 2: { constexpr int KW = 2; CALL; } break; \
    case 3: { constexpr int KW = 3; CALL; } break; \
    default: { constexpr int KW = 4; CALL; } break; \
  }

}  // namespace conv
}  // namespace kla

using namespace kla;
using namespace kla::conv;

extern "C" {

kla_status kla_conv_fwd(const void* x, long long ldx, const float* w, const float* bias,
                        const void* s0, const int* lengths, void* y, void* sT, int B, int T,
                        int D, int W, int silu, int dtype, void* stream) {
  kla_status s = check(B, T, D, W, dtype, ldx);
  if (s != KLA_OK) return s;
  if (T > 0 && (!x || !w || !y)) return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {w, bias, s0, y, sT};
  if (misaligned(ptrs) || misplaced(lengths, 4) || misplaced(x, elem(dtype))) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long rows = (long long)B * T, ns = (long long)B * (W - 1) * D;
  const Span in[] = {span(x, rows, D, ldx, es), span(w, (long long)D * W, 4),
                     span(bias, bias ? D : 0, 4), span(s0, s0 ? ns : 0, es),
                     span(lengths, lengths ? B : 0, 4)};
  const Span out[] = {span(y, rows * D, es), span(sT, sT ? ns : 0, es)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    if (sT)
      e = s0 ? cudaMemcpyAsync(sT, s0, ns * es, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(sT, 0, ns * es, st);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
  }
#define RUN(TY, V) \
  KLA_CONV_WIDTH(W, (e = launch_fwd<TY, V, KW>(x, ldx, w, bias, s0, lengths, y, sT, B, T, D, \
                                              silu != 0, st)))
  if (dtype == KLA_BF16) {
    if (rows_aligned(x, D, ldx, 4, es)) { RUN(__nv_bfloat16, 4) } else { RUN(__nv_bfloat16, 1) }
  } else {
    if (rows_aligned(x, D, ldx, 4, es)) { RUN(float, 4) } else { RUN(float, 1) }
  }
#undef RUN
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_conv_bwd_workspace_size(int B, int T, int D, int W) {
  if (check(B, T, D, W, KLA_BF16, D) != KLA_OK) return 0;
  // the larger of the two walks' part counts, whatever the pitch turns out to be
  const long long a = bwd_parts(B, T, D, 4), b = bwd_parts(B, T, D, 1);
  return (size_t)(a > b ? a : b) * (W + 1) * D * sizeof(float);
}

kla_status kla_conv_bwd(const void* x, long long ldx, const float* w, const float* bias,
                        const void* s0, const int* lengths, const void* grad_y,
                        const void* grad_sT, void* grad_x, float* grad_w, float* grad_bias,
                        void* grad_s0, int B, int T, int D, int W, int silu, int dtype,
                        void* workspace, size_t ws_bytes, void* stream) {
  kla_status s = check(B, T, D, W, dtype, ldx);
  if (s != KLA_OK) return s;
  if (T > 0 && (!x || !grad_y || !grad_x)) return KLA_ERR_INVALID_ARG;
  if (!w || !grad_w) return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {w,      bias,   s0,        grad_y,  grad_sT,
                              grad_x, grad_w, grad_bias, grad_s0, workspace};
  if (misaligned(ptrs) || misplaced(lengths, 4) || misplaced(x, elem(dtype))) return KLA_ERR_INVALID_ARG;
  const size_t need = kla_conv_bwd_workspace_size(B, T, D, W);
  if (ws_bytes < need || (need && !workspace)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long rows = (long long)B * T, ns = (long long)B * (W - 1) * D;
  const Span in[] = {span(x, rows, D, ldx, es), span(w, (long long)D * W, 4),
                     span(bias, bias ? D : 0, 4), span(s0, s0 ? ns : 0, es),
                     span(lengths, lengths ? B : 0, 4), span(grad_y, rows * D, es),
                     span(grad_sT, grad_sT ? ns : 0, es)};
  const Span out[] = {span(grad_x, rows * D, es), span(grad_w, (long long)D * W, 4),
                      span(grad_bias, grad_bias ? D : 0, 4),
                      span(grad_s0, grad_s0 ? ns : 0, es), span(workspace, (long long)need, 1)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    e = cudaMemsetAsync(grad_w, 0, (size_t)D * W * 4, st);
    if (e == cudaSuccess && grad_bias) e = cudaMemsetAsync(grad_bias, 0, (size_t)D * 4, st);
    if (e == cudaSuccess && grad_s0)
      e = grad_sT ? cudaMemcpyAsync(grad_s0, grad_sT, ns * es, cudaMemcpyDeviceToDevice, st)
                  : cudaMemsetAsync(grad_s0, 0, ns * es, st);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
  }
#define RUN(TY, V)                                                                          \
  KLA_CONV_WIDTH(W, (e = launch_bwd<TY, V, KW>(x, ldx, w, bias, s0, lengths, grad_y, grad_sT, \
                                              grad_x, grad_w, grad_bias, grad_s0, B, T, D,   \
                                              silu != 0, (float*)workspace, st)))
  const int v = rows_aligned(x, D, ldx, 4, es) ? 4 : 1;
  if (dtype == KLA_BF16) {
    if (v == 4) { RUN(__nv_bfloat16, 4) } else { RUN(__nv_bfloat16, 1) }
  } else {
    if (v == 4) { RUN(float, 4) } else { RUN(float, 1) }
  }
#undef RUN
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_conv_step(const void* x, long long ldx, const float* w, const float* bias,
                         void* state, void* y, int B, int D, int W, int silu, int dtype,
                         void* stream) {
  kla_status s = check(B, 1, D, W, dtype, ldx);
  if (s != KLA_OK) return s;
  if (!x || !w || !state || !y) return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {w, bias, state, y};
  if (misaligned(ptrs) || misplaced(x, elem(dtype))) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const Span in[] = {span(x, B, D, ldx, es), span(w, (long long)D * W, 4),
                     span(bias, bias ? D : 0, 4)};
  const Span out[] = {span(state, (long long)B * (W - 1) * D, es),
                      span(y, (long long)B * D, es)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
#define RUN(TY, V)                                                                           \
  KLA_CONV_WIDTH(W, (e = launch_step<TY, V, KW>(x, ldx, w, bias, state, y, B, D, silu != 0, \
                                               st)))
  if (dtype == KLA_BF16) {
    if (rows_aligned(x, D, ldx, 4, es)) { RUN(__nv_bfloat16, 4) } else { RUN(__nv_bfloat16, 1) }
  } else {
    if (rows_aligned(x, D, ldx, 4, es)) { RUN(float, 4) } else { RUN(float, 1) }
  }
#undef RUN
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
