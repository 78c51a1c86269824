// Norm of every query and key head and its rotation by position, in one pass,
// with the backward pass.
//
//   x^ = x r,   r = (sum x^2 + eps)^{-1/2}          (L2)
//               r = (sum x^2 / d + eps)^{-1/2}      (RMS), or r = 1 (no norm)
//   v = w x^,   out = scale R(pos) v on the first `rot` channels, v on the rest
//
// R turns channel pair i by the angle pos * inv_freq[i]; pairs are (i, i +
// rot/2) or (2i, 2i+1).  `scale` multiplies cosine and sine.  Backward, with
// g = scale R(-pos) grad:  dw = sum g x^,  dx = r (w g - x^ <w g, x^> / m), m = 1
// (L2) or d (RMS).
//
// Bound by HBM: q and k read and written once (backward: gradients too).  A
// row (one head of one token) lies on the smallest power of two of lanes that
// gives each 8 channels; a block takes a few tokens with all their heads.  A
// thread stays with one token and walks through some of its heads, so that
// cosines and sines are formed once a token and held in registers, and loads
// the rows of several heads before it needs the first.  Angles are formed and reduced to [-pi, pi] in fp64 (a position of
// 1e6 leaves 24-bit angles 0.06 off), their cosine and sine in fp32; norms
// and products are fp32, and only the results are rounded, once.
// Measured: 8 x 4096 tokens of 8 + 8 heads of 128, half of each turned, bf16:
// 50 us, 5.4 TB/s of the 6.45 that a copy reaches.  Backward, 4 x 8192 tokens of
// 32 + 8 heads of 64 with weights: 103 us, 4.9 TB/s.
#include "kla_layer.cuh"

namespace kla {
namespace qk {

using namespace layer;

constexpr int kNT = 256;
constexpr int kTrig = 1024;  // angles of a block's tokens at most: kNT / LPR tokens, 4 LPR pairs

struct Args {
  const void *q, *k, *gq, *gk;
  long long ldq, ldk;
  const float *wq, *wk, *inv_freq;
  const int* pos;
  long long pos_stride;  // 0: positions are shared by the sequences
  int pos0;
  void *oq, *ok;
  float* part;  // [blocks][2][d]
  long long tokens;
  int T, Hq, Hk, d, rot, TB, norm, interleaved;
  float eps, scale;
};

// Eight channels as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<__nv_bfloat16> {
  uint4 r;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    r = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
    const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f[i] = pack2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
  }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(f32x2 (&f)[4]) const {
    f[0] = pack2(a.x, a.y); f[1] = pack2(a.z, a.w);
    f[2] = pack2(b.x, b.y); f[3] = pack2(b.z, b.w);
  }
};
__device__ __forceinline__ void store8(__nv_bfloat16* p, const f32x2 (&f)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = unpack2(f[i]);
    __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store8(float* p, const f32x2 (&f)[4]) {
  reinterpret_cast<float4*>(p)[0] = flat(Quad{f[0], f[1]});
  reinterpret_cast<float4*>(p)[1] = flat(Quad{f[2], f[3]});
}

// How the partner of a channel is reached: PAIR (2i, 2i+1) lies in the lane,
// LANE (i, i + rot/2) in a lane at a fixed distance (rot/2 a multiple of 8),
// SMEM through shared memory (any even rot).
enum Reach { NONE = 0, PAIR = 1, LANE = 2, SMEM = 3 };

// Cosines and sines of the block's nt tokens, [token][pair], times scale.  fp32
// rows get them within 2.6 units of 2^-24 (the angle's rounding, as a multiple
// of pi in [-1, 1], and 1 ulp); bf16 rows, whose results are rounded by up to 2^-8,
// within 2^-21 by the fast form.
template <typename T>
__device__ __forceinline__ void make_angles(const Args& p, long long tok0, int nt, float* s_cos,
                                            float* s_sin) {
  const unsigned np = p.rot / 2;
  const long long b0 = tok0 / p.T;
  const unsigned first = (unsigned)(tok0 - b0 * p.T);
  for (unsigned i = threadIdx.x; i < nt * np; i += kNT) {
    const unsigned tt = i / np, j = i - tt * np;
    // first + tt < 2^30 + kNT
    const unsigned more = (first + tt) / (unsigned)p.T, t = first + tt - more * (unsigned)p.T;
    const int at = p.pos ? p.pos[(b0 + more) * p.pos_stride + t] : p.pos0 + (int)t;
    const double ang = (double)at * (double)p.inv_freq[j];
    const double turns = rint(ang * 0.15915494309189535);  // 1 / 2 pi
    const double r = fma(-turns, 6.283185307179586, ang);  // in [-pi, pi]
    float s, c;
    if constexpr (sizeof(T) == 4)
      sincospif((float)(r * 0.3183098861837907), &s, &c);
    else
      __sincosf((float)r, &s, &c);
    s_cos[i] = c * p.scale;
    s_sin[i] = s * p.scale;
  }
}

// This lane's part of its token's angles, for pairs of neighbouring channels:
// out = v co + o si, o the partners.  Channels that are not turned have (1, 0)
// and partner 0: an infinity beside them, or their own, stays where it is.
template <int REACH>
struct Turn {
  f32x2 co[4], si[4];
  int from;  // LANE: the partner's lane

  __device__ __forceinline__ void load(const Args& p, int c, const float* cosv,
                                       const float* sinv) {
    const int half = p.rot / 2, lane = threadIdx.x & 31;
    from = lane;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      co[e] = both(1.f);
      si[e] = both(0.f);
    }
    if constexpr (REACH == PAIR) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + 2 * e < p.rot) {
          const float s = sinv[c / 2 + e];
          co[e] = both(cosv[c / 2 + e]);
          si[e] = pack2(-s, s);
        }
    } else if constexpr (REACH == LANE) {  // half a multiple of 8: all 8 on one side
      if (c < p.rot) {
        const bool lo = c < half;
        from = lo ? lane + half / 8 : lane - half / 8;
        const float4* pc = reinterpret_cast<const float4*>(cosv + (lo ? c : c - half));
        const float4* ps = reinterpret_cast<const float4*>(sinv + (lo ? c : c - half));
        const f32x2 sign = both(lo ? -1.f : 1.f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Quad q = quad(pc[j]), r = quad(ps[j]);
          co[2 * j] = q.a; co[2 * j + 1] = q.b;
          si[2 * j] = mul2(r.a, sign); si[2 * j + 1] = mul2(r.b, sign);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float q[2] = {1.f, 1.f}, r[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = c + 2 * e + k;
          if (i < p.rot) {
            q[k] = cosv[i < half ? i : i - half];
            r[k] = i < half ? -sinv[i] : sinv[i - half];
          }
        }
        co[e] = pack2(q[0], q[1]);
        si[e] = pack2(r[0], r[1]);
      }
    }
  }

  // v turned; the backward pass turns back with si's sign flipped beforehand.
  // row: d floats of staging (SMEM)
  __device__ __forceinline__ void apply(f32x2 (&v)[4], const Args& p, int c, float* row) const {
    f32x2 o[4];
    if constexpr (REACH == PAIR) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = unpack2(v[e]);
        o[e] = c + 2 * e < p.rot ? pack2(a.y, a.x) : both(0.f);
      }
    } else if constexpr (REACH == LANE) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = unpack2(v[e]);
        o[e] = pack2(__shfl_sync(0xffffffffu, a.x, from), __shfl_sync(0xffffffffu, a.y, from));
        if (c >= p.rot) o[e] = both(0.f);
      }
    } else {
      const int half = p.rot / 2;
      if (c < p.d)
#pragma unroll
        for (int e = 0; e < 4; ++e) *reinterpret_cast<f32x2*>(row + c + 2 * e) = v[e];
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float q[2] = {0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int i = c + 2 * e + k;
          if (i < p.rot) q[k] = row[i < half ? i + half : i - half];
        }
        o[e] = pack2(q[0], q[1]);
      }
      __syncwarp();
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fma2(v[e], co[e], mul2(o[e], si[e]));
  }
  __device__ __forceinline__ void reverse() {
#pragma unroll
    for (int e = 0; e < 4; ++e) si[e] = mul2(si[e], both(-1.f));
  }
};
template <>
struct Turn<NONE> {
  __device__ __forceinline__ void load(const Args&, int, const float*, const float*) {}
  __device__ __forceinline__ void apply(f32x2 (&)[4], const Args&, int, float*) const {}
  __device__ __forceinline__ void reverse() {}
};

// sum of a lane's eight products, then of the row's lanes
template <int LPR>
__device__ __forceinline__ float row_dot(const f32x2 (&a)[4], const f32x2 (&b)[4]) {
  const float2 s = unpack2(fma2(a[3], b[3], fma2(a[2], b[2], fma2(a[1], b[1], mul2(a[0], b[0])))));
  float r = s.x + s.y;
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// LPR lanes a row; a block has kNT / LPR row places, TB tokens of them with
// the same number of places each.  BWD: q and k with their gradients to dq,
// dk, and the weights' parts.
template <typename T, int LPR, int REACH, bool BWD>
__global__ void __launch_bounds__(kNT, BWD ? 2 : 4)
qk_kernel(Args p, long long ntiles) {
  constexpr int RPB = kNT / LPR;
  constexpr int U = BWD || sizeof(T) == 4 ? 2 : 4;  // rows loaded ahead
  __shared__ __align__(16) float s_cos[REACH == NONE ? 1 : kTrig];
  __shared__ __align__(16) float s_sin[REACH == NONE ? 1 : kTrig];
  __shared__ __align__(16) float s_row[REACH == SMEM ? RPB : 1][REACH == SMEM ? LPR * 8 : 1];
  const int lr = threadIdx.x % LPR, rr = threadIdx.x / LPR, c = lr * 8;
  const int places = RPB / p.TB;  // of a token
  const int tt = rr / places, h0 = rr - tt * places;
  const int H = p.Hq + p.Hk;
  const float inv_m = p.norm == 2 ? 1.f / (float)p.d : 1.f;
  float* const row = s_row[REACH == SMEM ? rr : 0];
  f32x2 aq[4], ak[4];  // BWD: sums of the weights' gradients
#pragma unroll
  for (int e = 0; e < 4; ++e) aq[e] = ak[e] = both(0.f);
  __shared__ __align__(16) float s_w[2][LPR * 8];
  const bool weighted = p.wq || p.wk;
  if (weighted) {
    for (int i = threadIdx.x; i < LPR * 8; i += kNT) {
      s_w[0][i] = i < p.d && p.wq ? p.wq[i] : 1.f;
      s_w[1][i] = i < p.d && p.wk ? p.wk[i] : 1.f;
    }
    __syncthreads();
  }
  auto times_w = [&](f32x2 (&v)[4], bool isq) {
    if (!weighted) return;
    const float4* w = reinterpret_cast<const float4*>(&s_w[isq ? 0 : 1][c]);
    const Quad a = quad(w[0]), b = quad(w[1]);
    v[0] = mul2(v[0], a.a); v[1] = mul2(v[1], a.b);
    v[2] = mul2(v[2], b.a); v[3] = mul2(v[3], b.b);
  };
  // a token's rows, in bytes from each array's start: head h of q, or head h -
  // Hq of k, lies h * d elements on (k's starts are set back by Hq heads)
  constexpr long long es = sizeof(T);
  const long long back = (long long)p.Hq * p.d;
  struct Where {
    long long q_in, k_in, q_out, k_out;
    bool mine;
  };
  auto where = [&](long long tile) {
    const long long tok = tile * p.TB + tt;
    Where w;
    w.q_in = (tok * p.ldq + c) * es;
    w.k_in = (tok * p.ldk + c - back) * es;
    w.q_out = (tok * p.Hq * p.d + c) * es;
    w.k_out = (tok * p.Hk * p.d + c - back) * es;
    w.mine = c < p.d && tile < ntiles && tok < p.tokens;
    return w;
  };
  auto at = [&](const void* q, const void* k, long long qo, long long ko, int h) {
    const char* a = h < p.Hq ? (const char*)q + qo : (const char*)k + ko;
    return (T*)(a + (unsigned)(h * p.d * (int)es));  // below 2^31: h < 2^20, d <= 256
  };
  Raw8<T> xn[U], gn[BWD ? U : 1];  // the rows to come
  auto load = [&](const Where& w, int hb) {  // heads hb + h0, one place apart
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int hh = hb + i * places + h0;
      xn[i].zero();
      if (BWD) gn[i].zero();
      if (w.mine && hh < H) {
        xn[i].load(at(p.q, p.k, w.q_in, w.k_in, hh));
        if (BWD) gn[i].load(at(p.gq, p.gk, w.q_out, w.k_out, hh));
      }
    }
  };
  Where w = where(blockIdx.x);
  load(w, 0);
  for (long long tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {  // forward: once
    const long long tok0 = tile * p.TB;
    const int nt = (int)min((long long)p.TB, p.tokens - tok0);
    Where wn = w;
    if constexpr (BWD) wn = where(tile + gridDim.x);
    Turn<REACH> turn;
    if constexpr (REACH != NONE) {
      if (tile != blockIdx.x) __syncthreads();  // the last tile's angles are read
      make_angles<T>(p, tok0, nt, s_cos, s_sin);
      __syncthreads();
      const int mine_at = tt < nt ? tt * (p.rot / 2) : 0;
      turn.load(p, c, s_cos + mine_at, s_sin + mine_at);
      if (BWD) turn.reverse();
    }
    // every thread makes as many passes: all lanes take part in the exchanges
    for (int hb = 0; hb < H; hb += U * places) {
      // forward: four blocks an SM cover the loads; backward: two, so the rows
      // of the next pass (or tile) are on their way during this one
      if (!BWD && hb > 0) load(w, hb);
      Raw8<T> x[U], g[BWD ? U : 1];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = xn[i];
        if (BWD) g[i] = gn[i];
      }
      if (BWD) {
        if (hb + U * places < H)
          load(w, hb + U * places);
        else
          load(wn, 0);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (hb + i * places >= H) break;  // the same for all threads
        const int hh = hb + i * places + h0;
        const bool live = w.mine && hh < H, isq = hh < p.Hq;
        f32x2 v[4];
        float r = 1.f;
        x[i].get(v);
        if (p.norm) {
          // (not the flushing form: without an eps the sum may be subnormal)
          r = rsqrtf(fmaf(row_dot<LPR>(v, v), inv_m, p.eps));
          // a place without a row holds zeros: without an eps they would give
          // 0 / 0 to the weights' sums
          if (BWD && !live) r = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = mul2(v[e], both(r));
        }
        if constexpr (!BWD) {
          times_w(v, isq);
          turn.apply(v, p, c, row);
          if (live) store8(at(p.oq, p.ok, w.q_out, w.k_out, hh), v);
        } else {
          f32x2 d[4];
          g[i].get(d);
          turn.apply(d, p, c, row);
          if (isq)
#pragma unroll
            for (int e = 0; e < 4; ++e) aq[e] = fma2(d[e], v[e], aq[e]);
          else
#pragma unroll
            for (int e = 0; e < 4; ++e) ak[e] = fma2(d[e], v[e], ak[e]);
          times_w(d, isq);
          if (p.norm) {
            const f32x2 dot = both(-inv_m * row_dot<LPR>(d, v));
#pragma unroll
            for (int e = 0; e < 4; ++e) d[e] = mul2(both(r), fma2(v[e], dot, d[e]));
          }
          if (live) store8(at(p.oq, p.ok, w.q_out, w.k_out, hh), d);
        }
      }
    }
    if (BWD) w = wn;
  }
  if constexpr (BWD) {
    if (!p.part) return;
    // over the block's rows in order, 8 KB at a time
    __shared__ __align__(16) float s_sum[RPB][LPR * 8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x2*>(&s_sum[rr][c + 2 * e]) = w ? ak[e] : aq[e];
      __syncthreads();
      for (int i = threadIdx.x; i < p.d; i += kNT) {
        float s = 0.f;
#pragma unroll 8
        for (int j = 0; j < RPB; ++j) s += s_sum[j][i];
        p.part[((long long)blockIdx.x * 2 + w) * p.d + i] = s;
      }
    }
  }
}

// dwq, dwk: the blocks' parts [P][2][d] in order.
__global__ void __launch_bounds__(1024)
qk_reduce_kernel(const float* __restrict__ part, int P, int d, float* __restrict__ dwq,
                 float* __restrict__ dwk) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int i = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (i < 2 * d)
    for (int p = row; p < P; p += 32) s += part[(long long)p * 2 * d + i];
  red[row][lane] = s;
  __syncthreads();
  if (row == 0 && i < 2 * d) {
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += red[r][lane];
    if (i < d) {
      if (dwq) dwq[i] = s;
    } else if (dwk) {
      dwk[i - d] = s;
    }
  }
}

// ---------------------------------------------------------------- host side

static int lanes(int d) {
  int l = 4;
  while (l * 8 < d) l *= 2;
  return l;
}

// Tokens of a block, a power of two.  A thread walks at least 16 heads (or all)
// of its token, so that its angles serve many rows (8 x 4096 tokens of 8 + 8
// heads of 128: 48 us with all 16 heads a thread, 55 with 8, 81 with 4); while
// the blocks would not give every SM two, up to all heads lie side by side.
static int tokens_per_block(int H, int d, long long tokens) {
  const int places = kNT / lanes(d);
  int side = 1;
  while (side * 32 <= H && side < places) side *= 2;
  while (side < H && side < places && tokens < 2LL * 148 * (places / side)) side *= 2;
  return places / side;
}

// The backward pass keeps its sums of the weights' gradients over many tiles:
// two blocks an SM (4 x 8192 tokens of 32 + 8 heads of 64: 102 us, 107 with
// four), as many as are resident.
static long long blocks_of(long long tokens, int TB, bool bwd) {
  const long long n = (tokens + TB - 1) / TB;
  const long long most = bwd ? 148 * 2 : 0x7fffffffLL;
  return n < most ? n : most;
}

template <typename T, int LPR, bool BWD>
static void launch_reach(const Args& a, int reach, unsigned grid, long long ntiles,
                         cudaStream_t st) {
  switch (reach) {
    case NONE: qk_kernel<T, LPR, NONE, BWD><<<grid, kNT, 0, st>>>(a, ntiles); break;
    case PAIR: qk_kernel<T, LPR, PAIR, BWD><<<grid, kNT, 0, st>>>(a, ntiles); break;
    case LANE: qk_kernel<T, LPR, LANE, BWD><<<grid, kNT, 0, st>>>(a, ntiles); break;
    default: qk_kernel<T, LPR, SMEM, BWD><<<grid, kNT, 0, st>>>(a, ntiles); break;
  }
}

template <typename T, bool BWD>
static cudaError_t launch(Args a, cudaStream_t st) {
  a.TB = tokens_per_block(a.Hq + a.Hk, a.d, a.tokens);
  const long long ntiles = (a.tokens + a.TB - 1) / a.TB;
  const unsigned grid = (unsigned)blocks_of(a.tokens, a.TB, BWD);
  const int reach = a.rot == 0 ? NONE : a.interleaved ? PAIR : a.rot % 16 == 0 ? LANE : SMEM;
  switch (lanes(a.d)) {
    case 4: launch_reach<T, 4, BWD>(a, reach, grid, ntiles, st); break;
    case 8: launch_reach<T, 8, BWD>(a, reach, grid, ntiles, st); break;
    case 16: launch_reach<T, 16, BWD>(a, reach, grid, ntiles, st); break;
    default: launch_reach<T, 32, BWD>(a, reach, grid, ntiles, st); break;
  }
  return cudaGetLastError();
}

static kla_status check(int B, int T, int Hq, int Hk, int d, int rot, int norm, float eps,
                        float scale, long long ldq, long long ldk, int dtype) {
  if (B < 1 || T < 0 || Hq < 0 || Hk < 0 || Hq + (long long)Hk < 1 || d < 1 || !dtype_ok(dtype))
    return KLA_ERR_INVALID_ARG;
  if (norm < 0 || norm > 2 || !(eps >= 0.f) || !(scale - scale == 0.f))
    return KLA_ERR_INVALID_ARG;
  if (rot < 0 || rot > d || rot % 2 != 0) return KLA_ERR_INVALID_ARG;
  if ((long long)Hq * d > ldq || (long long)Hk * d > ldk) return KLA_ERR_INVALID_ARG;
  const long long rows = (long long)B * T;
  if (!size_ok(rows, ldq) || !size_ok(rows, ldk)) return KLA_ERR_INVALID_ARG;
  if (T > kMaxTokens || d % 8 != 0 || d > 256 || Hq > (1 << 19) || Hk > (1 << 19))
    return KLA_ERR_UNSUPPORTED;
  // rows are read 8 channels at a time
  const int v = 16 / elem(dtype);
  if (ldq % v != 0 || ldk % v != 0) return KLA_ERR_UNSUPPORTED;
  return KLA_OK;
}

// Read one by one, these need only their own alignment.
static bool scalars_misplaced(const float* wq, const float* wk, const int* pos,
                              const float* inv_freq) {
  return misplaced(wq, 4) || misplaced(wk, 4) || misplaced(pos, 4) || misplaced(inv_freq, 4);
}

static long long parts_of(long long tokens, int H, int d) {
  return tokens == 0 ? 0 : blocks_of(tokens, tokens_per_block(H, d, tokens), true);
}

}  // namespace qk
}  // namespace kla

using namespace kla;
using namespace kla::qk;

extern "C" {

kla_status kla_qk_norm_fwd(const void* q, const void* k, long long ldq, long long ldk,
                           const float* wq, const float* wk, const int* positions,
                           long long pos_stride, int pos0, const float* inv_freq, int rot,
                           int interleaved, float scale, int norm, float eps, void* oq,
                           void* ok, int B, int T, int Hq, int Hk, int d, int dtype,
                           void* stream) {
  kla_status s = check(B, T, Hq, Hk, d, rot, norm, eps, scale, ldq, ldk, dtype);
  if (s != KLA_OK) return s;
  if (T == 0) return KLA_OK;
  if (!positions && (long long)pos0 + T - 1 > 0x7fffffffLL) return KLA_ERR_INVALID_ARG;
  if ((Hq && (!q || !oq)) || (Hk && (!k || !ok)) || (rot && !inv_freq) ||
      (positions && pos_stride != 0 && pos_stride < T))
    return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {q, k, oq, ok};
  if (misaligned(ptrs) || scalars_misplaced(wq, wk, positions, inv_freq)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long rows = (long long)B * T, nq = (long long)Hq * d, nk = (long long)Hk * d;
  const Span in[] = {span(q, rows, nq, ldq, es), span(k, rows, nk, ldk, es),
                     span(wq, wq ? d : 0, 4), span(wk, wk ? d : 0, 4),
                     span(positions, positions ? B : 0, T, pos_stride, 4),
                     span(inv_freq, rot / 2, 4)};
  const Span out[] = {span(oq, rows * nq, es), span(ok, rows * nk, es)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  Args a = {};
  a.q = q; a.k = k; a.ldq = ldq; a.ldk = ldk; a.wq = wq; a.wk = wk; a.inv_freq = inv_freq;
  a.pos = positions; a.pos_stride = pos_stride; a.pos0 = pos0; a.oq = oq; a.ok = ok;
  a.tokens = rows; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot; a.norm = norm;
  a.interleaved = interleaved != 0; a.eps = eps; a.scale = scale;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = dtype == KLA_BF16 ? launch<__nv_bfloat16, false>(a, st)
                                          : launch<float, false>(a, st);
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_qk_norm_bwd_workspace_size(int B, int T, int Hq, int Hk, int d, int rot) {
  if (check(B, T, Hq, Hk, d, rot, 0, 0.f, 1.f, (long long)Hq * d, (long long)Hk * d, KLA_BF16) !=
      KLA_OK)
    return 0;
  return (size_t)parts_of((long long)B * T, Hq + Hk, d) * 2 * d * sizeof(float);
}

kla_status kla_qk_norm_bwd(const void* q, const void* k, long long ldq, long long ldk,
                           const float* wq, const float* wk, const int* positions,
                           long long pos_stride, int pos0, const float* inv_freq, int rot,
                           int interleaved, float scale, int norm, float eps,
                           const void* grad_oq, const void* grad_ok, void* grad_q,
                           void* grad_k, float* grad_wq, float* grad_wk, int B, int T, int Hq,
                           int Hk, int d, int dtype, void* workspace, size_t ws_bytes,
                           void* stream) {
  kla_status s = check(B, T, Hq, Hk, d, rot, norm, eps, scale, ldq, ldk, dtype);
  if (s != KLA_OK) return s;
  if (!positions && (long long)pos0 + T - 1 > 0x7fffffffLL) return KLA_ERR_INVALID_ARG;
  const bool weights = grad_wq || grad_wk;
  const void* const ptrs[] = {q,      k,      grad_oq, grad_ok,  grad_q,
                              grad_k, grad_wq, grad_wk, workspace};
  if (misaligned(ptrs) || scalars_misplaced(wq, wk, positions, inv_freq)) return KLA_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  const size_t need = weights ? kla_qk_norm_bwd_workspace_size(B, T, Hq, Hk, d, rot) : 0;
  if (ws_bytes < need || (need && !workspace)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long rows = (long long)B * T, nq = (long long)Hq * d, nk = (long long)Hk * d;
  if (T > 0 && ((Hq && (!q || !grad_oq || !grad_q)) || (Hk && (!k || !grad_ok || !grad_k)) ||
                (rot && !inv_freq) || (positions && pos_stride != 0 && pos_stride < T)))
    return KLA_ERR_INVALID_ARG;
  const Span in[] = {span(q, rows, nq, ldq, es), span(k, rows, nk, ldk, es),
                     span(wq, wq ? d : 0, 4), span(wk, wk ? d : 0, 4),
                     span(positions, positions ? B : 0, T, pos_stride, 4),
                     span(inv_freq, rot / 2, 4), span(grad_oq, rows * nq, es),
                     span(grad_ok, rows * nk, es)};
  const Span out[] = {span(grad_q, rows * nq, es), span(grad_k, rows * nk, es),
                      span(grad_wq, grad_wq ? d : 0, 4), span(grad_wk, grad_wk ? d : 0, 4),
                      span(workspace, (long long)need, 1)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  if (T == 0) {
    if (grad_wq) e = cudaMemsetAsync(grad_wq, 0, (size_t)d * 4, st);
    if (e == cudaSuccess && grad_wk) e = cudaMemsetAsync(grad_wk, 0, (size_t)d * 4, st);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
  }
  Args a = {};
  a.q = q; a.k = k; a.gq = grad_oq; a.gk = grad_ok; a.ldq = ldq; a.ldk = ldk;
  a.wq = wq; a.wk = wk; a.inv_freq = inv_freq;
  a.pos = positions; a.pos_stride = pos_stride; a.pos0 = pos0; a.oq = grad_q; a.ok = grad_k;
  a.part = weights ? (float*)workspace : nullptr;
  a.tokens = rows; a.T = T; a.Hq = Hq; a.Hk = Hk; a.d = d; a.rot = rot; a.norm = norm;
  a.interleaved = interleaved != 0; a.eps = eps; a.scale = scale;
  e = dtype == KLA_BF16 ? launch<__nv_bfloat16, true>(a, st) : launch<float, true>(a, st);
  if (e == cudaSuccess && weights) {
    const int P = (int)parts_of(rows, Hq + Hk, d);
    qk_reduce_kernel<<<(unsigned)((2 * d + 31) / 32), 1024, 0, st>>>(a.part, P, d, grad_wq,
                                                                     grad_wk);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
