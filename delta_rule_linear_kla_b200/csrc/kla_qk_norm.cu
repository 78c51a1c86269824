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
// gives each 8 channels; a block takes a few tokens with all their heads, so
// that an angle's cosine and sine are formed once a token and shared by the
// heads.  Angles are formed and reduced to [-pi, pi] in fp64 (a position of
// 1e6 leaves 24-bit angles 0.06 off), their cosine and sine in fp32; norms
// and products are fp32, and only the results are rounded, once.
#include "kla_layer.cuh"

namespace kla {
namespace qk {

using namespace layer;

constexpr int kNT = 256;
constexpr int kTrig = 2048;  // angles a block holds

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

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]);
template <>
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    u[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
template <>
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// How the partner of a channel is reached: PAIR (2i, 2i+1) lies in the lane,
// LANE (i, i + rot/2) in a lane at a fixed distance (rot/2 a multiple of 8),
// SMEM through shared memory (any even rot).
enum Reach { NONE = 0, PAIR = 1, LANE = 2, SMEM = 3 };

// cos and sin of the block's tokens: s_cs[token][pair]
__device__ __forceinline__ void make_angles(const Args& p, long long tok0, int nt,
                                            float2* s_cs) {
  const int np = p.rot / 2;
  for (int i = threadIdx.x; i < nt * np; i += kNT) {
    const int tt = i / np, j = i % np;
    const long long tok = tok0 + tt, b = tok / p.T;
    const int t = (int)(tok - b * p.T);
    const int at = p.pos ? p.pos[b * p.pos_stride + t] : p.pos0 + t;
    const double ang = (double)at * (double)p.inv_freq[j];
    const double turns = rint(ang * 0.15915494309189535);  // 1 / 2 pi
    const float r = (float)fma(-turns, 6.283185307179586, ang);
    float s, c;
    sincosf(r, &s, &c);
    s_cs[i] = make_float2(c * p.scale, s * p.scale);
  }
}

// v (this lane's 8 channels from c) turned by the token's angles; SIGN -1
// turns back.  row: this row's staging of d floats (SMEM).
template <int REACH>
__device__ __forceinline__ void turn(float (&v)[8], const Args& p, int c, const float2* cs,
                                     float* row, float sign) {
  if constexpr (REACH == PAIR) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      if (c + e < p.rot) {
        const float2 t = cs[(c + e) >> 1];
        const float a = v[e], b = v[e + 1], s = sign * t.y;
        v[e] = a * t.x - b * s;
        v[e + 1] = fmaf(b, t.x, a * s);
      }
  } else if constexpr (REACH == LANE) {
    const int half = p.rot / 2;
    const bool lo = c < half, in = c < p.rot;
    const int dist = half / 8, lane = threadIdx.x & 31;
    const int from = in ? (lo ? lane + dist : lane - dist) : lane;
    const int base = lo ? c : c - half;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float o = __shfl_sync(0xffffffffu, v[e], from);
      if (in) {
        const float2 t = cs[base + e];
        const float s = lo ? -sign * t.y : sign * t.y;
        v[e] = fmaf(v[e], t.x, o * s);
      }
    }
  } else if constexpr (REACH == SMEM) {
    const int half = p.rot / 2;
    if (c < p.d)
#pragma unroll
      for (int e = 0; e < 8; ++e) row[c + e] = v[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = c + e;
      if (i < p.rot) {
        const bool lo = i < half;
        const float2 t = cs[lo ? i : i - half];
        const float o = row[lo ? i + half : i - half];
        v[e] = fmaf(v[e], t.x, o * (lo ? -sign * t.y : sign * t.y));
      }
    }
    __syncwarp();
  }
}

// LPR lanes a row.  BWD: q and k with their gradients to dq, dk, and the
// weights' parts.
template <typename T, int LPR, int REACH, bool BWD>
__global__ void __launch_bounds__(kNT)
qk_kernel(Args p, long long ntiles) {
  constexpr int RPB = kNT / LPR;  // rows in flight
  __shared__ float2 s_cs[REACH == NONE ? 1 : kTrig];
  __shared__ float s_row[REACH == SMEM ? RPB : 1][REACH == SMEM ? LPR * 8 : 1];
  const int lr = threadIdx.x % LPR, rr = threadIdx.x / LPR, c = lr * 8;
  const bool in = c < p.d;
  const int H = p.Hq + p.Hk;
  const float inv_m = p.norm == 2 ? 1.f / (float)p.d : 1.f;
  float wq[8], wk[8], aq[8] = {}, ak[8] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    wq[e] = in && p.wq ? p.wq[c + e] : 1.f;
    wk[e] = in && p.wk ? p.wk[c + e] : 1.f;
  }
  for (long long tile = blockIdx.x; tile < ntiles; tile += gridDim.x) {
    const long long tok0 = tile * p.TB;
    const int nt = (int)min((long long)p.TB, p.tokens - tok0);
    if constexpr (REACH != NONE) {
      if (tile != blockIdx.x) __syncthreads();  // the last tile's angles are read
      make_angles(p, tok0, nt, s_cs);
      __syncthreads();
    }
    const int nrow = nt * H;
    // whole warps run every pass: lanes without a row take part in shuffles
    for (int r0 = 0; r0 < nrow; r0 += RPB) {
      const int r = r0 + rr;
      const bool live = in && r < nrow;
      const int tt = r < nrow ? r / H : 0, hh = r < nrow ? r - tt * H : 0;
      const long long tok = tok0 + tt;
      const bool isq = hh < p.Hq;
      const T* src = isq ? (const T*)p.q + tok * p.ldq + hh * p.d
                         : (const T*)p.k + tok * p.ldk + (hh - p.Hq) * p.d;
      const long long at = isq ? (tok * p.Hq + hh) * p.d : (tok * p.Hk + hh - p.Hq) * p.d;
      float x[8] = {}, g[8] = {};
      if (live) {
        load8(src + c, x);
        if (BWD) load8((isq ? (const T*)p.gq : (const T*)p.gk) + at + c, g);
      }
      float rs = 1.f;
      if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        rs = 1.f / sqrtf(fmaf(ss, inv_m, p.eps));
      }
      const float2* cs = s_cs + (REACH == NONE ? 0 : tt * (p.rot / 2));
      float* row = s_row[REACH == SMEM ? rr : 0];
      if constexpr (!BWD) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= rs * (isq ? wq[e] : wk[e]);
        turn<REACH>(x, p, c, cs, row, 1.f);
        if (live) store8((isq ? (T*)p.oq : (T*)p.ok) + at + c, x);
      } else {
        turn<REACH>(g, p, c, cs, row, -1.f);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] *= rs;
          if (live) {
            if (isq)
              aq[e] = fmaf(g[e], x[e], aq[e]);
            else
              ak[e] = fmaf(g[e], x[e], ak[e]);
          }
          g[e] *= isq ? wq[e] : wk[e];
          dot = fmaf(g[e], x[e], dot);
        }
        if (p.norm) {
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
          dot *= inv_m;
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] = rs * fmaf(-x[e], dot, g[e]);
        }
        if (live) store8((isq ? (T*)p.oq : (T*)p.ok) + at + c, g);
      }
    }
  }
  if constexpr (BWD) {
    if (!p.part) return;
    // over the block's rows in order, 8 KB at a time
    __shared__ float s_sum[RPB][LPR * 8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) s_sum[rr][c + e] = w ? ak[e] : aq[e];
      __syncthreads();
      for (int i = threadIdx.x; i < p.d; i += kNT) {
        float s = 0.f;
#pragma unroll 8
        for (int r = 0; r < RPB; ++r) s += s_sum[r][i];
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

// Tokens of a block: four passes of its rows, within its store of angles.
static int tokens_per_block(int H, int d, int rot, long long tokens) {
  const int rows = 4 * (kNT / lanes(d));
  long long tb = rows / H;
  const long long most = rot ? kTrig / (rot / 2) : tb;
  if (tb > most) tb = most;
  // few tokens: one each, so that every SM has work
  if (tokens < 148 * tb) tb = (tokens + 147) / 148;
  return (int)(tb < 1 ? 1 : tb);
}

static long long blocks_of(long long tokens, int TB, bool bwd) {
  const long long n = (tokens + TB - 1) / TB;
  const long long most = bwd ? 148 * 4 : 0x7fffffffLL;
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
  a.TB = tokens_per_block(a.Hq + a.Hk, a.d, a.rot, a.tokens);
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
  if (T > kMaxTokens || d % 8 != 0 || d > 256 || Hq > (1 << 20) || Hk > (1 << 20))
    return KLA_ERR_UNSUPPORTED;
  // rows are read 8 channels at a time
  const int v = 16 / elem(dtype);
  if (ldq % v != 0 || ldk % v != 0) return KLA_ERR_UNSUPPORTED;
  return KLA_OK;
}

static long long parts_of(long long tokens, int H, int d, int rot) {
  return tokens == 0 ? 0 : blocks_of(tokens, tokens_per_block(H, d, rot, tokens), true);
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
  if ((Hq && (!q || !oq)) || (Hk && (!k || !ok)) || (rot && !inv_freq) ||
      (positions && pos_stride != 0 && pos_stride < T))
    return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {q, k, wq, wk, positions, inv_freq, oq, ok};
  if (misaligned(ptrs)) return KLA_ERR_INVALID_ARG;
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
  return (size_t)parts_of((long long)B * T, Hq + Hk, d, rot) * 2 * d * sizeof(float);
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
  const bool weights = grad_wq || grad_wk;
  const void* const ptrs[] = {q, k, wq, wk, positions, inv_freq, grad_oq, grad_ok,
                              grad_q, grad_k, grad_wq, grad_wk, workspace};
  if (misaligned(ptrs)) return KLA_ERR_INVALID_ARG;
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
    const int P = (int)parts_of(rows, Hq + Hk, d, rot);
    qk_reduce_kernel<<<(unsigned)((2 * d + 31) / 32), 1024, 0, st>>>(a.part, P, d, grad_wq,
                                                                     grad_wk);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
