// Selective state space scan: a diagonal linear recurrence with step sizes,
// inputs and outputs that depend on the token, for prompts, their backward
// pass and single tokens.
//
//   dt'[t][d] = softplus(dt[t][d] + dt_bias[d])            (or dt + dt_bias)
//   h[d][n]  <- e^{dt' A[d][n]} h[d][n] + dt' u[t][d] B[t][g][n]
//   y[t][d]   = (sum_n C[t][g][n] h[d][n] + D[d] u[t][d]) silu(z[t][d])
//
// with channel d in group g = d / (D/G).  States and sums are fp32; only y
// (and the gradients of the activations) are rounded, once, to their type.
// Decays are formed as 2^{dt' (A log2 e)}.
//
// What bounds it: one exponential a state element and token.  The special
// function unit gives 16 a clock and SM, so N = 16 states take a clock of an
// SM per channel and token, against 8 bytes (u, dt, z, y in bf16): about
// three times what HBM needs.
//
// Split: a thread holds 4 states of CPT channels, the N/4 threads of a channel
// lie side by side in a warp, and a block's channels walk the tokens in tiles.
// Half of the block's warps run the recurrence; the other half prepare the
// next tile (softplus, dt' u, B and C to fp32) and finish the previous one
// (skip, gate, store), so the two kinds of work overlap.  With few channels
// the sequence is cut into segments: their end states from zero starts in
// parallel (MODE LOCAL), a short chain over segments, then all of them again
// from their true starts.
#include "kla_layer.cuh"

namespace kla {
namespace ssm {

using namespace layer;

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTile = 32;     // segments are multiples of this many tokens
constexpr int kCkpt = 16;     // tokens between the backward's saved states

enum Mode { FULL = 0, LOCAL = 1, CKPT = 2 };

template <int N>
struct Shape {
  static constexpr int LPC = N / 4;            // lanes of a channel
  static constexpr int CPT = 2;               // channels of a thread
  static constexpr int CW = N == 8 ? 2 : 4;    // warps that run the recurrence
  static constexpr int HW = 4;                 // helper warps
  static constexpr int CPW = (32 / LPC) * CPT; // channels of a warp
  static constexpr int CH = CW * CPW;          // channels of a block
  static constexpr int NT = (CW + HW) * 32;
  static constexpr int UN = LPC > 8 ? LPC : 8; // tokens in flight in the recurrence
};

// Tokens of a tile of the forward scan: what a helper thread's registers hold
// of three tiles, and at least four channels of one token each.
template <typename T, int N>
struct Tile {
  static constexpr int TK = sizeof(T) == 2 || N == 64 ? 32 : 16;
};

struct Args {
  const void *u, *dt, *Bm, *Cm, *z, *gy;
  long long ldu, lddt, ldb, ldc, ldz;
  const float *A, *Dw, *bias, *h0;
  const int* lengths;
  void* y;
  float* hT;
  float* ends;   // [B][S][D][N] local end states, then start states
  float* sums;   // [B][S][D] sums of dt' of a segment
  float* ckpt;   // [B][ceil(T/kCkpt)][D][N] states before every kCkpt-th token
  int B, T, D, G, S, seg;  // seg: tokens of a segment, a multiple of kTile
  int softplus;
  // whether four elements of a row of each can be accessed at once
  bool vu, vdt, vb, vc, vz;
};

// Sum over the LPC lanes of a channel of v[token][channel], LPC tokens at
// once: every exchange halves the tokens a lane is responsible for, so LPC
// tokens cost LPC - 1 exchanges a channel.  Lane nl ends with token nl in v[0].
template <int LPC, int CPT>
__device__ __forceinline__ void scatter_sum(float (&v)[LPC][CPT], int nl) {
#pragma unroll
  for (int off = LPC / 2; off > 0; off >>= 1) {
    const bool up = (nl & off) != 0;
#pragma unroll
    for (int i = 0; i < off; ++i)
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        const float keep = up ? v[i + off][c] : v[i][c];
        const float send = up ? v[i][c] : v[i + off][c];
        v[i][c] = keep + __shfl_xor_sync(0xffffffffu, send, off);
      }
  }
}

__device__ __forceinline__ float step_of(float raw, bool sp) { return sp ? softplus(raw) : raw; }

// Forward scan of one (channel tile, sequence, segment).
// REV (LOCAL only): the adjoint state e[t] = a[t] (e[t+1] + C[t] g[t]), g =
// gy silu(z), from the segment's last token to its first.
//
// A helper thread keeps its four channels through the sequence, loads its
// rows of the tile after the next into registers before it works on the next
// (a tile's time covers the latency), and holds u and z until the tile's y is
// there.
template <typename T, int N, int MODE, bool REV>
__global__ void __launch_bounds__(Shape<N>::NT, 2)
scan_kernel(Args p) {
  constexpr int LPC = Shape<N>::LPC, CPT = Shape<N>::CPT, CH = Shape<N>::CH;
  constexpr int TK = Tile<T, N>::TK;
  constexpr int CW = Shape<N>::CW, CPW = Shape<N>::CPW;
  constexpr int NH = Shape<N>::HW * 32;  // helper threads
  constexpr int IX = TK * CH / 4 / NH;                      // channel groups of a helper
  constexpr int IB = (TK * N / 4 + NH - 1) / NH;            // groups of B and of C
  static_assert(IX * NH * 4 == TK * CH && NH % (CH / 4) == 0, "helpers share a tile evenly");
  static_assert(!REV || MODE == LOCAL, "only end states run backward");
  constexpr bool USE_B = !REV, USE_C = MODE == FULL || REV;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  // [2][TK][CH] dt', then x = dt' u (or g), then y; [2][TK][N] B and C
  float* s_d = reinterpret_cast<float*>(smem_raw);
  float* s_x = s_d + 2 * TK * CH;
  float* s_y = s_x + 2 * TK * CH;
  float* s_b = s_y + (MODE == FULL ? 2 * TK * CH : 0);
  float* s_c = s_b + 2 * TK * N;

  const int Dg = p.D / p.G, TPG = (Dg + CH - 1) / CH;
  const int tiles = TPG * p.G;
  const int ct = blockIdx.x % tiles;
  const int rest = blockIdx.x / tiles;
  // nobody starts from the end of the chain's last segment
  const int ns = MODE == LOCAL ? p.S - 1 : p.S;
  const int sg = rest % ns + (REV ? 1 : 0), b = rest / ns;
  const int g = ct / TPG;
  const int c0 = g * Dg + (ct % TPG) * CH;       // first channel
  const int nc = min(CH, (g + 1) * Dg - c0);     // channels that exist
  const int t_lo = sg * p.seg, t_hi = min(p.T, t_lo + p.seg);
  const int t_live = min(t_hi, live_tokens(p.lengths, b, p.T));
  const int ntile = (t_hi - t_lo + TK - 1) / TK;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int first = REV ? ntile - 1 : 0, dir = REV ? -1 : 1;
  const long long row0 = (long long)b * p.T;

  if (warp >= CW) {
    // ------------------------------------------------ helpers
    const int hid = tid - CW * 32;
    const int c = (hid % (CH / 4)) * 4, tt0 = hid / (CH / 4);
    constexpr int TS = NH / (CH / 4);  // tokens between a helper's groups
    const int m = nc - c;              // channels that exist of this thread's four
    const bool vec = (Dg & 3) == 0;
    const bool vu = vec && p.vu, vdt = vec && p.vdt, vz = vec && p.vz;
    const T* src = REV ? (const T*)p.gy : (const T*)p.u;  // u, or gy
    const long long lds = REV ? p.D : p.ldu;
    const bool vs = REV ? vec : vu;
    src += row0 * lds + c0 + c;
    const T* dt = (const T*)p.dt + row0 * p.lddt + c0 + c;
    const bool has_z = p.z && (MODE == FULL || REV);
    const T* z = has_z ? (const T*)p.z + row0 * p.ldz + c0 + c : nullptr;
    const T* Bm = (const T*)p.Bm + row0 * p.ldb + (long long)g * N;
    const T* Cm = (const T*)p.Cm + row0 * p.ldc + (long long)g * N;
    T* y = MODE == FULL ? (T*)p.y + row0 * p.D + c0 + c : nullptr;
    const bool sp = p.softplus != 0;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f), skip = bias;
    if (p.bias) bias = ld4(p.bias + c0 + c, m, vec);
    if (MODE == FULL && p.Dw) skip = ld4(p.Dw + c0 + c, m, vec);

    Raw4<T> xn[IX], dn[IX], zn[IX], bn[IB], cn[IB];  // the tile to be staged next
    Raw4<T> xc[IX], zc[IX], xp[IX], zp[IX];          // u, z of the tiles in the scan and done
    // tiles of tokens that all exist take no care of ends
    const bool whole = vs && vdt && (vz || !has_z) && m >= 4;
    auto load = [&](int k) {
      const int t0 = t_lo + k * TK;
      if (whole && t0 + TK <= t_live) {
        const long long t = t0 + tt0;
        const T *px = src + t * lds, *pd = dt + t * p.lddt, *pz = z + (has_z ? t * p.ldz : 0);
        const long long sx = TS * lds, sd = TS * p.lddt, sz = TS * p.ldz;
#pragma unroll
        for (int i = 0; i < IX; ++i) {
          xn[i] = ld_raw4(px);
          dn[i] = ld_raw4(pd);
          if (has_z) zn[i] = ld_raw4(pz);
          px += sx; pd += sd; pz += sz;
        }
      } else {
#pragma unroll
        for (int i = 0; i < IX; ++i) {
          const int t = t0 + tt0 + i * TS;
          const int n = t < t_live ? m : 0;
          xn[i] = ld_raw4(src + (long long)t * lds, n, vs);
          dn[i] = ld_raw4(dt + (long long)t * p.lddt, n, vdt);
          if (has_z) zn[i] = ld_raw4(z + (long long)t * p.ldz, n, vz);
        }
      }
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        const int j = hid + i * NH, t = t0 + j / (N / 4), n = (j % (N / 4)) * 4;
        const int e = j < TK * N / 4 && t < t_live ? 4 : 0;
        if (USE_B) bn[i] = ld_raw4(Bm + (long long)t * p.ldb + n, e, p.vb);
        if (USE_C) cn[i] = ld_raw4(Cm + (long long)t * p.ldc + n, e, p.vc);
      }
    };
    auto stage = [&](int k) {
      const int t0 = t_lo + k * TK;
      float* sd = s_d + (k & 1) * TK * CH;
      float* sx = s_x + (k & 1) * TK * CH;
      const bool ends = m < 4 || t0 + TK > t_live;
#pragma unroll
      for (int i = 0; i < IX; ++i) {
        const int tt = tt0 + i * TS;
        float4 d = dn[i].get(), x = xn[i].get();
        d.x += bias.x; d.y += bias.y; d.z += bias.z; d.w += bias.w;
        if (sp) {
          d.x = softplus(d.x); d.y = softplus(d.y); d.z = softplus(d.z); d.w = softplus(d.w);
        }
        // tokens that do not exist, and channels past the last, step by 0:
        // their state stays as it is
        if (ends) {
          const int n = t0 + tt < t_live ? m : 0;
          if (n < 1) d.x = 0.f;
          if (n < 2) d.y = 0.f;
          if (n < 3) d.z = 0.f;
          if (n < 4) d.w = 0.f;
        }
        if (REV) {
          if (has_z) {
            const float4 q = zn[i].get();
            x.x *= silu(q.x); x.y *= silu(q.y); x.z *= silu(q.z); x.w *= silu(q.w);
          }
        } else {
          x.x *= d.x; x.y *= d.y; x.z *= d.z; x.w *= d.w;
        }
        *reinterpret_cast<float4*>(sd + tt * CH + c) = d;
        *reinterpret_cast<float4*>(sx + tt * CH + c) = x;
      }
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        const int j = hid + i * NH;
        if (j < TK * N / 4) {
          if (USE_B) reinterpret_cast<float4*>(s_b + (k & 1) * TK * N)[j] = bn[i].get();
          if (USE_C) reinterpret_cast<float4*>(s_c + (k & 1) * TK * N)[j] = cn[i].get();
        }
      }
    };
    auto finish = [&](int k, const Raw4<T>(&xs)[IX], const Raw4<T>(&zs)[IX]) {
      const int t0 = t_lo + k * TK;
      const float* sy = s_y + (k & 1) * TK * CH;
      if (vec && m >= 4 && t0 + TK <= t_live) {
        T* py = y + (long long)(t0 + tt0) * p.D;
#pragma unroll
        for (int i = 0; i < IX; ++i) {
          const float4 q = xs[i].get();
          float4 v = *reinterpret_cast<const float4*>(sy + (tt0 + i * TS) * CH + c);
          v.x = fmaf(skip.x, q.x, v.x); v.y = fmaf(skip.y, q.y, v.y);
          v.z = fmaf(skip.z, q.z, v.z); v.w = fmaf(skip.w, q.w, v.w);
          if (has_z) {
            const float4 w = zs[i].get();
            v.x *= silu(w.x); v.y *= silu(w.y); v.z *= silu(w.z); v.w *= silu(w.w);
          }
          IO<T>::st4(py, v);
          py += (long long)TS * p.D;
        }
        return;
      }
#pragma unroll
      for (int i = 0; i < IX; ++i) {
        const int tt = tt0 + i * TS, t = t0 + tt;
        if (t >= t_hi || m <= 0) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (t < t_live) {
          const float4 q = xs[i].get();
          v = *reinterpret_cast<const float4*>(sy + tt * CH + c);
          v.x = fmaf(skip.x, q.x, v.x); v.y = fmaf(skip.y, q.y, v.y);
          v.z = fmaf(skip.z, q.z, v.z); v.w = fmaf(skip.w, q.w, v.w);
          if (has_z) {
            const float4 w = zs[i].get();
            v.x *= silu(w.x); v.y *= silu(w.y); v.z *= silu(w.z); v.w *= silu(w.w);
          }
        }
        st4(y + (long long)t * p.D, v, m, vec);
      }
    };
    if (ntile > 0) {
      load(first);
      stage(first);
    }
#pragma unroll
    for (int i = 0; i < IX; ++i) { xc[i] = xn[i]; zc[i] = zn[i]; }
    if (ntile > 1) load(first + dir);
    __syncthreads();
    for (int i = 0; i < ntile; ++i) {
      const int k = first + dir * i;
      if (i + 1 < ntile) stage(k + dir);
      if (MODE == FULL && i > 0) finish(k - dir, xp, zp);
#pragma unroll
      for (int j = 0; j < IX; ++j) {
        xp[j] = xc[j]; zp[j] = zc[j];
        xc[j] = xn[j]; zc[j] = zn[j];
      }
      if (i + 2 < ntile) load(k + 2 * dir);
      __syncthreads();
    }
    if (MODE == FULL && ntile > 0) finish(ntile - 1, xp, zp);
    return;
  }

  // -------------------------------------------------- recurrence: 4 states of
  // CPT channels, as pairs
  const int nl = lane % LPC, cc = warp * CPW + (lane / LPC) * CPT;
  f32x2 a2[CPT][2], h[CPT][2];
  float sum[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    sum[k] = 0.f;
    a2[k][0] = a2[k][1] = h[k][0] = h[k][1] = pack2(0.f, 0.f);
    if (cc + k < nc) {
      const long long at = (long long)(c0 + cc + k) * N + nl * 4;
      const float4 v = *reinterpret_cast<const float4*>(p.A + at);
      a2[k][0] = pack2(v.x * kLog2e, v.y * kLog2e);
      a2[k][1] = pack2(v.z * kLog2e, v.w * kLog2e);
      const float* from = nullptr;
      if (MODE != LOCAL) {
        if (p.S > 1)
          from = p.ends + ((long long)b * p.S + sg) * p.D * N + at;
        else if (p.h0)
          from = p.h0 + (long long)b * p.D * N + at;
      }
      if (from) {
        const float4 q = *reinterpret_cast<const float4*>(from);
        h[k][0] = pack2(q.x, q.y);
        h[k][1] = pack2(q.z, q.w);
      }
    }
  }
  auto save = [&](float* to) {  // to: [D][N]
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (cc + k < nc) {
        const float2 u = unpack2(h[k][0]), v = unpack2(h[k][1]);
        *reinterpret_cast<float4*>(to + (long long)(c0 + cc + k) * N + nl * 4) =
            make_float4(u.x, u.y, v.x, v.y);
      }
  };
  auto scan = [&](int k) {
    const float* sd = s_d + (k & 1) * TK * CH + cc;
    const float* sx = s_x + (k & 1) * TK * CH + cc;
    const float* sb = s_b + (k & 1) * TK * N + nl * 4;
    const float* sc = s_c + (k & 1) * TK * N + nl * 4;
    float* sy = s_y + (k & 1) * TK * CH + cc;
    constexpr int UN = Shape<N>::UN;
#pragma unroll 1
    for (int tt = 0; tt < TK; tt += UN) {
      if (MODE == CKPT && tt % kCkpt == 0) {
        const int t = t_lo + k * TK + tt;
        if (t < t_hi)
          save(p.ckpt + ((long long)b * ((p.T + kCkpt - 1) / kCkpt) + t / kCkpt) * p.D * N);
      }
      float yv[UN][CPT];
#pragma unroll
      for (int i = 0; i < UN; ++i) {
        const int t = REV ? TK - 1 - tt - i : tt + i;
        f32x2 bv[2], cv[2];
        if (USE_B) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sb + t * N);
          bv[0] = v.x; bv[1] = v.y;
        }
        if (USE_C) {
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sc + t * N);
          cv[0] = v.x; cv[1] = v.y;
        }
        float d[CPT], x[CPT];
        if constexpr (CPT == 4) {
          const float4 v = *reinterpret_cast<const float4*>(sd + t * CH);
          const float4 w = *reinterpret_cast<const float4*>(sx + t * CH);
          d[0] = v.x; d[1] = v.y; d[2] = v.z; d[3] = v.w;
          x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
        } else if constexpr (CPT == 2) {
          const float2 v = *reinterpret_cast<const float2*>(sd + t * CH);
          const float2 w = *reinterpret_cast<const float2*>(sx + t * CH);
          d[0] = v.x; d[1] = v.y;
          x[0] = w.x; x[1] = w.y;
        } else {
          d[0] = sd[t * CH];
          x[0] = sx[t * CH];
        }
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
          const f32x2 d2 = pack2(d[c], d[c]), w2 = pack2(x[c], x[c]);
          const f32x2 e0 = ex2_2(mul2(d2, a2[c][0])), e1 = ex2_2(mul2(d2, a2[c][1]));
          if (REV) {
            h[c][0] = mul2(e0, fma2(w2, cv[0], h[c][0]));
            h[c][1] = mul2(e1, fma2(w2, cv[1], h[c][1]));
          } else {
            h[c][0] = fma2(e0, h[c][0], mul2(w2, bv[0]));
            h[c][1] = fma2(e1, h[c][1], mul2(w2, bv[1]));
          }
          if (MODE == LOCAL) sum[c] += d[c];
          if (MODE == FULL) {
            const float2 s = unpack2(fma2(cv[1], h[c][1], mul2(cv[0], h[c][0])));
            yv[i][c] = s.x + s.y;
          }
        }
      }
      if constexpr (MODE == FULL) {
#pragma unroll
        for (int j = 0; j < UN; j += LPC) {
          float (&part)[LPC][CPT] = *reinterpret_cast<float (*)[LPC][CPT]>(&yv[j]);
          scatter_sum<LPC, CPT>(part, nl);
#pragma unroll
          for (int c = 0; c < CPT; ++c) sy[(tt + j + nl) * CH + c] = part[0][c];
        }
      }
    }
  };
  __syncthreads();
  for (int i = 0; i < ntile; ++i) {
    scan(first + dir * i);
    __syncthreads();
  }
  if (MODE == LOCAL) {
    save(p.ends + ((long long)b * p.S + sg) * p.D * N);
#pragma unroll
    for (int c = 0; c < CPT; ++c)
      if (nl == 0 && cc + c < nc) p.sums[((long long)b * p.S + sg) * p.D + c0 + cc + c] = sum[c];
  }
  if (MODE == FULL && p.hT && sg == p.S - 1) save(p.hT + (long long)b * p.D * N);
}

// Chain over the segments: ends[b][s] (from a zero start) becomes the state
// that segment s starts from.  REV walks from the last segment to the first.
template <bool REV>
__global__ void __launch_bounds__(256)
chain_kernel(const float* __restrict__ A, const float* __restrict__ h0, float* __restrict__ ends,
             const float* __restrict__ sums, int S, int D, int N, long long total) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const long long dn = (long long)D * N;
  const long long b = id / dn, at = id % dn;
  const int d = (int)(at / N);
  const float a2 = A[at] * kLog2e;
  float h = h0 ? h0[id] : 0.f;
  for (int i = 0; i < S; ++i) {
    const int s = REV ? S - 1 - i : i;
    float* e = ends + (b * S + s) * dn + at;
    if (i == S - 1) {
      *e = h;
      return;
    }
    const float own = *e;
    *e = h;
    h = fmaf(ex2(a2 * sums[(b * S + s) * D + d]), h, own);
  }
}

// ---------------------------------------------------------------- backward
//
// With g = gy silu(z) and the adjoint state e (what flows into h[t-1]):
//   dh = e + C g;  dC = sum_d h g;  dB = sum_d dh dt' u;  e <- a dh
//   du = D g + dt' sum_n dh B;  ddt' = u sum_n dh B + sum_n A h[t-1] e
//   dA = sum_t dt' h[t-1] e;  dz = gy y0 silu'(z);  dD = sum g u
// A block takes kCkpt tokens at a time from the segment's end: a thread
// rebuilds the kCkpt states of its 4 from the saved one (decays and states
// stay in registers), then walks back.  Sums over n cross the lanes of a
// channel, sums over channels the other lanes and then the warps through
// shared memory; dB and dC leave as one part a channel tile, dA, dD and
// dt_bias as one part a segment, and reduce kernels add the parts in order:
// no atomics, the same bits every time.
constexpr int kBW = 8;  // warps of a backward block

template <int N>
struct BwdShape {
  static constexpr int LPC = N / 4;
  static constexpr int CPW = 32 / LPC;    // channels of a warp
  static constexpr int CH = kBW * CPW;    // channels of a block
};

struct BwdArgs {
  Args f;                       // forward arguments; f.ckpt, f.ends = adjoint starts
  const float* ghT;
  void *du, *ddt, *dz;
  float *dh0;
  float* part_bc;               // [TPG][B][T][G][2N]
  float* part_a;                // [B*S][D][N]
  float* part_d;                // [B*S][2][D]: dD, ddt_bias
};

template <typename T, int N>
__global__ void __launch_bounds__(kBW * 32, 1)
bwd_kernel(BwdArgs q) {
  constexpr int LPC = BwdShape<N>::LPC, CPW = BwdShape<N>::CPW, CH = BwdShape<N>::CH;
  constexpr int K = kCkpt;
  const Args& p = q.f;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float4* s_x = reinterpret_cast<float4*>(smem_raw);     // [K][CH] dt', dt' u, g, u
  float* s_b = reinterpret_cast<float*>(s_x + K * CH);   // [K][N]
  float* s_c = s_b + K * N;                              // [K][N]
  float4* s_o = reinterpret_cast<float4*>(s_c + K * N);  // [K][CH] sum dh B, sum A h e, y0
  float* s_bc = reinterpret_cast<float*>(s_o + K * CH);  // [kBW][K][2N]

  const int Dg = p.D / p.G, TPG = (Dg + CH - 1) / CH;
  const int tiles = TPG * p.G;
  const int ct = blockIdx.x % tiles;
  const int rest = blockIdx.x / tiles;
  const int sg = rest % p.S, b = rest / p.S;
  const int g = ct / TPG;
  const int c0 = g * Dg + (ct % TPG) * CH;
  const int nc = min(CH, (g + 1) * Dg - c0);
  const int t_lo = sg * p.seg, t_hi = min(p.T, t_lo + p.seg);
  const int n_live = live_tokens(p.lengths, b, p.T);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nl = lane % LPC, cg = lane / LPC, cl = warp * CPW + cg;
  const long long row0 = (long long)b * p.T;
  const T* u = (const T*)p.u + c0;
  const T* dt = (const T*)p.dt + c0;
  const T* z = p.z ? (const T*)p.z + c0 : nullptr;
  const T* gy = (const T*)p.gy + c0;
  const T* Bm = (const T*)p.Bm + (long long)g * N;
  const T* Cm = (const T*)p.Cm + (long long)g * N;
  const bool vec = (Dg & 3) == 0, vy = vec;
  const bool vu = vec && p.vu, vdt = vec && p.vdt, vz = vec && p.vz, vb = p.vb, vc = p.vc;

  const long long at = (long long)(c0 + cl) * N + nl * 4;
  const bool mine = cl < nc;
  float A[4] = {}, e[4] = {}, dA[4] = {};
  if (mine) {
    const float4 v = *reinterpret_cast<const float4*>(p.A + at);
    A[0] = v.x; A[1] = v.y; A[2] = v.z; A[3] = v.w;
    const float* from = p.S > 1 ? p.ends + ((long long)b * p.S + sg) * p.D * N + at
                        : q.ghT ? q.ghT + (long long)b * p.D * N + at
                                : nullptr;
    if (from) {
      const float4 w = *reinterpret_cast<const float4*>(from);
      e[0] = w.x; e[1] = w.y; e[2] = w.z; e[3] = w.w;
    }
  }
  // the 4 channels whose sums this thread keeps in the block's last step
  constexpr int VPT = K * CH / 4 / (kBW * 32) > 0 ? K * CH / 4 / (kBW * 32) : 1;
  static_assert((kBW * 32) % (CH / 4) == 0, "a thread keeps its channels");
  float4 accD = make_float4(0.f, 0.f, 0.f, 0.f), accT = accD;

  const int nchunk = (t_hi - t_lo + K - 1) / K;
  const int nck = (p.T + K - 1) / K;
  for (int ch = nchunk - 1; ch >= 0; --ch) {
    const int t0 = t_lo + ch * K;
    // inputs of the K tokens
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = tid + v * kBW * 32;
      if (i < K * CH / 4) {
        const int tt = i / (CH / 4), c = (i % (CH / 4)) * 4, t = t0 + tt;
        float4 d = make_float4(0.f, 0.f, 0.f, 0.f), x = d, gg = d;
        if (t < t_hi && t < n_live && c < nc) {
          const long long r = row0 + t;
          const int m = nc - c;
          d = ld4(dt + r * p.lddt + c, m, vdt);
          if (p.bias) {
            const float4 w = ld4(p.bias + c0 + c, m, vec);
            d.x += w.x; d.y += w.y; d.z += w.z; d.w += w.w;
          }
          d.x = step_of(d.x, p.softplus); d.y = step_of(d.y, p.softplus);
          d.z = step_of(d.z, p.softplus); d.w = step_of(d.w, p.softplus);
          x = ld4(u + r * p.ldu + c, m, vu);
          gg = ld4(gy + r * p.D + c, m, vy);
          if (z) {
            const float4 w = ld4(z + r * p.ldz + c, m, vz);
            gg.x *= silu(w.x); gg.y *= silu(w.y); gg.z *= silu(w.z); gg.w *= silu(w.w);
          }
          if (m < 4) {
            if (m < 2) d.y = x.y = gg.y = 0.f;
            if (m < 3) d.z = x.z = gg.z = 0.f;
            d.w = x.w = gg.w = 0.f;
          }
        }
        float4* o = s_x + tt * CH + c;
        o[0] = make_float4(d.x, d.x * x.x, gg.x, x.x);
        o[1] = make_float4(d.y, d.y * x.y, gg.y, x.y);
        o[2] = make_float4(d.z, d.z * x.z, gg.z, x.z);
        o[3] = make_float4(d.w, d.w * x.w, gg.w, x.w);
      }
    }
    for (int i = tid; i < K * N / 4; i += kBW * 32) {
      const int tt = i / (N / 4), n = (i % (N / 4)) * 4, t = t0 + tt;
      float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f), c4 = b4;
      if (t < t_hi && t < n_live) {
        b4 = ld4(Bm + (row0 + t) * p.ldb + n, 4, vb);
        c4 = ld4(Cm + (row0 + t) * p.ldc + n, 4, vc);
      }
      *reinterpret_cast<float4*>(s_b + tt * N + n) = b4;
      *reinterpret_cast<float4*>(s_c + tt * N + n) = c4;
    }
    float h0[4] = {};
    if (mine) {
      const float4 v = *reinterpret_cast<const float4*>(
          p.ckpt + ((long long)b * nck + t0 / K) * p.D * N + at);
      h0[0] = v.x; h0[1] = v.y; h0[2] = v.z; h0[3] = v.w;
    }
    __syncthreads();
    float a[K][4], h[K][4];
#pragma unroll
    for (int t = 0; t < K; ++t) {
      const float4 x = s_x[t * CH + cl];
      const float4 bv = *reinterpret_cast<const float4*>(s_b + t * N + nl * 4);
      const float bb[4] = {bv.x, bv.y, bv.z, bv.w};
      const float xd = x.x * kLog2e;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[t][i] = ex2(xd * A[i]);
        h[t][i] = fmaf(a[t][i], t ? h[t > 0 ? t - 1 : 0][i] : h0[i], x.y * bb[i]);
      }
    }
#pragma unroll
    for (int t = K - 1; t >= 0; --t) {
      const float4 x = s_x[t * CH + cl];
      const float4 bv = *reinterpret_cast<const float4*>(s_b + t * N + nl * 4);
      const float4 cv = *reinterpret_cast<const float4*>(s_c + t * N + nl * 4);
      const float bb[4] = {bv.x, bv.y, bv.z, bv.w}, cv4[4] = {cv.x, cv.y, cv.z, cv.w};
      float sB = 0.f, sA = 0.f, y0 = 0.f;
      float w[8];  // dB, dC of 4 states, to be summed over the warp's channels
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float dh = fmaf(cv4[i], x.z, e[i]);
        w[i] = dh * x.y;
        w[4 + i] = h[t][i] * x.z;
        y0 = fmaf(cv4[i], h[t][i], y0);
        sB = fmaf(dh, bb[i], sB);
        e[i] = a[t][i] * dh;
        const float f = e[i] * (t ? h[t > 0 ? t - 1 : 0][i] : h0[i]);
        sA = fmaf(A[i], f, sA);
        dA[i] = fmaf(x.x, f, dA[i]);
      }
#pragma unroll
      for (int off = LPC / 2; off > 0; off >>= 1) {
        sB += __shfl_xor_sync(0xffffffffu, sB, off);
        sA += __shfl_xor_sync(0xffffffffu, sA, off);
        y0 += __shfl_xor_sync(0xffffffffu, y0, off);
      }
      if (nl == 0) s_o[t * CH + cl] = make_float4(sB, sA, y0, 0.f);
      // over the CPW channels of the warp: halve the values a lane keeps
      // while there are values to share, then add plainly
      int keep = 8, first = 0;
#pragma unroll
      for (int off = CPW / 2; off > 0; off >>= 1) {
        if (keep > 1) {
          keep >>= 1;
          const bool up = (cg & off) != 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < keep) {
              const float k0 = up ? w[i + keep] : w[i], s0 = up ? w[i] : w[i + keep];
              w[i] = k0 + __shfl_xor_sync(0xffffffffu, s0, off * LPC);
            }
          first += up ? keep : 0;
        } else {
          w[0] += __shfl_xor_sync(0xffffffffu, w[0], off * LPC);
        }
      }
      // value v of 8: dB (v < 4) or dC of state nl*4 + v % 4
      float* o = s_bc + (warp * K + t) * 2 * N;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < keep) {
          const int v = first + i;
          if (CPW <= 8 || (cg & 1) == 0)
            o[(v >= 4 ? N : 0) + nl * 4 + (v & 3)] = w[i];
        }
    }
    __syncthreads();
    // dB, dC of the K tokens: the warps' sums in order
    float* pbc = q.part_bc + (((long long)(ct % TPG) * p.B + b) * p.T * p.G + g) * 2 * N;
    for (int i = tid; i < K * 2 * N; i += kBW * 32) {
      const int tt = i / (2 * N), n = i % (2 * N);
      if (t0 + tt < t_hi) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kBW; ++w) s += s_bc[(w * K + tt) * 2 * N + n];
        pbc[(long long)(t0 + tt) * p.G * 2 * N + n] = s;
      }
    }
    // du, ddt, dz
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      const int i = tid + v * kBW * 32;
      if (i < K * CH / 4) {
        const int tt = i / (CH / 4), c = (i % (CH / 4)) * 4, t = t0 + tt;
        if (t < t_hi && c < nc) {
          const long long r = row0 + t;
          const int m = nc - c;
          float4 vdu = make_float4(0.f, 0.f, 0.f, 0.f), vddt = vdu, vdz = vdu;
          if (t < n_live) {
            float4 raw = vdu, zz = vdu, g0 = vdu, dw = vdu;
            if (p.softplus) {
              raw = ld4(dt + r * p.lddt + c, m, vdt);
              if (p.bias) {
                const float4 w = ld4(p.bias + c0 + c, m, vec);
                raw.x += w.x; raw.y += w.y; raw.z += w.z; raw.w += w.w;
              }
            }
            if (p.Dw) dw = ld4(p.Dw + c0 + c, m, vec);
            if (z) {
              zz = ld4(z + r * p.ldz + c, m, vz);
              g0 = ld4(gy + r * p.D + c, m, vy);
            }
            auto one = [&](int k, float rw, float zv, float gv, float dv, float& du, float& ddt,
                           float& dzo, float& aD, float& aT) {
              const float4 x = s_x[tt * CH + c + k], o = s_o[tt * CH + c + k];
              du = fmaf(dv, x.z, o.x * x.x);
              ddt = fmaf(o.x, x.w, o.y);
              if (p.softplus) ddt *= sigmoid(rw);
              if (z) {
                const float s = sigmoid(zv);
                dzo = gv * fmaf(dv, x.w, o.z) * (s * fmaf(zv, 1.f - s, 1.f));
              }
              aD = fmaf(x.z, x.w, aD);
              aT += ddt;
            };
            one(0, raw.x, zz.x, g0.x, dw.x, vdu.x, vddt.x, vdz.x, accD.x, accT.x);
            one(1, raw.y, zz.y, g0.y, dw.y, vdu.y, vddt.y, vdz.y, accD.y, accT.y);
            one(2, raw.z, zz.z, g0.z, dw.z, vdu.z, vddt.z, vdz.z, accD.z, accT.z);
            one(3, raw.w, zz.w, g0.w, dw.w, vdu.w, vddt.w, vdz.w, accD.w, accT.w);
          }
          st4((T*)q.du + c0 + r * p.D + c, vdu, m, vy);
          st4((T*)q.ddt + c0 + r * p.D + c, vddt, m, vy);
          if (z) st4((T*)q.dz + c0 + r * p.D + c, vdz, m, vy);
        }
      }
    }
    __syncthreads();
  }
  const long long ps = (long long)b * p.S + sg;
  if (mine) {
    *reinterpret_cast<float4*>(q.part_a + ps * p.D * N + at) =
        make_float4(dA[0], dA[1], dA[2], dA[3]);
    if (q.dh0 && sg == 0)
      *reinterpret_cast<float4*>(q.dh0 + (long long)b * p.D * N + at) =
          make_float4(e[0], e[1], e[2], e[3]);
  }
  // dD, ddt_bias: over the threads that kept the same 4 channels
  float4* red = s_x;  // [2][kBW * 32], free after the last barrier
  red[tid] = accD;
  red[kBW * 32 + tid] = accT;
  __syncthreads();
  for (int i = tid; i < 2 * CH; i += kBW * 32) {
    const int w = i / CH, c = i % CH;
    if (c < nc) {
      float s = 0.f;
      for (int r = c / 4; r < kBW * 32; r += CH / 4)
        s += reinterpret_cast<const float*>(red + w * kBW * 32 + r)[c & 3];
      q.part_d[(ps * 2 + w) * p.D + c0 + c] = s;
    }
  }
}

// dB and dC: the channel tiles' parts [TPG][rows][2N] in order, rounded to T.
template <typename T>
__global__ void __launch_bounds__(256)
reduce_bc_kernel(const float* __restrict__ part, int P, long long rows, int N,
                 T* __restrict__ dB, T* __restrict__ dC) {
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x;  // groups of 4
  const long long per = rows * 2 * N / 4;
  if (i >= per) return;
  const long long r = i / (N / 2);
  const int n = (int)(i % (N / 2)) * 4;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < P; ++k) {
    const float4 v = reinterpret_cast<const float4*>(part)[(long long)k * per + i];
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  T* o = n < N ? dB + r * N + n : dC + r * N + n - N;
  IO<T>::st4(o, s);
}

// dA [D][N], dD and ddt_bias [D]: the segments' parts in order.
__global__ void __launch_bounds__(256)
reduce_param_kernel(const float* __restrict__ pa, const float* __restrict__ pd, int P, int D,
                    int N, float* __restrict__ dA, float* __restrict__ dD,
                    float* __restrict__ dbias) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
  const long long dn = (long long)D * N, all = dn + 2LL * D;
  const long long i = (long long)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (i < all) {
    const float* p = i < dn ? pa + i : pd + (i - dn);
    const long long step = i < dn ? dn : 2LL * D;
    for (int k = row; k < P; k += 8) s += p[(long long)k * step];
  }
  red[row][lane] = s;
  __syncthreads();
  if (row == 0 && i < all) {
    s = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) s += red[r][lane];
    if (i < dn)
      dA[i] = s;
    else if (i < dn + D) {
      if (dD) dD[i - dn] = s;
    } else if (dbias) {
      dbias[i - dn - D] = s;
    }
  }
}

// ---------------------------------------------------------------- one token
//
// One read and one write of the state; a thread holds 4 states, the N/4
// threads of a channel lie side by side.
template <typename T, int N>
__global__ void __launch_bounds__(256)
step_kernel(Args p, float* __restrict__ S, long long total) {
  constexpr int LPC = N / 4;
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id - (threadIdx.x & 31) >= total) return;  // whole warps only
  const bool live = id < total;
  const long long ch = live ? id / LPC : 0;
  const int nl = threadIdx.x % LPC;
  const int d = (int)(ch % p.D);
  const long long b = ch / p.D;
  const int g = d / (p.D / p.G);
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f), A = h, bv = h, cv = h;
  float dt = 0.f, u = 0.f, zz = 0.f;
  if (live) {
    h = reinterpret_cast<const float4*>(S)[id];
    A = *reinterpret_cast<const float4*>(p.A + (long long)d * N + nl * 4);
    bv = ld4((const T*)p.Bm + b * p.ldb + g * N + nl * 4, 4, p.vb);
    cv = ld4((const T*)p.Cm + b * p.ldc + g * N + nl * 4, 4, p.vc);
    dt = IO<T>::ld((const T*)p.dt + b * p.lddt + d);
    u = IO<T>::ld((const T*)p.u + b * p.ldu + d);
    if (p.z) zz = IO<T>::ld((const T*)p.z + b * p.ldz + d);
    if (p.bias) dt += p.bias[d];
    dt = step_of(dt, p.softplus);
  }
  const float x = dt * u, s = dt * kLog2e;
  h.x = fmaf(ex2(s * A.x), h.x, x * bv.x);
  h.y = fmaf(ex2(s * A.y), h.y, x * bv.y);
  h.z = fmaf(ex2(s * A.z), h.z, x * bv.z);
  h.w = fmaf(ex2(s * A.w), h.w, x * bv.w);
  float y = fmaf(cv.w, h.w, fmaf(cv.z, h.z, fmaf(cv.y, h.y, cv.x * h.x)));
#pragma unroll
  for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
  if (!live) return;
  reinterpret_cast<float4*>(S)[id] = h;
  if (nl == 0) {
    if (p.Dw) y = fmaf(p.Dw[d], u, y);
    if (p.z) y *= silu(zz);
    IO<T>::st((T*)p.y + ch, y);
  }
}

// ---------------------------------------------------------------- host side

static int channels(int N) { return N == 8 ? Shape<8>::CH : N == 16 ? Shape<16>::CH
                                  : N == 32 ? Shape<32>::CH : Shape<64>::CH; }
static int bwd_channels(int N) {
  return N == 8 ? BwdShape<8>::CH : N == 16 ? BwdShape<16>::CH
       : N == 32 ? BwdShape<32>::CH : BwdShape<64>::CH;
}

struct Split {
  int S, seg;
};

// Segments: none while the channel tiles alone give every SM a block.  A cut
// runs the exponentials twice, so it has to bring at least that: as many
// segments as fill two blocks an SM, of 256 tokens at least.
static Split split(long long base, int T) {
  int S = 1;
  if (base < 148) {
    const long long want = (2 * 148) / base;
    const int most = T / 256;
    S = (int)(want < most ? want : most);
    if (S < 3) S = 1;
  }
  const int tiles = (T + kTile - 1) / kTile;
  const int seg = ((tiles + S - 1) / S) * kTile;
  S = (T + seg - 1) / seg;
  return Split{S < 1 ? 1 : S, seg < kTile ? kTile : seg};
}

static long long tiles_of(int D, int G, int CH) { return (long long)G * ((D / G + CH - 1) / CH); }

static Split fwd_split(int B, int T, int D, int G, int N) {
  return split(B * tiles_of(D, G, channels(N)), T);
}
static Split bwd_split(int B, int T, int D, int G, int N) {
  return split(B * tiles_of(D, G, bwd_channels(N)), T);
}

static size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

static size_t chain_bytes(int B, int D, int N, int S) {
  return S > 1 ? up((size_t)B * S * D * N * 4) + up((size_t)B * S * D * 4) : 0;
}

template <typename T, int N, int MODE, bool REV>
static cudaError_t run_scan(const Args& a, cudaStream_t st) {
  constexpr int CH = Shape<N>::CH;
  const size_t smem = 2 * Tile<T, N>::TK * (CH * (8 + (MODE == FULL ? 4 : 0)) + 2 * N * 4);
  const long long blocks = tiles_of(a.D, a.G, CH) * a.B * (MODE == LOCAL ? a.S - 1 : a.S);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto k = scan_kernel<T, N, MODE, REV>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k<<<(unsigned)blocks, Shape<N>::NT, smem, st>>>(a);
  return cudaGetLastError();
}

template <bool REV>
static cudaError_t run_chain(const Args& a, int N, const float* h0, cudaStream_t st) {
  const long long total = (long long)a.B * a.D * N;
  if ((total + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidValue;
  chain_kernel<REV><<<(unsigned)((total + 255) / 256), 256, 0, st>>>(a.A, h0, a.ends, a.sums,
                                                                     a.S, a.D, N, total);
  return cudaGetLastError();
}

template <typename T, int N, int MODE>
static cudaError_t run_forward(const Args& a, cudaStream_t st) {
  if (a.S > 1) {
    cudaError_t e = run_scan<T, N, LOCAL, false>(a, st);
    if (e == cudaSuccess) e = run_chain<false>(a, N, a.h0, st);
    if (e != cudaSuccess) return e;
  }
  return run_scan<T, N, MODE, false>(a, st);
}

struct BwdPlan {
  Split f, r;
  int TPG;
  size_t ckpt, fends, fsums, rends, rsums, bc, pa, pd, total;
};

static BwdPlan bwd_plan(int B, int T, int D, int G, int N) {
  BwdPlan w;
  w.f = fwd_split(B, T, D, G, N);
  w.r = bwd_split(B, T, D, G, N);
  w.TPG = (D / G + bwd_channels(N) - 1) / bwd_channels(N);
  const size_t dn = (size_t)D * N * 4;
  size_t at = 0;
  auto take = [&](size_t n) { size_t r = at; at += up(n); return r; };
  w.ckpt = take((size_t)B * ((T + kCkpt - 1) / kCkpt) * dn);
  w.fends = take(w.f.S > 1 ? B * w.f.S * dn : 0);
  w.fsums = take(w.f.S > 1 ? (size_t)B * w.f.S * D * 4 : 0);
  w.rends = take(w.r.S > 1 ? B * w.r.S * dn : 0);
  w.rsums = take(w.r.S > 1 ? (size_t)B * w.r.S * D * 4 : 0);
  w.bc = take((size_t)w.TPG * B * T * G * 2 * N * 4);
  w.pa = take((size_t)B * w.r.S * dn);
  w.pd = take((size_t)B * w.r.S * 2 * D * 4);
  w.total = at;
  return w;
}

template <typename T, int N>
static cudaError_t run_backward(BwdArgs q, const BwdPlan& w, unsigned char* ws, float* dA,
                                float* dD, float* dbias, void* dB, void* dC, cudaStream_t st) {
  Args f = q.f;
  f.ckpt = (float*)(ws + w.ckpt);
  f.S = w.f.S; f.seg = w.f.seg;
  f.ends = (float*)(ws + w.fends);
  f.sums = (float*)(ws + w.fsums);
  cudaError_t e = run_forward<T, N, CKPT>(f, st);
  if (e != cudaSuccess) return e;
  q.f.ckpt = f.ckpt;
  q.f.S = w.r.S; q.f.seg = w.r.seg;
  q.f.ends = (float*)(ws + w.rends);
  q.f.sums = (float*)(ws + w.rsums);
  q.part_bc = (float*)(ws + w.bc);
  q.part_a = (float*)(ws + w.pa);
  q.part_d = (float*)(ws + w.pd);
  if (w.r.S > 1) {
    e = run_scan<T, N, LOCAL, true>(q.f, st);
    if (e == cudaSuccess) e = run_chain<true>(q.f, N, q.ghT, st);
    if (e != cudaSuccess) return e;
  }
  constexpr int CH = BwdShape<N>::CH, K = kCkpt;
  size_t smem = (size_t)K * CH * 32 + K * N * 8 + (size_t)kBW * K * 2 * N * 4;
  if (smem < 2 * kBW * 32 * 16) smem = 2 * kBW * 32 * 16;
  const long long blocks = tiles_of(q.f.D, q.f.G, CH) * q.f.B * q.f.S;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto k = bwd_kernel<T, N>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k<<<(unsigned)blocks, kBW * 32, smem, st>>>(q);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long rows = (long long)q.f.B * q.f.T * q.f.G, quads = rows * N / 2;
  if ((quads + 255) / 256 > 0x7fffffffLL) return cudaErrorInvalidValue;
  reduce_bc_kernel<T><<<(unsigned)((quads + 255) / 256), 256, 0, st>>>(q.part_bc, w.TPG, rows, N,
                                                                       (T*)dB, (T*)dC);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long all = (long long)q.f.D * N + 2LL * q.f.D;
  reduce_param_kernel<<<(unsigned)((all + 31) / 32), 256, 0, st>>>(
      q.part_a, q.part_d, q.f.B * q.f.S, q.f.D, N, dA, dD, dbias);
  return cudaGetLastError();
}

template <typename T, int N>
static cudaError_t run_step(const Args& a, float* S, cudaStream_t st) {
  const long long total = (long long)a.B * a.D * (N / 4), blocks = (total + 255) / 256;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  step_kernel<T, N><<<(unsigned)blocks, 256, 0, st>>>(a, S, total);
  return cudaGetLastError();
}

static kla_status check(int B, int T, int D, int G, int N, int dtype) {
  if (B < 1 || T < 0 || D < 1 || G < 1 || N < 1 || D % G != 0 || !dtype_ok(dtype))
    return KLA_ERR_INVALID_ARG;
  if (!size_ok((long long)B * (T > 0 ? T : 1), (long long)D) ||
      !size_ok((long long)B * D, (long long)N * (T / kCkpt + 1)) ||
      !size_ok((long long)B * (T > 0 ? T : 1), 2LL * G * N * 4))
    return KLA_ERR_INVALID_ARG;
  if (T > kMaxTokens || (N != 8 && N != 16 && N != 32 && N != 64)) return KLA_ERR_UNSUPPORTED;
  return KLA_OK;
}

static bool pitches_ok(long long rows, int D, int G, int N, long long ldu, long long lddt,
                       long long ldb, long long ldc, long long ldz, bool z) {
  return ldu >= D && lddt >= D && ldb >= (long long)G * N && ldc >= (long long)G * N &&
         (!z || ldz >= D) && size_ok(rows, ldu) && size_ok(rows, lddt) && size_ok(rows, ldb) &&
         size_ok(rows, ldc) && (!z || size_ok(rows, ldz));
}

static void set_rows(Args& a, long long ldu, long long lddt, long long ldb, long long ldc,
                     long long ldz, int N, int es) {
  a.ldu = ldu; a.lddt = lddt; a.ldb = ldb; a.ldc = ldc; a.ldz = ldz;
  a.vu = rows_aligned(a.u, a.D, ldu, 4, es);
  a.vdt = rows_aligned(a.dt, a.D, lddt, 4, es);
  a.vz = rows_aligned(a.z, a.D, ldz, 4, es);
  a.vb = rows_aligned(a.Bm, N, ldb, 4, es);
  a.vc = rows_aligned(a.Cm, N, ldc, 4, es);
}

static bool rows_misplaced(const void* u, const void* dt, const void* Bm, const void* Cm,
                           const void* z, int es) {
  return misplaced(u, es) || misplaced(dt, es) || misplaced(Bm, es) || misplaced(Cm, es) ||
         misplaced(z, es);
}

#define KLA_SSM_DISPATCH(CALL)                                   \
  if (dtype == KLA_BF16) {                                       \
    using TY = __nv_bfloat16;                                    \
    switch (N) {                                                 \
      case 8: { constexpr int KN = 8; CALL; } break;             \
      case 16: { constexpr int KN = 16; CALL; } break;           \
      case 32: { constexpr int KN = 32; CALL; } break;           \
      default: { constexpr int KN = 64; CALL; } break;           \
    }                                                            \
  } else {                                                       \
    using TY = float;                                            \
    switch (N) {                                                 \
      case 8: { constexpr int KN = 8; CALL; } break;             \
      case 16: { constexpr int KN = 16; CALL; } break;           \
      case 32: { constexpr int KN = 32; CALL; } break;           \
      default: { constexpr int KN = 64; CALL; } break;           \
    }                                                            \
  }

}  // namespace ssm
}  // namespace kla

using namespace kla;
using namespace kla::ssm;

extern "C" {

size_t kla_ssm_fwd_workspace_size(int B, int T, int D, int G, int N) {
  if (check(B, T, D, G, N, KLA_BF16) != KLA_OK || T == 0) return 0;
  return chain_bytes(B, D, N, fwd_split(B, T, D, G, N).S);
}

kla_status kla_ssm_fwd(const void* u, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dw, const void* z, const float* dt_bias,
                       const float* h0, const int* lengths, void* y, float* hT, int B, int T,
                       int D, int G, int N, long long ldu, long long lddt, long long ldb,
                       long long ldc, long long ldz, int softplus, int dtype, void* workspace,
                       size_t ws_bytes, void* stream) {
  kla_status s = check(B, T, D, G, N, dtype);
  if (s != KLA_OK) return s;
  const void* const ptrs[] = {A, Dw, dt_bias, h0, lengths, y, hT, workspace};
  if (misaligned(ptrs) || rows_misplaced(u, dt, Bm, Cm, z, elem(dtype))) return KLA_ERR_INVALID_ARG;
  const long long rows = (long long)B * T, dn = (long long)D * N, ns = B * dn;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (T > 0) {
    if (!u || !dt || !A || !Bm || !Cm || !y) return KLA_ERR_INVALID_ARG;
    if (!pitches_ok(rows, D, G, N, ldu, lddt, ldb, ldc, ldz, z != nullptr))
      return KLA_ERR_INVALID_ARG;
  }
  const size_t need = kla_ssm_fwd_workspace_size(B, T, D, G, N);
  if (ws_bytes < need || (need && !workspace)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const Span in[] = {span(u, rows, D, ldu, es), span(dt, rows, D, lddt, es), span(A, dn, 4),
                     span(Bm, rows, (long long)G * N, ldb, es),
                     span(Cm, rows, (long long)G * N, ldc, es), span(Dw, Dw ? D : 0, 4),
                     span(z, z ? rows : 0, D, ldz, es), span(dt_bias, dt_bias ? D : 0, 4),
                     span(lengths, lengths ? B : 0, 4)};
  const Span out[] = {span(y, rows * D, es), span(hT, hT ? ns : 0, 4),
                      span(workspace, (long long)need, 1)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  // the start state: hT may be exactly it (a block reads its states before it
  // writes them)
  const Span start[] = {span(h0, h0 ? ns : 0, 4)};
  const Span others[] = {out[0], hT == h0 ? span(hT, 0, 4) : out[1], out[2]};
  if (conflicts(start, others)) return KLA_ERR_INVALID_ARG;
  if (T == 0) {
    if (hT && hT != h0)
      e = h0 ? cudaMemcpyAsync(hT, h0, ns * 4, cudaMemcpyDeviceToDevice, st)
             : cudaMemsetAsync(hT, 0, ns * 4, st);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
  }
  const Split sp = fwd_split(B, T, D, G, N);
  Args a = {};
  a.u = u; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.z = z; a.gy = nullptr;
  a.A = A; a.Dw = Dw; a.bias = dt_bias; a.h0 = h0; a.lengths = lengths;
  a.y = y; a.hT = hT;
  a.ends = (float*)workspace;
  a.sums = (float*)((unsigned char*)workspace + up((size_t)B * sp.S * dn * 4));
  a.B = B; a.T = T; a.D = D; a.G = G; a.S = sp.S; a.seg = sp.seg;
  a.softplus = softplus != 0;
  set_rows(a, ldu, lddt, ldb, ldc, ldz, N, es);
  KLA_SSM_DISPATCH((e = run_forward<TY, KN, FULL>(a, st)))
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

size_t kla_ssm_bwd_workspace_size(int B, int T, int D, int G, int N) {
  if (check(B, T, D, G, N, KLA_BF16) != KLA_OK || T == 0) return 0;
  return bwd_plan(B, T, D, G, N).total;
}

kla_status kla_ssm_bwd(const void* u, const void* dt, const float* A, const void* Bm,
                       const void* Cm, const float* Dw, const void* z, const float* dt_bias,
                       const float* h0, const int* lengths, const void* grad_y,
                       const float* grad_hT, void* grad_u, void* grad_dt, float* grad_A,
                       void* grad_B, void* grad_C, float* grad_D, void* grad_z,
                       float* grad_dt_bias, float* grad_h0, int B, int T, int D, int G, int N,
                       long long ldu, long long lddt, long long ldb, long long ldc,
                       long long ldz, int softplus, int dtype, void* workspace, size_t ws_bytes,
                       void* stream) {
  kla_status s = check(B, T, D, G, N, dtype);
  if (s != KLA_OK) return s;
  const void* const ptrs[] = {A, Dw, dt_bias, h0, lengths, grad_y, grad_hT, grad_u, grad_dt,
                              grad_A, grad_B, grad_C, grad_D, grad_z, grad_dt_bias, grad_h0,
                              workspace};
  if (misaligned(ptrs) || rows_misplaced(u, dt, Bm, Cm, z, elem(dtype))) return KLA_ERR_INVALID_ARG;
  if (!grad_A || (z && T > 0 && !grad_z)) return KLA_ERR_INVALID_ARG;
  const long long rows = (long long)B * T, dn = (long long)D * N, ns = B * dn;
  if (T > 0) {
    if (!u || !dt || !A || !Bm || !Cm || !grad_y || !grad_u || !grad_dt || !grad_B || !grad_C)
      return KLA_ERR_INVALID_ARG;
    if (!pitches_ok(rows, D, G, N, ldu, lddt, ldb, ldc, ldz, z != nullptr))
      return KLA_ERR_INVALID_ARG;
  }
  const size_t need = kla_ssm_bwd_workspace_size(B, T, D, G, N);
  if (ws_bytes < need || (need && !workspace)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long gn = (long long)G * N;
  const Span in[] = {span(u, rows, D, ldu, es), span(dt, rows, D, lddt, es), span(A, dn, 4),
                     span(Bm, rows, gn, ldb, es), span(Cm, rows, gn, ldc, es),
                     span(Dw, Dw ? D : 0, 4), span(z, z ? rows : 0, D, ldz, es),
                     span(dt_bias, dt_bias ? D : 0, 4), span(h0, h0 ? ns : 0, 4),
                     span(lengths, lengths ? B : 0, 4), span(grad_y, rows * D, es),
                     span(grad_hT, grad_hT ? ns : 0, 4)};
  const Span out[] = {span(grad_u, rows * D, es), span(grad_dt, rows * D, es),
                      span(grad_A, dn, 4), span(grad_B, rows * gn, es),
                      span(grad_C, rows * gn, es), span(grad_D, grad_D ? D : 0, 4),
                      span(grad_z, grad_z ? rows * D : 0, es),
                      span(grad_dt_bias, grad_dt_bias ? D : 0, 4),
                      span(grad_h0, grad_h0 ? ns : 0, 4), span(workspace, (long long)need, 1)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  if (T == 0) {
    e = cudaMemsetAsync(grad_A, 0, dn * 4, st);
    if (e == cudaSuccess && grad_D) e = cudaMemsetAsync(grad_D, 0, (size_t)D * 4, st);
    if (e == cudaSuccess && grad_dt_bias) e = cudaMemsetAsync(grad_dt_bias, 0, (size_t)D * 4, st);
    if (e == cudaSuccess && grad_h0)
      e = grad_hT ? cudaMemcpyAsync(grad_h0, grad_hT, ns * 4, cudaMemcpyDeviceToDevice, st)
                  : cudaMemsetAsync(grad_h0, 0, ns * 4, st);
    return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
  }
  BwdArgs q = {};
  Args& a = q.f;
  a.u = u; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.z = z; a.gy = grad_y;
  a.A = A; a.Dw = Dw; a.bias = dt_bias; a.h0 = h0; a.lengths = lengths;
  a.B = B; a.T = T; a.D = D; a.G = G;
  a.softplus = softplus != 0;
  set_rows(a, ldu, lddt, ldb, ldc, ldz, N, es);
  q.ghT = grad_hT;
  q.du = grad_u; q.ddt = grad_dt; q.dz = grad_z; q.dh0 = grad_h0;
  const BwdPlan w = bwd_plan(B, T, D, G, N);
  KLA_SSM_DISPATCH((e = run_backward<TY, KN>(q, w, (unsigned char*)workspace, grad_A, grad_D,
                                             grad_dt_bias, grad_B, grad_C, st)))
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

kla_status kla_ssm_step(const void* u, const void* dt, const float* A, const void* Bm,
                        const void* Cm, const float* Dw, const void* z, const float* dt_bias,
                        float* state, void* y, int B, int D, int G, int N, long long ldu,
                        long long lddt, long long ldb, long long ldc, long long ldz,
                        int softplus, int dtype, void* stream) {
  kla_status s = check(B, 1, D, G, N, dtype);
  if (s != KLA_OK) return s;
  if (!u || !dt || !A || !Bm || !Cm || !state || !y) return KLA_ERR_INVALID_ARG;
  const void* const ptrs[] = {A, Dw, dt_bias, state, y};
  if (misaligned(ptrs) || rows_misplaced(u, dt, Bm, Cm, z, elem(dtype))) return KLA_ERR_INVALID_ARG;
  if (!pitches_ok(B, D, G, N, ldu, lddt, ldb, ldc, ldz, z != nullptr)) return KLA_ERR_INVALID_ARG;
  const int es = elem(dtype);
  const long long dn = (long long)D * N, gn = (long long)G * N;
  const Span in[] = {span(u, B, D, ldu, es), span(dt, B, D, lddt, es), span(A, dn, 4),
                     span(Bm, B, gn, ldb, es), span(Cm, B, gn, ldc, es),
                     span(Dw, Dw ? D : 0, 4), span(z, z ? B : 0, D, ldz, es),
                     span(dt_bias, dt_bias ? D : 0, 4)};
  const Span out[] = {span(state, B * dn, 4), span(y, (long long)B * D, es)};
  if (conflicts(in, out)) return KLA_ERR_INVALID_ARG;
  Args a = {};
  a.u = u; a.dt = dt; a.Bm = Bm; a.Cm = Cm; a.z = z;
  a.A = A; a.Dw = Dw; a.bias = dt_bias; a.y = y;
  a.B = B; a.T = 1; a.D = D; a.G = G;
  a.softplus = softplus != 0;
  set_rows(a, ldu, lddt, ldb, ldc, ldz, N, es);
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e = cudaSuccess;
  KLA_SSM_DISPATCH((e = run_step<TY, KN>(a, state, st)))
  return e == cudaSuccess ? KLA_OK : KLA_ERR_CUDA;
}

}  // extern "C"
