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
// SM per channel and token, three times what their bytes (u, dt, z, y in bf16)
// take of HBM.
//
// Split: a thread holds 4 states of 2 channels (their B and C are read once
// for both, and packed fp32 does two states an instruction), the N/4 threads
// of a channel lie side by side in a warp, and a block's channels walk the
// tokens in tiles.  Some warps run the recurrence; helper warps prepare the
// next tile (softplus, dt' u) and finish the previous one (skip, gate, store),
// so the two kinds of work overlap.  With few channels the sequence is cut into
// segments: their end states from zero starts in parallel (MODE LOCAL), a short
// chain over segments, then all of them again from their true starts.
//
// Measured, 8 x 4096 x 2048 x 16 bf16: 445 us, where the exponentials alone
// take 235 and with the softplus and the gate 280.  Two blocks an SM keep the
// special function unit 68 % busy over all SMs (256 blocks on 148), issue slots
// 51 %, the shared-memory pipe 48 %: a mix in which moving work from one to
// another lost (operands stored twice, 464 us; B and C kept in bf16, 462; an
// eighth or a quarter of the exponentials as polynomials, 464 and 481 when all
// on the special function unit took 466).
// 1 x 4096 x 2048 x 16, cut into segments: 99 us.
#include "kla_layer.cuh"

namespace kla {
namespace ssm {

using namespace layer;

constexpr float kLog2e = 1.4426950408889634f;
// ex2.approx is low on average, and a product of many decays adds that up.
// Measured (relative): by 0.5e-8 for exponents from -0.003 to -0.0001, 2.4e-8 from
// -0.05 to -0.005, 1.4 to 2e-8 to -0.5, 5e-8 below -1.  A token's decays get a
// constant added to their exponent, in the multiply-add that forms it, that takes
// 0.6e-8 away where a thread's exponents are small and 1.6e-8 elsewhere.  One
// constant a thread and segment, by the first token of the first tile that it
// comes to: one for all (2.3e-8) leaves memories of 300 tokens and more farther
// off than none (8 x 1024 tokens: states 4.2e-6 from the definition, 3.5e-6 with
// none, 2.9e-6 so), one a tile takes longer (backward 580 us, 573 so, 570 with one
// for all).  8 x 239 tokens: dA 2.7e-6 with none, 1.1e-6 so.  A step of 0 still
// has the decay 1.  (The decays of whole segments go without: carried().)
__device__ __forceinline__ float lift(float x) { return x > -4e-3f ? 0.9e-8f : 2.3e-8f; }
// A log2 e, -inf taken to the lowest finite value: the steps of 0 that stand
// for tokens that do not exist leave the state as it is for A = -inf, too.
__device__ __forceinline__ float rate(float A) {
  const float a = A * kLog2e;
  return a < -3.402823466e38f ? -3.402823466e38f : a;  // (NaN stays)
}
// 2^x h for the decay 2^x of many tokens, as 2^{x/2} h 2^{x/2}: the factor alone
// may leave fp32's range where the product does not.  A state of 0 stays 0
// under any growth.
__device__ __forceinline__ float carried(float x, float h) {
  const float f = ex2(0.5f * x);
  return h == 0.f ? 0.f : f * h * f;
}
constexpr int kTile = 32;     // segments are multiples of this many tokens
constexpr int kCkpt = 8;      // tokens between the backward's saved states, and of its tiles

// FULL: y, hT.  LOCAL: end states of the segments from zero starts.  CKPT: those
// and the states on the way.
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
  // before every kCkpt-th token, with the sequence's ceil(T/kCkpt) side by side:
  float* ckpt;   // [D][N] state, from a zero start of the segment where S > 1
  float* cums;   // [D] sum of dt' since the segment's start (S > 1)
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
  // tiles with tokens that exist; those behind leave the state as it is
  const int ntile = t_live > t_lo ? (t_live - t_lo + TK - 1) / TK : 0;
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
        Quad d4 = quad(dn[i].get()) + quad(bias), x4 = quad(xn[i].get());
        if (sp) d4 = softplus4(d4);
        // tokens that do not exist, and channels past the last, step by 0:
        // their state stays as it is
        float4 d = flat(d4);
        if (ends) {
          const int n = t0 + tt < t_live ? m : 0;
          if (n < 1) d.x = 0.f;
          if (n < 2) d.y = 0.f;
          if (n < 3) d.z = 0.f;
          if (n < 4) d.w = 0.f;
        }
        if (!REV)
          x4 = x4 * quad(d);
        else if (has_z)
          x4 = x4 * silu4(quad(zn[i].get()));
        const float4 x = flat(x4);
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
          Quad v = quad(*reinterpret_cast<const float4*>(sy + (tt0 + i * TS) * CH + c));
          v = fma4(quad(skip), quad(xs[i].get()), v);
          if (has_z) v = v * silu4(quad(zs[i].get()));
          IO<T>::st4(py, flat(v));
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
          Quad w = quad(*reinterpret_cast<const float4*>(sy + tt * CH + c));
          w = fma4(quad(skip), quad(xs[i].get()), w);
          if (has_z) w = w * silu4(quad(zs[i].get()));
          v = flat(w);
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
    if (MODE == FULL) {
      if (ntile > 0) finish(ntile - 1, xp, zp);
      if (m > 0)
        for (int t = t_lo + ntile * TK + tt0; t < t_hi; t += TS)
          st4(y + (long long)t * p.D, make_float4(0.f, 0.f, 0.f, 0.f), m, vec);
    }
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
      a2[k][0] = pack2(rate(v.x), rate(v.y));
      a2[k][1] = pack2(rate(v.z), rate(v.w));
      const float* from = nullptr;
      if (MODE != LOCAL) {
        if (p.S > 1)
          from = MODE == FULL ? p.ends + ((long long)b * p.S + sg) * p.D * N + at : nullptr;
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
  f32x2 up;  // what lifts the exponents of the tokens' decays
  auto scan = [&](int k) {
    const float* sd = s_d + (k & 1) * TK * CH + cc;
    const float* sx = s_x + (k & 1) * TK * CH + cc;
    const float* sb = s_b + (k & 1) * TK * N + nl * 4;
    const float* sc = s_c + (k & 1) * TK * N + nl * 4;
    float* sy = s_y + (k & 1) * TK * CH + cc;
    constexpr int UN = MODE == FULL ? Shape<N>::UN : kCkpt;
    static_assert(MODE != CKPT || UN == kCkpt, "a state is saved before every group");
#pragma unroll 1
    for (int tt = 0; tt < TK; tt += UN) {
      if (MODE == CKPT) {
        const int t = t_lo + k * TK + tt;
        const long long at = (long long)b * ((p.T + kCkpt - 1) / kCkpt) + t / kCkpt;
        if (t < t_hi) {
          save(p.ckpt + at * p.D * N);
          if (p.S > 1 && nl == 0) {
#pragma unroll
            for (int c = 0; c < CPT; ++c)
              if (cc + c < nc) p.cums[at * p.D + c0 + cc + c] = sum[c];
          }
        }
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
        const float2 dv = *reinterpret_cast<const float2*>(sd + t * CH);
        const float2 xv = *reinterpret_cast<const float2*>(sx + t * CH);
        const float d[CPT] = {dv.x, dv.y}, x[CPT] = {xv.x, xv.y};
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
          const f32x2 d2 = both(d[c]), w2 = both(x[c]);
          const f32x2 e0 = ex2_2(fma2(d2, a2[c][0], up));
          const f32x2 e1 = ex2_2(fma2(d2, a2[c][1], up));
          if (REV) {
            h[c][0] = mul2(e0, fma2(w2, cv[0], h[c][0]));
            h[c][1] = mul2(e1, fma2(w2, cv[1], h[c][1]));
          } else {
            h[c][0] = fma2(e0, h[c][0], mul2(w2, bv[0]));
            h[c][1] = fma2(e1, h[c][1], mul2(w2, bv[1]));
          }
          if (MODE != FULL) sum[c] += d[c];
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
  // (without a tile: whatever lies there, for nothing; a guard costs 1 %)
  up = both(lift(s_d[(first & 1) * TK * CH + cc] * unpack2(a2[0][0]).x));
  for (int i = 0; i < ntile; ++i) {
    scan(first + dir * i);
    __syncthreads();
  }
  if (MODE == LOCAL || (MODE == CKPT && p.S > 1)) {
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
chain_kernel(const float* __restrict__ A, const float* __restrict__ h0, float* ends,
             const float* __restrict__ sums, int S, int D, int N, long long total) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  if (id >= total) return;
  const long long dn = (long long)D * N;
  const long long b = id / dn, at = id % dn;
  const int d = (int)(at / N);
  const float a2 = rate(A[at]);
  float h = h0 ? h0[id] : 0.f;
  // eight segments' values are loaded before the first is needed
  for (int i0 = 0; i0 < S; i0 += 8) {
    float own[8], sum[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j, s = REV ? S - 1 - i : i;
      own[j] = sum[j] = 0.f;
      if (i < S - 1) {
        own[j] = ends[(b * S + s) * dn + at];
        sum[j] = sums[(b * S + s) * D + d];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + j, s = REV ? S - 1 - i : i;
      if (i < S) ends[(b * S + s) * dn + at] = h;
      h = carried(a2 * sum[j], h) + own[j];
    }
  }
}

// ---------------------------------------------------------------- backward
//
// With g = gy silu(z) and the adjoint state e (what flows into h[t-1]):
//   dh = e + C g;  dC = sum_d h g;  dB = sum_d dh dt' u;  e <- a dh
//   du = D g + dt' sum_n dh B;  ddt' = u sum_n dh B + sum_n A h[t-1] e
//   dA = sum_t dt' h[t-1] e;  dz = gy y0 silu'(z);  dD = sum g u
// Three passes: the states before every 8th token (scan_kernel, CKPT), the
// adjoint states between segments where the sequence is cut (LOCAL, REV), and
// bwd_kernel, which goes back through each segment 8 tokens at a time.
//
// bwd_kernel is split like the scan: recurrence warps with 4 states of 2
// channels a thread (pairs of states packed), helper warps for everything that
// is one value a channel.  A recurrence thread rebuilds 4 tokens' decays and
// states in registers from the saved state (the first 4 of the 8 twice) and
// walks them back.  Sums over n cross the lanes of a channel with 4 tokens
// exchanged at once.  Sums over channels (dB, dC) cross the other lanes: there
// register s of a thread holds state s ^ (its place among the channels), from
// copies of B and C in that order, so that every exchange sends fixed
// registers and needs no selection.  What bounds it are issue slots (about 170
// instructions a token for a thread's 8 states, 50 % of the slots used with two
// recurrence warps a scheduler, which is what the registers allow).
// 2 x 4096 x 2048 x 16 bf16: about 380 us of the pass's 575.
// dB and dC leave as one part a channel tile, dA, dD and dt_bias as one a
// segment, and reduce kernels add the parts in order: no atomics, the same
// bits every time.

template <int N>
struct BwdShape {
  static constexpr int LPC = N / 4;              // lanes of a channel
  static constexpr int CL = 32 / LPC;            // channel places of a warp
  static constexpr int PB = CL < 4 ? CL : 4;     // orders of 4 states
  static constexpr int CW = N == 8 ? 2 : 4;      // recurrence warps
  static constexpr int HW = 2;                   // helper warps
  static constexpr int CPW = 2 * CL;             // channels of a warp
  static constexpr int CH = CW * CPW;            // channels of a block
  static constexpr int NT = (CW + HW) * 32;
  // shared memory of one buffer, in floats: dt', x, g; the three sums; B and
  // C in every order; the warps' dB and dC
  static constexpr int XS = kCkpt * CH;
  static constexpr int BS = kCkpt * PB * N;
  static constexpr int PS = CW * kCkpt * 2 * N;
  static constexpr int BUF = 6 * XS + 2 * BS + PS;
};

struct BwdArgs {
  Args f;                       // forward arguments; S, seg, ends, sums of the adjoint
  int fS, fseg;                 // the forward's segments
  const float* fends;           // [B][fS][D][N] their start states
  const float* ghT;
  void *du, *ddt, *dz;
  float* dh0;
  float* part_bc;               // [TPG][B][T][G][2N]
  float* part_a;                // [B*S][D][N]
  float* part_d;                // [B*S][2][D]: dD, ddt_bias
};

// v[q][j], j < 4 tokens of 6 quantities: lane nl ends with the sum over the LPC
// lanes of a channel of token (nl & 3) (LPC >= 4: in v[q][0]) or of tokens nl,
// nl + 2 (LPC = 2).  All quantities cross together, so that their exchanges
// wait for each other once a round.
template <int LPC>
__device__ __forceinline__ void token_sums(float (&v)[6][4], int nl) {
  if constexpr (LPC == 2) {
#pragma unroll
    for (int q = 0; q < 6; ++q)
#pragma unroll
      for (int j = 0; j < 4; j += 2) {  // tokens j, j + 1
        const float keep = (nl & 1) ? v[q][j + 1] : v[q][j];
        const float send = (nl & 1) ? v[q][j] : v[q][j + 1];
        v[q][j] = keep + __shfl_xor_sync(0xffffffffu, send, 1);
      }
  } else {
#pragma unroll
    for (int off = LPC / 2; off >= 4; off >>= 1)
#pragma unroll
      for (int q = 0; q < 6; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[q][j] += __shfl_xor_sync(0xffffffffu, v[q][j], off);
#pragma unroll
    for (int off = 2; off > 0; off >>= 1) {
      const bool up = (nl & off) != 0;
      float got[6][2];
#pragma unroll
      for (int q = 0; q < 6; ++q)
#pragma unroll
        for (int j = 0; j < off; ++j)
          got[q][j] = __shfl_xor_sync(0xffffffffu, up ? v[q][j] : v[q][j + off], off);
#pragma unroll
      for (int q = 0; q < 6; ++q)
#pragma unroll
        for (int j = 0; j < off; ++j) v[q][j] = (up ? v[q][j + off] : v[q][j]) + got[q][j];
    }
  }
}

// (v.x, v.y, v.z, v.w) with register s holding component s ^ o; its own inverse.
__device__ __forceinline__ float4 reorder(float4 v, int o) {
  if (o & 1) v = make_float4(v.y, v.x, v.w, v.z);
  if (o & 2) v = make_float4(v.z, v.w, v.x, v.y);
  return v;
}

template <typename T, int N>
__global__ void __launch_bounds__(BwdShape<N>::NT, 2)
bwd_kernel(BwdArgs q) {
  using Sh = BwdShape<N>;
  constexpr int LPC = Sh::LPC, CL = Sh::CL, PB = Sh::PB, CW = Sh::CW, CPW = Sh::CPW;
  constexpr int CH = Sh::CH, K = kCkpt, NH = Sh::HW * 32;
  constexpr int XG = K * CH / 4;                   // channel groups of a tile
  constexpr int IX = (XG + NH - 1) / NH;           // of a helper
  constexpr int IB = (K * N / 4 + NH - 1) / NH;
  static_assert((XG % NH == 0 || XG < NH) && NH % (CH / 4) == 0, "helpers share a tile evenly");
  const Args& p = q.f;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  float* const smem = reinterpret_cast<float*>(smem_raw);

  const int Dg = p.D / p.G, TPG = (Dg + CH - 1) / CH;
  const int tiles = TPG * p.G;
  const int ct = blockIdx.x % tiles;
  const int rest = blockIdx.x / tiles;
  const int sg = rest % p.S, b = rest / p.S;
  const int g = ct / TPG;
  const int c0 = g * Dg + (ct % TPG) * CH;
  const int nc = min(CH, (g + 1) * Dg - c0);
  const int t_lo = sg * p.seg, t_hi = min(p.T, t_lo + p.seg);
  const int t_live = min(t_hi, live_tokens(p.lengths, b, p.T));
  // tiles with tokens that exist: behind them the gradients are zeros, and the
  // adjoint state comes through as it is
  const int ntile = t_live > t_lo ? (t_live - t_lo + K - 1) / K : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long row0 = (long long)b * p.T;
  const long long ps = (long long)b * p.S + sg;

  if (warp >= CW) {
    // ------------------------------------------------ helpers
    const int hid = tid - CW * 32;
    const int c = (hid % (CH / 4)) * 4, tt0 = hid / (CH / 4);
    constexpr int TS = NH / (CH / 4);
    const int m = XG < NH && hid >= XG ? 0 : nc - c;
    const bool vec = (Dg & 3) == 0;
    const bool vu = vec && p.vu, vdt = vec && p.vdt, vz = vec && p.vz;
    const bool has_z = p.z != nullptr, sp = p.softplus != 0;
    const T* u = (const T*)p.u + row0 * p.ldu + c0 + c;
    const T* dt = (const T*)p.dt + row0 * p.lddt + c0 + c;
    const T* gy = (const T*)p.gy + row0 * p.D + c0 + c;
    const T* z = has_z ? (const T*)p.z + row0 * p.ldz + c0 + c : nullptr;
    const T* Bm = (const T*)p.Bm + row0 * p.ldb + (long long)g * N;
    const T* Cm = (const T*)p.Cm + row0 * p.ldc + (long long)g * N;
    T* du = (T*)q.du + row0 * p.D + c0 + c;
    T* ddt = (T*)q.ddt + row0 * p.D + c0 + c;
    T* dz = has_z ? (T*)q.dz + row0 * p.D + c0 + c : nullptr;
    float* pbc = q.part_bc + (((long long)(ct % TPG) * p.B + b) * p.T * p.G + g) * 2 * N;
    float4 bias = make_float4(0.f, 0.f, 0.f, 0.f), skip = bias, accD = bias, accT = bias;
    if (p.bias) bias = ld4(p.bias + c0 + c, m, vec);
    if (p.Dw) skip = ld4(p.Dw + c0 + c, m, vec);

    struct Rows {
      Raw4<T> u[IX], dt[IX], gy[IX], z[IX];
    };
    Rows next, cur, done;  // to be staged, in the recurrence, finished
    Raw4<T> bn[IB], cn[IB];
    auto load = [&](int k) {
      const int t0 = t_lo + k * K;
#pragma unroll
      for (int i = 0; i < IX; ++i) {
        const int t = t0 + tt0 + i * TS;
        const int n = t < t_live ? m : 0;
        next.u[i] = ld_raw4(u + (long long)t * p.ldu, n, vu);
        next.dt[i] = ld_raw4(dt + (long long)t * p.lddt, n, vdt);
        next.gy[i] = ld_raw4(gy + (long long)t * p.D, n, vec);
        if (has_z) next.z[i] = ld_raw4(z + (long long)t * p.ldz, n, vz);
      }
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        const int j = hid + i * NH, t = t0 + j / (N / 4), n = (j % (N / 4)) * 4;
        const int have = j < K * N / 4 && t < t_live ? 4 : 0;
        bn[i] = ld_raw4(Bm + (long long)t * p.ldb + n, have, p.vb);
        cn[i] = ld_raw4(Cm + (long long)t * p.ldc + n, have, p.vc);
      }
    };
    auto stage = [&](int k) {
      float* buf = smem + (k & 1) * Sh::BUF;
      const int t0 = t_lo + k * K;
#pragma unroll
      for (int i = 0; i < IX; ++i) {
        const int tt = tt0 + i * TS;
        if (XG < NH && hid >= XG) continue;
        Quad d4 = quad(next.dt[i].get()) + quad(bias), g4 = quad(next.gy[i].get());
        if (sp) d4 = softplus4(d4);
        float4 d = flat(d4);
        const int n = t0 + tt < t_live ? m : 0;  // zero steps as in the scan
        if (n < 1) d.x = 0.f;
        if (n < 2) d.y = 0.f;
        if (n < 3) d.z = 0.f;
        if (n < 4) d.w = 0.f;
        if (has_z) g4 = g4 * silu4(quad(next.z[i].get()));
        const float4 x = flat(quad(next.u[i].get()) * quad(d)), gg = flat(g4);
        float* o = buf + tt * CH + c;
        *reinterpret_cast<float4*>(o) = d;
        *reinterpret_cast<float4*>(o + Sh::XS) = x;
        *reinterpret_cast<float4*>(o + 2 * Sh::XS) = gg;
      }
#pragma unroll
      for (int i = 0; i < IB; ++i) {
        const int j = hid + i * NH;
        if (j < K * N / 4) {
          float* o = buf + 6 * Sh::XS + (j / (N / 4)) * PB * N + (j % (N / 4)) * 4;
#pragma unroll
          for (int r = 0; r < PB; ++r) {
            *reinterpret_cast<float4*>(o + r * N) = reorder(bn[i].get(), r);
            *reinterpret_cast<float4*>(o + Sh::BS + r * N) = reorder(cn[i].get(), r);
          }
        }
      }
    };
    auto finish = [&](int k) {
      const float* buf = smem + (k & 1) * Sh::BUF;
      const int t0 = t_lo + k * K;
#pragma unroll
      for (int i = 0; i < IX; ++i) {
        const int tt = tt0 + i * TS, t = t0 + tt;
        if (t >= t_hi || m <= 0) continue;
        float4 vdu = make_float4(0.f, 0.f, 0.f, 0.f), vddt = vdu, vdz = vdu;
        if (t < t_live) {
          const float* o = buf + tt * CH + c;
          auto at = [&](int j) {
            return quad(*reinterpret_cast<const float4*>(o + j * Sh::XS));
          };
          const Quad d = at(0), gg = at(2), sB = at(3), uu = quad(done.u[i].get());
          vdu = flat(fma4(quad(skip), gg, sB * d));
          // the sum over A h e is with A log2 e
          Quad ds = fma4(sB, uu, at(4) * all4(0.6931471805599453f));
          if (sp) ds = ds * sigmoid4(quad(done.dt[i].get()) + quad(bias));
          vddt = flat(ds);
          accD = flat(fma4(gg, uu, quad(accD)));
          accT = flat(quad(accT) + ds);
          if (has_z) {
            const Quad zz = quad(done.z[i].get()), s = sigmoid4(zz), one = all4(1.f);
            const Quad slope = s * fma4(zz, fma4(s, all4(-1.f), one), one);
            vdz = flat(quad(done.gy[i].get()) * fma4(quad(skip), uu, at(5)) * slope);
          }
        }
        st4(du + (long long)t * p.D, vdu, m, vec);
        st4(ddt + (long long)t * p.D, vddt, m, vec);
        if (has_z) st4(dz + (long long)t * p.D, vdz, m, vec);
      }
      // dB, dC: the warps' sums in order (for a token that does not exist they
      // may be 0 times an infinite state)
      const float* bc = buf + 6 * Sh::XS + 2 * Sh::BS;
#pragma unroll
      for (int i = 0; i < K * 2 * N / 4; i += NH) {
        const int j = (i + hid) * 4, tt = j / (2 * N), n = j % (2 * N);
        if (i + hid < K * 2 * N / 4 && t0 + tt < t_hi) {
          float4 v = *reinterpret_cast<const float4*>(bc + j);
#pragma unroll
          for (int w = 1; w < CW; ++w) {
            const float4 a = *reinterpret_cast<const float4*>(bc + w * K * 2 * N + j);
            v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
          }
          if (t0 + tt >= t_live) v = make_float4(0.f, 0.f, 0.f, 0.f);
          *reinterpret_cast<float4*>(pbc + (long long)(t0 + tt) * p.G * 2 * N + n) = v;
        }
      }
    };
    if (ntile > 0) {
      load(ntile - 1);
      stage(ntile - 1);
      cur = next;
      if (ntile > 1) load(ntile - 2);
    }
    __syncthreads();
    for (int k = ntile - 1; k >= 0; --k) {
      if (k + 1 < ntile) finish(k + 1);  // before its buffer is filled anew
      if (k > 0) stage(k - 1);
      done = cur;
      cur = next;
      if (k > 1) load(k - 2);
      __syncthreads();
    }
    if (ntile > 0) finish(0);
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const int t_end = t_lo + ntile * K;
    if (m > 0)
      for (int t = t_end + tt0; t < t_hi; t += TS < K ? TS : K) {
        st4(du + (long long)t * p.D, zero, m, vec);
        st4(ddt + (long long)t * p.D, zero, m, vec);
        if (has_z) st4(dz + (long long)t * p.D, zero, m, vec);
      }
    for (int t = t_end + hid / (N / 2); t < t_hi; t += NH / (N / 2))
      *reinterpret_cast<float4*>(pbc + (long long)t * p.G * 2 * N + hid % (N / 2) * 4) = zero;
    // dD, ddt_bias: over the threads that kept the same 4 channels, through
    // the other buffer
    float* red = smem + Sh::BUF;
    asm volatile("bar.sync 1, %0;" ::"n"(NH) : "memory");
    *reinterpret_cast<float4*>(red + hid * 4) = accD;
    *reinterpret_cast<float4*>(red + NH * 4 + hid * 4) = accT;
    asm volatile("bar.sync 1, %0;" ::"n"(NH) : "memory");
    for (int i = hid; i < 2 * CH; i += NH) {
      const int w = i / CH, cc = i % CH;
      if (cc < nc) {
        float s = 0.f;
        for (int r = cc / 4; r < NH; r += CH / 4) s += red[(w * NH + r) * 4 + (cc & 3)];
        q.part_d[(ps * 2 + w) * p.D + c0 + cc] = s;
      }
    }
    return;
  }

  // -------------------------------------------------- recurrence
  const int nl = lane % LPC, cg = lane / LPC, cc = warp * CPW + cg * 2;
  const int ord = cg & (PB - 1);  // register s holds state nl * 4 + (s ^ ord)
  auto row = [&](const float* base, int k) {
    if (!base || cc + k >= nc) return make_float4(0.f, 0.f, 0.f, 0.f);
    return reorder(*reinterpret_cast<const float4*>(base + (long long)(c0 + cc + k) * N + nl * 4),
                   ord);
  };
  f32x2 a2[2][2], e[2][2], dA[2][2];
  const float* from = p.S > 1 ? p.ends + ps * p.D * N
                      : q.ghT ? q.ghT + (long long)b * p.D * N
                              : nullptr;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float4 v = row(p.A, c), w = row(from, c);
    a2[c][0] = pack2(rate(v.x), rate(v.y));
    a2[c][1] = pack2(rate(v.z), rate(v.w));
    e[c][0] = pack2(w.x, w.y);
    e[c][1] = pack2(w.z, w.w);
    dA[c][0] = dA[c][1] = pack2(0.f, 0.f);
  }
  const int nck = (p.T + K - 1) / K;
  // a tile's saved states come to places of this thread's own, one tile ahead:
  // [2][4][CW * 32] rows (state and segment start of both channels), [2][CW * 32]
  // sums of dt'
  float4* const s_h = reinterpret_cast<float4*>(smem + 2 * Sh::BUF) + tid;
  float2* const s_s = reinterpret_cast<float2*>(s_h - tid + 8 * CW * 32) + tid;
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (cc + c >= nc) {  // a channel that does not exist is never copied
#pragma unroll
      for (int i = 0; i < 8; i += 2) s_h[(i + c) * CW * 32] = make_float4(0.f, 0.f, 0.f, 0.f);
      reinterpret_cast<float*>(s_s)[c] = reinterpret_cast<float*>(s_s + CW * 32)[c] = 0.f;
    }
  auto fetch = [&](int k) {
    const int t = t_lo + k * K;
    const long long ck = (long long)b * nck + t / K;
    float4* v = s_h + (k & 1) * 4 * CW * 32;
    float* sum = reinterpret_cast<float*>(s_s + (k & 1) * CW * 32);
    const long long at = (long long)(c0 + cc) * N + nl * 4;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      if (cc + c < nc) {
        cp16(v + c * CW * 32, p.ckpt + ck * p.D * N + at + c * N);
        if (q.fS > 1) {
          cp16(v + (2 + c) * CW * 32,
               q.fends + ((long long)b * q.fS + t / q.fseg) * p.D * N + at + c * N);
          cp4(sum + c, p.cums + ck * p.D + c0 + cc + c);
        }
      }
    }
    cp_commit();
  };
  if (ntile > 0) fetch(ntile - 1);
  __syncthreads();
  const f32x2 up = both(lift(smem[((ntile - 1) & 1) * Sh::BUF + cc] * unpack2(a2[0][0]).x));
  for (int k = ntile - 1; k >= 0; --k) {
    float* buf = smem + (k & 1) * Sh::BUF;
    const float* sd = buf + cc;
    const float* sb = buf + 6 * Sh::XS + ord * N + nl * 4;
    // the state before the tile's first token
    f32x2 h0[2][2];
    if (k > 0) {
      fetch(k - 1);
      cp_wait<1>();
    } else {
      cp_wait<0>();
    }
    {
      const float4* v = s_h + (k & 1) * 4 * CW * 32;
      const float2 s = s_s[(k & 1) * CW * 32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float4 h = reorder(v[c * CW * 32], ord);
        h0[c][0] = pack2(h.x, h.y);
        h0[c][1] = pack2(h.z, h.w);
        if (q.fS > 1) {  // saved from a zero start: add what the segment's start left
          const float4 w = reorder(v[(2 + c) * CW * 32], ord);
          const f32x2 s2 = c ? pack2(s.y, s.y) : pack2(s.x, s.x);
          const float2 x0 = unpack2(mul2(s2, a2[c][0])), x1 = unpack2(mul2(s2, a2[c][1]));
          h0[c][0] = add2(h0[c][0], pack2(carried(x0.x, w.x), carried(x0.y, w.y)));
          h0[c][1] = add2(h0[c][1], pack2(carried(x1.x, w.z), carried(x1.y, w.w)));
        }
      }
    }
    f32x2 tA[2][2];
    tA[0][0] = tA[0][1] = tA[1][0] = tA[1][1] = pack2(0.f, 0.f);
    // one token forward: its decays, and h moved on
    auto forward = [&](int t, f32x2 (&h)[2][2], f32x2 (&a)[2][2]) {
      const float2 d = *reinterpret_cast<const float2*>(sd + t * CH);
      const float2 x = *reinterpret_cast<const float2*>(sd + Sh::XS + t * CH);
      const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(sb + t * PB * N);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const f32x2 d2 = c ? pack2(d.y, d.y) : pack2(d.x, d.x);
        const f32x2 x2 = c ? pack2(x.y, x.y) : pack2(x.x, x.x);
        a[c][0] = ex2_2(fma2(d2, a2[c][0], up));
        a[c][1] = ex2_2(fma2(d2, a2[c][1], up));
        h[c][0] = fma2(a[c][0], h[c][0], mul2(x2, bv.x));
        h[c][1] = fma2(a[c][1], h[c][1], mul2(x2, bv.y));
      }
    };
    auto half = [&](int tb, const f32x2 (&hs)[2][2]) {
      f32x2 a[4][2][2], h[5][2][2];
#pragma unroll
      for (int c = 0; c < 2; ++c) { h[0][c][0] = hs[c][0]; h[0][c][1] = hs[c][1]; }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < 2; ++c) { h[i + 1][c][0] = h[i][c][0]; h[i + 1][c][1] = h[i][c][1]; }
        forward(tb + i, h[i + 1], a[i]);
      }
      float v6[6][4];    // sum dh B, sum A h e, y0 of two channels
      f32x2 bc[4][4];    // dB, dC of the thread's 4 states
#pragma unroll
      for (int i = 3; i >= 0; --i) {
        const int t = tb + i;
        const float2 d = *reinterpret_cast<const float2*>(sd + t * CH);
        const float2 x = *reinterpret_cast<const float2*>(sd + Sh::XS + t * CH);
        const float2 gg = *reinterpret_cast<const float2*>(sd + 2 * Sh::XS + t * CH);
        const ulonglong2 bv = *reinterpret_cast<const ulonglong2*>(sb + t * PB * N);
        const ulonglong2 cv = *reinterpret_cast<const ulonglong2*>(sb + Sh::BS + t * PB * N);
        f32x2 wB[2], wC[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const f32x2 d2 = c ? pack2(d.y, d.y) : pack2(d.x, d.x);
          const f32x2 x2 = c ? pack2(x.y, x.y) : pack2(x.x, x.x);
          const f32x2 g2 = c ? pack2(gg.y, gg.y) : pack2(gg.x, gg.x);
          const f32x2 dh0 = fma2(cv.x, g2, e[c][0]), dh1 = fma2(cv.y, g2, e[c][1]);
          wB[0] = c ? fma2(dh0, x2, wB[0]) : mul2(dh0, x2);
          wB[1] = c ? fma2(dh1, x2, wB[1]) : mul2(dh1, x2);
          wC[0] = c ? fma2(h[i + 1][c][0], g2, wC[0]) : mul2(h[i + 1][c][0], g2);
          wC[1] = c ? fma2(h[i + 1][c][1], g2, wC[1]) : mul2(h[i + 1][c][1], g2);
          const float2 y = unpack2(fma2(cv.y, h[i + 1][c][1], mul2(cv.x, h[i + 1][c][0])));
          v6[4 + c][i] = y.x + y.y;
          const float2 sB = unpack2(fma2(dh1, bv.y, mul2(dh0, bv.x)));
          v6[c][i] = sB.x + sB.y;
          e[c][0] = mul2(a[i][c][0], dh0);
          e[c][1] = mul2(a[i][c][1], dh1);
          const f32x2 f0 = mul2(e[c][0], h[i][c][0]), f1 = mul2(e[c][1], h[i][c][1]);
          const float2 sA = unpack2(fma2(a2[c][1], f1, mul2(a2[c][0], f0)));
          v6[2 + c][i] = sA.x + sA.y;
          tA[c][0] = fma2(d2, f0, tA[c][0]);
          tA[c][1] = fma2(d2, f1, tA[c][1]);
        }
        bc[i][0] = wB[0]; bc[i][1] = wB[1];
        bc[i][2] = wC[0]; bc[i][3] = wC[1];
      }
      // dB, dC over the warp's channels, the 4 tokens of a round together
      float r[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          r[i][j] = __shfl_xor_sync(0xffffffffu, unpack2(bc[i][j]).y, LPC);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] += unpack2(bc[i][j]).x;
      float* o = buf + 6 * Sh::XS + 2 * Sh::BS + (warp * K + tb) * 2 * N + nl * 4;
      if constexpr (CL == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          o[i * 2 * N + ord] = r[i][0];
          o[i * 2 * N + (2 ^ ord)] = r[i][1];
          o[i * 2 * N + N + ord] = r[i][2];
          o[i * 2 * N + N + (2 ^ ord)] = r[i][3];
        }
      } else {
        float x[4][2];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            x[i][j] = __shfl_xor_sync(0xffffffffu, r[i][2 * j + 1], 2 * LPC);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) x[i][j] += r[i][2 * j];
        if constexpr (CL == 4) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            o[i * 2 * N + ord] = x[i][0];
            o[i * 2 * N + N + ord] = x[i][1];
          }
        } else {
          const bool up = (cg & 4) != 0;
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = __shfl_xor_sync(0xffffffffu, up ? x[i][0] : x[i][1], 4 * LPC);
#pragma unroll
          for (int i = 0; i < 4; ++i) w[i] += up ? x[i][1] : x[i][0];
          if constexpr (CL == 16)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] += __shfl_xor_sync(0xffffffffu, w[i], 8 * LPC);
          if (CL == 8 || cg < 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i * 2 * N + (up ? N : 0) + ord] = w[i];
        }
      }
      token_sums<LPC>(v6, nl);
      if (LPC <= 4 || nl < 4) {
#pragma unroll
        for (int j = 0; j < (LPC == 2 ? 4 : 1); j += 2) {
          float* o = buf + 3 * Sh::XS + (tb + j + nl) * CH + cc;
          *reinterpret_cast<float2*>(o) = make_float2(v6[0][j], v6[1][j]);
          *reinterpret_cast<float2*>(o + Sh::XS) = make_float2(v6[2][j], v6[3][j]);
          *reinterpret_cast<float2*>(o + 2 * Sh::XS) = make_float2(v6[4][j], v6[5][j]);
        }
      }
    };
    f32x2 hm[2][2], skip_a[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) { hm[c][0] = h0[c][0]; hm[c][1] = h0[c][1]; }
#pragma unroll
    for (int i = 0; i < 4; ++i) forward(i, hm, skip_a);
    half(4, hm);
    half(0, h0);
#pragma unroll
    for (int c = 0; c < 2; ++c) {  // per tile first: shorter chains of additions
      dA[c][0] = add2(dA[c][0], tA[c][0]);
      dA[c][1] = add2(dA[c][1], tA[c][1]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    if (cc + c >= nc) continue;
    const long long at = (long long)(c0 + cc + c) * N + nl * 4;
    const float2 v0 = unpack2(dA[c][0]), v1 = unpack2(dA[c][1]);
    *reinterpret_cast<float4*>(q.part_a + ps * p.D * N + at) =
        reorder(make_float4(v0.x, v0.y, v1.x, v1.y), ord);
    if (q.dh0 && sg == 0) {
      const float2 e0 = unpack2(e[c][0]), e1 = unpack2(e[c][1]);
      *reinterpret_cast<float4*>(q.dh0 + (long long)b * p.D * N + at) =
          reorder(make_float4(e0.x, e0.y, e1.x, e1.y), ord);
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
// Bound by HBM: one read and one write of the state.  A thread holds 4 states,
// the N/4 threads of a channel lie side by side, and a block takes neighbouring
// channels of one sequence (64 x 2048 x 16: 6.6 us, in 2.3 waves of blocks; x 64 states: 22 us, 6.2 TB/s;
// two channels a thread: 6.5 and 23 us, and slower for a single sequence).
template <typename T, int N>
__global__ void __launch_bounds__(256)
step_kernel(Args p, float* __restrict__ S, unsigned tiles) {
  constexpr int LPC = N / 4, CB = 256 / LPC;
  const unsigned bb = blockIdx.x / tiles;
  const long long b = bb;
  const int d = (int)(blockIdx.x - bb * tiles) * CB + threadIdx.x / LPC;
  const int nl = threadIdx.x % LPC;
  const bool live = d < p.D;
  float* const at = S + (b * p.D + d) * N + nl * 4;
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f), A = h, bv = h, cv = h;
  float raw = 0.f, u = 0.f, z = 0.f, skip = 0.f;
  if (live) {
    const int g = d / (p.D / p.G);
    h = *reinterpret_cast<const float4*>(at);
    A = *reinterpret_cast<const float4*>(p.A + (long long)d * N + nl * 4);
    const long long gn = (long long)g * N + nl * 4;
    bv = ld4((const T*)p.Bm + b * p.ldb + gn, 4, p.vb);
    cv = ld4((const T*)p.Cm + b * p.ldc + gn, 4, p.vc);
    raw = IO<T>::ld((const T*)p.dt + b * p.lddt + d);
    u = IO<T>::ld((const T*)p.u + b * p.ldu + d);
    if (p.z) z = IO<T>::ld((const T*)p.z + b * p.ldz + d);
    if (p.bias) raw += p.bias[d];
    if (p.Dw) skip = p.Dw[d];
  }
  const float s = p.softplus ? softplus(raw) : raw, x = s * u;
  const float up = lift(s * rate(A.x));
  h.x = fmaf(ex2(fmaf(s, rate(A.x), up)), h.x, x * bv.x);
  h.y = fmaf(ex2(fmaf(s, rate(A.y), up)), h.y, x * bv.y);
  h.z = fmaf(ex2(fmaf(s, rate(A.z), up)), h.z, x * bv.z);
  h.w = fmaf(ex2(fmaf(s, rate(A.w), up)), h.w, x * bv.w);
  float y = fmaf(cv.w, h.w, fmaf(cv.z, h.z, fmaf(cv.y, h.y, cv.x * h.x)));
#pragma unroll
  for (int off = LPC / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
  if (!live) return;
  *reinterpret_cast<float4*>(at) = h;
  if (nl == 0) {
    y = fmaf(skip, u, y);
    if (p.z) y *= silu(z);
    IO<T>::st((T*)p.y + b * p.D + d, y);
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

// Segments of a sequence.  `tiles` blocks would run uncut; a block's time a
// token is, in units of a scan block that shares an SM, 1.2 alone and n on an
// SM with n of them (8 x 4096 x 2048 x 16, two an SM: 220 clocks a token; one:
// 130).  A cut scan first needs all segments but one for their end states
// (about 0.8 of a scan each), so the parts have to bring more than that: the
// fewest segments of at least 128 tokens whose modelled time is within 3 % of
// the best.
//   ends: what a segment's end state costs beside `own`, its time in the pass
//   itself (1 for the scan; 3.5 for the backward pass: 780 clocks, two an SM)
static Split split(long long tiles, int T, double own, double ends) {
  auto block = [](long long n) { return n <= 148 ? 1.2 : (double)((n + 147) / 148); };
  auto time = [&](int S) {
    return (own * block(tiles * S) + (S > 1 ? ends * block(tiles * (S - 1)) : 0.0)) / S;
  };
  const int most = T / 128 < 64 ? T / 128 : 64;
  double best = time(1);
  for (int S = 2; S <= most; ++S) best = time(S) < best ? time(S) : best;
  int S = 1;
  while (S < most && time(S) > 1.03 * best) ++S;
  const int blocks = (T + kTile - 1) / kTile;
  const int seg = ((blocks + S - 1) / S) * kTile;
  return Split{(T + seg - 1) / seg, seg};
}

static long long tiles_of(int D, int G, int CH) { return (long long)G * ((D / G + CH - 1) / CH); }

static Split fwd_split(int B, int T, int D, int G, int N) {
  return split(B * tiles_of(D, G, channels(N)), T, 1.0, 0.8);
}
// the saved states need no second pass: the backward kernel adds what a
// segment's start leaves
static Split save_split(int B, int T, int D, int G, int N) {
  return split(B * tiles_of(D, G, channels(N)), T, 0.8, 0.0);
}
static Split bwd_split(int B, int T, int D, int G, int N) {
  return split(B * tiles_of(D, G, bwd_channels(N)), T, 3.5, 0.8);
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

template <typename T, int N>
static cudaError_t run_forward(const Args& a, cudaStream_t st) {
  if (a.S > 1) {
    cudaError_t e = run_scan<T, N, LOCAL, false>(a, st);
    if (e == cudaSuccess) e = run_chain<false>(a, N, a.h0, st);
    if (e != cudaSuccess) return e;
  }
  return run_scan<T, N, FULL, false>(a, st);
}

struct BwdPlan {
  Split f, r;
  int TPG;
  size_t ckpt, cums, fends, fsums, rends, rsums, bc, pa, pd, total;
};

static BwdPlan bwd_plan(int B, int T, int D, int G, int N) {
  BwdPlan w;
  w.f = save_split(B, T, D, G, N);
  w.r = bwd_split(B, T, D, G, N);
  w.TPG = (D / G + bwd_channels(N) - 1) / bwd_channels(N);
  const size_t dn = (size_t)D * N * 4, nck = (size_t)B * ((T + kCkpt - 1) / kCkpt);
  size_t at = 0;
  auto take = [&](size_t n) { size_t r = at; at += up(n); return r; };
  w.ckpt = take(nck * dn);
  w.cums = take(w.f.S > 1 ? nck * D * 4 : 0);
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
  f.cums = (float*)(ws + w.cums);
  f.S = w.f.S; f.seg = w.f.seg;
  f.ends = (float*)(ws + w.fends);
  f.sums = (float*)(ws + w.fsums);
  cudaError_t e = run_scan<T, N, CKPT, false>(f, st);
  if (e == cudaSuccess && f.S > 1) e = run_chain<false>(f, N, f.h0, st);
  if (e != cudaSuccess) return e;
  q.fS = f.S; q.fseg = f.seg; q.fends = f.ends;
  q.f.ckpt = f.ckpt; q.f.cums = f.cums;
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
  using Sh = BwdShape<N>;
  // two buffers, and two tiles' saved states of every recurrence thread
  constexpr size_t smem = 2 * (Sh::BUF * sizeof(float) + Sh::CW * 32 * (4 * 16 + 8));
  static_assert(Sh::BUF >= Sh::HW * 32 * 8, "room for the helpers' sums");
  const long long blocks = tiles_of(q.f.D, q.f.G, Sh::CH) * q.f.B * q.f.S;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto k = bwd_kernel<T, N>;
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  k<<<(unsigned)blocks, Sh::NT, smem, st>>>(q);
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
  constexpr int per = 256 / (N / 4);  // channels of a block
  const long long tiles = (a.D + per - 1) / per, blocks = tiles * a.B;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  step_kernel<T, N><<<(unsigned)blocks, 256, 0, st>>>(a, S, (unsigned)tiles);
  return cudaGetLastError();
}

static kla_status check(int B, int T, int D, int G, int N, int dtype) {
  if (B < 1 || T < 0 || D < 1 || G < 1 || N < 1 || D % G != 0 || !dtype_ok(dtype))
    return KLA_ERR_INVALID_ARG;
  if (!size_ok((long long)B * (T > 0 ? T : 1), (long long)D) ||
      !size_ok((long long)B * D, (long long)N * (T / kCkpt + 1)) ||
      !size_ok((long long)B * (T > 0 ? T : 1), 2LL * G * N * 4))
    return KLA_ERR_INVALID_ARG;
  if (T > kMaxTokens || D > kMaxTokens || (N != 8 && N != 16 && N != 32 && N != 64))
    return KLA_ERR_UNSUPPORTED;
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
  const void* const ptrs[] = {A, Dw, dt_bias, h0, y, hT, workspace};
  if (misaligned(ptrs) || misplaced(lengths, 4) || rows_misplaced(u, dt, Bm, Cm, z, elem(dtype))) return KLA_ERR_INVALID_ARG;
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
  KLA_SSM_DISPATCH((e = run_forward<TY, KN>(a, st)))
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
  const void* const ptrs[] = {A, Dw, dt_bias, h0, grad_y, grad_hT, grad_u, grad_dt, grad_A,
                              grad_B, grad_C, grad_D, grad_z, grad_dt_bias, grad_h0, workspace};
  if (misaligned(ptrs) || misplaced(lengths, 4) || rows_misplaced(u, dt, Bm, Cm, z, elem(dtype))) return KLA_ERR_INVALID_ARG;
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
