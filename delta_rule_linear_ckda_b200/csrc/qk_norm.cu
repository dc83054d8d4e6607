// Norm of every head of the queries and the keys, and the rotation by
// position, in one pass, and its backward.
//
// Per row x (one token's head, d channels), with c = 1 (unit length) or 1/d
// (unit mean square):
//   r = (c |x|^2 + eps)^(-1/2),  y = (r x) * w,  z = R y,
// R turning the channel pair p of the first `rot` channels by the angle
// pos * inv_freq[p]: pairs (p, p + rot / 2), or (2p, 2p + 1) interleaved.
// Backward, with u = R^T dz (the turn by the opposite angle):
//   dx = r (w * u) - c r^3 x (x . (w * u)),   dw = sum over rows of u * (r x).
//
// Both read a row once and write it once; that traffic is their floor.  At 16384
// tokens, 16 + 16 heads of 128: fp32 forward 89 us, backward 130 (92 and 94 % of
// the copy rate, bound by HBM); bf16 61.5 and 83 (67 and 74 %): with half the
// bytes per row the arithmetic and the angles show, 57 and 61 % of the issue
// slots with the 16 warps that 106 and 128 registers leave an SM, and a warp
// has nothing of its next token in flight.  The last reduction of the weights'
// gradients takes 7 us of the backward.
//
// A thread owns two units of G adjacent channels (G = 8: 16 bytes of bf16)
// that hold whole pairs, so that the turn needs no exchange between threads;
// the d / (2 G) threads of a row are adjacent lanes and sum over it by shuffles.
// A warp takes some of one token's query heads, or key heads, so that a
// thread computes the sines and cosines of its own pairs once for all of them
// and no barrier stands between the rows.  It requests several rows per lane
// at once (64 to 128 bytes) before it uses the first.
//
// Angles: the turns, position * inv_freq / (2 pi), and their reduction to
// [-1/2, 1/2] are computed in 64 bits (error below 2^-50 of the turns), and
// only the reduced angle is rounded to 32 bits, to 2^-25 of a turn.
#include "qk_norm.cuh"

namespace ckda {
namespace qkn {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// G elements as they lie in memory.
template <typename T, int G>
struct Raw {
  static constexpr int kWords = (int)sizeof(T) * G / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint32_t*>(p) + i);
        w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void get(float* x) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < G; ++i) x[i] = __uint_as_float(w[i]);
    }
  }
};

template <typename T, int G>
__device__ __forceinline__ void store_unit(T* p, const float* x) {
  if constexpr (sizeof(T) == 2 && G == 8) {
    uint4 raw;
    uint32_t* u = reinterpret_cast<uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      u[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = raw;
  } else {
#pragma unroll
    for (int i = 0; i < G; i += 4) store4(p + i, make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
  }
}

// The channel offsets of thread c's two units in a row, and whether they turn.
// Split pairs: units u and u + rot / (2 G) for the turned channels; the rest,
// and interleaved pairs, in adjacent units.
template <int G>
__device__ __forceinline__ void units(int c, int rot, int interleaved, int* a, int* b,
                                      bool* turn) {
  const int nrot = rot / (2 * G);  // threads whose units turn
  *turn = c < nrot;
  if (*turn && !interleaved) {
    *a = c * G;
    *b = *a + rot / 2;
  } else {
    *a = 2 * c * G;
    *b = *a + G;
  }
}

// The pairs of a thread's two units turned by (cs.x, sgn * cs.y).
template <int G>
__device__ __forceinline__ void turn(float* x, float* y, const float2* cs, int interleaved,
                                     float sgn) {
#pragma unroll
  for (int i = 0; i < G; ++i) {
    const float c = cs[i].x, s = sgn * cs[i].y;
    if (!interleaved) {
      const float x0 = x[i], y0 = y[i];
      x[i] = x0 * c - y0 * s;
      y[i] = y0 * c + x0 * s;
    } else {
      float* z = 2 * i < G ? x + 2 * i : y + 2 * i - G;
      const float x0 = z[0], y0 = z[1];
      z[0] = x0 * c - y0 * s;
      z[1] = y0 * c + x0 * s;
    }
  }
}

// (c |x|^2 + eps)^(-1/2); 0 for a row of zeros when eps is 0, whose output
// and gradient are then zeros.
__device__ __forceinline__ float inv_norm(float ss, const Args& p) {
  const float m = fmaf(ss, p.c, p.eps);
  return m == 0.f ? 0.f : rsqrtf(m);
}

// cos and sin of pos[t] * inv_freq for a thread's G pairs (unit offset a).
template <int G>
__device__ __forceinline__ void angles(const Args& p, int64_t t, int a, float2* cs) {
  constexpr double kInv2Pi = 0.15915494309189533577;
  const double pos = (double)__ldg(p.pos + t) * kInv2Pi;
  const float* f = p.inv_freq + (p.interleaved ? a / 2 : a);
#pragma unroll
  for (int i = 0; i < G; ++i) {
    double turns = pos * (double)__ldg(f + i);
    turns -= rint(turns);
    sincospif(2.0f * (float)turns, &cs[i].y, &cs[i].x);
  }
}

// A warp's rows: heads [h0, h1) of token t.
struct Unit {
  int64_t t;
  int h0, h1;
};

__device__ __forceinline__ Unit unit_of(const Side& s, int64_t u) {
  Unit x;
  const int groups = (s.H + s.heads_warp - 1) / s.heads_warp;
  x.t = groups == 1 ? u : u / groups;
  x.h0 = (int)(u - x.t * groups) * s.heads_warp;
  x.h1 = min(s.H, x.h0 + s.heads_warp);
  return x;
}

template <int G>
__device__ __forceinline__ void load_w(const float* p, int a, int b, float* w) {
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) w[i] = p != nullptr ? __ldg(p + (i < G ? a + i : b + i - G)) : 1.f;
}

// Rows that a lane requests at once.
template <typename T, bool BWD>
constexpr int kBatch = (sizeof(T) == 2 ? 4 : 2) / (BWD ? 2 : 1);

template <typename Tin, typename Tout, int D, int G>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);  // threads per row
  constexpr int RPW = 32 / TPR;     // rows per warp and pass
  constexpr int NB = kBatch<Tin, false>;
  const int lane = threadIdx.x & 31;
  const int c = lane % TPR, rg = lane / TPR;
  const bool keys = blockIdx.x >= p.s[0].ctas;
  const Side& sd = keys ? p.s[1] : p.s[0];
  const int64_t u =
      (int64_t)(blockIdx.x - (keys ? p.s[0].ctas : 0u)) * kWarps + (threadIdx.x >> 5);
  if (u >= sd.units) return;
  const Unit un = unit_of(sd, u);
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  const Tin* src = static_cast<const Tin*>(sd.x) + un.t * sd.stride;
  Tout* dst = static_cast<Tout*>(sd.out) + un.t * sd.H * D;
  Raw<Tin, G> ra[NB], rb[NB];
  float w[2 * G];
  float2 cs[G];
  // (every lane takes the same trips, so the shuffles meet)
  for (int r0 = un.h0; r0 < un.h1; r0 += RPW * NB) {
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int hh = r0 + n * RPW + rg;
      if (hh < un.h1) {
        ra[n].load(src + (int64_t)hh * D + a);
        rb[n].load(src + (int64_t)hh * D + b);
      } else {
        ra[n].zero();
        rb[n].zero();
      }
    }
    if (r0 == un.h0) {
      load_w<G>(sd.w, a, b, w);
      if (trn) angles<G>(p, un.t, a, cs);
    }
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      if (r0 + n * RPW >= un.h1) break;
      const int hh = r0 + n * RPW + rg;
      float x[G], y[G];
      ra[n].get(x);
      rb[n].get(y);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int o = TPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      const float r = inv_norm(ss, p);
#pragma unroll
      for (int i = 0; i < G; ++i) {
        x[i] *= r * w[i];
        y[i] *= r * w[G + i];
      }
      if (trn) turn<G>(x, y, cs, p.interleaved, 1.f);
      if (hh < un.h1) {
        store_unit<Tout, G>(dst + (int64_t)hh * D + a, x);
        store_unit<Tout, G>(dst + (int64_t)hh * D + b, y);
      }
    }
  }
}

// The warps walk the units of their side with a stride of its CTAs, so that
// each adds its rows' shares of dw up in registers and a CTA leaves one
// partial sum per channel; dw_kernel adds those in a fixed order.
template <typename T, int D, int G, bool SUMS>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);
  constexpr int RPW = 32 / TPR;
  constexpr int NB = kBatch<T, true>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % TPR, rg = lane / TPR;
  const bool keys = blockIdx.x >= p.s[0].ctas;
  const Side& sd = keys ? p.s[1] : p.s[0];
  const unsigned cta = blockIdx.x - (keys ? p.s[0].ctas : 0u);
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  float w[2 * G], dw[SUMS ? 2 * G : 1];
  load_w<G>(sd.w, a, b, w);
  if constexpr (SUMS) {
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) dw[i] = 0.f;
  }
  for (int64_t uu = (int64_t)cta * kWarps + warp; uu < sd.units;
       uu += (int64_t)sd.ctas * kWarps) {
    const Unit un = unit_of(sd, uu);
    const T* src = static_cast<const T*>(sd.x) + un.t * sd.stride;
    const T* gr = static_cast<const T*>(sd.g) + un.t * sd.H * D;
    T* dst = static_cast<T*>(sd.out) + un.t * sd.H * D;
    Raw<T, G> ra[NB], rb[NB], ga[NB], gb[NB];
    float2 cs[G];
    for (int r0 = un.h0; r0 < un.h1; r0 += RPW * NB) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const int hh = r0 + n * RPW + rg;
        if (hh < un.h1) {
          ra[n].load(src + (int64_t)hh * D + a);
          rb[n].load(src + (int64_t)hh * D + b);
          ga[n].load(gr + (int64_t)hh * D + a);
          gb[n].load(gr + (int64_t)hh * D + b);
        } else {
          ra[n].zero();
          rb[n].zero();
          ga[n].zero();
          gb[n].zero();
        }
      }
      if (trn && r0 == un.h0) angles<G>(p, un.t, a, cs);
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        if (r0 + n * RPW >= un.h1) break;
        const int hh = r0 + n * RPW + rg;
        float x[G], y[G], u[G], v[G];
        ra[n].get(x);
        rb[n].get(y);
        ga[n].get(u);
        gb[n].get(v);
        if (trn) turn<G>(u, v, cs, p.interleaved, -1.f);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
          dot = fmaf(x[i] * u[i], w[i], dot);
          dot = fmaf(y[i] * v[i], w[G + i], dot);
        }
#pragma unroll
        for (int o = TPR / 2; o >= 1; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          dot += __shfl_xor_sync(0xffffffffu, dot, o);
        }
        const float r = inv_norm(ss, p);
        // c r^3 x dot as products of x r and r dot, which stay in range where
        // r^3 does not (rows below 1e-13 without an eps)
        const float m = p.c * r * (r * dot);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          x[i] *= r;
          y[i] *= r;
        }
        if constexpr (SUMS) {  // (a lane without a row adds zeros)
#pragma unroll
          for (int i = 0; i < G; ++i) {
            dw[i] = fmaf(u[i], x[i], dw[i]);
            dw[G + i] = fmaf(v[i], y[i], dw[G + i]);
          }
        }
#pragma unroll
        for (int i = 0; i < G; ++i) {
          u[i] = fmaf(r * w[i], u[i], -m * x[i]);
          v[i] = fmaf(r * w[G + i], v[i], -m * y[i]);
        }
        if (hh < un.h1) {
          store_unit<T, G>(dst + (int64_t)hh * D + a, u);
          store_unit<T, G>(dst + (int64_t)hh * D + b, v);
        }
      }
    }
  }
  if constexpr (SUMS) {
    __shared__ float sw[kWarps][D];
    // lanes c, c + TPR, ... of a warp hold the same channels
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
#pragma unroll
      for (int o = TPR; o < 32; o <<= 1) dw[i] += __shfl_xor_sync(0xffffffffu, dw[i], o);
      if (lane < TPR) sw[warp][i < G ? a + i : b + i - G] = dw[i];
    }
    __syncthreads();
    for (int ch = threadIdx.x; ch < D; ch += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += sw[k][ch];
      p.part[(size_t)blockIdx.x * D + ch] = s;
    }
  }
}

// dw[ch] = the sum of the CTAs' partial sums: a CTA per 32 channels of one
// weight, 64-bit sums in a fixed order.  A warp has four partial sums on
// their way at a time: with one, the chain of loads took 26 us for 444 CTAs.
__global__ void __launch_bounds__(1024) dw_kernel(const float* __restrict__ part, int nq, int nk,
                                                  int d, float* __restrict__ dwq,
                                                  float* __restrict__ dwk) {
  __shared__ double red[32][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ch = blockIdx.x * 32 + lane;
  const int i0 = blockIdx.y ? nq : 0, i1 = blockIdx.y ? nq + nk : nq;
  float* o = blockIdx.y ? dwk : dwq;
  if (o == nullptr) return;
  double s = 0.0;
  if (ch < d) {
    for (int i = i0 + w; i < i1; i += 128) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        x[e] = i + 32 * e < i1 ? __ldg(part + (size_t)(i + 32 * e) * d + ch) : 0.f;
      s += ((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3]);
    }
  }
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && ch < d) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += red[i][lane];
    o[ch] = (float)s;
  }
}

// CTAs of a side at most, with sums.  us with 1, 2, 3 and 4 per SM, 32768
// tokens, bf16: 16 query heads of 128 alone 112, 80, 101, 85; 32 + 8 heads of
// 128 245, 181, 182, 186; 32 + 1 241, 170, 177, 175; 16 + 16 of 64 86, 90, 94,
// 96; fp32, 16 + 16 of 128 258, 247, 248, 247.
constexpr int kBwdCtas = 148 * 2;

// Heads of a token that one warp takes: all of them (in up to `most` passes)
// when that leaves every SM three warps of a side, else one pass's.  us with one
// pass / all heads (16 + 16 of 128, bf16), forward: 148 tokens 3.0 / 3.9,
// 296: 4.0 / 4.3, 592: 6.4 / 4.8, 1184: 11.2 / 6.4; backward: 6.1 / 8.0,
// 7.9 / 8.5, 11.8 / 8.9, 19.4 / 11.1; fp32 and 32 + 32 heads change over
// between 296 and 592 tokens too.
static void plan(Args* p, int rpw, int most, unsigned cap) {
  for (Side& s : p->s) {
    const int64_t all = p->tokens * ((s.H + most * rpw - 1) / (most * rpw));
    s.heads_warp = all >= 148 * 3 ? most * rpw : rpw;
    s.units = p->tokens * ((s.H + s.heads_warp - 1) / s.heads_warp);
    const int64_t ctas = (s.units + kWarps - 1) / kWarps;
    s.ctas = cap != 0 && ctas > cap ? cap : (unsigned)ctas;
  }
}

template <typename Tin, typename Tout, int D, int G>
static cudaError_t launch_fwd(Args p, cudaStream_t st) {
  plan(&p, 32 / (D / (2 * G)), 8, 0);
  fwd_kernel<Tin, Tout, D, G><<<p.s[0].ctas + p.s[1].ctas, kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, int G>
static cudaError_t launch_bwd(Args p, float* dwq, float* dwk, cudaStream_t st) {
  plan(&p, 32 / (D / (2 * G)), 8, p.part != nullptr ? kBwdCtas : 0);
  const unsigned grid = p.s[0].ctas + p.s[1].ctas;  // 0 without tokens: dw = 0
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    if (p.part != nullptr)
      bwd_kernel<T, D, G, true><<<grid, kThreads, 0, st>>>(p);
    else
      bwd_kernel<T, D, G, false><<<grid, kThreads, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && p.part != nullptr) {
    dw_kernel<<<dim3((D + 31) / 32, 2), 1024, 0, st>>>(p.part, (int)p.s[0].ctas, (int)p.s[1].ctas, D,
                                                      dwq, dwk);
    e = cudaGetLastError();
  }
  return e;
}

// Units of 8 channels where the turned channels split into them, else 4.
template <typename Tin, typename Tout, int D>
static cudaError_t fwd_g(const Args& p, cudaStream_t st) {
  return p.rot % 16 == 0 ? launch_fwd<Tin, Tout, D, 8>(p, st) : launch_fwd<Tin, Tout, D, 4>(p, st);
}

template <typename Tin, typename Tout>
static cudaError_t fwd_d(const Args& p, cudaStream_t st) {
  switch (p.d) {
    case 16: return fwd_g<Tin, Tout, 16>(p, st);
    case 32: return fwd_g<Tin, Tout, 32>(p, st);
    case 64: return fwd_g<Tin, Tout, 64>(p, st);
    case 128: return fwd_g<Tin, Tout, 128>(p, st);
  }
  return cudaErrorInvalidValue;
}

template <typename T, int D>
static cudaError_t bwd_g(const Args& p, float* dwq, float* dwk, cudaStream_t st) {
  return p.rot % 16 == 0 ? launch_bwd<T, D, 8>(p, dwq, dwk, st)
                         : launch_bwd<T, D, 4>(p, dwq, dwk, st);
}

template <typename T>
static cudaError_t bwd_d(const Args& p, float* dwq, float* dwk, cudaStream_t st) {
  switch (p.d) {
    case 16: return bwd_g<T, 16>(p, dwq, dwk, st);
    case 32: return bwd_g<T, 32>(p, dwq, dwk, st);
    case 64: return bwd_g<T, 64>(p, dwq, dwk, st);
    case 128: return bwd_g<T, 128>(p, dwq, dwk, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace qkn

cudaError_t launch_qk_norm_fwd(const qkn::Args& p, int dtype, int out_dtype, cudaStream_t st) {
  using bf = __nv_bfloat16;
  if (dtype == CKDA_BF16)
    return out_dtype == CKDA_BF16 ? qkn::fwd_d<bf, bf>(p, st) : qkn::fwd_d<bf, float>(p, st);
  return out_dtype == CKDA_BF16 ? qkn::fwd_d<float, bf>(p, st) : qkn::fwd_d<float, float>(p, st);
}

cudaError_t launch_qk_norm_bwd(const qkn::Args& p, int dtype, float* dwq, float* dwk,
                               cudaStream_t st) {
  return dtype == CKDA_BF16 ? qkn::bwd_d<__nv_bfloat16>(p, dwq, dwk, st)
                            : qkn::bwd_d<float>(p, dwq, dwk, st);
}

size_t qk_norm_bwd_workspace_bytes(int d) { return (size_t)qkn::kBwdCtas * 2 * d * 4; }

}  // namespace ckda
