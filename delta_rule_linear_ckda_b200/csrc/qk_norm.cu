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
// Both are bound by HBM bandwidth: a row is read once and written once.  A
// thread owns two units of G adjacent channels (G = 8: 16 bytes of bf16) that
// hold whole pairs, so that the turn needs no exchange between threads; the
// d / (2 G) threads of a row are adjacent lanes and sum over it by shuffles.
// A warp takes some heads of one token, queries' and keys' alike, so that a
// thread computes the sines and cosines of its own pairs once for all of them
// and no barrier stands between the rows; the next rows are requested before
// the present ones are used.
//
// Angles: the turns, position * inv_freq / (2 pi), and their reduction to
// [-1/2, 1/2] are computed in 64 bits (error below 2^-50 of the turns), and
// only the reduced angle is rounded to 32 bits, to 2^-25 of a turn.
#include "qk_norm.cuh"

namespace ckda {
namespace qkn {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

template <typename T, int G>
__device__ __forceinline__ void load_unit(const T* p, float* x);
template <>
__device__ __forceinline__ void load_unit<float, 4>(const float* p, float* x) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
template <>
__device__ __forceinline__ void load_unit<float, 8>(const float* p, float* x) { load8_f32(p, x); }
template <>
__device__ __forceinline__ void load_unit<__nv_bfloat16, 4>(const __nv_bfloat16* p, float* x) {
  const float4 a = load4_f32(p);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
}
template <>
__device__ __forceinline__ void load_unit<__nv_bfloat16, 8>(const __nv_bfloat16* p, float* x) {
  load8_f32(p, x);
}

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

// A warp's rows: heads [h0, h1) of token t, RPW of them at a time.
struct Unit {
  int64_t t;
  int h0, h1;
};

__device__ __forceinline__ Unit unit_of(const Args& p, int64_t u) {
  Unit x;
  const int groups = (p.Hq + p.Hk + p.heads_warp - 1) / p.heads_warp;
  x.t = u / groups;
  x.h0 = (int)(u - x.t * groups) * p.heads_warp;
  x.h1 = min(p.Hq + p.Hk, x.h0 + p.heads_warp);
  return x;
}

template <int G>
struct Weights {
  float q[2 * G], k[2 * G];
  __device__ __forceinline__ void load(const Args& p, int a, int b) {
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
      const int ch = i < G ? a + i : b + i - G;
      q[i] = p.wq != nullptr ? __ldg(p.wq + ch) : 1.f;
      k[i] = p.wk != nullptr ? __ldg(p.wk + ch) : 1.f;
    }
  }
};

template <typename T, int D>
__device__ __forceinline__ const T* row_in(const Args& p, int64_t t, int hh) {
  return hh < p.Hq ? static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)hh * D
                   : static_cast<const T*>(p.k) + t * p.k_stride + (int64_t)(hh - p.Hq) * D;
}

// A row's offset in a contiguous [tokens, heads, D] tensor of its own.
template <int D>
__device__ __forceinline__ int64_t row_at(const Args& p, int64_t t, int hh) {
  return hh < p.Hq ? (t * p.Hq + hh) * D : (t * p.Hk + hh - p.Hq) * D;
}

template <typename Tin, typename Tout, int D, int G>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);  // threads per row
  constexpr int RPW = 32 / TPR;     // rows per warp and pass
  const int lane = threadIdx.x & 31;
  const int c = lane % TPR, rg = lane / TPR;
  const int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (u >= p.units) return;
  const Unit un = unit_of(p, u);
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  float x[G], y[G];
  auto fetch = [&](int hh) {
#pragma unroll
    for (int i = 0; i < G; ++i) x[i] = y[i] = 0.f;
    if (hh < un.h1) {
      const Tin* src = row_in<Tin, D>(p, un.t, hh);
      load_unit<Tin, G>(src + a, x);
      load_unit<Tin, G>(src + b, y);
    }
  };
  fetch(un.h0 + rg);
  Weights<G> w;
  w.load(p, a, b);
  float2 cs[G];
  if (trn) angles<G>(p, un.t, a, cs);
  // (every lane takes the same trips, so the shuffles meet)
  for (int r0 = un.h0; r0 < un.h1; r0 += RPW) {
    const int hh = r0 + rg;
    const bool isq = hh < p.Hq;
    float u0[G], v0[G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
      u0[i] = x[i];
      v0[i] = y[i];
    }
    fetch(hh + RPW);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) ss = fmaf(u0[i], u0[i], fmaf(v0[i], v0[i], ss));
#pragma unroll
    for (int o = TPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = inv_norm(ss, p);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      u0[i] *= r * (isq ? w.q[i] : w.k[i]);
      v0[i] *= r * (isq ? w.q[G + i] : w.k[G + i]);
    }
    if (trn) turn<G>(u0, v0, cs, p.interleaved, 1.f);
    if (hh < un.h1) {
      Tout* dst = static_cast<Tout*>(isq ? p.oq : p.ok) + row_at<D>(p, un.t, hh);
      store_unit<Tout, G>(dst + a, u0);
      store_unit<Tout, G>(dst + b, v0);
    }
  }
}

// The warps walk the units with a stride of the grid, so that each adds its
// rows' shares of dw up in registers and a CTA leaves one partial sum per
// weight; dw_kernel adds those in a fixed order.
template <typename T, int D, int G, bool SUMS>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);
  constexpr int RPW = 32 / TPR;
  __shared__ float sw[2][kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = lane % TPR, rg = lane / TPR;
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  Weights<G> w;
  w.load(p, a, b);
  float dwq[2 * G], dwk[2 * G];
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) dwq[i] = dwk[i] = 0.f;
  for (int64_t uu = (int64_t)blockIdx.x * kWarps + warp; uu < p.units;
       uu += (int64_t)gridDim.x * kWarps) {
    const Unit un = unit_of(p, uu);
    float2 cs[G];
    if (trn) angles<G>(p, un.t, a, cs);
    for (int r0 = un.h0; r0 < un.h1; r0 += RPW) {
      const int hh = r0 + rg;
      const bool ok = hh < un.h1, isq = hh < p.Hq;
      float x[G], y[G], u[G], v[G];
#pragma unroll
      for (int i = 0; i < G; ++i) x[i] = y[i] = u[i] = v[i] = 0.f;
      const int64_t at = row_at<D>(p, un.t, hh);
      if (ok) {
        const T* src = row_in<T, D>(p, un.t, hh);
        const T* gr = static_cast<const T*>(isq ? p.gq : p.gk) + at;
        load_unit<T, G>(src + a, x);
        load_unit<T, G>(src + b, y);
        load_unit<T, G>(gr + a, u);
        load_unit<T, G>(gr + b, v);
      }
      if (trn) turn<G>(u, v, cs, p.interleaved, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int i = 0; i < G; ++i) {
        dot = fmaf(x[i] * u[i], isq ? w.q[i] : w.k[i], dot);
        dot = fmaf(y[i] * v[i], isq ? w.q[G + i] : w.k[G + i], dot);
      }
#pragma unroll
      for (int o = TPR / 2; o >= 1; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float r = inv_norm(ss, p);
      const float m = p.c * r * r * r * dot;
      if (SUMS) {  // (a lane without a row adds zeros)
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const float e = u[i] * (x[i] * r), f = v[i] * (y[i] * r);
          dwq[i] += isq ? e : 0.f;
          dwq[G + i] += isq ? f : 0.f;
          dwk[i] += isq ? 0.f : e;
          dwk[G + i] += isq ? 0.f : f;
        }
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        u[i] = fmaf(r * (isq ? w.q[i] : w.k[i]), u[i], -m * x[i]);
        v[i] = fmaf(r * (isq ? w.q[G + i] : w.k[G + i]), v[i], -m * y[i]);
      }
      if (ok) {
        T* dst = static_cast<T*>(isq ? p.oq : p.ok) + at;
        store_unit<T, G>(dst + a, u);
        store_unit<T, G>(dst + b, v);
      }
    }
  }
  if constexpr (SUMS) {
    // lanes c, c + TPR, ... of a warp hold the same channels
#pragma unroll
    for (int i = 0; i < 2 * G; ++i) {
#pragma unroll
      for (int o = TPR; o < 32; o <<= 1) {
        dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
        dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
      }
      const int ch = i < G ? a + i : b + i - G;
      if (lane < TPR) {
        sw[0][warp][ch] = dwq[i];
        sw[1][warp][ch] = dwk[i];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
      const int which = e / D, ch = e - which * D;
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) s += sw[which][k][ch];
      p.part[((size_t)blockIdx.x * 2 + which) * D + ch] = s;
    }
  }
}

// dw[ch] = the sum of `n` partial sums: a CTA per 32 channels of one weight,
// 64-bit sums in a fixed order.
__global__ void __launch_bounds__(256) dw_kernel(const float* __restrict__ part, int n, int d,
                                                 float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double red[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ch = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (ch < d)
    for (int i = w; i < n; i += 8) s += (double)part[((size_t)i * 2 + blockIdx.y) * d + ch];
  red[w][lane] = s;
  __syncthreads();
  if (w == 0 && ch < d) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    float* o = blockIdx.y ? dwk : dwq;
    if (o != nullptr) o[ch] = (float)s;
  }
}

constexpr int kBwdGrid = 148 * 4;

// Heads of a token that one warp takes: all of them (in up to 8 passes) when
// the tokens alone give every SM 16 warps, else one pass's.
static void plan(Args* p, int rpw) {
  const int heads = p->Hq + p->Hk;
  const int64_t all = p->tokens * ((heads + 8 * rpw - 1) / (8 * rpw));
  p->heads_warp = all >= 148 * 16 ? 8 * rpw : rpw;
  p->units = p->tokens * ((heads + p->heads_warp - 1) / p->heads_warp);
}

template <typename Tin, typename Tout, int D, int G>
static cudaError_t launch_fwd(Args p, cudaStream_t st) {
  plan(&p, 32 / (D / (2 * G)));
  fwd_kernel<Tin, Tout, D, G><<<(unsigned)((p.units + kWarps - 1) / kWarps), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, int G>
static cudaError_t launch_bwd(Args p, float* dwq, float* dwk, cudaStream_t st) {
  plan(&p, 32 / (D / (2 * G)));
  const int64_t ctas = (p.units + kWarps - 1) / kWarps;
  const int grid = (int)(ctas < kBwdGrid ? ctas : kBwdGrid);  // 0 without tokens: dw = 0
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    if (p.part != nullptr)
      bwd_kernel<T, D, G, true><<<grid, kThreads, 0, st>>>(p);
    else
      bwd_kernel<T, D, G, false><<<(unsigned)ctas, kThreads, 0, st>>>(p);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && p.part != nullptr) {
    dw_kernel<<<dim3((D + 31) / 32, 2), 256, 0, st>>>(p.part, grid, D, dwq, dwk);
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

size_t qk_norm_bwd_workspace_bytes(int d) { return (size_t)qkn::kBwdGrid * 2 * d * 4; }

}  // namespace ckda
