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
// 16 / G ... d / (2 G) threads of a row are adjacent lanes and sum over it by
// shuffles.  A CTA takes whole tokens, queries' and keys' heads alike, so
// the angles' sines and cosines are computed once per token and pair and
// shared through shared memory, while the first rows are on their way.
//
// Angles: the position times the fp32 frequency is exact in 64 bits up to
// 53 bits, so the reduction to turns in [-1/2, 1/2] is made there and only
// the reduced angle is rounded to 32 bits (error below 2^-24 of a turn at
// any int32 position).
#include "qk_norm.cuh"

namespace ckda {
namespace qkn {

constexpr int kThreads = 256;

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
__device__ __forceinline__ void turn(float* x, float* y, const float2* cs, int a, int interleaved,
                                     float sgn) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      const float2 w = cs[a + i];
      const float s = sgn * w.y, x0 = x[i], y0 = y[i];
      x[i] = x0 * w.x - y0 * s;
      y[i] = y0 * w.x + x0 * s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2 * G; i += 2) {
      float* z = i < G ? x + i : y + i - G;
      const float2 w = cs[(a + i) >> 1];
      const float s = sgn * w.y, x0 = z[0], y0 = z[1];
      z[0] = x0 * w.x - y0 * s;
      z[1] = y0 * w.x + x0 * s;
    }
  }
}

// (c |x|^2 + eps)^(-1/2); 0 for a row of zeros when eps is 0, whose output
// and gradient are then zeros.
__device__ __forceinline__ float inv_norm(float ss, const Args& p) {
  const float m = fmaf(ss, p.c, p.eps);
  return m == 0.f ? 0.f : rsqrtf(m);
}

// cos and sin of pos[t] * inv_freq[p] for `nt` tokens from t0.
__device__ __forceinline__ void angles(const Args& p, int64_t t0, int nt, float2* cs) {
  const int half = p.rot / 2;
  constexpr double kInv2Pi = 0.15915494309189533577;
  for (int e = threadIdx.x; e < nt * half; e += kThreads) {
    const int t = e / half, i = e - t * half;
    double turns = (double)__ldg(p.pos + t0 + t) * (double)__ldg(p.inv_freq + i) * kInv2Pi;
    turns -= rint(turns);
    float s, c;
    sincospif(2.0f * (float)turns, &s, &c);
    cs[e] = make_float2(c, s);
  }
}

template <typename Tin, typename Tout, int D, int G>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);       // threads per row
  constexpr int RPP = kThreads / TPR;    // rows per pass
  extern __shared__ float2 cs[];
  const int heads = p.Hq + p.Hk;
  const int c = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  float wq[2 * G], wk[2 * G];
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) {
    const int ch = i < G ? a + i : b + i - G;
    wq[i] = p.wq != nullptr ? __ldg(p.wq + ch) : 1.f;
    wk[i] = p.wk != nullptr ? __ldg(p.wk + ch) : 1.f;
  }
  const int64_t t0 = (int64_t)blockIdx.x * p.tok_cta;
  const int nt = (int)min((int64_t)p.tok_cta, p.tokens - t0);
  const int nrows = nt * heads;
  // (every thread of a row's lanes takes the same trips, so the shuffles meet)
  for (int r0 = 0; r0 < nrows; r0 += RPP) {
    const int row = r0 + rg;
    const bool ok = row < nrows;
    const int t = ok ? row / heads : 0, hh = ok ? row - t * heads : 0;
    const bool isq = hh < p.Hq;
    float x[G], y[G];
#pragma unroll
    for (int i = 0; i < G; ++i) x[i] = y[i] = 0.f;
    if (ok) {
      const Tin* src = isq ? static_cast<const Tin*>(p.q) + (t0 + t) * p.q_stride + (int64_t)hh * D
                           : static_cast<const Tin*>(p.k) + (t0 + t) * p.k_stride +
                                 (int64_t)(hh - p.Hq) * D;
      load_unit<Tin, G>(src + a, x);
      load_unit<Tin, G>(src + b, y);
    }
    if (r0 == 0) {
      if (p.rot > 0) angles(p, t0, nt, cs);
      __syncthreads();
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < G; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
    for (int o = TPR / 2; o >= 1; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const float r = inv_norm(ss, p);
#pragma unroll
    for (int i = 0; i < G; ++i) {
      x[i] *= r * (isq ? wq[i] : wk[i]);
      y[i] *= r * (isq ? wq[G + i] : wk[G + i]);
    }
    if (trn) turn<G>(x, y, cs + t * (p.rot / 2), a, p.interleaved, 1.f);
    if (ok) {
      Tout* dst = isq ? static_cast<Tout*>(p.oq) + ((t0 + t) * p.Hq + hh) * D
                      : static_cast<Tout*>(p.ok) + ((t0 + t) * p.Hk + hh - p.Hq) * D;
      store_unit<Tout, G>(dst + a, x);
      store_unit<Tout, G>(dst + b, y);
    }
  }
}

// The CTAs walk the token groups with a stride of the grid, so that each adds
// its rows' shares of dw up in registers and leaves one partial sum per
// weight; dw_kernel adds those in a fixed order.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Args p) {
  constexpr int TPR = D / (2 * G);
  constexpr int RPP = kThreads / TPR;
  extern __shared__ float2 cs[];
  __shared__ float sw[2][kThreads / 32][D];
  const int heads = p.Hq + p.Hk;
  const int c = threadIdx.x % TPR, rg = threadIdx.x / TPR;
  int a, b;
  bool trn;
  units<G>(c, p.rot, p.interleaved, &a, &b, &trn);
  float wq[2 * G], wk[2 * G], dwq[2 * G], dwk[2 * G];
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) {
    const int ch = i < G ? a + i : b + i - G;
    wq[i] = p.wq != nullptr ? __ldg(p.wq + ch) : 1.f;
    wk[i] = p.wk != nullptr ? __ldg(p.wk + ch) : 1.f;
    dwq[i] = dwk[i] = 0.f;
  }
  for (int64_t t0 = (int64_t)blockIdx.x * p.tok_cta; t0 < p.tokens;
       t0 += (int64_t)gridDim.x * p.tok_cta) {
    const int nt = (int)min((int64_t)p.tok_cta, p.tokens - t0);
    const int nrows = nt * heads;
    for (int r0 = 0; r0 < nrows; r0 += RPP) {
      const int row = r0 + rg;
      const bool ok = row < nrows;
      const int t = ok ? row / heads : 0, hh = ok ? row - t * heads : 0;
      const bool isq = hh < p.Hq;
      float x[G], y[G], u[G], w[G];
#pragma unroll
      for (int i = 0; i < G; ++i) x[i] = y[i] = u[i] = w[i] = 0.f;
      const int64_t at = isq ? ((t0 + t) * p.Hq + hh) * D : ((t0 + t) * p.Hk + hh - p.Hq) * D;
      if (ok) {
        const T* src = isq ? static_cast<const T*>(p.q) + (t0 + t) * p.q_stride + (int64_t)hh * D
                           : static_cast<const T*>(p.k) + (t0 + t) * p.k_stride +
                                 (int64_t)(hh - p.Hq) * D;
        const T* gr = static_cast<const T*>(isq ? p.gq : p.gk) + at;
        load_unit<T, G>(src + a, x);
        load_unit<T, G>(src + b, y);
        load_unit<T, G>(gr + a, u);
        load_unit<T, G>(gr + b, w);
      }
      if (r0 == 0 && p.rot > 0) {
        __syncthreads();  // the last tokens' angles have been read
        angles(p, t0, nt, cs);
        __syncthreads();
      }
      if (trn) turn<G>(u, w, cs + t * (p.rot / 2), a, p.interleaved, -1.f);
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int i = 0; i < G; ++i) ss = fmaf(x[i], x[i], fmaf(y[i], y[i], ss));
#pragma unroll
      for (int i = 0; i < G; ++i) {
        dot = fmaf(x[i] * u[i], isq ? wq[i] : wk[i], dot);
        dot = fmaf(y[i] * w[i], isq ? wq[G + i] : wk[G + i], dot);
      }
#pragma unroll
      for (int o = TPR / 2; o >= 1; o >>= 1) {
        ss += __shfl_xor_sync(0xffffffffu, ss, o);
        dot += __shfl_xor_sync(0xffffffffu, dot, o);
      }
      const float r = inv_norm(ss, p);
      const float m = p.c * r * r * r * dot;
      if (p.part != nullptr && ok) {
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const float e = u[i] * (x[i] * r), f = w[i] * (y[i] * r);
          if (isq) {
            dwq[i] += e;
            dwq[G + i] += f;
          } else {
            dwk[i] += e;
            dwk[G + i] += f;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < G; ++i) {
        u[i] = fmaf(r * (isq ? wq[i] : wk[i]), u[i], -m * x[i]);
        w[i] = fmaf(r * (isq ? wq[G + i] : wk[G + i]), w[i], -m * y[i]);
      }
      if (ok) {
        T* dst = static_cast<T*>(isq ? p.oq : p.ok) + at;
        store_unit<T, G>(dst + a, u);
        store_unit<T, G>(dst + b, w);
      }
    }
  }
  if (p.part == nullptr) return;
  // lanes c, c + TPR, ... of a warp hold the same channels
#pragma unroll
  for (int i = 0; i < 2 * G; ++i) {
#pragma unroll
    for (int o = TPR; o < 32; o <<= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
    }
    const int ch = i < G ? a + i : b + i - G;
    if ((threadIdx.x & 31) < TPR) {
      sw[0][threadIdx.x / 32][ch] = dwq[i];
      sw[1][threadIdx.x / 32][ch] = dwk[i];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += kThreads) {
    const int which = e / D, ch = e - which * D;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) s += sw[which][w][ch];
    p.part[((size_t)blockIdx.x * 2 + which) * D + ch] = s;
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

// Tokens per CTA: enough rows for every thread, at most 32 tokens (so that
// the angles of 64 pairs each take 16 KB of shared memory).
static int tokens_per_cta(int heads, int rpp) {
  int t = (rpp + heads - 1) / heads;
  return t < 1 ? 1 : (t > 32 ? 32 : t);
}

constexpr int kBwdGrid = 148 * 4;

static int bwd_grid(int64_t tokens, int tok_cta) {
  const int64_t groups = (tokens + tok_cta - 1) / tok_cta;
  return (int)(groups < kBwdGrid ? groups : kBwdGrid);
}

template <typename Tin, typename Tout, int D, int G>
static cudaError_t launch_fwd(Args p, cudaStream_t st) {
  p.tok_cta = tokens_per_cta(p.Hq + p.Hk, kThreads / (D / (2 * G)));
  const unsigned grid = (unsigned)((p.tokens + p.tok_cta - 1) / p.tok_cta);
  fwd_kernel<Tin, Tout, D, G><<<grid, kThreads, (size_t)p.tok_cta * p.rot / 2 * 8, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, int G>
static cudaError_t launch_bwd(Args p, float* dwq, float* dwk, cudaStream_t st) {
  p.tok_cta = tokens_per_cta(p.Hq + p.Hk, kThreads / (D / (2 * G)));
  const int grid = bwd_grid(p.tokens, p.tok_cta);  // 0 without tokens: dw = 0
  cudaError_t e = cudaSuccess;
  if (grid > 0) {
    bwd_kernel<T, D, G><<<grid, kThreads, (size_t)p.tok_cta * p.rot / 2 * 8, st>>>(p);
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
