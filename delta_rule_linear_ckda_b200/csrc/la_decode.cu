// One token of head-decay linear attention, in place on the fp32 state:
//   S <- a S + k v^T,   o = S^T q.
//
// The step moves 8 d_k d_v bytes of state per (sequence, head) and does four
// fp32 operations per element: it is bound by HBM bandwidth (B = 256, H = 32,
// d = 128: 160 us, the copy rate; issue slots 17 %).  Each thread
// owns four adjacent columns (one 16-byte vector) of NR rows and requests
// them all before it uses one.  Unlike the delta-rule steps nothing has to
// be summed over the rows before the state can be written back, so the new
// state leaves at once and the column sums follow it.
//
// A CTA owns CV columns of one (sequence, head): all of them or, for few heads
// of the largest state, 16 (the columns are independent), so that one token
// of one sequence uses d_v / 16 = 8 times as many SMs.  The choice and both
// sides' times stand at launch_la_decode.
#include "la_common.cuh"

namespace ckda {
namespace la {

template <int DK, int CV>
struct StepShape {
  static constexpr int kCpr = CV / 4;  // threads across a row
  static constexpr int kThreads = (DK * CV / 4 < 256) ? DK * CV / 4 : 256;
  static constexpr int kRpp = kThreads / kCpr;  // rows covered per pass
  static constexpr int kRows = DK / kRpp;       // rows per thread
  static_assert(DK % kRpp == 0 && kThreads >= DK, "row split");
};

template <int DK, int CV, typename Tin, typename Tout>
__global__ void __launch_bounds__(StepShape<DK, CV>::kThreads)
la_step_kernel(const Tin* __restrict__ q, const Tin* __restrict__ k, const Tin* __restrict__ v,
               const float* __restrict__ alpha, int per_head, float* __restrict__ S,
               Tout* __restrict__ out, int H, int DV) {
  using Sh = StepShape<DK, CV>;
  constexpr int CPR = Sh::kCpr, RPP = Sh::kRpp, NR = Sh::kRows;
  __shared__ float vk[DK], vq[DK];
  __shared__ float4 red[RPP][CPR];
  const int slices = DV / CV;
  const int64_t bh = blockIdx.x / slices;
  const int j0 = (int)(blockIdx.x % slices) * CV;
  const int t = threadIdx.x, c = t % CPR, g = t / CPR;
  float lk = 0.f, lq = 0.f;
  if (t < DK) {
    lk = Elem<Tin>::to_f32(k[bh * DK + t]);
    lq = Elem<Tin>::to_f32(q[bh * DK + t]);
  }
  float* Sb = S + bh * DK * DV + j0 + 4 * c;
  float4 s[NR];
#pragma unroll
  for (int m = 0; m < NR; ++m)
    s[m] = __ldcs(reinterpret_cast<const float4*>(Sb + (size_t)(g + RPP * m) * DV));
  const float4 vv = load4_f32(v + bh * DV + j0 + 4 * c);
  const float a = __ldg(alpha + (per_head ? bh % H : bh));
  if (t < DK) {
    vk[t] = lk;
    vq[t] = lq;
  }
  __syncthreads();
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int m = 0; m < NR; ++m) {
    const int i = g + RPP * m;
    const float kk = vk[i], qq = vq[i];
    float4 x = s[m];
    x.x = fmaf(a, x.x, kk * vv.x); x.y = fmaf(a, x.y, kk * vv.y);
    x.z = fmaf(a, x.z, kk * vv.z); x.w = fmaf(a, x.w, kk * vv.w);
    __stcs(reinterpret_cast<float4*>(Sb + (size_t)i * DV), x);
    o.x = fmaf(x.x, qq, o.x); o.y = fmaf(x.y, qq, o.y);
    o.z = fmaf(x.z, qq, o.z); o.w = fmaf(x.w, qq, o.w);
  }
  red[g][c] = o;
  __syncthreads();
  if (g == 0) {
#pragma unroll 8
    for (int gg = 1; gg < RPP; ++gg) {
      const float4 b = red[gg][c];
      o.x += b.x; o.y += b.y; o.z += b.z; o.w += b.w;
    }
    store4(out + bh * DV + j0 + 4 * c, o);
  }
}

struct StepArgs {
  const void *q, *k, *v;
  const float* alpha;
  int per_head;
  float* S;
  void* out;
  int BH, H, dv;
  bool narrow;  // column slices of 16
};

template <int DK, int CV, typename Tin, typename Tout>
static cudaError_t step_launch(const StepArgs& p, cudaStream_t st) {
  la_step_kernel<DK, CV, Tin, Tout>
      <<<(unsigned)p.BH * (p.dv / CV), StepShape<DK, CV>::kThreads, 0, st>>>(
          static_cast<const Tin*>(p.q), static_cast<const Tin*>(p.k), static_cast<const Tin*>(p.v),
          p.alpha, p.per_head, p.S, static_cast<Tout*>(p.out), p.H, p.dv);
  return cudaGetLastError();
}

template <int DK, typename Tin, typename Tout>
static cudaError_t step_cols(const StepArgs& p, cudaStream_t st) {
  if (p.narrow || p.dv == 16) return step_launch<DK, 16, Tin, Tout>(p, st);
  switch (p.dv) {
    case 32: return step_launch<DK, 32, Tin, Tout>(p, st);
    case 64: return step_launch<DK, 64, Tin, Tout>(p, st);
    case 128: return step_launch<DK, 128, Tin, Tout>(p, st);
  }
  return cudaErrorInvalidValue;
}

template <typename Tin, typename Tout>
static cudaError_t step_rows(int dk, const StepArgs& p, cudaStream_t st) {
  switch (dk) {
    case 16: return step_cols<16, Tin, Tout>(p, st);
    case 32: return step_cols<32, Tin, Tout>(p, st);
    case 64: return step_cols<64, Tin, Tout>(p, st);
    case 128: return step_cols<128, Tin, Tout>(p, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace la

cudaError_t launch_la_decode(int dtype, int out_dtype, int dk, int dv, const void* q, const void* k,
                             const void* v, const float* alpha, int per_head, float* S, void* out,
                             int B, int H, cudaStream_t stream) {
  const int BH = B * H;
  // Slices of 16 columns for at most half as many heads as SMs with a state of
  // 64 KB.  us, slices / whole heads, bf16 inputs, one call after another:
  //   d_k = d_v = 128: 16 heads 2.1 / 2.9, 32: 2.8 / 3.6, 64: 3.9 / 4.0, 80: 4.2 / 4.2,
  //   128: 5.1 / 4.9, 256: 8.3 / 7.3
  // Smaller states are not worth it at any number (d_k = 64, d_v = 128: 32 heads
  // 2.3 / 2.1, 128: 4.0 / 3.4; d_k = 128, d_v = 64: 2.2 / 2.2, 3.9 / 3.4).
  const la::StepArgs p{q, k, v, alpha, per_head, S, out, BH, H, dv,
                       dk == 128 && dv == 128 && BH <= 148 / 2};
  if (dtype == CKDA_BF16)
    return out_dtype == CKDA_BF16 ? la::step_rows<__nv_bfloat16, __nv_bfloat16>(dk, p, stream)
                                  : la::step_rows<__nv_bfloat16, float>(dk, p, stream);
  return out_dtype == CKDA_BF16 ? la::step_rows<float, __nv_bfloat16>(dk, p, stream)
                                : la::step_rows<float, float>(dk, p, stream);
}

}  // namespace ckda
