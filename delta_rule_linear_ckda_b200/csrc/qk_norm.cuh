// Arguments of the query / key norm kernels (qk_norm.cu), filled by the C ABI.
#pragma once

#include "common.cuh"

namespace ckda {
namespace qkn {

struct Args {
  const void *q, *k;      // rows of token t at q + t * q_stride + head * d
  const float *wq, *wk;   // [d] or NULL (ones)
  const int32_t* pos;     // [tokens]
  const float* inv_freq;  // [rot / 2]
  void *oq, *ok;          // forward: z; backward: dx; [tokens, heads, d]
  const void *gq, *gk;    // backward: dz [tokens, heads, d]
  float* part;            // backward: [gridDim.x][2][d] sums of dw, or NULL
  int64_t q_stride, k_stride;
  int64_t tokens;
  int Hq, Hk, d, rot, interleaved;
  int tok_cta;            // tokens a CTA takes at a time
  float c, eps;
};

}  // namespace qkn
}  // namespace ckda
