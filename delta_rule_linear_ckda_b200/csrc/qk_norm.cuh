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
  int heads_warp;         // heads of a token that one warp takes (set at launch, as units)
  float c, eps;
  int64_t units;          // warps' shares
};

}  // namespace qkn
}  // namespace ckda
