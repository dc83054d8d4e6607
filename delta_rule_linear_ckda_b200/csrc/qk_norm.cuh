// Arguments of the query / key norm kernels (qk_norm.cu), filled by the C ABI.
#pragma once

#include "common.cuh"

namespace ckda {
namespace qkn {

// The queries (0) or the keys (1).
struct Side {
  const void* x;      // row of token t and head h at x + t * stride + h * d
  const float* w;     // [d] or NULL (ones)
  void* out;          // forward: z; backward: dx; [tokens, H, d]
  const void* g;      // backward: dz [tokens, H, d]
  int64_t stride;
  int H;
  // set at launch
  int heads_warp;     // heads of a token that one warp takes
  int64_t units;      // warps' shares
  unsigned ctas;      // of the grid, the queries' first
};

struct Args {
  Side s[2];
  const int32_t* pos;     // [tokens]
  const float* inv_freq;  // [rot / 2]
  float* part;            // backward: [ctas][d] sums of dw, or NULL
  int64_t tokens;
  int d, rot, interleaved;
  float c, eps;
};

}  // namespace qkn
}  // namespace ckda
