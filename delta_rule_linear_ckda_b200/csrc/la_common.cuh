// Shared by the kernels of head-decay linear attention,
//   S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,
// with one decay a_t in [-1, 1] per (token, head), or one per head.
#pragma once

#include "common.cuh"

namespace ckda {
namespace la {

// A decay: alpha[token, h], or alpha[h] when it is given per head.
struct Decay {
  const float* p;
  int H;
  int per_head;
  __device__ __forceinline__ float at(int64_t tok, int h) const {
    return __ldg(per_head ? p + h : p + tok * H + h);
  }
  // The same, issued where it stands: the compiler may move a plain load past
  // waits, down to its use.
  __device__ __forceinline__ float now(int64_t tok, int h) const {
    float x;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(per_head ? p + h : p + tok * H + h));
    return x;
  }
};

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 z, x, y, w;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Chunks of `C` tokens, numbered over the batch: a sequence's first slot.
// Packed batches use floor(cu[n] / C) + n, so that every sequence has room
// for its partial chunk whatever the lengths (slots in between stay unused).
__host__ __device__ __forceinline__ int64_t chunk_slots(bool varlen, int n_seqs, int T, int C) {
  return varlen ? (int64_t)T / C + n_seqs : (int64_t)n_seqs * (((int64_t)T + C - 1) / C);
}

__device__ __forceinline__ int64_t slot_of(const int32_t* cu, int n, int T, int C) {
  return cu != nullptr ? (int64_t)(cu[n] / C) + n : (int64_t)n * ((T + C - 1) / C);
}

// The sequence and chunk of a slot; false for a slot that holds no token.
// Only offsets that seq_range accepts for sequence n are used: the caller
// checks them.
__device__ __forceinline__ bool slot_chunk(const int32_t* cu, int n_seqs, int T, int C, int64_t slot,
                                           int* n_out, int* c_out) {
  if (cu == nullptr) {
    const int per = (T + C - 1) / C;
    *n_out = (int)(slot / per);
    *c_out = (int)(slot % per);
    return *n_out < n_seqs;
  }
  // the last n with slot_of(n) <= slot; slot_of grows by at least one per
  // sequence where the offsets do not decrease
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (slot_of(cu, mid, T, C) <= slot) lo = mid; else hi = mid - 1;
  }
  *n_out = lo;
  *c_out = (int)(slot - slot_of(cu, lo, T, C));
  return *c_out >= 0 && (int64_t)*c_out * C < (int64_t)cu[lo + 1] - cu[lo];
}

}  // namespace la
}  // namespace ckda
