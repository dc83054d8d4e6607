// Pieces shared by the tensor-core kernels of head-decay linear attention.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

#include "la_common.cuh"
#include "sm100.cuh"

namespace ckda {
namespace la {

// Products over a warp's lanes: through this lane, and behind it.
template <typename T>
__device__ __forceinline__ T warp_prefix(T a, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T b = __shfl_up_sync(0xffffffffu, a, o);
    a = lane >= o ? a * b : a;
  }
  return a;
}

template <typename T>
__device__ __forceinline__ T warp_suffix(T a, int lane) {
  T s = __shfl_down_sync(0xffffffffu, a, 1);
  s = lane == 31 ? T(1) : s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T b = __shfl_down_sync(0xffffffffu, s, o);
    s = lane + o < 32 ? s * b : s;
  }
  return s;
}

// A chunk's decays (four blocks of 32 tokens, a lane one of each) for the other
// warps: {a[128], sufW[128], tot[4], gamma}.  gamma, whose error the state
// takes on again with every chunk, is multiplied up in 64 bits and rounded
// once: in 32 bits the errors all lie on one side when the decay is the same
// for every token (1e-6 of S_final after 4096 tokens instead of 2e-7).  The
// others stay in 32 bits: 64-bit shuffles for all of them cost a tenth of the
// forward's time, which shared memory bounds.
constexpr int kDecFloats = 264;
__device__ __forceinline__ void put_decays(float* o, const float* a, int lane) {
  double all = ((double)a[0] * (double)a[1]) * ((double)a[2] * (double)a[3]);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) all *= __shfl_xor_sync(0xffffffffu, all, d);
#pragma unroll
  for (int bk = 0; bk < 4; ++bk) {
    const float pw = warp_prefix(a[bk], lane), sw = warp_suffix(a[bk], lane);
    o[32 * bk + lane] = a[bk];
    o[128 + 32 * bk + lane] = sw;
    if (lane == 31) o[256 + bk] = pw;
  }
  if (lane == 0) o[260] = (float)all;
}

__device__ __forceinline__ float lo_f(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi_f(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// A pair of bf16 values times w as the sum of three bf16 pairs: 24 bits.
__device__ __forceinline__ void split3(uint32_t in, float2 w, uint32_t* t1, uint32_t* t2,
                                       uint32_t* t3) {
  const float2 m1 = make_float2(-1.f, -1.f);
  float2 x = mul2(make_float2(lo_f(in), hi_f(in)), w);
  *t1 = sm100::pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(lo_f(*t1), hi_f(*t1)), m1, x);
  *t2 = sm100::pack_bf16x2(x.x, x.y);
  x = fma2(make_float2(lo_f(*t2), hi_f(*t2)), m1, x);
  *t3 = sm100::pack_bf16x2(x.x, x.y);
}

__device__ __forceinline__ uint4 pack8(const float* x) {
  return make_uint4(sm100::pack_bf16x2(x[0], x[1]), sm100::pack_bf16x2(x[2], x[3]),
                    sm100::pack_bf16x2(x[4], x[5]), sm100::pack_bf16x2(x[6], x[7]));
}

template <int N>
__device__ __forceinline__ void store_cols(__nv_bfloat16* o, const float* x) {
#pragma unroll
  for (int e = 0; e < N; e += 8) *reinterpret_cast<uint4*>(o + e) = pack8(x + e);
}

template <int N>
__device__ __forceinline__ void store_cols(float* o, const float* x) {
#pragma unroll
  for (int e = 0; e < N; e += 4)
    *reinterpret_cast<float4*>(o + e) = make_float4(x[e], x[e + 1], x[e + 2], x[e + 3]);
}

// ---- host side ---------------------------------------------------------------------

// A [rows, cols] bf16 tensor in boxes of `box_rows` x 64, 128-byte swizzle.
inline bool bf16_map(CUtensorMap* m, const void* ptr, uint64_t cols, uint64_t rows,
                     uint32_t box_rows) {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  auto f = fn.load(std::memory_order_acquire);
  if (f == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    fn.store(f, std::memory_order_release);
  }
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Allows kernel `id` its dynamic shared memory, once per device.
template <int id, typename K>
inline cudaError_t max_smem(K kern, size_t bytes) {
  constexpr int kMaxDevices = 64;
  static std::atomic<bool> done[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < kMaxDevices && done[dev].load(std::memory_order_acquire))
    return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices)
    done[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace la
}  // namespace ckda
