// Backward of head-decay linear attention on the tensor cores (tcgen05): bf16
// inputs, d_k and d_v 64 or 128 (sm_100a).
//
// Per chunk of C = 128 tokens, S the state at its start, G the adjoint of the
// state at its end, D(i, j) = a_{j+1} .. a_i (zero for j > i):
//   E = D o (dO V^T),  P = D o (Q K^T)
//   dQ = E K   + diag(pre) dO S^T        pre_i = a_0 .. a_i
//   dK = E^T Q + diag(suf) V G^T         suf_j = a_{j+1} .. a_{C-1}
//   dV = P^T dO + diag(suf) K G
//   da_t = sum_{i >= t > j} D(i, t) D(t-1, j) W_ij + head_t X_t + tail_t Y_t
//          + head_t tail_t <S, G>,   W = (Q K^T) o (dO V^T)
// with X_t = sum_{i >= t} D(i, t) x_i, x_i = q_i . (dO S^T)_i,
// Y_t = sum_{j < t} D(t-1, j) y_j, y_j = v_j . (K G)_j, head_t = a_0 .. a_{t-1},
// tail_t = suf_t: nothing is divided by a decay.
//
// Two kernels:
//  1. la_states_kernel walks every sequence's chunks forward for S and
//     backward for G and leaves both at every chunk's bound (fp32).  It is the
//     forward's state path alone: one product per chunk, diag(w) V split into
//     three bf16 terms side by side.
//  2. la_chunk_kernel takes one (chunk, head) at a time, all of them in
//     parallel.  S and G enter their products as three bf16 terms each
//     (V G^T: one), because x, y and so the decays' gradient keep fp32
//     accuracy; dq, dk, dv are rounded to bf16 in the end (1.66e-3 in 2-norm),
//     and E, P and V G^T's G once on the way (2.35e-3 with it): E and P as
//     operands fill what shared memory the states' terms leave.
// E and P are zero right of the diagonal, but zero times a value that is not
// finite is not, and E K, E^T Q and P^T dO would carry it to tokens that do
// not depend on it.  A chunk with such a value shows it in the scores'
// diagonal; it takes those values out of K, Q and dO before these products (E K
// then waits for the other readers of K) and sets what does depend on them to
// NaN afterwards.
// B = 4, T = 4096, H = 16, d = 128: 345 us.  The first launch (123 us alone, DRAM
// 50 %) waits for each chunk's product in turn; the second (235 us) is bound by
// its chain of phases, one block of 8 warps per SM: DRAM 37 %, tensor pipe 21 %,
// issue slots 28 %.  The two states of 64 KB per (chunk, head), written and read
// once, are more than half of the traffic.
#include "la_tc.cuh"

namespace ckda {
namespace la {

using namespace sm100;

namespace bw {

constexpr int C = 128;
constexpr int DK = 128;
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait

// A state in the workspace (always 128 rows): columns in groups of four, [d_v / 4][128 rows][4],
// so that a warp whose lanes are rows reads and writes whole lines.
__host__ __device__ constexpr size_t state_floats(int dv) { return (size_t)DK * dv; }

// ---- kernel 1: states at the chunks' bounds -------------------------------------------

namespace st {

constexpr int BV = 64;
constexpr int kHalf = BV / 2;
constexpr uint32_t OFF_A = 0;                     // k or q [128][128]
constexpr uint32_t OFF_B = 32768;                 // v or do [128][64]
constexpr uint32_t OFF_VW = OFF_B + 16384;        // diag(w) of it, three terms
constexpr uint32_t OFF_DEC = OFF_VW + 3 * 16384;  // 2 x the decays (put_decays)
constexpr uint32_t kDecBytes = kDecFloats * 4;
constexpr uint32_t OFF_BAR = OFF_DEC + 2 * kDecBytes;
constexpr uint32_t B_A = 0, B_B = 8, B_VW = 16, B_D = 24, B_DEC = 32, B_DECE = 48;
constexpr uint32_t OFF_MISC = OFF_BAR + 64;
constexpr uint32_t kSmem = OFF_MISC + 16;
constexpr uint32_t kTmemCols = 256;
constexpr int kThreads = 352;

struct Args {
  Decay al;
  const float *S0, *dSf;
  float *Sk, *Gk;  // kept states
  float* dS0;      // or NULL
  const int32_t* cu;
  int n_seqs, T, H, DV;
  int* status;
};

// KD: d_k
template <int KD>
__global__ void __launch_bounds__(kThreads, 2)
la_states_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                 const Args p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if ((sb & 1023u) != 0) {
    set_status(p.status, CKDA_ERR_CUDA);
    return;
  }
  // block index: column slice, direction, head, sequence (longest first)
  const int slices = p.DV / BV;
  int b = blockIdx.x;
  const int j0 = (b % slices) * BV;
  b /= slices;
  const bool rev = b & 1;
  b >>= 1;
  const int h = b % p.H;
  const int n =
      seq_longest_first(p.cu, p.n_seqs, b / p.H, reinterpret_cast<int*>(sm + OFF_MISC + 4));
  const SeqRange sr = seq_range(p.cu, n, p.n_seqs, p.T, p.status);
  if (!sr.ok) return;
  const uint32_t bar = sb + OFF_BAR;
  const CUtensorMap* tm_a = rev ? &tm_q : &tm_k;
  const CUtensorMap* tm_b = rev ? &tm_do : &tm_v;
  if (tid == 0) {
    mbar_init(bar + B_A, 1);
    mbar_init(bar + B_B, 1);
    mbar_init(bar + B_VW, 8);
    mbar_init(bar + B_D, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B_DEC + 8 * i, 1);
      mbar_init(bar + B_DECE + 8 * i, 8);
    }
    fence_mbar_init();
    prefetch_tmap(tm_a);
    prefetch_tmap(tm_b);
  }
  if (warp == 0) {
    tmem_alloc(sb + OFF_MISC, kTmemCols);
    tmem_relinquish();
  }
  if constexpr (KD < DK) {  // no load writes a's second 64 columns
    for (int e = tid; e < 1024; e += kThreads)
      *reinterpret_cast<uint4*>(sm + OFF_A + 16384 + e * 16) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sm + OFF_MISC), 0);
  const int nck = __shfl_sync(0xffffffffu, (int)((sr.end - sr.begin + C - 1) / C), 0);
  // the it-th chunk taken
  auto chunk = [&](int it) -> int { return rev ? nck - 1 - it : it; };
  auto tok = [&](int it) -> int64_t { return sr.begin + (int64_t)chunk(it) * C; };
  auto len_of = [&](int it) -> int {
    const int64_t left = sr.end - tok(it);
    return left < C ? (int)left : C;
  };
  auto wait = [&](uint32_t off, uint32_t par) -> bool {
    return mbar_wait_small(bar + off, par & 1u, kWaitNs);
  };
  auto arrive = [&](uint32_t off) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + off);
  };
  const float* dec0 = reinterpret_cast<const float*>(sm + OFF_DEC);
  auto decs = [&](int it) { return dec0 + (it & 1) * (kDecBytes / 4); };
  bool ok = true;
  bool open_a = false, open_b = false, mma_open = false;
  uint32_t par_last = 0;

  if (warp < 8) {
    // ---- state: row r of d_k, half of the slice's columns ------------------------------
    const int q4 = warp & 3, hf = warp >> 2;
    const int r = 32 * q4 + lane;
    const uint32_t row = tmem + ((uint32_t)(32 * q4) << 16);
    const size_t unit = (size_t)n * p.H + h, stsz = (size_t)KD * p.DV;
    const bool row_in = KD == DK || r < KD;
    const size_t at = (size_t)r * p.DV + j0 + kHalf * hf;
    float S[kHalf];
    {
      const float* src = rev ? p.dSf : p.S0;
#pragma unroll
      for (int e = 0; e < kHalf; e += 4) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src != nullptr && row_in)
          x = *reinterpret_cast<const float4*>(src + unit * stsz + at + e);
        S[e] = x.x; S[e + 1] = x.y; S[e + 2] = x.z; S[e + 3] = x.w;
      }
    }
    float* kept = (rev ? p.Gk : p.Sk) + (size_t)(j0 + kHalf * hf) * DK + 4 * r;
    const int64_t slot0 = slot_of(p.cu, n, p.T, C);
    float gamma = 1.f;
#pragma unroll 1
    for (int it = 0; it <= nck; ++it) {
      if (it > 0) {
        if (!(ok = wait(B_D, it - 1))) break;
        tc_fence_after();
        const float2 g2 = make_float2(gamma, gamma);
#pragma unroll
        for (int e = 0; e < kHalf; e += 8) {
          float x[8], y[8], z[8];
          tmem_ld8(row + kHalf * hf + e, x);
          tmem_ld8(row + BV + kHalf * hf + e, y);
          tmem_ld8(row + 2 * BV + kHalf * hf + e, z);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 8; u += 2) {
            const float2 d = add2(make_float2(x[u], x[u + 1]),
                                  add2(make_float2(y[u], y[u + 1]), make_float2(z[u], z[u + 1])));
            const float2 s = fma2(g2, make_float2(S[e + u], S[e + u + 1]), d);
            S[e + u] = s.x;
            S[e + u + 1] = s.y;
          }
        }
      }
      if (it == nck) break;
      {
        float* o = kept + ((size_t)(slot0 + chunk(it)) * p.H + h) * state_floats(p.DV);
#pragma unroll
        for (int e = 0; e < kHalf; e += 4)
          *reinterpret_cast<float4*>(o + (size_t)e * DK) =
              make_float4(S[e], S[e + 1], S[e + 2], S[e + 3]);
      }
      const int len = len_of(it);
      if (!(ok = wait(B_DEC + 8 * (it & 1), it >> 1))) break;
      const float* dc = decs(it);
      const float4 tot = *reinterpret_cast<const float4*>(dc + 256);
      float wgt;
      if (rev)
        wgt = warp_prefix(dc[r], lane) * (q4 > 0 ? tot.x : 1.f) * (q4 > 1 ? tot.y : 1.f) *
              (q4 > 2 ? tot.z : 1.f);
      else
        wgt = dc[128 + r] * (q4 < 1 ? tot.y : 1.f) * (q4 < 2 ? tot.z : 1.f) *
              (q4 < 3 ? tot.w : 1.f);
      gamma = dc[260];
      arrive(B_DECE + 8 * (it & 1));
      if (!(ok = wait(B_B, it))) break;
      if (len < C && !(ok = wait(B_A, it))) break;
      if (r < len) {
        const float2 w2 = make_float2(wgt, wgt);
#pragma unroll 1
        for (int h2 = 0; h2 < 2; ++h2) {
          const uint32_t o0 = sw128_chunk(r, kHalf * hf + 16 * h2, 128);
          const uint32_t o1 = o0 ^ 16u;  // the next 16 bytes under the swizzle
          const uint4 ra = *reinterpret_cast<const uint4*>(sm + OFF_B + o0);
          const uint4 rb = *reinterpret_cast<const uint4*>(sm + OFF_B + o1);
          const uint32_t in[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
          uint32_t t1[8], t2[8], t3[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) split3(in[e], w2, &t1[e], &t2[e], &t3[e]);
          uint8_t* d = sm + OFF_VW;
          *reinterpret_cast<uint4*>(d + o0) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
          *reinterpret_cast<uint4*>(d + o1) = make_uint4(t1[4], t1[5], t1[6], t1[7]);
          *reinterpret_cast<uint4*>(d + 16384 + o0) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
          *reinterpret_cast<uint4*>(d + 16384 + o1) = make_uint4(t2[4], t2[5], t2[6], t2[7]);
          *reinterpret_cast<uint4*>(d + 32768 + o0) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
          *reinterpret_cast<uint4*>(d + 32768 + o1) = make_uint4(t3[4], t3[5], t3[6], t3[7]);
        }
      } else {
        // what lies past the sequence's end takes no part, finite or not
        const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int c8 = 0; c8 < kHalf / 8; ++c8)
          for (int e = 0; e < 3; ++e)
            *reinterpret_cast<uint4*>(sm + OFF_VW + e * 16384 +
                                      sw128_chunk(r, kHalf * hf + 8 * c8, 128)) = z;
#pragma unroll 1
        for (int c8 = 0; c8 < KD / 16; ++c8)
          *reinterpret_cast<uint4*>(sm + OFF_A + sw128_chunk(r, (KD / 2) * hf + 8 * c8, 128)) = z;
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(B_VW);
    }
    if (ok && rev && p.dS0 != nullptr && row_in) store_cols<kHalf>(p.dS0 + unit * stsz + at, S);
  } else if (warp == 8) {
    // ---- MMA (the whole warp waits, one lane issues) ---------------------------------------
    const uint64_t d_a = smem_desc(sb + OFF_A, 16384, 1024, kSwizzle128);
    const uint64_t d_vw = smem_desc(sb + OFF_VW, 16384, 1024, kSwizzle128);
    constexpr uint32_t id = idesc_bf16(128, 3 * BV, 1, 1);
#pragma unroll 1
    for (int it = 0; it < nck; ++it) {
      if (!(ok = wait(B_VW, it) && wait(B_A, it))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16(tmem, d_a + 128 * kk, d_vw + 128 * kk, id, kk > 0 ? 1u : 0u);
        mma_commit(bar + B_D);
      }
      __syncwarp();
      mma_open = true;
      par_last = it;
    }
  } else if (warp == 9) {
    // ---- loads: b of the next chunk once its rows are converted, a once the
    // product is done (the two blocks of an SM cover for one another) -----------------------
    if (lane == 0) {
#pragma unroll 1
      for (int it = 0; it < nck; ++it) {
        const int t = (int)tok(it);
        if (it > 0 && !(ok = wait(B_VW, it - 1))) break;
        mbar_expect_tx(bar + B_B, 16384);
        tma_load_2d(sb + OFF_B, tm_b, h * p.DV + j0, t, bar + B_B);
        open_b = true;
        par_last = it;
        if (it + 1 < nck) {
          const int t1 = (int)tok(it + 1);
          for (int x = 0; x < KD; x += 64) tma_prefetch_2d(tm_a, h * KD + x, t1);
          tma_prefetch_2d(tm_b, h * p.DV + j0, t1);
        }
        if (it > 0 && !(ok = wait(B_D, it - 1))) break;
        mbar_expect_tx(bar + B_A, 256 * KD);
        for (int x = 0; x < KD; x += 64)
          tma_load_2d(sb + OFF_A + 256 * x, tm_a, h * KD + x, t, bar + B_A);
        open_a = true;
      }
      if (!ok) {  // give the loads in flight their time
        if (open_b) mbar_wait_small(bar + B_B, par_last & 1u, kWaitNs);
        if (open_a && par_last > 0) mbar_wait_small(bar + B_A, (par_last - 1) & 1u, kWaitNs);
      }
    }
  } else {
    // ---- decays ---------------------------------------------------------------------------
    auto load = [&](int it, float* a) {
      const int len = it < nck ? len_of(it) : 0;
      const int64_t t0 = it < nck ? tok(it) : 0;
#pragma unroll
      for (int bk = 0; bk < 4; ++bk) {
        const int t = 32 * bk + lane;
        a[bk] = t < len ? p.al.now(t0 + t, h) : 1.f;
      }
    };
    float a[4], nx[4];
    load(0, a);
#pragma unroll 1
    for (int it = 0; it < nck; ++it) {
      load(it + 1, nx);
      if (it >= 2 && !(ok = wait(B_DECE + 8 * (it & 1), (it >> 1) - 1))) break;
      put_decays(reinterpret_cast<float*>(sm + OFF_DEC) + (it & 1) * kDecFloats, a, lane);
#pragma unroll
      for (int bk = 0; bk < 4; ++bk) a[bk] = nx[bk];
      arrive(B_DEC + 8 * (it & 1));
    }
  }
  if (!ok) {
    set_status(p.status, CKDA_ERR_DEVICE_TIMEOUT);
    if (warp == 8 && mma_open) mbar_wait_small(bar + B_D, par_last & 1u, kWaitNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace st

// ---- kernel 2: the gradients of one (chunk, head) ----------------------------------------

namespace ck {

constexpr uint32_t OFF_Q = 0, OFF_K = 32768;         // [128][128] bf16, two 64-column atoms
constexpr uint32_t OFF_V = 65536, OFF_DO = 98304;    // [128][DV]
constexpr uint32_t OFF_E = 131072, OFF_P = 163840;   // first two terms of S, then E and P
constexpr uint32_t OFF_T = 196608;                   // third term of S, then the terms of G
constexpr uint32_t OFF_F = 229376;                   // floats, below
// decays; sufW; block products; <S, G> by warp; x by column half; column sums
// of the six row and column blocks below the diagonal
constexpr uint32_t F_A = 0, F_SW = 128, F_TOT = 256, F_Z = 260, F_X = 268, F_COL = 524;
// later in their places: y by column half, the sums within the chunk
constexpr uint32_t F_Y0 = F_COL, F_Y1 = F_SW, F_IN = F_X + 128;
// bytes, of a chunk with values that are not finite: the row behind a
// column's last one in Q, in dO (the first one in K: OFF_KBAD)
constexpr uint32_t OFF_QBAD = OFF_F + 4 * 652, OFF_OBAD = OFF_QBAD + 128;
constexpr uint32_t OFF_BAR = OFF_F + 4 * 716;
constexpr uint32_t B_LD = 0;    // tiles loaded
constexpr uint32_t B_SC = 8;    // scores complete (tensor core)
constexpr uint32_t B_DS = 16;   // dO S^T complete
constexpr uint32_t B_G = 24;    // a term of G is done with (three times per unit)
constexpr uint32_t B_FIN = 32;  // the gradients complete
constexpr uint32_t OFF_MISC = OFF_BAR + 40;  // tensor-memory base, whether there are such values
constexpr uint32_t OFF_KBAD = OFF_MISC + 16;
constexpr uint32_t kSmem = OFF_KBAD + 128;
static_assert(OFF_OBAD + 128 <= OFF_BAR, "bytes of a chunk with values that are not finite");
static_assert(kSmem <= 232448, "shared memory");

constexpr uint32_t TM_S1 = 0, TM_S2 = 128;           // Q K^T, dO V^T
constexpr uint32_t TM_DV = 0, TM_DK = 128, TM_DQ = 256;
constexpr uint32_t kTmemCols = 512;
constexpr int kCompute = 256;
constexpr int kThreads = kCompute;  // more warps would leave a thread less than 255 registers

struct Args {
  Decay al;
  const float *Sk, *Gk;
  __nv_bfloat16 *dq, *dk, *dv;
  float* da;
  const int32_t* cu;
  int n_seqs, T, H;
  int64_t units;  // slots * H
  int* status;
};

// 16 bytes, requested where this stands (a plain load may be moved down to its
// use).
__device__ __forceinline__ void ld4(const float* p, float* x) {
  asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
               : "l"(p));
}

// Pulls `bytes` (a multiple of 16) into L2.
__device__ __forceinline__ void prefetch_l2_bulk(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}

// V_t = c_t V_{t-1} + b_t over 128 positions, four per lane; V_{-1} = 0.
__device__ __forceinline__ void lin_scan(const float* c, const float* b, float* v, int lane) {
  float A = c[0], B = b[0];
#pragma unroll
  for (int e = 1; e < 4; ++e) {
    B = fmaf(c[e], B, b[e]);
    A *= c[e];
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float pa = __shfl_up_sync(0xffffffffu, A, o), pb = __shfl_up_sync(0xffffffffu, B, o);
    if (lane >= o) {
      B = fmaf(A, pb, B);
      A *= pa;
    }
  }
  float x = __shfl_up_sync(0xffffffffu, B, 1);
  if (lane == 0) x = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x = fmaf(c[e], x, b[e]);
    v[e] = x;
  }
}

// A row's N columns of an accumulator times f, in place; returns the row's
// product (before f) with the same columns of a 128-byte-swizzled bf16 tile.
template <int N>
__device__ __forceinline__ float scale_rows(uint32_t addr, float f, const uint8_t* tile, int i,
                                            int col) {
  float s = 0.f;
#pragma unroll 1
  for (int e = 0; e < N; e += 16) {
    float x[16];
    tmem_ld16(addr + e, x);
    tmem_ld_wait();
    if (tile != nullptr) {
#pragma unroll
      for (int o = 0; o < 16; o += 8) {
        const uint4 r = *reinterpret_cast<const uint4*>(tile + sw128_chunk(i, col + e + o, 128));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int t = 0; t < 4; ++t)
          s = fmaf(x[o + 2 * t], lo_f(w[t]), fmaf(x[o + 2 * t + 1], hi_f(w[t]), s));
      }
    }
    uint32_t y[16];
#pragma unroll
    for (int t = 0; t < 16; ++t) y[t] = __float_as_uint(f * x[t]);
    tmem_st16(addr + e, y);
  }
  tmem_st_wait();
  return s;
}

// Takes the values that are not finite out of a column of a 128-row tile; their
// first row (128 if there is none) and the row behind the last (0).
__device__ __forceinline__ void clean_column(uint8_t* tile, int col, int* first, int* end) {
  *first = 128;
  *end = 0;
#pragma unroll 1
  for (int r = 0; r < 128; ++r) {
    uint16_t* x = reinterpret_cast<uint16_t*>(tile + sw128_chunk(r, col & ~7, 128)) + (col & 7);
    if ((*x & 0x7f80) == 0x7f80) {
      *x = 0;
      if (*end == 0) *first = r;
      *end = r + 1;
    }
  }
}

// Sets row i of N columns of an accumulator to NaN where it lies in rows
// [at[col], 128) or, for `before`, in rows [0, at[col]).
template <int N>
__device__ __forceinline__ void poison_rows(uint32_t addr, int i, const uint8_t* at, bool before) {
#pragma unroll 1
  for (int e = 0; e < N; e += 16) {
    float x[16];
    tmem_ld16(addr + e, x);
    tmem_ld_wait();
    uint32_t y[16];
#pragma unroll
    for (int t = 0; t < 16; ++t)
      y[t] = (i < at[e + t]) == before ? 0x7fffffffu : __float_as_uint(x[t]);
    tmem_st16(addr + e, y);
  }
  tmem_st_wait();
}

template <int KD, int DV>  // d_k, d_v
__global__ void __launch_bounds__(kThreads, 1)
la_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ CUtensorMap tm_dk,
                const __grid_constant__ CUtensorMap tm_dv, const Args p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if ((sb & 1023u) != 0) {
    set_status(p.status, CKDA_ERR_CUDA);
    return;
  }
  const uint32_t bar = sb + OFF_BAR;
  float* F = reinterpret_cast<float*>(sm + OFF_F);
  if (tid == 0) {
    for (int i = 0; i < 5; ++i) mbar_init(bar + 8 * i, 1);
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_do);
  }
  if (warp == 0) {
    tmem_alloc(sb + OFF_MISC, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sm + OFF_MISC), 0);
  auto wait = [&](uint32_t off, uint32_t par) -> bool {
    return mbar_wait_small(bar + off, par & 1u, kWaitNs);
  };
  // the unit's first token, its tokens and its head; 0 tokens: no such chunk
  auto decode = [&](int64_t u, int64_t* t0, int* h) -> int {
    *h = (int)(u % p.H);
    int n, c;
    if (!slot_chunk(p.cu, p.n_seqs, p.T, C, u / p.H, &n, &c)) return 0;
    const SeqRange sr = seq_range(p.cu, n, p.n_seqs, p.T, p.status);
    if (!sr.ok) return 0;
    *t0 = sr.begin + (int64_t)c * C;
    const int64_t left = sr.end - *t0;
    return left < C ? (int)left : C;
  };
  auto load = [&](int64_t t0, int h) {
    const int t = (int)t0;
    mbar_expect_tx(bar + B_LD, 2 * 256 * (KD + DV));
    for (int x = 0; x < KD; x += 64) {
      tma_load_2d(sb + OFF_Q + 256 * x, &tm_q, h * KD + x, t, bar + B_LD);
      tma_load_2d(sb + OFF_K + 256 * x, &tm_k, h * KD + x, t, bar + B_LD);
    }
    for (int x = 0; x < DV; x += 64) {
      tma_load_2d(sb + OFF_DO + 256 * x, &tm_do, h * DV + x, t, bar + B_LD);
      tma_load_2d(sb + OFF_V + 256 * x, &tm_v, h * DV + x, t, bar + B_LD);
    }
  };

  const bool lead = warp == 0;  // this warp also issues the products, loads and stores
  const uint64_t q_k = smem_desc(sb + OFF_Q, 16, 1024, kSwizzle128);      // K-major
  const uint64_t q_m = smem_desc(sb + OFF_Q, 16384, 1024, kSwizzle128);   // MN-major
  constexpr uint64_t kTile = 32768 >> 4;
  // tiles by index: 0 Q, 1 K, 2 V, 3 dO, 4 E, 5 P, 6 T
  auto km = [&](int tile, int kk) { return q_k + tile * kTile + 1024 * (kk >> 2) + 2 * (kk & 3); };
  auto mn = [&](int tile, int kk) { return q_m + tile * kTile + 128 * kk; };

  // compute threads: row (token or d_k) and column half
  const int w4 = warp & 3, hf = (warp >> 2) & 1;
  const int i = 32 * w4 + lane;
  const uint32_t row = tmem + ((uint32_t)(32 * w4) << 16);
  bool ok = true, loaded = false;
  uint32_t ld_par = 0, issued = 0, issued_par = 0;  // the MMA warp's last load and commit
  int64_t t0 = 0, t0n = 0;
  int h = 0, hn = 0;
  int64_t u = blockIdx.x;
  int len = 0;
  for (; u < p.units; u += gridDim.x)
    if ((len = decode(u, &t0, &h)) > 0) break;
  if (u < p.units && lead && lane == 0) load(t0, h);
  if (u < p.units) loaded = true;
  // this thread's row and columns of S and of G: what is left of them to split
  float S[DV / 2], G[DV / 2];
  const size_t mine = (size_t)(DV / 2 * hf) * DK + 4 * i;
  auto states = [&](float (&X)[DV / 2], const float* kept, int64_t w) {
    const float* a = kept + w * state_floats(DV) + mine;  // (rows behind d_k are zero there)
#pragma unroll
    for (int e = 0; e < DV / 2; e += 4) ld4(a + (size_t)e * DK, X + e);
  };
  if (u < p.units) {
    states(S, p.Sk, u);
    states(G, p.Gk, u);
  }
  uint32_t ph = 0, g3 = 0;
#pragma unroll 1
  while (u < p.units) {
    // the next unit with tokens
    int64_t un = u + gridDim.x;
    int lenn = 0;
    for (; un < p.units; un += gridDim.x)
      if ((lenn = decode(un, &t0n, &hn)) > 0) break;

    // one bf16 term of X into a tile, X keeps the rest
    auto term = [&](uint32_t off, float (&X)[DV / 2]) {
#pragma unroll
      for (int e = 0; e < DV / 2; e += 8) {
        uint32_t w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          w[x] = pack_bf16x2(X[e + 2 * x], X[e + 2 * x + 1]);
          X[e + 2 * x] -= lo_f(w[x]);
          X[e + 2 * x + 1] -= hi_f(w[x]);
        }
        *reinterpret_cast<uint4*>(sm + off + sw128_chunk(i, DV / 2 * hf + e, 128)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    volatile int* odd = reinterpret_cast<volatile int*>(sm + OFF_MISC + 4);
    if (tid == 0) *odd = 0;  // (the last unit's was read before its last barriers)
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < DV / 2; ++e) z = fmaf(S[e], G[e], z);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (lead) {
      if (lane == 0 && un < p.units) {
        prefetch_l2_bulk(p.Sk + un * state_floats(DV), state_floats(DV) * 4);
        prefetch_l2_bulk(p.Gk + un * state_floats(DV), state_floats(DV) * 4);
      }
      ok = wait(B_LD, ph);
      if (ok && elect_one()) {
        constexpr uint32_t id = idesc_bf16(128, 128, 0, 0);
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk)
          mma_f16(tmem + TM_S1, km(0, kk), km(1, kk), id, kk > 0);
#pragma unroll
        for (int kk = 0; kk < DV / 16; ++kk) mma_f16(tmem + TM_S2, km(3, kk), km(2, kk), id, kk > 0);
        mma_commit(bar + B_SC);
      }
      __syncwarp();
      issued = B_SC;
      issued_par = ph;
      // the last unit's gradients have left their tiles
      if (lane == 0) bulk_wait_read_all();
    }
    __syncthreads();
    if (lane == 0) F[F_Z + warp] = z;
    term(OFF_E, S);
    term(OFF_P, S);
    term(OFF_T, S);
    fence_proxy_async_smem();
    if (warp >= 4) {  // decays
      const float a = i < len ? p.al.at(t0 + i, h) : 1.f;
      const float pw = warp_prefix(a, lane);
      F[F_A + i] = a;
      F[F_SW + i] = warp_suffix(a, lane);
      if (lane == 31) F[F_TOT + w4] = pw;
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    const float4 tot = *reinterpret_cast<const float4*>(F + F_TOT);
    const float pw = i < 128 ? warp_prefix(F[F_A + (i & 127)], lane) : 1.f;
    const float pre = pw * (w4 > 0 ? tot.x : 1.f) * (w4 > 1 ? tot.y : 1.f) * (w4 > 2 ? tot.z : 1.f);
    const float suf = F[F_SW + i] * (w4 < 1 ? tot.y : 1.f) * (w4 < 2 ? tot.z : 1.f) *
                      (w4 < 3 ? tot.w : 1.f);
    if (lead) {
      // dO S^T, the three terms of S one after another
      if (elect_one()) {
        constexpr uint32_t id = idesc_bf16(128, KD, 0, 0);
#pragma unroll 1
        for (int e = 0; e < 3; ++e)
#pragma unroll
          for (int kk = 0; kk < DV / 16; ++kk)
            mma_f16(tmem + TM_DQ, km(3, kk), km(4 + e, kk), id, (e > 0 || kk > 0) ? 1u : 0u);
        mma_commit(bar + B_DS);
      }
      __syncwarp();
      issued = B_DS;
      issued_par = ph;
    }
    {
      // what lies past the sequence's end takes no part, finite or not (the
      // scores' products may read these rows before or after: rows and
      // columns that are masked)
      ok = wait(B_LD, ph);
      if (ok && i >= len) {
        const uint4 zz = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
        for (int e = 0; e < KD / 16; ++e) {
          *reinterpret_cast<uint4*>(sm + OFF_Q + sw128_chunk(i, KD / 2 * hf + 8 * e, 128)) = zz;
          *reinterpret_cast<uint4*>(sm + OFF_K + sw128_chunk(i, KD / 2 * hf + 8 * e, 128)) = zz;
        }
#pragma unroll 1
        for (int e = 0; e < DV / 16; ++e) {
          *reinterpret_cast<uint4*>(sm + OFF_V + sw128_chunk(i, DV / 2 * hf + 8 * e, 128)) = zz;
          *reinterpret_cast<uint4*>(sm + OFF_DO + sw128_chunk(i, DV / 2 * hf + 8 * e, 128)) = zz;
        }
        fence_proxy_async_smem();
      }
      ok = ok && wait(B_SC, ph) && wait(B_DS, ph);
      tc_fence_after();
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    float intra = 0.f;
    // ---- E and P, the decays' sums within the chunk; x and dO S^T scaled; the
    // first term of G ----------------------------------------------------------------------
    {
      term(OFF_T, G);
      fence_proxy_async_smem();
      const bool in = i < len;
      // the decays between block J and this row's
      auto between = [&](int J) -> float {
        return (w4 > 1 && J < 1 ? tot.y : 1.f) * (w4 > 2 && J < 2 ? tot.z : 1.f);
      };
      if (hf == 0) {
        // R(t) = sum_{j < t} D(t - 1, j) W_ij runs along the row; column t of
        // the block then sums D(i, t) R(t) over its rows
        float R = 0.f;
#pragma unroll 1
        for (int J = 0; J <= w4; ++J) {
          float dd[32];
          if (J == w4) {
            // D(i, t) in the diagonal block, from t = i down
            float run = 1.f;
            const float a = F[F_A + i];
#pragma unroll
            for (int t = 31; t >= 0; --t) {
              const float at = __shfl_sync(0xffffffffu, a, t);
              dd[t] = t <= lane ? run : 0.f;
              run = t <= lane ? run * at : run;
            }
          } else {
            const float d = pw * between(J);
#pragma unroll
            for (int t = 0; t < 32; t += 4) {
              const float4 f = *reinterpret_cast<const float4*>(F + F_SW + 32 * J + t);
              dd[t] = d * f.x; dd[t + 1] = d * f.y; dd[t + 2] = d * f.z; dd[t + 3] = d * f.w;
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            float s1[8], s2[8];
            tmem_ld8(row + TM_S1 + 32 * J + e, s1);
            tmem_ld8(row + TM_S2 + 32 * J + e, s2);
            tmem_ld_wait();
            if (J == w4 || len < C) {
              const int last = in ? (J == w4 ? lane : 31) : -1;
#pragma unroll
              for (int t = 0; t < 8; ++t) s1[t] = e + t <= last ? s1[t] * s2[t] : 0.f;
            } else {
#pragma unroll
              for (int t = 0; t < 8; ++t) s1[t] *= s2[t];
            }
#pragma unroll
            for (int t = 0; t < 8; t += 4) {
              const float4 f = *reinterpret_cast<const float4*>(F + F_A + 32 * J + e + t);
              dd[e + t] *= R;
              R = fmaf(f.x, R, s1[t]);
              dd[e + t + 1] *= R;
              R = fmaf(f.y, R, s1[t + 1]);
              dd[e + t + 2] *= R;
              R = fmaf(f.z, R, s1[t + 2]);
              dd[e + t + 3] *= R;
              R = fmaf(f.w, R, s1[t + 3]);
            }
          }
          if (J == w4 || len < C) {
            // (after the product with R, which need not be finite by now)
            const int last = in ? (J == w4 ? lane : 31) : -1;
#pragma unroll
            for (int t = 0; t < 32; ++t) dd[t] = t <= last ? dd[t] : 0.f;
          }
          // lane t gets the sum of dd[t] over the lanes
#pragma unroll
          for (int o = 16; o >= 1; o >>= 1) {
            const bool up = lane & o;
#pragma unroll
            for (int t = 0; t < o; ++t) {
              const float give = up ? dd[t] : dd[t + o];
              const float keep = up ? dd[t + o] : dd[t];
              dd[t] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
          }
          const float cs = dd[0];
          if (J == w4)
            intra = cs;
          else
            F[F_COL + 32 * (w4 * (w4 - 1) / 2 + J) + lane] = cs;
        }
      } else {
        float2 zero = make_float2(0.f, 0.f);  // NaN, if the diagonal block is not finite
#pragma unroll 1
        for (int J = 0; J < 4; ++J) {
          const float d = J < w4 ? pw * between(J) : 0.f;
          float run = in ? 1.f : 0.f;
          const float a = F[F_A + i];
#pragma unroll 1
          for (int e = 16; e >= 0; e -= 16) {
            float s1[16], s2[16];
            if (J <= w4) {
              tmem_ld16(row + TM_S1 + 32 * J + e, s1);
              tmem_ld16(row + TM_S2 + 32 * J + e, s2);
              tmem_ld_wait();
            }
            if (J == w4) {
#pragma unroll
              for (int t = 15; t >= 0; --t) {
                const float at = __shfl_sync(0xffffffffu, a, e + t);
                const bool on = e + t <= lane;
                s1[t] = on ? s1[t] * run : 0.f;
                s2[t] = on ? s2[t] * run : 0.f;
                run = on ? run * at : run;
              }
            } else if (J < w4) {
              const float2 d2 = make_float2(d, d);
#pragma unroll
              for (int t = 0; t < 16; t += 2) {
                const float2 f = mul2(d2, *reinterpret_cast<const float2*>(F + F_SW + 32 * J + e + t));
                const float2 x = mul2(make_float2(s1[t], s1[t + 1]), f);
                const float2 y = mul2(make_float2(s2[t], s2[t + 1]), f);
                s1[t] = x.x; s1[t + 1] = x.y;
                s2[t] = y.x; s2[t + 1] = y.y;
              }
            }
            if (J > w4 || !in) {
#pragma unroll
              for (int t = 0; t < 16; ++t) s1[t] = s2[t] = 0.f;
            }
            if (J == w4) {
#pragma unroll
              for (int t = 0; t < 16; ++t)
                zero = fma2(make_float2(s1[t], s2[t]), make_float2(0.f, 0.f), zero);
            }
#pragma unroll
            for (int t = 0; t < 16; t += 8) {
              const uint32_t o = sw128_chunk(i, 32 * J + e + t, 128);
              *reinterpret_cast<uint4*>(sm + OFF_P + o) = pack8(s1 + t);
              *reinterpret_cast<uint4*>(sm + OFF_E + o) = pack8(s2 + t);
            }
          }
        }
        if (!(zero.x + zero.y == 0.f)) *odd = 1;
        fence_proxy_async_smem();
      }
      tc_fence_before();
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    const bool rare = *odd != 0;  // (of the whole block)

    // ---- K G and V G^T with G's first term; x; diag(pre) dO S^T ---------------------------
    constexpr uint32_t id_kg = idesc_bf16(128, DV, 0, 1), id_vg = idesc_bf16(128, KD, 0, 0);
    constexpr uint32_t id_ek = idesc_bf16(128, KD, 0, 1);
    if (lead) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk)
          mma_f16(tmem + TM_DV, km(1, kk), mn(6, kk), id_kg, kk > 0);
#pragma unroll
        for (int kk = 0; kk < DV / 16; ++kk)
          mma_f16(tmem + TM_DK, km(2, kk), km(6, kk), id_vg, kk > 0);
        mma_commit(bar + B_G);
      }
      __syncwarp();
      issued = B_G;
      issued_par = g3;
    }
    {
      if (hf == 0) {
#pragma unroll
        for (int w = 1; w < 4; ++w)
          if (w > w4) intra += F[F_COL + 32 * (w * (w - 1) / 2 + w4) + lane];
      }
      const float x = scale_rows<KD / 2>(row + TM_DQ + KD / 2 * hf, pre, sm + OFF_Q, i, KD / 2 * hf);
      F[F_X + 128 * hf + i] = i < len ? x : 0.f;
      ok = wait(B_G, g3);
      term(OFF_T, G);
      fence_proxy_async_smem();
      tc_fence_before();
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    // ---- second term; E K -----------------------------------------------------------------
    if (lead) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk)
          mma_f16(tmem + TM_DV, km(1, kk), mn(6, kk), id_kg, 1u);
        mma_commit(bar + B_G);
        if (!rare) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_f16(tmem + TM_DQ, km(4, kk), mn(1, kk), id_ek, 1u);
        }
      }
      __syncwarp();
      issued = B_G;
      issued_par = g3 + 1;
    }
    {
      if (hf == 0) {
        F[F_X + i] += F[F_X + 128 + i];
        F[F_IN + i] = intra;
      }
      ok = wait(B_G, g3 + 1);
      term(OFF_T, G);
      fence_proxy_async_smem();
      if (un < p.units) {  // in registers until the next unit
        states(S, p.Sk, un);
        states(G, p.Gk, un);
      }
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    // ---- third term; y; diag(suf) K G, diag(suf) V G^T --------------------------------------
    if (lead) {
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk)
          mma_f16(tmem + TM_DV, km(1, kk), mn(6, kk), id_kg, 1u);
        mma_commit(bar + B_G);
      }
      __syncwarp();
      issued = B_G;
      issued_par = g3 + 2;
    }
    {
      ok = wait(B_G, g3 + 2);
      tc_fence_after();
      const float y = scale_rows<DV / 2>(row + TM_DV + DV / 2 * hf, suf, sm + OFF_V, i, DV / 2 * hf);
      F[(hf ? F_Y1 : F_Y0) + i] = i < len ? y : 0.f;
      scale_rows<KD / 2>(row + TM_DK + KD / 2 * hf, suf, nullptr, i, 0);
      if (__builtin_expect(rare && ok, 0)) {
        // (all readers of K but E K are through, and of Q and dO but E^T Q and P^T dO)
#pragma unroll 1
        for (int x = tid; x < 2 * KD + DV; x += kCompute) {
          int first, end;
          if (x < KD) {
            clean_column(sm + OFF_K, x, &first, &end);
            sm[OFF_KBAD + x] = (uint8_t)first;
          } else if (x < 2 * KD) {
            clean_column(sm + OFF_Q, x - KD, &first, &end);
            sm[OFF_QBAD + x - KD] = (uint8_t)end;
          } else {
            clean_column(sm + OFF_DO, x - 2 * KD, &first, &end);
            sm[OFF_OBAD + x - 2 * KD] = (uint8_t)end;
          }
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;

    // ---- P^T dO, E^T Q; the decays' gradient ------------------------------------------------
    if (lead) {
      tc_fence_after();
      if (elect_one()) {
        constexpr uint32_t id_dv = idesc_bf16(128, DV, 1, 1), id_dk = idesc_bf16(128, KD, 1, 1);
        if (rare) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) mma_f16(tmem + TM_DQ, km(4, kk), mn(1, kk), id_ek, 1u);
        }
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_f16(tmem + TM_DV, mn(5, kk), mn(3, kk), id_dv, 1u);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) mma_f16(tmem + TM_DK, mn(4, kk), mn(0, kk), id_dk, 1u);
        mma_commit(bar + B_FIN);
      }
      __syncwarp();
      issued = B_FIN;
      issued_par = ph;
    }
    {
      if (warp == 4) {
        float a[4], c[4], b[4], v[4], y[4], hd[4], tl[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 4 * lane + e, s = 127 - t;
          a[e] = F[F_A + t];
          y[e] = F[F_Y0 + t] + F[F_Y1 + t];
          c[e] = t > 0 ? F[F_A + s + 1] : 0.f;
          b[e] = F[F_X + s];
        }
        lin_scan(c, b, v, lane);  // X, from the end
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) F[F_X + 127 - 4 * lane - e] = v[e];
        lin_scan(a, y, v, lane);  // Y of the next position
        float Y = __shfl_up_sync(0xffffffffu, v[3], 1);
        if (lane == 0) Y = 0.f;
        const float all = (a[0] * a[1]) * (a[2] * a[3]);
        float up = __shfl_up_sync(0xffffffffu, warp_prefix(all, lane), 1);
        float down = warp_suffix(all, lane);
        if (lane == 0) up = 1.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          hd[e] = up;
          up *= a[e];
          tl[3 - e] = down;
          down *= a[3 - e];
        }
        float zz = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) zz += F[F_Z + e];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = 4 * lane + e;
          float g = F[F_IN + t];
          g = fmaf(hd[e], F[F_X + t], g);
          g = fmaf(tl[e], e > 0 ? v[e - 1] : Y, g);
          g = fmaf(hd[e] * tl[e], zz, g);
          if (t < len) p.da[(t0 + t) * p.H + h] = g;
        }
      }
      ok = wait(B_FIN, ph);
      tc_fence_after();
      if (lead) {
        loaded = false;
        if (ok && un < p.units) {
          if (lane == 0) load(t0n, hn);
          loaded = true;
          ld_par = ph ^ 1u;
        }
      }
      if (__builtin_expect(rare && ok, 0)) {
        poison_rows<KD / 2>(row + TM_DQ + KD / 2 * hf, i, sm + OFF_KBAD + KD / 2 * hf, false);
        poison_rows<KD / 2>(row + TM_DK + KD / 2 * hf, i, sm + OFF_QBAD + KD / 2 * hf, true);
        poison_rows<DV / 2>(row + TM_DV + DV / 2 * hf, i, sm + OFF_OBAD + DV / 2 * hf, true);
      }
      // the gradients' rows: whole chunks leave by TMA from the tiles of E, P
      // and G's terms, a partial one row by row
      auto give = [&](uint32_t col, uint32_t off, __nv_bfloat16* g, int D, int n0, int nn) {
#pragma unroll 1
        for (int e = n0; e < n0 + nn; e += 32) {
          float x[32];
          tmem_ld32(row + col + e, x);
          tmem_ld_wait();
          if (len == C) {
#pragma unroll
            for (int o = 0; o < 32; o += 8)
              *reinterpret_cast<uint4*>(sm + off + sw128_chunk(i, e + o, 128)) = pack8(x + o);
          } else if (i < len) {
            store_cols<32>(g + ((t0 + i) * p.H + h) * D + e, x);
          }
        }
      };
      if (ok) {
        give(TM_DQ, OFF_E, p.dq, KD, KD / 2 * hf, KD / 2);
        give(TM_DK, OFF_P, p.dk, KD, KD / 2 * hf, KD / 2);
        give(TM_DV, OFF_T, p.dv, DV, DV / 2 * hf, DV / 2);
      }
      fence_proxy_async_smem();
      tc_fence_before();
    }
    ok = __syncthreads_and(ok);
    if (!ok) break;
    if (lead && lane == 0 && len == C) {
      const int t = (int)t0;
      for (int x = 0; x < KD; x += 64) {
        tma_store_2d(&tm_dq, sb + OFF_E + 256 * x, h * KD + x, t);
        tma_store_2d(&tm_dk, sb + OFF_P + 256 * x, h * KD + x, t);
      }
      for (int x = 0; x < DV; x += 64) tma_store_2d(&tm_dv, sb + OFF_T + 256 * x, h * DV + x, t);
      bulk_commit();
    }
    tc_fence_after();
    u = un;
    len = lenn;
    t0 = t0n;
    h = hn;
    ph ^= 1u;
    g3 += 3;
  }
  if (lead && lane == 0) bulk_wait_all();
  if (!ok) {
    set_status(p.status, CKDA_ERR_DEVICE_TIMEOUT);
    // loads and products in flight get their time
    if (lead) {
      if (loaded) wait(B_LD, ld_par);
      if (issued != 0) wait(issued, issued_par);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace ck

}  // namespace bw
}  // namespace la

bool la_bwd_tc_supported(int dtype, int dk, int dv, int n_seqs, int T, int H, bool varlen) {
  const uint64_t rows = varlen ? (uint64_t)T : (uint64_t)n_seqs * (uint64_t)T;
  return dtype == CKDA_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128) && rows > 0 &&
         rows <= 0x7fffffffull - la::bw::C && (uint64_t)H * (dk > dv ? dk : dv) <= 0x7fffffffull;
}

size_t la_bwd_tc_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen,
                                 bool per_head) {
  const size_t slots = (size_t)la::chunk_slots(varlen, n_seqs, T, la::bw::C);
  const size_t tokens = varlen ? (size_t)T : (size_t)n_seqs * T;
  return 2 * slots * H * la::bw::state_floats(dv) * 4 + (per_head ? (tokens * H * 4 + 255) / 256 * 256 : 0);
}

cudaError_t launch_la_dalpha_sum(const float* part, float* da, int64_t tokens, int H,
                                 cudaStream_t stream);

cudaError_t launch_la_bwd_tc(int dk_, int dv_, const void* q, const void* k, const void* v,
                             const float* alpha, int per_head, const float* S0, const int32_t* cu,
                             const void* dO, const float* dSf, void* dq, void* dk, void* dv,
                             float* dalpha, float* dS0, void* ws, int n_seqs, int T, int H,
                             int* status, cudaStream_t stream) {
  using namespace la;
  const bool varlen = cu != nullptr;
  const uint64_t rows = varlen ? (uint64_t)T : (uint64_t)n_seqs * (uint64_t)T;
  const int64_t slots = chunk_slots(varlen, n_seqs, T, bw::C);
  float* Sk = static_cast<float*>(ws);
  const size_t all = (size_t)slots * H * bw::state_floats(dv_);
  float* Gk = Sk + all;
  float* part = per_head ? Gk + all : dalpha;
  const Decay al{alpha, H, per_head};
  CUtensorMap mq, mk, mv, mo, nq, nk, nv;
  const uint64_t ck_ = (uint64_t)H * dk_, cv = (uint64_t)H * dv_;
  if (!bf16_map(&mq, q, ck_, rows, bw::C) || !bf16_map(&mk, k, ck_, rows, bw::C) ||
      !bf16_map(&mv, v, cv, rows, bw::C) || !bf16_map(&mo, dO, cv, rows, bw::C) ||
      !bf16_map(&nq, dq, ck_, rows, bw::C) || !bf16_map(&nk, dk, ck_, rows, bw::C) ||
      !bf16_map(&nv, dv, cv, rows, bw::C))
    return cudaErrorInvalidValue;
  cudaError_t e;
  {
    auto ks = dk_ == 128 ? bw::st::la_states_kernel<128> : bw::st::la_states_kernel<64>;
    e = dk_ == 128 ? max_smem<10>(ks, bw::st::kSmem) : max_smem<11>(ks, bw::st::kSmem);
    if (e != cudaSuccess) return e;
    const bw::st::Args a{al, S0, dSf, Sk, Gk, dS0, cu, n_seqs, T, H, dv_, status};
    ks<<<(unsigned)n_seqs * H * 2 * (dv_ / bw::st::BV), bw::st::kThreads, bw::st::kSmem, stream>>>(
        mq, mk, mv, mo, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const bw::ck::Args a{al,
                       Sk,
                       Gk,
                       static_cast<__nv_bfloat16*>(dq),
                       static_cast<__nv_bfloat16*>(dk),
                       static_cast<__nv_bfloat16*>(dv),
                       part,
                       cu,
                       n_seqs,
                       T,
                       H,
                       slots * H,
                       status};
  const unsigned grid = (unsigned)(a.units < 148 ? a.units : 148);
  auto run = [&](auto kc, cudaError_t attr) -> cudaError_t {
    if (attr != cudaSuccess) return attr;
    kc<<<grid, bw::ck::kThreads, bw::ck::kSmem, stream>>>(mq, mk, mv, mo, nq, nk, nv, a);
    return cudaGetLastError();
  };
#define CKDA_LA_CHUNK(KD, DV)                      \
  run(bw::ck::la_chunk_kernel<KD, DV>,             \
      max_smem<20 + KD + DV / 64>(bw::ck::la_chunk_kernel<KD, DV>, bw::ck::kSmem))
  if (dk_ == 128)
    e = dv_ == 128 ? CKDA_LA_CHUNK(128, 128) : CKDA_LA_CHUNK(128, 64);
  else
    e = dv_ == 128 ? CKDA_LA_CHUNK(64, 128) : CKDA_LA_CHUNK(64, 64);
#undef CKDA_LA_CHUNK
  if (e != cudaSuccess) return e;
  return per_head ? launch_la_dalpha_sum(part, dalpha, (int64_t)rows, H, stream) : cudaSuccess;
}

}  // namespace ckda
