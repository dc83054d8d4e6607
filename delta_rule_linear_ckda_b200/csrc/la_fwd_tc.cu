// Head-decay linear attention on the tensor cores (tcgen05): bf16 inputs,
// d_k 64 or 128, d_v a multiple of 64 (sm_100a).
//
// Per chunk of C = 128 tokens (start state S, D(i, j) = a_{j+1} .. a_i):
//   O = (D o Q K^T) V + diag(pre) Q S,   S' = gamma S + K^T diag(suf) V,
// pre_i = a_0 .. a_i, suf_j = a_{j+1} .. a_{C-1}, gamma = a_0 .. a_{C-1}: two
// products on either side of the scores, and the state touched once per
// chunk.  The work is one read of q, k, v and one write of out: bound by HBM
// bandwidth, if the products and what feeds them keep up.
//
// One CTA walks the chunks of a (sequence, head) for 64 of the d_v columns
// (the slices of a head read the same q and k at about the same time, from L2
// but once).  Its warps have fixed roles and pass each chunk on through
// mbarriers:
//   warps 0..7   scores: tensor memory -> times the decays, masked -> bf16
//                operand in the same place; out: pre_i (Q S) + (P V), stored
//                (thread = row i; two warps share the columns of 32 rows)
//   warps 8..15  state: V's rows times suf as bf16 operands in shared memory;
//                S' = gamma S + product, in fp32 registers (thread = row of
//                d_k, half of the columns), its bf16 copy for the next chunk
//   warp 16      every MMA (one lane issues)
//   warp 17      every TMA load (one thread): q, k, v two chunks deep
//   warp 18      the decays' products of each chunk
//
// Decays are running products within aligned blocks of 32 tokens: prefW_i
// from the block's start through i, sufW_j from j + 1 to the block's end,
// tot_b of whole blocks; D(i, j) across blocks is prefW_i tot .. tot sufW_j.
// No logarithm and no division: zero and negative decays are exact, and
// underflow goes to zero.
//
// Roundings: the scores (after their decays) and the state's copy that the
// queries read are rounded once to bf16, like the inputs; both only reach
// out, whose error is 2.35e-3 (2-norm) in bf16 where the result's own rounding
// is 1.66e-3, and 1.66e-3 in fp32.  Second terms have no room: the 512 columns of
// tensor memory and all but 500 bytes of shared memory are in use.  Inputs in
// fp32 take the fp32 kernels.
//
// The state itself stays at fp32 accuracy: diag(suf) V is split into three bf16
// terms (24 bits) whose products with the exact bf16 K are one MMA with the
// terms side by side (N = 192): shared memory, whose bandwidth bounds this
// kernel, is read for K once instead of three times.
//
// P is zero right of the diagonal, but zero times a v that is not finite is
// not: such values are taken out of V's tile (never out of the state's
// operand) and the rows from their token on set to NaN, which is what the
// state, now NaN in that column, gives the later chunks.  Rows before it keep
// their values.  The check costs 1 % (B = 4, T = 4096, H = 16, d = 128: 88.8 ->
// 89.8 us; on V itself instead of the third terms 91.1).
//
// A sequence may be split into segments that run at the same time (few
// sequences and heads): a first launch computes each segment's own end state
// (K, V only), the second starts every segment from their decayed sum.

#include "la_common.cuh"
#include "sm100.cuh"
#include "la_tc.cuh"

namespace ckda {
namespace la {

using namespace sm100;

namespace fw {

constexpr int C = 128;
constexpr int DK = 128;  // rows of the state's product; those behind a d_k of 64 are zero
constexpr int BV = 64;  // d_v columns per CTA
constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s per wait

// shared memory
constexpr uint32_t OFF_Q = 0;                    // 2 stages [128][128] bf16, two 64-column atoms
constexpr uint32_t OFF_K = 65536;                // 2 stages, the same
constexpr uint32_t OFF_V = 131072;               // 2 stages [128][64]
constexpr uint32_t OFF_VW = 163840;              // diag(suf) V: 3 terms [128][64]
constexpr uint32_t OFF_SB = OFF_VW + 3 * 16384;  // bf16 state [128][64]
constexpr uint32_t OFF_DEC = OFF_SB + 16384;     // 2 x the decays (put_decays)
constexpr uint32_t kDecBytes = kDecFloats * 4;
constexpr uint32_t OFF_BAR = OFF_DEC + 2 * kDecBytes;
constexpr uint32_t OFF_MISC = OFF_BAR + 176;     // tensor-memory base, the sequence, whether any
                                                 // column has what follows
constexpr uint32_t OFF_BAD = OFF_MISC + 16;      // a column's first token (of this block's) whose v
                                                 // is not finite
constexpr uint32_t kSmem = OFF_BAD + 4 * BV;
static_assert(kSmem <= 232448, "shared memory");

// mbarriers, byte offsets from OFF_BAR; each completes once per chunk (those
// with two stages once per two)
constexpr uint32_t B_Q = 0, B_K = 16, B_V = 32;  // stage loaded, + 8 (c & 1)
constexpr uint32_t B_SC = 48;    // Q K^T complete (tensor core); the last chunk's P is free too
constexpr uint32_t B_P = 56;     // P written, the scores read
constexpr uint32_t B_VW = 64;    // diag(suf) V written, V's and K's tail rows cleared, the last
                                 // chunk's product read
constexpr uint32_t B_SB = 72;    // the state's operand written, V finite
constexpr uint32_t B_O = 80;     // Q S and P V complete (tensor core)
constexpr uint32_t B_OE = 88;    // and read
// complete (tensor core), + 8 (c & 1): the copy thread, which nothing holds
// to the chunk, waits for these too
constexpr uint32_t B_D = 96;     // K^T diag(suf) V
constexpr uint32_t B_QS = 112;   // Q S
constexpr uint32_t B_ST = 128;   // out staged where V was (or stored), + 8 (c & 1)
constexpr uint32_t B_DEC = 144;  // decays of a chunk written, + 8 (c & 1)
constexpr uint32_t B_DECE = 160; // and read, + 8 (c & 1)

// tensor-memory columns
constexpr uint32_t TM_SC = 0;    // Q K^T
constexpr uint32_t TM_P = 128;   // P, bf16 pairs
constexpr uint32_t TM_O1 = 192;  // Q S
constexpr uint32_t TM_O2 = 256;  // P V
constexpr uint32_t TM_D = 320;   // K^T diag(suf) V, three terms
constexpr uint32_t kTmemCols = 512;

constexpr int kThreads = 608;
constexpr int kHalf = BV / 2;  // columns per state or output thread

struct Args {
  Decay al;
  const float* S0;
  const int32_t* cu;
  void* out;
  float* Sf;
  int n_seqs, T, H, DV;
  int* status;
  // segments per sequence, and pieces per segment that the first launch takes
  // (np = seg_n piece_n of them); part[(n H + h) np + g]: for g > 0 the end
  // state of piece g - 1 (piece 0's from S0, the others' from zero), for
  // g = 0 a copy of S0; dec: the pieces' decays
  int seg_n, piece_n;
  float* part;
  float* dec;
};

// SUM: the pieces' own end states only (those of segments 0 .. seg_n - 2)
// KD: d_k
template <typename Tout, bool SUM, int KD>
__global__ void __launch_bounds__(kThreads, 1)
la_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
              const __grid_constant__ CUtensorMap tm_v,
              const __grid_constant__ CUtensorMap tm_o, const Args p) {
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t sb = smem_u32(sm);
  // (through a shuffle, so that the compiler knows the warp index as uniform)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // (the swizzled tiles need this; the base of dynamic shared memory has it)
  if ((sb & 1023u) != 0) {
    set_status(p.status, CKDA_ERR_CUDA);
    return;
  }

  const int slices = p.DV / BV;
  const int np = p.seg_n * p.piece_n;
  const int nseg = SUM ? np - p.piece_n : p.seg_n;
  // block index: column slice, then segment, then head, then sequence (longest first)
  int b = blockIdx.x;
  const int j0 = (b % slices) * BV;
  b /= slices;
  const int seg = b % nseg;
  b /= nseg;
  const int h = b % p.H;
  int* pick = reinterpret_cast<int*>(sm + OFF_MISC + 4);
  const int n = seq_longest_first(p.cu, p.n_seqs, b / p.H, pick);
  const SeqRange sr = seq_range(p.cu, n, p.n_seqs, p.T, p.status);
  if (!sr.ok) return;

  const uint32_t bar = sb + OFF_BAR;
  if (tid == 0) {
    for (int i = 0; i < 7; ++i) mbar_init(bar + 8 * i, 1);  // Q, K, V, scores
    mbar_init(bar + B_P, 8);
    mbar_init(bar + B_VW, 8);
    mbar_init(bar + B_SB, 8);
    mbar_init(bar + B_O, 1);
    mbar_init(bar + B_OE, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar + B_D + 8 * i, 1);
      mbar_init(bar + B_QS + 8 * i, 1);
      mbar_init(bar + B_ST + 8 * i, 8);
      mbar_init(bar + B_DEC + 8 * i, 1);
      mbar_init(bar + B_DECE + 8 * i, SUM ? 8 : 16);
    }
    fence_mbar_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    if (!SUM && sizeof(Tout) == 2) prefetch_tmap(&tm_o);  // (fp32 rows are stored by threads)
  }
  if (warp == 0) {
    tmem_alloc(sb + OFF_MISC, kTmemCols);
    tmem_relinquish();
  }
  int* bad_any = reinterpret_cast<int*>(sm + OFF_MISC + 8);
  int* bad_from = reinterpret_cast<int*>(sm + OFF_BAD);
  if constexpr (!SUM) {
    if (tid < BV) bad_from[tid] = INT32_MAX;
    if (tid == 0) *bad_any = 0;
  }
  if constexpr (KD < DK) {  // no load writes K's second 64 columns
    for (int e = tid; e < 2 * 16384 / 16; e += kThreads)
      *reinterpret_cast<uint4*>(sm + OFF_K + (e >> 10) * 32768 + 16384 + (e & 1023) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem =
      __shfl_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t*>(sm + OFF_MISC), 0);

  const int nck_all = (int)((sr.end - sr.begin + C - 1) / C);
  const int parts = SUM ? np : p.seg_n;  // (a segment ends where its last piece does)
  const int cbeg = (int)((int64_t)seg * nck_all / parts);
  const int nck =
      __shfl_sync(0xffffffffu, (int)((int64_t)(seg + 1) * nck_all / parts) - cbeg, 0);
  const int64_t tok0 = sr.begin + (int64_t)cbeg * C;
  auto len_of = [&](int c) -> int {
    const int64_t left = sr.end - (tok0 + (int64_t)c * C);
    return left < C ? (int)left : C;
  };
  auto wait = [&](uint32_t off, uint32_t par) -> bool {
    return mbar_wait_small(bar + off, par & 1u, kWaitNs);
  };
  const float* dec0 = reinterpret_cast<const float*>(sm + OFF_DEC);
  auto decs = [&](int c) { return dec0 + (c & 1) * (kDecBytes / 4); };
  auto suff = [&](int c) { return decs(c) + 128; };
  auto tots = [&](int c) { return decs(c) + 256; };
  // Whole chunks of bf16 leave by TMA from the V tile, which the products are
  // done with by then: a thread's own row would be four stores to 32 different
  // lines per warp, and 1024 cycles of the load / store unit per chunk.
  auto staged = [&](int c) -> bool { return sizeof(Tout) == 2 && len_of(c) == C; };
  // One arrival per warp, once all of its lanes are here: a lane's arrivals
  // on one mbarrier follow each other, 256 of them take some 500 cycles.
  auto arrive = [&](uint32_t off) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + off);
  };
  bool ok = true;
  // the copy thread's loads, bit 2 (Q, K, V) + stage: issued, and the parity of the last one
  uint32_t pend = 0, pend_par = 0;
  bool mma_open = false;
  uint32_t mma_off = 0, mma_par = 0;

  // Loops whose code would not stay in the instruction cache when unrolled
  // (19 warps run five different programs) are kept rolled on purpose.
  if (warp < 8) {
    // ---- scores and out ---------------------------------------------------------------------
    if constexpr (!SUM) {
      const int w4 = warp & 3, hf = warp >> 2;  // row block; which of its two warps
      const int i = 32 * w4 + lane;             // row
      const uint32_t row = tmem + ((uint32_t)(32 * w4) << 16);
      if (hf == 0) {
        // blocks right of the diagonal stay zero
        uint32_t z[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll 1
        for (int J = w4 + 1; J < 4; ++J) tmem_st16(row + TM_P + 16 * J, z);
        tmem_st_wait();
      }
      float pre = 0.f;
#pragma unroll 1
      for (int c = 0; c <= nck; ++c) {
        if (c > 0) {
          // out of the last chunk: its products end while this one's scores
          // are computed
          const int e = c - 1;
          if (!(ok = wait(B_O, e))) break;
          tc_fence_after();
          const bool st = staged(e), in = i < len_of(e);
          const bool bad = *reinterpret_cast<volatile int*>(bad_any) != 0;
          Tout* o = static_cast<Tout*>(p.out) +
                    ((size_t)(tok0 + (int64_t)e * C + i) * p.H + h) * p.DV + j0 + kHalf * hf;
#pragma unroll 1
          for (int u0 = 0; u0 < kHalf; u0 += 16) {
            float x[16], y[16];
            tmem_ld16(row + TM_O1 + kHalf * hf + u0, y);
            tmem_ld16(row + TM_O2 + kHalf * hf + u0, x);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < 16; ++u) x[u] = fmaf(pre, y[u], x[u]);
            if (__builtin_expect(bad, 0)) {
#pragma unroll
              for (int u = 0; u < 16; ++u)
                if (reinterpret_cast<volatile int*>(bad_from)[kHalf * hf + u0 + u] <= e * C + i)
                  x[u] = __int_as_float(0x7fffffff);
            }
            if (st) {
#pragma unroll
              for (int c8 = 0; c8 < 2; ++c8)
                *reinterpret_cast<uint4*>(sm + OFF_V + (e & 1) * 16384 +
                                          sw128_chunk(i, kHalf * hf + u0 + 8 * c8, 128)) =
                    pack8(x + 8 * c8);
            } else if (in) {
              store_cols<16>(o + u0, x);
            }
          }
          tc_fence_before();
          fence_proxy_async_smem();
          arrive(B_OE);
          if (lane == 0) mbar_arrive(bar + B_ST + 8 * (e & 1));
        }
        if (c == nck) break;
        if (!(ok = wait(B_DEC + 8 * (c & 1), c >> 1))) break;
        const float* sw = suff(c);
        const float4 tot = *reinterpret_cast<const float4*>(tots(c));
        const float a = decs(c)[i], pw = warp_prefix(a, lane);
        if (!(ok = wait(B_SC, c))) break;
        tc_fence_after();
        float s[32];
        uint32_t w[16];
        if (hf == 0) {
          // the diagonal block: D(i, j) runs down from 1 at j = i
          tmem_ld32(row + TM_SC + 32 * w4, s);
          tmem_ld_wait();
          float run = 1.f;
#pragma unroll
          for (int j = 31; j >= 0; --j) {
            const float aj = __shfl_sync(0xffffffffu, a, j);
            s[j] = j <= lane ? s[j] * run : 0.f;
            run = j <= lane ? run * aj : run;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(s[2 * e], s[2 * e + 1]);
          tmem_st16(row + TM_P + 16 * w4, w);
        }
        // blocks left of it: of the last rows the first warp takes block 0,
        // the second warp takes the others
        const int Jlo = hf == 0 ? 0 : (w4 == 3 ? 1 : 0);
        const int Jhi = hf == 0 ? (w4 == 3 ? 0 : -1) : w4 - 1;
#pragma unroll 1
        for (int J = Jhi; J >= Jlo; --J) {
          tmem_ld32(row + TM_SC + 32 * J, s);
          // the decays between block J and this row's
          float d = pw;
          if (w4 > 1 && J < 1) d *= tot.y;
          if (w4 > 2 && J < 2) d *= tot.z;
          const float2 d2 = make_float2(d, d);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float4 f = *reinterpret_cast<const float4*>(sw + 32 * J + 4 * e);
            const float2 x = mul2(make_float2(s[4 * e], s[4 * e + 1]),
                                  mul2(d2, make_float2(f.x, f.y)));
            const float2 y = mul2(make_float2(s[4 * e + 2], s[4 * e + 3]),
                                  mul2(d2, make_float2(f.z, f.w)));
            w[2 * e] = pack_bf16x2(x.x, x.y);
            w[2 * e + 1] = pack_bf16x2(y.x, y.y);
          }
          tmem_st16(row + TM_P + 16 * J, w);
        }
        tmem_st_wait();
        tc_fence_before();
        arrive(B_P);
        if (lane == 0) mbar_arrive(bar + B_DECE + 8 * (c & 1));
        pre = pw * (w4 > 0 ? tot.x : 1.f) * (w4 > 1 ? tot.y : 1.f) * (w4 > 2 ? tot.z : 1.f);
      }
    }
  } else if (warp < 16) {
    // ---- state ----------------------------------------------------------------------------
    const int q4 = warp & 3, hf = (warp >> 2) & 1;
    const int r = 32 * q4 + lane;  // token j of V, row i of the state
    const uint32_t row = tmem + ((uint32_t)(32 * q4) << 16);
    float S[kHalf];
#pragma unroll
    for (int e = 0; e < kHalf; ++e) S[e] = 0.f;
    const size_t unit = (size_t)n * p.H + h;
    const size_t at = ((size_t)r * p.DV) + j0 + kHalf * hf;  // this thread's columns of a state
    const size_t stsz = (size_t)KD * p.DV;
    const bool row_in = KD == DK || r < KD;
    float* part = p.part + unit * np * stsz + at;
    {
      // segment 0 starts from S0; with segments, from a copy of it that the
      // first launch keeps (the last segment may write S_final over S0 before
      // this block starts); the others from the decayed sum of the pieces' end
      // states before them
      float f = 1.f;
#pragma unroll 1
      for (int g = SUM ? seg : seg * p.piece_n; g >= 0; --g) {
        const float* src = nullptr;
        if (g > 0)
          src = SUM ? nullptr : part + g * stsz;
        else if (seg == 0 && p.S0 != nullptr)
          src = !SUM && p.seg_n > 1 ? part : p.S0 + unit * stsz + at;
        if (src != nullptr && row_in) {
#pragma unroll
          for (int e = 0; e < kHalf; e += 4) {
            const float4 x = *reinterpret_cast<const float4*>(src + e);
            S[e] = fmaf(f, x.x, S[e]);
            S[e + 1] = fmaf(f, x.y, S[e + 1]);
            S[e + 2] = fmaf(f, x.z, S[e + 2]);
            S[e + 3] = fmaf(f, x.w, S[e + 3]);
          }
        }
        if (!SUM && g > 0) f *= p.dec[unit * np + g - 1];
      }
      if (SUM && seg == 0 && p.S0 != nullptr && row_in) store_cols<kHalf>(part, S);
    }
    float gamma = 1.f, total = 1.f;
#pragma unroll 1
    for (int c = 0; c <= nck; ++c) {
      if (c > 0) {
        if (!(ok = wait(B_D + 8 * ((c - 1) & 1), (c - 1) >> 1))) break;
        tc_fence_after();
        const float2 g2 = make_float2(gamma, gamma);
#pragma unroll
        for (int e = 0; e < kHalf; e += 16) {
          float x[16], y[16], z3[16];
          tmem_ld16(row + TM_D + kHalf * hf + e, x);
          tmem_ld16(row + TM_D + BV + kHalf * hf + e, y);
          tmem_ld16(row + TM_D + 2 * BV + kHalf * hf + e, z3);
          tmem_ld_wait();
#pragma unroll
          for (int u = 0; u < 16; u += 2) {
            const float2 d = add2(make_float2(x[u], x[u + 1]),
                                  add2(make_float2(y[u], y[u + 1]), make_float2(z3[u], z3[u + 1])));
            const float2 z = fma2(g2, make_float2(S[e + u], S[e + u + 1]), d);
            S[e + u] = z.x;
            S[e + u + 1] = z.y;
          }
        }
        total *= gamma;
      }
      if (c == nck) break;
      // diag(suf) V into the product's operand, before the state's: it does
      // not wait for the queries' product with the last chunk's state
      const int st = c & 1;
      const int len = len_of(c);
      uint32_t odd = 0;  // the third terms' bits: NaN for a v that is not finite
      if (!(ok = wait(B_DEC + 8 * st, c >> 1))) break;
      {
        const float4 tot = *reinterpret_cast<const float4*>(tots(c));
        const float wgt = suff(c)[r] * (q4 < 1 ? tot.y : 1.f) * (q4 < 2 ? tot.z : 1.f) *
                          (q4 < 3 ? tot.w : 1.f);
        gamma = decs(c)[260];
        arrive(B_DECE + 8 * st);
        if (!(ok = wait(B_V + 8 * st, c >> 1))) break;
        if (len < C && !(ok = wait(B_K + 8 * st, c >> 1))) break;
        if (r < len) {
          const float2 w2 = make_float2(wgt, wgt);
#pragma unroll 1
          for (int h2 = 0; h2 < 2; ++h2) {
            const uint32_t o0 = sw128_chunk(r, kHalf * hf + 16 * h2, 128);
            const uint32_t o1 = o0 ^ 16u;  // the next 16 bytes under the swizzle
            const uint4 ra = *reinterpret_cast<const uint4*>(sm + OFF_V + st * 16384 + o0);
            const uint4 rb = *reinterpret_cast<const uint4*>(sm + OFF_V + st * 16384 + o1);
            const uint32_t in[8] = {ra.x, ra.y, ra.z, ra.w, rb.x, rb.y, rb.z, rb.w};
            uint32_t t1[8], t2[8], t3[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) split3(in[e], w2, &t1[e], &t2[e], &t3[e]);
            if constexpr (!SUM) {
#pragma unroll
              for (int e = 0; e < 8; e += 2) odd |= t3[e] | t3[e + 1];
            }
            uint8_t* d = sm + OFF_VW;
            *reinterpret_cast<uint4*>(d + o0) = make_uint4(t1[0], t1[1], t1[2], t1[3]);
            *reinterpret_cast<uint4*>(d + o1) = make_uint4(t1[4], t1[5], t1[6], t1[7]);
            *reinterpret_cast<uint4*>(d + 16384 + o0) = make_uint4(t2[0], t2[1], t2[2], t2[3]);
            *reinterpret_cast<uint4*>(d + 16384 + o1) = make_uint4(t2[4], t2[5], t2[6], t2[7]);
            *reinterpret_cast<uint4*>(d + 32768 + o0) = make_uint4(t3[0], t3[1], t3[2], t3[3]);
            *reinterpret_cast<uint4*>(d + 32768 + o1) = make_uint4(t3[4], t3[5], t3[6], t3[7]);
          }
        } else {
          // past the sequence's end lie other tokens, or none: V and K rows
          // cleared, so that no product meets what is not finite there
          const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
          for (int c8 = 0; c8 < kHalf / 8; ++c8) {
            const uint32_t o = sw128_chunk(r, kHalf * hf + 8 * c8, 128);
            *reinterpret_cast<uint4*>(sm + OFF_V + st * 16384 + o) = z;
#pragma unroll
            for (int e = 0; e < 3; ++e)
              *reinterpret_cast<uint4*>(sm + OFF_VW + e * 16384 + o) = z;
          }
#pragma unroll 1
          for (int c8 = 0; c8 < KD / 16; ++c8)
            *reinterpret_cast<uint4*>(sm + OFF_K + st * 32768 +
                                      sw128_chunk(r, (KD / 2) * hf + 8 * c8, 128)) = z;
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      arrive(B_VW);
      if constexpr (!SUM) {
        // (the highest bit of an exponent: set in NaN, and in the third term of a
        // v of 2^17 or more, which is let through here)
        if (__builtin_expect((odd & 0x40004000u) != 0, 0)) {
#pragma unroll 1
          for (int e = kHalf * hf; e < kHalf * (hf + 1); e += 8) {
            uint16_t* x =
                reinterpret_cast<uint16_t*>(sm + OFF_V + st * 16384 + sw128_chunk(r, e, 128));
            const uint4 w = *reinterpret_cast<const uint4*>(x);
            uint32_t zero = 0;  // times zero: a pair of zeros, or NaN
            asm("fma.rn.bf16x2 %0, %1, %5, %0;\n\tfma.rn.bf16x2 %0, %2, %5, %0;\n\t"
                "fma.rn.bf16x2 %0, %3, %5, %0;\n\tfma.rn.bf16x2 %0, %4, %5, %0;"
                : "+r"(zero)
                : "r"(w.x), "r"(w.y), "r"(w.z), "r"(w.w), "r"(0));
            if ((zero & 0x7fff7fffu) == 0) continue;
#pragma unroll 1
            for (int u = 0; u < 8; ++u)
              if ((x[u] & 0x7f80) == 0x7f80) {
                x[u] = 0;
                atomicMin(bad_from + e + u, c * C + r);
              }
            *reinterpret_cast<volatile int*>(bad_any) = 1;
          }
        }
        // (the old operand has been read)
        if (c > 0 && !(ok = wait(B_QS + 8 * (st ^ 1), (c - 1) >> 1))) break;
#pragma unroll
        for (int c8 = 0; c8 < kHalf / 8; ++c8)
          *reinterpret_cast<uint4*>(sm + OFF_SB + sw128_chunk(r, kHalf * hf + 8 * c8, 128)) =
              pack8(S + 8 * c8);
        fence_proxy_async_smem();
        arrive(B_SB);
      }
    }
    if (ok) {
      if (SUM) {
        if (row_in) store_cols<kHalf>(part + (seg + 1) * stsz, S);
        if (r == 0 && hf == 0 && j0 == 0) p.dec[unit * np + seg] = total;
      } else if (p.Sf != nullptr && seg == p.seg_n - 1 && row_in) {
        store_cols<kHalf>(p.Sf + unit * stsz + at, S);
      }
    }
  } else if (warp == 16) {
    // ---- MMA ------------------------------------------------------------------------------
    // (the whole warp waits, one lane issues)
    const uint64_t d_q = smem_desc(sb + OFF_Q, 16, 1024, kSwizzle128);
    const uint64_t d_k = smem_desc(sb + OFF_K, 16, 1024, kSwizzle128);
    const uint64_t d_km = smem_desc(sb + OFF_K, 16384, 1024, kSwizzle128);  // K^T (MN-major)
    const uint64_t d_v = smem_desc(sb + OFF_V, 16384, 1024, kSwizzle128);
    const uint64_t d_vw = smem_desc(sb + OFF_VW, 16384, 1024, kSwizzle128);
    const uint64_t d_sb = smem_desc(sb + OFF_SB, 16384, 1024, kSwizzle128);
    constexpr uint32_t id_sc = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t id_qs = idesc_bf16(128, BV, 0, 1);
    constexpr uint32_t id_pv = idesc_bf16(128, BV, 0, 1);
    constexpr uint32_t id_kv = idesc_bf16(128, 3 * BV, 1, 1);
    auto scores = [&](int c) {
      const uint64_t so = (uint64_t)(c & 1) * (32768 >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < KD / 16; ++kk) {
          const uint64_t ko = so + 1024 * (kk >> 2) + 2 * (kk & 3);
          mma_f16(tmem + TM_SC, d_q + ko, d_k + ko, id_sc, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar + B_SC);
      }
      __syncwarp();
      mma_open = true; mma_off = B_SC; mma_par = c;
    };
    if constexpr (!SUM) {
      if (nck > 0 && (ok = wait(B_Q, 0) && wait(B_K, 0))) scores(0);
    }
    for (int c = 0; ok && c < nck; ++c) {
      const uint32_t st = c & 1;
      const uint64_t so = (uint64_t)st * (32768 >> 4);
      // (V's rows written implies V loaded; K is waited for in full here)
      if (!(ok = wait(B_VW, c) && wait(B_K + 8 * st, c >> 1))) break;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_f16(tmem + TM_D, d_km + so + 128 * kk, d_vw + 128 * kk, id_kv, kk > 0 ? 1u : 0u);
        mma_commit(bar + B_D + 8 * st);
      }
      __syncwarp();
      mma_open = true; mma_off = B_D + 8 * st; mma_par = c >> 1;
      if constexpr (!SUM) {
        if (!(ok = wait(B_SB, c) && (c == 0 || wait(B_OE, c - 1)))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < KD / 16; ++kk)
            mma_f16(tmem + TM_O1, d_q + so + 1024 * (kk >> 2) + 2 * (kk & 3), d_sb + 128 * kk,
                    id_qs, kk > 0 ? 1u : 0u);
          mma_commit(bar + B_QS + 8 * st);
        }
        __syncwarp();
        mma_open = true; mma_off = B_QS + 8 * st; mma_par = c >> 1;
      }
      if constexpr (!SUM) {
        if (!(ok = wait(B_P, c))) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(tmem + TM_O2, tmem + TM_P + 8 * kk, d_v + (so >> 1) + 128 * kk,
                       id_pv, kk > 0 ? 1u : 0u);
          mma_commit(bar + B_O);
        }
        __syncwarp();
        mma_off = B_O; mma_par = c;
        // the next chunk's scores, last: K comes into its stage only after
        // the last chunk's product with it, and is then still on its way
        if (c + 1 < nck) {
          if (!(ok = wait(B_Q + 8 * (st ^ 1), (c + 1) >> 1) &&
                     wait(B_K + 8 * (st ^ 1), (c + 1) >> 1)))
            break;
          scores(c + 1);
        }
      }
    }
  } else if (warp == 17) {
    // ---- loads ----------------------------------------------------------------------------
    if (lane == 0) {
      auto issued = [&](int kind, int c) {
        const uint32_t bit = 1u << (2 * kind + (c & 1));
        pend |= bit;
        pend_par = (c >> 1 & 1) ? pend_par | bit : pend_par & ~bit;
      };
      auto tok = [&](int c) { return (int)(tok0 + (int64_t)c * C); };
      auto load_q = [&](int c) {
        const uint32_t bq = bar + B_Q + 8 * (c & 1), dst = sb + OFF_Q + (c & 1) * 32768;
        mbar_expect_tx(bq, 256 * KD);
        for (int x = 0; x < KD; x += 64) tma_load_2d(dst + 256 * x, &tm_q, h * KD + x, tok(c), bq);
        issued(0, c);
      };
      auto load_k = [&](int c) {
        const uint32_t bk = bar + B_K + 8 * (c & 1), dst = sb + OFF_K + (c & 1) * 32768;
        mbar_expect_tx(bk, 256 * KD);
        for (int x = 0; x < KD; x += 64) tma_load_2d(dst + 256 * x, &tm_k, h * KD + x, tok(c), bk);
        issued(1, c);
      };
      auto load_v = [&](int c) {
        const uint32_t bv = bar + B_V + 8 * (c & 1);
        mbar_expect_tx(bv, 16384);
        tma_load_2d(sb + OFF_V + (c & 1) * 16384, &tm_v, h * p.DV + j0, tok(c), bv);
        issued(2, c);
      };
      // into L2 two chunks ahead of the loads
      auto prefetch = [&](int c) {
        if (c >= nck) return;
        for (int x = 0; x < KD; x += 64) {
          if (!SUM) tma_prefetch_2d(&tm_q, h * KD + x, tok(c));
          tma_prefetch_2d(&tm_k, h * KD + x, tok(c));
        }
        tma_prefetch_2d(&tm_v, h * p.DV + j0, tok(c));
      };
      // out of chunk c; on return its stage of V is free
      auto send = [&](int c) -> bool {
        if (!wait(B_ST + 8 * (c & 1), c >> 1)) return false;
        if (staged(c)) {
          tma_store_2d(&tm_o, sb + OFF_V + (c & 1) * 16384, h * p.DV + j0, tok(c));
          bulk_commit();
          bulk_wait_read_all();
        }
        return true;
      };
      int c = 0;
      for (; c < 2 && c < nck; ++c) {
        if (!SUM) load_q(c);
        load_k(c);
        load_v(c);
      }
      prefetch(2);
      prefetch(3);
      // chunk c takes the stage of chunk c - 2 as its parts become free
      for (; c < nck; ++c) {
        if (!(ok = wait(B_D + 8 * (c & 1), (c >> 1) - 1))) break;
        load_k(c);
        if constexpr (!SUM) {
          if (!(ok = wait(B_QS + 8 * (c & 1), (c >> 1) - 1))) break;
          load_q(c);
        }
        if (!SUM && !(ok = send(c - 2))) break;
        load_v(c);
        prefetch(c + 2);
      }
      if constexpr (!SUM) {
        for (int e = nck > 2 ? nck - 2 : 0; ok && e < nck; ++e) ok = send(e);
        bulk_wait_all();
      }
      if (!ok) {
        // give the loads in flight their time before the block leaves
        for (int s = 0; s < 6; ++s)
          if (pend >> s & 1u) mbar_wait_bounded(bar + 8 * s, pend_par >> s & 1u, kWaitNs);
      }
    }
  } else if (warp == 18) {
    // ---- decays ---------------------------------------------------------------------------
    auto load = [&](int c, float* a) {
      const int len = c < nck ? len_of(c) : 0;
#pragma unroll
      for (int bk = 0; bk < 4; ++bk) {
        const int t = 32 * bk + lane;
        a[bk] = t < len ? p.al.now(tok0 + (int64_t)c * C + t, h) : 1.f;
      }
    };
    float a[4], nx[4];
    load(0, a);
    for (int c = 0; c < nck; ++c) {
      load(c + 1, nx);
      if (c >= 2 && !(ok = wait(B_DECE + 8 * (c & 1), (c >> 1) - 1))) break;
      put_decays(reinterpret_cast<float*>(sm + OFF_DEC) + (c & 1) * kDecFloats, a, lane);
#pragma unroll
      for (int bk = 0; bk < 4; ++bk) a[bk] = nx[bk];
      arrive(B_DEC + 8 * (c & 1));
    }
  }
  if (!ok) {
    set_status(p.status, CKDA_ERR_DEVICE_TIMEOUT);
    if (warp == 16 && mma_open) mbar_wait_bounded(bar + mma_off, mma_par & 1u, kWaitNs);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace fw

// Segments per sequence: as many as fill the SMs once, when whole sequences
// leave half of them or more without a CTA, and each keeps 8 chunks.
static int fwd_segments(int n_seqs, int T, int H, int dv, bool varlen) {
  const int64_t ctas = (int64_t)n_seqs * H * (dv / fw::BV);
  int64_t g = 148 / (ctas > 0 ? ctas : 1);
  const int64_t most = (int64_t)T / (n_seqs > 0 && varlen ? n_seqs : 1) / (8 * fw::C);
  if (g > most) g = most;
  return g < 1 ? 1 : (int)g;
}

// The first launch leaves the last segment out: smaller pieces fill the SMs.
// A segment adds up the states of all pieces before it, about 0.7 us each, so
// that there are no more than eight of them unless the segments alone are more.
// us with 1 / 2 / 4 / 8 pieces, d = 128: T = 4096, one head, 4 segments 44 / 42 /
// 46 / 57; T = 16384, one head, 16 segments 57 / 67 / 98 / 168; T = 65536, 32
// heads, 2 segments 1048 / 851 / 857.
static int fwd_pieces(int n_seqs, int H, int dv, int segs) {
  if (segs == 1) return 1;
  const int64_t ctas = (int64_t)n_seqs * H * (dv / fw::BV) * (segs - 1);
  const int64_t fill = 148 / ctas, most = 8 / (segs - 1);
  const int64_t n = fill < most ? fill : most;
  return n < 1 ? 1 : (int)n;
}

}  // namespace la

bool la_fwd_tc_supported(int dtype, int dk, int dv, int n_seqs, int T, int H, bool varlen) {
  const uint64_t rows = varlen ? (uint64_t)T : (uint64_t)n_seqs * (uint64_t)T;
  return dtype == CKDA_BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128) && rows > 0 &&
         rows <= 0x7fffffffull - la::fw::C &&
         (uint64_t)H * (dk > dv ? dk : dv) <= 0x7fffffffull;
}

size_t la_fwd_tc_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen) {
  const int g = la::fwd_segments(n_seqs, T, H, dv, varlen);
  const int np = g * la::fwd_pieces(n_seqs, H, dv, g);
  return g > 1 ? (size_t)n_seqs * H * np * ((size_t)dk * dv + 64) * 4 : 0;
}

namespace la {

template <int KD>
static cudaError_t fwd_run(int out_dtype, unsigned units, fw::Args a, const CUtensorMap& mq,
                           const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                           cudaStream_t stream) {
  cudaError_t e;
  if (a.seg_n > 1) {
    auto ks = fw::la_fwd_kernel<float, true, KD>;
    if ((e = max_smem<KD>(ks, fw::kSmem)) != cudaSuccess) return e;
    ks<<<units * (a.seg_n - 1) * a.piece_n, fw::kThreads, fw::kSmem, stream>>>(mq, mk, mv, mo, a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (out_dtype == CKDA_BF16) {
    auto kb = fw::la_fwd_kernel<__nv_bfloat16, false, KD>;
    if ((e = max_smem<KD + 1>(kb, fw::kSmem)) != cudaSuccess) return e;
    kb<<<units * a.seg_n, fw::kThreads, fw::kSmem, stream>>>(mq, mk, mv, mo, a);
  } else {
    auto kf = fw::la_fwd_kernel<float, false, KD>;
    if ((e = max_smem<KD + 2>(kf, fw::kSmem)) != cudaSuccess) return e;
    kf<<<units * a.seg_n, fw::kThreads, fw::kSmem, stream>>>(mq, mk, mv, mo, a);
  }
  return cudaGetLastError();
}

}  // namespace la

cudaError_t launch_la_fwd_tc(int out_dtype, int dk, int dv, const void* q, const void* k,
                             const void* v, const float* alpha, int per_head, const float* S0,
                             const int32_t* cu, void* out, float* S_final, void* ws, int n_seqs,
                             int T, int H, int* status, cudaStream_t stream) {
  using namespace la;
  const bool varlen = cu != nullptr;
  const uint64_t rows = varlen ? (uint64_t)T : (uint64_t)n_seqs * (uint64_t)T;
  CUtensorMap mq, mk, mv;
  CUtensorMap mo = {};
  if (!bf16_map(&mq, q, (uint64_t)H * dk, rows, fw::C) ||
      !bf16_map(&mk, k, (uint64_t)H * dk, rows, fw::C) ||
      !bf16_map(&mv, v, (uint64_t)H * dv, rows, fw::C))
    return cudaErrorInvalidValue;
  if (out_dtype == CKDA_BF16 && !bf16_map(&mo, out, (uint64_t)H * dv, rows, fw::C))
    return cudaErrorInvalidValue;
  const int g = fwd_segments(n_seqs, T, H, dv, varlen);
  const int np = g * fwd_pieces(n_seqs, H, dv, g);
  fw::Args a{{alpha, H, per_head}, S0, cu, out, S_final, n_seqs, T, H, dv, status, g, np / g,
             nullptr, nullptr};
  const unsigned units = (unsigned)n_seqs * H * (dv / fw::BV);
  if (g > 1) {
    a.part = static_cast<float*>(ws);
    a.dec = a.part + (size_t)n_seqs * H * np * dk * dv;
  }
  return dk == 128 ? fwd_run<128>(out_dtype, units, a, mq, mk, mv, mo, stream)
                   : fwd_run<64>(out_dtype, units, a, mq, mk, mv, mo, stream);
}

}  // namespace ckda
