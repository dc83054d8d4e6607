// Head-decay linear attention on fp32 CUDA cores: every head size and type
// that the tensor-core kernels do not take.
//
// Forward, token by token: S_t = a_t S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.
// With G_t the adjoint of S_t (G_t = q_t do_t^T + a_{t+1} G_{t+1}) the
// gradients are the same recurrence with other operands:
//   dq_t = S_t do_t    queries do, keys v, values k  (state S^T, forward in time)
//   dk_t = G_t v_t     queries v, keys do, values q  (state G^T, backward in time)
//   dv_t = G_t^T k_t   queries k, keys q, values do  (state G, backward in time)
// so one kernel runs all four.  The decay's gradient da_t = <S_{t-1}, G_t>
// is put together chunk by chunk from the states at the chunk's bounds,
// which the dq and dv runs leave behind (la_dalpha_kernel).
//
// A recurrence costs 3 d_k d_v fp32 operations per token (the decay and the
// outer product, the product with the queries): as many as the chunked form
// with 64-token chunks needs without tensor cores, and it keeps full fp32
// accuracy.  The kernel is bound by instruction issue and, with few CTAs, by the
// latency of a token's chain.  A CTA owns 32 (16) columns of one (sequence,
// head)'s state in registers; row groups of 128 threads, of one or two columns
// each, split the rows.  Two rows share one packed fp32 instruction.
// Tokens come 16 at a time through shared memory, the next 16 already on
// their way in registers; the row groups' shares of the outputs are summed
// once per 16 tokens, so no barrier stands between tokens.
//
// A recurrence of few heads leaves most SMs empty and takes as long as its
// tokens take one after another.  Its sequences are then split into segments
// of whole chunks that run at the same time: a first launch carries each
// segment's own state to its end (keys and values only), the second starts
// every segment from their decayed sum (backward of B = 2, T = 1000, H = 4,
// d = 64, fp32, with the decays' gradient: 174 -> 78 us).
#include <type_traits>

#include "la_common.cuh"

namespace ckda {
namespace la {

constexpr int kTile = 16;     // tokens per shared-memory tile
constexpr int kRecThreads = 128;
constexpr int kChunk = 64;    // tokens per chunk of the decay gradient
static_assert(kChunk % kTile == 0, "tiles per chunk");

struct RecArgs {
  const void *q, *k, *v;
  Decay al;
  // element (i, j) of a state of (n, h): base + (n H + h) DK DV + i si + j sj
  const float* X0;  // or NULL
  float* Xf;        // or NULL
  int si, sj;
  void* out;
  // the state at each chunk's near bound (forward: its start, backward: its
  // end), [slot, h, DK, DV], or NULL
  float* kept;
  const int32_t* cu;
  int n_seqs, T, H, DV;
  int* status;
  // segments per sequence, numbered in the order of the recurrence;
  // part[(n H + h) seg_n + g], [DK, DV]: for g > 0 the end state of segment
  // g - 1 (segment 0's from X0, the others' from zero), for g = 0 a copy of
  // X0; dec: the segments' decays
  int seg_n;
  float* part;
  float* dec;
};

// Columns per thread: what a thread reads of k and q from shared memory serves
// all of its columns.  Two, if that leaves a thread four rows (the backward's
// second launch, d = 128, B = 4, T = 2048, H = 4: 339 us with one column, 318
// with two).
template <int DK, int COLS>
constexpr int kCpt = DK * COLS / kRecThreads >= 8 ? 2 : 1;

template <int DK, int COLS>
struct RecSmem {
  float sq[kTile][DK], sk[kTile][DK], sv[kTile][COLS], sa[kTile];
  float red[kTile][kRecThreads * kCpt<DK, COLS> / COLS][COLS];
};

// SUM: the segments' own end states only (all but the last segment)
template <int DK, int COLS, typename Tin, typename Tout, bool REV, bool SUM>
__device__ __forceinline__ void rec_body(const RecArgs& p, unsigned block, RecSmem<DK, COLS>& sm) {
  constexpr int CPT = kCpt<DK, COLS>;           // columns per thread
  constexpr int RG = kRecThreads * CPT / COLS;  // row groups
  constexpr int RPT = DK / RG;                  // rows per thread
  constexpr int LQ = kTile * DK / kRecThreads;
  constexpr int LV = kTile * COLS / kRecThreads;
  static_assert(RPT % 2 == 0 && LQ >= 1 && LV >= 1, "shape");
  auto& sq = sm.sq;
  auto& sk = sm.sk;
  auto& sv = sm.sv;
  auto& sa = sm.sa;
  auto& red = sm.red;

  const int tid = threadIdx.x;
  const int col = tid % (COLS / CPT) * CPT, g = tid / (COLS / CPT);
  // block index: column slice, then segment, then head, then sequence (longest first)
  const int slices = p.DV / COLS, nseg = SUM ? p.seg_n - 1 : p.seg_n;
  const int j0 = (int)(block % slices) * COLS;
  block /= slices;
  const int seg = (int)(block % nseg);
  block /= nseg;
  const int h = (int)(block % p.H);
  const int n = seq_longest_first(p.cu, p.n_seqs, (int)(block / p.H));
  const SeqRange sr = seq_range(p.cu, n, p.n_seqs, p.T, p.status);
  if (!sr.ok) return;
  const int len = (int)(sr.end - sr.begin);
  const int ntiles = (len + kTile - 1) / kTile;
  constexpr int per = kChunk / kTile;
  // this segment's tiles [tb, te)
  int tb = 0, te = ntiles;
  if (p.seg_n > 1) {
    const int64_t nck = (len + kChunk - 1) / kChunk;
    const int g = REV ? p.seg_n - 1 - seg : seg;
    tb = (int)(g * nck / p.seg_n) * per;
    te = min(ntiles, (int)((g + 1) * nck / p.seg_n) * per);
  }
  const Tin* q = static_cast<const Tin*>(p.q);
  const Tin* k = static_cast<const Tin*>(p.k);
  const Tin* v = static_cast<const Tin*>(p.v);

  const size_t unit = (size_t)n * p.H + h, st0 = unit * DK * p.DV;
  const int i0 = g * RPT;
  // this thread's columns of part's states
  float* part = p.part + unit * p.seg_n * DK * p.DV + (size_t)i0 * p.DV + j0 + col;
  float2 X[CPT][RPT / 2];
  auto put = [&](float* o) {  // rows of p.DV columns
#pragma unroll
    for (int r = 0; r < RPT / 2; ++r)
#pragma unroll
      for (int c = 0; c < CPT; ++c) {
        o[(size_t)(2 * r) * p.DV + c] = X[c][r].x;
        o[(size_t)(2 * r + 1) * p.DV + c] = X[c][r].y;
      }
  };
#pragma unroll
  for (int c = 0; c < CPT; ++c)
#pragma unroll
    for (int r = 0; r < RPT / 2; ++r) X[c][r] = make_float2(0.f, 0.f);
  if (p.X0 != nullptr && (SUM ? seg == 0 : p.seg_n == 1)) {
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      const float* b = p.X0 + st0 + (size_t)(j0 + col + c) * p.sj;
#pragma unroll
      for (int r = 0; r < RPT / 2; ++r)
        X[c][r] = make_float2(b[(size_t)(i0 + 2 * r) * p.si], b[(size_t)(i0 + 2 * r + 1) * p.si]);
    }
    // (the second launch starts from a copy: its last segment may write Xf
    // over X0 before its first one starts)
    if constexpr (SUM) put(part);
  }
  if (!SUM && p.seg_n > 1) {
    float f = 1.f;
#pragma unroll 1
    for (int e = seg; e >= 0; --e) {
      if (e > 0 || (seg == 0 && p.X0 != nullptr)) {
        const float* b = part + (size_t)e * DK * p.DV;
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int c = 0; c < CPT; ++c)
#pragma unroll
          for (int r = 0; r < RPT / 2; ++r)
            X[c][r] = fma2(f2, make_float2(b[(size_t)(2 * r) * p.DV + c],
                                           b[(size_t)(2 * r + 1) * p.DV + c]), X[c][r]);
      }
      if (e > 0) f *= p.dec[unit * p.seg_n + e - 1];
    }
  }
  double total = 1.0;  // SUM: this thread's share of the segment's decay

  float rq[LQ], rk[LQ], rv[LV], ra = 0.f;
  // the tile's rows past the sequence's end are zero, so that what lies
  // behind it is never read
  auto fetch = [&](int tl) {
    const int64_t t0 = sr.begin + (int64_t)tl * kTile;
    const int rows = min(kTile, len - tl * kTile);
#pragma unroll
    for (int e = 0; e < LQ; ++e) {
      const int x = tid + e * kRecThreads, t = x / DK, i = x % DK;
      const size_t at = ((size_t)(t0 + t) * p.H + h) * DK + i;
      if constexpr (!SUM) rq[e] = t < rows ? Elem<Tin>::to_f32(q[at]) : 0.f;
      rk[e] = t < rows ? Elem<Tin>::to_f32(k[at]) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < LV; ++e) {
      const int x = tid + e * kRecThreads, t = x / COLS, j = x % COLS;
      rv[e] = t < rows ? Elem<Tin>::to_f32(v[((size_t)(t0 + t) * p.H + h) * p.DV + j0 + j]) : 0.f;
    }
    if (tid < kTile) ra = tid < rows ? p.al.at(t0 + tid, h) : 1.f;
  };

  const int64_t slot0 = p.kept != nullptr ? slot_of(p.cu, n, p.T, kChunk) : 0;
  const int mine = te - tb;
  if (mine > 0) fetch(REV ? te - 1 : tb);
  for (int it = 0; it < mine; ++it) {
    const int tl = REV ? te - 1 - it : tb + it;
    const int64_t t0 = sr.begin + (int64_t)tl * kTile;
    const int rows = min(kTile, len - tl * kTile);
    __syncthreads();  // the last tile's reads are done
#pragma unroll
    for (int e = 0; e < LQ; ++e) {
      const int x = tid + e * kRecThreads;
      if constexpr (!SUM) sq[x / DK][x % DK] = rq[e];
      sk[x / DK][x % DK] = rk[e];
    }
#pragma unroll
    for (int e = 0; e < LV; ++e) {
      const int x = tid + e * kRecThreads;
      sv[x / COLS][x % COLS] = rv[e];
    }
    if (tid < kTile) {
      sa[tid] = ra;
      if constexpr (SUM) total *= (double)ra;
    }
    __syncthreads();
    if (it + 1 < mine) fetch(REV ? tl - 1 : tl + 1);

    if (!SUM && p.kept != nullptr && (REV ? (tl % per == per - 1 || tl == ntiles - 1) : tl % per == 0)) {
      put(p.kept + ((size_t)(slot0 + tl / per) * p.H + h) * DK * p.DV + (size_t)i0 * p.DV + j0 + col);
    }
    // Backward in time the decay of token t acts behind its own term: it is
    // applied with token t - 1's, and the tile's first token's at the end.
    // Four tokens at a time, so that one's loads from shared memory and sums
    // run under another's.
    auto token = [&](int t, float a) {
      const float2 a2 = make_float2(a, a);
      float2 o[CPT], o1[CPT];
#pragma unroll
      for (int c = 0; c < CPT; ++c) o[c] = o1[c] = make_float2(0.f, 0.f);
#pragma unroll
      for (int r = 0; r < RPT / 2; ++r) {
        const float2 k2 = *reinterpret_cast<const float2*>(&sk[t][i0 + 2 * r]);
        float2 q2 = k2;
        if constexpr (!SUM) q2 = *reinterpret_cast<const float2*>(&sq[t][i0 + 2 * r]);
#pragma unroll
        for (int c = 0; c < CPT; ++c) {
          const float vv = sv[t][col + c];
          X[c][r] = fma2(X[c][r], a2, mul2(k2, make_float2(vv, vv)));
          if constexpr (!SUM) {
            if (r & 1)
              o1[c] = fma2(q2, X[c][r], o1[c]);
            else
              o[c] = fma2(q2, X[c][r], o[c]);
          }
        }
      }
      if constexpr (!SUM) {
#pragma unroll
        for (int c = 0; c < CPT; ++c)
          red[t][g][col + c] = (o[c].x + o1[c].x) + (o[c].y + o1[c].y);
      }
    };
    if (rows == kTile) {
#pragma unroll 4
      for (int tt = 0; tt < kTile; ++tt) {
        const int t = REV ? kTile - 1 - tt : tt;
        token(t, REV ? (tt == 0 ? 1.f : sa[t + 1]) : sa[t]);
      }
    } else {
#pragma unroll 1
      for (int tt = 0; tt < rows; ++tt) {
        const int t = REV ? rows - 1 - tt : tt;
        token(t, REV ? (tt == 0 ? 1.f : sa[t + 1]) : sa[t]);
      }
    }
    if (REV) {
      const float2 a2 = make_float2(sa[0], sa[0]);
#pragma unroll
      for (int c = 0; c < CPT; ++c)
#pragma unroll
        for (int r = 0; r < RPT / 2; ++r) X[c][r] = mul2(X[c][r], a2);
    }
    if constexpr (SUM) continue;
    __syncthreads();
    if (p.out != nullptr) {
      Tout* out = static_cast<Tout*>(p.out);
#pragma unroll
      for (int e = 0; e < LV; ++e) {
        const int x = tid + e * kRecThreads, t = x / COLS, j = x % COLS;
        if (t < rows) {
          float s = red[t][0][j];
#pragma unroll
          for (int gg = 1; gg < RG; ++gg) s += red[t][gg][j];
          out[((size_t)(t0 + t) * p.H + h) * p.DV + j0 + j] = Elem<Tout>::from_f32(s);
        }
      }
    }
  }
  if constexpr (SUM) {
    put(part + (size_t)(seg + 1) * DK * p.DV);
    if (tid < kTile) {
#pragma unroll
      for (int o = kTile / 2; o >= 1; o >>= 1)
        total *= __shfl_xor_sync(0xffffffffu >> (32 - kTile), total, o);
      if (tid == 0 && j0 == 0) p.dec[unit * p.seg_n + seg] = (float)total;
    }
  } else if (p.Xf != nullptr && seg == p.seg_n - 1) {
#pragma unroll
    for (int c = 0; c < CPT; ++c) {
      float* b = p.Xf + st0 + (size_t)(j0 + col + c) * p.sj;
#pragma unroll
      for (int r = 0; r < RPT / 2; ++r) {
        b[(size_t)(i0 + 2 * r) * p.si] = X[c][r].x;
        b[(size_t)(i0 + 2 * r + 1) * p.si] = X[c][r].y;
      }
    }
  }
}

template <int DK, int COLS, typename Tin, typename Tout, bool REV, bool SUM>
__global__ void __launch_bounds__(kRecThreads, 4) la_rec_kernel(const RecArgs p) {
  __shared__ __align__(16) RecSmem<DK, COLS> sm;
  rec_body<DK, COLS, Tin, Tout, REV, SUM>(p, blockIdx.x, sm);
}

// The backward's three recurrences at once, when d_k = d_v: they do not depend
// on one another, and a recurrence by itself leaves most SMs empty when there
// are few heads.
struct Rec3Args {
  RecArgs fwd, rev[2];
};

template <int DK, int COLS, typename T, bool SUM>
__global__ void __launch_bounds__(kRecThreads, 4) la_rec3_kernel(const Rec3Args p) {
  __shared__ __align__(16) RecSmem<DK, COLS> sm;
  const unsigned which = blockIdx.x % 3, block = blockIdx.x / 3;
  if (which == 0)
    rec_body<DK, COLS, T, T, false, SUM>(p.fwd, block, sm);
  else
    rec_body<DK, COLS, T, T, true, SUM>(p.rev[which - 1], block, sm);
}

constexpr int rec_columns(int dv) { return dv == 16 ? 16 : 32; }

// Segments per sequence of recurrences with `dv` columns that run together:
// as many as give every SM four CTAs, if each keeps a chunk, and at most
// sqrt(T / 2), since the last segment adds up the states of all others.  One
// head forward, fp32, us with 16 / 32 / 64 / 128 segments:
//   T = 2048   d = 16: 18 / 18,             64: 30 / 24,             128: 42 / 33
//   T = 8192   d = 16: 47 / 32 / 28 / 36,   64: 87 / 52 / 42 / 50,   128: 127 / 75 / 70 / 95
//   T = 32768  d = 16: 161 / 89 / 56 / 49,  64: 316 / 167 / 99 / 90, 128: 469 / 247 / 204 / 212
// A launch takes as long as its longest segment, so that the count is one which
// gives them all about the same number of chunks (T = 8192, d = 128: 40 segments
// of 3 or 4 chunks 99 us, 64 of 2 chunks 70).
static int rec_segments(int together, int n_seqs, int T, int H, int dv, bool varlen) {
  const int64_t ctas = (int64_t)together * n_seqs * H * (dv / rec_columns(dv));
  const int64_t len = (int64_t)T / (n_seqs > 0 && varlen ? n_seqs : 1);
  int64_t g = 148 * 4 / (ctas > 0 ? ctas : 1);
  if (g > len / kChunk) g = len / kChunk;
  while (g > 1 && 2 * g * g > len) --g;
  if (g < 2) return 1;
  const int64_t chunks = (len + kChunk - 1) / kChunk, per = (chunks + g - 1) / g;
  return (int)((chunks + per - 1) / per);
}

// Floats of the segments' states and decays.
static size_t part_floats(int dk, int dv, int n_seqs, int H, int seg_n) {
  return seg_n > 1 ? (size_t)n_seqs * H * seg_n * ((size_t)dk * dv + 64) : 0;
}

static void set_parts(RecArgs* a, int dk, int seg_n, float* ws) {
  a->seg_n = seg_n;
  a->part = ws;
  a->dec = seg_n > 1 ? ws + (size_t)a->n_seqs * a->H * seg_n * dk * a->DV : nullptr;
}

template <int DK, int COLS, typename T>
static cudaError_t rec3_launch(const Rec3Args& a, cudaStream_t st) {
  const RecArgs& f = a.fwd;
  const unsigned n = 3u * (unsigned)(f.DV / COLS) * f.H * f.n_seqs;
  if (f.seg_n > 1) {
    la_rec3_kernel<DK, COLS, T, true><<<n * (f.seg_n - 1), kRecThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  la_rec3_kernel<DK, COLS, T, false><<<n * f.seg_n, kRecThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
static cudaError_t rec3(int d, const Rec3Args& a, cudaStream_t st) {
  switch (d) {
    case 16: return rec3_launch<16, 16, T>(a, st);
    case 32: return rec3_launch<32, 32, T>(a, st);
    case 64: return rec3_launch<64, 32, T>(a, st);
    case 128: return rec3_launch<128, 32, T>(a, st);
  }
  return cudaErrorInvalidValue;
}

template <int DK, int COLS, typename Tin, typename Tout, bool REV>
static cudaError_t rec_run(const RecArgs& a, cudaStream_t st) {
  const unsigned n = (unsigned)(a.DV / COLS) * a.H * a.n_seqs;
  if (a.seg_n > 1) {
    // (which has no output)
    la_rec_kernel<DK, COLS, Tin, Tin, REV, true><<<n * (a.seg_n - 1), kRecThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  la_rec_kernel<DK, COLS, Tin, Tout, REV, false><<<n * a.seg_n, kRecThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <int DK, int COLS, typename Tin, typename Tout>
static cudaError_t rec_launch(const RecArgs& a, bool rev, cudaStream_t st) {
  // Backward in time there is one type, and d_k = d_v = 16 runs in la_rec3_kernel.
  if constexpr (std::is_same<Tin, Tout>::value && DK + COLS > 32) {
    if (rev) return rec_run<DK, COLS, Tin, Tout, true>(a, st);
  }
  return rev ? cudaErrorInvalidValue : rec_run<DK, COLS, Tin, Tout, false>(a, st);
}

template <int DK, typename Tin, typename Tout>
static cudaError_t rec_cols(const RecArgs& a, bool rev, cudaStream_t st) {
  return a.DV == 16 ? rec_launch<DK, 16, Tin, Tout>(a, rev, st)
                    : rec_launch<DK, 32, Tin, Tout>(a, rev, st);
}

template <typename Tin, typename Tout>
static cudaError_t rec_rows(int dk, const RecArgs& a, bool rev, cudaStream_t st) {
  switch (dk) {
    case 16: return rec_cols<16, Tin, Tout>(a, rev, st);
    case 32: return rec_cols<32, Tin, Tout>(a, rev, st);
    case 64: return rec_cols<64, Tin, Tout>(a, rev, st);
    case 128: return rec_cols<128, Tin, Tout>(a, rev, st);
  }
  return cudaErrorInvalidValue;
}

static cudaError_t rec(int dtype, int out_dtype, int dk, const RecArgs& a, bool rev,
                       cudaStream_t st) {
  if (dtype == CKDA_BF16)
    return out_dtype == CKDA_BF16 ? rec_rows<__nv_bfloat16, __nv_bfloat16>(dk, a, rev, st)
                                  : rec_rows<__nv_bfloat16, float>(dk, a, rev, st);
  return out_dtype == CKDA_BF16 ? rec_rows<float, __nv_bfloat16>(dk, a, rev, st)
                                : rec_rows<float, float>(dk, a, rev, st);
}

// ---- the decay's gradient --------------------------------------------------------
//
// Within a chunk (positions 0..L-1, start state S, adjoint G of the state at
// its end, D(i, j) = a_{j+1} .. a_i):
//   da_t = sum_{i >= t > j} D(i, t) D(t-1, j) (q_i.k_j) (do_i.v_j)
//        + head_t sum_{i >= t} D(i, t) x_i + tail_t sum_{j < t} D(t-1, j) y_j
//        + head_t tail_t <S, G>
// with x_i = do_i . S^T q_i, y_j = v_j . G^T k_j, head_t = a_0 .. a_{t-1} and
// tail_t = a_{t+1} .. a_{L-1}: the products leave a_t out instead of dividing
// by it, so a zero decay has its gradient too.  The double sum is
//   U_t[j] = W[t][j] + a_{t+1} U_{t+1}[j],   sum_j D(t-1, j) U_t[j],
// one column j per thread.
struct DalphaArgs {
  const void *q, *k, *v, *dO;
  Decay al;
  const float* St;  // S^T at the chunks' starts [slot, h, DV, DK]
  const float* G;   // G at the chunks' ends [slot, h, DK, DV]
  float* da;        // [tokens, H]
  const int32_t* cu;
  int n_seqs, T, H, DK, DV;
  int* status;
};

constexpr int kDaThreads = 256;
constexpr int kSlab = 16;  // inner dimension per shared-memory slab (head sizes are multiples)

// Two C x C products at a time (q k^T with do v^T, then q S with k G, whose
// slabs of S and G also give <S, G>): the next slab's four tiles are on their
// way in registers while this one's are multiplied.  With few chunks the
// kernel's time is this chain of slabs; one product at a time without the
// loads ahead took 105 us per CTA at d_k = 64, d_v = 128.
template <typename Tin>
__global__ void __launch_bounds__(kDaThreads, 2) la_dalpha_kernel(const DalphaArgs p) {
  constexpr int C = kChunk, PT = C * kSlab / kDaThreads;
  __shared__ float sa[C], sx[C], sy[C], head[C], tail[C], zs[kDaThreads / 32];
  // the tiles, and E in their place once the products are done
  struct Tiles {
    float t[4][kSlab][C + 4];
  };
  union Scratch {
    Tiles tiles;
    float e[C][C + 1];
  };
  __shared__ __align__(16) Scratch sc;
  __shared__ float W[C][C + 1];
  auto& tl = sc.tiles.t;
  auto& E = sc.e;
  const int tid = threadIdx.x;
  const int h = blockIdx.y;
  int n, c;
  if (!slot_chunk(p.cu, p.n_seqs, p.T, C, blockIdx.x, &n, &c)) return;
  const SeqRange sr = seq_range(p.cu, n, p.n_seqs, p.T, p.status);
  if (!sr.ok) return;
  const int64_t t0 = sr.begin + (int64_t)c * C;
  const int L = (int)min((int64_t)C, sr.end - t0);
  const Tin* q = static_cast<const Tin*>(p.q);
  const Tin* k = static_cast<const Tin*>(p.k);
  const Tin* v = static_cast<const Tin*>(p.v);
  const Tin* dO = static_cast<const Tin*>(p.dO);
  const int ty = tid / 16, tx = tid % 16;  // this thread's 4 x 4 block of a C x C product

  if (tid < C) {
    sa[tid] = tid < L ? p.al.at(t0 + tid, h) : 1.f;
    sx[tid] = 0.f;
    sy[tid] = 0.f;
  }
  float r[4][PT];  // the next slab's tiles
  // columns d0 .. d0 + kSlab of a tensor's rows (zero behind the chunk and the head)
  auto get_rows = [&](float* o, const Tin* x, int D, int d0) {
#pragma unroll
    for (int e = 0; e < PT; ++e) {
      const int at = tid + e * kDaThreads, row = at / kSlab, d = d0 + at % kSlab;
      o[e] = row < L && d < D ? Elem<Tin>::to_f32(x[((size_t)(t0 + row) * p.H + h) * D + d]) : 0.f;
    }
  };
  auto put_rows = [&](int tile, const float* x) {
#pragma unroll
    for (int e = 0; e < PT; ++e) {
      const int at = tid + e * kDaThreads;
      tl[tile][at % kSlab][at / kSlab] = x[e];
    }
  };
  // acc[a][b] += sum_d A[d][ty * 4 + a] * B[d][tx * 4 + b], two b at a time
  struct Acc {
    float2 x[4][2];
    __device__ __forceinline__ Acc() {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i][0] = x[i][1] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ float at(int i, int j) const {
      return j & 1 ? x[i][j / 2].y : x[i][j / 2].x;
    }
  };
  auto mac = [&](Acc& acc, int A, int B) {
#pragma unroll
    for (int d = 0; d < kSlab; ++d) {
      const float4 a4 = *reinterpret_cast<const float4*>(&tl[A][d][ty * 4]);
      const float4 b4 = *reinterpret_cast<const float4*>(&tl[B][d][tx * 4]);
      const float a[4] = {a4.x, a4.y, a4.z, a4.w};
      const float2 b0 = make_float2(b4.x, b4.y), b1 = make_float2(b4.z, b4.w);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 aa = make_float2(a[i], a[i]);
        acc.x[i][0] = fma2(aa, b0, acc.x[i][0]);
        acc.x[i][1] = fma2(aa, b1, acc.x[i][1]);
      }
    }
  };
  Acc s1, s2;
  {
    const int D = max(p.DK, p.DV);
    auto fetch = [&](int d0) {
      get_rows(r[0], q, p.DK, d0);
      get_rows(r[1], k, p.DK, d0);
      get_rows(r[2], dO, p.DV, d0);
      get_rows(r[3], v, p.DV, d0);
    };
    fetch(0);
    for (int d0 = 0; d0 < D; d0 += kSlab) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 4; ++e) put_rows(e, r[e]);
      __syncthreads();
      if (d0 + kSlab < D) fetch(d0 + kSlab);
      if (d0 < p.DK) mac(s1, 0, 1);
      if (d0 < p.DV) mac(s2, 2, 3);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) W[ty * 4 + i][tx * 4 + j] = s1.at(i, j) * s2.at(i, j);

  // x and y: rows of [q S] . do and [k G] . v, C columns of the products at a time
  const size_t st = ((size_t)blockIdx.x * p.H + h) * p.DK * p.DV;
  const float* St = p.St + st;
  const float* G = p.G + st;
  float z = 0.f;
  {
    // S^T rows run over d_k, G rows over d_v: read along the rows
    auto fetch = [&](int j0, int d0) {
      get_rows(r[0], q, p.DK, d0);
      get_rows(r[1], k, p.DK, d0);
#pragma unroll
      for (int e = 0; e < PT; ++e) {
        const int at = tid + e * kDaThreads;
        const int js = j0 + at / kSlab, ds = d0 + at % kSlab;
        const int jg = j0 + at % C, dg = d0 + at / C;
        r[2][e] = js < p.DV ? St[(size_t)js * p.DK + ds] : 0.f;
        r[3][e] = jg < p.DV ? G[(size_t)dg * p.DV + jg] : 0.f;
      }
    };
    fetch(0, 0);
    for (int j0 = 0; j0 < p.DV; j0 += C) {
      Acc s, g;
      for (int d0 = 0; d0 < p.DK; d0 += kSlab) {
        __syncthreads();
        put_rows(0, r[0]);
        put_rows(1, r[1]);
        put_rows(2, r[2]);
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          const int at = tid + e * kDaThreads;
          tl[3][at / C][at % C] = r[3][e];
        }
        __syncthreads();
        if (d0 + kSlab < p.DK)
          fetch(j0, d0 + kSlab);
        else if (j0 + C < p.DV)
          fetch(j0 + C, 0);
        mac(s, 0, 2);
        mac(g, 1, 3);
#pragma unroll
        for (int e = 0; e < PT; ++e) {
          const int at = tid + e * kDaThreads;
          z = fmaf(tl[2][at / C][at % C], tl[3][at / C][at % C], z);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = ty * 4 + i;
        float x = 0.f, y = 0.f;
        if (row < L) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int jj = j0 + tx * 4 + j;
            if (jj < p.DV) {
              const size_t at = ((size_t)(t0 + row) * p.H + h) * p.DV + jj;
              x = fmaf(s.at(i, j), Elem<Tin>::to_f32(dO[at]), x);
              y = fmaf(g.at(i, j), Elem<Tin>::to_f32(v[at]), y);
            }
          }
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) {
          x += __shfl_xor_sync(0xffffffffu, x, o);
          y += __shfl_xor_sync(0xffffffffu, y, o);
        }
        if (tx == 0) {  // one writer per row
          sx[row] += x;
          sy[row] += y;
        }
      }
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  if (tid % 32 == 0) zs[tid / 32] = z;
  __syncthreads();

  if (tid < C) {
    // E[t][j] = D(t - 1, j), then times U_t[j]
    const int j = tid;
    float d = 1.f;
    for (int t = j + 1; t < L; ++t) {
      E[t][j] = d;
      d *= sa[t];
    }
    float u = 0.f;
    for (int t = L - 1; t > j; --t) {
      u = fmaf(t + 1 < L ? sa[t + 1] : 0.f, u, W[t][j]);
      E[t][j] *= u;
    }
  } else if (tid == C) {
    float d = 1.f;
    for (int t = 0; t < L; ++t) {
      head[t] = d;
      d *= sa[t];
    }
    float x = 0.f;
    for (int t = L - 1; t >= 0; --t) {
      x = fmaf(t + 1 < L ? sa[t + 1] : 0.f, x, sx[t]);
      sx[t] = x;
    }
  } else if (tid == C + 32) {
    float d = 1.f;
    for (int t = L - 1; t >= 0; --t) {
      tail[t] = d;
      d *= sa[t];
    }
    float y = 0.f;
    for (int t = 0; t < L; ++t) {
      const float own = sy[t];
      sy[t] = y;
      y = fmaf(sa[t], y, own);
    }
  }
  __syncthreads();
  if (tid < L) {
    const int t = tid;
    float zz = 0.f;
#pragma unroll
    for (int w = 0; w < kDaThreads / 32; ++w) zz += zs[w];
    float s = 0.f;
    for (int j = 0; j < t; ++j) s += E[t][j];
    s = fmaf(head[t], sx[t], s);
    s = fmaf(tail[t], sy[t], s);
    s = fmaf(head[t] * tail[t], zz, s);
    p.da[(size_t)(t0 + t) * p.H + h] = s;
  }
}

// da[h] = the sum over the tokens of per-token gradients [tokens, H]: one CTA
// per head, a fixed order, sums in 64 bits.  A thread has eight loads on their
// way at a time: a head's sum is a chain of latencies, not of bytes.
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads) la_dalpha_sum_kernel(const float* __restrict__ part,
                                                                    float* __restrict__ da,
                                                                    int64_t tokens, int H) {
  __shared__ double red[kSumThreads];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t t = threadIdx.x; t < tokens; t += 8 * kSumThreads) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t at = t + e * kSumThreads;
      x[e] = at < tokens ? __ldg(part + at * H + h) : 0.f;
    }
    s += (((double)x[0] + (double)x[1]) + ((double)x[2] + (double)x[3])) +
         (((double)x[4] + (double)x[5]) + ((double)x[6] + (double)x[7]));
  }
  red[threadIdx.x] = s;
  __syncthreads();
#pragma unroll
  for (int w = kSumThreads / 2; w >= 1; w >>= 1) {
    if (threadIdx.x < w) red[threadIdx.x] += red[threadIdx.x + w];
    __syncthreads();
  }
  if (threadIdx.x == 0) da[h] = (float)red[0];
}

}  // namespace la

size_t la_fwd_simt_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen) {
  return 4 * la::part_floats(dk, dv, n_seqs, H, la::rec_segments(1, n_seqs, T, H, dv, varlen));
}

cudaError_t launch_la_fwd_simt(int dtype, int out_dtype, int dk, int dv, const void* q,
                               const void* k, const void* v, const float* alpha, int per_head,
                               const float* S0, const int32_t* cu, void* out, float* S_final,
                               void* ws, int n_seqs, int T, int H, int* status,
                               cudaStream_t stream) {
  la::RecArgs a{q,   k,       v,  {alpha, H, per_head}, S0, S_final, dv, 1,
                out, nullptr, cu, n_seqs, T, H, dv, status};
  la::set_parts(&a, dk, la::rec_segments(1, n_seqs, T, H, dv, cu != nullptr),
                static_cast<float*>(ws));
  return la::rec(dtype, out_dtype, dk, a, false, stream);
}

cudaError_t launch_la_dalpha_sum(const float* part, float* da, int64_t tokens, int H,
                                 cudaStream_t stream) {
  la::la_dalpha_sum_kernel<<<H, la::kSumThreads, 0, stream>>>(part, da, tokens, H);
  return cudaGetLastError();
}

namespace la {

// Segments of the three recurrences (dq, dv, dk), which run together, each
// with states of its own, when d_k = d_v, and one after another otherwise.
static void bwd_segments(int dk, int dv, int n_seqs, int T, int H, bool varlen, int* g) {
  const int together = dk == dv ? 3 : 1;
  g[0] = g[2] = rec_segments(together, n_seqs, T, H, dk, varlen);
  g[1] = rec_segments(together, n_seqs, T, H, dv, varlen);
}

}  // namespace la

// S^T and G at the chunks' bounds, then (decay per head) its gradient per
// token, then the segments' states.
size_t la_bwd_simt_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen,
                                   bool per_head) {
  const size_t slots = (size_t)la::chunk_slots(varlen, n_seqs, T, la::kChunk);
  const size_t tokens = varlen ? (size_t)T : (size_t)n_seqs * T;
  int g[3];
  la::bwd_segments(dk, dv, n_seqs, T, H, varlen, g);
  const size_t a = la::part_floats(dk, dv, n_seqs, H, g[0]);
  const size_t b = la::part_floats(dk, dv, n_seqs, H, g[1]);
  return 2 * slots * H * dk * dv * 4 + (per_head ? (tokens * H * 4 + 255) / 256 * 256 : 0) +
         4 * (dk == dv ? 3 * a : (a > b ? a : b));
}

cudaError_t launch_la_bwd_simt(int dtype, int dk_, int dv_, const void* q, const void* k,
                               const void* v, const float* alpha, int per_head, const float* S0,
                               const int32_t* cu, const void* dO, const float* dSf, void* dq,
                               void* dk, void* dv, float* dalpha, float* dS0, void* ws, int n_seqs,
                               int T, int H, int* status, cudaStream_t stream) {
  const bool varlen = cu != nullptr;
  const size_t slots = (size_t)la::chunk_slots(varlen, n_seqs, T, la::kChunk);
  const int64_t tokens = varlen ? (int64_t)T : (int64_t)n_seqs * T;
  float* St = static_cast<float*>(ws);
  float* G = St + slots * H * dk_ * dv_;
  float* part = per_head ? G + slots * H * dk_ * dv_ : dalpha;
  const la::Decay al{alpha, H, per_head};
  // (state, stride of its first index, stride of its second): S^T, G, G^T
  la::RecArgs aq{dO, v, k, al, S0, nullptr, 1, dv_, dq, St, cu, n_seqs, T, H, dk_, status};
  la::RecArgs av{k, q, dO, al, dSf, dS0, dv_, 1, dv, G, cu, n_seqs, T, H, dv_, status};
  la::RecArgs ak{v, dO, q, al, dSf, nullptr, 1, dv_, dk, nullptr, cu, n_seqs, T, H, dk_, status};
  int g[3];
  la::bwd_segments(dk_, dv_, n_seqs, T, H, varlen, g);
  float* ps = G + slots * H * dk_ * dv_ + (per_head ? ((size_t)tokens * H + 63) / 64 * 64 : 0);
  const size_t one = dk_ == dv_ ? la::part_floats(dk_, dv_, n_seqs, H, g[0]) : 0;
  la::set_parts(&aq, dv_, g[0], ps);
  la::set_parts(&av, dk_, g[1], ps + one);
  la::set_parts(&ak, dv_, g[2], ps + 2 * one);
  cudaError_t e;
  if (dk_ == dv_) {
    const la::Rec3Args a{aq, {av, ak}};
    e = dtype == CKDA_BF16 ? la::rec3<__nv_bfloat16>(dk_, a, stream)
                           : la::rec3<float>(dk_, a, stream);
  } else {
    e = la::rec(dtype, dtype, dv_, aq, false, stream);
    if (e == cudaSuccess) e = la::rec(dtype, dtype, dk_, av, true, stream);
    if (e == cudaSuccess) e = la::rec(dtype, dtype, dv_, ak, true, stream);
  }
  if (e != cudaSuccess) return e;
  if (slots > 0) {
    const la::DalphaArgs d{q, k, v, dO, al, St, G, part, cu, n_seqs, T, H, dk_, dv_, status};
    const dim3 grid((unsigned)slots, H);
    if (dtype == CKDA_BF16)
      la::la_dalpha_kernel<__nv_bfloat16><<<grid, la::kDaThreads, 0, stream>>>(d);
    else
      la::la_dalpha_kernel<float><<<grid, la::kDaThreads, 0, stream>>>(d);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  return per_head ? launch_la_dalpha_sum(part, dalpha, tokens, H, stream) : cudaSuccess;
}

}  // namespace ckda
