// Host side of the head-decay linear attention and of the query / key norm:
// argument validation and dispatch.  Every check happens before any CUDA
// call, so an argument error launches nothing and touches no memory.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ckda.h"
#include "qk_norm.cuh"

namespace ckda {
int* status_word();
cudaError_t launch_la_fwd_simt(int dtype, int out_dtype, int dk, int dv, const void* q,
                               const void* k, const void* v, const float* alpha, int per_head,
                               const float* S0, const int32_t* cu, void* out, float* S_final,
                               void* ws, int n_seqs, int T, int H, int* status,
                               cudaStream_t stream);
size_t la_fwd_simt_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen);
bool la_fwd_tc_supported(int dtype, int dk, int dv, int n_seqs, int T, int H, bool varlen);
size_t la_fwd_tc_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen);
cudaError_t launch_la_fwd_tc(int out_dtype, int dk, int dv, const void* q, const void* k,
                             const void* v, const float* alpha, int per_head, const float* S0,
                             const int32_t* cu, void* out, float* S_final, void* ws, int n_seqs,
                             int T, int H, int* status, cudaStream_t stream);
cudaError_t launch_la_decode(int dtype, int out_dtype, int dk, int dv, const void* q, const void* k,
                             const void* v, const float* alpha, int per_head, float* S, void* out,
                             int B, int H, cudaStream_t stream);
cudaError_t launch_la_dalpha_sum(const float* part, float* da, int64_t tokens, int H,
                                 cudaStream_t stream);
size_t la_bwd_simt_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen,
                                   bool per_head);
cudaError_t launch_la_bwd_simt(int dtype, int dk_, int dv_, const void* q, const void* k,
                               const void* v, const float* alpha, int per_head, const float* S0,
                               const int32_t* cu, const void* dO, const float* dSf, void* dq,
                               void* dk, void* dv, float* dalpha, float* dS0, void* ws, int n_seqs,
                               int T, int H, int* status, cudaStream_t stream);
bool la_bwd_tc_supported(int dtype, int dk, int dv, int n_seqs, int T, int H, bool varlen);
size_t la_bwd_tc_workspace_bytes(int dk, int dv, int n_seqs, int T, int H, bool varlen,
                                 bool per_head);
cudaError_t launch_la_bwd_tc(int dk_, int dv_, const void* q, const void* k, const void* v,
                             const float* alpha, int per_head, const float* S0, const int32_t* cu,
                             const void* dO, const float* dSf, void* dq, void* dk, void* dv,
                             float* dalpha, float* dS0, void* ws, int n_seqs, int T, int H,
                             int* status, cudaStream_t stream);
cudaError_t launch_qk_norm_fwd(const qkn::Args& p, int dtype, int out_dtype, cudaStream_t st);
cudaError_t launch_qk_norm_bwd(const qkn::Args& p, int dtype, float* dwq, float* dwk,
                               cudaStream_t st);
size_t qk_norm_bwd_workspace_bytes(int d);
}  // namespace ckda

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }
bool known_dtype(int t) { return t == CKDA_F32 || t == CKDA_BF16; }

// Sizes of a head-decay linear attention call.  The grids count (sequence,
// head, column slice) triples, slices of 16 columns at the least, in 31 bits.
int la_sizes(int B, int T, int H, int d_k, int d_v, int per_head, int dtype, bool varlen) {
  if (B < 0 || T < 0 || H <= 0 || (per_head != 0 && per_head != 1)) return CKDA_ERR_INVALID_ARG;
  if (!known_dtype(dtype)) return CKDA_ERR_UNSUPPORTED;
  if (!supported_d(d_k) || !supported_d(d_v)) return CKDA_ERR_UNSUPPORTED;
  if (varlen && B == 0 && T != 0) return CKDA_ERR_INVALID_ARG;
  if (!varlen && (int64_t)B * T * H > (int64_t)INT32_MAX) return CKDA_ERR_UNSUPPORTED;
  if (H > 65535 || (int64_t)B * H * 8 > (int64_t)INT32_MAX) return CKDA_ERR_UNSUPPORTED;
  return CKDA_OK;
}

struct Span {
  const void* p;
  size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.bytes == 0 || b.bytes == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// A workspace of `need` bytes that touches none of the tensors.
int check_workspace(const void* ws, size_t bytes, size_t need, const Span* t, int nt) {
  if (need == 0) return CKDA_OK;
  if (ws == nullptr || bytes < need || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0)
    return CKDA_ERR_WORKSPACE;
  for (int i = 0; i < nt; ++i)
    if (overlap({ws, need}, t[i])) return CKDA_ERR_WORKSPACE;
  return CKDA_OK;
}

int qk_sizes(int64_t tokens, int Hq, int Hk, int d, int rot, int norm, float eps, int interleaved,
             int64_t q_stride, int64_t k_stride, int dtype) {
  if (tokens < 0 || Hq < 0 || Hk < 0 || Hq + (int64_t)Hk < 1) return CKDA_ERR_INVALID_ARG;
  if (norm != CKDA_NORM_L2 && norm != CKDA_NORM_RMS) return CKDA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return CKDA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || isinf(eps)) return CKDA_ERR_INVALID_ARG;
  if (!known_dtype(dtype) || !supported_d(d)) return CKDA_ERR_UNSUPPORTED;
  if (rot < 0 || rot > d) return CKDA_ERR_INVALID_ARG;
  if (rot % 8 != 0) return CKDA_ERR_UNSUPPORTED;
  if (q_stride < (int64_t)Hq * d || k_stride < (int64_t)Hk * d) return CKDA_ERR_INVALID_ARG;
  const int per16 = dtype == CKDA_BF16 ? 8 : 4;
  if (q_stride % per16 != 0 || k_stride % per16 != 0) return CKDA_ERR_MISALIGNED;
  if (tokens > (int64_t)INT32_MAX || (int64_t)Hq + Hk > 65535) return CKDA_ERR_UNSUPPORTED;
  // (the rows' extent in bytes stays in 63 bits)
  const int64_t most = (INT64_MAX >> 4) / (tokens > 0 ? tokens : 1);
  if (q_stride > most || k_stride > most) return CKDA_ERR_INVALID_ARG;
  return CKDA_OK;
}

}  // namespace

extern "C" {

int64_t ckda_la_fwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int dtype, int varlen) {
  const int rc = la_sizes(B, T, H, d_k, d_v, 0, dtype, varlen != 0);
  if (rc != CKDA_OK) return rc;
  if (B == 0) return 0;
  const bool vl = varlen != 0;
  return (int64_t)(ckda::la_fwd_tc_supported(dtype, d_k, d_v, B, T, H, vl)
                       ? ckda::la_fwd_tc_workspace_bytes(d_k, d_v, B, T, H, vl)
                       : ckda::la_fwd_simt_workspace_bytes(d_k, d_v, B, T, H, vl));
}

int ckda_la_fwd_chunked(const void* q, const void* k, const void* v, const float* alpha,
                        const float* S0, const int32_t* cu_seqlens, void* out, float* S_final,
                        int B, int T, int H, int d_k, int d_v, int alpha_per_head, int dtype,
                        int out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  int rc = la_sizes(B, T, H, d_k, d_v, alpha_per_head, dtype, varlen);
  if (rc != CKDA_OK) return rc;
  if (!known_dtype(out_dtype)) return CKDA_ERR_UNSUPPORTED;
  const int64_t tokens = varlen ? (int64_t)T : (int64_t)B * T;
  if (tokens > 0 && (!q || !k || !v || !alpha || !out)) return CKDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, alpha, S0, out, S_final};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return CKDA_ERR_MISALIGNED;
  if (B == 0) return CKDA_OK;
  const size_t e = dtype == CKDA_BF16 ? 2 : 4, eo = out_dtype == CKDA_BF16 ? 2 : 4;
  const size_t th = (size_t)tokens * H, st = (size_t)B * H * d_k * d_v * 4;
  const Span tens[] = {{q, th * d_k * e},
                       {k, th * d_k * e},
                       {v, th * d_v * e},
                       {alpha, (alpha_per_head ? (size_t)H : th) * 4},
                       {S0, st},
                       {cu_seqlens, (size_t)(B + 1) * 4},
                       {out, th * d_v * eo},
                       {S_final, st}};
  // out touches nothing else; S_final only S0, and then all of it
  for (int i = 0; i < 8; ++i) {
    if (i != 6 && overlap(tens[6], tens[i])) return CKDA_ERR_INVALID_ARG;
    if (i != 6 && i != 7 && !(i == 4 && S0 == S_final) && overlap(tens[7], tens[i]))
      return CKDA_ERR_INVALID_ARG;
  }
  const size_t need = (size_t)ckda_la_fwd_workspace_bytes(B, T, H, d_k, d_v, dtype, varlen);
  rc = check_workspace(workspace, workspace_bytes, need, tens, 8);
  if (rc != CKDA_OK) return rc;
  int* status = ckda::status_word();
  if (status == nullptr) return CKDA_ERR_CUDA;
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  const cudaError_t err =
      ckda::la_fwd_tc_supported(dtype, d_k, d_v, B, T, H, varlen)
          ? ckda::launch_la_fwd_tc(out_dtype, d_k, d_v, q, k, v, alpha, alpha_per_head, S0,
                                   cu_seqlens, out, S_final, workspace, B, T, H, status, st_)
          : ckda::launch_la_fwd_simt(dtype, out_dtype, d_k, d_v, q, k, v, alpha, alpha_per_head, S0,
                                     cu_seqlens, out, S_final, workspace, B, T, H, status, st_);
  return err == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

int64_t ckda_la_bwd_workspace_bytes(int B, int T, int H, int d_k, int d_v, int alpha_per_head,
                                    int dtype, int varlen) {
  const int rc = la_sizes(B, T, H, d_k, d_v, alpha_per_head, dtype, varlen != 0);
  if (rc != CKDA_OK) return rc;
  if (B == 0) return 0;
  const bool vl = varlen != 0, ph = alpha_per_head != 0;
  return (int64_t)(ckda::la_bwd_tc_supported(dtype, d_k, d_v, B, T, H, vl)
                       ? ckda::la_bwd_tc_workspace_bytes(d_k, d_v, B, T, H, vl, ph)
                       : ckda::la_bwd_simt_workspace_bytes(d_k, d_v, B, T, H, vl, ph));
}

int ckda_la_bwd_chunked(const void* q, const void* k, const void* v, const float* alpha,
                        const float* S0, const int32_t* cu_seqlens, const void* dO,
                        const float* dS_final, void* dq, void* dk, void* dv, float* dalpha,
                        float* dS0, int B, int T, int H, int d_k, int d_v, int alpha_per_head,
                        int dtype, void* workspace, size_t workspace_bytes, void* stream) {
  const bool varlen = cu_seqlens != nullptr;
  int rc = la_sizes(B, T, H, d_k, d_v, alpha_per_head, dtype, varlen);
  if (rc != CKDA_OK) return rc;
  const int64_t tokens = varlen ? (int64_t)T : (int64_t)B * T;
  if (tokens > 0 && (!q || !k || !v || !alpha || !dO || !dq || !dk || !dv || !dalpha))
    return CKDA_ERR_INVALID_ARG;
  if (alpha_per_head && !dalpha) return CKDA_ERR_INVALID_ARG;  // [H], whatever B and T
  const void* ptrs[] = {q, k, v, alpha, S0, dO, dS_final, dq, dk, dv, dalpha, dS0};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return CKDA_ERR_MISALIGNED;
  const cudaStream_t st_ = static_cast<cudaStream_t>(stream);
  if (B == 0) {  // a gradient of [H] is zero without a sequence too
    if (!alpha_per_head) return CKDA_OK;
    return ckda::launch_la_dalpha_sum(nullptr, dalpha, 0, H, st_) == cudaSuccess ? CKDA_OK
                                                                                 : CKDA_ERR_CUDA;
  }
  const size_t e = dtype == CKDA_BF16 ? 2 : 4;
  const size_t th = (size_t)tokens * H, st = (size_t)B * H * d_k * d_v * 4;
  const size_t al = (alpha_per_head ? (size_t)H : th) * 4;
  const Span tens[] = {{q, th * d_k * e},  {k, th * d_k * e},  {v, th * d_v * e}, {alpha, al},
                       {S0, st},           {dO, th * d_v * e}, {dS_final, st},
                       {cu_seqlens, (size_t)(B + 1) * 4},
                       {dq, th * d_k * e}, {dk, th * d_k * e}, {dv, th * d_v * e}, {dalpha, al},
                       {dS0, st}};
  // no output touches an input or another output
  for (int i = 8; i < 13; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(tens[i], tens[j])) return CKDA_ERR_INVALID_ARG;
  const size_t need = (size_t)ckda_la_bwd_workspace_bytes(B, T, H, d_k, d_v, alpha_per_head, dtype,
                                                          varlen);
  rc = check_workspace(workspace, workspace_bytes, need, tens, 13);
  if (rc != CKDA_OK) return rc;
  int* status = ckda::status_word();
  if (status == nullptr) return CKDA_ERR_CUDA;
  const cudaError_t err =
      ckda::la_bwd_tc_supported(dtype, d_k, d_v, B, T, H, varlen)
          ? ckda::launch_la_bwd_tc(d_k, d_v, q, k, v, alpha, alpha_per_head, S0, cu_seqlens, dO,
                                   dS_final, dq, dk, dv, dalpha, dS0, workspace, B, T, H, status,
                                   st_)
          : ckda::launch_la_bwd_simt(dtype, d_k, d_v, q, k, v, alpha, alpha_per_head, S0,
                                     cu_seqlens, dO, dS_final, dq, dk, dv, dalpha, dS0, workspace,
                                     B, T, H, status, st_);
  return err == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

int ckda_la_decode_step(const void* q, const void* k, const void* v, const float* alpha,
                        float* S_inout, void* out, int B, int H, int d_k, int d_v,
                        int alpha_per_head, int dtype, int out_dtype, void* stream) {
  int rc = la_sizes(B, 1, H, d_k, d_v, alpha_per_head, dtype, false);
  if (rc != CKDA_OK) return rc;
  if (!known_dtype(out_dtype)) return CKDA_ERR_UNSUPPORTED;
  if (B == 0) return CKDA_OK;
  if (!q || !k || !v || !alpha || !S_inout || !out) return CKDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, v, alpha, S_inout, out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
  const size_t e = dtype == CKDA_BF16 ? 2 : 4, bh = (size_t)B * H;
  const Span tens[] = {{q, bh * d_k * e},
                       {k, bh * d_k * e},
                       {v, bh * d_v * e},
                       {alpha, (alpha_per_head ? (size_t)H : bh) * 4},
                       {S_inout, bh * d_k * d_v * 4},
                       {out, bh * d_v * (out_dtype == CKDA_BF16 ? 2u : 4u)}};
  for (int i = 0; i < 4; ++i)
    if (overlap(tens[4], tens[i]) || overlap(tens[5], tens[i])) return CKDA_ERR_INVALID_ARG;
  if (overlap(tens[4], tens[5])) return CKDA_ERR_INVALID_ARG;
  const cudaError_t err =
      ckda::launch_la_decode(dtype, out_dtype, d_k, d_v, q, k, v, alpha, alpha_per_head, S_inout,
                             out, B, H, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

int ckda_qk_norm_rope(const void* q, const void* k, const float* wq, const float* wk,
                      const int32_t* positions, const float* inv_freq, void* q_out, void* k_out,
                      int64_t tokens, int Hq, int Hk, int d, int rot, int interleaved, int norm,
                      float eps, int64_t q_stride, int64_t k_stride, int dtype, int out_dtype,
                      void* stream) {
  int rc = qk_sizes(tokens, Hq, Hk, d, rot, norm, eps, interleaved, q_stride, k_stride, dtype);
  if (rc != CKDA_OK) return rc;
  if (!known_dtype(out_dtype)) return CKDA_ERR_UNSUPPORTED;
  if (tokens == 0) return CKDA_OK;
  if ((Hq > 0 && (!q || !q_out)) || (Hk > 0 && (!k || !k_out))) return CKDA_ERR_INVALID_ARG;
  if (rot > 0 && (!positions || !inv_freq)) return CKDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, q_out, k_out};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
  const void* words[] = {wq, wk, positions, inv_freq};
  for (const void* p : words)
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return CKDA_ERR_MISALIGNED;
  const size_t e = dtype == CKDA_BF16 ? 2 : 4, eo = out_dtype == CKDA_BF16 ? 2 : 4;
  // the outputs touch no input, but for a contiguous one that is replaced
  const Span in[] = {{Hq ? q : nullptr, ((tokens - 1) * q_stride + (size_t)Hq * d) * e},
                     {Hk ? k : nullptr, ((tokens - 1) * k_stride + (size_t)Hk * d) * e},
                     {wq, (size_t)d * 4},
                     {wk, (size_t)d * 4},
                     {positions, (size_t)tokens * 4},
                     {inv_freq, (size_t)rot * 2}};
  const Span out[] = {{Hq ? q_out : nullptr, (size_t)tokens * Hq * d * eo},
                      {Hk ? k_out : nullptr, (size_t)tokens * Hk * d * eo}};
  const bool in_place[] = {q_out == q && q_stride == (int64_t)Hq * d && e == eo,
                           k_out == k && k_stride == (int64_t)Hk * d && e == eo};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 6; ++j)
      if (!(i == j && in_place[i]) && overlap(out[i], in[j])) return CKDA_ERR_INVALID_ARG;
  if (overlap(out[0], out[1])) return CKDA_ERR_INVALID_ARG;
  const ckda::qkn::Args p{{{q, wq, q_out, nullptr, q_stride, Hq, 0, 0, 0},
                           {k, wk, k_out, nullptr, k_stride, Hk, 0, 0, 0}},
                          positions, inv_freq, nullptr, tokens, d, rot, interleaved,
                          norm == CKDA_NORM_RMS ? 1.f / (float)d : 1.f, eps};
  const cudaError_t err =
      ckda::launch_qk_norm_fwd(p, dtype, out_dtype, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

int64_t ckda_qk_norm_rope_bwd_workspace_bytes(int d) {
  if (!supported_d(d)) return CKDA_ERR_UNSUPPORTED;
  return (int64_t)ckda::qk_norm_bwd_workspace_bytes(d);
}

int ckda_qk_norm_rope_bwd(const void* q, const void* k, const float* wq, const float* wk,
                          const int32_t* positions, const float* inv_freq, const void* dq_out,
                          const void* dk_out, void* dq, void* dk, float* dwq, float* dwk,
                          int64_t tokens, int Hq, int Hk, int d, int rot, int interleaved, int norm,
                          float eps, int64_t q_stride, int64_t k_stride, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  int rc = qk_sizes(tokens, Hq, Hk, d, rot, norm, eps, interleaved, q_stride, k_stride, dtype);
  if (rc != CKDA_OK) return rc;
  if (tokens > 0 && ((Hq > 0 && (!q || !dq_out || !dq)) || (Hk > 0 && (!k || !dk_out || !dk))))
    return CKDA_ERR_INVALID_ARG;
  if (tokens > 0 && rot > 0 && (!positions || !inv_freq)) return CKDA_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, dq_out, dk_out, dq, dk};
  for (const void* p : ptrs)
    if (!aligned16(p)) return CKDA_ERR_MISALIGNED;
  const void* words[] = {wq, wk, positions, inv_freq, dwq, dwk};
  for (const void* p : words)
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return CKDA_ERR_MISALIGNED;
  const size_t e = dtype == CKDA_BF16 ? 2 : 4;
  const size_t nq = (size_t)tokens * Hq * d * e, nk = (size_t)tokens * Hk * d * e;
  const size_t last = tokens > 0 ? (size_t)(tokens - 1) : 0;
  const Span tens[] = {{nq ? q : nullptr, (last * q_stride + (size_t)Hq * d) * e},
                       {nk ? k : nullptr, (last * k_stride + (size_t)Hk * d) * e},
                       {wq, (size_t)d * 4},
                       {wk, (size_t)d * 4},
                       {positions, (size_t)tokens * 4},
                       {inv_freq, (size_t)rot * 2},
                       {dq_out, nq},
                       {dk_out, nk},
                       {dq, nq},
                       {dk, nk},
                       {dwq, (size_t)d * 4},
                       {dwk, (size_t)d * 4}};
  for (int i = 8; i < 12; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(tens[i], tens[j])) return CKDA_ERR_INVALID_ARG;
  const bool sums = dwq != nullptr || dwk != nullptr;
  rc = check_workspace(workspace, workspace_bytes,
                       sums ? ckda::qk_norm_bwd_workspace_bytes(d) : 0, tens, 12);
  if (rc != CKDA_OK) return rc;
  const ckda::qkn::Args p{{{q, wq, dq, dq_out, q_stride, Hq, 0, 0, 0},
                           {k, wk, dk, dk_out, k_stride, Hk, 0, 0, 0}},
                          positions, inv_freq, sums ? static_cast<float*>(workspace) : nullptr,
                          tokens, d, rot, interleaved,
                          norm == CKDA_NORM_RMS ? 1.f / (float)d : 1.f, eps};
  if (tokens == 0 && !sums) return CKDA_OK;
  const cudaError_t err =
      ckda::launch_qk_norm_bwd(p, dtype, dwq, dwk, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? CKDA_OK : CKDA_ERR_CUDA;
}

}  // extern "C"
