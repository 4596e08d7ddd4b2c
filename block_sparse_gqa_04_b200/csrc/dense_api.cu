// C ABI of the dense-attention operators: argument checks, workspace layout and
// launches.  Declarations and the contract of every entry point are in
// include/msa.h.
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/msa.h"
#include "dense_common.cuh"
#include "internal.h"

using msa::Dense;
using msa::SeqRec;
using msa::Tree;

namespace {

constexpr size_t kAlign = 256;
constexpr size_t kHeadBytes = msa::kHeadWords * sizeof(int32_t);
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxNodes = 128;
// Tokens of a sequence: the idle warps of the tensor-core kernels wait for a row of key
// tiles, 65536 of them about 0.1 s, and a bounded wait gives up after a second or so.
constexpr int kMaxTokens = 1 << 23;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename... P>
bool pointers_ok(const P*... p) {
  return ((p && aligned16(p)) && ...);
}

int tiles(long long n) { return int((n + msa::kDenseTile - 1) / msa::kDenseTile); }

// The checks that do not depend on the layout.
msa_status_t resolve_heads(const msa_problem_t* p, Dense* P) {
  if (!p || p->batch < 1 || p->num_kv_heads < 1 || p->num_q_heads < 1 ||
      p->num_q_heads % p->num_kv_heads != 0 || p->head_dim < 1)
    return MSA_ERR_INVALID_ARG;
  if (p->dtype != MSA_BF16 && p->dtype != MSA_F32) return MSA_ERR_INVALID_ARG;
  if (!(p->softmax_scale >= 0.0f) || isinf(p->softmax_scale)) return MSA_ERR_INVALID_ARG;
  if (p->num_pages < 0 || (p->num_pages > 0 && !p->block_table)) return MSA_ERR_INVALID_ARG;
  if (p->qk_dtype != 0) return MSA_ERR_UNSUPPORTED;
  if (p->head_dim != 64 && p->head_dim != 128) return MSA_ERR_UNSUPPORTED;
  if (p->num_q_heads > 65536) return MSA_ERR_UNSUPPORTED;
  *P = Dense{};
  P->B = p->batch;
  P->Hq = p->num_q_heads;
  P->Hkv = p->num_kv_heads;
  P->G = p->num_q_heads / p->num_kv_heads;
  P->D = p->head_dim;
  P->scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / sqrtf((float)p->head_dim);
  P->f32 = p->dtype == MSA_F32;
  P->pages = p->num_pages;
  P->table = p->num_pages > 0 ? p->block_table : nullptr;
  return MSA_OK;
}

// Rows and work items have to be addressable with 32 bits.
msa_status_t check_sizes(const Dense& P, long long qtiles, long long ktiles, long long pairs) {
  constexpr long long kMax = 1LL << 31;
  if (P.rows_pad >= kMax || P.rows_k >= kMax || qtiles * 2 * P.Hq >= kMax ||
      ktiles * 2 * P.Hq >= kMax || pairs >= kMax || P.rows_q * P.Hq >= kMax * 4 ||
      ktiles * P.Hkv * P.G >= kMax)
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

msa_status_t resolve_batched(const msa_problem_t* p, Dense* P) {
  msa_status_t st = resolve_heads(p, P);
  if (st != MSA_OK) return st;
  if (p->q_len < 0 || p->kv_len < 1 || p->q_pos0 < 0 ||
      p->q_pos0 > (int64_t)p->kv_len - p->q_len)
    return MSA_ERR_INVALID_ARG;
  if (p->kv_len > kMaxTokens) return MSA_ERR_UNSUPPORTED;
  P->Sq = p->q_len;
  P->Skv = p->kv_len;
  P->pos0 = int(p->q_pos0);
  P->table_w = tiles(p->kv_len);
  P->rows_q = (long long)P->B * P->Sq;
  P->rows_pad = (long long)P->B * ((P->Sq + 15LL) / 16 * 16);
  P->rows_k = P->table ? (long long)P->pages * msa::kDenseTile : (long long)P->B * P->Skv;
  const long long qt = (long long)P->B * tiles(P->Sq), kt = (long long)P->B * tiles(P->Skv);
  const long long pairs = (long long)P->B * P->Hkv * msa::dense_pairs(tiles(P->Sq), P->G);
  if ((st = check_sizes(*P, qt, kt, pairs)) != MSA_OK) return st;
  P->qtiles = int(qt);
  P->ktiles = int(kt);
  P->pairs = int(pairs);
  return MSA_OK;
}

// The records of a packed batch; recs (p->batch of them) may be null: sizes only.
msa_status_t resolve_packed(const msa_problem_t* p, const int32_t* cu_q, const int32_t* cu_k,
                            Dense* P, SeqRec* recs) {
  msa_status_t st = resolve_heads(p, P);
  if (st != MSA_OK) return st;
  if (p->batch > kMaxSeqs || !cu_q || !cu_k || cu_q[0] != 0 || cu_k[0] != 0)
    return MSA_ERR_INVALID_ARG;
  if (p->num_pages != 0) return MSA_ERR_UNSUPPORTED;
  long long qt = 0, kt = 0, pairs = 0, pad = 0;
  for (int b = 0; b < p->batch; ++b) {
    const long long nq = (long long)cu_q[b + 1] - cu_q[b], nk = (long long)cu_k[b + 1] - cu_k[b];
    if (nq < 0 || nk < 0 || nq > nk) return MSA_ERR_INVALID_ARG;
    if (nk > kMaxTokens) return MSA_ERR_UNSUPPORTED;
    pad += (nq + 15) / 16 * 16;
    qt += tiles(nq);
    kt += tiles(nk);
    pairs += (long long)P->Hkv * msa::dense_pairs(tiles(nq), P->G);
    if (recs) recs[b] = SeqRec{cu_q[b], cu_k[b], int(nq), int(nk), int(nk - nq), 0, 0, 0, 0};
  }
  P->rows_q = cu_q[p->batch];
  P->rows_pad = pad;
  P->rows_k = cu_k[p->batch];
  if ((st = check_sizes(*P, qt, kt, pairs)) != MSA_OK) return st;
  P->qtiles = int(qt);
  P->ktiles = int(kt);
  P->pairs = int(pairs);
  if (recs) {
    std::sort(recs, recs + p->batch, [](const SeqRec& a, const SeqRec& b) {
      return a.nk != b.nk ? a.nk > b.nk : a.k0 != b.k0 ? a.k0 < b.k0 : a.q0 < b.q0;
    });
    SeqRec at{};
    for (int b = 0; b < p->batch; ++b) {
      SeqRec& r = recs[b];
      r.qt0 = at.qt0;
      r.kt0 = at.kt0;
      r.pr0 = at.pr0;
      r.qp0 = at.qp0;
      at.qp0 += msa::pad16(r.nq);
      at.qt0 += tiles(r.nq);
      at.kt0 += tiles(r.nk);
      at.pr0 += P->Hkv * msa::dense_pairs(tiles(r.nq), P->G);
    }
  }
  return MSA_OK;
}

msa_status_t resolve_dense(const msa_problem_t* p, const int32_t* cu_q, const int32_t* cu_k,
                           Dense* P, SeqRec* recs) {
  if (cu_q || cu_k) return resolve_packed(p, cu_q, cu_k, P, recs);
  return resolve_batched(p, P);
}

struct DenseLayout {
  size_t status, recs, nl, delta, room, part, total;
};

DenseLayout dense_layout(const Dense& P, bool packed, bool backward) {
  DenseLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  L.status = take(kHeadBytes);
  if (packed) L.recs = take(size_t(P.B) * sizeof(SeqRec));
  if (backward) {
    const size_t rows = P.f32 ? size_t(P.rows_q) * P.Hq
                              : size_t(P.rows_pad) * P.Hq + msa::kDenseTile;
    const int splits = msa::dense_bwd_splits(P);
    if (!P.f32) L.nl = take(rows * sizeof(float));
    L.delta = take(rows * sizeof(float));
    if (!P.f32) L.room = take(rows * sizeof(float));
    if (splits > 1) L.part = take(size_t(splits) * 2 * P.rows_k * P.Hkv * P.D * sizeof(float));
  }
  L.total = off;
  return L;
}

template <typename T>
T* at(void* ws, size_t off) { return reinterpret_cast<T*>(static_cast<char*>(ws) + off); }

msa_status_t check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) % kAlign) != 0) return MSA_ERR_INVALID_ARG;
  return have < need ? MSA_ERR_WORKSPACE : MSA_OK;
}

// A packed batch's records on the host for the length of a call.
struct Records {
  SeqRec* r = nullptr;
  bool make(const msa_problem_t* p, const int32_t* cu_q, const int32_t* cu_k) {
    if (!(cu_q || cu_k) || !p || p->batch < 1 || p->batch > kMaxSeqs) return true;
    r = new (std::nothrow) SeqRec[p->batch];
    return r != nullptr;
  }
  ~Records() { delete[] r; }
};

// A call without rows: it reports no error, whatever the workspace held.
msa_status_t nothing_to_do(void* ws, size_t have, cudaStream_t s) {
  if (check_ws(ws, have, sizeof(int32_t)) != MSA_OK) return MSA_OK;
  return msa::status_of(cudaMemsetAsync(ws, 0, sizeof(int32_t), s));
}

// Clears the head of the workspace and puts the records in place.
msa_status_t begin(Dense* P, const Records& R, const DenseLayout& L, void* ws, cudaStream_t s) {
  int32_t* head = at<int32_t>(ws, L.status);
  if (R.r) P->seqs = at<SeqRec>(ws, L.recs);
  cudaError_t e = msa::launch_dense_begin(head, R.r, R.r ? at<SeqRec>(ws, L.recs) : nullptr,
                                          R.r ? P->B : 0, s);
  if (e == cudaSuccess) e = msa::launch_dense_check_table(*P, head, s);
  return msa::status_of(e);
}

// Tree problems: the cache is a batched problem with kv_len rows per sequence.
msa_status_t resolve_tree(const msa_problem_t* p, Tree* T) {
  if (!p) return MSA_ERR_INVALID_ARG;
  msa_problem_t c = *p;
  c.q_pos0 = 0;
  msa_status_t st = resolve_batched(&c, &T->d);
  if (st != MSA_OK) return st;
  if (p->q_len > kMaxNodes || T->d.G > 128) return MSA_ERR_UNSUPPORTED;
  T->rows = T->d.f32 ? msa::kSimtTreeRows : msa::kTcTreeRows;
  T->groups = (T->d.Sq * T->d.G + T->rows - 1) / T->rows;
  if ((long long)T->d.B * T->d.Hkv * T->groups * (T->d.D / 8) >= (1LL << 31) ||
      (long long)T->d.B * T->d.Hkv * T->groups >= (1LL << 31))
    return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

struct TreeLayout {
  size_t status, bits, part_o, part_ml, total;
};

TreeLayout tree_layout(const Tree& T) {
  TreeLayout L{};
  size_t off = 0;
  auto take = [&](size_t bytes) { size_t o = off; off += align_up(bytes); return o; };
  const size_t rows = size_t(msa::tree_ctas(T.d.f32)) * 2 * T.rows;
  L.status = take(sizeof(int32_t));
  if (!T.d.f32) L.bits = take(size_t(T.d.B) * (T.d.Sq + 1) * sizeof(uint4));
  L.part_o = take(rows * T.d.D * sizeof(float));
  L.part_ml = take(rows * sizeof(float2));
  L.total = off;
  return L;
}

msa_status_t resolve_norm(const msa_norm_rope_t* p, msa::NormRope* P) {
  if (!p || p->rows < 0 || p->num_q_heads < 1 || p->num_kv_heads < 0 || p->head_dim < 1 ||
      p->rotary_dim < 0 || p->rotary_dim > p->head_dim || p->reserved != 0)
    return MSA_ERR_INVALID_ARG;
  if (p->dtype != MSA_BF16 && p->dtype != MSA_F32) return MSA_ERR_INVALID_ARG;
  if (!(p->eps >= 0.0f) || isinf(p->eps)) return MSA_ERR_INVALID_ARG;
  if (p->head_dim != 32 && p->head_dim != 64 && p->head_dim != 128) return MSA_ERR_UNSUPPORTED;
  if (p->rotary_dim % 16 != 0) return MSA_ERR_UNSUPPORTED;
  if (p->num_q_heads > 65536 || p->num_kv_heads > 65536 || p->rows >= (1LL << 31))
    return MSA_ERR_UNSUPPORTED;
  *P = msa::NormRope{p->rows, p->num_q_heads, p->num_kv_heads, p->head_dim, p->rotary_dim,
                     p->interleaved != 0, p->dtype == MSA_F32, p->eps, p->q_stride, p->k_stride,
                     p->q_out_stride, p->k_out_stride, p->dq_stride, p->dk_stride};
  return MSA_OK;
}

// An output that starts on the other heads' input or output (it may lie on its own input).
bool crossed(const msa::NormRope& P, const void* q_in, const void* k_in, const void* q_out,
             const void* k_out) {
  return P.hk && (q_out == k_in || k_out == q_in || q_out == k_out);
}

// A row stride holds the heads and keeps rows on 16-byte boundaries.
bool stride_ok(const msa::NormRope& P, long long stride, int heads) {
  return stride >= (long long)heads * P.D && stride % (P.f32 ? 4 : 8) == 0 &&
         stride < (1LL << 40);
}

}  // namespace

extern "C" {

size_t msa_dense_workspace_size(const msa_problem_t* p, const int32_t* cu_seqlens_q_opt,
                                const int32_t* cu_seqlens_k_opt, int32_t backward) {
  Dense P;
  if (resolve_dense(p, cu_seqlens_q_opt, cu_seqlens_k_opt, &P, nullptr) != MSA_OK) return 0;
  return dense_layout(P, cu_seqlens_q_opt != nullptr, backward != 0).total;
}

msa_status_t msa_dense_attend(const msa_problem_t* p, const int32_t* cu_seqlens_q_opt,
                              const int32_t* cu_seqlens_k_opt, const void* q, const void* k,
                              const void* v, void* out, float* lse_opt, void* ws,
                              size_t ws_bytes, void* stream) {
  Records R;
  Dense P;
  if (!R.make(p, cu_seqlens_q_opt, cu_seqlens_k_opt)) return MSA_ERR_TOO_LARGE;
  msa_status_t st = resolve_dense(p, cu_seqlens_q_opt, cu_seqlens_k_opt, &P, R.r);
  if (st != MSA_OK) return st;
  if (P.rows_q == 0) return nothing_to_do(ws, ws_bytes, (cudaStream_t)stream);
  if (!pointers_ok(q, k, v, out) || (lse_opt && !aligned16(lse_opt))) return MSA_ERR_INVALID_ARG;
  const DenseLayout L = dense_layout(P, R.r != nullptr, false);
  if ((st = check_ws(ws, ws_bytes, L.total)) != MSA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if ((st = begin(&P, R, L, ws, s)) != MSA_OK) return st;
  int32_t* head = at<int32_t>(ws, L.status);
  return msa::status_of(P.f32
                            ? msa::launch_dense_fwd_simt(P, q, k, v, out, lse_opt, s)
                            : msa::launch_dense_fwd_tc(P, q, k, v, out, lse_opt, head + 1, head, s));
}

msa_status_t msa_dense_backward(const msa_problem_t* p, const int32_t* cu_seqlens_q_opt,
                                const int32_t* cu_seqlens_k_opt, const void* dout, const void* q,
                                const void* k, const void* v, const void* out, const float* lse,
                                void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                                void* stream) {
  Records R;
  Dense P;
  if (!R.make(p, cu_seqlens_q_opt, cu_seqlens_k_opt)) return MSA_ERR_TOO_LARGE;
  msa_status_t st = resolve_dense(p, cu_seqlens_q_opt, cu_seqlens_k_opt, &P, R.r);
  if (st != MSA_OK) return st;
  if (P.table) return MSA_ERR_UNSUPPORTED;
  if (P.rows_k == 0) return nothing_to_do(ws, ws_bytes, (cudaStream_t)stream);
  if (!pointers_ok(k, v, dk, dv)) return MSA_ERR_INVALID_ARG;
  if (P.rows_q > 0 && !pointers_ok(dout, q, out, lse, dq)) return MSA_ERR_INVALID_ARG;
  const DenseLayout L = dense_layout(P, R.r != nullptr, true);
  if ((st = check_ws(ws, ws_bytes, L.total)) != MSA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  // without records the gradients' first kernel clears the head
  const bool own_begin = !P.f32 && !R.r && P.rows_q > 0;
  if (!own_begin && (st = begin(&P, R, L, ws, s)) != MSA_OK) return st;
  int32_t* head = at<int32_t>(ws, L.status);
  const msa::DenseBwdSpace W{at<float>(ws, L.nl), at<float>(ws, L.delta), at<float>(ws, L.room),
                             at<float>(ws, L.part)};
  if (P.f32)
    return msa::status_of(
        msa::launch_dense_bwd_simt(P, dout, q, k, v, out, lse, W, dq, dk, dv, s));
  return msa::status_of(
      msa::launch_dense_bwd_tc(P, dout, q, k, v, out, lse, W, dq, dk, dv, head, s));
}

size_t msa_tree_workspace_size(const msa_problem_t* p) {
  Tree T{};
  if (resolve_tree(p, &T) != MSA_OK) return 0;
  return tree_layout(T).total;
}

msa_status_t msa_tree_attend(const msa_problem_t* p, const void* q, const void* k, const void* v,
                             const uint8_t* tree_mask, int64_t mask_batch_stride,
                             const int32_t* kv_lens, void* out, float* lse_opt, void* ws,
                             size_t ws_bytes, void* stream) {
  Tree T{};
  msa_status_t st = resolve_tree(p, &T);
  if (st != MSA_OK) return st;
  if (T.d.rows_q == 0) return nothing_to_do(ws, ws_bytes, (cudaStream_t)stream);
  if (!pointers_ok(q, k, v, out) || (lse_opt && !aligned16(lse_opt)) || !tree_mask || !kv_lens ||
      (reinterpret_cast<uintptr_t>(kv_lens) & 3u) != 0)
    return MSA_ERR_INVALID_ARG;
  if (mask_batch_stride != 0 && mask_batch_stride < (int64_t)T.d.Sq * T.d.Sq)
    return MSA_ERR_INVALID_ARG;
  const TreeLayout L = tree_layout(T);
  if ((st = check_ws(ws, ws_bytes, L.total)) != MSA_OK) return st;
  T.mask = tree_mask;
  T.mask_stride = mask_batch_stride;
  T.kv_lens = kv_lens;
  T.bits = at<uint4>(ws, L.bits);
  T.part_o = at<float>(ws, L.part_o);
  T.part_ml = at<float2>(ws, L.part_ml);
  cudaStream_t s = (cudaStream_t)stream;
  int32_t* status = at<int32_t>(ws, L.status);
  if (!T.d.f32)
    return msa::status_of(msa::launch_tree_tc(T, q, k, v, out, lse_opt, status, s));
  cudaError_t e = cudaMemsetAsync(status, 0, sizeof(int32_t), s);
  if (e == cudaSuccess) e = msa::launch_tree_simt(T, q, k, v, out, lse_opt, status, s);
  return msa::status_of(e);
}

size_t msa_norm_rope_workspace_size(const msa_norm_rope_t* p) {
  msa::NormRope P;
  if (resolve_norm(p, &P) != MSA_OK) return 0;
  return align_up(size_t(std::max(1, msa::norm_rope_partials(P))) * P.D * sizeof(float));
}

msa_status_t msa_qk_norm_rope(const msa_norm_rope_t* p, const void* q, const void* k,
                              const void* q_weight, const void* k_weight, const double* inv_freq,
                              const int64_t* positions, void* q_out, void* k_out, void* stream) {
  msa::NormRope P;
  msa_status_t st = resolve_norm(p, &P);
  if (st != MSA_OK) return st;
  if (P.rows == 0) return MSA_OK;
  if (!pointers_ok(q, q_weight, q_out) || !stride_ok(P, P.qs, P.hq) || !stride_ok(P, P.qos, P.hq))
    return MSA_ERR_INVALID_ARG;
  if (P.hk && (!pointers_ok(k, k_weight, k_out) || !stride_ok(P, P.ks, P.hk) ||
               !stride_ok(P, P.kos, P.hk)))
    return MSA_ERR_INVALID_ARG;
  if (P.rot && (!inv_freq || !positions || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
                (reinterpret_cast<uintptr_t>(positions) & 7u)))
    return MSA_ERR_INVALID_ARG;
  if (crossed(P, q, k, q_out, k_out)) return MSA_ERR_INVALID_ARG;
  return msa::status_of(msa::launch_norm_rope(P, q, k, q_weight, k_weight, inv_freq, positions,
                                              q_out, k_out, (cudaStream_t)stream));
}

msa_status_t msa_qk_norm_rope_backward(const msa_norm_rope_t* p, const void* dq_out,
                                       const void* dk_out, const void* q, const void* k,
                                       const void* q_weight, const void* k_weight,
                                       const double* inv_freq, const int64_t* positions, void* dq,
                                       void* dk, float* dq_weight, float* dk_weight, void* ws,
                                       size_t ws_bytes, void* stream) {
  msa::NormRope P;
  msa_status_t st = resolve_norm(p, &P);
  if (st != MSA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (!pointers_ok(dq_weight) || (P.hk && !pointers_ok(dk_weight))) return MSA_ERR_INVALID_ARG;
  if (P.rows == 0) {  // sums over nothing
    cudaError_t e = cudaMemsetAsync(dq_weight, 0, P.D * sizeof(float), s);
    if (e == cudaSuccess && P.hk) e = cudaMemsetAsync(dk_weight, 0, P.D * sizeof(float), s);
    return msa::status_of(e);
  }
  if (!pointers_ok(dq_out, q, q_weight, dq) || !stride_ok(P, P.qs, P.hq) ||
      !stride_ok(P, P.qos, P.hq) || !stride_ok(P, P.dqs, P.hq))
    return MSA_ERR_INVALID_ARG;
  if (P.hk && (!pointers_ok(dk_out, k, k_weight, dk) || !stride_ok(P, P.ks, P.hk) ||
               !stride_ok(P, P.kos, P.hk) || !stride_ok(P, P.dks, P.hk)))
    return MSA_ERR_INVALID_ARG;
  if (P.rot && (!inv_freq || !positions || (reinterpret_cast<uintptr_t>(inv_freq) & 7u) ||
                (reinterpret_cast<uintptr_t>(positions) & 7u)))
    return MSA_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, msa_norm_rope_workspace_size(p))) != MSA_OK) return st;
  if (crossed(P, q, k, dq, dk) || crossed(P, dq_out, dk_out, dq, dk)) return MSA_ERR_INVALID_ARG;
  return msa::status_of(msa::launch_norm_rope_backward(
      P, dq_out, dk_out, q, k, q_weight, k_weight, inv_freq, positions, dq, dk, dq_weight,
      dk_weight, static_cast<float*>(ws), s));
}

}  // extern "C"

namespace msa {
namespace {

// Records per launch: as many as fit the 4 KB of kernel parameters.
constexpr int kChunkRecs = 112;
struct Chunk {
  SeqRec r[kChunkRecs];
};

__global__ void dense_begin_kernel(const __grid_constant__ Chunk c, SeqRec* dst, int n,
                                   int32_t* head) {
  tc::griddep_launch();
  if (head && threadIdx.x < kHeadWords) head[threadIdx.x] = 0;
  if (int(threadIdx.x) < n) dst[threadIdx.x] = c.r[threadIdx.x];
}

__global__ void dense_check_table_kernel(const int32_t* table, long long n, int pages,
                                         int32_t* status) {
  const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n && (table[i] < 0 || table[i] >= pages)) atomicOr(status, kStatusBadPage);
}

}  // namespace

cudaError_t launch_dense_begin(int32_t* head, const SeqRec* host, SeqRec* dst, int n,
                               cudaStream_t s) {
  for (int i = 0; i == 0 || i < n; i += kChunkRecs) {
    Chunk c;
    const int m = std::min(kChunkRecs, n - i);
    std::copy(host + i, host + i + m, c.r);
    std::fill(c.r + m, c.r + kChunkRecs, SeqRec{});
    dense_begin_kernel<<<1, 128, 0, s>>>(c, dst + i, m, i == 0 ? head : nullptr);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_dense_check_table(const Dense& P, int32_t* status, cudaStream_t s) {
  if (!P.table) return cudaSuccess;
  const long long n = (long long)P.B * P.table_w;
  dense_check_table_kernel<<<unsigned((n + 255) / 256), 256, 0, s>>>(P.table, n, P.pages, status);
  return cudaGetLastError();
}

int tree_ctas(bool f32) {
  // the SM count of a B200: a fixed number, so that the workspace size and the way
  // the work is cut do not depend on the device that happens to be current; the small
  // blocks of the fp32 kernel run two to an SM
  return f32 ? 2 * 148 : 148;
}

}  // namespace msa
