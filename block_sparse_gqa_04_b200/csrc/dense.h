// Internal launch interface of the dense-attention operators (dense_api.cu and
// their kernel files).  Not part of the public header.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/msa.h"
#include "internal.h"

namespace msa {

constexpr int kDenseTile = 128;  // query rows and keys of a tile, tokens of a page
constexpr int kStatusBadLength = 8;  // a kv_lens entry outside the cache

// One sequence of a packed batch.  q0, k0: its first rows; pos0: position of its
// first query row; qt0, kt0, pr0: query tiles, key tiles and (tensor-core forward)
// row-tile pairs x key heads of the sequences before it in this list, which is
// sorted by length, longest first, so that the heaviest work is dealt out first.
// qp0: its first row where every sequence's rows are padded to a multiple of 16.
struct SeqRec {
  int q0, k0, nq, nk, pos0, qt0, kt0, pr0, qp0;
};

__host__ __device__ inline int pad16(int n) { return (n + 15) & ~15; }

struct Dense {
  int B, Sq, Skv;      // batched layout (seqs == nullptr); B is the number of records otherwise
  int Hq, Hkv, G, D;
  float scale;
  bool f32;
  int pos0;            // batched layout: position of query row 0
  long long rows_q, rows_k;  // rows of q and of k in memory
  long long rows_pad;        // rows of q, every sequence's padded to a multiple of 16
  int qtiles, ktiles;  // 128-row query tiles and key tiles of all sequences
  int pairs;           // row-tile pairs x key heads of all sequences
  const SeqRec* seqs;  // device, B records, or nullptr
  const int32_t* table;  // block table or nullptr
  int pages, table_w;
};

// Row-tile pairs of one key head of a sequence with nqt query tiles: the G heads'
// tiles of one query tile one after another, two at a time.
__host__ __device__ inline int dense_pairs(int nqt, int G) { return (nqt * G + 1) / 2; }

struct Tree {
  Dense d;               // Sq = nodes per sequence, Skv = cache capacity
  const uint8_t* mask;   // [.., nodes, nodes]
  long long mask_stride; // bytes from one sequence's mask to the next, 0 = shared
  const int32_t* kv_lens;
  int rows;              // (node, head) rows of one work unit
  int groups;            // units per (sequence, key head)
  bool q_boxes;          // tensor cores: 128 rows are the heads of whole nodes
  uint4* bits;           // tensor cores: the masks as bits, [masks, nodes + 1]
  float* part_o;         // [2 * CTAs, D, rows] unnormalised partial outputs
  float2* part_ml;       // [2 * CTAs, rows] base-2 running maximum and sum
};

// Head of a workspace: the status word, then work counters of the tensor-core kernels.
constexpr int kHeadWords = 4;
// Zeroes the head and brings a packed batch's n records (or none) into device memory, as
// kernel parameters: nothing is read from host memory after the launch.
cudaError_t launch_dense_begin(int32_t* head, const SeqRec* host, SeqRec* dst, int n,
                               cudaStream_t s);
// Flags a block table's entries outside the pool (no launch without a table).
cudaError_t launch_dense_check_table(const Dense& P, int32_t* status, cudaStream_t s);

cudaError_t launch_dense_fwd_simt(const Dense& P, const void* q, const void* k, const void* v,
                                  void* out, float* lse, cudaStream_t s);
// bf16 on the tensor cores; counter: a zeroed word.
cudaError_t launch_dense_fwd_tc(const Dense& P, const void* q, const void* k, const void* v,
                                void* out, float* lse, int32_t* counter, int32_t* status,
                                cudaStream_t s);
// Scratch of the gradients: on the tensor cores -lse log2 e, -delta and what the rounding
// of out can have taken from delta, [Hq, rows_pad] + 128 values each, in fp32 delta
// [rows_q, Hq]; with several splits their partial sums, [splits][2][rows_k, Hkv, D].
struct DenseBwdSpace {
  float *nl, *dl, *room, *part;
};
int dense_bwd_splits(const Dense& P);
// Zeroes the head words itself.
cudaError_t launch_dense_bwd_tc(const Dense& P, const void* dout, const void* q, const void* k,
                                const void* v, const void* out, const float* lse,
                                const DenseBwdSpace& W, void* dq, void* dk, void* dv,
                                int32_t* head, cudaStream_t s);
// fp32 on the CUDA cores (nl and room unused).
cudaError_t launch_dense_bwd_simt(const Dense& P, const void* dout, const void* q, const void* k,
                                  const void* v, const void* out, const float* lse,
                                  const DenseBwdSpace& W, void* dq, void* dk, void* dv,
                                  cudaStream_t s);
// dk, dv = the sum of the splits' partial sums [splits][dv, dk][n], dk scaled.
template <typename T>
cudaError_t launch_dkv_sum(const float* part, int splits, long long n, float scale, T* dk, T* dv,
                           cudaStream_t s);

constexpr int kSimtTreeRows = 32;  // rows of a work unit on the CUDA cores
constexpr int kTcTreeRows = 128;   // and on the tensor cores
int tree_ctas(bool f32);           // CTAs of a tree launch
// Joins the partial states (second launch of either tree kernel).
cudaError_t launch_tree_combine(const Tree& T, void* out, float* lse, cudaStream_t s);
cudaError_t launch_tree_simt(const Tree& T, const void* q, const void* k, const void* v, void* out,
                             float* lse, int32_t* status, cudaStream_t s);

// Clears the status word itself.
cudaError_t launch_tree_tc(const Tree& T, const void* q, const void* k, const void* v, void* out,
                           float* lse, int32_t* status, cudaStream_t s);

struct NormRope {
  long long rows;
  int hq, hk, D, rot;
  bool inter, f32;
  float eps;
  long long qs, ks, qos, kos, dqs, dks;
};
int norm_rope_partials(const NormRope& P);  // partial weight gradients of the backward pass
cudaError_t launch_norm_rope(const NormRope& P, const void* q, const void* k, const void* qw,
                             const void* kw, const double* inv_freq, const int64_t* pos,
                             void* qo, void* ko, cudaStream_t s);
cudaError_t launch_norm_rope_backward(const NormRope& P, const void* gq, const void* gk,
                                      const void* q, const void* k, const void* qw,
                                      const void* kw, const double* inv_freq, const int64_t* pos,
                                      void* dq, void* dk, float* dqw, float* dkw, float* part,
                                      cudaStream_t s);

}  // namespace msa
