// Device helpers of the dense-attention kernels: which sequence, rows and keys a
// piece of work covers.
#pragma once

#include "common.cuh"
#include "dense.h"
#include "tc_common.cuh"

namespace msa {

// Last record whose prefix (member F) is <= x: the one that owns item x.
template <int SeqRec::*F>
__device__ __forceinline__ int find_seq(const SeqRec* seqs, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (seqs[mid].*F <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ SeqRec batch_seq(const Dense& P, int b) {
  // the rows of q, and of an unpaged k, are below 2^31; a paged k has no k0
  return SeqRec{b * P.Sq, P.table ? 0 : b * P.Skv, P.Sq, P.Skv, P.pos0, 0, 0, 0,
                b * pad16(P.Sq)};
}

// Query tile `t` of all sequences: its sequence and its tile there, last (heaviest)
// tiles first within a sequence and, in a batch, across it.
__device__ __forceinline__ SeqRec query_tile(const Dense& P, int t, int* qt) {
  if (P.seqs) {
    const SeqRec s = P.seqs[find_seq<&SeqRec::qt0>(P.seqs, P.B, t)];
    *qt = (s.nq + kDenseTile - 1) / kDenseTile - 1 - (t - s.qt0);
    return s;
  }
  const int n = (P.Sq + kDenseTile - 1) / kDenseTile;
  *qt = n - 1 - t / P.B;
  return batch_seq(P, t % P.B);
}

// Key tile `t` of all sequences: first (heaviest: seen by most rows) tiles first.
__device__ __forceinline__ SeqRec key_tile(const Dense& P, int t, int* kt) {
  if (P.seqs) {
    const SeqRec s = P.seqs[find_seq<&SeqRec::kt0>(P.seqs, P.B, t)];
    *kt = t - s.kt0;
    return s;
  }
  *kt = t / P.B;
  return batch_seq(P, t % P.B);
}

// Memory row of key tile kt of a sequence: contiguous, or the page that the block
// table names (page 0 for an entry outside the pool).
__device__ __forceinline__ long long tile_row(const Dense& P, int b, int k0, int kt) {
  if (!P.table) return (long long)k0 + (long long)kt * kDenseTile;
  const int pg = P.table[(long long)b * P.table_w + kt];
  return (pg >= 0 && pg < P.pages) ? (long long)pg * kDenseTile : 0;
}

// ---------------------------------------------------------------------------
// Tree attention: the key tiles of all work units, in unit order, are cut into
// equal contiguous shares, one per CTA, so that every CTA streams the same amount
// of cache whatever the sequences' lengths.  A unit is (sequence, key head, group of
// `rows` (node, head) rows) over ceil((len + nodes) / 128) key tiles.  A unit inside
// one share is finished there; one cut by a share's border leaves partial states:
// slot 2*cta for the piece that began in an earlier share, 2*cta + 1 for the piece
// that starts in this share and goes on.
// ---------------------------------------------------------------------------
struct TreeSeq {
  int len, tiles;  // cached tokens, key tiles of one unit
};

__device__ __forceinline__ TreeSeq tree_seq(const Tree& T, int b) {
  const int len = max(0, min(T.kv_lens[b], T.d.Skv - T.d.Sq));
  return TreeSeq{len, (len + T.d.Sq + kDenseTile - 1) / kDenseTile};
}

struct TreeSpan {
  long long total;  // key tiles of all units
  long long share;  // of one CTA
};

__device__ __forceinline__ long long tree_share(long long total, int ctas) {
  return (total + ctas - 1) / ctas;
}

// Called by whole warps.
__device__ __forceinline__ TreeSpan tree_span(const Tree& T, int ctas) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  for (int b = lane; b < T.d.B; b += 32) sum += tree_seq(T, b).tiles;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(MSA_FULL_MASK, sum, o);
  const long long total = sum * T.d.Hkv * T.groups;
  return TreeSpan{total, tree_share(total, ctas)};
}

// Walks the pieces of the share [at, end).
struct TreeWalk {
  long long at, end, first;  // first: tile at which sequence b's units start
  int b;
  TreeSeq s;

  // Called by whole warps.  Up to 32 sequences take one read of their lengths.
  __device__ __forceinline__ void begin(const Tree& T, int cta, int ctas) {
    const int lane = threadIdx.x & 31, per = T.d.Hkv * T.groups;
    const bool few = T.d.B <= 32;
    long long total = few ? 0 : tree_span(T, ctas).total;
    at = end = first = 0;
    b = 0;
    // the sequence that holds tile `at`: 32 sequences at a time
    for (int base = 0;; base += 32) {
      long long mine = base + lane < T.d.B ? (long long)tree_seq(T, base + lane).tiles * per : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(MSA_FULL_MASK, mine, o);
        if (lane >= o) mine += up;
      }
      if (base == 0) {
        if (few) total = __shfl_sync(MSA_FULL_MASK, mine, 31);
        const long long share = tree_share(total, ctas);
        at = min(share * cta, total);
        end = min(at + share, total);
        if (at >= end) break;
      }
      const unsigned past = __ballot_sync(MSA_FULL_MASK, first + mine > at);
      if (past) {
        const int w = __ffs(past) - 1;
        const long long before = __shfl_sync(MSA_FULL_MASK, mine, max(w - 1, 0));
        if (w > 0) first += before;
        b = base + w;
        break;
      }
      first += __shfl_sync(MSA_FULL_MASK, mine, 31);
    }
    s = tree_seq(T, b);
  }

  struct Piece {
    int b, g, group;     // sequence, key head, row group
    int kt0, kt1;        // key tiles [kt0, kt1) of the unit
    int len;             // cached tokens
    int slot;            // -1: the whole unit; 0: began earlier; 1: begins here, goes on
  };

  // The next piece, or false at the share's end.  b advances with the lengths read
  // one sequence ahead of need only.
  __device__ __forceinline__ bool next(const Tree& T, Piece* p) {
    if (at >= end) return false;
    const int per = T.d.Hkv * T.groups;
    while (at >= first + (long long)s.tiles * per) {
      first += (long long)s.tiles * per;
      s = tree_seq(T, ++b);
    }
    const long long into = at - first;
    const bool narrow = into < (1LL << 32);  // a 64-bit division takes hundreds of cycles
    const int unit = narrow ? int(unsigned(into) / unsigned(s.tiles)) : int(into / s.tiles);
    const int kt0 = int(into - (long long)unit * s.tiles);
    const int n = int(min((long long)(s.tiles - kt0), end - at));
    *p = Piece{b, unit / T.groups, unit % T.groups, kt0, kt0 + n, s.len,
               kt0 > 0 ? 0 : (n < s.tiles ? 1 : -1)};
    at += n;
    return true;
  }
};

// Launches a kernel whose set-up may run while its predecessor in the stream finishes
// (the kernel calls griddep_wait()).
template <typename... P, typename... A>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                                cudaStream_t s, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...);
}

}  // namespace msa
