// Gradients of dense causal attention on tcgen05 tensor cores (bf16, head_dim 64 or
// 128), in two passes so that every sum has one owner and a fixed order (no atomics):
//   dk, dv: a CTA owns 128 keys of a key head and walks the group's heads and the query
//           tiles that see them.  With keys as rows (lanes of TMEM),
//             S^T = K Q^T,  dP^T = V dO^T,  P^T = 2^(c S^T - c lse),
//             dS^T = P^T (dP^T - delta),  dV += P^T dO,  dK += dS^T Q:
//           P^T and dS^T are written to TMEM over S^T and dP^T as bf16 and are A operands
//           there; Q and dO serve as K-major operands of the first two products and as
//           MN-major operands of the last two, so nothing is stored twice.
//   dq:     a CTA owns 128 query rows of a head and walks the keys they see, with the
//           rows as lanes: S = Q K^T, dP = dO V^T, dS as above, dQ += dS K.
// The two passes take 4 + 4 products of 128 x 128 x D per pair of tiles where a single
// pass would take 5; in exchange no gradient leaves the chip before it is finished (the
// single pass would add 64 KB of dQ per pair of tiles to memory, 4.4 GB for 2 x 4096 rows
// x 64 heads, in an order that changes).
//
// Roundings.  P and dS meet the MMAs as bf16.  For dq, where nothing but dS is rounded
// before the result, dS is the sum of two bf16 numbers (the fourth product): its error
// falls from 0.0025 to 0.0019, of which a bf16 result's own rounding is 0.0017.  delta =
// sum_d dout out is formed from the rounded out; where P sums to 1, the dq pass knows
// what delta lacks, sum_j P (dP - delta), and leaves delta completed for dk (error of dk
// 0.0024 instead of 0.02 to 0.06 with values of 100 +- 8).  It does so only where the sum
// differs from 1 by no more than fp32 leaves of it, and by no more than a rounding can
// have taken from out: half a step of sum_d |dout out|.  So out and lse may be those of
// more keys than the call's, whatever weight and values the others have.
//
// One thread issues all MMAs in an order that keeps the pipe fed while the sixteen
// elementwise warps (four warpgroups, a quarter of the columns each) work on the other
// half of a step: dK, dV pass ... dV(i) S(i+1) | dK(i) dP(i+1) | ..., dq pass ... dP(i+1)
// dQ(i) S(i+2) ... with dS over the scores that made it, so that dP is free at once.  A
// second warp gathers every other condition of the products into the barrier that the
// elementwise warps complete, so that the issuing thread waits for one thing at a time.
//
// What bounds them (2 x 4096 rows x 64 heads x 128: dk, dv 0.87 ms, dq 0.85 ms; the tensor
// pipe 66 % busy in both): a dk, dv step has 2048 cycles of MMA and takes ~2900, the chain
// dV, S, P (its exponentials) and the barriers between them; a dq step has 2048 and takes
// ~2900, of which the elementwise warps are busy 2500.
//
// Rows behind the end of a sequence come in with its last tiles.  Query rows there have
// lse = inf, hence P = 0 (and are masked: a key may hold anything); the products that sum
// over rows stop at whole groups of 16, and the rest of the last group is zeroed in shared
// memory before use.
#include <algorithm>

#include "dense_tc.cuh"

namespace msa {
namespace {

// warp 0 items and TMA, warp 1 MMA, warp 2 waits for it, warp 3 idle, warps 4-19 elementwise
constexpr int kWarpgroups = 4;  // elementwise; each takes 32 columns of a tile
constexpr int kThreads = 128 + 128 * kWarpgroups;
constexpr uint32_t kTmemCols = 512;
constexpr int kItems = 2;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kHalf = 128 * 64 * 2;
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, 128, 0, 0);
  static constexpr uint32_t kIdescG = tc::idesc_bf16_f32(128, D, 0, 1);
};

__device__ __forceinline__ uint64_t pair_of(const uint32_t* v) {
  return (uint64_t(v[1]) << 32) | v[0];
}
__device__ __forceinline__ float lo_of(uint64_t x) { return __uint_as_float(uint32_t(x)); }
__device__ __forceinline__ float hi_of(uint64_t x) { return __uint_as_float(uint32_t(x >> 32)); }

// P of the pair of columns `pair`, POLY of every 8 pairs on the FMA pipe.  The dk, dv pass
// waits for P on the exp2 unit's 1024 cycles a step: 3 of 8 take it from 0.886 to 0.865 ms
// (2 x 4096 rows; 1 of 8 0.878, 2 0.866, 4 0.909).  The dq pass does not gain (0.847 with
// none, 0.871 with 3 of 8), nor does the forward pass (0.885 ms for 8192 rows with none,
// 0.954 with 1 of 8): there a warp alone on its scheduler pays for every instruction.
template <int POLY>
__device__ __forceinline__ void exp2_pair(uint32_t* p, uint64_t z, int pair) {
  if ((pair * POLY) % 8 < POLY) {
    const uint64_t y = exp2_poly(z);
    p[0] = uint32_t(y);
    p[1] = uint32_t(y >> 32);
  } else {
    p[0] = __float_as_uint(ex2_f32(lo_of(z)));
    p[1] = __float_as_uint(ex2_f32(hi_of(z)));
  }
}

// Low words of the tiles' descriptors, and the upper word that they share.
constexpr uint32_t kHi = uint32_t(tc::kDescHi | (1024 >> 4));
__device__ __forceinline__ uint32_t kmajor(const uint8_t* tile) {
  return uint32_t(tc::sdesc_sw128(tc::smem_addr(tile), 16, 1024));
}
template <int D>
__device__ __forceinline__ uint32_t mnmajor(const uint8_t* tile) {
  return uint32_t(tc::sdesc_sw128(tc::smem_addr(tile), Cfg<D>::kHalf, 1024));
}

// S = A B^T over D, both tiles K-major.
template <int D>
__device__ __forceinline__ void issue_nt(uint32_t d, uint32_t a, uint32_t b) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk >> 2) * (Cfg<D>::kHalf / 16) + (kk & 3) * 2;
    tc::mma_ss_lo(d, a + off, b + off, kHi, Cfg<D>::kIdescS, kk > 0 ? 1u : 0u);
  }
}

// G += A B over `groups` groups of 16 rows of B (MN-major tile); A in TMEM as bf16, 32
// columns of elements in 16 TMEM columns at a, the next 32 at a + 32 and so on (each
// warpgroup writes over what it has read itself).
template <int D>
__device__ __forceinline__ void issue_ts(uint32_t d, uint32_t a, uint32_t b, int groups,
                                         uint32_t accumulate) {
  if (groups == 8) {
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)
      tc::mma_ts_lo(d, a + (kk >> 1) * 32 + (kk & 1) * 8, b + kk * 128, kHi, Cfg<D>::kIdescG,
                    kk > 0 ? 1u : accumulate);
  } else {
#pragma unroll 1
    for (int kk = 0; kk < groups; ++kk)
      tc::mma_ts_lo(d, a + (kk >> 1) * 32 + (kk & 1) * 8, b + kk * 128, kHi, Cfg<D>::kIdescG,
                    kk > 0 ? 1u : accumulate);
  }
}

// ---------------------------------------------------------------------------
// -c lse, -delta = -sum_d dout out and room = 2^-8 sum_d |dout out|, half a step of bf16,
// per (head, row), rows of a sequence padded to groups of 16 (padding: -inf, so that P = 0,
// and 0): one warp per (16 rows, head).
// ---------------------------------------------------------------------------
template <int D>
__global__ void __launch_bounds__(256)
dense_prep_kernel(Dense P, const __nv_bfloat16* __restrict__ dout,
                  const __nv_bfloat16* __restrict__ out, const float* __restrict__ lse,
                  float* __restrict__ nl, float* __restrict__ dl, float* __restrict__ room,
                  int* __restrict__ head) {
  tc::griddep_wait();  // the records are in place
  tc::griddep_launch();
  if (blockIdx.x == 0 && threadIdx.x < kHeadWords) head[threadIdx.x] = 0;
  constexpr int kLanes = D / 8, kRowsAtOnce = 32 / kLanes;
  const long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int h = int(w % P.Hq);
  const long long x0 = w / P.Hq * 16;  // padded row
  if (x0 >= P.rows_pad) return;
  SeqRec s;
  if (P.seqs) {
    s = P.seqs[find_seq<&SeqRec::qp0>(P.seqs, P.B, int(x0))];
  } else {
    s = batch_seq(P, int(x0 / pad16(P.Sq)));
  }
  const int i0 = int(x0) - s.qp0;
  float mine = 0.f, size = 0.f;
#pragma unroll
  for (int r0 = 0; r0 < 16; r0 += kRowsAtOnce) {
    const int i = i0 + r0 + lane / kLanes;
    float sum = 0.f, mag = 0.f;
    if (i < s.nq) {
      const long long at = ((long long)(s.q0 + i) * P.Hq + h) * D + (lane % kLanes) * 8;
      float a[8], b[8];
      load_vec<__nv_bfloat16, 8>(dout + at, a);
      load_vec<__nv_bfloat16, 8>(out + at, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum += a[e] * b[e];
        mag += fabsf(a[e] * b[e]);
      }
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(MSA_FULL_MASK, sum, o);
      mag += __shfl_xor_sync(MSA_FULL_MASK, mag, o);
    }
    // lane r of the warp keeps row r
    const int from = (lane % kRowsAtOnce) * kLanes;
    const float got = __shfl_sync(MSA_FULL_MASK, sum, from);
    const float got_mag = __shfl_sync(MSA_FULL_MASK, mag, from);
    if (lane / kRowsAtOnce == r0 / kRowsAtOnce) {
      mine = got;
      size = got_mag;
    }
  }
  if (lane < 16) {
    const bool there = i0 + lane < s.nq;
    const long long at = (long long)h * P.rows_pad + x0 + lane;
    nl[at] = there ? -kLog2e * lse[(long long)(s.q0 + i0 + lane) * P.Hq + h] : -INFINITY;
    dl[at] = there ? -mine : 0.f;
    room[at] = there ? 0x1p-8f * size : 0.f;
  }
}

// ---------------------------------------------------------------------------
// dk, dv
// ---------------------------------------------------------------------------
struct KeyItem {
  int live;
  int nk, j0, k0, g;      // keys of the sequence; first key of the tile; its first row in k
  int h0, heads;          // heads of this item
  int qt0, nqt;           // query tiles that see the tile
  int q0, qp0, nq, pos0;
  int split;
};

struct KeyBars {
  uint64_t kv_full, kv_empty;
  uint64_t q_full[3], q_empty[3], g_full[2], g_empty[2];  // stages of Q and of dO
  uint64_t nd_full[2];   // lse and delta; a slot is free with the Q stage of its step
  // first_full: the item's K, V and first Q, dO are there; p_full, ds_full: P and dS
  // written, and the next step's Q and dO are there
  uint64_t first_full, s_full, p_full, dp_full, ds_full, acc_full, acc_empty;
  uint64_t i_full[kItems], i_empty[kItems];
  uint64_t mma_done;
  KeyItem item[kItems];
  alignas(16) float nl[2][128];
  alignas(16) float dl[2][128];
  uint32_t tmem_base;
  int abort;
};

// The dynamic part starts on a 1024-byte boundary, there is no room to align it by hand
// (the kernel looks, and refuses to run otherwise).
template <int D>
constexpr size_t key_smem() {
  return size_t(7) * Cfg<D>::kTileBytes + sizeof(KeyBars);
}
static_assert(key_smem<128>() <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void make_key_item(const Dense& P, int t, int splits, KeyItem* it) {
  const int split = t % splits;
  t /= splits;
  const int g = t % P.Hkv;
  int kt;
  const SeqRec s = key_tile(P, t / P.Hkv, &kt);
  const int per = (P.G + splits - 1) / splits;
  it->live = 1;
  it->nk = s.nk;
  it->j0 = kt * kDenseTile;
  it->k0 = s.k0 + it->j0;
  it->g = g;
  it->h0 = g * P.G + split * per;
  it->heads = max(0, min(per, P.G - split * per));
  // the first query row that sees key j0 sits at position j0
  const int nqt = tiles_of(s.nq);
  it->qt0 = min(max(0, it->j0 - s.pos0) / kDenseTile, nqt);
  it->nqt = nqt;
  it->q0 = s.q0;
  it->qp0 = s.qp0;
  it->nq = s.nq;
  it->pos0 = s.pos0;
  it->split = split;
}

template <int D, bool PART>
__global__ void __launch_bounds__(kThreads, 1)
dense_dkv_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_g,
                    const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v, Dense P, int splits, int items,
                    const float* nl, const float* dl,
                    __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv,
                    float* __restrict__ part, int* __restrict__ next_item,
                    int* __restrict__ status) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (tc::smem_addr(smem) & 1023) {
    tc::griddep_wait();
    if (threadIdx.x == 0) atomicOr(status, tc::kStatusWaitTimeout);
    return;
  }
  uint8_t* kbuf = smem;
  uint8_t* vbuf = kbuf + C::kTileBytes;
  uint8_t* qbuf = vbuf + C::kTileBytes;        // [3]
  uint8_t* gbuf = qbuf + 3 * C::kTileBytes;    // [2]
  KeyBars* bars = reinterpret_cast<KeyBars*>(gbuf + 2 * C::kTileBytes);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->kv_full, 1);
    tc::mbar_init(&bars->kv_empty, 1);
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(&bars->q_full[s], 1);
      tc::mbar_init(&bars->q_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->g_full[s], 1);
      tc::mbar_init(&bars->g_empty[s], 1);
      tc::mbar_init(&bars->nd_full[s], 1);
    }
    tc::mbar_init(&bars->first_full, 1);
    tc::mbar_init(&bars->s_full, 1);
    tc::mbar_init(&bars->p_full, 4 * kWarpgroups + 1);   // elementwise warps and warp 2
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->ds_full, 4 * kWarpgroups + 1);
    tc::mbar_init(&bars->acc_full, 1);
    tc::mbar_init(&bars->acc_empty, 4 * kWarpgroups);
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&bars->i_full[i], 1);
      tc::mbar_init(&bars->i_empty[i], 4 * kWarpgroups + 2);  // warps 1, 2, elementwise
    }
    tc::mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch(&tmap_q);
    tc::tma_prefetch(&tmap_g);
    tc::tma_prefetch(&tmap_k);
    tc::tma_prefetch(&tmap_v);
  }
  if (warp == 1) tc::tmem_alloc(&bars->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  tc::griddep_wait();    // the dq pass has completed delta
  tc::griddep_launch();
  // S^T | dP^T | dV | dK
  const uint32_t ts = tmem, tp = tmem + 128, tv = tmem + 256, tk = tmem + 256 + D;
  bool failed = false;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0) {
      tc::ArmedRing kv_armed, q_armed, g_armed, nd_armed;
      int qs = 0;
      uint32_t qp = 0;
      int n = 0, used = 0;  // steps and items with steps so far
      int t = blockIdx.x;   // the first item is the CTA's own
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        if (!tc::mbar_wait(&bars->i_empty[slot], ((ii / kItems) & 1) ^ 1, abort)) {
          failed = true;
          break;
        }
        if (t < items) make_key_item(P, t, splits, &bars->item[slot]);
        else bars->item[slot].live = 0;
        const KeyItem it = bars->item[slot];
        tc::mbar_arrive(&bars->i_full[slot]);
        if (!it.live) break;
        if (it.heads == 0 || it.qt0 >= it.nqt) {
          t = gridDim.x + atomicAdd(next_item, 1);
          continue;
        }
        if (!tc::mbar_wait(&bars->kv_empty, (used & 1) ^ 1, abort)) { failed = true; break; }
        tc::mbar_arrive_expect_tx(&bars->kv_full, 2 * C::kTileBytes);
        kv_armed.note(0, used & 1);
        ++used;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tc::tma_load_3d(kbuf + h * C::kHalf, &tmap_k, &bars->kv_full, 64 * h, it.g, it.k0);
          tc::tma_load_3d(vbuf + h * C::kHalf, &tmap_v, &bars->kv_full, 64 * h, it.g, it.k0);
        }
        for (int hh = it.h0; hh < it.h0 + it.heads && !failed; ++hh) {
          for (int qt = it.qt0; qt < it.nqt; ++qt, ++n) {
            const int s = n & 1, par = (n >> 1) & 1, row = it.q0 + qt * 128;
            const long long at = (long long)hh * P.rows_pad + it.qp0 + qt * 128;
            if (!tc::mbar_wait(&bars->q_empty[qs], qp ^ 1, abort)) { failed = true; break; }
            tc::mbar_arrive_expect_tx(&bars->q_full[qs], C::kTileBytes);
            q_armed.note(qs, qp);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_load_3d(qbuf + qs * C::kTileBytes + h * C::kHalf, &tmap_q, &bars->q_full[qs],
                              64 * h, hh, row);
            if (!tc::mbar_wait(&bars->g_empty[s], par ^ 1, abort)) { failed = true; break; }
            tc::mbar_arrive_expect_tx(&bars->g_full[s], C::kTileBytes);
            g_armed.note(s, par);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_load_3d(gbuf + s * C::kTileBytes + h * C::kHalf, &tmap_g, &bars->g_full[s],
                              64 * h, hh, row);
            // lse and delta: their slot was step n - 2's
            if (n >= 2) {
              const int x = qs == 2 ? 0 : qs + 1;  // (n - 2) % 3
              const uint32_t xp = qs == 2 ? qp : qp ^ 1;
              if (!tc::mbar_wait(&bars->q_empty[x], xp, abort)) { failed = true; break; }
            }
            tc::mbar_arrive_expect_tx(&bars->nd_full[s], 1024);
            nd_armed.note(s, par);
            tc::bulk_load(bars->nl[s], nl + at, 512, &bars->nd_full[s]);
            tc::bulk_load(bars->dl[s], dl + at, 512, &bars->nd_full[s]);
            if (++qs == 3) { qs = 0; qp ^= 1; }
          }
        }
        t = gridDim.x + atomicAdd(next_item, 1);  // late, so that no CTA holds two items
      }
      if (!(kv_armed.drain(&bars->kv_full) && q_armed.drain(bars->q_full) &&
            g_armed.drain(bars->g_full) && nd_armed.drain(bars->nd_full)))
        failed = true;
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (tc::elect_one()) {
      const uint32_t ka = kmajor(kbuf), va = kmajor(vbuf);
      const uint32_t qa = kmajor(qbuf), ga = kmajor(gbuf);
      const uint32_t qb = mnmajor<D>(qbuf), gb = mnmajor<D>(gbuf);
      constexpr uint32_t kTile16 = C::kTileBytes / 16;
      uint32_t n = 0, used = 0;
      int qs = 0;  // Q stage of this step
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        if (!tc::mbar_spin(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
        const KeyItem it = bars->item[slot];
        tc::mbar_arrive(&bars->i_empty[slot]);
        if (!it.live) break;
        const int tiles = it.nqt - it.qt0, steps = it.heads * tiles;
        if (steps <= 0) continue;
        const int last = (min(128, it.nq - (it.nqt - 1) * 128) + 15) >> 4;
        if (!tc::mbar_spin(&bars->first_full, used & 1, abort)) { failed = true; break; }
        tc::tc_fence_after();
        uint32_t off = (n & 1) * kTile16;  // of this step's dO stage
        issue_nt<D>(ts, ka, qa + qs * kTile16);
        tc::mma_commit(&bars->s_full);
        issue_nt<D>(tp, va, ga + off);
        tc::mma_commit(&bars->dp_full);
        int left = tiles;  // query tiles left of the head
        for (int i = 0; i < steps; ++i, ++n, off ^= kTile16) {
          const int s = n & 1, next = qs == 2 ? 0 : qs + 1;
          const int groups = --left == 0 ? last : 8;
          if (left == 0) left = tiles;
          if (!tc::mbar_spin(&bars->p_full, n & 1, abort)) { failed = true; break; }
          tc::tc_fence_after();
          issue_ts<D>(tv, ts, gb + off, groups, i > 0);
          tc::mma_commit(&bars->g_empty[s]);
          if (i + 1 < steps) {
            issue_nt<D>(ts, ka, qa + next * kTile16);
            tc::mma_commit(&bars->s_full);
          }
          if (!tc::mbar_spin(&bars->ds_full, n & 1, abort)) { failed = true; break; }
          tc::tc_fence_after();
          issue_ts<D>(tk, tp, qb + qs * kTile16, groups, i > 0);
          tc::mma_commit(&bars->q_empty[qs]);
          qs = next;
          if (i + 1 < steps) {
            issue_nt<D>(tp, va, ga + (off ^ kTile16));
            tc::mma_commit(&bars->dp_full);
          }
        }
        if (failed) break;
        tc::mma_commit(&bars->kv_empty);
        tc::mma_commit(&bars->acc_full);
        ++used;
      }
      if (!tc::mma_drain(&bars->mma_done)) failed = true;
    }
  } else if (warp == 2) {
    // ---------------- what else the products need ----------------
    uint32_t n = 0, used = 0, qp = 0;
    int qs = 0;
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const KeyItem it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      const int tiles = it.nqt - it.qt0, steps = it.heads * tiles;
      if (steps <= 0) continue;
      const int rows = min(128, it.nq - (it.nqt - 1) * 128);  // of each head's last tile
      // the next step's tile has landed; rows behind the sequence are zero
      auto next_q = [&](bool tail) -> bool {
        if (!warp_wait(&bars->q_full[qs], qp, abort)) return false;
        if (tail && (rows & 15)) zero_rows<D>(qbuf + qs * C::kTileBytes, rows, (rows + 15) & ~15);
        if (++qs == 3) { qs = 0; qp ^= 1; }
        return true;
      };
      auto next_g = [&](uint32_t x, bool tail) -> bool {
        if (!warp_wait(&bars->g_full[x & 1], (x >> 1) & 1, abort)) return false;
        if (tail && (rows & 15))
          zero_rows<D>(gbuf + (x & 1) * C::kTileBytes, rows, (rows + 15) & ~15);
        return true;
      };
      if (!warp_wait(&bars->kv_full, used & 1, abort) || !next_q(tiles == 1) ||
          !next_g(n, tiles == 1)) {
        failed = true;
        break;
      }
      if (lane == 0) tc::mbar_arrive(&bars->first_full);
      int left = tiles;
      for (int i = 0; i < steps; ++i, ++n) {
        if (--left == 0) left = tiles;
        const bool tail = left == 1;  // the next step's tile is its head's last
        // an arrival belongs to this step: the step before is over
        if ((n > 0 && !warp_wait(&bars->p_full, (n & 1) ^ 1, abort)) ||
            (i == 0 && !warp_wait(&bars->acc_empty, (used & 1) ^ 1, abort)) ||
            (i + 1 < steps && !next_q(tail))) {
          failed = true;
          break;
        }
        if (lane == 0) tc::mbar_arrive(&bars->p_full);
        if ((n > 0 && !warp_wait(&bars->ds_full, (n & 1) ^ 1, abort)) ||
            (i + 1 < steps && !next_g(n + 1, tail))) {
          failed = true;
          break;
        }
        if (lane == 0) tc::mbar_arrive(&bars->ds_full);
      }
      ++used;
    }
  } else if (warp >= 4) {
    // ---------------- elementwise: P, dS, then the tile's dV (first half) or dK ----------------
    const int wg = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t sa = ts + lanes + wg * 32, pa = tp + lanes + wg * 32;
    const float sl2 = P.scale * kLog2e;
    const uint64_t sl2x2 = f2(sl2, sl2);
    int n = 0, used = 0;
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const KeyItem it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      const int tiles = it.nqt - it.qt0, steps = it.heads * tiles;
      // first column of this warpgroup's that sees the thread's key, at the first tile
      const int from0 = it.j0 + row - it.pos0 - it.qt0 * 128 - wg * 32;
      const int rows = it.nq - (it.nqt - 1) * 128 - wg * 32;  // of the last tile, from here on
      int from = from0, left = tiles;
      for (int i = 0; i < steps; ++i, ++n) {
        const int s = n & 1;
        const uint32_t par = n & 1;
        if (!warp_wait(&bars->nd_full[s], (n >> 1) & 1, abort)) { failed = true; break; }
        // read before the wait for S: the MMAs' operands keep shared memory so busy that
        // these reads, waited for one by one, took 650 cycles of a step (and delta's 400)
        float4 col[8];
        {
          const float4* src = reinterpret_cast<const float4*>(bars->nl[s] + wg * 32);
#pragma unroll
          for (int x = 0; x < 8; ++x) col[x] = src[x];
        }
        if (!warp_wait(&bars->s_full, par, abort)) { failed = true; break; }
        tc::tc_fence_after();
        uint32_t p[32];
        tc::tmem_ld32(sa, p);
        tc::tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; x += 4) {
          const float4 f = col[x / 4];
          const uint64_t a = fma2(pair_of(&p[x]), sl2x2, f2(f.x, f.y));
          const uint64_t b = fma2(pair_of(&p[x + 2]), sl2x2, f2(f.z, f.w));
          exp2_pair<3>(&p[x], a, x / 2);
          exp2_pair<3>(&p[x + 2], b, x / 2 + 1);
        }
        // columns that do not see the key, and those behind the last row: P = 0, and dS
        // too (the key and its value may hold anything)
        const int to = left == 1 ? rows : 32;
        const bool cut = to < 32 || __any_sync(MSA_FULL_MASK, from > 0);
        if (cut) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x < from || x >= to) p[x] = 0u;
        }
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x)
          w[x] = pack_bf16(__uint_as_float(p[2 * x]), __uint_as_float(p[2 * x + 1]));
        tmem_st8(sa, w);
        tmem_st8(sa + 8, w + 8);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full);
        {
          const float4* src = reinterpret_cast<const float4*>(bars->dl[s] + wg * 32);
#pragma unroll
          for (int x = 0; x < 4; ++x) col[x] = src[x];
          if (!warp_wait(&bars->dp_full, par, abort)) { failed = true; break; }
          tc::tc_fence_after();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t d[16];
            tc::tmem_ld16(pa + h * 16, d);
            tc::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; x += 4) {
              const float4 f = col[x / 4];  // -delta
              const uint32_t* q2 = &p[h * 16 + x];
              if (cut) {
#pragma unroll
                for (int y = 0; y < 4; ++y)
                  if (h * 16 + x + y < from || h * 16 + x + y >= to) d[x + y] = 0u;
              }
              w[h * 8 + x / 2] = to_bf16x2(mul2(pair_of(q2), add2(pair_of(&d[x]), f2(f.x, f.y))));
              w[h * 8 + x / 2 + 1] =
                  to_bf16x2(mul2(pair_of(q2 + 2), add2(pair_of(&d[x + 2]), f2(f.z, f.w))));
            }
            if (h == 0) {
#pragma unroll
              for (int x = 0; x < 4; ++x) col[x] = src[4 + x];
            }
          }
        }
        tmem_st8(pa, w);
        tmem_st8(pa + 8, w + 8);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->ds_full);
        from -= 128;
        if (--left == 0) {  // the next head
          left = tiles;
          from = from0;
        }
      }
      if (failed) break;
      const bool any = steps > 0;
      if (any) {
        if (!warp_wait(&bars->acc_full, used & 1, abort)) { failed = true; break; }
        tc::tc_fence_after();
        ++used;
      }
      const int half = wg >> 1, col0 = (wg & 1) * (D / 2);
      const float scale = half ? P.scale : 1.f;
      const bool mine = it.j0 + row < it.nk;
      const long long at = ((long long)(it.k0 + row) * P.Hkv + it.g) * D + col0;
      const uint32_t acc = (half ? tk : tv) + lanes + col0;
      __nv_bfloat16* dst = half ? dk : dv;
      float* pdst = part + ((long long)(it.split * 2 + half) * P.rows_k * P.Hkv) * D;
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t o[16];
        __syncwarp();
        if (any) {
          tc::tmem_ld16(acc + c, o);
          tc::tmem_ld_wait();
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) o[x] = 0u;
        }
        if (mine && PART) {
#pragma unroll
          for (int x = 0; x < 16; x += 4)
            *reinterpret_cast<uint4*>(pdst + at + c + x) =
                make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
        } else if (mine) {
          uint32_t w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x)
            w[x] = pack_bf16(__uint_as_float(o[2 * x]) * scale,
                             __uint_as_float(o[2 * x + 1]) * scale);
          *reinterpret_cast<uint4*>(dst + at + c) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(dst + at + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      if (any) {
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->acc_empty);
      }
    }
  }
  if (failed) {
    bars->abort = 1;
    atomicOr(status, tc::kStatusWaitTimeout);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// dq
// ---------------------------------------------------------------------------
struct RowItem {
  int live;
  int n;                  // key tiles
  int rows, pos, row0, pad0, head, nk;
};

struct RowBars {
  uint64_t q_full, q_empty;
  uint64_t k_full[3], k_empty[3], v_full[2], v_empty[2];
  // first_full: Q, dO and the first K and V tiles are there; ds_full: dS written, and the
  // next V tile is there; kz_full: the K tile after the next is
  uint64_t first_full, kz_full[2], s_full[2], dp_full, ds_full, acc_full, acc_empty, r_full[2];
  uint64_t i_full[kItems], i_empty[kItems];
  uint64_t mma_done;
  RowItem item[kItems];
  float2 rest[2][128];
  uint32_t tmem_base;
  int abort;
};

// Aligned by its declaration, as above.
template <int D>
constexpr size_t row_smem() {
  return size_t(7) * Cfg<D>::kTileBytes + sizeof(RowBars);
}
static_assert(kWarpgroups == 4, "sums of four warpgroups");
static_assert(row_smem<128>() <= 232448 && row_smem<64>() <= 232448, "shared memory of a CTA");

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_dq_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                   const __grid_constant__ CUtensorMap tmap_g,
                   const __grid_constant__ CUtensorMap tmap_k,
                   const __grid_constant__ CUtensorMap tmap_v, Dense P, int items,
                   const float* nl, float* dl, const float* room,
                   __nv_bfloat16* __restrict__ dq, int* __restrict__ next_item,
                   int* __restrict__ status) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (tc::smem_addr(smem) & 1023) {
    tc::griddep_wait();
    if (threadIdx.x == 0) atomicOr(status, tc::kStatusWaitTimeout);
    return;
  }
  uint8_t* qbuf = smem;
  uint8_t* gbuf = qbuf + C::kTileBytes;
  uint8_t* kbuf = gbuf + C::kTileBytes;      // [3]
  uint8_t* vbuf = kbuf + 3 * C::kTileBytes;  // [2]
  RowBars* bars = reinterpret_cast<RowBars*>(vbuf + 2 * C::kTileBytes);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->q_full, 1);
    tc::mbar_init(&bars->q_empty, 1);
    for (int s = 0; s < 3; ++s) {
      tc::mbar_init(&bars->k_full[s], 1);
      tc::mbar_init(&bars->k_empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&bars->v_full[s], 1);
      tc::mbar_init(&bars->v_empty[s], 1);
    }
    tc::mbar_init(&bars->first_full, 1);
    tc::mbar_init(&bars->kz_full[0], 1);
    tc::mbar_init(&bars->kz_full[1], 1);
    tc::mbar_init(&bars->r_full[0], 8);   // warpgroups 2 and 3
    tc::mbar_init(&bars->r_full[1], 4);   // warpgroup 1
    tc::mbar_init(&bars->s_full[0], 1);
    tc::mbar_init(&bars->s_full[1], 1);
    tc::mbar_init(&bars->dp_full, 1);
    tc::mbar_init(&bars->ds_full, 4 * kWarpgroups + 1);   // elementwise warps and warp 2
    tc::mbar_init(&bars->acc_full, 1);
    tc::mbar_init(&bars->acc_empty, 4 * kWarpgroups);
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&bars->i_full[i], 1);
      tc::mbar_init(&bars->i_empty[i], 4 * kWarpgroups + 2);
    }
    tc::mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch(&tmap_q);
    tc::tma_prefetch(&tmap_g);
    tc::tma_prefetch(&tmap_k);
    tc::tma_prefetch(&tmap_v);
  }
  if (warp == 1) tc::tmem_alloc(&bars->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  tc::griddep_wait();    // lse and delta are in place
  tc::griddep_launch();
  // S of even and of odd key tiles | dP | dQ
  const uint32_t tp = tmem + 256, tq = tmem + 384;
  bool failed = false;

  if (warp == 0) {
    // ---------------- producer ----------------
    if (lane == 0) {
      tc::ArmedRing q_armed, k_armed, v_armed;
      int ks = 0, vs = 0;
      uint32_t kp = 0, vp = 0;
      int t = blockIdx.x;  // the first item is the CTA's own
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        if (!tc::mbar_wait(&bars->i_empty[slot], ((ii / kItems) & 1) ^ 1, abort)) {
          failed = true;
          break;
        }
        RowItem it{};
        int k0 = 0;
        if (t < items) {
          int qt;
          const SeqRec s = query_tile(P, t / P.Hq, &qt);
          const int i0 = qt * kDenseTile;
          it.live = 1;
          it.rows = min(kDenseTile, s.nq - i0);
          it.pos = s.pos0 + i0;
          it.n = tiles_of(min(s.nk, it.pos + it.rows));
          it.row0 = s.q0 + i0;
          it.pad0 = s.qp0 + i0;
          it.head = t % P.Hq;
          it.nk = s.nk;
          k0 = s.k0;
        }
        bars->item[slot] = it;
        tc::mbar_arrive(&bars->i_full[slot]);
        if (!it.live) break;
        const int g = it.head / P.G;
        if (!tc::mbar_wait(&bars->q_empty, (ii & 1) ^ 1, abort)) { failed = true; break; }
        tc::mbar_arrive_expect_tx(&bars->q_full, 2 * C::kTileBytes);
        q_armed.note(0, ii & 1);
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tc::tma_load_3d(qbuf + h * C::kHalf, &tmap_q, &bars->q_full, 64 * h, it.head, it.row0);
          tc::tma_load_3d(gbuf + h * C::kHalf, &tmap_g, &bars->q_full, 64 * h, it.head, it.row0);
        }
        for (int j = 0; j < it.n && !failed; ++j) {
          if (!tc::mbar_wait(&bars->k_empty[ks], kp ^ 1, abort)) { failed = true; break; }
          tc::mbar_arrive_expect_tx(&bars->k_full[ks], C::kTileBytes);
          k_armed.note(ks, kp);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(kbuf + ks * C::kTileBytes + h * C::kHalf, &tmap_k, &bars->k_full[ks],
                            64 * h, g, k0 + j * 128);
          if (++ks == 3) { ks = 0; kp ^= 1; }
          if (!tc::mbar_wait(&bars->v_empty[vs], vp ^ 1, abort)) { failed = true; break; }
          tc::mbar_arrive_expect_tx(&bars->v_full[vs], C::kTileBytes);
          v_armed.note(vs, vp);
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(vbuf + vs * C::kTileBytes + h * C::kHalf, &tmap_v, &bars->v_full[vs],
                            64 * h, g, k0 + j * 128);
          if (++vs == 2) { vs = 0; vp ^= 1; }
        }
        t = gridDim.x + atomicAdd(next_item, 1);
      }
      if (!(q_armed.drain(&bars->q_full) && k_armed.drain(bars->k_full) &&
            v_armed.drain(bars->v_full)))
        failed = true;
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer ----------------
    if (tc::elect_one()) {
      const uint32_t qa = kmajor(qbuf), ga = kmajor(gbuf), ka = kmajor(kbuf), va = kmajor(vbuf);
      const uint32_t kb = mnmajor<D>(kbuf);
      constexpr uint32_t kTile16 = C::kTileBytes / 16;
      uint32_t n = 0, kz = 0;
      int k0 = 0, k2 = 0, vs = 0;  // K stages of dQ and of S, V stage of dP
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        if (!tc::mbar_spin(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
        const RowItem it = bars->item[slot];
        tc::mbar_arrive(&bars->i_empty[slot]);
        if (!it.live) break;
        const int last = (min(128, min(it.nk, it.pos + it.rows) - (it.n - 1) * 128) + 15) >> 4;
        if (!tc::mbar_spin(&bars->first_full, ii & 1, abort)) { failed = true; break; }
        tc::tc_fence_after();
        auto scores = [&](int j) {
          issue_nt<D>(tmem + uint32_t(j & 1) * 128, qa, ka + k2 * kTile16);
          tc::mma_commit(&bars->s_full[j & 1]);
          k2 = k2 == 2 ? 0 : k2 + 1;
        };
        auto products = [&]() {
          issue_nt<D>(tp, ga, va + vs * kTile16);
          tc::mma_commit(&bars->dp_full);
          tc::mma_commit(&bars->v_empty[vs]);
          vs ^= 1;
        };
        scores(0);
        products();
        if (it.n > 1) scores(1);
        for (int j = 0; j < it.n; ++j, ++n) {
          if (!tc::mbar_spin(&bars->ds_full, n & 1, abort)) { failed = true; break; }
          tc::tc_fence_after();
          // dP is read: the next one first, the elementwise warps want it soonest
          if (j + 1 < it.n) products();
          const uint32_t ds = tmem + uint32_t(j & 1) * 128, k = kb + k0 * kTile16;
          const int groups = j == it.n - 1 ? last : 8;
          issue_ts<D>(tq, ds, k, groups, j > 0);
          issue_ts<D>(tq, ds + 16, k, groups, 1);
          tc::mma_commit(&bars->k_empty[k0]);
          k0 = k0 == 2 ? 0 : k0 + 1;
          if (j + 2 < it.n) {
            if (!tc::mbar_spin(&bars->kz_full[kz & 1], (kz >> 1) & 1, abort)) { failed = true; break; }
            ++kz;
            tc::tc_fence_after();
            scores(j + 2);
          }
        }
        if (failed) break;
        tc::mma_commit(&bars->q_empty);
        tc::mma_commit(&bars->acc_full);
      }
      if (!tc::mma_drain(&bars->mma_done)) failed = true;
    }
  } else if (warp == 2) {
    // ---------------- what else the products need ----------------
    uint32_t n = 0, kz = 0;
    int ks = 0, vs = 0;
    uint32_t kp = 0, vp = 0;
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const RowItem it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      const int keys = min(128, min(it.nk, it.pos + it.rows) - (it.n - 1) * 128);  // last tile's
      // K tile j has landed; rows behind what is seen are zero
      auto key_tile = [&](int j) -> bool {
        if (!warp_wait(&bars->k_full[ks], kp, abort)) return false;
        if (j == it.n - 1 && (keys & 15))
          zero_rows<D>(kbuf + ks * C::kTileBytes, keys, (keys + 15) & ~15);
        if (++ks == 3) { ks = 0; kp ^= 1; }
        return true;
      };
      auto value_tile = [&]() -> bool {
        if (!warp_wait(&bars->v_full[vs], vp, abort)) return false;
        if (++vs == 2) { vs = 0; vp ^= 1; }
        return true;
      };
      if (!warp_wait(&bars->q_full, ii & 1, abort) || !key_tile(0) || !value_tile() ||
          (it.n > 1 && !key_tile(1))) {
        failed = true;
        break;
      }
      if (lane == 0) tc::mbar_arrive(&bars->first_full);
      for (int j = 0; j < it.n; ++j, ++n) {
        // the arrival belongs to this step: the step before is over
        if ((n > 0 && !warp_wait(&bars->ds_full, (n & 1) ^ 1, abort)) ||
            (j == 0 && !warp_wait(&bars->acc_empty, (ii & 1) ^ 1, abort)) ||
            (j + 1 < it.n && !value_tile())) {
          failed = true;
          break;
        }
        if (lane == 0) tc::mbar_arrive(&bars->ds_full);
        if (j + 2 < it.n) {
          if (!key_tile(j + 2)) { failed = true; break; }
          if (lane == 0) tc::mbar_arrive(&bars->kz_full[kz & 1]);
          ++kz;
        }
      }
    }
  } else if (warp >= 4) {
    // ---------------- elementwise, then a share of the tile's dQ columns ----------------
    const int wg = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = uint32_t(quarter * 32) << 16;
    const uint32_t pa = tp + lanes + wg * 32;
    const float sl2 = P.scale * kLog2e;
    const uint64_t sl2x2 = f2(sl2, sl2);
    long long n = 0;
    int sn[2] = {0, 0};  // score tiles read of each buffer
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const RowItem it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      const bool mine = row < it.rows;
      const long long at = (long long)it.head * P.rows_pad + it.pad0 + row;
      const float nlse = mine ? nl[at] : -INFINITY, ndelta = mine ? dl[at] : 0.f;
      const uint64_t nl2 = f2(nlse, nlse), nd2 = f2(ndelta, ndelta);
      uint64_t rest = 0, mass = 0;  // sums of P (dP - delta) and of P over these columns
      for (int j = 0; j < it.n; ++j, ++n) {
        const int b = j & 1;
        const uint32_t sa = tmem + b * 128 + lanes + wg * 32;
        if (!warp_wait(&bars->s_full[b], sn[b] & 1, abort)) { failed = true; break; }
        ++sn[b];
        tc::tc_fence_after();
        uint32_t p[32];
        tc::tmem_ld32(sa, p);
        tc::tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const uint64_t a = fma2(pair_of(&p[x]), sl2x2, nl2);
          exp2_pair<0>(&p[x], a, x / 2);
        }
        if (!warp_wait(&bars->dp_full, uint32_t(n & 1), abort)) { failed = true; break; }
        tc::tc_fence_after();
        uint32_t d[32];
        tc::tmem_ld32(pa, d);
        tc::tmem_ld_wait();
        const int lim = it.pos + row - j * 128 - wg * 32;  // last visible column of these 32
        const bool cut = __any_sync(MSA_FULL_MASK, lim < 31);
#pragma unroll
        for (int x = 0; x < 32; x += 2) {
          const uint64_t y = mul2(pair_of(&p[x]), add2(pair_of(&d[x]), nd2));
          d[x] = uint32_t(y);
          d[x + 1] = uint32_t(y >> 32);
        }
        if (cut) {
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (x > lim) d[x] = p[x] = 0u;
        }
        // dS as the sum of two bf16 numbers, over the scores that made it
        uint32_t hi[16], lo[16];
        uint64_t here = 0;  // P summed tile by tile: fewer roundings
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const uint64_t y = pair_of(&d[2 * x]);
          rest = add2(rest, y);
          here = add2(here, pair_of(&p[2 * x]));
          hi[x] = to_bf16x2(y);
          lo[x] = to_bf16x2(add2(y, f2(-__uint_as_float(hi[x] << 16),
                                       -__uint_as_float(hi[x] & 0xffff0000u))));
        }
        mass = add2(mass, here);
        tmem_st8(sa, hi);
        tmem_st8(sa + 8, hi + 8);
        tmem_st8(sa + 16, lo);
        tmem_st8(sa + 24, lo + 8);
        tc::tmem_st_wait();
        tc::tc_fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->ds_full);
      }
      if (failed) break;
      // delta was formed from the rounded out: P sums to 1, so what is left of the sum
      // of P (dP - delta) is what delta lacks; dk gets the better one.
      float r = lo_of(rest) + hi_of(rest), sum = lo_of(mass) + hi_of(mass);
      const float most = wg == 0 && mine ? room[at] : 0.f;  // that rounding out can take
      if (!warp_wait(&bars->acc_full, ii & 1, abort)) { failed = true; break; }
      tc::tc_fence_after();
      // Not before acc_full: it takes every warp's last dS of this item, so the previous
      // item's sums have been read.  (In an item of one key tile nothing else orders them.)
      if (wg >= 2) {
        bars->rest[wg - 2][row] = make_float2(r, sum);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->r_full[0]);
      }
      __nv_bfloat16* dst = dq + ((long long)(it.row0 + row) * P.Hq + it.head) * D + wg * (D / 4);
#pragma unroll 1
      for (int c = 0; c < D / 4; c += 16) {
        uint32_t o[16];
        __syncwarp();
        tc::tmem_ld16(tq + lanes + wg * (D / 4) + c, o);
        tc::tmem_ld_wait();
        if (mine) {
          uint32_t w[8];
#pragma unroll
          for (int x = 0; x < 8; ++x)
            w[x] = pack_bf16(__uint_as_float(o[2 * x]) * P.scale,
                             __uint_as_float(o[2 * x + 1]) * P.scale);
          *reinterpret_cast<uint4*>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
          *reinterpret_cast<uint4*>(dst + c + 8) = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->acc_empty);
      // the four sums in a fixed order: 0 + 2, 1 + 3, both
      if (wg < 2) {
        if (!warp_wait(&bars->r_full[0], ii & 1, abort)) { failed = true; break; }
        r += bars->rest[wg][row].x;
        sum += bars->rest[wg][row].y;
        if (wg == 1) {
          bars->rest[1][row] = make_float2(r, sum);
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars->r_full[1]);
        } else {
          if (!warp_wait(&bars->r_full[1], ii & 1, abort)) { failed = true; break; }
          const float2 other = bars->rest[1][row];
          // Not where more keys than this call's are in lse and out.  Units of 2^-24 that
          // a whole row's sum may be off by: the exponentials of both passes and log2 l,
          // 2^-22 each and more for a large l; the sums, 32 and 16 addends a tile and a
          // tile after another, with signs that mostly cancel; 2.8 |c lse| by the three
          // roundings between l and c lse.  A whole row that misses it keeps its delta.
          const float off = 0x1p-24f * (256.f + 4.f * fabsf(nlse));
          r += other.x;
          if (mine && fabsf(sum + other.y - 1.f) <= off && fabsf(r) <= most) dl[at] = ndelta - r;
        }
      }
    }
  }
  if (failed) {
    bars->abort = 1;
    atomicOr(status, tc::kStatusWaitTimeout);
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
cudaError_t bwd_tc(const Dense& P, const void* dout, const void* q, const void* k, const void* v,
                   const void* out, const float* lse, const DenseBwdSpace& W, void* dq, void* dk,
                   void* dv, int32_t* head, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  cudaError_t e = cudaSuccess;
  const int splits = dense_bwd_splits(P);
  const long long kelems = P.rows_k * P.Hkv * D;
  if (P.rows_q == 0) {  // no row sees anything
    e = cudaMemsetAsync(dk, 0, kelems * 2, s);
    return e == cudaSuccess ? cudaMemsetAsync(dv, 0, kelems * 2, s) : e;
  }
  static std::atomic<uint64_t> done[3];
  CUtensorMap mq, mg, mk, mv;
  e = encode_rows(&mq, q, D, P.Hq, P.rows_q);
  if (e == cudaSuccess) e = encode_rows(&mg, dout, D, P.Hq, P.rows_q);
  if (e == cudaSuccess) e = encode_rows(&mk, k, D, P.Hkv, P.rows_k);
  if (e == cudaSuccess) e = encode_rows(&mv, v, D, P.Hkv, P.rows_k);
  auto dkv = splits > 1 ? dense_dkv_tc_kernel<D, true> : dense_dkv_tc_kernel<D, false>;
  if (e == cudaSuccess) e = prepare_kernel(&done[splits > 1], dkv, key_smem<D>(), 0, kThreads);
  if (e == cudaSuccess)
    e = prepare_kernel(&done[2], dense_dq_tc_kernel<D>, row_smem<D>(), 0, kThreads);
  if (e != cudaSuccess) return e;
  const long long warps = P.rows_pad / 16 * P.Hq;
  if (P.seqs) {
    e = launch_after(dense_prep_kernel<D>, unsigned((warps + 7) / 8), 256, 0, s, P,
                     static_cast<const bf16*>(dout), static_cast<const bf16*>(out), lse, W.nl, W.dl,
                     W.room, head);
  } else {  // nothing of this call ran before: an ordinary launch
    dense_prep_kernel<D><<<unsigned((warps + 7) / 8), 256, 0, s>>>(
        P, static_cast<const bf16*>(dout), static_cast<const bf16*>(out), lse, W.nl, W.dl, W.room,
        head);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const int qitems = P.qtiles * P.Hq;
  e = launch_after(dense_dq_tc_kernel<D>, std::min(sm_count(), qitems), kThreads, row_smem<D>(), s,
                   mq, mg, mk, mv, P, qitems, W.nl, W.dl, W.room, static_cast<bf16*>(dq), head + 2,
                   head);
  if (e != cudaSuccess) return e;
  const int kitems = P.ktiles * P.Hkv * splits;
  e = launch_after(dkv, std::min(sm_count(), kitems), kThreads, key_smem<D>(), s, mq, mg, mk, mv, P,
                   splits, kitems, W.nl, W.dl, static_cast<bf16*>(dk), static_cast<bf16*>(dv),
                   W.part, head + 1, head);
  if (e != cudaSuccess) return e;
  if (splits > 1) {
    e = launch_dkv_sum(W.part, splits, kelems, P.scale, static_cast<bf16*>(dk),
                       static_cast<bf16*>(dv), s);
    if (e != cudaSuccess) return e;
  }
  return e;
}

}  // namespace

cudaError_t launch_dense_bwd_tc(const Dense& P, const void* dout, const void* q, const void* k,
                                const void* v, const void* out, const float* lse,
                                const DenseBwdSpace& W, void* dq, void* dk, void* dv,
                                int32_t* head, cudaStream_t s) {
  return (P.D == 128 ? bwd_tc<128> : bwd_tc<64>)(P, dout, q, k, v, out, lse, W, dq, dk, dv,
                                                 head, s);
}

}  // namespace msa
