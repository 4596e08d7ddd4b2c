// Dense causal attention on tcgen05 tensor cores (bf16, head_dim 64 or 128).
//
// A work item is a pair of 128-row query tiles that share a key head: two heads of
// the group at the same query tile (their keys are loaded once and both tiles see
// the same number of them), or, where the group has an odd number of heads, two
// neighbours in the list of (query tile, head).  Persistent CTAs, one per SM, take
// items from a counter in the workspace, heaviest first.  Per key tile of 128 keys
// and per query tile, with the running maximum m and sum l of the softmax held by
// the thread that owns the row:
//   S = Q K^T          (both K-major in shared memory, fp32 in TMEM, a row per lane)
//   P = 2^(c S - c m)  (c = scale log2 e; bf16, written over S in TMEM), l += sum P
//   O += P V           (P from TMEM, V as an MN-major shared-memory operand)
// m moves only when a row's maximum has grown by more than 2^kSlack: O, kept in
// TMEM, is then scaled by the softmax warps; otherwise P just exceeds 1, which fp32
// sums and a bf16 P carry with the same relative error.  P as one bf16 number is what the
// MMAs take at their full rate (two would add half to their cycles): out is 0.0020 to 0.0023
// of its 2-norm from 64 bits, of which its own rounding is 0.0016.  l sums P unrounded.
//
// Each tile of the pair has its own TMEM columns (S|P 128, O) and softmax warpgroup;
// one thread issues the MMAs of both in turn, so one tile's MMAs run while the other is
// in its softmax.  A fourth warpgroup normalises and stores the finished tiles.  A stage
// of the TMA ring is a V tile and the K tile after it, in the order of use.
//
// What bounds it: a step (one key tile, both query tiles) has 2048 cycles of MMA and as
// many of the exp2 unit, and takes ~3050: from S to P a tile's softmax takes ~1800 cycles
// (exponentials 1024 at the unit's rate), P to the MMA thread ~250, the rest of P V and
// the next S ~640, S to the softmax ~170.  8192 rows x 64 heads x 128: 0.89 ms, 1235
// TFLOP/s (the tensor pipe 53 % busy); 512 rows at the end of 8000 tokens 0.134 ms, 970
// TFLOP/s.  What brought it there: MMAs issued under elect.sync, so that their operands
// stay in uniform registers (1.14 -> 0.92 ms: under `lane == 0` every MMA first moved
// them there); the fixed order of one issuing thread (1.57 -> 1.25 ms against a thread
// per tile, whose products interleaved so that both tiles were in their softmax at the
// same time); all other waits in a second warp (1.25 -> 1.19 ms).
//
// Tokens behind the last key of a sequence (the next sequence's, or an unused part
// of a page) come in with its last tile.  Their scores are cut by the causal mask;
// their V rows must not meet a weight of zero as infinities or NaN, so P V runs over
// whole groups of 16 keys only as far as keys exist, and the rest of the last group
// is zeroed in shared memory first.
#include <algorithm>

#include "dense_tc.cuh"

namespace msa {
namespace {

// warp 0 items and TMA, warp 1 MMA, warp 2 waits for it, warp 3 idle, warps 4-11 softmax, 12-15 epilogue
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;
constexpr int kItems = 3;     // items in flight
constexpr float kSlack = 8.f;
constexpr int kFirst = 6;   // groups of 16 keys of P that P V starts on (1-2 % over 4)
// 96 + 64 + 2 x 176 = 512 = 4 x 128: the registers the CTA is launched with
constexpr int kRegsCtl = 96, kRegsEpi = 64, kRegsSoftmax = 176;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kHalf = 128 * 64 * 2;            // 64 dims of 128 rows
  static constexpr int kPairs = D == 128 ? 2 : 4;       // stages of a V and a K tile
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, 128, 0, 0);
  static constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, D, 0, 1);  // V is MN-major
};

struct Item {
  int live;               // 0: no more items
  int n;                  // key tiles to pass through (the larger of nkt)
  int nkt[2];             // key tiles of each query tile; 0: no such tile
  int rows[2];            // its rows
  int pos[2];             // position of its first row
  int head[2];
  int row0[2];            // its first row in q
  int nk;                 // keys of the sequence
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k0_full;                     // the CTA's first K tile
  uint64_t vk_full[4], vk_empty[4];     // a V tile and the K tile after it
  // per query tile: S computed, the first kFirst groups of P written (and what else its
  // products need is there), all of P written, the tile's last P V done, O read by the
  // epilogue, sums written, sums read
  uint64_t s_full[2], p_half[2], p_full[2], o_done[2], o_empty[2], l_full[2], l_empty[2];
  uint64_t i_full[kItems], i_empty[kItems];
  uint64_t mma_done;
  Item item[kItems];
  float l[2][128];        // sums of the rows, softmax -> epilogue
  uint32_t tmem_base;
  int abort;
};

template <int D>
constexpr size_t smem_bytes() {
  return 1024 + size_t(3 + 2 * Cfg<D>::kPairs) * Cfg<D>::kTileBytes + sizeof(Bars) + 64;
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory of a CTA");

// Item t of the launch; b and k0 locate its keys (b: batch index for a block table).
__device__ __forceinline__ void make_item(const Dense& P, int t, Item* it, int* b, int* k0, int* g) {
  SeqRec s;
  int p;
  if (P.seqs) {
    s = P.seqs[find_seq<&SeqRec::pr0>(P.seqs, P.B, t)];
    p = (t - s.pr0) / P.Hkv;
    *g = (t - s.pr0) % P.Hkv;
    *b = 0;
  } else {
    p = t / (P.B * P.Hkv);
    *b = (t / P.Hkv) % P.B;
    *g = t % P.Hkv;
    s = batch_seq(P, *b);
  }
  *k0 = s.k0;
  const int nqt = tiles_of(s.nq);
  it->live = 1;
  it->nk = s.nk;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int x = 2 * p + e;
    const bool there = x < nqt * P.G;
    const int i0 = (nqt - 1 - (there ? x / P.G : 0)) * kDenseTile;  // last tiles first
    it->rows[e] = there ? min(kDenseTile, s.nq - i0) : 0;
    it->pos[e] = s.pos0 + i0;
    it->head[e] = *g * P.G + (there ? x % P.G : 0);
    it->row0[e] = s.q0 + i0;
    it->nkt[e] = there ? tiles_of(min(s.nk, s.pos0 + i0 + it->rows[e])) : 0;
  }
  it->n = max(it->nkt[0], it->nkt[1]);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
dense_fwd_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
                    const __grid_constant__ CUtensorMap tmap_k,
                    const __grid_constant__ CUtensorMap tmap_v,
                    const __grid_constant__ CUtensorMap tmap_o, Dense P,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse,
                    int* __restrict__ next_item, int* __restrict__ status) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = smem;                          // [2]
  uint8_t* k0buf = qbuf + 2 * C::kTileBytes;
  uint8_t* vkbuf = k0buf + C::kTileBytes;        // [pairs][V, K]
  Bars* bars = reinterpret_cast<Bars*>(vkbuf + C::kPairs * 2 * C::kTileBytes);
  volatile int* abort = &bars->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bars->k0_full, 1);
    for (int s = 0; s < C::kPairs; ++s) {
      tc::mbar_init(&bars->vk_full[s], 1);
      tc::mbar_init(&bars->vk_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&bars->q_full[b], 1);
      tc::mbar_init(&bars->q_empty[b], 1);
      tc::mbar_init(&bars->s_full[b], 1);
      tc::mbar_init(&bars->p_half[b], 5);    // the tile's softmax warps and warp 2
      tc::mbar_init(&bars->p_full[b], 4);
      tc::mbar_init(&bars->o_done[b], 1);
      tc::mbar_init(&bars->o_empty[b], 4);   // the epilogue warps
      tc::mbar_init(&bars->l_full[b], 4);
      tc::mbar_init(&bars->l_empty[b], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&bars->i_full[i], 1);
      tc::mbar_init(&bars->i_empty[i], 14);  // warps 1, 2, softmax, epilogue
    }
    tc::mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch(&tmap_q);
    tc::tma_prefetch(&tmap_k);
    tc::tma_prefetch(&tmap_v);
    tc::tma_prefetch(&tmap_o);
  }
  if (warp == 1) tc::tmem_alloc(&bars->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  tc::griddep_wait();  // the records and the counter are written
  bool failed = false;

  if (warp < 4) {
    regs_dec<kRegsCtl>();
    if (warp == 0) {
      // ---------------- producer: items and TMA ----------------
      if (lane == 0) {
        tc::ArmedRing q_armed, vk_armed;
        bool k0_armed = false;
        int stage = 0, qn[2] = {0, 0};
        uint32_t phase = 0;
        struct Where {
          int live, n, b, k0, g;
          int nkt[2], head[2], row0[2];
        } cur, nxt;
        // The first item is the CTA's own, the others are taken late, two key tiles before
        // the copies need them, so that no CTA holds an item while another has none.
        int ii = 0, ticket = blockIdx.x;  // items, the next one's number
        // the next item to the other warps, and what the copies need of it
        auto publish = [&](Where* w) -> bool {
          const int slot = ii % kItems, t = ticket;
          if (!tc::mbar_wait(&bars->i_empty[slot], ((ii / kItems) & 1) ^ 1, abort)) return false;
          ++ii;
          Item& it = bars->item[slot];
          w->live = t < P.pairs;
          it.live = w->live;
          if (w->live) {
            make_item(P, t, &it, &w->b, &w->k0, &w->g);
            w->n = it.n;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              w->nkt[e] = it.nkt[e];
              w->head[e] = it.head[e];
              w->row0[e] = it.row0[e];
            }
          }
          tc::mbar_arrive(&bars->i_full[slot]);
          return true;
        };
        auto copy = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, const Where& w, int j) {
          const int row = int(tile_row(P, w.b, w.k0, j));
#pragma unroll
          for (int h = 0; h < D / 64; ++h)
            tc::tma_load_3d(dst + h * C::kHalf, map, bar, 64 * h, w.g, row);
        };
        failed = !publish(&cur);
        bool start = true;
        while (!failed && cur.live) {
          if (start) {
            tc::mbar_arrive_expect_tx(&bars->k0_full, C::kTileBytes);
            k0_armed = true;
            copy(&tmap_k, k0buf, &bars->k0_full, cur, 0);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (cur.nkt[e] == 0 || failed) continue;
            if (!tc::mbar_wait(&bars->q_empty[e], (qn[e] & 1) ^ 1, abort)) { failed = true; continue; }
            tc::mbar_arrive_expect_tx(&bars->q_full[e], C::kTileBytes);
            q_armed.note(e, qn[e] & 1);
            ++qn[e];
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_load_3d(qbuf + e * C::kTileBytes + h * C::kHalf, &tmap_q, &bars->q_full[e],
                              64 * h, cur.head[e], cur.row0[e]);
          }
          start = false;
          for (int j = 0; j < cur.n && !failed; ++j) {
            if (j == max(cur.n - 3, 0)) ticket = gridDim.x + atomicAdd(next_item, 1);
            if (j == cur.n - 1 && !publish(&nxt)) { failed = true; break; }
            if (!tc::mbar_wait(&bars->vk_empty[stage], phase ^ 1, abort)) { failed = true; break; }
            const bool more = j + 1 < cur.n || nxt.live;
            uint64_t* fb = &bars->vk_full[stage];
            uint8_t* dst = vkbuf + stage * 2 * C::kTileBytes;
            tc::mbar_arrive_expect_tx(fb, (more ? 2 : 1) * C::kTileBytes);
            vk_armed.note(stage, phase);
            copy(&tmap_v, dst, fb, cur, j);
            if (more)
              copy(&tmap_k, dst + C::kTileBytes, fb, j + 1 < cur.n ? cur : nxt,
                   j + 1 < cur.n ? j + 1 : 0);
            if (++stage == C::kPairs) { stage = 0; phase ^= 1; }
          }
          cur = nxt;
        }
        // every copy issued has landed before the CTA can leave
        if (k0_armed && !tc::mbar_drain(&bars->k0_full, 0)) failed = true;
        if (!(q_armed.drain(bars->q_full) && vk_armed.drain(bars->vk_full))) failed = true;
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      // In the fixed order P V of tile 0, its next S, P V of tile 1, its next S (the next
      // item's first S at an item's end): the two tiles stay half a step apart, each in
      // its softmax while the other's products run.  The pipe queues few instructions, so
      // whatever this thread waits for or does between them shows: it waits for P alone
      // (its first keys, then the others), to whose first barrier warp 2 adds its arrival
      // once all else that the products need is there.
      if (tc::elect_one()) {
        int ii = 0, ps = 0;                  // items, stage
        uint32_t pp = 0, qpar = 0, ppar = 0; // parities: stage; per query tile Q and P (bit e)
        // low words of the descriptors; steps of 16 columns or rows are added to them
        const uint32_t qd = uint32_t(tc::sdesc_sw128(tc::smem_addr(qbuf), 16, 1024));
        const uint32_t k0d = uint32_t(tc::sdesc_sw128(tc::smem_addr(k0buf), 16, 1024));
        const uint32_t kd = uint32_t(tc::sdesc_sw128(tc::smem_addr(vkbuf + C::kTileBytes), 16, 1024));
        const uint32_t vd = uint32_t(tc::sdesc_sw128(tc::smem_addr(vkbuf), C::kHalf, 1024));
        constexpr uint32_t kHi = uint32_t(tc::kDescHi | (1024 >> 4));
        constexpr uint32_t kTile16 = C::kTileBytes / 16, kHalf16 = C::kHalf / 16;
        auto fetch = [&](Item* it) -> bool {
          const int slot = ii % kItems;
          if (!tc::mbar_spin(&bars->i_full[slot], (ii++ / kItems) & 1, abort)) return false;
          *it = bars->item[slot];
          tc::mbar_arrive(&bars->i_empty[slot]);
          return true;
        };
        // S of query tile e
        auto scores = [&](int e, uint32_t b, bool last) {
          const uint32_t st = tmem + e * 256;
          const uint32_t a = qd + e * kTile16;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
            tc::mma_ss_lo(st, a + off, b + off, kHi, C::kIdescS, kk > 0 ? 1u : 0u);
          }
          tc::mma_commit(&bars->s_full[e]);
          if (last) tc::mma_commit(&bars->q_empty[e]);
        };
        Item cur{};
        failed = !fetch(&cur);
        if (!failed && cur.live) {
          failed = !tc::mbar_spin(&bars->k0_full, 0, abort);
#pragma unroll 1
          for (int e = 0; e < 2; ++e) {
            const int nkt = e ? cur.nkt[1] : cur.nkt[0];
            if (nkt == 0 || failed) continue;
            failed = !tc::mbar_spin(&bars->q_full[e], 0, abort);
            qpar ^= 1u << e;
            tc::tc_fence_after();
            if (!failed) scores(e, k0d, nkt == 1);
          }
        }
        while (!failed && cur.live) {
          const int nkt0 = cur.nkt[0], nkt1 = cur.nkt[1], n = cur.n;
          const int seen0 = min(cur.nk, cur.pos[0] + cur.rows[0]);
          const int seen1 = min(cur.nk, cur.pos[1] + cur.rows[1]);
          int j = 0;
          // Steps in which both tiles have whole key tiles left run without a decision on
          // the way: the general form below takes hundreds of cycles more.
          for (const int fast = min(nkt0, nkt1) - 1; j < fast && (ppar == 0 || ppar == 3); ++j) {
            const uint32_t par = ppar & 1;
            const uint32_t v = vd + ps * 2 * kTile16, k = kd + ps * 2 * kTile16;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t st = tmem + e * 256, q = qd + e * kTile16;
              if (!tc::mbar_spin(&bars->p_half[e], par, abort)) { failed = true; break; }
              tc::tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kFirst; ++kk)
                tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO,
                              kk > 0 ? 1u : uint32_t(j));
              if (!tc::mbar_spin(&bars->p_full[e], par, abort)) { failed = true; break; }
              tc::tc_fence_after();
#pragma unroll
              for (int kk = kFirst; kk < 8; ++kk)
                tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO, 1u);
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
                tc::mma_ss_lo(st, q + off, k + off, kHi, C::kIdescS, kk > 0 ? 1u : 0u);
              }
              tc::mma_commit(&bars->s_full[e]);
            }
            if (failed) break;
            tc::mma_commit(&bars->vk_empty[ps]);
            ppar ^= 3;
            if (++ps == C::kPairs) { ps = 0; pp ^= 1; }
            if (j + 2 == nkt0) tc::mma_commit(&bars->q_empty[0]);
            if (j + 2 == nkt1) tc::mma_commit(&bars->q_empty[1]);
          }
          for (; j < n && !failed; ++j) {
            const bool end = j == n - 1;
            if (end && !fetch(&cur)) { failed = true; break; }
#pragma unroll 1
            for (int e = 0; e < 2; ++e) {
              const uint32_t st = tmem + e * 256;
              const int nkt = e ? nkt1 : nkt0;
              const int left = !end ? nkt - j - 1 : cur.live ? (e ? cur.nkt[1] : cur.nkt[0]) : 0;
              if (j < nkt) {
                // the first keys' products run while the softmax finishes the others
                const int groups = (min(128, (e ? seen1 : seen0) - j * 128) + 15) >> 4;
                const uint32_t v = vd + ps * 2 * kTile16;
                if (!tc::mbar_spin(&bars->p_half[e], (ppar >> e) & 1, abort)) { failed = true; break; }
                tc::tc_fence_after();
                if (groups >= kFirst) {
#pragma unroll
                  for (int kk = 0; kk < kFirst; ++kk)
                    tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO,
                                  kk > 0 ? 1u : uint32_t(j));
                } else {
#pragma unroll 1
                  for (int kk = 0; kk < groups; ++kk)
                    tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO,
                                  uint32_t(kk + j));
                }
                if (!tc::mbar_spin(&bars->p_full[e], (ppar >> e) & 1, abort)) { failed = true; break; }
                ppar ^= 1u << e;
                tc::tc_fence_after();
                if (groups == 8) {
#pragma unroll
                  for (int kk = kFirst; kk < 8; ++kk)
                    tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO, 1u);
                } else {
#pragma unroll 1
                  for (int kk = kFirst; kk < groups; ++kk)
                    tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO, 1u);
                }
                if (j == nkt - 1) tc::mma_commit(&bars->o_done[e]);
              } else if (left > 0) {  // only scores: this tile's products were shorter
                if (!tc::mbar_spin(&bars->vk_full[ps], pp, abort) ||
                    !tc::mbar_spin(&bars->q_full[e], (qpar >> e) & 1, abort)) {
                  failed = true;
                  break;
                }
                tc::tc_fence_after();
              }
              if (left > 0) {
                if (end) qpar ^= 1u << e;
                scores(e, kd + ps * 2 * kTile16, left == 1);
              }
            }
            tc::mma_commit(&bars->vk_empty[ps]);
            if (++ps == C::kPairs) { ps = 0; pp ^= 1; }
          }
        }
        // every MMA issued has completed before TMEM is freed
        if (!tc::mma_drain(&bars->mma_done)) failed = true;
      }
    } else if (warp == 2) {
      // ---------------- what else the products need ----------------
      // Per key tile and query tile, one arrival at p_half: the V tile and the K tile
      // after it have landed (V's rows behind the last key zeroed), the epilogue has read
      // the previous O, the next item's Q has landed.
      int ii = 0, ps = 0;
      uint32_t pp = 0;
      uint32_t qn[2] = {0, 0}, on[2] = {0, 0}, in[2] = {0, 0};  // Q tiles, key tiles, items
      auto fetch = [&](Item* it) -> bool {
        const int slot = ii % kItems;
        if (!warp_wait(&bars->i_full[slot], (ii++ / kItems) & 1, abort)) return false;
        *it = bars->item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
        return true;
      };
      Item cur{}, nxt{};
      failed = !fetch(&cur);
#pragma unroll
      for (int e = 0; e < 2; ++e) qn[e] = !failed && cur.live && cur.nkt[e] > 0;
      while (!failed && cur.live) {
        int all = 0;  // keys that some row of the item sees
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (cur.nkt[e] > 0) all = max(all, min(cur.nk, cur.pos[e] + cur.rows[e]));
        for (int j = 0; j < cur.n && !failed; ++j) {
          const bool end = j == cur.n - 1;
          if (end && !fetch(&nxt)) { failed = true; break; }
          if (!warp_wait(&bars->vk_full[ps], pp, abort)) { failed = true; break; }
          const int keys = min(128, all - j * 128);
          if (keys & 15) zero_rows<D>(vkbuf + ps * 2 * C::kTileBytes, keys, (keys + 15) & ~15);
          if (++ps == C::kPairs) { ps = 0; pp ^= 1; }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const bool follow = end && nxt.live && nxt.nkt[e] > 0;
            if (j < cur.nkt[e] && !failed) {
              // the arrival belongs to the phase of this key tile: the one before is over
              if ((on[e] > 0 && !warp_wait(&bars->p_half[e], (on[e] & 1) ^ 1, abort)) ||
                  (j == 0 && !warp_wait(&bars->o_empty[e], (in[e]++ & 1) ^ 1, abort)) ||
                  (follow && !warp_wait(&bars->q_full[e], qn[e] & 1, abort))) {
                failed = true;
                break;
              }
              ++on[e];
              if (lane == 0) tc::mbar_arrive(&bars->p_half[e]);
            }
            if (follow) ++qn[e];
          }
        }
        cur = nxt;
      }
    }
  } else if (warp < 12) {
    // ---------------- softmax of query tile e ----------------
    regs_inc<kRegsSoftmax>();
    const int e = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t st = tmem + (uint32_t(quarter * 32) << 16) + e * 256, ot = st + 128;
    const float sl2 = P.scale * kLog2e;
    const uint64_t sl2x2 = f2(sl2, sl2);
    int qn = 0, on = 0;
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const Item& it = bars->item[slot];
      const int live = it.live, nkt = it.nkt[e];
      // last key that the row sees (rows behind the tile's last one: its last)
      const int last = it.pos[e] + min(row, it.rows[e] - 1);
      const long long lse_at =
          lse && row < it.rows[e] ? (long long)(it.row0[e] + row) * P.Hq + it.head[e] : -1;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!live) break;
      if (nkt == 0) continue;
      float m = -INFINITY, ms = 0.f, l = 0.f;  // running maximum, c m, sum
      for (int j = 0; j < nkt; ++j, ++on) {
        if (!warp_wait(&bars->s_full[e], on & 1, abort)) { failed = true; break; }
        tc::tc_fence_after();
        uint32_t v[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) tc::tmem_ld32(st + q4 * 32, v[q4]);
        tc::tmem_ld_wait();
        const int lim = last - j * 128;  // last visible column
        if (!__all_sync(MSA_FULL_MASK, lim >= 127)) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (q4 * 32 + x > lim) v[q4][x] = __float_as_uint(-INFINITY);
        }
        float top = max32(v[0], -INFINITY);
        top = fmaxf(fmaxf(top, max32(v[1], -INFINITY)), fmaxf(max32(v[2], -INFINITY),
                                                             max32(v[3], -INFINITY)));
        // the first tile sets the maximum; later ones move it only past the slack
        const bool grow = j == 0 || (top - m) * sl2 > kSlack;
        float keep = 1.f;
        if (grow) {
          const float nms = top == -INFINITY ? 0.f : top * sl2;
          keep = m == -INFINITY ? 0.f : ex2_f32(ms - nms);
          m = top;
          ms = nms;
        }
        if (j > 0 && __any_sync(MSA_FULL_MASK, grow)) {
          // the previous P V was issued before this S: O is there; scale it
          const uint64_t k2 = f2(keep, keep);
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            tc::tmem_ld16(ot + c, o);
            tc::tmem_ld_wait();
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const uint64_t y = mul2((uint64_t(o[x + 1]) << 32) | o[x], k2);
              o[x] = uint32_t(y);
              o[x + 1] = uint32_t(y >> 32);
            }
            tmem_st8(ot + c, o);
            tmem_st8(ot + c + 8, o + 8);
          }
        }
        const uint64_t nmsx2 = f2(-ms, -ms);
        uint64_t lsum[2] = {0, 0};
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
#pragma unroll
          for (int x8 = 0; x8 < 2; ++x8) {
            uint32_t pw[8];
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const uint32_t* s2 = v[q4] + x8 * 16 + x;
              const uint64_t z = fma2((uint64_t(s2[1]) << 32) | s2[0], sl2x2, nmsx2);
              const float pa = ex2_f32(__uint_as_float(uint32_t(z)));
              const float pb = ex2_f32(__uint_as_float(uint32_t(z >> 32)));
              lsum[(x >> 1) & 1] = add2(lsum[(x >> 1) & 1], f2(pa, pb));
              pw[x >> 1] = pack_bf16(pa, pb);
            }
            tmem_st8(st + q4 * 16 + x8 * 8, pw);
          }
          if (q4 == kFirst / 2 - 1 || q4 == 3) {
            tc::tmem_st_wait();
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(q4 < 3 ? &bars->p_half[e] : &bars->p_full[e]);
          }
        }
        const uint64_t lsx = add2(lsum[0], lsum[1]);
        l = l * keep + (__uint_as_float(uint32_t(lsx)) + __uint_as_float(uint32_t(lsx >> 32)));
      }
      if (failed || !warp_wait(&bars->l_empty[e], (qn & 1) ^ 1, abort)) { failed = true; break; }
      bars->l[e][row] = l;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->l_full[e]);
      if (lse_at >= 0) lse[lse_at] = (ms + log2f(l)) * kLn2;
      ++qn;
    }
  } else {
    // ---------------- epilogue of both query tiles ----------------
    regs_dec<kRegsEpi>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    uint8_t* wst = k0buf + quarter * (32 * D * 2);  // free once the first item's scores are done
    int qn[2] = {0, 0};
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const Item& it = bars->item[slot];
      const int live = it.live;
      int nkt[2], rows[2], head[2], row0[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        nkt[e] = it.nkt[e];
        rows[e] = it.rows[e];
        head[e] = it.head[e];
        row0[e] = it.row0[e];
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!live) break;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (nkt[e] == 0 || failed) continue;
        const uint32_t par = qn[e] & 1;
        ++qn[e];
        if (!warp_wait(&bars->l_full[e], par, abort)) { failed = true; continue; }
        const float inv = 1.f / bars->l[e][row];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->l_empty[e]);
        if (!warp_wait(&bars->o_done[e], par, abort)) { failed = true; continue; }
        tc::tc_fence_after();
        const uint32_t ot = tmem + (uint32_t(quarter * 32) << 16) + e * 256 + 128;
        // Each warp owns 32 rows and stores them itself with TMA, from a staging area in
        // the 128-byte swizzle (16-byte chunk k of a row at chunk k ^ (row % 8)); plain
        // 16-byte stores of a row per thread kept the softmax warps' TMEM accesses waiting
        // behind them.
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        const uint64_t inv2 = f2(inv, inv);
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          __syncwarp();
          tc::tmem_ld32(ot + c * 32, o);
          tc::tmem_ld_wait();
          if (c == D / 32 - 1) {
            tc::tc_fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars->o_empty[e]);
          }
          uint8_t* hp = wst + (c >> 1) * 4096 + lane * 128;
#pragma unroll
          for (int k8 = 0; k8 < 4; ++k8) {
            const uint32_t* w8 = o + 8 * k8;
            uint4 u;
            u.x = to_bf16x2(mul2((uint64_t(w8[1]) << 32) | w8[0], inv2));
            u.y = to_bf16x2(mul2((uint64_t(w8[3]) << 32) | w8[2], inv2));
            u.z = to_bf16x2(mul2((uint64_t(w8[5]) << 32) | w8[4], inv2));
            u.w = to_bf16x2(mul2((uint64_t(w8[7]) << 32) | w8[6], inv2));
            *reinterpret_cast<uint4*>(hp + ((((c & 1) * 4 + k8) ^ (lane & 7)) << 4)) = u;
          }
        }
        const int left = rows[e] - quarter * 32;  // rows of the warp that exist
        if (left >= 32) {
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_store_3d(&tmap_o, wst + h * 4096, 64 * h, head[e], row0[e] + quarter * 32);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else {
          __syncwarp();
          constexpr int per = D / 8;
          for (int i = lane; i < left * per; i += 32) {
            const int r = i / per, c = i % per;
            const uint4 u = *reinterpret_cast<const uint4*>(wst + (c >> 3) * 4096 + r * 128 +
                                                            (((c & 7) ^ (r & 7)) << 4));
            *reinterpret_cast<uint4*>(
                out + ((long long)(row0[e] + quarter * 32 + r) * P.Hq + head[e]) * D + c * 8) = u;
          }
          __syncwarp();
        }
      }
    }
    // every store has completed before the CTA exits
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
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
cudaError_t fwd_tc(const Dense& P, const void* q, const void* k, const void* v, void* out,
                   float* lse, int32_t* counter, int32_t* status, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap mq, mk, mv, mo;
  cudaError_t e = encode_rows(&mq, q, D, P.Hq, P.rows_q);
  if (e == cudaSuccess) e = encode_rows(&mo, out, D, P.Hq, P.rows_q, 32);
  if (e == cudaSuccess) e = encode_rows(&mk, k, D, P.Hkv, P.rows_k);
  if (e == cudaSuccess) e = encode_rows(&mv, v, D, P.Hkv, P.rows_k);
  if (e == cudaSuccess)
    e = prepare_kernel(&done, dense_fwd_tc_kernel<D>, smem_bytes<D>(),
                       kRegsCtl + kRegsEpi + 2 * kRegsSoftmax, kThreads);
  if (e != cudaSuccess) return e;
  return launch_after(dense_fwd_tc_kernel<D>, std::min(sm_count(), P.pairs), kThreads,
                      smem_bytes<D>(), s, mq, mk, mv, mo, P, static_cast<__nv_bfloat16*>(out), lse,
                      counter, status);
}

}  // namespace

cudaError_t launch_dense_fwd_tc(const Dense& P, const void* q, const void* k, const void* v,
                                void* out, float* lse, int32_t* counter, int32_t* status,
                                cudaStream_t s) {
  return (P.D == 128 ? fwd_tc<128> : fwd_tc<64>)(P, q, k, v, out, lse, counter, status, s);
}

}  // namespace msa
