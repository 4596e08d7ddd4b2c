// Attention of drafted tokens over a KV cache on tcgen05 tensor cores (bf16, head_dim
// 64 or 128), a single drafted token being a decoding step.
//
// The cache is read once per group of 128 (node, head) rows of a key head and that
// reading is the bound: 64 KB per key tile of 128 against 1024 cycles of MMA.  The key
// tiles of all units (sequence, key head, row group) form one list that is cut into
// equal shares, one per CTA, so that every SM streams the same amount whatever the
// lengths; a unit that a share's border cuts leaves partial states for a second, small
// launch to join.
//
// Inside a CTA the even and the odd key tiles of a piece are two independent chains,
// each with its own softmax warpgroup, running maximum and sum, and accumulator O, so that
// one chain's MMAs and copies run under the other's softmax; the epilogue joins the two.
// Scores, probabilities (bf16 for P V: out is 0.0023 of its 2-norm from 64 bits, 0.0017 by
// its own rounding) and the moving maximum are as in the forward pass over whole prompts.
// K and V tiles come through a ring of TMA stages (160 KB); Q comes a piece ahead.
//
// 8 drafted tokens each over four contexts of 128K (1.07 GB): 178 us, 6.0 TB/s, nearly the
// rate of a copy; 32 sequences of 2000 to 6000 tokens, one token each: 56 us, 4.7 TB/s (the
// first tiles' latency and the border pieces weigh more).  The order of use in the ring took
// the former from 222 us: with K and V of a tile requested together the V tiles held three
// of the five stages through the softmax.
//
// Which drafted tokens a node sees comes as one bit mask per node, and which are seen
// at all as one per sequence, formed by a small launch before.  V rows of unseen tokens
// are zeroed in shared memory, for they may hold anything.
#include <algorithm>

#include "dense_tc.cuh"

namespace msa {
namespace {

// warp 0 pieces and TMA, warp 1 MMA, warp 2 waits for it, warp 3 Q rows, warps 4-11 softmax, 12-15 epilogue
constexpr int kThreads = 512;
constexpr uint32_t kTmemCols = 512;
constexpr int kItems = 2;
constexpr float kSlack = 8.f;
constexpr int kRegsCtl = 96, kRegsEpi = 64, kRegsSoftmax = 176;

template <int D>
struct Cfg {
  static constexpr int kTileBytes = 128 * D * 2;
  static constexpr int kHalf = 128 * 64 * 2;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kIdescS = tc::idesc_bf16_f32(128, 128, 0, 0);
  static constexpr uint32_t kIdescO = tc::idesc_bf16_f32(128, D, 0, 1);
};

struct Item {
  int live;
  int b, g, row0, rows;   // sequence, key head, first (node, head) row, rows
  int kt0, n;             // first key tile, key tiles
  int len;                // cached tokens
  int slot;
};

struct Bars {
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[8], kv_empty[8];
  // first_full: the CTA's first Q and K tiles are there; per chain: S computed, P written
  // (and what its products need is there), the piece's last P V done, O read, (maximum,
  // sum) written, read
  uint64_t first_full, s_full[2], p_full[2], o_done[2], o_empty[2], l_full[2], l_empty[2];
  uint64_t i_full[kItems], i_empty[kItems];
  uint64_t mma_done;
  Item item[kItems];
  uint32_t tmem_base;
  int abort;
  float2 ml[2][128];
};

// The dynamic part starts on a 1024-byte boundary, there is no room to align it by hand
// (the kernel looks, and refuses to run otherwise).
template <int D>
constexpr size_t smem_bytes() {
  return size_t(2 + Cfg<D>::kStages) * Cfg<D>::kTileBytes + sizeof(Bars);
}
static_assert(smem_bytes<128>() <= 232448 && smem_bytes<64>() <= 232448, "shared memory of a CTA");

// Bits of the drafted tokens that each node sees, [masks][nodes + 1], the last of a
// sequence those that any node sees; clears the status word.
__global__ void __launch_bounds__(256)
tree_prep_kernel(const uint8_t* __restrict__ mask, long long stride, int nodes,
                 uint4* __restrict__ bits, int32_t* __restrict__ status) {
  __shared__ uint32_t any[4];
  tc::griddep_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
  if (threadIdx.x < 4) any[threadIdx.x] = 0;
  __syncthreads();
  mask += blockIdx.x * stride;
  bits += (long long)blockIdx.x * (nodes + 1);
  uint32_t mine[4] = {};
#pragma unroll 4
  for (int i = warp; i < nodes; i += 8) {
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int j = 32 * x + lane;
      w[x] = __ballot_sync(MSA_FULL_MASK, j < nodes && mask[i * nodes + j] != 0);
      mine[x] |= w[x];
    }
    if (lane == 0) bits[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (lane < 4) atomicOr(&any[lane], lane == 0 ? mine[0] : lane == 1 ? mine[1]
                                     : lane == 2 ? mine[2] : mine[3]);
  __syncthreads();
  if (threadIdx.x == 0) bits[nodes] = make_uint4(any[0], any[1], any[2], any[3]);
}

// 32 bits from position pos of: ones below 0, the 128 bits of m, zeros above.
__device__ __forceinline__ uint32_t bits_at(const uint4& m, int pos) {
  auto word = [&](int i) {
    return i < 0 ? 0xffffffffu : i == 0 ? m.x : i == 1 ? m.y : i == 2 ? m.z : i == 3 ? m.w : 0u;
  };
  const int w = pos >> 5;
  return __funnelshift_r(word(w), word(w + 1), pos & 31);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap tmap_q,
               const __grid_constant__ CUtensorMap tmap_k,
               const __grid_constant__ CUtensorMap tmap_v, Tree A,
               const __nv_bfloat16* __restrict__ q, __nv_bfloat16* __restrict__ out,
               float* __restrict__ lse, int* __restrict__ status) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const Dense& P = A.d;
  uint8_t* qbuf = smem;                          // [2]
  uint8_t* kvbuf = qbuf + 2 * C::kTileBytes;     // [stages], K and V tiles in turn
  Bars* bars = reinterpret_cast<Bars*>(kvbuf + C::kStages * C::kTileBytes);
  volatile int* abort = &bars->abort;
  const int nodes = P.Sq;

  if (tc::smem_addr(smem) & 1023) {
    tc::griddep_wait();
    if (threadIdx.x == 0) atomicOr(status, tc::kStatusWaitTimeout);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      tc::mbar_init(&bars->kv_full[s], 1);
      tc::mbar_init(&bars->kv_empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init(&bars->q_full[b], 1);
      tc::mbar_init(&bars->q_empty[b], 1);
      tc::mbar_init(&bars->s_full[b], 1);
      tc::mbar_init(&bars->p_full[b], 5);    // the chain's softmax warps and warp 2
      tc::mbar_init(&bars->o_done[b], 1);
      tc::mbar_init(&bars->o_empty[b], 4);
      tc::mbar_init(&bars->l_full[b], 4);
      tc::mbar_init(&bars->l_empty[b], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&bars->i_full[i], 1);
      tc::mbar_init(&bars->i_empty[i], 15);  // warps 1-3, 8 softmax, 4 epilogue warps
    }
    tc::mbar_init(&bars->first_full, 1);
    tc::mbar_init(&bars->mma_done, 1);
    bars->abort = 0;
    tc::fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tc::tma_prefetch(&tmap_k);
    tc::tma_prefetch(&tmap_v);
  }
  if (warp == 1) tc::tmem_alloc(&bars->tmem_base, kTmemCols);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  tc::griddep_wait();    // the masks' bits are in place, the status word is clear
  tc::griddep_launch();
  bool failed = false;

  if (warp < 4) {
    regs_dec<kRegsCtl>();
    if (warp == 0) {
      // ---------------- producer: pieces and TMA ----------------
      if (blockIdx.x == 0)
        for (int b = lane; b < P.B; b += 32)
          if (A.kv_lens[b] < 0 || A.kv_lens[b] > P.Skv - nodes) atomicOr(status, kStatusBadLength);
      TreeWalk w;
      w.begin(A, blockIdx.x, gridDim.x);
      if (tc::elect_one()) {
        tc::ArmedRing kv_armed, q_armed;
        int stage = 0;
        uint32_t phase = 0;
        for (int ii = 0; !failed; ++ii) {
          const int slot = ii % kItems;
          TreeWalk::Piece p{};
          const bool live = w.next(A, &p);
          if (!tc::mbar_wait(&bars->i_empty[slot], ((ii / kItems) & 1) ^ 1, abort)) {
            failed = true;
            break;
          }
          const int row0 = p.group * 128;
          bars->item[slot] = Item{live, p.b, p.g, row0, min(128, nodes * P.G - row0),
                                  p.kt0, p.kt1 - p.kt0, p.len, p.slot};
          tc::mbar_arrive(&bars->i_full[slot]);
          if (!live) break;
          // Q rows of (node, head) are heads of consecutive nodes: one box per half
          if (A.q_boxes) {
            const int qs = ii & 1;
            if (!tc::mbar_wait(&bars->q_empty[qs], ((ii >> 1) & 1) ^ 1, abort)) {
              failed = true;
              break;
            }
            tc::mbar_arrive_expect_tx(&bars->q_full[qs], C::kTileBytes);
            q_armed.note(qs, (ii >> 1) & 1);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_load_3d(qbuf + qs * C::kTileBytes + h * C::kHalf, &tmap_q, &bars->q_full[qs],
                              64 * h, p.g * P.G, p.b * nodes + row0 / P.G);
          }
          // In the order of use, K0 K1 V0 K2 V1 K3 ..: a V tile that came with its K tile
          // would hold a stage through the whole softmax.
          const int32_t* pages = P.table ? P.table + (long long)p.b * P.table_w : nullptr;
          const int n = p.kt1 - p.kt0;
          int page = pages ? pages[p.kt0] : 0, next = 0;   // next: K tile whose row comes next
          auto next_row = [&]() -> int {
            const int t = p.kt0 + next++;
            if (!pages) return p.b * P.Skv + t * kDenseTile;
            const bool in = page >= 0 && page < P.pages;
            if (!in) atomicOr(status, kStatusBadPage);
            const int row = in ? page * kDenseTile : 0;
            if (next < n) page = pages[t + 1];  // on its way during this tile's copies
            return row;
          };
          auto copy = [&](const CUtensorMap* map, int row) {
            if (!tc::mbar_wait(&bars->kv_empty[stage], phase ^ 1, abort)) { failed = true; return; }
            uint64_t* fb = &bars->kv_full[stage];
            uint8_t* dst = kvbuf + stage * C::kTileBytes;
            tc::mbar_arrive_expect_tx(fb, C::kTileBytes);
            kv_armed.note(stage, phase);
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tc::tma_load_3d(dst + h * C::kHalf, map, fb, 64 * h, p.g, row);
            if (++stage == C::kStages) { stage = 0; phase ^= 1; }
          };
          int r0 = next_row(), r1 = 0;
          copy(&tmap_k, r0);
          if (n > 1 && !failed) copy(&tmap_k, r1 = next_row());
          for (int x = 0; x < n && !failed; ++x) {
            copy(&tmap_v, r0);
            r0 = r1;
            if (x + 2 < n && !failed) copy(&tmap_k, r1 = next_row());
          }
        }
        if (!q_armed.drain(bars->q_full)) failed = true;
        if (!kv_armed.drain(bars->kv_full)) failed = true;
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer ----------------
      // S of tiles 0 and 1, then P V of tile x followed by S of tile x + 2 (of the next
      // piece's first tiles at the end); one barrier per pair of products (warp 2).
      if (tc::elect_one()) {
        constexpr uint32_t kHi = uint32_t(tc::kDescHi | (1024 >> 4));
        constexpr uint32_t kTile16 = C::kTileBytes / 16, kHalf16 = C::kHalf / 16;
        const uint32_t qd = uint32_t(tc::sdesc_sw128(tc::smem_addr(qbuf), 16, 1024));
        const uint32_t kd = uint32_t(tc::sdesc_sw128(tc::smem_addr(kvbuf), 16, 1024));
        const uint32_t vd = uint32_t(tc::sdesc_sw128(tc::smem_addr(kvbuf), C::kHalf, 1024));
        int ii = 0, rx = 0;   // pieces; ring position of the next tile, in order of use
        uint32_t ppar = 0;
        auto advance = [&]() { rx = rx + 1 == C::kStages ? 0 : rx + 1; };
        auto fetch = [&](Item* it) -> bool {
          const int slot = ii % kItems;
          if (!tc::mbar_spin(&bars->i_full[slot], (ii / kItems) & 1, abort)) return false;
          *it = bars->item[slot];
          tc::mbar_arrive(&bars->i_empty[slot]);
          ++ii;
          return true;
        };
        // S of tile x of the piece whose Q stage is qs
        auto scores = [&](int x, int qs, bool last) {
          const uint32_t a = qd + qs * kTile16, b = kd + rx * kTile16;
          const uint32_t st = tmem + (x & 1) * 256;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kHalf16 + (kk & 3) * 2;
            tc::mma_ss_lo(st, a + off, b + off, kHi, C::kIdescS, kk > 0 ? 1u : 0u);
          }
          tc::mma_commit(&bars->s_full[x & 1]);
          tc::mma_commit(&bars->kv_empty[rx]);
          if (last) tc::mma_commit(&bars->q_empty[qs]);
          advance();
        };
        Item cur{};
        failed = !fetch(&cur);
        if (!failed && cur.live) {
          failed = !tc::mbar_spin(&bars->first_full, 0, abort);
          tc::tc_fence_after();
          if (!failed) {
            scores(0, 0, cur.n == 1);
            if (cur.n > 1) scores(1, 0, cur.n == 2);
          }
        }
        while (!failed && cur.live) {
          const int n = cur.n, qs = (ii - 1) & 1;
          int off = cur.len - cur.kt0 * 128;   // tile's row of drafted token 0
          for (int x = 0; x < n; ++x, off -= 128) {
            const int e = x & 1;
            const uint32_t st = tmem + e * 256, v = vd + rx * kTile16;
            if (x == n - 1 && !fetch(&cur)) { failed = true; break; }
            if (!tc::mbar_spin(&bars->p_full[e], (ppar >> e) & 1, abort)) { failed = true; break; }
            ppar ^= 1u << e;
            tc::tc_fence_after();
            const int groups = (min(128, off + nodes) + 15) >> 4;
            if (groups == 8) {
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO,
                              kk > 0 ? 1u : uint32_t(x >= 2));
            } else {
#pragma unroll 1
              for (int kk = 0; kk < groups; ++kk)
                tc::mma_ts_lo(st + 128, st + kk * 8, v + kk * 128, kHi, C::kIdescO,
                              kk > 0 ? 1u : uint32_t(x >= 2));
            }
            tc::mma_commit(&bars->kv_empty[rx]);
            advance();
            if (x + 2 >= n) tc::mma_commit(&bars->o_done[e]);
            if (x + 2 < n) {
              scores(x + 2, qs, x + 3 == n);
            } else if (x == n - 1 && cur.live) {
              scores(0, qs ^ 1, cur.n == 1);
              if (cur.n > 1) scores(1, qs ^ 1, cur.n == 2);
            }
          }
        }
        if (!tc::mma_drain(&bars->mma_done)) failed = true;
      }
    } else if (warp == 2) {
      // ---------------- what else the products need ----------------
      // One arrival per tile at p_full of its chain: V has landed, with the rows that no
      // node sees zeroed, K of the scores that follow too, the epilogue has read the
      // chain's previous O.
      int ii = 0, rx = 0;
      uint32_t rp = 0, un[2] = {0, 0}, on[2] = {0, 0};
      auto fetch = [&](Item* it) -> bool {
        const int slot = ii % kItems;
        if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) return false;
        *it = bars->item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
        ++ii;
        return true;
      };
      auto landed = [&]() -> bool {  // the next tile in the order of use
        if (!warp_wait(&bars->kv_full[rx], rp, abort)) return false;
        if (++rx == C::kStages) { rx = 0; rp ^= 1; }
        return true;
      };
      // Q of the piece just fetched, and its first K tiles
      auto start = [&](const Item& it) -> bool {
        return warp_wait(&bars->q_full[(ii - 1) & 1], ((ii - 1) >> 1) & 1, abort) &&
               landed() && (it.n == 1 || landed());
      };
      Item cur{}, nxt{};
      failed = !fetch(&cur) || (cur.live && !start(cur));
      if (!failed && cur.live && lane == 0) tc::mbar_arrive(&bars->first_full);
      while (!failed && cur.live) {
        int off = cur.len - cur.kt0 * 128;
        for (int x = 0; x < cur.n; ++x, off -= 128) {
          const int e = x & 1, vs = rx;
          if (!landed()) { failed = true; break; }
          if (off < 128) {
            uint8_t* v = kvbuf + vs * C::kTileBytes;
            const int rows = (min(128, off + nodes) + 15) & ~15;
            const uint4 seen = A.bits[(long long)(A.mask_stride ? cur.b : 0) * (nodes + 1) + nodes];
            for (int r0 = max(0, off) & ~31; r0 < rows; r0 += 32) {
              uint32_t w = ~bits_at(seen, r0 - off);
              if (rows - r0 < 32) w &= (1u << (rows - r0)) - 1u;
              while (w) {
                const int r = r0 + __ffs(w) - 1;
                w &= w - 1;
                if (lane < 8 * (D / 64))
                  *reinterpret_cast<uint4*>(v + (lane >> 3) * C::kHalf + r * 128 +
                                            (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
              }
            }
            tc::fence_async_smem();
            __syncwarp();
          }
          // the arrival belongs to this tile: the chain's tile before is over
          if ((on[e] > 0 && !warp_wait(&bars->p_full[e], (on[e] & 1) ^ 1, abort)) ||
              (x < 2 && !warp_wait(&bars->o_empty[e], (un[e]++ & 1) ^ 1, abort)) ||
              (x + 2 < cur.n && !landed()) ||
              (x == cur.n - 1 && (!fetch(&nxt) || (nxt.live && !start(nxt))))) {
            failed = true;
            break;
          }
          ++on[e];
          if (lane == 0) tc::mbar_arrive(&bars->p_full[e]);
        }
        cur = nxt;
      }
    } else {
      // ---------------- Q rows, where a box does not fetch them ----------------
      constexpr int kChunks = D / 8;   // 16-byte chunks of a row
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems, qs = ii & 1;
        if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
        const Item it = bars->item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
        if (!it.live) break;
        if (A.q_boxes) continue;  // the producer's
        if (!warp_wait(&bars->q_empty[qs], ((ii >> 1) & 1) ^ 1, abort)) { failed = true; break; }
        uint8_t* dst = qbuf + qs * C::kTileBytes;
        const int total = it.rows * kChunks;
        for (int i0 = lane; i0 < total; i0 += 32 * 8) {
          uint4 x[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = i0 + 32 * u, r = it.row0 + i / kChunks;
            if (i < total)
              x[u] = *reinterpret_cast<const uint4*>(
                  q + (((long long)it.b * nodes + r / P.G) * P.Hq + it.g * P.G + r % P.G) * D +
                  (i % kChunks) * 8);
          }
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = i0 + 32 * u, r = i / kChunks, c = i % kChunks;
            if (i < total)
              *reinterpret_cast<uint4*>(dst + (c >> 3) * C::kHalf + r * 128 +
                                        (((c & 7) ^ (r & 7)) << 4)) = x[u];
          }
        }
        tc::fence_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->q_full[qs]);
      }
    }
  } else if (warp < 12) {
    // ---------------- softmax of chain e ----------------
    regs_inc<kRegsSoftmax>();
    const int e = (warp - 4) >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t st = tmem + (uint32_t(quarter * 32) << 16) + e * 256, ot = st + 128;
    const float sl2 = P.scale * kLog2e;
    const uint64_t sl2x2 = f2(sl2, sl2);
    int un = 0, on = 0;
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const Item it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      if (it.n <= e) continue;
      const bool work = quarter * 32 < it.rows;  // some row of the warp exists
      float m = -INFINITY, ms = 0.f, l = 0.f;
      uint4 seen = make_uint4(0, 0, 0, 0);
      if (work && (it.kt0 + it.n) * 128 > it.len) {
        const int node = (it.row0 + min(row, it.rows - 1)) / P.G;
        seen = A.bits[(long long)(A.mask_stride ? it.b : 0) * (nodes + 1) + node];
      }
      for (int j = e; j < it.n; j += 2, ++on) {
        if (!warp_wait(&bars->s_full[e], on & 1, abort)) { failed = true; break; }
        if (work) {
          tc::tc_fence_after();
          // 32 columns at a time, each read twice: a loop over the whole row at once is
          // 700 instructions that every launch fetches anew, 4000 cycles and more of a
          // piece's first tiles
          const int off = it.len - (it.kt0 + j) * 128;
          auto chunk = [&](int q4, uint32_t (&v)[32]) {
            tc::tmem_ld32(st + q4 * 32, v);
            tc::tmem_ld_wait();
            if (off < 128) {
              const uint32_t w = bits_at(seen, q4 * 32 - off);
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!((w >> x) & 1u)) v[x] = __float_as_uint(-INFINITY);
            }
          };
          float top = -INFINITY;
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t v[32];
            chunk(q4, v);
            top = max32(v, top);
          }
          const bool grow = j == e || (top - m) * sl2 > kSlack;
          float keep = 1.f;
          if (grow) {
            const float nms = top == -INFINITY ? 0.f : top * sl2;
            keep = m == -INFINITY ? 0.f : ex2_f32(ms - nms);
            m = top;
            ms = nms;
          }
          const uint64_t nmsx2 = f2(-ms, -ms);
          uint64_t lsum[2] = {0, 0};
          // P of columns 32 q4 .. goes over columns 16 q4 .., which have been read
#pragma unroll 1
          for (int q4 = 0; q4 < 4; ++q4) {
            uint32_t v[32], pw[16];
            chunk(q4, v);
#pragma unroll
            for (int x = 0; x < 32; x += 2) {
              const uint64_t z = fma2((uint64_t(v[x + 1]) << 32) | v[x], sl2x2, nmsx2);
              const float pa = ex2_f32(__uint_as_float(uint32_t(z)));
              const float pb = ex2_f32(__uint_as_float(uint32_t(z >> 32)));
              lsum[(x >> 1) & 1] = add2(lsum[(x >> 1) & 1], f2(pa, pb));
              pw[x >> 1] = pack_bf16(pa, pb);
            }
            tmem_st8(st + q4 * 16, pw);
            tmem_st8(st + q4 * 16 + 8, pw + 8);
          }
          if (j > e && __any_sync(MSA_FULL_MASK, grow)) {
            // the previous P V was issued before this S: O is there
            const uint64_t k2 = f2(keep, keep);
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tc::tmem_ld32(ot + c, o);
              tc::tmem_ld_wait();
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                const uint64_t y = mul2((uint64_t(o[x + 1]) << 32) | o[x], k2);
                o[x] = uint32_t(y);
                o[x + 1] = uint32_t(y >> 32);
              }
              tc::tmem_st32(ot + c, o);
            }
          }
          tc::tmem_st_wait();
          tc::tc_fence_before();
          const uint64_t lsx = add2(lsum[0], lsum[1]);
          l = l * keep + (__uint_as_float(uint32_t(lsx)) + __uint_as_float(uint32_t(lsx >> 32)));
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->p_full[e]);
      }
      if (failed || !warp_wait(&bars->l_empty[e], (un & 1) ^ 1, abort)) { failed = true; break; }
      bars->ml[e][row] = make_float2(m == -INFINITY ? -INFINITY : ms, l);
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->l_full[e]);
      ++un;
    }
  } else {
    // ---------------- epilogue: joins the chains ----------------
    regs_dec<kRegsEpi>();
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t ot = tmem + (uint32_t(quarter * 32) << 16) + 128;
    int un1 = 0;   // pieces with a second chain
    for (int ii = 0; !failed; ++ii) {
      const int slot = ii % kItems;
      if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
      const Item it = bars->item[slot];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
      if (!it.live) break;
      const bool two = it.n > 1;
      const uint32_t par0 = ii & 1, par1 = un1 & 1;
      if (!warp_wait(&bars->l_full[0], par0, abort) ||
          (two && !warp_wait(&bars->l_full[1], par1, abort))) {
        failed = true;
        break;
      }
      const float2 a = bars->ml[0][row];
      const float2 b = two ? bars->ml[1][row] : make_float2(-INFINITY, 0.f);
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bars->l_empty[0]);
        if (two) tc::mbar_arrive(&bars->l_empty[1]);
      }
      const float m = fmaxf(a.x, b.x), base = m == -INFINITY ? 0.f : m;
      float wa = ex2_f32(a.x - base), wb = ex2_f32(b.x - base);
      const float l = a.y * wa + b.y * wb;
      const bool whole = it.slot < 0, mine = row < it.rows;
      const int r = it.row0 + row;
      const long long at = whole ? ((long long)it.b * nodes + r / P.G) * P.Hq + it.g * P.G + r % P.G
                                 : (long long)(blockIdx.x * 2 + it.slot) * 128 + row;
      float* part = A.part_o + (long long)(blockIdx.x * 2 + it.slot) * 128 * D + row;
      if (mine) {
        if (!whole) A.part_ml[at] = make_float2(m, l);
        else if (lse) lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        wa *= inv;
        wb *= inv;
      }
      if (!warp_wait(&bars->o_done[0], par0, abort) ||
          (two && !warp_wait(&bars->o_done[1], par1, abort))) {
        failed = true;
        break;
      }
      tc::tc_fence_after();
      if (quarter * 32 < it.rows) {
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t x[16], y[16];
          __syncwarp();
          tc::tmem_ld16(ot + c, x);
          if (two) tc::tmem_ld16(ot + 256 + c, y);
          tc::tmem_ld_wait();
          float o[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i] = __uint_as_float(x[i]) * wa;
            if (two) o[i] += __uint_as_float(y[i]) * wb;
          }
          if (mine && whole) {
#pragma unroll
            for (int i = 0; i < 16; i += 8)
              *reinterpret_cast<uint4*>(out + at * D + c + i) =
                  make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                             pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7]));
          } else if (mine) {
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128] = o[i];
          }
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&bars->o_empty[0]);
        if (two) tc::mbar_arrive(&bars->o_empty[1]);
      }
      if (two) ++un1;
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
cudaError_t tree_tc(const Tree& A_, const void* q, const void* k, const void* v, void* out,
                    float* lse, int32_t* status, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  CUtensorMap mq, mk, mv;
  Tree A = A_;
  A.q_boxes = 128 % A.d.G == 0;
  cudaError_t e = encode_rows(&mq, q, D, A.d.Hq, A.d.rows_q, A.q_boxes ? 128 / A.d.G : 1,
                              A.q_boxes ? A.d.G : 1);
  if (e == cudaSuccess) e = encode_rows(&mk, k, D, A.d.Hkv, A.d.rows_k);
  if (e == cudaSuccess) e = encode_rows(&mv, v, D, A.d.Hkv, A.d.rows_k);
  if (e == cudaSuccess)
    e = prepare_kernel(&done, tree_tc_kernel<D>, smem_bytes<D>(), kRegsCtl + kRegsEpi + 2 * kRegsSoftmax,
                       kThreads);
  if (e != cudaSuccess) return e;
  tree_prep_kernel<<<A.mask_stride ? A.d.B : 1, 256, 0, s>>>(A.mask, A.mask_stride, A.d.Sq, A.bits,
                                                             status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_after(tree_tc_kernel<D>, tree_ctas(A.d.f32), kThreads, smem_bytes<D>(), s, mq, mk, mv,
                   A, static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(out), lse,
                   status);
  if (e != cudaSuccess) return e;
  return launch_tree_combine(A, out, lse, s);
}

}  // namespace

cudaError_t launch_tree_tc(const Tree& A, const void* q, const void* k, const void* v, void* out,
                           float* lse, int32_t* status, cudaStream_t s) {
  return (A.d.D == 128 ? tree_tc<128> : tree_tc<64>)(A, q, k, v, out, lse, status, s);
}

}  // namespace msa
