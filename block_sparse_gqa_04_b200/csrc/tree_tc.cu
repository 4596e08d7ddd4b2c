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
// each with its own MMA-issuing thread, softmax warpgroup, running maximum and sum, and
// accumulator O, so that one chain's MMAs and copies run under the other's softmax;
// the epilogue joins the two.  Scores, probabilities and the moving maximum are as in
// the forward pass over whole prompts.  K and V tiles come through a ring of TMA
// stages (160 KB in flight); Q rows are gathered by one warp, a piece ahead.
//
// Which drafted tokens a node sees comes as one bit mask per node, and which are seen
// at all as one per sequence, formed by a small launch before.  V rows of unseen tokens
// are zeroed in shared memory, for they may hold anything.
#include <algorithm>

#include "dense_tc.cuh"

namespace msa {
namespace {

// warp 0 pieces and TMA, warps 1-2 MMA, warp 3 Q rows, warps 4-11 softmax, 12-15 epilogue
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
  // per chain: S computed, P written, each P V done, the piece's last P V done, O read,
  // (maximum, sum) written, read
  uint64_t s_full[2], p_full[2], o_step[2], o_done[2], o_empty[2], l_full[2], l_empty[2];
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
tree_tc_kernel(const __grid_constant__ CUtensorMap tmap_k,
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
      tc::mbar_init(&bars->q_empty[b], 2);   // both chains' issuers
      tc::mbar_init(&bars->s_full[b], 1);
      tc::mbar_init(&bars->p_full[b], 4);
      tc::mbar_init(&bars->o_step[b], 1);
      tc::mbar_init(&bars->o_done[b], 1);
      tc::mbar_init(&bars->o_empty[b], 4);
      tc::mbar_init(&bars->l_full[b], 4);
      tc::mbar_init(&bars->l_empty[b], 4);
    }
    for (int i = 0; i < kItems; ++i) {
      tc::mbar_init(&bars->i_full[i], 1);
      tc::mbar_init(&bars->i_empty[i], 15);  // 2 MMA, Q, 8 softmax, 4 epilogue warps
    }
    tc::mbar_init(&bars->mma_done, 2);
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
  bool failed = false;

  if (warp < 4) {
    regs_dec<kRegsCtl>();
    if (warp == 0) {
      // ---------------- producer: pieces and TMA ----------------
      tc::ArmedRing kv_armed;
      int stage = 0;
      uint32_t phase = 0;
      if (blockIdx.x == 0)
        for (int b = lane; b < P.B; b += 32)
          if (A.kv_lens[b] < 0 || A.kv_lens[b] > P.Skv - nodes) atomicOr(status, kStatusBadLength);
      TreeWalk w;
      w.begin(A, blockIdx.x, tree_span(A, gridDim.x));
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        TreeWalk::Piece p{};
        const bool live = w.next(A, &p);
        bool good = true;
        if (lane == 0) {
          good = tc::mbar_wait(&bars->i_empty[slot], ((ii / kItems) & 1) ^ 1, abort);
          if (good) {
            const int row0 = p.group * 128;
            bars->item[slot] = Item{live, p.b, p.g, row0, min(128, nodes * P.G - row0),
                                    p.kt0, p.kt1 - p.kt0, p.len, p.slot};
            tc::mbar_arrive(&bars->i_full[slot]);
          }
        }
        if (!__shfl_sync(MSA_FULL_MASK, good, 0)) { failed = true; break; }
        if (!live) break;
        for (int j0 = p.kt0; j0 < p.kt1 && !failed; j0 += 32) {
          // the rows of 32 tiles at a time: their pages come with one load
          int row = 0;
          if (j0 + lane < p.kt1) {
            if (P.table) {
              const int pg = P.table[(long long)p.b * P.table_w + j0 + lane];
              const bool in = pg >= 0 && pg < P.pages;
              if (!in) atomicOr(status, kStatusBadPage);
              row = in ? pg * kDenseTile : 0;
            } else {
              row = p.b * P.Skv + (j0 + lane) * kDenseTile;
            }
          }
          for (int j = 0; j < 32 && j0 + j < p.kt1; ++j) {
            const int r = __shfl_sync(MSA_FULL_MASK, row, j);
            if (lane == 0) {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                good = good && tc::mbar_wait(&bars->kv_empty[stage], phase ^ 1, abort);
                if (!good) break;
                uint64_t* fb = &bars->kv_full[stage];
                uint8_t* dst = kvbuf + stage * C::kTileBytes;
                tc::mbar_arrive_expect_tx(fb, C::kTileBytes);
                kv_armed.note(stage, phase);
#pragma unroll
                for (int h = 0; h < D / 64; ++h)
                  tc::tma_load_3d(dst + h * C::kHalf, x ? &tmap_v : &tmap_k, fb, 64 * h, p.g, r);
                if (++stage == C::kStages) { stage = 0; phase ^= 1; }
              }
            }
            if (!__shfl_sync(MSA_FULL_MASK, good, 0)) { failed = true; break; }
          }
        }
      }
      if (lane == 0 && !kv_armed.drain(bars->kv_full)) failed = true;
    } else if (warp < 3) {
      // ---------------- MMA issuer of chain e ----------------
      const int e = warp - 1;
      const uint32_t st = tmem + e * 256, ot = st + 128;
      long long n0 = 0;      // key tiles of the pieces before
      int on = 0, un = 0;    // key tiles of this chain, pieces in which it has any
      auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        const bool ok = lane != 0 || tc::mbar_spin(bar, parity, abort);
        return __shfl_sync(MSA_FULL_MASK, ok ? 1 : 0, 0) != 0;
      };
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems;
        if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
        const Item it = bars->item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
        if (!it.live) break;
        const int qs = ii & 1;
        if (!wait(&bars->q_full[qs], (ii >> 1) & 1)) { failed = true; break; }
        const int last = it.n - 1 - ((it.n - 1 - e) & 1);  // the chain's last tile, if any
        for (int j = e; j < it.n; j += 2) {
          const long long x = 2 * (n0 + j);
          const int ks = int(x % C::kStages), vs = int((x + 1) % C::kStages);
          if (!wait(&bars->kv_full[ks], uint32_t((x / C::kStages) & 1))) { failed = true; break; }
          if (lane == 0) {
            tc::tc_fence_after();
            const uint32_t qa = tc::smem_addr(qbuf + qs * C::kTileBytes);
            const uint32_t ka = tc::smem_addr(kvbuf + ks * C::kTileBytes);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * C::kHalf + (kk & 3) * 32;
              tc::mma_ss(st, tc::sdesc_sw128(qa + off, 16, 1024),
                         tc::sdesc_sw128(ka + off, 16, 1024), C::kIdescS, kk > 0 ? 1u : 0u);
            }
            tc::mma_commit(&bars->s_full[e]);
            tc::mma_commit(&bars->kv_empty[ks]);
          }
          if (!wait(&bars->kv_full[vs], uint32_t(((x + 1) / C::kStages) & 1))) {
            failed = true;
            break;
          }
          uint8_t* v = kvbuf + vs * C::kTileBytes;
          const int off = it.len - (it.kt0 + j) * 128;     // tile's row of drafted token 0
          const int keys = min(128, off + nodes), groups = (keys + 15) >> 4;
          if (off < 128) {
            // drafted tokens that nobody sees, and what is behind them
            const uint4 seen = A.bits[(long long)(A.mask_stride ? it.b : 0) * (nodes + 1) + nodes];
            for (int r0 = max(0, off) & ~31; r0 < groups * 16; r0 += 32) {
              uint32_t w = ~bits_at(seen, r0 - off);
              if (groups * 16 - r0 < 32) w &= (1u << (groups * 16 - r0)) - 1u;
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
          if (!wait(&bars->p_full[e], on & 1) ||
              (j == e && !wait(&bars->o_empty[e], (un & 1) ^ 1))) {
            failed = true;
            break;
          }
          if (lane == 0) {
            tc::tc_fence_after();
            const uint32_t va = tc::smem_addr(v);
            for (int kk = 0; kk < groups; ++kk)
              tc::mma_ts(ot, st + kk * 8, tc::sdesc_sw128(va + kk * 2048, C::kHalf, 1024),
                         C::kIdescO, (j > e || kk > 0) ? 1u : 0u);
            tc::mma_commit(&bars->kv_empty[vs]);
            tc::mma_commit(&bars->o_step[e]);
            if (j == last) tc::mma_commit(&bars->o_done[e]);
          }
          ++on;
        }
        if (failed) break;
        // the chain is done with the piece's Q
        if (lane == 0) {
          if (it.n > e) tc::mma_commit(&bars->q_empty[qs]);
          else tc::mbar_arrive(&bars->q_empty[qs]);
        }
        if (it.n > e) ++un;
        n0 += it.n;
      }
      if (lane == 0 && !tc::mma_drain(&bars->mma_done)) failed = true;
    } else {
      // ---------------- Q rows ----------------
      constexpr int kChunks = D / 8;   // 16-byte chunks of a row
      for (int ii = 0; !failed; ++ii) {
        const int slot = ii % kItems, qs = ii & 1;
        if (!warp_wait(&bars->i_full[slot], (ii / kItems) & 1, abort)) { failed = true; break; }
        const Item it = bars->item[slot];
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars->i_empty[slot]);
        if (!it.live) break;
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
          uint32_t v[4][32];
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) tc::tmem_ld32(st + q4 * 32, v[q4]);
          tc::tmem_ld_wait();
          const int off = it.len - (it.kt0 + j) * 128;
          if (off < 128) {
#pragma unroll
            for (int q4 = 0; q4 < 4; ++q4) {
              const uint32_t w = bits_at(seen, q4 * 32 - off);
#pragma unroll
              for (int x = 0; x < 32; ++x)
                if (!((w >> x) & 1u)) v[q4][x] = __float_as_uint(-INFINITY);
            }
          }
          float top = max32(v[0], -INFINITY);
          top = fmaxf(fmaxf(top, max32(v[1], -INFINITY)), fmaxf(max32(v[2], -INFINITY),
                                                               max32(v[3], -INFINITY)));
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
          }
          if (j > e && __any_sync(MSA_FULL_MASK, grow)) {
            if (!warp_wait(&bars->o_step[e], (on & 1) ^ 1, abort)) { failed = true; break; }
            tc::tc_fence_after();
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
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(A.part_o + at * D + c + i) =
                  make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
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
cudaError_t tree_tc(const Tree& A, const void* q, const void* k, const void* v, void* out,
                    float* lse, int32_t* status, cudaStream_t s) {
  CUtensorMap mk, mv;
  cudaError_t e = encode_rows(&mk, k, D, A.d.Hkv, A.d.rows_k);
  if (e == cudaSuccess) e = encode_rows(&mv, v, D, A.d.Hkv, A.d.rows_k);
  if (e == cudaSuccess)
    e = prepare_kernel(tree_tc_kernel<D>, smem_bytes<D>(), kRegsCtl + kRegsEpi + 2 * kRegsSoftmax,
                       kThreads);
  if (e != cudaSuccess) return e;
  tree_prep_kernel<<<A.mask_stride ? A.d.B : 1, 256, 0, s>>>(A.mask, A.mask_stride, A.d.Sq, A.bits,
                                                             status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  tree_tc_kernel<D><<<tree_ctas(), kThreads, smem_bytes<D>(), s>>>(
      mk, mv, A, static_cast<const __nv_bfloat16*>(q), static_cast<__nv_bfloat16*>(out), lse,
      status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_combine(A, out, lse, s);
}

}  // namespace

cudaError_t launch_tree_tc(const Tree& A, const void* q, const void* k, const void* v, void* out,
                           float* lse, int32_t* status, cudaStream_t s) {
  return (A.d.D == 128 ? tree_tc<128> : tree_tc<64>)(A, q, k, v, out, lse, status, s);
}

}  // namespace msa
