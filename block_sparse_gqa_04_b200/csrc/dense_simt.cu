// Dense attention in fp32 on the CUDA cores: forward, gradients, and the tree form
// over a cache.
//
// One block holds 32 rows (queries, or keys for their gradients) and walks the 64-row
// tiles of the other side that they see, with the running maximum and sum of the softmax
// (one pass over the keys):
//   S = Q K^T, m' = max(m, max S), P = 2^(S - m'), l = l 2^(m - m') + sum P,
//   O = O 2^(m - m') + P V
// in base 2 with the scale folded into the exponent.  128 threads form an 8 x 16 grid; a
// thread owns 4 rows (8 apart) x 4 columns (16 apart) of S and the same rows of D/16
// columns of O.  The products are register-tiled from shared memory: 64 FMAs per 8
// 16-byte loads, which bound them (4 cycles of shared memory each against 64 cycles of the
// FMA pipe for four warps).  A tile is copied while the other operand's product runs.  32
// rows rather than 64 give small problems twice the blocks and half the longest one; 8 or 2
// rows to a thread instead of 4 (64 or 256 threads) take 1.0 to 1.5 times as long, for want
// of warps or for more loads.  Training step of 1024 rows x 8 heads x 64: 0.28 ms; attention
// of 1500 rows x 32 heads x 128: 0.49 ms, 38 TFLOP/s.
#include <algorithm>

#include "dense_common.cuh"
#include "tc_warp.cuh"

namespace msa {
namespace {

constexpr int kThreads = 128;
constexpr int kRows = 32;    // rows of a block
constexpr int kTile = 64;    // columns at a time
constexpr int kTy = kThreads / 16;   // threads along the rows
constexpr int kR = kRows / kTy;      // rows of a thread, kTy apart
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Smem {
  static constexpr int kPitch = D + 4;  // rows 4 banks apart: 16-byte loads of 8 rows do not collide
  static constexpr int kRowFloats = kRows * kPitch, kTileFloats = kTile * kPitch;
  static constexpr int kPPitch = kTile + 4;
  static constexpr int kPFloats = kRows * kPPitch;
};

// Rows 0 .. N-1 of `src` (row r at src + r * stride elements) on their way into a tile;
// rows from `valid` on become zero.  One group of copies: tile_wait() waits for all but
// the latest `left` groups of the thread.
template <int D, int N>
__device__ __forceinline__ void load_tile(float* dst, const float* src, long long stride,
                                          int valid) {
#pragma unroll 8
  for (int i = threadIdx.x; i < N * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4, bytes = r < valid ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     tc::smem_addr(dst + r * Smem<D>::kPitch + c)),
                 "l"(src + (r < valid ? r * stride : 0) + c), "r"(bytes)
                 : "memory");
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void tile_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
  __syncthreads();
}

// acc[i][j] = A[row ty + kTy i] . B[row tx + 16 j] over D columns.  Two FMAs to an
// instruction, here and below (neighbouring columns lie side by side in both operands), and
// 16 passes unrolled: against scalar FMAs, 4 and 2 passes unrolled, the attention of 4000
// rows x 8 heads x 64 went from 518 to 458 us and its gradients from 1.69 to 1.66 ms, that of
// 1500 rows x 32 heads x 128 from 560 to 491 us and from 2.31 to 1.96 ms (32 passes: 2.15).
template <int D>
__device__ __forceinline__ void product_nt(const float* A, const float* B, int ty, int tx,
                                           float (&acc)[kR][4]) {
  constexpr int P = Smem<D>::kPitch;
  uint64_t sum[kR][4] = {};  // of even and of odd columns
#pragma unroll 16
  for (int d = 0; d < D; d += 4) {
    ulonglong2 a[kR], b[4];
#pragma unroll
    for (int i = 0; i < kR; ++i)
      a[i] = *reinterpret_cast<const ulonglong2*>(A + (ty + kTy * i) * P + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const ulonglong2*>(B + (tx + 16 * j) * P + d);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sum[i][j] = fma2(a[i].x, b[j].x, sum[i][j]);
        sum[i][j] = fma2(a[i].y, b[j].y, sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[i][j] = __uint_as_float(uint32_t(sum[i][j])) + __uint_as_float(uint32_t(sum[i][j] >> 32));
}

// acc[i][c] += sum_k W[row ty + kTy i][k] * B[k][col], W [32][kPPitch], columns
// tx * 4 + 64 * (c / 4) + c % 4 (D = 64: 4 columns, 128: 8), two to an accumulator.
template <int D>
__device__ __forceinline__ void product_nn(const float* W, const float* B, int ty, int tx,
                                           uint64_t (&acc)[kR][D / 32]) {
  constexpr int P = Smem<D>::kPitch, PP = Smem<D>::kPPitch;
#pragma unroll
  for (int k = 0; k < kTile; k += 4) {
    float4 w[kR];
#pragma unroll
    for (int i = 0; i < kR; ++i) w[i] = *reinterpret_cast<const float4*>(W + (ty + kTy * i) * PP + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint64_t x[kR];
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const float y = reinterpret_cast<const float*>(&w[i])[kk];
        x[i] = f2(y, y);
      }
#pragma unroll
      for (int c = 0; c < D / 32; c += 2) {
        const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(B + (k + kk) * P + tx * 4 + c * 32);
#pragma unroll
        for (int i = 0; i < kR; ++i) {
          acc[i][c] = fma2(x[i], b.x, acc[i][c]);
          acc[i][c + 1] = fma2(x[i], b.y, acc[i][c + 1]);
        }
      }
    }
  }
}

__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(MSA_FULL_MASK, v, o));
  return v;
}
__device__ __forceinline__ float sum16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(MSA_FULL_MASK, v, o);
  return v;
}

// Running softmax of a thread's 4 rows (each shared by the 16 threads of a row).
template <int D>
struct Running {
  float m[kR], l[kR];
  uint64_t o[kR][D / 32];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[i][c] = 0;
    }
  }
  // Scores (already scaled to base 2, -inf where hidden) of one key tile: P into Ps.
  __device__ __forceinline__ void step(float (&s)[kR][4], float* Ps, int ty, int tx) {
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      float mx = fmaxf(fmaxf(s[i][0], s[i][1]), fmaxf(s[i][2], s[i][3]));
      mx = fmaxf(m[i], max16(mx));
      const float base = mx == -INFINITY ? 0.f : mx;  // a row that has seen nothing yet
      const float keep = exp2f(m[i] - base);
      m[i] = mx;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(s[i][j] - base);
        sum += p;
        Ps[(ty + kTy * i) * Smem<D>::kPPitch + tx + 16 * j] = p;
      }
      l[i] = l[i] * keep + sum16(sum);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[i][c] = mul2(o[i][c], f2(keep, keep));
    }
  }
};

__device__ __forceinline__ float part_of(const uint64_t* x, int e) {  // e: a constant
  return __uint_as_float(uint32_t(x[e >> 1] >> (e & 1 ? 32 : 0)));
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, const uint64_t* x, float scale) {
#pragma unroll
  for (int e = 0; e < 4; ++e) dst[e] = from_f32<T>(part_of(x, e) * scale);
}

template <int D>
constexpr size_t fwd_smem() {
  return sizeof(float) * (Smem<D>::kRowFloats + 2 * Smem<D>::kTileFloats + Smem<D>::kPFloats);
}

// Blocks of a 128-row tile.
constexpr int kParts = kDenseTile / kRows;

// ---------------------------------------------------------------------------
// Forward over whole prompts: block = (32 query rows, head)
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
dense_fwd_simt_kernel(Dense P, const T* __restrict__ q, const T* __restrict__ k,
                      const T* __restrict__ v, T* __restrict__ out, float* __restrict__ lse) {
  extern __shared__ float sm[];
  float* Qs = sm;
  float* Ks = Qs + Smem<D>::kRowFloats;
  float* Vs = Ks + Smem<D>::kTileFloats;
  float* Ps = Vs + Smem<D>::kTileFloats;
  const int h = blockIdx.x % P.Hq, t = blockIdx.x / P.Hq;
  int qt;
  const SeqRec s = query_tile(P, t / kParts, &qt);
  const int i0 = qt * kDenseTile + (kParts - 1 - t % kParts) * kRows;
  if (i0 >= s.nq) return;
  const int rows = min(kRows, s.nq - i0), g = h / P.G;
  const int b = P.seqs ? 0 : s.q0 / P.Sq;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  load_tile<D, kRows>(Qs, q + ((long long)(s.q0 + i0) * P.Hq + h) * D, (long long)P.Hq * D, rows);
  Running<D> R;
  R.clear();
  const float sl2 = P.scale * kLog2e;
  const int seen = min(s.nk, s.pos0 + i0 + rows);  // keys that the block's last row sees
  // rows behind what is seen are zero: a value there must not meet a weight of zero as NaN
  auto load = [&](float* dst, const T* src, int j0) {
    if (j0 >= seen) {  // keeps the count of groups
      asm volatile("cp.async.commit_group;" ::: "memory");
      return;
    }
    const long long row = tile_row(P, b, s.k0, j0 / kDenseTile) + (j0 % kDenseTile);
    load_tile<D, kTile>(dst, src + (row * P.Hkv + g) * D, (long long)P.Hkv * D,
                        min(kTile, seen - j0));
  };
  load(Ks, k, 0);
  load(Vs, v, 0);
  for (int j0 = 0; j0 < seen; j0 += kTile) {
    tile_wait<1>();  // K is there (and the previous P is read)
    float sc[kR][4] = {};
    product_nt<D>(Qs, Ks, ty, tx, sc);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool sees = j0 + tx + 16 * j <= s.pos0 + i0 + ty + kTy * i;
        sc[i][j] = sees ? sc[i][j] * sl2 : -INFINITY;
      }
    R.step(sc, Ps, ty, tx);
    __syncthreads();  // K is read, P written
    load(Ks, k, j0 + kTile);
    tile_wait<1>();   // V is there
    product_nn<D>(Ps, Vs, ty, tx, R.o);
    __syncthreads();  // V is read
    load(Vs, v, j0 + kTile);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = ty + kTy * i;
    if (r >= rows) continue;
    const long long at = (long long)(s.q0 + i0 + r) * P.Hq + h;
    const float inv = 1.f / R.l[i];
#pragma unroll
    for (int c = 0; c < D / 16; c += 4) store4(out + at * D + tx * 4 + c * 16, &R.o[i][c / 2], inv);
    if (lse && tx == 0) lse[at] = (R.m[i] + log2f(R.l[i])) * kLn2;
  }
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------
// delta[row, head] = sum_d dout out, one warp per (row, head).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
dense_delta_kernel(const T* __restrict__ dout, const T* __restrict__ out, float* __restrict__ delta,
                   long long n) {
  const long long r = (long long)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= n) return;
  constexpr int N = D / 32;
  float a[N], b[N], s = 0.f;
  load_vec<T, N>(dout + r * D + lane * N, a);
  load_vec<T, N>(out + r * D + lane * N, b);
#pragma unroll
  for (int i = 0; i < N; ++i) s += a[i] * b[i];
  s = warp_sum_f32(s);
  if (lane == 0) delta[r] = s;
}

// dk and dv: block = (32 keys, key head, split of the group's heads); walks those heads
// and the 64-query tiles that see the keys, with keys as rows:
//   P^T = 2^(c K Q^T - c lse), dS^T = P^T (V dO^T - delta), dV += P^T dO, dK += dS^T Q.
template <int D>
constexpr size_t dkv_smem() {
  return sizeof(float) * (2 * Smem<D>::kRowFloats + 2 * Smem<D>::kTileFloats +
                          2 * Smem<D>::kPFloats + 2 * kTile);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
dense_dkv_simt_kernel(Dense P, int splits, const T* __restrict__ dout, const T* __restrict__ q,
                      const T* __restrict__ k, const T* __restrict__ v,
                      const float* __restrict__ lse, const float* __restrict__ delta,
                      T* __restrict__ dk, T* __restrict__ dv, float* __restrict__ part) {
  extern __shared__ float sm[];
  float* Ks = sm;
  float* Vs = Ks + Smem<D>::kRowFloats;
  float* Qs = Vs + Smem<D>::kRowFloats;
  float* Gs = Qs + Smem<D>::kTileFloats;
  float* Ps = Gs + Smem<D>::kTileFloats;
  float* Ss = Ps + Smem<D>::kPFloats;
  float* lse_s = Ss + Smem<D>::kPFloats;
  float* delta_s = lse_s + kTile;
  const int split = blockIdx.x % splits, g = (blockIdx.x / splits) % P.Hkv;
  const int t = blockIdx.x / splits / P.Hkv;
  int kt;
  const SeqRec s = key_tile(P, t / kParts, &kt);
  const int j0 = kt * kDenseTile + (t % kParts) * kRows;
  if (j0 >= s.nk) return;
  const int keys = min(kRows, s.nk - j0);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long kst = (long long)P.Hkv * D, qst = (long long)P.Hq * D;
  const long long kat = ((long long)(s.k0 + j0) * P.Hkv + g) * D;
  load_tile<D, kRows>(Ks, k + kat, kst, keys);
  load_tile<D, kRows>(Vs, v + kat, kst, keys);
  uint64_t ak[kR][D / 32] = {}, av[kR][D / 32] = {};
  // the first query row that sees key j0 sits at position j0
  const int i_first = max(0, j0 - s.pos0) / kTile * kTile;
  const int per = (P.G + splits - 1) / splits;
  const int h0 = g * P.G + split * per, h1 = min(h0 + per, (g + 1) * P.G);
  const int tiles = max(0, (s.nq - i_first + kTile - 1) / kTile), steps = max(0, h1 - h0) * tiles;
  // step x: query tile x % tiles of head h0 + x / tiles
  auto place = [&](int x) {
    return (long long)(s.q0 + i_first + x % tiles * kTile) * P.Hq + h0 + x / tiles;
  };
  auto load = [&](float* dst, const T* src, int x) {
    if (x < steps)
      load_tile<D, kTile>(dst, src + place(x) * D, qst,
                          min(kTile, s.nq - i_first - x % tiles * kTile));
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  };
  float lse_r = 0.f, delta_r = 0.f;  // of the thread's query row in the coming step
  auto stats = [&](int x) {
    if (x >= steps || threadIdx.x >= kTile) return;
    const bool ok = int(threadIdx.x) < s.nq - i_first - x % tiles * kTile;
    const long long at = place(x) + (long long)threadIdx.x * P.Hq;
    lse_r = ok ? lse[at] * kLog2e : 0.f;
    delta_r = ok ? delta[at] : 0.f;
  };
  load(Gs, dout, 0);
  load(Qs, q, 0);
  stats(0);
  for (int x = 0; x < steps; ++x) {
    const int i0 = i_first + x % tiles * kTile, rows = min(kTile, s.nq - i0);
    if (threadIdx.x < kTile) {
      lse_s[threadIdx.x] = lse_r;
      delta_s[threadIdx.x] = delta_r;
    }
    tile_wait<1>();  // dO is there
    stats(x + 1);
    float sc[kR][4] = {}, dp[kR][4] = {};
    product_nt<D>(Vs, Gs, ty, tx, dp);
    tile_wait<0>();  // Q is there
    product_nt<D>(Ks, Qs, ty, tx, sc);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = ty + kTy * i, c = tx + 16 * j;
        const bool sees = c < rows && j0 + key <= s.pos0 + i0 + c;
        const float p = sees ? exp2f(sc[i][j] * (P.scale * kLog2e) - lse_s[c]) : 0.f;
        Ps[key * Smem<D>::kPPitch + c] = p;
        Ss[key * Smem<D>::kPPitch + c] = sees ? p * (dp[i][j] - delta_s[c]) : 0.f;
      }
    __syncthreads();
    product_nn<D>(Ps, Gs, ty, tx, av);
    __syncthreads();  // dO is read
    load(Gs, dout, x + 1);
    product_nn<D>(Ss, Qs, ty, tx, ak);
    __syncthreads();  // Q is read
    load(Qs, q, x + 1);
  }
  const long long all = P.rows_k * P.Hkv * D;
  float* pv = part + (long long)split * 2 * all;
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = ty + kTy * i;
    if (r >= keys) continue;
    const long long at = kat + r * kst + tx * 4;
#pragma unroll
    for (int c = 0; c < D / 16; c += 4) {
      if (splits > 1) {
        store4(pv + at + c * 16, &av[i][c / 2], 1.f);
        store4(pv + all + at + c * 16, &ak[i][c / 2], 1.f);
      } else {
        store4(dk + at + c * 16, &ak[i][c / 2], P.scale);
        store4(dv + at + c * 16, &av[i][c / 2], 1.f);
      }
    }
  }
}

// dq: block = (32 query rows, head); walks the keys that its rows see.
template <int D>
constexpr size_t dq_smem() {
  return sizeof(float) * (2 * Smem<D>::kRowFloats + 2 * Smem<D>::kTileFloats +
                          Smem<D>::kPFloats + 2 * kRows);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
dense_dq_simt_kernel(Dense P, const T* __restrict__ dout, const T* __restrict__ q,
                     const T* __restrict__ k, const T* __restrict__ v,
                     const float* __restrict__ lse, const float* __restrict__ delta,
                     T* __restrict__ dq) {
  extern __shared__ float sm[];
  float* Qs = sm;
  float* Gs = Qs + Smem<D>::kRowFloats;
  float* Ks = Gs + Smem<D>::kRowFloats;
  float* Vs = Ks + Smem<D>::kTileFloats;
  float* Ss = Vs + Smem<D>::kTileFloats;
  float* lse_s = Ss + Smem<D>::kPFloats;
  float* delta_s = lse_s + kRows;
  const int h = blockIdx.x % P.Hq, t = blockIdx.x / P.Hq, g = h / P.G;
  int qt;
  const SeqRec s = query_tile(P, t / kParts, &qt);
  const int i0 = qt * kDenseTile + (kParts - 1 - t % kParts) * kRows;
  if (i0 >= s.nq) return;
  const int rows = min(kRows, s.nq - i0);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long kst = (long long)P.Hkv * D, qst = (long long)P.Hq * D;
  const long long at = (long long)(s.q0 + i0) * P.Hq + h;
  load_tile<D, kRows>(Qs, q + at * D, qst, rows);
  load_tile<D, kRows>(Gs, dout + at * D, qst, rows);
  if (threadIdx.x < kRows) {
    const bool ok = int(threadIdx.x) < rows;
    lse_s[threadIdx.x] = ok ? lse[at + (long long)threadIdx.x * P.Hq] * kLog2e : 0.f;
    delta_s[threadIdx.x] = ok ? delta[at + (long long)threadIdx.x * P.Hq] : 0.f;
  }
  uint64_t aq[kR][D / 32] = {};
  const int seen = min(s.nk, s.pos0 + i0 + rows);
  // rows behind what is seen are zero: they must not meet a weight of zero as NaN
  auto load = [&](float* dst, const T* src, int j0) {
    if (j0 < seen)
      load_tile<D, kTile>(dst, src + ((long long)(s.k0 + j0) * P.Hkv + g) * D, kst,
                          min(kTile, seen - j0));
    else
      asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load(Vs, v, 0);
  load(Ks, k, 0);
  for (int j0 = 0; j0 < seen; j0 += kTile) {
    float sc[kR][4] = {}, dp[kR][4] = {};
    tile_wait<1>();  // V is there
    product_nt<D>(Gs, Vs, ty, tx, dp);
    tile_wait<0>();  // K is there, V read
    load(Vs, v, j0 + kTile);
    product_nt<D>(Qs, Ks, ty, tx, sc);
#pragma unroll
    for (int i = 0; i < kR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = ty + kTy * i, c = tx + 16 * j;
        const bool sees = r < rows && j0 + c <= s.pos0 + i0 + r;
        const float p = sees ? exp2f(sc[i][j] * (P.scale * kLog2e) - lse_s[r]) : 0.f;
        Ss[r * Smem<D>::kPPitch + c] = sees ? p * (dp[i][j] - delta_s[r]) : 0.f;
      }
    __syncthreads();
    product_nn<D>(Ss, Ks, ty, tx, aq);
    __syncthreads();  // K is read
    load(Ks, k, j0 + kTile);
  }
#pragma unroll
  for (int i = 0; i < kR; ++i) {
    const int r = ty + kTy * i;
    if (r >= rows) continue;
#pragma unroll
    for (int c = 0; c < D / 16; c += 4)
      store4(dq + (at + (long long)r * P.Hq) * D + tx * 4 + c * 16, &aq[i][c / 2], P.scale);
  }
}

template <typename T>
__global__ void __launch_bounds__(256)
dense_dkv_sum_kernel(const float* part, int splits, long long n, float scale,
                     T* __restrict__ dk, T* __restrict__ dv) {
  tc::griddep_wait();
  const long long i = ((long long)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  const int which = blockIdx.y;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < splits; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(part + (s * 2 + which) * n + i);
    sum.x += x.x;
    sum.y += x.y;
    sum.z += x.z;
    sum.w += x.w;
  }
  const float f = which ? scale : 1.f;
  T* dst = (which ? dk : dv) + i;
  dst[0] = from_f32<T>(sum.x * f);
  dst[1] = from_f32<T>(sum.y * f);
  dst[2] = from_f32<T>(sum.z * f);
  dst[3] = from_f32<T>(sum.w * f);
}

// ---------------------------------------------------------------------------
// Tree attention over a cache
// ---------------------------------------------------------------------------
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
tree_simt_kernel(Tree A, const T* __restrict__ q, const T* __restrict__ k,
                 const T* __restrict__ v, T* __restrict__ out, float* __restrict__ lse,
                 int32_t* __restrict__ status) {
  extern __shared__ float sm[];
  __shared__ uint8_t seen_s[kTile];  // a draft's row of this key tile is seen by some node
  const Dense& P = A.d;
  float* Qs = sm;
  float* Ks = Qs + Smem<D>::kRowFloats;
  float* Vs = Ks + Smem<D>::kTileFloats;
  float* Ps = Vs + Smem<D>::kTileFloats;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, nodes = P.Sq;
  const float sl2 = P.scale * kLog2e;
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < P.B; b += kThreads)
      if (A.kv_lens[b] < 0 || A.kv_lens[b] > P.Skv - nodes) atomicOr(status, kStatusBadLength);
  TreeWalk w;
  w.begin(A, blockIdx.x, gridDim.x);
  TreeWalk::Piece p;
  while (w.next(A, &p)) {
    const uint8_t* mask = A.mask + p.b * A.mask_stride;
    const int row0 = p.group * A.rows, rows = min(A.rows, nodes * P.G - row0);
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int r = i / (D / 4), c = (i % (D / 4)) * 4, node = (row0 + r) / P.G;
      float x[4] = {};
      if (r < rows)
        load_vec<T, 4>(q + (((long long)p.b * nodes + node) * P.Hq + p.g * P.G +
                            (row0 + r) % P.G) * D + c, x);
      *reinterpret_cast<float4*>(Qs + r * Smem<D>::kPitch + c) = make_float4(x[0], x[1], x[2], x[3]);
    }
    Running<D> R;
    R.clear();
    const int total = p.len + nodes;
    for (int j0 = p.kt0 * kDenseTile; j0 < min(total, p.kt1 * kDenseTile); j0 += kTile) {
      const long long row =
          tile_row(P, p.b, P.table ? 0 : p.b * P.Skv, j0 / kDenseTile) + (j0 % kDenseTile);
      if (P.table && threadIdx.x == 0) {
        const int pg = P.table[(long long)p.b * P.table_w + j0 / kDenseTile];
        if (pg < 0 || pg >= P.pages) atomicOr(status, kStatusBadPage);
      }
      const int valid = min(kTile, total - j0);
      const bool drafts = j0 + kTile > p.len;  // the tile reaches the drafted tokens
      __syncthreads();
      load_tile<D, kTile>(Ks, k + (row * P.Hkv + p.g) * D, (long long)P.Hkv * D, valid);
      load_tile<D, kTile>(Vs, v + (row * P.Hkv + p.g) * D, (long long)P.Hkv * D, valid);
      if (drafts && threadIdx.x < kTile) {
        const int j = j0 + int(threadIdx.x) - p.len;
        bool any = j < 0;
        for (int i = 0; i < nodes && j >= 0 && j < nodes; ++i) any |= mask[i * nodes + j] != 0;
        seen_s[threadIdx.x] = any;
      }
      tile_wait<0>();
      if (drafts) {  // a row that no node sees must not reach the products
        for (int i = threadIdx.x; i < kTile * D; i += kThreads)
          if (!seen_s[i / D]) Vs[i / D * Smem<D>::kPitch + i % D] = 0.f;
      }
      float sc[kR][4] = {};
      product_nt<D>(Qs, Ks, ty, tx, sc);
#pragma unroll
      for (int i = 0; i < kR; ++i) {
        const int node = min((row0 + ty + kTy * i) / P.G, nodes - 1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int draft = j0 + tx + 16 * j - p.len;
          const bool sees = draft < 0 || (draft < nodes && mask[node * nodes + draft] != 0);
          sc[i][j] = sees ? sc[i][j] * sl2 : -INFINITY;
        }
      }
      R.step(sc, Ps, ty, tx);
      __syncthreads();
      product_nn<D>(Ps, Vs, ty, tx, R.o);
    }
#pragma unroll
    for (int i = 0; i < kR; ++i) {
      const int r = ty + kTy * i;
      if (r >= rows) continue;
      if (p.slot >= 0) {
        const long long at = (long long)(blockIdx.x * 2 + p.slot) * A.rows;
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
          A.part_o[at * D + (tx * 4 + (c / 4) * 64 + c % 4) * A.rows + r] = part_of(R.o[i], c);
        if (tx == 0) A.part_ml[at + r] = make_float2(R.m[i], R.l[i]);
        continue;
      }
      const long long at = ((long long)p.b * nodes + (row0 + r) / P.G) * P.Hq + p.g * P.G +
                           (row0 + r) % P.G;
      const float inv = R.l[i] == 0.f ? 0.f : 1.f / R.l[i];
#pragma unroll
      for (int c = 0; c < D / 16; c += 4) store4(out + at * D + tx * 4 + c * 16, &R.o[i][c / 2], inv);
      if (lse && tx == 0) lse[at] = R.l[i] == 0.f ? -INFINITY : (R.m[i] + log2f(R.l[i])) * kLn2;
    }
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Merge of the partial states of units that a share's border cut: a thread per row (the
// partial outputs have rows innermost) and 8 columns; a block of 128 threads holds
// `rows` rows (a power of two) of one unit and as many groups of columns as fit.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 128;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
tree_combine_kernel(Tree A, int ctas, int rows, T* __restrict__ out, float* __restrict__ lse) {
  const Dense& P = A.d;
  const int nodes = P.Sq, per = P.Hkv * A.groups, blocks = max(1, D / 8 * rows / kJoinThreads);
  const int c0d = (blockIdx.x % blocks * (kJoinThreads / rows) + threadIdx.x / rows) * 8;
  const int unit = (blockIdx.x / blocks) % per;
  const int b = blockIdx.x / blocks / per, lane = threadIdx.x & 31;
  long long total = 0, before = 0;  // key tiles of all sequences, of those before b
  for (int i = lane; i < P.B; i += 32) {
    const int t = tree_seq(A, i).tiles;
    total += t;
    if (i < b) before += t;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    total += __shfl_xor_sync(MSA_FULL_MASK, total, o);
    before += __shfl_xor_sync(MSA_FULL_MASK, before, o);
  }
  const long long share = tree_share(total * per, ctas);
  const int n = tree_seq(A, b).tiles;
  const long long t0 = before * per + (long long)unit * n;
  const int c0 = int(t0 / share), c1 = int((t0 + n - 1) / share);
  tc::griddep_wait();  // the partial states are written
  if (c0 == c1) return;
  const int g = unit / A.groups, row0 = (unit % A.groups) * A.rows, r = threadIdx.x % rows;
  if (r >= min(A.rows, nodes * P.G - row0) || c0d >= D) return;
  // Four pieces' loads at a time: the join is a few round trips to L2 long.  The unit's
  // first piece lies in c0's slot 1, the others in their CTA's slot 0.
  float m = -INFINITY, o[8] = {}, l = 0.f;
  for (int c = c0; c <= c1; c += 4) {
    float2 ml[4];
    float x[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const bool there = c + u <= c1;
      const long long at = (long long)(2 * (there ? c + u : c) + (c + u == c0 ? 1 : 0)) * A.rows;
      const float* src = A.part_o + at * D + (long long)c0d * A.rows + r;
      ml[u] = there ? A.part_ml[at + r] : make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u][i] = there ? src[i * A.rows] : 0.f;
    }
    float top = m;
#pragma unroll
    for (int u = 0; u < 4; ++u) top = fmaxf(top, ml[u].x);
    const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m - base);
    m = top;
    l *= keep;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= keep;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float w = exp2f(ml[u].x - base);
      l += w * ml[u].y;
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] += w * x[u][i];
    }
  }
  const long long row = ((long long)b * nodes + (row0 + r) / P.G) * P.Hq + g * P.G + (row0 + r) % P.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  T* dst = out + row * D + c0d;
  constexpr int vec = 16 / int(sizeof(T));
#pragma unroll
  for (int i = 0; i < 8; i += vec) {
    uint4 u;
    T* e = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int x = 0; x < vec; ++x) e[x] = from_f32<T>(o[i + x] * inv);
    *reinterpret_cast<uint4*>(dst + i) = u;
  }
  if (lse && c0d == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

namespace {

template <typename K>
cudaError_t allow_smem(K kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
}

template <typename T, int D>
cudaError_t fwd(const Dense& P, const void* q, const void* k, const void* v, void* out, float* lse,
                cudaStream_t s) {
  cudaError_t e = allow_smem(dense_fwd_simt_kernel<T, D>, fwd_smem<D>());
  if (e != cudaSuccess) return e;
  dense_fwd_simt_kernel<T, D><<<unsigned(P.qtiles) * kParts * P.Hq, kThreads, fwd_smem<D>(), s>>>(
      P, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
      static_cast<T*>(out), lse);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t bwd(const Dense& P, const void* dout, const void* q, const void* k, const void* v,
                const void* out, const float* lse, const DenseBwdSpace& W, void* dq, void* dk,
                void* dv, cudaStream_t s) {
  cudaError_t e = allow_smem(dense_dkv_simt_kernel<T, D>, dkv_smem<D>());
  if (e == cudaSuccess) e = allow_smem(dense_dq_simt_kernel<T, D>, dq_smem<D>());
  if (e != cudaSuccess) return e;
  const long long n = P.rows_q * P.Hq;
  const T *g_ = static_cast<const T*>(dout), *q_ = static_cast<const T*>(q);
  const T *k_ = static_cast<const T*>(k), *v_ = static_cast<const T*>(v);
  T *dk_ = static_cast<T*>(dk), *dv_ = static_cast<T*>(dv);
  if (n > 0)
    dense_delta_kernel<T, D><<<unsigned((n + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s>>>(
        g_, static_cast<const T*>(out), W.dl, n);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int splits = dense_bwd_splits(P);
  dense_dkv_simt_kernel<T, D>
      <<<unsigned(P.ktiles) * kParts * P.Hkv * splits, kThreads, dkv_smem<D>(), s>>>(
          P, splits, g_, q_, k_, v_, lse, W.dl, dk_, dv_, W.part);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (splits > 1) e = launch_dkv_sum(W.part, splits, P.rows_k * P.Hkv * D, P.scale, dk_, dv_, s);
  if (e != cudaSuccess) return e;
  if (P.qtiles > 0)
    dense_dq_simt_kernel<T, D><<<unsigned(P.qtiles) * kParts * P.Hq, kThreads, dq_smem<D>(), s>>>(
        P, g_, q_, k_, v_, lse, W.dl, static_cast<T*>(dq));
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t tree(const Tree& A, const void* q, const void* k, const void* v, void* out, float* lse,
                 int32_t* status, cudaStream_t s) {
  cudaError_t e = allow_smem(tree_simt_kernel<T, D>, fwd_smem<D>());
  if (e != cudaSuccess) return e;
  tree_simt_kernel<T, D><<<tree_ctas(A.d.f32), kThreads, fwd_smem<D>(), s>>>(
      A, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v),
      static_cast<T*>(out), lse, status);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  return launch_tree_combine(A, out, lse, s);
}

}  // namespace

cudaError_t launch_tree_combine(const Tree& A, void* out, float* lse, cudaStream_t s) {
  int rows = 8;
  while (rows < std::min(A.rows, A.d.Sq * A.d.G)) rows *= 2;
  const long long blocks = (long long)A.d.B * A.d.Hkv * A.groups *
                           std::max(1, A.d.D / 8 * rows / kJoinThreads);
  const int ctas = tree_ctas(A.d.f32);
  if (A.d.f32) {
    auto kern = A.d.D == 128 ? tree_combine_kernel<float, 128> : tree_combine_kernel<float, 64>;
    return launch_after(kern, unsigned(blocks), kJoinThreads, 0, s, A, ctas, rows,
                        static_cast<float*>(out), lse);
  } else {
    auto kern = A.d.D == 128 ? tree_combine_kernel<__nv_bfloat16, 128>
                             : tree_combine_kernel<__nv_bfloat16, 64>;
    return launch_after(kern, unsigned(blocks), kJoinThreads, 0, s, A, ctas, rows,
                        static_cast<__nv_bfloat16*>(out), lse);
  }
}

// bf16 problems run on the tensor cores: only fp32 comes here.
cudaError_t launch_dense_fwd_simt(const Dense& P, const void* q, const void* k, const void* v,
                                  void* out, float* lse, cudaStream_t s) {
  return (P.D == 128 ? fwd<float, 128> : fwd<float, 64>)(P, q, k, v, out, lse, s);
}

cudaError_t launch_dense_bwd_simt(const Dense& P, const void* dout, const void* q, const void* k,
                                  const void* v, const void* out, const float* lse,
                                  const DenseBwdSpace& W, void* dq, void* dk, void* dv,
                                  cudaStream_t s) {
  return (P.D == 128 ? bwd<float, 128> : bwd<float, 64>)(P, dout, q, k, v, out, lse, W, dq, dk, dv,
                                                         s);
}

cudaError_t launch_tree_simt(const Tree& A, const void* q, const void* k, const void* v, void* out,
                             float* lse, int32_t* status, cudaStream_t s) {
  return (A.d.D == 128 ? tree<float, 128> : tree<float, 64>)(A, q, k, v, out, lse, status, s);
}

// The heads of a group are split over several items where there would otherwise be
// fewer than three items (tensor cores; 128 keys each) or four blocks (32 keys each) per
// SM to balance the load with; each split costs one more write and read of dk and dv in
// fp32.
int dense_bwd_splits(const Dense& P) {
  const long long items = (long long)P.ktiles * P.Hkv * (P.f32 ? kParts : 1);
  int n = 1;
  while (n < P.G && items * n < (P.f32 ? 4LL : 3LL) * 148) n *= 2;
  return std::min(n, P.G);
}

template <typename T>
cudaError_t launch_dkv_sum(const float* part, int splits, long long n, float scale, T* dk, T* dv,
                           cudaStream_t s) {
  return launch_after(dense_dkv_sum_kernel<T>, dim3(unsigned((n / 4 + 255) / 256), 2), 256, 0, s,
                      part, splits, n, scale, dk, dv);
}
template cudaError_t launch_dkv_sum(const float*, int, long long, float, float*, float*,
                                    cudaStream_t);
template cudaError_t launch_dkv_sum(const float*, int, long long, float, __nv_bfloat16*,
                                    __nv_bfloat16*, cudaStream_t);

}  // namespace msa
