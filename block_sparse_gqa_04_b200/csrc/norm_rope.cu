// RMS norm of query and key heads with the position rotation in the same pass,
// and its gradients.
//
// A head row x of D elements becomes y = w x r, r = (mean x^2 + eps)^-1/2, and its
// first rot elements turn pairwise by f = position * inv_freq.  Backward, with the
// rotation undone on the incoming gradient (its transpose): g, u = r x, t = w g,
//   dw = sum g u,   dx = r (t - u mean(t u)).
//
// Both directions read and write every element once and are bound by HBM, if little
// enough else goes through the load/store pipe: shuffles and shared-memory reads were the
// bound while a row's lanes held neighbouring elements and fetched the partners of their
// pairs (2.6 TB/s).  So a thread holds both elements of its pairs: of D / 16 lanes per
// row, each has two chunks of 8 elements, a chunk of the first half of the rotated part
// and its partner in the second (or two neighbours, where pairs are adjacent or nothing
// is rotated).  Its 8 angles are the same for all heads of a token: it keeps them in
// registers and walks the heads, the next rows' loads in flight.  The angles are formed
// once per block and token, in fp64 (positions x frequencies reach 10^6 turns, where fp32
// keeps no fraction), reduced to a quarter turn before the fp32 sine and cosine.  Blocks
// take query heads or key heads, so that a thread needs one set of weights and sums.
// 32768 tokens x 68 heads x 128: 0.212 ms, 5.4 TB/s; gradients of 8191 tokens 82 us, 5.2
// TB/s, and 6 us for the sum of the blocks' weight gradients.
#include "common.cuh"
#include "dense.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxHalf = 64;  // rotated pairs of a head
constexpr int kTokens = 32;   // tokens of a block at a time, at most

// cos and sin of position * freq: turns reduced in fp64, then at most a quarter
// turn in fp32.
__device__ __forceinline__ float2 cos_sin(long long pos, double freq) {
  const double quarters = double(pos) * freq * 0.63661977236758134308;  // 2 / pi
  const double k = rint(quarters);
  float s, c;
  sincospif(0.5f * float(quarters - k), &s, &c);
  const int quad = int((long long)k & 3);
  const float cc = (quad & 1) ? s : c, ss = (quad & 1) ? c : s;
  // quadrant 0: (c, s), 1: (-s, c), 2: (-c, -s), 3: (s, -c)
  return make_float2((quad == 1 || quad == 2) ? -cc : cc, quad >= 2 ? -ss : ss);
}

// A thread's part of a row: elements a .. a+7 and b .. b+7.
struct Place {
  int a, b;
  bool turned;  // they are rotated, by the angles 8 * lane .. 8 * lane + 7
};

__device__ __forceinline__ Place place_of(int lane, int rot, bool inter) {
  if (inter) return Place{16 * lane, 16 * lane + 8, 16 * lane < rot};
  if (16 * lane < rot) return Place{8 * lane, 8 * lane + rot / 2, true};
  return Place{16 * lane, 16 * lane + 8, false};
}

// 16 elements of a row, as stored.
template <typename T>
struct Raw {
  static constexpr int kWords = int(sizeof(T));  // 16-byte words of 16 elements: 2 or 4
  uint4 w[kWords];
  __device__ __forceinline__ void load(const T* row, const Place& p) {
#pragma unroll
    for (int i = 0; i < kWords / 2; ++i) {
      w[i] = *reinterpret_cast<const uint4*>(row + p.a + i * (16 / sizeof(T)));
      w[kWords / 2 + i] = *reinterpret_cast<const uint4*>(row + p.b + i * (16 / sizeof(T)));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(T* row, const Place& p) const {
#pragma unroll
    for (int i = 0; i < kWords / 2; ++i) {
      *reinterpret_cast<uint4*>(row + p.a + i * (16 / sizeof(T))) = w[i];
      *reinterpret_cast<uint4*>(row + p.b + i * (16 / sizeof(T))) = w[kWords / 2 + i];
    }
  }
  __device__ __forceinline__ float get(int i) const {  // i: a constant
    return to_f32(reinterpret_cast<const T*>(w)[i]);
  }
  __device__ __forceinline__ void set(int i, float x) {
    reinterpret_cast<T*>(w)[i] = from_f32<T>(x);
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(MSA_FULL_MASK, v, o);
  return v;
}

// Turns y (elements a.. and b.. of a row) by the angles cs, or back with sign -1.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&y)[16], const float2 (&cs)[8], float sign) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int u = INTER ? 2 * i : i, v = INTER ? 2 * i + 1 : i + 8;
    const float a = y[u], b = y[v], s = sign * cs[i].y;
    y[u] = a * cs[i].x - b * s;
    y[v] = b * cs[i].x + a * s;
  }
}

// Angles of a block's tokens, of which nt are there.  The others get no turn: what the
// memory held may be NaN, which times their rows of zeros would reach the weights' gradients.
__device__ __forceinline__ void fill_angles(float2 (*cs)[kMaxHalf], long long t0, int nt,
                                            int tokens, int half, const double* inv_freq,
                                            const int64_t* pos) {
  for (int i = threadIdx.x; i < tokens * half; i += kThreads) {
    const int t = i / half, f = i % half;
    cs[t][f] = t < nt ? cos_sin(pos[t0 + t], inv_freq[f]) : make_float2(1.f, 0.f);
  }
}

// A thread's angles of token `tok`; no turn where nothing is rotated.
__device__ __forceinline__ void my_angles(float2 (&a)[8], const float2 (*cs)[kMaxHalf], int tok,
                                          int lane, bool turned) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = turned ? cs[tok][8 * lane + i] : make_float2(1.f, 0.f);
}

// How the query heads (or the key heads) are cut: `tokens` tokens at a time, `span` heads
// of them (in `chunks` parts), `blocks` blocks that share all of it.
struct Cut {
  int heads, tokens, span, chunks;
  long long sets;  // ceil(rows / tokens) * chunks
  int blocks;
};

template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3)
norm_rope_kernel(NormRope P, Cut cq, Cut ck, const T* q, const T* k, const T* qw, const T* kw,
                 const double* inv_freq, const int64_t* pos, T* qo, T* ko) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  __shared__ float2 cs[kTokens][kMaxHalf];
  const bool isq = int(blockIdx.x) < cq.blocks;
  const Cut c = isq ? cq : ck;
  const T* src = isq ? q : k;
  T* dst = isq ? qo : ko;
  const long long ss = isq ? P.qs : P.ks, ds = isq ? P.qos : P.kos;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int per = kGroups / c.tokens, tok = group / per, g = group % per;
  const Place at = place_of(lane, P.rot, INTER);
  float w[16];
  {
    Raw<T> x;
    x.load(isq ? qw : kw, at);
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = x.get(i);
  }
  bool first = true;
  for (long long set = isq ? blockIdx.x : blockIdx.x - cq.blocks; set < c.sets; set += c.blocks) {
    const long long t0 = set / c.chunks * c.tokens, r = t0 + tok;
    const int h0 = int(set % c.chunks) * c.span, h1 = min(c.heads, h0 + c.span);
    const int nt = int(min((long long)c.tokens, P.rows - t0));
    const bool there = tok < nt;
    auto fetch = [&](int base, Raw<T>& x) {
      const int h = base + g;
      if (there && h < h1) x.load(src + r * ss + h * D, at); else x.clear();
    };
    Raw<T> cur, nxt;
    fetch(h0, cur);  // the angles are formed under the first loads
    if (!first) __syncthreads();
    first = false;
    fill_angles(cs, t0, nt, c.tokens, P.rot >> 1, inv_freq, pos);
    __syncthreads();
    float2 ang[8];
    my_angles(ang, cs, tok, lane, at.turned);
    for (int base = h0; base < h1; base += per) {
      fetch(base + per, nxt);
      float x[16], sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = cur.get(i);
        sum += x[i] * x[i];
      }
      const float rr = rsqrtf(row_sum<kLanes>(sum) * (1.f / D) + P.eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = x[i] * rr * w[i];
      rotate<INTER>(x, ang, 1.f);
#pragma unroll
      for (int i = 0; i < 16; ++i) cur.set(i, x[i]);
      if (there && base + g < h1) cur.store(dst + r * ds + (base + g) * D, at);
      cur = nxt;
    }
  }
}

// Gradients; part[block][D] receives the block's sums of its weight's gradient.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2)
norm_rope_backward_kernel(NormRope P, Cut cq, Cut ck, const T* gq, const T* gk, const T* q,
                          const T* k, const T* qw, const T* kw, const double* inv_freq,
                          const int64_t* pos, T* dq, T* dk, float* part) {
  constexpr int kLanes = D / 16, kGroups = kThreads / kLanes;
  __shared__ float2 cs[kTokens][kMaxHalf];
  __shared__ float sums[kGroups][D];
  const bool isq = int(blockIdx.x) < cq.blocks;
  const Cut c = isq ? cq : ck;
  const T *src = isq ? q : k, *gsrc = isq ? gq : gk;
  T* dst = isq ? dq : dk;
  const long long ss = isq ? P.qs : P.ks, gs = isq ? P.qos : P.kos, ds = isq ? P.dqs : P.dks;
  const int lane = threadIdx.x % kLanes, group = threadIdx.x / kLanes;
  const int per = kGroups / c.tokens, tok = group / per, g = group % per;
  const Place at = place_of(lane, P.rot, INTER);
  float w[16], acc[16];
  {
    Raw<T> x;
    x.load(isq ? qw : kw, at);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w[i] = x.get(i);
      acc[i] = 0.f;
    }
  }
  for (long long set = isq ? blockIdx.x : blockIdx.x - cq.blocks; set < c.sets; set += c.blocks) {
    const long long t0 = set / c.chunks * c.tokens, r = t0 + tok;
    const int h0 = int(set % c.chunks) * c.span, h1 = min(c.heads, h0 + c.span);
    const int nt = int(min((long long)c.tokens, P.rows - t0));
    const bool there = tok < nt;
    auto fetch = [&](int base, Raw<T>& x, Raw<T>& y) {
      const int h = base + g;
      if (there && h < h1) {
        x.load(src + r * ss + h * D, at);
        y.load(gsrc + r * gs + h * D, at);
      } else {
        x.clear();  // adds nothing to the sums
        y.clear();
      }
    };
    Raw<T> cx, cg, nx, ng;
    fetch(h0, cx, cg);
    __syncthreads();  // the previous tokens' angles are read
    fill_angles(cs, t0, nt, c.tokens, P.rot >> 1, inv_freq, pos);
    __syncthreads();
    float2 ang[8];
    my_angles(ang, cs, tok, lane, at.turned);
    for (int base = h0; base < h1; base += per) {
      fetch(base + per, nx, ng);
      float x[16], y[16], sum = 0.f, tu = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] = cx.get(i);
        y[i] = cg.get(i);
        sum += x[i] * x[i];
      }
      const float mean = row_sum<kLanes>(sum) * (1.f / D);
      // a row that is not there adds nothing (eps may be 0)
      const float rr = there && base + g < h1 ? rsqrtf(mean + P.eps) : 0.f;
      rotate<INTER>(y, ang, -1.f);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[i] *= rr;
        acc[i] += y[i] * x[i];
        y[i] *= w[i];
        tu += y[i] * x[i];
      }
      const float m = row_sum<kLanes>(tu) * (1.f / D);
#pragma unroll
      for (int i = 0; i < 16; ++i) cx.set(i, rr * (y[i] - x[i] * m));
      if (there && base + g < h1) cx.store(dst + r * ds + (base + g) * D, at);
      cx = nx;
      cg = ng;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) sums[group][i < 8 ? at.a + i : at.b + i - 8] = acc[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float s = 0.f;
    for (int x = 0; x < kGroups; ++x) s += sums[x][threadIdx.x];
    part[(long long)blockIdx.x * D + threadIdx.x] = s;
  }
}

// dw[d] = sum over blocks of part[block][d], in a fixed order: 32 columns of one weight
// per block (blockIdx.x: query or key heads, y: columns).
__global__ void __launch_bounds__(1024)
norm_rope_weights_kernel(const float* part, int blocks_q, int blocks_k, int D, float* dqw,
                         float* dkw) {
  __shared__ double sums[32][32];
  float* dst = blockIdx.x ? dkw : dqw;
  const int c = threadIdx.x & 31, lane = threadIdx.x >> 5, d = blockIdx.y * 32 + c;
  const int n = blockIdx.x ? blocks_k : blocks_q;
  if (blockIdx.x) part += (long long)blocks_q * D;
  double s = 0.0;
#pragma unroll 8
  for (int b = lane; b < n; b += 32) s += part[(long long)b * D + d];
  sums[lane][c] = s;
  __syncthreads();
  if (lane == 0 && dst) {
    for (int l = 1; l < 32; ++l) s += sums[l][c];
    dst[d] = float(s);
  }
}

// Few tokens: one at a time and a block per row group, so that every row is its own
// thread group's (32 tokens x 68 heads 2.9 us, against 3.8 with four tokens a block); many:
// enough that a thread walks several heads of its token with the next row's load in flight
// (32768 tokens 0.212 ms, against 0.288 with four tokens and loads in batches).
Cut cut_of(long long rows, int heads, int D, int max_blocks) {
  const int groups = kThreads / (D / 16);
  Cut c{};
  c.heads = heads;
  if (heads == 0) return c;
  c.tokens = rows <= 148 * 8 ? 1 : heads >= 32 ? 8 : 32;
  c.span = c.tokens == 1 ? groups : heads;
  c.chunks = (heads + c.span - 1) / c.span;
  c.sets = (rows + c.tokens - 1) / c.tokens * c.chunks;
  c.blocks = int(min(c.sets, (long long)max_blocks));
  return c;
}

template <typename T, int D>
cudaError_t forward(const NormRope& P, const void* q, const void* k, const void* qw,
                    const void* kw, const double* f, const int64_t* pos, void* qo, void* ko,
                    cudaStream_t s) {
  const Cut cq = cut_of(P.rows, P.hq, D, 1 << 30), ck = cut_of(P.rows, P.hk, D, 1 << 30);
  auto kern = P.inter ? norm_rope_kernel<T, D, true> : norm_rope_kernel<T, D, false>;
  kern<<<unsigned(cq.blocks + ck.blocks), kThreads, 0, s>>>(
      P, cq, ck, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(qw),
      static_cast<const T*>(kw), f, pos, static_cast<T*>(qo), static_cast<T*>(ko));
  return cudaGetLastError();
}

// Blocks of the backward pass: each leaves one partial sum per weight.
constexpr int kBackwardBlocks = 148 * 8;

template <typename T, int D>
cudaError_t backward(const NormRope& P, const void* gq, const void* gk, const void* q,
                     const void* k, const void* qw, const void* kw, const double* f,
                     const int64_t* pos, void* dq, void* dk, float* dqw, float* dkw, float* part,
                     cudaStream_t s) {
  const Cut cq = cut_of(P.rows, P.hq, D, kBackwardBlocks);
  const Cut ck = cut_of(P.rows, P.hk, D, kBackwardBlocks);
  auto kern = P.inter ? norm_rope_backward_kernel<T, D, true>
                      : norm_rope_backward_kernel<T, D, false>;
  kern<<<cq.blocks + ck.blocks, kThreads, 0, s>>>(
      P, cq, ck, static_cast<const T*>(gq), static_cast<const T*>(gk), static_cast<const T*>(q),
      static_cast<const T*>(k), static_cast<const T*>(qw), static_cast<const T*>(kw), f, pos,
      static_cast<T*>(dq), static_cast<T*>(dk), part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_rope_weights_kernel<<<dim3(P.hk ? 2 : 1, D / 32), 1024, 0, s>>>(part, cq.blocks, ck.blocks,
                                                                       D, dqw, dkw);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_partials(const NormRope& P) {
  return cut_of(P.rows, P.hq, P.D, kBackwardBlocks).blocks +
         cut_of(P.rows, P.hk, P.D, kBackwardBlocks).blocks;
}

cudaError_t launch_norm_rope(const NormRope& P, const void* q, const void* k, const void* qw,
                             const void* kw, const double* f, const int64_t* pos, void* qo,
                             void* ko, cudaStream_t s) {
  auto fn = P.f32 ? (P.D == 128  ? forward<float, 128>
                     : P.D == 64 ? forward<float, 64>
                                 : forward<float, 32>)
                  : (P.D == 128  ? forward<__nv_bfloat16, 128>
                     : P.D == 64 ? forward<__nv_bfloat16, 64>
                                 : forward<__nv_bfloat16, 32>);
  return fn(P, q, k, qw, kw, f, pos, qo, ko, s);
}

cudaError_t launch_norm_rope_backward(const NormRope& P, const void* gq, const void* gk,
                                      const void* q, const void* k, const void* qw,
                                      const void* kw, const double* f, const int64_t* pos,
                                      void* dq, void* dk, float* dqw, float* dkw, float* part,
                                      cudaStream_t s) {
  auto fn = P.f32 ? (P.D == 128  ? backward<float, 128>
                     : P.D == 64 ? backward<float, 64>
                                 : backward<float, 32>)
                  : (P.D == 128  ? backward<__nv_bfloat16, 128>
                     : P.D == 64 ? backward<__nv_bfloat16, 64>
                                 : backward<__nv_bfloat16, 32>);
  return fn(P, gq, gk, q, k, qw, kw, f, pos, dq, dk, dqw, dkw, part, s);
}

}  // namespace msa
