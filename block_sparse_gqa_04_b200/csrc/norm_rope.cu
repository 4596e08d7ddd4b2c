// RMS norm of query and key heads with the position rotation in the same pass,
// and its gradients.
//
// A head row x of D elements becomes y = w x r, r = (mean x^2 + eps)^-1/2, and its
// first rot elements turn pairwise by f = position * inv_freq.  Backward, with the
// rotation undone on the incoming gradient (its transpose): g, u = r x, t = w g,
//   dw = sum g u,   dx = r (t - u mean(t u)).
//
// Both directions read and write every element once and are bound by HBM.  A row
// is held by D / (16 bytes) neighbouring lanes, 16 bytes each, so its sums and the
// partners of its pairs are a few shuffles away and nothing but the angles goes
// through shared memory; a thread has kUnroll rows' loads in flight.  The angles
// of a token are the same for all its heads: a block takes all heads of a few
// tokens and forms them once, in fp64 (positions x frequencies reach 10^6 turns,
// where fp32 keeps no fraction), reduced to a quarter turn before the fp32 sine
// and cosine.
#include "common.cuh"
#include "dense.h"

namespace msa {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;
constexpr int kMaxHalf = 64;  // rotated pairs of a head
// Tokens of a block: one for a decode step's few rows, where every block counts,
// else enough rows to fill the unrolled loop.
constexpr int kTokens = 4;

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

template <typename T, int D>
struct Shape {
  static constexpr int kVec = 16 / int(sizeof(T));
  static constexpr int kLanes = D / kVec;          // lanes of a row
  static constexpr int kSlots = kThreads / kLanes;  // rows of a block at a time
};

template <int N, int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(MSA_FULL_MASK, v, o);
  return v;
}

template <typename T, int N>
__device__ __forceinline__ void widen(const uint4& u, float (&x)[N]) {
  const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
}

template <typename T, int N>
__device__ __forceinline__ uint4 narrow(const float (&x)[N]) {
  uint4 u;
  T* e = reinterpret_cast<T*>(&u);
#pragma unroll
  for (int i = 0; i < N; ++i) e[i] = from_f32<T>(x[i]);
  return u;
}

// Turns this lane's elements e0 .. e0+N-1 of a row by the angles cs (sign -1: back).
// Every lane of the warp takes part.
template <int N>
__device__ __forceinline__ void rotate(float (&y)[N], int e0, int rot, bool inter,
                                       const float2* cs, float sign) {
  if (rot == 0) return;
  if (inter) {
    if (e0 < rot) {
#pragma unroll
      for (int i = 0; i < N; i += 2) {
        const float2 f = cs[(e0 + i) >> 1];
        const float a = y[i], b = y[i + 1], s = sign * f.y;
        y[i] = a * f.x - b * s;
        y[i + 1] = b * f.x + a * s;
      }
    }
    return;
  }
  const int half = rot >> 1, lane = threadIdx.x & 31;
  const bool first = e0 < half, turned = e0 < rot;
  const int other = turned ? (first ? lane + half / N : lane - half / N) : lane;
  // first half: a cos - b sin with b the partner; second: b cos + a sin
  const float s0 = first ? -sign : sign;
  const int i0 = first ? e0 : e0 - half;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float p = __shfl_sync(MSA_FULL_MASK, y[i], other);
    if (turned) {
      const float2 f = cs[i0 + i];
      y[i] = y[i] * f.x + p * (s0 * f.y);
    }
  }
}

__device__ __forceinline__ void fill_angles(float2 (*cs)[kMaxHalf], long long t0, int nt, int half,
                                            const double* inv_freq, const int64_t* pos) {
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, f = i % half;
    cs[t][f] = cos_sin(pos[t0 + t], inv_freq[f]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
norm_rope_kernel(NormRope P, int tokens, const T* q, const T* k, const T* qw, const T* kw,
                 const double* inv_freq, const int64_t* pos, T* qo, T* ko) {
  using S = Shape<T, D>;
  __shared__ float2 cs[kTokens][kMaxHalf];
  const long long t0 = (long long)blockIdx.x * tokens;
  const int nt = int(min((long long)tokens, P.rows - t0));
  const int heads = P.hq + P.hk, items = nt * heads;
  const int slot = threadIdx.x / S::kLanes, e0 = (threadIdx.x % S::kLanes) * S::kVec;
  fill_angles(cs, t0, nt, P.rot >> 1, inv_freq, pos);
  float wq[S::kVec], wk[S::kVec];
  load_vec<T, S::kVec>(qw + e0, wq);
  if (P.hk) load_vec<T, S::kVec>(kw + e0, wk);
  __syncthreads();
  for (int base = 0; base < items; base += S::kSlots * kUnroll) {
    uint4 raw[kUnroll];
    int tok[kUnroll], head[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int it = base + u * S::kSlots + slot;
      tok[u] = it < items ? it / heads : -1;
      head[u] = it - max(tok[u], 0) * heads;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (tok[u] >= 0) {
        const long long r = t0 + tok[u];
        const T* src = head[u] < P.hq ? q + r * P.qs + head[u] * D
                                      : k + r * P.ks + (head[u] - P.hq) * D;
        raw[u] = *reinterpret_cast<const uint4*>(src + e0);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (base + u * S::kSlots >= items) break;
      float x[S::kVec], ss = 0.f;
      widen<T>(raw[u], x);
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) ss += x[i] * x[i];
      const float r = rsqrtf(row_sum<S::kVec, S::kLanes>(ss) * (1.f / D) + P.eps);
      const bool isq = head[u] < P.hq;
#pragma unroll
      for (int i = 0; i < S::kVec; ++i) x[i] = x[i] * r * (isq ? wq[i] : wk[i]);
      rotate(x, e0, P.rot, P.inter, cs[max(tok[u], 0)], 1.f);
      if (tok[u] >= 0) {
        const long long row = t0 + tok[u];
        T* dst = isq ? qo + row * P.qos + head[u] * D : ko + row * P.kos + (head[u] - P.hq) * D;
        *reinterpret_cast<uint4*>(dst + e0) = narrow<T>(x);
      }
    }
  }
}

// Gradients; part[block][2][D] receives the block's sums of the weights' gradients.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
norm_rope_backward_kernel(NormRope P, int tokens, const T* gq, const T* gk, const T* q, const T* k,
                          const T* qw, const T* kw, const double* inv_freq, const int64_t* pos,
                          T* dq, T* dk, float* part) {
  using S = Shape<T, D>;
  constexpr int kLoads = 2;  // rows in flight per thread, two loads each
  __shared__ float2 cs[kTokens][kMaxHalf];
  __shared__ float sums[S::kSlots][D];
  const int heads = P.hq + P.hk;
  const int slot = threadIdx.x / S::kLanes, e0 = (threadIdx.x % S::kLanes) * S::kVec;
  float wq[S::kVec], wk[S::kVec], aq[S::kVec], ak[S::kVec];
  load_vec<T, S::kVec>(qw + e0, wq);
  if (P.hk) load_vec<T, S::kVec>(kw + e0, wk);
#pragma unroll
  for (int i = 0; i < S::kVec; ++i) aq[i] = ak[i] = 0.f;
  for (long long t0 = (long long)blockIdx.x * tokens; t0 < P.rows;
       t0 += (long long)gridDim.x * tokens) {
    const int nt = int(min((long long)tokens, P.rows - t0));
    const int items = nt * heads;
    __syncthreads();  // the previous tokens' angles are read
    fill_angles(cs, t0, nt, P.rot >> 1, inv_freq, pos);
    __syncthreads();
    for (int base = 0; base < items; base += S::kSlots * kLoads) {
      uint4 rx[kLoads], rg[kLoads];
      int tok[kLoads], head[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int it = base + u * S::kSlots + slot;
        tok[u] = it < items ? it / heads : -1;
        head[u] = it - max(tok[u], 0) * heads;
        rx[u] = rg[u] = make_uint4(0, 0, 0, 0);
        if (tok[u] >= 0) {
          const long long r = t0 + tok[u];
          const bool isq = head[u] < P.hq;
          const int h = (isq ? head[u] : head[u] - P.hq) * D + e0;
          rx[u] = *reinterpret_cast<const uint4*>((isq ? q + r * P.qs : k + r * P.ks) + h);
          rg[u] = *reinterpret_cast<const uint4*>((isq ? gq + r * P.qos : gk + r * P.kos) + h);
        }
      }
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        if (base + u * S::kSlots >= items) break;
        const bool isq = head[u] < P.hq;
        float x[S::kVec], g[S::kVec], ss = 0.f, tu = 0.f;
        widen<T>(rx[u], x);
        widen<T>(rg[u], g);
#pragma unroll
        for (int i = 0; i < S::kVec; ++i) ss += x[i] * x[i];
        const float r = rsqrtf(row_sum<S::kVec, S::kLanes>(ss) * (1.f / D) + P.eps);
        rotate(g, e0, P.rot, P.inter, cs[max(tok[u], 0)], -1.f);
#pragma unroll
        for (int i = 0; i < S::kVec; ++i) {
          x[i] *= r;
          const float gu = tok[u] >= 0 ? g[i] * x[i] : 0.f;
          if (isq) aq[i] += gu; else ak[i] += gu;
          g[i] *= isq ? wq[i] : wk[i];
          tu += g[i] * x[i];
        }
        const float m = row_sum<S::kVec, S::kLanes>(tu) * (1.f / D);
#pragma unroll
        for (int i = 0; i < S::kVec; ++i) x[i] = r * (g[i] - x[i] * m);
        if (tok[u] >= 0) {
          const long long row = t0 + tok[u];
          T* dst = isq ? dq + row * P.dqs + head[u] * D : dk + row * P.dks + (head[u] - P.hq) * D;
          *reinterpret_cast<uint4*>(dst + e0) = narrow<T>(x);
        }
      }
    }
  }
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::kVec; ++i) sums[slot][e0 + i] = which ? ak[i] : aq[i];
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
      for (int r = 0; r < S::kSlots; ++r) s += sums[r][threadIdx.x];
      part[((long long)blockIdx.x * 2 + which) * D + threadIdx.x] = s;
    }
  }
}

// dw[which][d] = sum over blocks of part[block][which][d], in a fixed order.
__global__ void __launch_bounds__(1024)
norm_rope_weights_kernel(const float* part, int blocks, int D, float* dqw, float* dkw) {
  __shared__ double sums[1024];
  float* dst = blockIdx.x ? dkw : dqw;
  const int d = threadIdx.x % D, lane = threadIdx.x / D, lanes = 1024 / D;
  double s = 0.0;
  for (int b = lane; b < blocks; b += lanes) s += part[((long long)b * 2 + blockIdx.x) * D + d];
  sums[threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.x < D && dst) {
    for (int l = 1; l < lanes; ++l) s += sums[l * D + d];
    dst[d] = float(s);
  }
}

// A block per token until every SM has several, then kTokens each.
int tokens_per_block(long long rows) { return rows <= 148 * 8 ? 1 : kTokens; }

template <typename T, int D>
cudaError_t forward(const NormRope& P, const void* q, const void* k, const void* qw,
                    const void* kw, const double* f, const int64_t* pos, void* qo, void* ko,
                    cudaStream_t s) {
  const int tok = tokens_per_block(P.rows);
  norm_rope_kernel<T, D><<<unsigned((P.rows + tok - 1) / tok), kThreads, 0, s>>>(
      P, tok, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(qw),
      static_cast<const T*>(kw), f, pos, static_cast<T*>(qo), static_cast<T*>(ko));
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t backward(const NormRope& P, const void* gq, const void* gk, const void* q,
                     const void* k, const void* qw, const void* kw, const double* f,
                     const int64_t* pos, void* dq, void* dk, float* dqw, float* dkw, float* part,
                     cudaStream_t s) {
  const int blocks = norm_rope_partials(P);
  norm_rope_backward_kernel<T, D><<<blocks, kThreads, 0, s>>>(
      P, tokens_per_block(P.rows), static_cast<const T*>(gq), static_cast<const T*>(gk),
      static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(qw),
      static_cast<const T*>(kw), f, pos, static_cast<T*>(dq), static_cast<T*>(dk), part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_rope_weights_kernel<<<2, 1024, 0, s>>>(part, blocks, D, dqw, P.hk ? dkw : nullptr);
  return cudaGetLastError();
}

}  // namespace

int norm_rope_partials(const NormRope& P) {
  const int tok = tokens_per_block(P.rows);
  return int(min((P.rows + tok - 1) / tok, 148LL * 6));
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
