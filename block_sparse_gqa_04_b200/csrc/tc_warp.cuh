// What the tensor-core attention kernels do with their accumulators: bounded waits by
// whole warps, packed fp32 arithmetic, bf16 packing, register trades between
// warpgroups; and on the host the tensor-map encoder and the SM count.
#pragma once

#include <cudaTypedefs.h>

#include "common.cuh"
#include "tc_common.cuh"

namespace msa {

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
  return __all_sync(MSA_FULL_MASK, tc::mbar_wait(bar, parity, abort));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&h);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Maximum of 32 values (four independent chains of three-input maxima).
__device__ __forceinline__ float max32(const uint32_t (&v)[32], float m) {
  float a[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int x = 0; x < 32; x += 2)
    a[(x >> 1) & 3] = max3(a[(x >> 1) & 3], __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
  return fmaxf(fmaxf(a[0], a[1]), fmaxf(a[2], a[3]));
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}

// setmaxnreg acts on a whole warpgroup.
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// Two-wide fp32 helpers (sm_100 packed FMA / add / mul on a 64-bit pair).
__device__ __forceinline__ uint64_t f2(float lo, float hi) {
  return (uint64_t(__float_as_uint(hi)) << 32) | __float_as_uint(lo);
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// bf16x2 of the two fp32 halves (low half -> low 16 bits), round to nearest even
__device__ __forceinline__ uint32_t to_bf16x2(uint64_t x) {
  return pack_bf16(__uint_as_float(uint32_t(x)), __uint_as_float(uint32_t(x >> 32)));
}
// 2^x in fp32 on the exp2 unit (flushes subnormal results to zero)
__device__ __forceinline__ float ex2_f32(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The larger of two values, NaN if either is (fmaxf takes the other).
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 2^x of two values on the FMA pipe, for part of a tile's exponentials where the exp2
// unit (16 values per SM and cycle) is what everything waits for.  x = n + f, n the
// nearest integer, found by adding 1.5 x 2^23; 2^f on [-1/2, 1/2] by a quartic, the minimax
// fit of the relative error by Remez exchange (3e-6, against 2^-9 of a bf16 rounding);
// times 2^n, made of n's bits by an integer add.  (Added to the quartic's exponent instead,
// n's bits would turn a NaN into a number.)  For x up to 127; below -126 it is taken as
// -126.
__device__ __forceinline__ uint64_t exp2_poly(uint64_t x) {
  constexpr float c[5] = {0.9999992847442627f, 0.6931217908859253f, 0.240247443318367f,
                          0.05591785907745361f, 0.009570102207362652f};
  constexpr float kMagic = 12582912.f;
  constexpr uint32_t kOne = 0x3f800000u;  // 1.f
  x = f2(max_nan(__uint_as_float(uint32_t(x)), -126.f),
         max_nan(__uint_as_float(uint32_t(x >> 32)), -126.f));
  const uint64_t t = add2(x, f2(kMagic, kMagic));
  const uint64_t n = add2(t, f2(-kMagic, -kMagic));
  const uint64_t f = fma2(n, f2(-1.f, -1.f), x);
  uint64_t p = f2(c[4], c[4]);
#pragma unroll
  for (int i = 3; i >= 0; --i) p = fma2(p, f, f2(c[i], c[i]));
  const uint32_t lo = (uint32_t(t) << 23) + kOne;
  const uint32_t hi = (uint32_t(t >> 32) << 23) + kOne;
  return mul2(p, (uint64_t(hi) << 32) | lo);
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  return fn;
}

inline int sm_count() {
  static int n = 0;
  if (!n) {
    int dev = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (n <= 0) n = 148;
  }
  return n;
}

}  // namespace msa
