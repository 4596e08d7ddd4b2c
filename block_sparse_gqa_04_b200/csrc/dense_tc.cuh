// Shared pieces of the tensor-core kernels of the dense operators.
#pragma once

#include <atomic>

#include "dense_common.cuh"
#include "tc_warp.cuh"

namespace msa {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int tiles_of(int n) { return (n + kDenseTile - 1) / kDenseTile; }

// Zeroes rows r0 .. r1-1 of a [128, D] tile (64-dim halves of 128-byte rows; a whole
// row is the same bytes whatever the swizzle) and hands them to the async proxy.  By a
// whole warp, after the tile's copy has landed.
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int r0, int r1) {
  constexpr int per = 8 * (D / 64);
  for (int i = threadIdx.x & 31; i < (r1 - r0) * per; i += 32) {
    const int r = r0 + i / per, c = i % per;
    *reinterpret_cast<uint4*>(tile + (c >> 3) * (128 * 128) + r * 128 + (c & 7) * 16) =
        make_uint4(0, 0, 0, 0);
  }
  tc::fence_async_smem();
  __syncwarp();
}

// Rows of `heads` heads of D: tiles of box_rows rows of box_heads
// heads, 64 dims at a time.
inline cudaError_t encode_rows(CUtensorMap* map, const void* base, int D, int heads, long long rows,
                               int box_rows = kDenseTile, int box_heads = 1) {
  auto enc = encode_fn();
  if (!enc) return cudaErrorNotSupported;
  cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(heads), cuuint64_t(rows)};
  cuuint64_t strides[2] = {cuuint64_t(D) * 2, cuuint64_t(heads) * D * 2};
  cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_rows)}, estr[3] = {1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// Shared memory of a kernel, and the registers that its setmaxnreg split needs, 0
// without one (a build with fewer would leave warpgroups waiting for registers forever).
// Done once per device (`done`: a bit per device, one word per kernel).
template <typename K>
inline cudaError_t prepare_kernel(std::atomic<uint64_t>* done, K kern, size_t smem, int split,
                                  int threads) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (done->load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  cudaFuncAttributes fa;
  e = cudaFuncGetAttributes(&fa, kern);
  if (e != cudaSuccess) return e;
  if (fa.numRegs * (threads / 128) < split) return cudaErrorInvalidConfiguration;
  done->fetch_or(bit, std::memory_order_release);
  return cudaSuccess;
}

}  // namespace msa
