// chunk.cuh -- what the kernels of a chunk over bf16 pages share: the checked
// lengths, and where a position lies.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "tensor_ops.cuh"

namespace dkv {
namespace tc {

// Every length in range and their sum T; `before` gets the tokens of the
// requests before r.  Warp 0 works, every thread of the block calls it.
__device__ __forceinline__ bool chunk_lens(const ChunkArgs &a, int32_t r, int64_t &before) {
  __shared__ int64_t before_s;
  __shared__ int32_t ok_s;
  if (threadIdx.x < 32) {
    int64_t b = 0, t = 0;
    int bad = 0;
    for (int32_t i = threadIdx.x; i < a.R; i += 32) {
      const int32_t n = __ldg(a.new_lens + i), c = __ldg(a.ctx_lens + i);
      if (n < 0 || n > a.max_new || c < 0 || static_cast<int64_t>(c) + n > a.cap) bad = 1;
      t += n;
      if (i < r) b += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b += __shfl_xor_sync(kFull, b, o);
      t += __shfl_xor_sync(kFull, t, o);
      bad |= __shfl_xor_sync(kFull, bad, o);
    }
    if (threadIdx.x == 0) {
      before_s = b;
      ok_s = !bad && t == a.T;
      if (!ok_s) set_error(a.status, DKV_E_LENS);
    }
  }
  __syncthreads();
  before = before_s;
  return ok_s != 0;
}

// The page of positions [B j, B j + B) of request r; -1 when the table names none of the pool.
__device__ __forceinline__ int32_t chunk_page(const ChunkArgs &a, int32_t r, int32_t j) {
  const int32_t id = __ldg(a.table + static_cast<int64_t>(r) * a.tmax + j);
  if (id >= 0 && id < a.F) return id;
  set_error(a.status, DKV_E_INTERNAL);
  return -1;
}

// One lane of a converged warp.  Under this predicate the compiler keeps the
// operands of the products in uniform registers; under `lane == 0` a product
// took 106 cycles to issue where the tensor cores take 64.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(p));
  return p != 0;
}

// TMA copy of one box of a 3-D tensor map at (channel, head, row).
__device__ __forceinline__ void copy_box(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(saddr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(saddr(bar))
      : "memory");
}

// 3-D tensor map over bf16 channels of 128: extents n1 and n2 with strides s1
// and s2 (elements), whose box is 64 channels by b1 by b2, written to shared
// memory with the 128-byte swizzle (what lies past an extent reads as zeros).
inline cudaError_t chunk_map(CUtensorMap *map, const void *base, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int32_t b1,
                             int32_t b2) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    cudaDriverEntryPointQueryResult qr;
    void *fn = nullptr;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &qr);
    return e == cudaSuccess && qr == cudaDriverEntryPointSuccess ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn)
                                                                 : nullptr;
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s1) * 2, static_cast<cuuint64_t>(s2) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
  const cuuint32_t one[3] = {1, 1, 1};
  const CUresult res = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return res == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace tc
}  // namespace dkv
