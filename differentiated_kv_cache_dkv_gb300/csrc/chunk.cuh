// chunk.cuh -- what the kernels of a chunk over bf16 pages share: the checked
// lengths, and where a position lies.
#pragma once

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

}  // namespace tc
}  // namespace dkv
