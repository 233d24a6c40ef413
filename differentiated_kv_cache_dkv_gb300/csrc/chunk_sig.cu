// chunk_sig.cu -- what a chunk's rows give every token's significance
// (dkv_chunk_significance).
#include <algorithm>
#include <cmath>

#include "chunk.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kKeyWarps = 8;

// A warp per (position, query head): blocks (positions of a request, request, layer).
__global__ void __launch_bounds__(32 * kKeyWarps) k_chunk_sig_rows(const __grid_constant__ ChunkArgs a) {
  const int32_t r = blockIdx.y, li = blockIdx.z, lane = threadIdx.x & 31;
  int64_t before;
  if (!chunk_lens(a, r, before)) return;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kKeyWarps + (threadIdx.x >> 5);
  const int32_t t = static_cast<int32_t>(row / a.Hq), hq = static_cast<int32_t>(row % a.Hq), h = hq / a.G;
  const int32_t n = __ldg(a.new_lens + r), ctx = __ldg(a.ctx_lens + r);
  if (n == 0 || t >= ctx + n) return;
  const int32_t id = max(chunk_page(a, r, t / a.B), 0);
  const int64_t at = ((((static_cast<int64_t>(a.layer0) + li) * a.F + id) * a.B + t % a.B) * a.Hkv + h) * 128;
  const uint2 k = *(reinterpret_cast<const uint2 *>(a.k + at) + lane);
  const float k0 = bf16_lo(k.x), k1 = bf16_hi(k.x), k2 = bf16_lo(k.y), k3 = bf16_hi(k.y);
  const float sl2 = a.scale * kLog2e;
  float sum = 0.0f;
  for (int32_t i = max(0, t - ctx); i < n; ++i) {
    const int64_t tok = static_cast<int64_t>(li) * a.T + before + i;
    const uint2 q = __ldg(reinterpret_cast<const uint2 *>(a.q + tok * a.q_stride + hq * 128) + lane);
    float x = k0 * bf16_lo(q.x) + k1 * bf16_hi(q.x) + k2 * bf16_lo(q.y) + k3 * bf16_hi(q.y);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(kFull, x, s);
    const float e = __ldg(a.lse + tok * a.Hq + hq);
    if (e != -INFINITY) sum += exp2f(x * sl2 - e * kLog2e);
  }
  if (lane == 0) {
    float *p = a.sig_sum + ((static_cast<int64_t>(a.layer0) + li) * a.R * a.cap + static_cast<int64_t>(r) * a.cap + t) * a.Hq + hq;
    *p = t < ctx ? *p + sum : sum;
  }
}

}  // namespace

cudaError_t launch_chunk_sig(const ChunkArgs &a, cudaStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.cap) * a.Hq;
  k_chunk_sig_rows<<<dim3(static_cast<unsigned>((rows + kKeyWarps - 1) / kKeyWarps), a.R, a.n_layers), 32 * kKeyWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace dkv
