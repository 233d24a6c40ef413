// chunk.cu -- attention of a chunk of new tokens a request over bf16 pages
// (dkv_chunk_attention).
#include <algorithm>
#include <cmath>

#include "chunk.cuh"

namespace dkv {

namespace {

using namespace tc;

// ------------------------------------------------------------------ append --

constexpr int kAppendThreads = 256, kAppendTokens = 16;

// Both halves of w finite?
__device__ __forceinline__ bool finite2(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}
// ... and w with halves that are not finite as 0.
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  return w;
}

// The new tokens' K and V to their places in the pages: blocks (tokens of a
// request, request, layer), a lane per 16 bytes.
__global__ void __launch_bounds__(kAppendThreads) k_chunk_append(const __grid_constant__ ChunkArgs a) {
  const int32_t r = blockIdx.y, li = blockIdx.z, t0 = blockIdx.x * kAppendTokens;
  int64_t before;
  if (!chunk_lens(a, r, before)) return;
  const int32_t n = min(__ldg(a.new_lens + r) - t0, kAppendTokens), ctx = __ldg(a.ctx_lens + r);
  const int32_t units = a.Hkv * 16;  // 16-byte units of a token's K (or V) rows
  bool bad = false;
  for (int32_t i = threadIdx.x; i < n * units; i += kAppendThreads) {
    const int32_t t = t0 + i / units, c = i % units, p = ctx + t;
    const int32_t id = chunk_page(a, r, p / a.B);
    if (id < 0) continue;
    const int64_t from = (static_cast<int64_t>(li) * a.T + before + t) * a.kv_stride + c * 8;
    const int64_t to = (((static_cast<int64_t>(a.layer0) + li) * a.F + id) * a.B + p % a.B) * (a.Hkv * int64_t{128}) + c * 8;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4 x = *reinterpret_cast<const uint4 *>((kv ? a.v_new : a.k_new) + from);
      if (!(finite2(x.x) && finite2(x.y) && finite2(x.z) && finite2(x.w))) {
        bad = true;
        x = make_uint4(finite_only(x.x), finite_only(x.y), finite_only(x.z), finite_only(x.w));
      }
      *reinterpret_cast<uint4 *>((kv ? a.v : a.k) + to) = x;
    }
  }
  if (bad) set_error(a.status, DKV_E_RANGE);
}

// --------------------------------------------------------------- attention --

constexpr int kRowWarps = 8;

// A warp per (new token, query head): blocks (rows of a request, request, layer).
__global__ void __launch_bounds__(32 * kRowWarps) k_chunk_rows(const __grid_constant__ ChunkArgs a) {
  const int32_t r = blockIdx.y, li = blockIdx.z, lane = threadIdx.x & 31;
  int64_t before;
  if (!chunk_lens(a, r, before)) return;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRowWarps + (threadIdx.x >> 5);
  const int32_t i = static_cast<int32_t>(row / a.Hq), hq = static_cast<int32_t>(row % a.Hq), h = hq / a.G;
  if (i >= __ldg(a.new_lens + r)) return;
  const int32_t end = __ldg(a.ctx_lens + r) + i + 1;
  const int64_t tok = static_cast<int64_t>(li) * a.T + before + i;
  const uint2 qw = __ldg(reinterpret_cast<const uint2 *>(a.q + tok * a.q_stride + hq * 128) + lane);
  const float q0 = bf16_lo(qw.x), q1 = bf16_hi(qw.x), q2 = bf16_lo(qw.y), q3 = bf16_hi(qw.y);
  float m = -INFINITY, l = 0.0f, o0 = 0.0f, o1 = 0.0f, o2 = 0.0f, o3 = 0.0f;
  const float sl2 = a.scale * kLog2e;
  int32_t id = 0;
  for (int32_t t = 0; t < end; ++t) {
    if (t % a.B == 0) id = max(chunk_page(a, r, t / a.B), 0);
    const int64_t at = ((((static_cast<int64_t>(a.layer0) + li) * a.F + id) * a.B + t % a.B) * a.Hkv + h) * 128;
    const uint2 k = *(reinterpret_cast<const uint2 *>(a.k + at) + lane), v = *(reinterpret_cast<const uint2 *>(a.v + at) + lane);
    float x = q0 * bf16_lo(k.x) + q1 * bf16_hi(k.x) + q2 * bf16_lo(k.y) + q3 * bf16_hi(k.y);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(kFull, x, s);
    x *= sl2;
    const float mn = fmaxf(m, x), f = exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * f + p;
    o0 = o0 * f + p * bf16_lo(v.x);
    o1 = o1 * f + p * bf16_hi(v.x);
    o2 = o2 * f + p * bf16_lo(v.y);
    o3 = o3 * f + p * bf16_hi(v.y);
  }
  const float w = 1.0f / l;
  *(reinterpret_cast<uint2 *>(a.out + (tok * a.Hq + hq) * 128) + lane) = make_uint2(bf16x2_rn(o0 * w, o1 * w), bf16x2_rn(o2 * w, o3 * w));
  if (a.lse && lane == 0) a.lse[tok * a.Hq + hq] = (m + log2f(l)) * 0.693147180559945309f;
}

}  // namespace

size_t chunk_workspace(const ChunkArgs &) { return 256; }

cudaError_t launch_chunk(const ChunkArgs &a, void *, cudaStream_t s) {
  if (a.k_new) {
    k_chunk_append<<<dim3((a.max_new + kAppendTokens - 1) / kAppendTokens, a.R, a.n_layers), kAppendThreads, 0, s>>>(a);
    if (cudaError_t e = cudaGetLastError()) return e;
  }
  const int64_t rows = static_cast<int64_t>(a.max_new) * a.Hq;
  k_chunk_rows<<<dim3(static_cast<unsigned>((rows + kRowWarps - 1) / kRowWarps), a.R, a.n_layers), 32 * kRowWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace dkv
