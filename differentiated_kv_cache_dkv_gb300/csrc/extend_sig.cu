// extend_sig.cu -- significance of the accepted new tokens of a request
// (dkv_extend_significance).
#include <algorithm>
#include <cmath>

#include "tensor_ops.cuh"

namespace dkv {

namespace {

using namespace tc;

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }

// Page and slot of token t of a unit's lists (the high list, then the low
// list); null when the table's page id is out of range.
__device__ __forceinline__ const uint8_t *token_page(const ExtendArgs &a, const PageGeom &g, const Unit &x, int32_t t,
                                                     bool &high, int32_t &slot) {
  high = t < x.n_hi;
  int32_t k;
  if (high) {
    k = t / a.P;
    slot = t - k * a.P;
  } else {
    const int32_t j = t - x.n_hi;
    k = j / (2 * a.P);
    slot = j - k * 2 * a.P;
    k += x.p_hi;
  }
  const int32_t id = __ldg(a.fwd + x.u * a.pmax + k);
  if (id < 0 || id >= a.F) {
    set_error(a.status, DKV_E_INTERNAL);
    return nullptr;
  }
  return a.pages + id * g.bytes;
}

__device__ __forceinline__ float code_of(const uint8_t *row, int ch, int bits) {
  return static_cast<float>((row[(ch * bits) >> 3] >> ((ch * bits) & 7)) & ((1 << bits) - 1));
}

constexpr int kTok = 32;

// Simple form: a block per 32 tokens of a unit (held or new), one warp per
// query head of the group in turn, a lane per token; the rows pass through
// shared memory 16 at a time.
__global__ void __launch_bounds__(128) k_extend_sig(ExtendArgs a, int32_t tiles) {
  __shared__ float ks[kTok][129], qs[4][128];
  __shared__ int32_t ok_s[kTok], pos_s[kTok];
  const int64_t ui = blockIdx.x / tiles;
  const int32_t tile = blockIdx.x % tiles;
  const int32_t h = ui % a.Hkv, r = (ui / a.Hkv) % a.R, li = ui / (static_cast<int64_t>(a.Hkv) * a.R);
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t acc = __ldg(a.acc_lens + r), ctx = __ldg(a.ctx_lens + r);
  const PageGeom g = page_geom(a.scheme, a.P);
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t held = x.n_hi + x.n_lo, total = held + (a.k_new ? acc : 0), t0 = tile * kTok;
  if (acc == 0 || t0 >= total) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  {
    const int t = threadIdx.x / 4, c0 = 32 * (threadIdx.x % 4);
    const int32_t tt = t0 + t;
    int32_t ok = 0, pos = 0;
    if (tt < held) {
      bool high;
      int32_t slot;
      const uint8_t *pg = token_page(a, g, x, tt, high, slot);
      if (pg) {
        pos = *reinterpret_cast<const int32_t *>(pg + g.pos + 4 * slot);
        ok = pos >= 0 && pos < ctx;
        if (!ok) set_error(a.status, DKV_E_INTERNAL);
        const int kb = high ? g.kh : g.kh / 2;
        const __half *md = reinterpret_cast<const __half *>(pg + g.meta + 8 * slot);
        const float sk = __half2float(md[0]), zk = __half2float(md[1]);
        for (int c = c0; c < c0 + 32; ++c) ks[t][c] = fmaf(code_of(pg + slot * 16 * kb, c, kb), sk, zk);
      }
    } else if (tt < total) {
      ok = 1;
      pos = ctx + tt - held;
      const int64_t row = ((tok0 + tt - held) * a.Hkv + h) * 128;
      for (int c = c0; c < c0 + 32; ++c) {
        const float k = bf16f(a.k_new[row + c]);
        if (!isfinite(k)) set_error(a.status, DKV_E_RANGE);
        ks[t][c] = isfinite(k) ? k : 0.0f;
      }
    }
    if (c0 == 0) {
      ok_s[t] = ok;
      pos_s[t] = pos;
    }
  }
  __syncthreads();
  const int32_t tt = t0 + lane;
  for (int32_t gq = warp; gq < a.G; gq += 4) {
    float sum = 0.0f;
    for (int32_t i = 0; i < acc; ++i) {
      const int64_t at = (tok0 + i) * a.Hq + h * a.G + gq;
      __syncwarp();
      for (int c = lane; c < 128; c += 32) qs[warp][c] = bf16f(a.q[at * 128 + c]);
      __syncwarp();
      const float lse = a.lse[at];
      float s = 0.0f;
      for (int c = 0; c < 128; ++c) s = fmaf(qs[warp][c], ks[lane][c], s);
      if (ok_s[lane] && lse != -INFINITY && (tt < held || tt - held <= i)) sum += expf(s * a.scale - lse);
    }
    if (ok_s[lane]) {
      float *dst = a.sig_sum + ((static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.cap + pos_s[lane]) * a.Hq +
                   h * a.G + gq;
      *dst = tt < held ? *dst + sum : sum;
    }
  }
}

}  // namespace

cudaError_t launch_extend_sig(const ExtendArgs &a, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.cap) + a.max_new + kTok - 1) / kTok;
  const int64_t grid = static_cast<int64_t>(a.n_layers) * a.R * a.Hkv * tiles;
  if (grid == 0) return cudaSuccess;
  k_extend_sig<<<static_cast<unsigned>(grid), 128, 0, s>>>(a, static_cast<int32_t>(tiles));
  return cudaGetLastError();
}

}  // namespace dkv
