// extend.cu -- attention of several new tokens a request over the unified
// pages (dkv_extend_attention), and the significance their accepted ones give
// (dkv_extend_significance).
//
// A row is one (new token i, query head g of the KV head's group), numbered
// i G + g within its unit.  With codes c, scale s and zero z of a token,
//   x = scale (s (q . c) + z (sum of q)),  out = sum_t exp(x_t - lse) v_t.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "dkv_internal.cuh"

namespace dkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float bf16f(uint16_t x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
__device__ __forceinline__ uint16_t f2bf16(float x) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(0.0f), "f"(x));
  return static_cast<uint16_t>(r);
}

// Every length in range and their sum T; `before` gets the tokens of the
// requests before r.  Warp 0 works, every thread of the block calls it.
__device__ __forceinline__ bool lens_valid(const ExtendArgs &a, int32_t r, int64_t &before) {
  __shared__ int64_t before_s;
  __shared__ int32_t ok_s;
  if (threadIdx.x < 32) {
    int64_t b = 0, t = 0;
    int bad = 0;
    for (int32_t i = threadIdx.x; i < a.R; i += 32) {
      const int32_t n = __ldg(a.new_lens + i), c = __ldg(a.ctx_lens + i);
      if (n < 0 || n > a.max_new || c < 0 || static_cast<int64_t>(c) + n > a.cap) bad = 1;
      if (a.acc_lens && (__ldg(a.acc_lens + i) < 0 || __ldg(a.acc_lens + i) > n)) bad = 1;
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

// The lists of a unit (empty when its header contradicts itself).
struct Unit {
  int64_t u;             // index in the tables
  int32_t n_hi, n_lo, p_hi;
};

__device__ __forceinline__ Unit load_unit(const ExtendArgs &a, int64_t u) {
  const int4 h = *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * u);
  Unit x{u, h.x, h.y, h.z};
  if (h.x < 0 || h.y < 0 || h.z != (static_cast<int64_t>(h.x) + a.P - 1) / a.P ||
      h.w != (static_cast<int64_t>(h.y) + 2 * a.P - 1) / (2 * a.P) || h.z + h.w > a.pmax) {
    set_error(a.status, DKV_E_INTERNAL);
    x.n_hi = x.n_lo = x.p_hi = 0;
  }
  return x;
}

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

constexpr int kRows = 16, kTok = 32;

// Simple form: 16 rows a block, 32 tokens at a time dequantised into shared
// memory, one warp for four rows, a lane per token (logits) and per four
// channels (values).
__global__ void __launch_bounds__(128) k_extend(ExtendArgs a, int32_t tiles) {
  __shared__ float ks[kTok][129], qs[kRows][128];
  __shared__ __align__(16) float vs[kTok][132];  // read as float4
  __shared__ int32_t ok_s[kTok];
  const int64_t ui = blockIdx.x / tiles;
  const int32_t tile = blockIdx.x % tiles;
  const int32_t h = ui % a.Hkv, r = (ui / a.Hkv) % a.R, li = ui / (static_cast<int64_t>(a.Hkv) * a.R);
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t n = __ldg(a.new_lens + r), rows = n * a.G, row0 = tile * kRows;
  if (row0 >= rows) return;
  const PageGeom g = page_geom(a.scheme, a.P);
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t held = x.n_hi + x.n_lo, last_i = min(row0 + kRows - 1, rows - 1) / a.G;
  const int32_t total = held + (a.k_new ? last_i + 1 : 0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  for (int e = threadIdx.x; e < kRows * 128; e += 128) {
    const int32_t row = row0 + e / 128;
    qs[e / 128][e % 128] =
        row < rows ? bf16f(a.q[((tok0 + row / a.G) * a.Hq + h * a.G + row % a.G) * 128 + e % 128]) : 0.0f;
  }
  float m[4], l[4], o[4][4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    m[k] = -INFINITY;
    l[k] = o[k][0] = o[k][1] = o[k][2] = o[k][3] = 0.0f;
  }
  for (int32_t t0 = 0; t0 < total; t0 += kTok) {
    __syncthreads();
    {
      const int t = threadIdx.x / 4, c0 = 32 * (threadIdx.x % 4);
      const int32_t tt = t0 + t;
      int32_t ok = 0;
      if (tt < held) {
        bool high;
        int32_t slot;
        const uint8_t *pg = token_page(a, g, x, tt, high, slot);
        if (pg) {
          ok = 1;
          const int kb = high ? g.kh : g.kh / 2, vb = high ? g.vh : g.vh / 2;
          const __half *md = reinterpret_cast<const __half *>(pg + g.meta + 8 * slot);
          const float sk = __half2float(md[0]), zk = __half2float(md[1]), sv = __half2float(md[2]),
                      zv = __half2float(md[3]);
          const uint8_t *kr = pg + slot * 16 * kb, *vr = pg + g.vbase + slot * 16 * vb;
          for (int c = c0; c < c0 + 32; ++c) {
            ks[t][c] = fmaf(code_of(kr, c, kb), sk, zk);
            vs[t][c] = fmaf(code_of(vr, c, vb), sv, zv);
          }
        }
      } else if (tt < total) {
        ok = 1;
        const int64_t row = ((tok0 + tt - held) * a.Hkv + h) * 128;
        for (int c = c0; c < c0 + 32; ++c) {
          float k = bf16f(a.k_new[row + c]), v = bf16f(a.v_new[row + c]);
          if (!isfinite(k) || !isfinite(v)) set_error(a.status, DKV_E_RANGE);
          ks[t][c] = isfinite(k) ? k : 0.0f;
          vs[t][c] = isfinite(v) ? v : 0.0f;
        }
      }
      if (!ok)
        for (int c = c0; c < c0 + 32; ++c) ks[t][c] = vs[t][c] = 0.0f;
      if (c0 == 0) ok_s[t] = ok;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = row0 + 4 * warp + k;
      const int32_t i = row / a.G, tt = t0 + lane;
      float s = 0.0f;
      for (int c = 0; c < 128; ++c) s = fmaf(qs[4 * warp + k][c], ks[lane][c], s);
      s = ok_s[lane] && (tt < held || tt - held <= i) ? s * a.scale : -INFINITY;
      float mx = s;
      for (int w = 16; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, w));
      const float mn = fmaxf(m[k], mx);
      if (mn == -INFINITY) continue;
      const float f = expf(m[k] - mn), p = expf(s - mn);
      float sum = p;
      for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(kFull, sum, w);
      l[k] = l[k] * f + sum;
      m[k] = mn;
      for (int c = 0; c < 4; ++c) o[k][c] *= f;
      for (int t = 0; t < kTok; ++t) {
        const float pt = __shfl_sync(kFull, p, t);
        const float4 v = *reinterpret_cast<const float4 *>(&vs[t][4 * lane]);
        o[k][0] = fmaf(pt, v.x, o[k][0]);
        o[k][1] = fmaf(pt, v.y, o[k][1]);
        o[k][2] = fmaf(pt, v.z, o[k][2]);
        o[k][3] = fmaf(pt, v.w, o[k][3]);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int32_t row = row0 + 4 * warp + k;
    if (row >= rows) continue;
    const int64_t at = (tok0 + row / a.G) * a.Hq + h * a.G + row % a.G;
    const float inv = l[k] > 0.0f ? 1.0f / l[k] : 0.0f;
    for (int c = 0; c < 4; ++c) a.out[at * 128 + 4 * lane + c] = f2bf16(o[k][c] * inv);
    if (a.lse && lane == 0) a.lse[at] = l[k] > 0.0f ? m[k] + logf(l[k]) : -INFINITY;
  }
}

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

cudaError_t launch_extend(const ExtendArgs &a, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.max_new) * a.G + kRows - 1) / kRows;
  const int64_t grid = static_cast<int64_t>(a.n_layers) * a.R * a.Hkv * tiles;
  if (grid == 0) return cudaSuccess;
  k_extend<<<static_cast<unsigned>(grid), 128, 0, s>>>(a, static_cast<int32_t>(tiles));
  return cudaGetLastError();
}

cudaError_t launch_extend_sig(const ExtendArgs &a, cudaStream_t s) {
  const int64_t tiles = (static_cast<int64_t>(a.cap) + a.max_new + kTok - 1) / kTok;
  const int64_t grid = static_cast<int64_t>(a.n_layers) * a.R * a.Hkv * tiles;
  if (grid == 0) return cudaSuccess;
  k_extend_sig<<<static_cast<unsigned>(grid), 128, 0, s>>>(a, static_cast<int32_t>(tiles));
  return cudaGetLastError();
}

}  // namespace dkv
