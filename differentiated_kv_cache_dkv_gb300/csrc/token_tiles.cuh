// token_tiles.cuh -- token tiles of a unit as tensor-core operands: where 128
// tokens of a list lie in the pages, their codes into registers and from there
// into the swizzled rows of an operand (extend.cu, extend_sig.cu).
#pragma once

#include "tensor_ops.cuh"

namespace dkv {
namespace tc {

// Quotient and remainder by P with M = 2^32 / P + 1 (the quotient is at most
// one too large below 2^31).
__device__ __forceinline__ void split(int32_t t, int32_t P, uint32_t M, int32_t &k, int32_t &r) {
  k = static_cast<int32_t>(__umulhi(static_cast<uint32_t>(t), M));
  r = t - k * P;
  if (r < 0) {
    --k;
    r += P;
  }
}

// Largest |value| of a bf16 row as bits; 0 when it is not finite.
__device__ __forceinline__ uint32_t row_max(const uint16_t *src) {
  float mx = 0.0f;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src) + i);
    mx = max3(mx, max3(fabsf(bf16_lo(v.x)), fabsf(bf16_hi(v.x)), fabsf(bf16_lo(v.y))),
              max3(fabsf(bf16_hi(v.y)), fabsf(bf16_lo(v.z)), fabsf(bf16_hi(v.z))));
    mx = max3(mx, fabsf(bf16_lo(v.w)), fabsf(bf16_hi(v.w)));
  }
  const uint32_t b = __float_as_uint(mx);
  return b < 0x7f800000u ? b : 0;
}

// The exponent e that puts a largest value (its bits) into [2^14, 2^15).
__device__ __forceinline__ int lift_exponent(uint32_t bits) {
  return bits ? min(max(14 + 127 - static_cast<int>(bits >> 23), -120), 120) : 0;
}

// The dequant warps' view of one tile.
struct Tile {
  int32_t kind, t0, n;  // 0 high, 1 low, 2 new; first token in its list; tokens
};

__device__ __forceinline__ Tile tile_at(const Tiles &ts, const Unit &x, int32_t fresh, int32_t j) {
  Tile t;
  if (j < ts.hi) t = {0, 128 * j, x.n_hi};
  else if (j < ts.hi + ts.lo) t = {1, 128 * (j - ts.hi), x.n_lo};
  else t = {2, 128 * (j - ts.hi - ts.lo), fresh};
  t.n = min(128, t.n - t.t0);
  return t;
}

// ------------------------------------------------------- dequantising warps --
//
// Four threads a token, 32 channels each, two tokens (tk and tk + 64) a
// thread.  The thread of channels 64 .. takes its two 16-channel halves in the
// other order, so that the eight threads of two neighbouring rows always
// write eight different 16-byte chunks of the swizzled rows.
struct DeqCtx {
  const ExtendArgs *a;
  Unit x;
  uint32_t m1, m2;  // split() by P and 2 P
  int64_t bytes;
  int32_t vbase, meta;
  int tk, c, hs;    // token, quarter of the channels, which half comes first
  uint32_t off[4];  // operand-tile offsets of the thread's four groups (token tk)
};

struct Held {
  uint32_t k[2][2][4], v[2][2][4];  // [token][half][words]
  uint2 md[2];
  bool ok[2];
};

// Where the two tokens of a tile lie: page ids (-1: no token) and slots.
struct Where {
  int32_t id[2], slot[2];
};

__device__ __forceinline__ void locate(const DeqCtx &d, const Tile &t, Where &w) {
  if (t.kind == 2) return;
  const bool high = t.kind == 0;
  const int32_t per = high ? d.a->P : 2 * d.a->P, first = high ? 0 : d.x.p_hi;
  const uint32_t M = high ? d.m1 : d.m2;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int32_t i = d.tk + 64 * p;
    int32_t k;
    split(t.t0 + i, per, M, k, w.slot[p]);
    w.id[p] = i < t.n ? __ldg(d.a->fwd + d.x.u * d.a->pmax + first + k) : -1;
  }
}

template <int KW, int VW>
__device__ __forceinline__ void fetch(const DeqCtx &d, const Where &w, Held &h, bool k, bool v) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bool ok = w.id[p] >= 0 && w.id[p] < d.a->F;
    const uint8_t *pg = d.a->pages + (ok ? w.id[p] : 0) * d.bytes;  // page 0 stands in: masked, or its scale is 0
    if (k) {
      const uint8_t *src = pg + w.slot[p] * (16 * KW) + d.c * (4 * KW);
      load16<KW>(h.k[p][0], src + d.hs * (2 * KW));
      load16<KW>(h.k[p][1], src + (d.hs ^ 1) * (2 * KW));
    }
    if (v) {
      const uint8_t *src = pg + d.vbase + w.slot[p] * (16 * VW) + d.c * (4 * VW);
      load16<VW>(h.v[p][0], src + d.hs * (2 * VW));
      load16<VW>(h.v[p][1], src + (d.hs ^ 1) * (2 * VW));
      h.md[p] = __ldg(reinterpret_cast<const uint2 *>(pg + d.meta + 8 * w.slot[p]));
      h.ok[p] = ok;
      if (!ok) h.md[p] = make_uint2(0, 0);
    }
  }
}

__device__ __forceinline__ void put(uint8_t *tile, uint32_t at, const __half2 (&o)[4]) {
  *reinterpret_cast<uint4 *>(tile + at) = make_uint4(h2u(o[0]), h2u(o[1]), h2u(o[2]), h2u(o[3]));
}

template <int W, class S>
__device__ __forceinline__ void convert_k(const DeqCtx &d, const Held &h, S &sm, uint8_t *dst, int slot, float f) {
  constexpr float kMid = 1 << (W - 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(h.k[p][i >> 1], i & 1, w0, w1);
      group_codes<W>(w0, w1, kMid, o);
      put(dst, d.off[i] + p * (64 * 128), o);
    }
    if (d.c == 0) {
      const int row = d.tk + 64 * p;
      const __half2 m = u2h(h.md[p].x);
      const float s = __low2float(m), z = __high2float(m);
      sm.s[slot][row] = s * f;
      sm.z[slot][row] = fmaf(kMid, s, z) * f;
      sm.valid[slot][row] = h.ok[p];
    }
  }
}

template <int W>
__device__ __forceinline__ void convert_v(const DeqCtx &d, const Held &h, uint8_t *dst) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const __half2 m = u2h(h.md[p].y);
    const __half2 s = __low2half2(m), z = __high2half2(m);
    // a dequantised value can pass fp16's largest by half a scale step
    const bool big = fmaf(static_cast<float>((1 << W) - 1), __low2float(m), fabsf(__high2float(m))) > 65000.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(h.v[p][i >> 1], i & 1, w0, w1);
      group_codes<W>(w0, w1, 0.0f, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __hfma2(o[e], s, z);
      if (big) {
        const __half2 top = __float2half2_rn(65504.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = __hmax2(__hmin2(o[e], top), __hneg2(top));
      }
      put(dst, d.off[i] + p * (64 * 128), o);
    }
  }
}

// 16 bf16 of a new token's row (0 when it has none), not finite -> 0: half
// `half` (in the thread's order) of its 32 channels.
__device__ __forceinline__ void load_new(const DeqCtx &d, const uint16_t *base, int64_t row, bool have, int half,
                                         uint4 (&x)[2]) {
  x[0] = x[1] = make_uint4(0, 0, 0, 0);
  if (!have) return;
  const uint4 *src = reinterpret_cast<const uint4 *>(base + row * 128) + 4 * d.c + 2 * (half ^ d.hs);
  x[0] = __ldg(src);
  x[1] = __ldg(src + 1);
  uint32_t *w = reinterpret_cast<uint32_t *>(x);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u, bad = true;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu, bad = true;
  }
  if (bad) set_error(d.a->status, DKV_E_RANGE);
}

// K of the new tokens: each row times the power of two that puts its largest
// value into [2^14, 2^15), in fp16; the scale carries it back.
template <bool kValid, class S>
__device__ __forceinline__ void new_k(const DeqCtx &d, const Tile &t, int64_t tok0, int32_t h, S &sm, uint8_t *dst,
                                      int slot, float f) {
#pragma unroll 1
  for (int p = 0; p < 2; ++p) {
    const int row = d.tk + 64 * p;
    uint4 x[2][2];
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      load_new(d, d.a->k_new, (tok0 + t.t0 + row) * d.a->Hkv + h, row < t.n, e, x[e]);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(x[e]);
#pragma unroll
      for (int i = 0; i < 8; ++i) mx = max3(mx, fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i])));
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
    const int e = lift_exponent(__float_as_uint(mx));
    const float sc = pow2f(e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = x[i >> 1][i & 1];
      *reinterpret_cast<uint4 *>(dst + d.off[i] + p * (64 * 128)) = make_uint4(
          f16x2_rn(bf16_lo(v.x) * sc, bf16_lo(v.z) * sc), f16x2_rn(bf16_hi(v.x) * sc, bf16_hi(v.z) * sc),
          f16x2_rn(bf16_lo(v.y) * sc, bf16_lo(v.w) * sc), f16x2_rn(bf16_hi(v.y) * sc, bf16_hi(v.w) * sc));
    }
    if (d.c == 0) {
      sm.s[slot][row] = pow2f(-e) * f;
      sm.z[slot][row] = 0.0f;
      if constexpr (kValid) sm.valid[slot][row] = 1;
    }
  }
}

__device__ __forceinline__ void new_v(const DeqCtx &d, const Tile &t, int64_t tok0, int32_t h, uint8_t *dst) {
#pragma unroll 1
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = d.tk + 64 * p;
      uint4 x[2];
      load_new(d, d.a->v_new, (tok0 + t.t0 + row) * d.a->Hkv + h, row < t.n, e, x);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t g[4];
        group_bf16(x[i], g);
        *reinterpret_cast<uint4 *>(dst + d.off[2 * e + i] + p * (64 * 128)) = make_uint4(g[0], g[1], g[2], g[3]);
      }
    }
  }
}

}  // namespace tc
}  // namespace dkv
