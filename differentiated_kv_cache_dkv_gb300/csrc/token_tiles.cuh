// token_tiles.cuh -- token tiles of a unit as tensor-core operands: where 128
// tokens of a list lie in the pages, their codes into registers and from there
// into the swizzled rows of an operand (extend.cu, extend_few.cu, extend_sig.cu).
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
// Four threads a token, 32 channels each, NP tokens a thread: tk + p 128 / NP.
// The thread of channels 64 .. takes its two 16-channel halves in the other
// order, so that the eight threads of two neighbouring rows always write eight
// different 16-byte chunks of the swizzled rows.  (u, m1 .. meta: for locate and
// fetch, where the codes come straight from the pages.)
struct DeqCtx {
  const ExtendArgs *a;
  Unit x;
  const volatile int64_t *u;  // x.u in shared memory
  uint32_t m1, m2;  // split() by P and 2 P
  int32_t bytes;
  uint32_t vbase, meta;
  int tk, c, hs;    // token, quarter of the channels, which half comes first
  uint32_t off[4];  // operand-tile offsets of the thread's four groups (token tk)
};

template <int NP>
struct Held {
  uint32_t k[NP][2][4], v[NP][2][4];  // [token][half][words]
  uint2 md[NP];
  bool ok[NP];
};

// Where the thread's tokens of a tile lie: page ids (-1: no token) and slots.
template <int NP>
struct Where {
  int32_t id[NP], slot[NP];
};

template <int NP>
__device__ __forceinline__ void locate(const DeqCtx &d, const Tile &t, Where<NP> &w) {
  if (t.kind == 2) return;
  const bool high = t.kind == 0;
  const int32_t per = high ? d.a->P : 2 * d.a->P, first = high ? 0 : d.x.p_hi;
  const uint32_t M = high ? d.m1 : d.m2;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int32_t i = d.tk + 128 / NP * p;
    int32_t k;
    split(t.t0 + i, per, M, k, w.slot[p]);
    w.id[p] = i < t.n ? __ldg(d.a->fwd + *d.u * d.a->pmax + first + k) : -1;
  }
}

// Codes of the thread's tokens: its two 16-channel halves of a W-bit row lie
// 2 W (8 slot + 2 c + half) bytes into the rows.
template <int KW, int VW, int NP>
__device__ __forceinline__ void fetch(const DeqCtx &d, const Where<NP> &w, Held<NP> &h, bool k, bool v) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const bool ok = w.id[p] >= 0 && w.id[p] < d.a->F;
    // page 0 stands in for none: masked, or its scale is 0
    const uint8_t *pg = d.a->pages + static_cast<int64_t>(ok ? w.id[p] : 0) * d.bytes;
    const uint32_t u0 = 8 * w.slot[p] + 2 * d.c + d.hs, u1 = u0 ^ 1u;
    if (k) {
      load16<KW>(h.k[p][0], pg + 2 * KW * u0);
      load16<KW>(h.k[p][1], pg + 2 * KW * u1);
    }
    if (v) {
      load16<VW>(h.v[p][0], pg + (d.vbase + 2 * VW * u0));
      load16<VW>(h.v[p][1], pg + (d.vbase + 2 * VW * u1));
      h.md[p] = __ldg(reinterpret_cast<const uint2 *>(pg + (d.meta + 8u * w.slot[p])));
      h.ok[p] = ok;
      if (!ok) h.md[p] = make_uint2(0, 0);
    }
  }
}

// Sixteen W-bit codes of a row in shared memory.
template <int W>
__device__ __forceinline__ void read16(uint32_t (&x)[4], const uint8_t *src) {
  if constexpr (W == 8) {
    const uint4 v = *reinterpret_cast<const uint4 *>(src);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else if constexpr (W == 4) {
    const uint2 v = *reinterpret_cast<const uint2 *>(src);
    x[0] = v.x, x[1] = v.y;
  } else if constexpr (W == 2) {
    x[0] = *reinterpret_cast<const uint32_t *>(src);
  } else {
    x[0] = *reinterpret_cast<const uint16_t *>(src);
  }
}

__device__ __forceinline__ void put(uint8_t *tile, uint32_t at, const __half2 (&o)[4]) {
  *reinterpret_cast<uint4 *>(tile + at) = make_uint4(h2u(o[0]), h2u(o[1]), h2u(o[2]), h2u(o[3]));
}

template <int W, class S, int NP>
__device__ __forceinline__ void convert_k(const DeqCtx &d, const Held<NP> &h, S &sm, uint8_t *dst, int slot, float f) {
  constexpr int kMid = 1 << (W - 1);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(h.k[p][i >> 1], i & 1, w0, w1);
      group_codes<W, kMid>(w0, w1, o);
      put(dst, d.off[i] + p * (128 / NP * 128), o);
    }
    if (d.c == 0) {
      const int row = d.tk + 128 / NP * p;
      const __half2 m = u2h(h.md[p].x);
      const float s = __low2float(m), z = __high2float(m);
      sm.s[slot][row] = s * f;
      sm.z[slot][row] = fmaf(kMid, s, z) * f;
      sm.valid[slot][row] = h.ok[p];
    }
  }
}

template <int W, int NP>
__device__ __forceinline__ void convert_v(const DeqCtx &d, const Held<NP> &h, uint8_t *dst) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const __half2 m = u2h(h.md[p].y);
    const __half2 s = __low2half2(m), z = __high2half2(m);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(h.v[p][i >> 1], i & 1, w0, w1);
      group_codes<W, 0>(w0, w1, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = __hfma2(o[e], s, z);
      put(dst, d.off[i] + p * (128 / NP * 128), o);
    }
    // a dequantised value can pass fp16's largest by half a scale step: the
    // infinities go back to it (out of the way of the usual tokens' code)
    if (__builtin_expect(fmaf(static_cast<float>((1 << W) - 1), __low2float(m), fabsf(__high2float(m))) > 65000.0f, 0)) {
#pragma unroll 1
      for (int i = 0; i < 16; ++i) {
        const uint32_t off = group_at(d.tk + 128 / NP * p, 4 * d.c + (i >> 2)) + 4 * (i & 3);
        __half2 *x = reinterpret_cast<__half2 *>(dst + off);
        *x = __hmax2(__hmin2(*x, u2h(0x7bff7bffu)), u2h(0xfbfffbffu));
      }
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
template <int NP, bool kValid, class S>
__device__ __forceinline__ void new_k(const DeqCtx &d, const Tile &t, int64_t tok0, int32_t h, S &sm, uint8_t *dst,
                                      int slot, float f) {
#pragma unroll 1
  for (int p = 0; p < NP; ++p) {
    const int row = d.tk + 128 / NP * p;
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
      *reinterpret_cast<uint4 *>(dst + d.off[i] + p * (128 / NP * 128)) = make_uint4(
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

template <int NP>
__device__ __forceinline__ void new_v(const DeqCtx &d, const Tile &t, int64_t tok0, int32_t h, uint8_t *dst) {
#pragma unroll 1
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int row = d.tk + 128 / NP * p;
      uint4 x[2];
      load_new(d, d.a->v_new, (tok0 + t.t0 + row) * d.a->Hkv + h, row < t.n, e, x);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t g[4];
        group_bf16(x[i], g);
        *reinterpret_cast<uint4 *>(dst + d.off[2 * e + i] + p * (128 / NP * 128)) = make_uint4(g[0], g[1], g[2], g[3]);
      }
    }
  }
}

}  // namespace tc
}  // namespace dkv
