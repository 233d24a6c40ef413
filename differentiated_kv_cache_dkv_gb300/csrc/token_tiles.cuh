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

// The exponent of a block of Q, and how much further a row of it is shifted.  A
// block's rows share one power of two, which the tokens' scales undo; a row
// whose largest value lies 2^12 and more below the block's would lose bits of
// fp16, and is shifted by its own d (its products are multiplied by 2^-d, as is
// the sum of its values).  The block's largest counts as 2^35 at most, so that
// scales times 2^20 stay finite in fp32; rows above that have d < 0.
__device__ __forceinline__ int block_exponent(uint32_t bits) { return max(lift_exponent(bits), -20); }
__device__ __forceinline__ int row_shift(uint32_t ex, int e) {  // ex: the biased exponent of the row's largest
  if (!ex) return 0;  // zeros (or as good as), or not finite
  const int d = lift_exponent(ex << 23) - e;
  return d < 0 || d > 12 ? min(d, 126) : 0;
}
// References and normalisers above this (log2 units) leave y - m, summed in one
// multiply-add, off by more than the weights' range allows: y is rounded first.
constexpr float kFar = 1048576.0f;

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
// Which of its two 16-channel halves a thread takes first alternates with the
// channels and the rows (hs), so that neighbouring threads read different banks
// of the raw rows and the eight threads of two neighbouring rows always write
// eight different 16-byte chunks of the swizzled rows.
struct DeqCtx {
  const ExtendArgs *a;
  int tk, c, hs;    // token, quarter of the channels, which half comes first
  uint32_t off[4];  // operand-tile offsets of the thread's four groups (token tk)
};

template <int NP>
struct Held {
  uint32_t k[NP][2][4], v[NP][2][4];  // [token][half][words]
  uint2 md[NP];
  bool ok[NP];
};

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

// How a raw tile lies in shared memory: token i is slot i mod 2^lg of "page"
// i >> lg, pages `stride` bytes apart, with V codes and scales at vb and mo.
// Where pages divide a tile those are the pages themselves, as they lie in
// memory up to their last used scale: one copy a page.  Otherwise it is one
// page of 128 slots, which three copies per page and tile put together.
struct RawForm {
  int32_t lg, stride, vb, mo;
  bool whole;
};

template <int KW, int VW>
__device__ __forceinline__ RawForm raw_form(int32_t P, bool high) {
  const int32_t per = high ? P : 2 * P;
  const bool whole = per <= 128 && (per & (per - 1)) == 0;
  const int32_t n = whole ? per : 128;
  // per W-bit slots take 16 W per bytes, scales 8 per
  return RawForm{31 - __clz(n), n * (16 * (KW + VW) + 8), n * 16 * KW, n * 16 * (KW + VW), whole};
}

// The two 16-channel halves of each of the thread's tokens, in its order.
template <int W, int NP>
__device__ __forceinline__ void read_raw(const DeqCtx &d, const RawForm &f, const uint8_t *raw, uint32_t (&x)[NP][2][4]) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int i = d.tk + 128 / NP * p, slot = i & ((1 << f.lg) - 1);
    const uint8_t *row = raw + (i >> f.lg) * f.stride + slot * (16 * W);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const uint8_t *src = row + 2 * W * (2 * d.c + (d.hs ^ e));
      read16<W>(x[p][e], src);
    }
  }
}

__device__ __forceinline__ uint2 read_md(const RawForm &f, const uint8_t *raw, int i) {
  return *reinterpret_cast<const uint2 *>(raw + (i >> f.lg) * f.stride + f.mo + 8 * (i & ((1 << f.lg) - 1)));
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
