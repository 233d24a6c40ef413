// extend.cu -- attention of several new tokens a request over the unified
// pages (dkv_extend_attention), on the fifth-generation tensor cores.
//
// A row is one (new token i, query head g of the KV head's group), numbered
// i G + g within its unit.  With codes c, scale s and zero z of a token,
//   x = scale (s (q . c) + z (sum of q)),  out = sum_t exp(x_t - lse) v_t.
// A block takes 128 MT rows of one unit (MT = 1 or 2) and a contiguous range of the
// unit's token tiles: 128 tokens of the high list, of the low list, or of the
// request's new tokens.  Its roles, pipelined through mbarriers:
//   dequant warps (8)  copy the pages of a tile into shared memory by bulk
//     copies, one tile ahead, read their codes into registers and write two
//     operands to shared memory: K as
//     the codes themselves in fp16, less the middle code (exact; scale and
//     zero stay in fp32 and are applied to the logits), and V as
//     fp16(fma(c, s, z)) -- every cached value is a multiple of 2^-24, so
//     fp16 holds it to half a step of its 11 bits, subnormals exactly;
//   softmax warps (2 x 4)  a thread per row: logits, running maximum and sum
//     in fp32, P = 2^(y - m) in fp16 back into the columns of S.  One thread of
//     each warpgroup issues its products: O += P V of a tile (P read from
//     tensor memory) as soon as its P is complete, then S = Q K^T of its next
//     tile into the same columns (the tensor cores run one thread's products
//     in order), while the other warpgroup is in its softmax.  A separate
//     issuing warp would be the seventeenth and cost every thread a quarter of
//     its registers.
// The block's rows of Q are scaled by one power of two that puts their largest
// finite value into [2^14, 2^15) (the tokens' scales undo it), and a row whose
// own largest lies 2^12 and more below by a further one of its own (row_shift):
// values 19 binades below a row's largest still have all their bits in fp16, so
// q . c is exact up to the fp32 accumulation, whatever the rows beside it are.
// New tokens: K is scaled per token the same way; V stays the bf16 it is, and
// that product takes P as the sum of two bf16 values in two products (both
// operands of one MMA have one type; one bf16 value alone showed as a third of
// the output's error where few tokens are attended).
//
// The maximum is lazy: P = 2^(y - m + 7) with a row's reference m (a whole
// number, log2 units) that is set by the first chunk of columns the row attends
// and moves only when the sum of 32 weights passes 2^15, so the usual chunk needs
// no maximum at all; then the softmax warp raises m to the chunk's maximum and
// multiplies its row of O by the exact power of two.
// Weights stay at or below 2^15 (fp16's largest is 2^16); those down to 2^-21
// of the row's largest keep all 11 bits and 2^-32 is where they vanish.
//
// MT = 2 (more than 128 rows): the two softmax warpgroups take 128 rows each
// and every tile serves both, which halves the conversions per logit.  MT = 1:
// both take the same rows and every other tile; their two partial results
// meet, as those of the blocks that share a row's tiles do, in k_extend_merge.
// Units with at most 32 rows have a kernel of their own (extend_few.cu).
//
// Measured (32 heads over 8, 4 requests of 1024 new tokens over 16384 held, half
// of those in the high list, 39% in the low one): 1490 us, 1.01 TFLOP, 680 TFLOP/s,
// 35% of the measured bf16 rate.  The tensor pipe is busy for 30% of the
// cycles: a warpgroup's tile takes 6640 (traced with a call at 1513 us), of which
// its softmax 3730 (932 for 32 columns, one warp a scheduler: the latencies of the tensor-memory load, of
// the scales' broadcast reads and of the exponentials follow one another) and
// the issue of its products, their completion and the hand-overs 2900; at full
// rate a tile's products for both warpgroups take 2048.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "token_tiles.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kSoftWarps = 8, kDeqWarps = 8;
constexpr int kThreads = 32 * (kSoftWarps + kDeqWarps);
constexpr uint32_t kTmemCols = 512;  // S (and P) of warpgroup w at 128 w, O at 256 + 128 w
constexpr int kMeta = 4;             // ring of the tiles' scales and zeros
constexpr float kLift = 7.0f;        // P = 2^(y - m + kLift)
constexpr float kMost = 32768.0f;    // sum of 32 weights that moves m

template <int MT>
struct __align__(1024) Smem {
  uint8_t q[MT][kTileBytes];
  uint8_t k[2][kTileBytes];
  uint8_t v[2][kTileBytes];
  float s[kMeta][128], z[kMeta][128];  // per token: scale s and z + mid s, times scale log2 e
  uint8_t valid[kMeta][128];           // looked at only when a page id of the unit is bad
  uint8_t raw[200 * 128];              // a tile's pages: codes, scales and zeros (200 bytes a token at most)
  uint64_t rfull, rempty, qready, kfull[2], kempty[2], vfull[2], vempty[2], mfull[kMeta];
  uint64_t sfull[2], pready[2], odone[2], turn[2], done[2];
  uint32_t tmem;
  uint32_t qmax;  // largest finite |q| of the block's rows (bits)
  float w[256];   // 2^-d of the softmax threads' rows (row_shift)
  int32_t abort, bad;
  int64_t u, tok0;  // unit and first new token, for the conversion (which has no registers for them)
};
template <int MT>
constexpr size_t smem_bytes() { return sizeof(Smem<MT>) + 1024; }
static_assert(smem_bytes<2>() <= 227 * 1024, "shared memory");
static_assert(offsetof(Smem<1>, raw) % 16 == 0 && offsetof(Smem<2>, raw) % 16 == 0, "bulk copies");

// ------------------------------------------------------------ softmax warps --

// A row of Q times sc into operand form (`dst` may be null); returns its sum.
__device__ __forceinline__ float stage_q(const uint16_t *src, bool have, uint8_t *dst, int row, float sc) {
  float sum = 0.0f;
#pragma unroll 4
  for (int i = 0; i < 16; ++i) {
    const uint4 v = have ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
    const float c0 = bf16_lo(v.x) * sc, c1 = bf16_hi(v.x) * sc, c2 = bf16_lo(v.y) * sc, c3 = bf16_hi(v.y) * sc;
    const float c4 = bf16_lo(v.z) * sc, c5 = bf16_hi(v.z) * sc, c6 = bf16_lo(v.w) * sc, c7 = bf16_hi(v.w) * sc;
    sum += ((c0 + c1) + (c2 + c3)) + ((c4 + c5) + (c6 + c7));
    if (dst)
      *reinterpret_cast<uint4 *>(dst + group_at(row, i)) =
          make_uint4(f16x2_rn(c0, c4), f16x2_rn(c1, c5), f16x2_rn(c2, c6), f16x2_rn(c3, c7));
  }
  return sum;
}

// Columns a row keeps of 32: the first `lim`, and of those the valid ones.
__device__ __forceinline__ uint32_t column_mask(int32_t lim, const uint8_t *valid) {
  uint32_t k = lim >= 32 ? 0xffffffffu : (lim <= 0 ? 0u : (1u << lim) - 1u);
  if (valid)
    for (int i = 0; i < 32; ++i)
      if (!valid[i]) k &= ~(1u << i);
  return k;
}

// Columns of one row of O: 32 values in operand order, to channel order.
__device__ __forceinline__ void channel_order(const uint32_t *r, float *x) {
#pragma unroll
  for (int g = 0; g < 4; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[8 * g + i] = __uint_as_float(r[8 * g + 2 * i]);
      x[8 * g + 4 + i] = __uint_as_float(r[8 * g + 2 * i + 1]);
    }
}

// The first `full` blocks do a row tile each, the others one of `splits` parts
// of a row tile's token tiles.
template <int SC, int MT>
__global__ void __launch_bounds__(kThreads, 1)
    k_extend(const __grid_constant__ ExtendArgs a, int32_t row_tiles, uint32_t full, int32_t splits, ExtendPartial part) {
  constexpr int KH = scheme_kh(SC), VH = scheme_vh(SC);
  // with MT = 1 it costs more than it hides (16 new tokens over 16384: 41 us
  // without, 47 with; drafts of two requests 23.6 with, 25.7 without)
  if constexpr (MT == 2) let_merge_start();
  extern __shared__ unsigned char smem_raw[];
  // aligned by an offset, not by an integer address: the compiler then knows that these are shared accesses
  Smem<MT> &sm = *reinterpret_cast<Smem<MT> *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // in the order (request, the longest first; layer, head; row tile; part): the
  // blocks of short requests fill the gaps that those of long ones leave (16
  // ragged requests: 188 -> 164 us)
  const bool whole = blockIdx.x < full;
  const uint32_t pb = blockIdx.x - full, ur = whole ? blockIdx.x : full + pb / splits, ui = ur / row_tiles;
  const uint32_t lh = static_cast<uint32_t>(a.n_layers) * a.Hkv, k = ui / lh, rest = ui - k * lh;
  const int32_t sp = whole ? 0 : static_cast<int32_t>(pb % splits), ns = whole ? 1 : splits;
  const int32_t rt = static_cast<int32_t>(ur - ui * row_tiles);
  const int32_t li = static_cast<int32_t>(rest / a.Hkv), h = static_cast<int32_t>(rest - li * a.Hkv);
  const int32_t r = longest_first(a, static_cast<int32_t>(k));
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t rows = __ldg(a.new_lens + r) * a.G, row0 = rt * (128 * MT);
  if (row0 >= rows) return;
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t fresh = a.k_new ? (min(row0 + 128 * MT, rows) - 1) / a.G + 1 : 0;
  const Tiles ts{(x.n_hi + 127) / 128, (x.n_lo + 127) / 128, (fresh + 127) / 128};
  // this block's share of the tiles
  const int32_t nt = ts.count(), per = (nt + ns - 1) / ns;
  const int32_t j0 = min(nt, sp * per), n = min(nt, j0 + per) - j0;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  volatile int32_t *abort = &sm.abort;

  if (tid == 0) {
    mbar_init(&sm.qready, kSoftWarps);
    mbar_init(&sm.rfull, kDeqWarps);
    mbar_init(&sm.rempty, kDeqWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.kfull[i], kDeqWarps);
      mbar_init(&sm.kempty[i], MT);
      mbar_init(&sm.vfull[i], kDeqWarps);
      mbar_init(&sm.vempty[i], MT);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pready[i], 4);
      mbar_init(&sm.odone[i], 1);
      mbar_init(&sm.turn[i], 1);
      mbar_init(&sm.done[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&sm.mfull[i], kDeqWarps);
    sm.abort = 0;
    sm.bad = 0;
    sm.u = x.u;
    sm.tok0 = tok0;
    sm.qmax = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  uint32_t qbits = 0;
  if (warp < kSoftWarps) {
    const int32_t grow = row0 + (MT == 2 ? tid : tid & 127);
    qbits = grow < rows ? row_max(a.q + ((tok0 + grow / a.G) * a.Hq + h * a.G + grow % a.G) * 128) : 0;
    const uint32_t w = __reduce_max_sync(kFull, qbits);
    if (lane == 0 && w) atomicMax(&sm.qmax, w);
  }
  // a page id out of range anywhere in the unit: logits are masked token by token
  for (int32_t k = tid; k < (x.n_hi + a.P - 1) / a.P + (x.n_lo + 2 * a.P - 1) / (2 * a.P); k += kThreads) {
    const int32_t id = __ldg(a.fwd + x.u * a.pmax + k);
    if (id < 0 || id >= a.F) {
      sm.bad = 1;
      set_error(a.status, DKV_E_INTERNAL);
    }
  }
  __syncthreads();
  const int e = block_exponent(sm.qmax);
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, abort, a.status); };
  // the same answer in every lane: the loops below hold warp-wide instructions
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };

  if (warp < kSoftWarps) {
    // ================= softmax warps: a thread per row
    const int wg = warp >> 2, row = tid & 127;
    const int32_t grow = row0 + (MT == 2 ? 128 * wg : 0) + row;  // row of the unit
    const bool have = grow < rows;
    const int32_t qi = grow / a.G, qg = grow - qi * a.G;
    const int64_t at = (tok0 + qi) * a.Hq + h * a.G + qg;
    const int shift = row_shift(qbits >> 23, e);
    const float qsum = pow2f(-shift) * stage_q(a.q + at * 128, have, MT == 2 || wg == 0 ? sm.q[MT == 2 ? wg : 0] : nullptr,
                                               row, pow2f(e + shift));
    sm.w[tid] = pow2f(-shift);
    bool odd = __any_sync(kFull, shift != 0);  // rows with a shift of their own, or references beyond kFar
    fence_async();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.qready);
    const uint64_t qs2 = f2_pack(qsum, qsum);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts_s = tmem + lanes + 128 * wg, ts_o = tmem + lanes + 256 + 128 * wg;
    float m = -INFINITY;
    uint64_t l2 = 0;  // running sum, even and odd columns
    const bool some = __any_sync(kFull, have);
    // one thread issues the warpgroup's products
    const bool issuer = (warp & 3) == 0 && lane == 0;
    constexpr uint32_t kStep = kTileBytes >> 4;
    const uint64_t dq = sw128_desc(saddr(sm.q[MT == 2 ? wg : 0]), 16, 1024);
    const uint64_t dk = sw128_desc(saddr(sm.k[0]), 16, 1024), dv = sw128_desc(saddr(sm.v[0]), kBox, 1024);
    // S of tile j: 16 channels a step
    auto issue_s = [&](int32_t j) {
      const uint64_t db = dk + (j & 1) * kStep;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t o = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
        mma_ss(tmem + 128 * wg, dq + o, db + o, idesc(false, 128, 128, false), kk > 0 ? 1u : 0u);
      }
      mma_commit(&sm.sfull[wg]);
      mma_commit(&sm.kempty[j & 1]);
    };
    // O += P V of tile j: 16 tokens a step (8 columns of P, 16 rows of V).  P of
    // 32 tokens takes the first 16 of their 32 columns of S; against new tokens
    // P is the sum of two bf16 values, the second ones in the other 16.
    auto issue_o = [&](int32_t j, bool bf16, bool first) {
      const uint32_t id = bf16 ? idesc(true, 128, 128, true) : idesc(false, 128, 128, true);
      const uint64_t db = dv + (j & 1) * kStep;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts(tmem + 256 + 128 * wg, tmem + 128 * wg + 32 * (kk >> 1) + 8 * (kk & 1), db + ((kk * 2048) >> 4), id,
               first && kk == 0 ? 0u : 1u);
      if (bf16) {  // the weights' second halves
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ts(tmem + 256 + 128 * wg, tmem + 128 * wg + 32 * (kk >> 1) + 16 + 8 * (kk & 1), db + ((kk * 2048) >> 4), id, 1u);
      }
      mma_commit(&sm.odone[wg]);
      mma_commit(&sm.vempty[j & 1]);
    };
    const int32_t first = MT == 2 ? 0 : wg, step = MT == 2 ? 1 : 2;
    if (issuer && first < n && wait(&sm.qready, 0) && wait(&sm.kfull[first & 1], 0)) {
      fence_after();
      issue_s(first);
    }
    __syncwarp();
    bool ok = true;
    int32_t t = 0;  // tiles of this warpgroup
    for (int32_t j = first; j < n && ok; j += step, ++t) {
      const Tile tl = tile_at(ts, x, fresh, j0 + j);
      const int ms = j % kMeta;
      if (!(ok = warp_wait(&sm.mfull[ms], (j / kMeta) & 1u) && warp_wait(&sm.sfull[wg], t & 1u))) break;
      fence_after();
      const int32_t lim = tl.kind == 2 ? min(tl.n, qi - tl.t0 + 1) : tl.n;
      const bool masked = __any_sync(kFull, lim < 128) || sm.bad;
      const float *sv = sm.s[ms], *zv = sm.z[ms];
      const uint8_t *valid = sm.bad ? sm.valid[ms] : nullptr;
      auto mask = [&](uint32_t (&u)[32], int c) {
        if (__builtin_expect(masked, 0)) {
          const uint32_t keep = column_mask(lim - 32 * c, valid ? valid + 32 * c : nullptr);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(keep >> i & 1u)) u[i] = 0xff800000u;
        }
      };
      // 2^(x - mo) in the place of x; returns the sum, even and odd columns
      auto weigh = [&](uint32_t (&u)[32], float mo) -> uint64_t {
        uint64_t sum[4] = {0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p0 = ex2(__uint_as_float(u[2 * i]) - mo), p1 = ex2(__uint_as_float(u[2 * i + 1]) - mo);
          sum[i & 3] = f2_add(sum[i & 3], f2_pack(p0, p1));
          u[2 * i] = __float_as_uint(p0);
          u[2 * i + 1] = __float_as_uint(p1);
        }
        return f2_add(f2_add(sum[0], sum[1]), f2_add(sum[2], sum[3]));
      };
      // P of columns 32 c .. + 31, the usual way: y - mo in one multiply-add a
      // value, -inf where masked, and the sum
      auto usual = [&](uint32_t (&u)[32], int c) -> uint64_t {
        const float mo = m == -INFINITY ? 0.0f : m - kLift;
        const uint64_t nm2 = f2_pack(-mo, -mo);
        tmem_ld32(ts_s + 32 * c, u);
        tmem_wait32(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 s = *reinterpret_cast<const float4 *>(sv + 32 * c + 4 * i);
          const float4 z = *reinterpret_cast<const float4 *>(zv + 32 * c + 4 * i);
          float y0, y1;
          f2_unpack(f2_fma(f2_pack(s.x, s.y), f2_pack(__uint_as_float(u[4 * i]), __uint_as_float(u[4 * i + 1])),
                           f2_fma(f2_pack(z.x, z.y), qs2, nm2)), y0, y1);
          u[4 * i] = __float_as_uint(y0);
          u[4 * i + 1] = __float_as_uint(y1);
          f2_unpack(f2_fma(f2_pack(s.z, s.w), f2_pack(__uint_as_float(u[4 * i + 2]), __uint_as_float(u[4 * i + 3])),
                           f2_fma(f2_pack(z.z, z.w), qs2, nm2)), y0, y1);
          u[4 * i + 2] = __float_as_uint(y0);
          u[4 * i + 3] = __float_as_uint(y1);
        }
        mask(u, c);
        return weigh(u, 0.0f);
      };
      // The same with y rounded before m is taken off, rows' own shifts, and m
      // moved to the columns' maximum where that is larger: the sum, P of the
      // tile's columns before and O of the tiles before follow.
      auto careful = [&](uint32_t (&u)[32], int c, uint64_t &sum) -> bool {
        auto y_of = [&] {
          const float w = sm.w[tid];
          tmem_ld32(ts_s + 32 * c, u);
          tmem_wait32(u);
#pragma unroll
          for (int i = 0; i < 32; ++i)
            u[i] = __float_as_uint(fmaf(sv[32 * c + i], __uint_as_float(u[i]) * w, zv[32 * c + i] * qsum));
          mask(u, c);
        };
        y_of();
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < 32; i += 2) mx = max3(mx, __uint_as_float(u[i]), __uint_as_float(u[i + 1]));
        const float mn = fmaxf(m, ceilf(mx));
        const float f = mn == m ? 1.0f : ex2(m - mn);  // a power of two, 0 at first
        if (__any_sync(kFull, f != 1.0f)) {
          l2 = f2_mul(l2, f2_pack(f, f));
          m = mn;
          odd |= __any_sync(kFull, fabsf(m) > kFar && m != -INFINITY);
          // P of earlier columns, and O where m has moved in this tile before, were
          // stored by this thread: a load sees a store only after this wait
          tmem_wait_st();
#pragma unroll 1
          for (int i = 0; i < (tl.kind == 2 ? 2 * c : c); ++i) {
            const uint32_t at_p = ts_s + (tl.kind == 2 ? 16 * i : 32 * i);
            tmem_ld16(at_p, u);
            tmem_wait16(u);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 p2 = tl.kind == 2 ? make_float2(bf16_lo(u[e]), bf16_hi(u[e])) : __half22float2(u2h(u[e]));
              u[e] = tl.kind == 2 ? bf16x2_rn(p2.x * f, p2.y * f) : f16x2_rn(p2.x * f, p2.y * f);
            }
            tmem_st16(at_p, u);
          }
          if (t > 0) {
            if (!warp_wait(&sm.odone[wg], (t - 1) & 1u)) return false;
            fence_after();
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
              tmem_ld16(ts_o + 16 * i, u);
              tmem_wait16(u);
#pragma unroll
              for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
              tmem_st16(ts_o + 16 * i, u);
            }
          }
          y_of();
        }
        sum = weigh(u, m == -INFINITY ? 0.0f : m - kLift);
        return true;
      };
      // 32 columns at a time: the short loop stays in the instruction cache.  A
      // warp of padding rows leaves its rows of P as they are.
#pragma unroll 1
      for (int c = some ? 0 : 4; c < 4; ++c) {
        uint32_t u[32];
        uint64_t sum = 0;
        bool rare = odd;
        if (!rare) {
          sum = usual(u, c);
          // a row's first columns set its reference whatever their sum: against 0
          // the weights of logits below -87 are all zero
          rare = __any_sync(kFull, f2_sum(sum) > kMost || (m == -INFINITY && lim > 32 * c));
        }
        if (__builtin_expect(rare, 0) && !(ok = careful(u, c, sum))) break;
        l2 = f2_add(l2, sum);
        if (tl.kind == 2) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float p0 = __uint_as_float(u[2 * i]), p1 = __uint_as_float(u[2 * i + 1]);
            w[i] = bf16x2_rn(p0, p1);
            u[i] = bf16x2_rest(p0, p1, w[i]);
          }
          tmem_st16(ts_s + 32 * c, w);
          tmem_st16(ts_s + 32 * c + 16, u);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) u[i] = f16x2_rn(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
          tmem_st16(ts_s + 32 * c, u);
        }
      }
      if (!ok) break;
      tmem_wait_st();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pready[wg]);
      // the warpgroups issue in turn: products that interleave would all finish
      // late and keep both warpgroups in their softmax at the same time
      if (issuer && (ok = wait(&sm.vfull[j & 1], (j >> 1) & 1u) && wait(&sm.pready[wg], t & 1u) &&
                          (wg == 0 && t == 0 || wait(&sm.turn[wg], (wg == 0 ? t - 1 : t) & 1u)))) {
        fence_after();
        issue_o(j, tl.kind == 2, t == 0);
        const int32_t jn = j + step;
        if (jn < n && (ok = wait(&sm.kfull[jn & 1], (jn >> 1) & 1u))) {
          fence_after();
          issue_s(jn);
        }
        mbar_arrive(&sm.turn[wg ^ 1]);
      }
      ok = __all_sync(kFull, ok);
    }
    if (issuer) {  // every product of the warpgroup done (also after an abort)
      mma_commit(&sm.done[wg]);
      mbar_wait(&sm.done[wg], 0, nullptr);
    }
    ok = __all_sync(kFull, ok);
    // ---- this warpgroup's rows: sums and O
    float l0, l1;
    f2_unpack(l2, l0, l1);
    const float l = l0 + l1, mo = m == -INFINITY ? 0.0f : m - kLift;
    if (ok && t > 0) ok = warp_wait(&sm.odone[wg], (t - 1) & 1u);
    fence_after();
    const int64_t n_rows = a.n_layers * a.T * a.Hq;
    const bool direct = MT == 2 && (whole || splits == 1);
    const int64_t slot = (MT == 2 ? sp : 2 * sp + wg) * part.rows + at;
    if (ok) {
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);  // NaN stays NaN
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        float f[32];
        __syncwarp();  // rows that are padding have skipped ahead
        if (t > 0) {
          tmem_ld32(ts_o + 32 * c, o);
          tmem_wait32(o);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0;
        }
        channel_order(o, f);
        if (!have || !in_range(at, n_rows, a.status)) continue;
        if (direct) {
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + at * 128 + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            dst[i] = make_uint4(bf16x2_rn(f[8 * i] * inv, f[8 * i + 1] * inv), bf16x2_rn(f[8 * i + 2] * inv, f[8 * i + 3] * inv),
                                bf16x2_rn(f[8 * i + 4] * inv, f[8 * i + 5] * inv),
                                bf16x2_rn(f[8 * i + 6] * inv, f[8 * i + 7] * inv));
        } else if (t > 0) {
          float4 *dst = reinterpret_cast<float4 *>(part.o + slot * 128 + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
        }
      }
      if (have && in_range(at, n_rows, a.status)) {
        if (!direct) part.ml[slot] = make_float2(t > 0 ? mo : -INFINITY, l);
        else if (part.ml) part.ml[at] = make_float2(0.0f, -1.0f);  // nothing to merge
        if (direct && a.lse) a.lse[at] = l == 0.0f ? -INFINITY : (mo + log2f(l)) * 0.693147180559945309f;
      }
    }
    fence_before();
  } else {
    // ================= dequantising warps
    const int dt = tid - 32 * kSoftWarps;
    const PageGeom g = page_geom(SC, a.P);
    DeqCtx d{&a, dt >> 2, dt & 3, ((dt & 3) >> 1) ^ (__popc(dt >> 2 & 7) & 1), {}};
#pragma unroll
    for (int i = 0; i < 4; ++i) d.off[i] = group_at(d.tk, 4 * d.c + (i ^ (2 * d.hs)));
    const float f = a.scale * kLog2e * pow2f(-e);
    Held<2> hd;
    bool ok = true;
    const int32_t *const fwd = a.fwd + *const_cast<volatile int64_t *>(&sm.u) * a.pmax;
    // The pages of a tile: this warp copies those numbered warp, warp + 8, ...,
    // a lane each (pages of two tokens: 65 in a tile); `page` is the lane's id.
    int32_t page = -1, k0 = 0, pages = 0;
    Tile tn{};
    auto ahead = [&](int32_t j) {
      tn = tile_at(ts, x, fresh, j0 + j);
      if (tn.kind == 2) return;
      const int32_t per = tn.kind == 0 ? a.P : 2 * a.P, k = (warp - kSoftWarps) + kDeqWarps * lane;
      k0 = tn.t0 / per;
      pages = (tn.t0 + tn.n - 1) / per - k0 + 1;
      page = k < pages ? __ldg(fwd + (tn.kind == 0 ? 0 : x.p_hi) + k0 + k) : -1;
    };
    auto copy = [&] {  // tile tn into the raw tile
      uint32_t sum = 0;
      const bool high = tn.kind == 0;
      const int32_t per = high ? a.P : 2 * a.P, k = (warp - kSoftWarps) + kDeqWarps * lane;
      const RawForm rf = high ? raw_form<KH, VH>(a.P, true) : raw_form<KH / 2, VH / 2>(a.P, false);
      const int32_t kb = high ? 16 * KH : 8 * KH, vb = high ? 16 * VH : 8 * VH;
      const int32_t p0 = (k0 + k) * per, first = max(tn.t0 - p0, 0), to = p0 + first - tn.t0;
      const int32_t n_in = min(p0 + per, tn.t0 + tn.n) - p0 - first, md = 8 * ((n_in + 1) & ~1);
      const bool mine = tn.kind != 2 && k < pages && page >= 0 && page < a.F &&  // else the tokens are masked (sm.bad)
                        in_range(to, 129 - n_in, a.status) && in_range(first, per + 1 - n_in, a.status);
      if (mine) sum = rf.whole ? rf.stride : n_in * (kb + vb) + md;
      sum = __reduce_add_sync(kFull, sum);
      if (lane == 0) mbar_expect_tx(&sm.rfull, sum);  // before any copy can land
      __syncwarp();
      if (mine) {
        const uint8_t *src = a.pages + page * g.bytes;
        if (rf.whole) {
          copy_bulk(sm.raw + (to >> rf.lg) * rf.stride, src, rf.stride, &sm.rfull);
        } else {
          copy_bulk(sm.raw + to * kb, src + first * kb, n_in * kb, &sm.rfull);
          copy_bulk(sm.raw + rf.vb + to * vb, src + g.vbase + first * vb, n_in * vb, &sm.rfull);
          copy_bulk(sm.raw + rf.mo + to * 8, src + g.meta + 8 * first, md, &sm.rfull);
        }
      }
      __syncwarp();
    };
    if (n > 0) {
      ahead(0);
      copy();
    }
    int32_t last = 0;  // the tile copied last
#pragma unroll 1
    for (int32_t j = 0; j < n; ++j) {
      const int b = j & 1, ms = j % kMeta;
      const Tile t = tn;
      if (j + 1 < n) ahead(j + 1);
      if (!(ok = warp_wait(&sm.rfull, j & 1u))) break;
      if (t.kind != 2) {  // into registers, so that the next tile's copies can go ahead
        const bool high = t.kind == 0;
        const RawForm rf = high ? raw_form<KH, VH>(a.P, true) : raw_form<KH / 2, VH / 2>(a.P, false);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const int row = d.tk + 64 * p;
          bool have = row < t.n;
          if (__builtin_expect(sm.bad, 0) && have) {
            const int32_t id = __ldg(fwd + (high ? 0 : x.p_hi) + (t.t0 + row) / (high ? a.P : 2 * a.P));
            have = id >= 0 && id < a.F;
          }
          hd.ok[p] = have;
          hd.md[p] = have ? read_md(rf, sm.raw, row) : make_uint2(0, 0);
        }
        if (high) {
          read_raw<KH>(d, rf, sm.raw, hd.k);
          read_raw<VH>(d, rf, sm.raw + rf.vb, hd.v);
        } else {
          read_raw<KH / 2>(d, rf, sm.raw, hd.k);
          read_raw<VH / 2>(d, rf, sm.raw + rf.vb, hd.v);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.rempty);
      if (j + 1 < n) {
        if (!(ok = warp_wait(&sm.rempty, j & 1u))) break;
        copy();
        last = j + 1;
      }
      if (j >= 2 && !(ok = warp_wait(&sm.kempty[b], ((j >> 1) - 1) & 1u))) break;
      if (t.kind == 0) convert_k<KH>(d, hd, sm, sm.k[b], ms, f);
      else if (t.kind == 1) convert_k<KH / 2>(d, hd, sm, sm.k[b], ms, f);
      else new_k<2, true>(d, t, *const_cast<volatile int64_t *>(&sm.tok0), h, sm, sm.k[b], ms, f);
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.kfull[b]);
        mbar_arrive(&sm.mfull[ms]);
      }
      if (j >= 2 && !(ok = warp_wait(&sm.vempty[b], ((j >> 1) - 1) & 1u))) break;
      if (t.kind == 0) convert_v<VH>(d, hd, sm.v[b]);
      else if (t.kind == 1) convert_v<VH / 2>(d, hd, sm.v[b]);
      else new_v<2>(d, t, *const_cast<volatile int64_t *>(&sm.tok0), h, sm.v[b]);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.vfull[b]);
    }
    // after an abort: this warp's last copies land before the block leaves (bounded)
    if (!ok) mbar_wait(&sm.rfull, last & 1u, nullptr);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

// Joins the partial results of a row: a warp per row, four channels a lane.
__global__ void __launch_bounds__(256) k_extend_merge(ExtendArgs a, int32_t parts, ExtendPartial part) {
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
  __shared__ int32_t ok_s;
  if (threadIdx.x < 32) {  // the lengths were wrong: the attention wrote nothing
    int64_t t = 0;
    int bad = 0;
    for (int32_t i = threadIdx.x; i < a.R; i += 32) {
      const int32_t n = __ldg(a.new_lens + i), c = __ldg(a.ctx_lens + i);
      if (n < 0 || n > a.max_new || c < 0 || static_cast<int64_t>(c) + n > a.cap) bad = 1;
      t += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      t += __shfl_xor_sync(kFull, t, o);
      bad |= __shfl_xor_sync(kFull, bad, o);
    }
    if (threadIdx.x == 0) ok_s = !bad && t == a.T;
  }
  __syncthreads();
  if (!ok_s) return;
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= part.rows) return;
  if (part.ml[at].y < 0.0f) return;  // written by its one block
  // a lane per part for the references and sums, then the parts' O one by one
  float M = -INFINITY;
  for (int32_t p = lane; p < parts; p += 32) {
    const float2 ml = part.ml[p * part.rows + at];
    if (ml.y != 0.0f) M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int32_t p0 = 0; p0 < parts; p0 += 32) {
    const float2 ml = p0 + lane < parts ? part.ml[(p0 + lane) * part.rows + at] : make_float2(0.0f, 0.0f);
    const bool some = ml.y != 0.0f;  // else it attends nothing there (or has no tile): O may not be written
    const float f = some ? ex2(ml.x - M) : 0.0f;
    if (some) l = fmaf(f, ml.y, l);
    const uint32_t live = __ballot_sync(kFull, some);
#pragma unroll 4
    for (int i = 0; i < min(32, parts - p0); ++i) {
      const float fi = __shfl_sync(kFull, f, i);
      const float4 v = live >> i & 1u
                           ? *reinterpret_cast<const float4 *>(part.o + ((p0 + i) * part.rows + at) * 128 + 4 * lane)
                           : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      o.x = fmaf(fi, v.x, o.x);
      o.y = fmaf(fi, v.y, o.y);
      o.z = fmaf(fi, v.z, o.z);
      o.w = fmaf(fi, v.w, o.w);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(kFull, l, d);
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2 *>(a.out + at * 128 + 4 * lane) =
      make_uint2(bf16x2_rn(o.x * inv, o.y * inv), bf16x2_rn(o.z * inv, o.w * inv));
  if (a.lse && lane == 0) a.lse[at] = l == 0.0f ? -INFINITY : (M + log2f(l)) * 0.693147180559945309f;
}

template <int SC, int MT>
cudaError_t launch_kernel(const ExtendArgs &a, const ExtendPlan &p, const ExtendPartial &part, cudaStream_t s) {
  const int smem = static_cast<int>(smem_bytes<MT>());
  if (cudaError_t e = cudaFuncSetAttribute(k_extend<SC, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  k_extend<SC, MT><<<static_cast<unsigned>(p.blocks), kThreads, smem, s>>>(a, p.row_tiles, static_cast<uint32_t>(p.full),
                                                                          p.splits, part);
  return cudaGetLastError();
}

template <int SC>
cudaError_t launch(const ExtendArgs &a, const ExtendPlan &p, const ExtendPartial &part, cudaStream_t s) {
  return p.mt == 1 ? launch_kernel<SC, 1>(a, p, part, s) : launch_kernel<SC, 2>(a, p, part, s);
}

}  // namespace

// Parts of a context, while the blocks with at most 32 rows do not pass two
// waves of the 152 multiprocessors, with six tiles each at least (requests of
// 2048 .. 8192 tokens with 8 heads, one wave / two / three: 1 request 30 / 30 /
// 30 us, 8: 58 / 52 / 62, 16: 90 / 80 / 87, 24: 92 / 92 / 113; powers of two up
// to three waves: 42, 72, 94 and 116).  Blocks of 128 or 256 rows: one wave (a
// request with 512 new tokens over 8192: 138 / 155 / 162 us).
constexpr int64_t kFewBlocks = 152 * 2;

ExtendPlan extend_plan(int64_t units, bool equal, int32_t max_new, int32_t G, int32_t cap, int64_t rows) {
  ExtendPlan p{};
  const int64_t most = static_cast<int64_t>(max_new) * G;
  const int64_t tiles = (static_cast<int64_t>(cap) + 127) / 128 + 2;
  p.splits = 1;
  if (most <= 32) {
    p.mt = 0;
    p.row_tiles = 1;
    p.splits = static_cast<int32_t>(
        std::clamp<int64_t>(kFewBlocks / std::max<int64_t>(units, 1), 1, std::max<int64_t>(tiles / 6, 1)));
  } else {
    p.mt = most > 128 ? 2 : 1;
    p.row_tiles = static_cast<int32_t>((most + 128 * p.mt - 1) / (128 * p.mt));
    const int64_t items = units * p.row_tiles, rest = items % 152;
    if (items < 152 || p.mt == 1) {
      p.splits = static_cast<int32_t>(std::clamp<int64_t>(152 / std::max<int64_t>(items, 1), 1, std::max<int64_t>(tiles / 4, 1)));
    } else if (equal && rest > 0 && items < 16 * 152) {
      // the last, incomplete wave in parts, as many as fill it, where every
      // request has max_new new tokens (512 row tiles: 4 waves of 1, or 3 and one
      // of 1/2).  Requests with 32 heads over 8, without parts and with them:
      //   512 new over 8192, 3 requests 436 / 324, 8: 870 / 805 us
      //   333 new over 5000, 4: 285 / 215, 11: 571 / 538, 16: 834 / 753 us
      // Of ragged ones the order fills the last wave, and parts cost more than
      // they bring (100 .. 333 new over 5000, 4: 154 / 160, 16: 558 / 569; over
      // 1000 .. 5000, 11: 250 / 250, 16: 346 / 358 us).
      p.splits = static_cast<int32_t>(std::clamp<int64_t>(152 / rest, 1, std::min<int64_t>(8, std::max<int64_t>(tiles / 4, 1))));
      if (p.splits > 1) p.full = items - rest;
    }
  }
  const int64_t items = units * p.row_tiles;
  p.blocks = p.full + (items - p.full) * p.splits;
  p.parts = p.mt == 1 ? 2 * p.splits : (p.splits == 1 ? 0 : p.splits);
  size_t o = align256(sizeof(float2) * static_cast<size_t>(p.parts) * rows);
  p.o = o;
  p.bytes = o + align256(512 * static_cast<size_t>(p.parts) * rows);
  return p;
}

cudaError_t launch_extend(const ExtendArgs &a, const ExtendPlan &p, void *ws, cudaStream_t s) {
  if (p.blocks == 0 || p.row_tiles == 0) return cudaSuccess;
  ExtendPartial part{};
  part.rows = a.n_layers * a.T * a.Hq;
  part.ml = p.parts ? static_cast<float2 *>(ws) : nullptr;
  part.o = reinterpret_cast<float *>(static_cast<uint8_t *>(ws) + p.o);
  cudaError_t e;
  if (p.mt == 0)
    e = launch_extend_few(a, p, part, s);
  else
    e = a.scheme == 0 ? launch<0>(a, p, part, s) : a.scheme == 1 ? launch<1>(a, p, part, s) : launch<2>(a, p, part, s);
  if (e != cudaSuccess || p.parts == 0) return e;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(static_cast<unsigned>((part.rows + 7) / 8));
  c.blockDim = dim3(256);
  c.stream = s;
  c.attrs = &attr;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, k_extend_merge, a, p.parts, part);
}

}  // namespace dkv
