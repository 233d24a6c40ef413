// extend_few.cu -- attention of several new tokens a request when a unit has at
// most 32 rows (drafted tokens: new tokens x query heads of the group).
//
// With so few rows the work is the conversion of the cache, and a product of
// 128 rows would be mostly padding.  Here the tokens are the long side:
//   S^T = K Q^T     a token per tensor-memory lane, 64 columns of which `rows`
//                   are real;
//   O^T += V^T P^T  channels x rows; against new tokens P in two bf16 parts.
//   copy warps (3)     bulk copies of the pages (K codes, V codes, scales and
//     zeros) into a ring of raw tiles, one tile each: loads of single threads,
//     or their asynchronous copies, cost the load unit about 1500 cycles a
//     tile, the bulk copies none, but issuing one costs its warp 54 cycles;
//   convert warps (8)  four threads a token: K codes less their middle and V =
//     fma(c, s, z), both fp16;
//   softmax warps (8)  two threads per token: the token's logits against half of
//     the rows lie in its own lane, its scale and zero are two registers;
//   MMA warp           issues every product.
//
// A row's reference m is as in extend.cu (set by the first tile), and so are its
// power of two and the care where logits are large, but a row is a column here: the
// softmax warps meet at a named barrier once per tile, which also tells whether any
// weight passed 2^15 and the references have to move (rarely).
//
// Measured (64 requests with 1 .. 8 drafts over 2048 .. 8192 tokens, 32 heads
// over 8): 224 us for 374 MB, 1.67 TB/s, 25% of the measured copy rate.  A tile
// takes about 2400 cycles: the conversion of K (880) and V (830) by eight warps,
// K behind the product that read the tile before.  The kernel for 128 rows takes
// 315 us there.  A call of four tokens over 512 takes 18 us, almost all of it
// the latency of one block's start, its few tiles and its end.
#include <algorithm>
#include <cmath>
#include <cstddef>

#include "token_tiles.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kSoftWarps = 8, kConvWarps = 8;
constexpr int kMmaWarp = kSoftWarps + kConvWarps, kCopyWarp = kMmaWarp + 1, kCopyWarps = 3;
constexpr int kThreads = 32 * (kCopyWarp + kCopyWarps);
constexpr int kNP = 2;               // tokens a convert thread holds
constexpr int kRaw = kCopyWarps;     // raw tiles in flight, one a copy warp
constexpr uint32_t kTmemCols = 256;  // S^T at 0 and 64, O^T at 128
constexpr uint32_t kColO = 128;
constexpr int kMeta = 4;             // ring of the tiles' scales and zeros
constexpr int kCols = 32;            // most rows of a unit
constexpr float kLift = 7.0f;        // P = 2^(y - m + kLift)
constexpr float kMost = 32768.0f;    // a weight above it moves m

struct __align__(1024) Smem {
  uint8_t k[kTileBytes];      // tokens x 128 channels (two boxes)
  uint8_t v[2][kTileBytes];
  uint8_t p[128 * 128];       // tokens x 64 rows
  uint8_t q[2][64 * 128];     // 64 rows x 64 channels, twice
  uint8_t raw[kRaw][200 * 128];  // a tile's pages: codes, scales and zeros (200 bytes a token at most)
  uint32_t there[kRaw][4];       // which of its tokens exist
  float s[kMeta][128], z[kMeta][128];
  uint8_t valid[kMeta][128];
  float4 col[kCols / 2];      // per pair of rows: sums of Q, -(m - lift)
  float m[kCols], f[kCols];   // references; what O is multiplied by when they move
  float l[4][kCols];          // sums per warp
  float inv[kCols];           // 1 / sum
  int64_t at[kCols];          // output rows
  uint32_t top[kCols];        // maxima of a tile, as ordered integers
  uint64_t rfull[kRaw], rempty[kRaw], kfull, kempty, mfull[kMeta], vfull[2], vempty[2], sfull[2], pready, odone, done;
  float w[kCols];             // 2^-d of the rows (row_shift)
  uint32_t qmax, tmem;
  int32_t abort, unset, odd;  // odd: a row has a shift of its own, or a reference beyond kFar
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(offsetof(Smem, q) % 1024 == 0 && offsetof(Smem, p) % 1024 == 0, "swizzled operands");
static_assert(offsetof(Smem, raw) % 1024 == 0 && sizeof(Smem::raw[0]) % 1024 == 0, "bulk copies, weights of new tokens");

__device__ __forceinline__ uint32_t ordered(float x) {
  const int32_t i = __float_as_int(x);
  return static_cast<uint32_t>(i < 0 ? ~i : i ^ static_cast<int32_t>(0x80000000u));
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __int_as_float(u & 0x80000000u ? static_cast<int32_t>(u ^ 0x80000000u) : static_cast<int32_t>(~u));
}

// Barrier of all warps but the copy warps.
__device__ __forceinline__ void meet_all() { asm volatile("bar.sync 2, %0;" ::"n"(32 * kCopyWarp) : "memory"); }

// Barrier of the softmax warps that also reduces a predicate.
__device__ __forceinline__ bool meet(bool p) {
  uint32_t r;
  asm volatile(
      "{ .reg .pred q, o; setp.ne.u32 q, %1, 0; barrier.cta.red.or.pred o, 1, 256, q; selp.u32 %0, 1, 0, o; }"
      : "=r"(r)
      : "r"(p ? 1u : 0u)
      : "memory");
  return r != 0;
}

// Pages [k0, k0 + n) of a unit's list that a tile lies in: fwd, their ids; id,
// the lane's of the first 32.
struct PageRange {
  int32_t per, k0, n, id;
  const int32_t *fwd;
};

// One warp: the pages of tile t into a raw tile (issuing a bulk copy takes a
// warp about 54 cycles, whatever its size).  P is even, so that a page's first
// slot here and an even count keep the 8-byte scales on 16-byte boundaries (an
// odd last token takes its neighbour's along, still inside the page).
template <int KH, int VH>
__device__ __forceinline__ void copy_tile(const ExtendArgs &a, const Tile &t, const PageRange &g, const PageGeom &pg,
                                          uint8_t *raw, uint32_t *there, uint64_t *bar) {
  const int lane = threadIdx.x & 31;
  const RawForm f = t.kind == 0 ? raw_form<KH, VH>(a.P, true) : raw_form<KH / 2, VH / 2>(a.P, false);
  const int32_t kb = t.kind == 0 ? 16 * KH : 8 * KH, vb = t.kind == 0 ? 16 * VH : 8 * VH;
  if (lane < 4) there[lane] = 0;
  __syncwarp();
  // bytes to come, then the copies
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t sum = 0;
#pragma unroll 1
    for (int32_t k = lane; k < g.n; k += 32) {
      const int32_t id = k < 32 ? g.id : __ldg(g.fwd + k);
      if (id < 0 || id >= a.F) {
        set_error(a.status, DKV_E_INTERNAL);
        continue;
      }
      const int32_t p0 = (g.k0 + k) * g.per, first = max(t.t0 - p0, 0);
      const int32_t n = min(p0 + g.per, t.t0 + t.n) - p0 - first, to = p0 + first - t.t0, md = 8 * ((n + 1) & ~1);
      if (!in_range(to, 129 - n, a.status) || !in_range(first, g.per + 1 - n, a.status)) continue;
      if (pass == 0) {
        sum += f.whole ? f.stride : n * (kb + vb) + md;
        for (int32_t b = to; b < to + n; b += 32 - (b & 31))  // bits [to, to + n)
          atomicOr(there + (b >> 5), (0xffffffffu >> (32 - min(32 - (b & 31), to + n - b))) << (b & 31));
        continue;
      }
      const uint8_t *src = a.pages + id * pg.bytes;
      if (f.whole) {
        copy_bulk(raw + (to >> f.lg) * f.stride, src, f.stride, bar);
      } else {
        copy_bulk(raw + to * kb, src + first * kb, n * kb, bar);
        copy_bulk(raw + f.vb + to * vb, src + pg.vbase + first * vb, n * vb, bar);
        copy_bulk(raw + f.mo + to * 8, src + pg.meta + 8 * first, md, bar);
      }
    }
    if (pass) break;
    sum = __reduce_add_sync(kFull, sum);
    __syncwarp();  // the bits above are part of what the arrival publishes
    if (lane == 0) mbar_expect_tx(bar, sum);  // before any copy can land
    __syncwarp();
  }
}

template <int SC>
__global__ void __launch_bounds__(kThreads, 1)
    k_extend_few(const __grid_constant__ ExtendArgs a, int32_t splits, ExtendPartial part) {
  constexpr int KH = scheme_kh(SC), VH = scheme_vh(SC);
  let_merge_start();
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // blocks in the order (request, the longest first; layer, head; part): the
  // short ones fill the gaps at the end (this and the copies that start before Q
  // is read: 256 -> 221 us for 64 requests of 2048 .. 8192 tokens)
  const uint32_t ui = blockIdx.x / splits, lh = static_cast<uint32_t>(a.n_layers) * a.Hkv, k = ui / lh, rest = ui - k * lh;
  const int32_t sp = static_cast<int32_t>(blockIdx.x - ui * splits);
  const int32_t li = static_cast<int32_t>(rest / a.Hkv), h = static_cast<int32_t>(rest - li * a.Hkv);
  const int32_t r = longest_first(a, static_cast<int32_t>(k));
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t nn = __ldg(a.new_lens + r), rows = nn * a.G;
  if (rows == 0) return;
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t fresh = a.k_new ? nn : 0;
  const Tiles ts{(x.n_hi + 127) / 128, (x.n_lo + 127) / 128, (fresh + 127) / 128};
  const int32_t nt = ts.count(), per = (nt + splits - 1) / splits;
  const int32_t j0 = min(nt, sp * per), n = min(nt, j0 + per) - j0;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  // output row of row c of the unit
  auto row_at = [&](int32_t c) { return (tok0 + c / a.G) * a.Hq + h * a.G + c % a.G; };
  if (n == 0) {  // no tile here: nothing to add to the row
    if (tid < rows) {
      if (part.ml) part.ml[sp * part.rows + row_at(tid)] = make_float2(-INFINITY, 0.0f);
      else if (a.lse) a.lse[row_at(tid)] = -INFINITY;
    }
    if (!part.ml)
      for (int32_t i = tid; i < rows * 16; i += kThreads)
        *reinterpret_cast<uint4 *>(a.out + row_at(i / 16) * 128 + 8 * (i % 16)) = make_uint4(0, 0, 0, 0);
    return;
  }
  volatile int32_t *abort = &sm.abort;
  if (tid == 0) {
    mbar_init(&sm.kfull, kConvWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.vfull[i], kConvWarps);
      mbar_init(&sm.vempty[i], 1);
    }
    for (int i = 0; i < kMeta; ++i) mbar_init(&sm.mfull[i], kConvWarps);
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.rfull[i], 1);
      mbar_init(&sm.rempty[i], kConvWarps);
    }
    mbar_init(&sm.kempty, 1);
    mbar_init(&sm.sfull[0], 1);
    mbar_init(&sm.sfull[1], 1);
    mbar_init(&sm.pready, kSoftWarps);
    mbar_init(&sm.odone, 1);
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    sm.qmax = 0;
    sm.odd = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  // four warps stage Q: two threads per row, 64 rows
  const int qrow = (tid & 127) >> 1, qhalf = tid & 1;
  uint4 qv[8];
  uint32_t rm = 0;  // bits of the row's largest |value|
  fence_before();
  __syncthreads();
  fence_after();
  if (warp < 4) {
    const bool have = qrow < rows;
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (have ? row_at(qrow) : 0) * 128) + 8 * qhalf;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      qv[k] = have ? __ldg(src + k) : make_uint4(0, 0, 0, 0);
      const uint32_t *w = reinterpret_cast<const uint32_t *>(&qv[k]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        rm = max(rm, max((w[q] << 16) & 0x7fffffffu, w[q] & 0x7fff0000u));  // bits of |value|: they order like it
    }
    rm = max(rm, __shfl_xor_sync(kFull, rm, 1));
    if (rm >= 0x7f800000u) rm = 0;  // a row that is not finite spoils itself alone
    const uint32_t wm = __reduce_max_sync(kFull, rm);
    if (lane == 0 && wm) atomicMax(&sm.qmax, wm);
  }
  if (warp < kCopyWarp) meet_all();  // the copy warps have gone ahead
  const int e = block_exponent(sm.qmax);
  if (warp < 4) {
    const int shift = row_shift(rm >> 23, e);
    const float sc = pow2f(e + shift);
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 y = qv[k];
      const float c0 = bf16_lo(y.x) * sc, c1 = bf16_hi(y.x) * sc, c2 = bf16_lo(y.y) * sc, c3 = bf16_hi(y.y) * sc;
      const float c4 = bf16_lo(y.z) * sc, c5 = bf16_hi(y.z) * sc, c6 = bf16_lo(y.w) * sc, c7 = bf16_hi(y.w) * sc;
      sum += ((c0 + c1) + (c2 + c3)) + ((c4 + c5) + (c6 + c7));
      *reinterpret_cast<uint4 *>(sm.q[qhalf] + qrow * 128 + ((k ^ (qrow & 7)) << 4)) =
          make_uint4(f16x2_rn(c0, c4), f16x2_rn(c1, c5), f16x2_rn(c2, c6), f16x2_rn(c3, c7));
    }
    sum += __shfl_xor_sync(kFull, sum, 1);
    if (qhalf == 0 && qrow < kCols) {
      float *dst = reinterpret_cast<float *>(&sm.col[qrow >> 1]) + (qrow & 1);
      dst[0] = sum * pow2f(-shift);
      dst[2] = 0.0f;
      sm.w[qrow] = pow2f(-shift);
      if (shift != 0) sm.odd = 1;
      sm.m[qrow] = -INFINITY;
      sm.top[qrow] = 0;
    }
    fence_async();
  }
  if (warp < kCopyWarp) meet_all();
  const uint32_t tmem = sm.tmem;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, abort, a.status); };
  // the same answer in every lane: the loops below hold warp-wide instructions
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };

  if (warp < kSoftWarps) {
    // ================= softmax warps: two threads per token
    constexpr int kMine = kCols / 2;  // rows 16 half .. + 15
    const int row = tid & 127, half = warp >> 2;  // the token of a tile
    const bool some = kMine * half < rows;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    bool ok = true, force = true;  // force: some row has no reference yet
    float l[kMine];
#pragma unroll
    for (int c = 0; c < kMine; ++c) l[c] = 0.0f;
#pragma unroll 1
    for (int32_t j = 0; j < n; ++j) {
      const int ms = j % kMeta;
      ok = ok && warp_wait(&sm.mfull[ms], (j / kMeta) & 1u);
      const Tile cur = tile_at(ts, x, fresh, j0 + j);
      const float s_cur = sm.s[ms][row], z_cur = sm.z[ms][row];
      // a new token is attended from row jt G on
      const int32_t from = (row >= cur.n || !sm.valid[ms][row] ? kCols : cur.kind == 2 ? (cur.t0 + row) * a.G : 0) - kMine * half;
      ok = ok && warp_wait(&sm.sfull[j & 1], (j >> 1) & 1u);
      fence_after();
      const uint32_t ts_s = tmem + lanes + 64 * (j & 1) + kMine * half;
      const bool masked = __any_sync(kFull, from > 0);
      const uint64_t s2 = f2_pack(s_cur, s_cur), z2 = f2_pack(z_cur, z_cur);
      const float4 *col = sm.col + (kMine / 2) * half;
      const bool odd = sm.odd != 0;
      uint32_t u[kMine];
      auto mask = [&] {
        if (masked) {
#pragma unroll
          for (int c = 0; c < kMine; ++c) u[c] = c >= from ? u[c] : 0xff800000u;
        }
      };
      // 2^x in the place of x; returns the largest
      auto weigh = [&] {
        float mx = 0.0f;
#pragma unroll
        for (int c = 0; c < kMine; c += 2) {
          const float p0 = ex2(__uint_as_float(u[c])), p1 = ex2(__uint_as_float(u[c + 1]));
          u[c] = __float_as_uint(p0);
          u[c + 1] = __float_as_uint(p1);
          mx = max3(mx, p0, p1);
        }
        return mx;
      };
      float mx = 0.0f;
      if (ok && some && !odd) {  // y - m + lift in one multiply-add a value, -inf where masked
        tmem_ld16(ts_s, u);
        tmem_wait16(u);
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) {
          const float4 cv = col[i];
          float y0, y1;
          f2_unpack(f2_fma(s2, f2_pack(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                           f2_fma(z2, f2_pack(cv.x, cv.y), f2_pack(cv.z, cv.w))), y0, y1);
          u[2 * i] = __float_as_uint(y0);
          u[2 * i + 1] = __float_as_uint(y1);
        }
        mask();
        mx = weigh();
      }
      fence_before();
      if (__builtin_expect(meet(!ok || mx > kMost || force || odd), 0)) {
        // ---- the references move to the tile's maxima where those are larger; y is
        // rounded before they are taken off, and rows' own shifts are taken back
        bool stop = meet(!ok);
        __syncwarp();
        if (!stop && some) {
          tmem_ld16(ts_s, u);
          tmem_wait16(u);
#pragma unroll
          for (int i = 0; i < kMine / 2; ++i) {
            const float4 cv = col[i];
            const float2 w = *reinterpret_cast<const float2 *>(sm.w + kMine * half + 2 * i);
            u[2 * i] = __float_as_uint(fmaf(s_cur, __uint_as_float(u[2 * i]) * w.x, z_cur * cv.x));
            u[2 * i + 1] = __float_as_uint(fmaf(s_cur, __uint_as_float(u[2 * i + 1]) * w.y, z_cur * cv.y));
          }
          mask();
#pragma unroll 1
          for (int c = 0; c < kMine; ++c) {
            uint32_t v = 0;  // u[c], with the loop kept short
#pragma unroll
            for (int i = 0; i < kMine; ++i) v = i == c ? u[i] : v;
            const uint32_t k = __reduce_max_sync(kFull, ordered(__uint_as_float(v)));
            if (lane == 0) atomicMax(&sm.top[kMine * half + c], k);
          }
        }
        if (!stop && j > 0) ok = warp_wait(&sm.odone, (j - 1) & 1u);
        stop = stop || meet(!ok);
        if (stop) {
          ok = false;
          break;
        }
        if (tid < kCols) {
          const float m0 = sm.m[tid], m1 = fmaxf(m0, ceilf(unordered(sm.top[tid])));
          sm.f[tid] = m1 == m0 ? 1.0f : ex2(m0 - m1);  // a power of two, 0 at first
          sm.m[tid] = m1;
          sm.top[tid] = 0;
          (reinterpret_cast<float *>(&sm.col[tid >> 1]) + (tid & 1))[2] = m1 == -INFINITY ? 0.0f : kLift - m1;
          const uint32_t un = __ballot_sync(kFull, tid < rows && m1 == -INFINITY);
          if (tid == 0) sm.unset = un != 0;
          if (fabsf(m1) > kFar && m1 != -INFINITY) sm.odd = 1;
        }
        meet(false);  // the next tile's first meeting keeps f until everyone has used it
        force = sm.unset != 0;
#pragma unroll
        for (int c = 0; c < kMine; ++c) l[c] *= sm.f[kMine * half + c];
        if (j > 0) {
          __syncwarp();
          fence_after();
          uint32_t o[kMine];
          tmem_ld16(tmem + lanes + kColO + kMine * half, o);
          tmem_wait16(o);
#pragma unroll
          for (int i = 0; i < kMine; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * sm.f[kMine * half + i]);
          tmem_st16(tmem + lanes + kColO + kMine * half, o);
          tmem_wait_st();
        }
        if (some) {
#pragma unroll
          for (int i = 0; i < kMine / 2; ++i) {
            u[2 * i] = __float_as_uint(__uint_as_float(u[2 * i]) + col[i].z);
            u[2 * i + 1] = __float_as_uint(__uint_as_float(u[2 * i + 1]) + col[i].w);
          }
          weigh();
        }
      }
      // P of the tile before must have been read
      if (ok && j > 0) ok = warp_wait(&sm.odone, (j - 1) & 1u);
      if (ok && some) {
        uint32_t w[kMine / 2];
#pragma unroll
        for (int c = 0; c < kMine; ++c) l[c] += __uint_as_float(u[c]);
        if (cur.kind == 2) {  // the sum of two bf16 values; the second ones go where the tile has no codes
          uint32_t rest[kMine / 2];
#pragma unroll
          for (int c = 0; c < kMine / 2; ++c) {
            const float p0 = __uint_as_float(u[2 * c]), p1 = __uint_as_float(u[2 * c + 1]);
            w[c] = bf16x2_rn(p0, p1);
            rest[c] = bf16x2_rest(p0, p1, w[c]);
          }
#pragma unroll
          for (int c = 0; c < kMine / 8; ++c)
            *reinterpret_cast<uint4 *>(sm.raw[j % kRaw] + row * 128 + (((2 * half + c) ^ (row & 7)) << 4)) =
                make_uint4(rest[4 * c], rest[4 * c + 1], rest[4 * c + 2], rest[4 * c + 3]);
        } else {
#pragma unroll
          for (int c = 0; c < kMine / 2; ++c) w[c] = f16x2_rn(__uint_as_float(u[2 * c]), __uint_as_float(u[2 * c + 1]));
        }
#pragma unroll
        for (int c = 0; c < kMine / 8; ++c)
          *reinterpret_cast<uint4 *>(sm.p + row * 128 + (((2 * half + c) ^ (row & 7)) << 4)) =
              make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
      }
      fence_async();
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.pready);
    }
    // ---- sums over the tokens: lanes, then warps
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      float v = l[c];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
      if (lane == 0) sm.l[warp & 3][kMine * half + c] = v;
    }
    meet(false);
    const int64_t n_rows = a.n_layers * a.T * a.Hq;
    if (tid < rows) {  // a thread per row: sum, reference, where it goes
      const float ls = (sm.l[0][tid] + sm.l[1][tid]) + (sm.l[2][tid] + sm.l[3][tid]);
      const float mo = sm.m[tid] == -INFINITY ? 0.0f : sm.m[tid] - kLift;
      const int64_t at = row_at(tid);
      sm.at[tid] = at;
      sm.inv[tid] = part.ml ? 1.0f : (ls == 0.0f ? 0.0f : 1.0f / ls);
      if (!in_range(at, n_rows, a.status)) sm.inv[tid] = 0.0f;
      else if (part.ml) part.ml[sp * part.rows + at] = make_float2(mo, ls);
      else if (a.lse) a.lse[at] = ls == 0.0f ? -INFINITY : (mo + log2f(ls)) * 0.693147180559945309f;
    }
    meet(false);
    ok = ok && warp_wait(&sm.odone, (n - 1) & 1u);
    fence_after();
    if (ok) {
      // this lane's channel of every row (operand order 0 4 1 5 2 6 3 7 within eight)
      const int ch = (row & ~7) | ((row & 1) << 2) | ((row & 7) >> 1);
#pragma unroll 1
      for (int c0 = kMine * half; c0 < min(rows, kMine * half + kMine); c0 += 4) {
        uint32_t o[4];
        __syncwarp();
        tmem_ld4(tmem + lanes + kColO + c0, o);
        tmem_wait4(o);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (c0 + i >= rows || !in_range(sm.at[c0 + i], n_rows, a.status)) break;
          const float v = __uint_as_float(o[i]) * sm.inv[c0 + i];
          const int64_t to = sm.at[c0 + i] * 128 + ch;
          if (part.ml) part.o[sp * part.rows * 128 + to] = v;
          else a.out[to] = static_cast<uint16_t>(bf16x2_rn(v, v));
        }
      }
    }
    fence_before();
  } else if (warp < kMmaWarp) {
    // ================= convert warps
    const int dt = tid - 32 * kSoftWarps;
    DeqCtx d{&a, dt >> 2, dt & 3, ((dt & 3) >> 1) ^ (__popc(dt >> 2 & 7) & 1), {}};
#pragma unroll
    for (int i = 0; i < 4; ++i) d.off[i] = group_at(d.tk, 4 * d.c + (i ^ (2 * d.hs)));
    const float f = a.scale * kLog2e * pow2f(-e);
    bool ok = true;
#pragma unroll 1
    for (int32_t j = 0; j < n; ++j) {
      const Tile t = tile_at(ts, x, fresh, j0 + j);
      const int ms = j % kMeta, st = j % kRaw;
      Held<kNP> hd;
      if (!(ok = warp_wait(&sm.rfull[st], (j / kRaw) & 1u))) break;
      const RawForm rf = t.kind == 0 ? raw_form<KH, VH>(a.P, true) : raw_form<KH / 2, VH / 2>(a.P, false);
#pragma unroll
      for (int p = 0; p < kNP; ++p) {
        const int row = d.tk + 128 / kNP * p;
        hd.ok[p] = sm.there[st][row >> 5] >> (row & 31) & 1u;
        hd.md[p] = hd.ok[p] ? read_md(rf, sm.raw[st], row) : make_uint2(0, 0);
      }
      if (j >= 1 && !(ok = warp_wait(&sm.kempty, (j - 1) & 1u))) break;
      if (t.kind == 0) {
        read_raw<KH>(d, rf, sm.raw[st], hd.k);
        convert_k<KH>(d, hd, sm, sm.k, ms, f);
        read_raw<VH>(d, rf, sm.raw[st] + rf.vb, hd.v);
      } else if (t.kind == 1) {
        read_raw<KH / 2>(d, rf, sm.raw[st], hd.k);
        convert_k<KH / 2>(d, hd, sm, sm.k, ms, f);
        read_raw<VH / 2>(d, rf, sm.raw[st] + rf.vb, hd.v);
      } else {
        new_k<kNP, true>(d, t, tok0, h, sm, sm.k, ms, f);
      }
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.kfull);
        mbar_arrive(&sm.mfull[ms]);
        mbar_arrive(&sm.rempty[st]);
      }
      if (j >= 2 && !(ok = warp_wait(&sm.vempty[j & 1], ((j >> 1) - 1) & 1u))) break;
      if (t.kind == 0) convert_v<VH>(d, hd, sm.v[j & 1]);
      else if (t.kind == 1) convert_v<VH / 2>(d, hd, sm.v[j & 1]);
      else new_v<kNP>(d, t, tok0, h, sm.v[j & 1]);
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.vfull[j & 1]);
    }
    (void)ok;
  } else if (warp >= kCopyWarp) {
    // ================= copy warps: a raw tile each
    const PageGeom pg = page_geom(SC, a.P);
    const int st = warp - kCopyWarp;
    bool ok = true;
    int32_t uses = 0;
    Tile t{};
    PageRange g{};
    auto ahead = [&](int32_t j) {  // tile j, and the lane's page of it
      t = tile_at(ts, x, fresh, j0 + j);
      if (t.kind == 2) return;
      const bool high = t.kind == 0;
      g.per = high ? a.P : 2 * a.P;
      g.k0 = t.t0 / g.per;
      g.n = (t.t0 + t.n - 1) / g.per - g.k0 + 1;
      g.fwd = a.fwd + x.u * a.pmax + (high ? 0 : x.p_hi) + g.k0;
      g.id = lane < g.n ? __ldg(g.fwd + lane) : -1;
    };
    if (st < n) ahead(st);
#pragma unroll 1
    for (int32_t j = st; j < n; j += kRaw) {
      if (uses > 0 && !(ok = warp_wait(&sm.rempty[st], (uses - 1) & 1u))) break;
      if (t.kind != 2) copy_tile<KH, VH>(a, t, g, pg, sm.raw[st], sm.there[st], &sm.rfull[st]);
      else if (lane == 0) mbar_arrive(&sm.rfull[st]);  // new tokens are read where they are converted
      ++uses;
      if (j + kRaw < n) ahead(j + kRaw);
    }
    // every copy has landed before the block leaves (bounded)
    if (uses > 0) mbar_wait(&sm.rfull[st], (uses - 1) & 1u, nullptr);
    (void)ok;
  } else if (lane == 0) {
    // ================= MMA warp, one lane
    const uint64_t dk = sw128_desc(saddr(sm.k), 16, 1024), dq = sw128_desc(saddr(sm.q[0]), 16, 1024);
    const uint64_t dv = sw128_desc(saddr(sm.v[0]), kBox, 1024), dp = sw128_desc(saddr(sm.p), kBox, 1024);
    bool ok = true;
#pragma unroll 1
    for (int32_t j = -1; j < n && ok; ++j) {
      if (j + 1 < n) {  // S^T of tile j + 1: 16 channels a step
        if (!(ok = wait(&sm.kfull, (j + 1) & 1u))) break;
        fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem + 64 * ((j + 1) & 1), dk + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4),
                 dq + (((kk >> 2) * (64 * 128) + (kk & 3) * 32) >> 4), idesc(false, 128, 64, false), kk > 0 ? 1u : 0u);
        mma_commit(&sm.sfull[(j + 1) & 1]);
        mma_commit(&sm.kempty);
      }
      if (j >= 0) {  // O^T += V^T P^T of tile j: 16 tokens a step
        if (!(ok = wait(&sm.vfull[j & 1], (j >> 1) & 1u) && wait(&sm.pready, j & 1u))) break;
        fence_after();
        const bool bf16 = j0 + j >= ts.hi + ts.lo;
        const uint32_t id = idesc(bf16, 128, 64, true) | kAMn;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          mma_ss(tmem + kColO, dv + (((j & 1) * kTileBytes + kk * 2048) >> 4), dp + ((kk * 2048) >> 4), id,
                 j > 0 || kk > 0 ? 1u : 0u);
        if (bf16) {  // the weights' second halves
          const uint64_t dr = sw128_desc(saddr(sm.raw[j % kRaw]), kBox, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_ss(tmem + kColO, dv + (((j & 1) * kTileBytes + kk * 2048) >> 4), dr + ((kk * 2048) >> 4), id, 1u);
        }
        mma_commit(&sm.odone);
        mma_commit(&sm.vempty[j & 1]);
      }
    }
    // every product done (also after an abort)
    mma_commit(&sm.done);
    mbar_wait(&sm.done, 0, nullptr);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

template <int SC>
cudaError_t launch(const ExtendArgs &a, const ExtendPlan &p, const ExtendPartial &part, cudaStream_t s) {
  const int smem = static_cast<int>(kSmemBytes);
  if (cudaError_t e = cudaFuncSetAttribute(k_extend_few<SC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  k_extend_few<SC><<<static_cast<unsigned>(p.blocks), kThreads, smem, s>>>(a, p.splits, part);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_few(const ExtendArgs &a, const ExtendPlan &p, const ExtendPartial &part, cudaStream_t s) {
  return a.scheme == 0 ? launch<0>(a, p, part, s) : a.scheme == 1 ? launch<1>(a, p, part, s) : launch<2>(a, p, part, s);
}

}  // namespace dkv
