// extend_sig.cu -- significance of the accepted new tokens of a request
// (dkv_extend_significance), on the fifth-generation tensor cores.
//
// Each attended token t of a unit receives, per query head of its group,
//   sum_{i < acc} p(i, t),   p(i, t) = 2^(s (q_i . c) + z (sum q_i) - lse_i)
// (s, z with scale log2 e in them, lse in log2 units), recomputed from the
// stored lse: a token's sum needs the final normaliser of every row, which the
// attention only has when it is done, and only the accepted rows count.
//
// S^T = K Q^T puts a token on a tensor-memory lane, so its scale and zero are
// two registers and its sums plain additions of one thread in a fixed order.
// A block takes a contiguous range of one unit's token tiles,
// four tiles (a group) at a time, K converted once and resident, and streams
// the rows of Q past them in blocks of 128 columns: `nb` columns per head, as
// many heads as fit (a draft of eight tokens: 16 columns for each of four
// heads), so every 16 columns belong to one head.
//   convert warps (8)  K tiles as in the attention (codes less their middle,
//     fp16); Q blocks as fp16 times one power of two per block (and one of a
//     column's own where it is far smaller), with the sums of their rows and
//     -lse (log2) per column;
//   copy warps (3)     K codes by bulk copies, their scales and positions by
//     asynchronous ones, into a ring of raw tiles;
//   MMA warp           S^T of every (block, tile) into four tensor-memory
//     buffers, one per tile of the group;
//   sum warps          a thread per token, two or four warpgroups in turn.  A
//     token's sums go to memory as additions without a result (each address
//     has one adder a call, so their order cannot show).
//
// Measured (32 heads over 8): the drafts of 64 requests over 2048 .. 8192
// tokens 160 us for 330 MB, 2.06 TB/s, 31% of the measured copy rate (a tile
// takes its conversion, about 1000 cycles, and hand-overs: 2050); 4 requests of
// 1024 tokens over 8192 560 us for 0.262 TFLOP, 468 TFLOP/s, 24% of the measured
// bf16 rate: a block of 128 columns against four tiles takes 7200 cycles, where
// the products would take 2048, the exponentials 2048 and the broadcast reads of
// the columns' sums and lse 2150 of shared memory's time, which the products'
// operands want as well.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "token_tiles.cuh"

namespace dkv {

namespace {

using namespace tc;

// Two warpgroups sum where one block of Q holds every head (then the conversion
// of K bounds the kernel, and its threads want 96 registers), four where
// several blocks stream past a group (then the sums do, and they want more
// warps): 199 and 703 us with two, 235 and 549 us with four, for 64 requests
// with drafts and for a chunk of 4 x 1024 tokens.
template <bool kMany>
struct Roles {
  static constexpr int kWg = kMany ? 4 : 2, kConv = 4 * kWg, kMma = kConv + 8, kCopy = kMma + 1;
  static constexpr int kThreads = 32 * (kCopy + 3);
};
constexpr int kConvWarps = 8, kCopyWarps = 3;
constexpr uint32_t kTmemCols = 512;
constexpr int kGroup = 4;    // token tiles resident at once
constexpr int kHeads = 8;    // most heads of a block of Q

// Raw tiles: K codes of 128 tokens, K's scales and zeros, positions.  The ring lies behind the first
// block of Q and takes the second one's place too where there is none.
template <int KH>
struct Raw {
  static constexpr int kMd = 128 * 16 * KH, kPos = kMd + 128 * 4, kSlot = kPos + 128 * 4;
};
constexpr int kExtra = 3 * Raw<8>::kSlot - kTileBytes;
constexpr int kRaw = kCopyWarps;  // a slot each

struct __align__(1024) Smem {
  uint8_t k[kGroup][kTileBytes];
  uint8_t q[2][kTileBytes];
  uint8_t extra[kExtra];
  float s[kGroup][128], z[kGroup][128];
  int32_t pos[kGroup][128];     // -1: not a token
  float4 col[4][64];            // per column pair: row sums of Q, -lse (log2)
  uint32_t there[kRaw][4];   // which of a raw tile's tokens exist
  uint64_t kfull[kGroup], kempty[kGroup], sfull[kGroup], sfree[kGroup];
  uint64_t qfull[2], qempty[2], cfull[4], cempty[4], qm[4], done, rfull[kRaw], rempty[kRaw];
  int8_t d[4][128];         // per column: row_shift
  alignas(8) uint8_t odd[4][kConvWarps];  // a convert warp's columns have such shifts, or normalisers beyond kFar
  uint32_t qmax[4];
  float qf[4];  // 2^-e of the block's Q
  uint32_t tmem;
  int32_t abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");
static_assert(offsetof(Smem, extra) == offsetof(Smem, q) + 2 * kTileBytes, "one region");

// Pages [k0, k0 + n) of a unit's list that a tile lies in: fwd, their ids; id,
// the lane's of the first 32.
struct PageRange {
  int32_t per, k0, n, id;
  uint32_t M;
  const int32_t *fwd;
};

// One warp: the tile's K codes, scales and positions into a raw tile.  The
// codes go by one bulk copy a page (issuing one takes a warp about 54 cycles,
// whatever its size), the rest by asynchronous copies of four bytes.
template <int KH>
__device__ __forceinline__ void copy_keys(const ExtendArgs &a, const Tile &t, const PageRange &g, const PageGeom &pg,
                                          uint8_t *raw, uint32_t *there, uint64_t *bar) {
  const int lane = threadIdx.x & 31;
  const int32_t rowb = t.kind == 0 ? 16 * KH : 8 * KH;
  int32_t k, slot;
  split(t.t0 + lane, g.per, g.M, k, slot);
  uint32_t have = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t in = k - g.k0, other = __shfl_sync(kFull, g.id, in & 31);
    const int32_t id = lane + 32 * i >= t.n ? -1 : in < 32 ? other : __ldg(g.fwd + in);
    const bool ok = id >= 0 && id < a.F && in_range(slot, g.per, a.status);
    if (ok) {
      const uint8_t *src = a.pages + id * pg.bytes;
      copy_async4(raw + Raw<KH>::kMd + 4 * (lane + 32 * i), src + pg.meta + 8 * slot);
      copy_async4(raw + Raw<KH>::kPos + 4 * (lane + 32 * i), src + pg.pos + 4 * slot);
    } else if (lane + 32 * i < t.n) {
      set_error(a.status, DKV_E_INTERNAL);
    }
    const uint32_t b = __ballot_sync(kFull, ok);
    have += __popc(b);
    if (lane == 0) there[i] = b;
    for (slot += 32; slot >= g.per; slot -= g.per) ++k;
  }
  if (lane == 0) mbar_expect_tx(bar, have * rowb);  // before any copy can land
  __syncwarp();
#pragma unroll 1
  for (int32_t k = lane; k < g.n; k += 32) {
    const int32_t id = k < 32 ? g.id : __ldg(g.fwd + k);
    if (id < 0 || id >= a.F) continue;
    const int32_t p0 = (g.k0 + k) * g.per, first = max(t.t0 - p0, 0);
    const int32_t n = min(p0 + g.per, t.t0 + t.n) - p0 - first;
    if (!in_range(p0 + first - t.t0, 129 - n, a.status) || !in_range(first, g.per + 1 - n, a.status)) continue;
    copy_bulk(raw + (p0 + first - t.t0) * rowb, a.pages + id * pg.bytes + first * rowb, n * rowb, bar);
  }
  arrive_async(bar);
}

// Tokens tk and tk + 64 of a raw tile: codes, scale and zero, position.
template <int W, int KH>
__device__ __forceinline__ void convert_key(const DeqCtx &d, const uint8_t *raw, const uint32_t *there, Smem &sm, int q,
                                            float f, int32_t ctx) {
  constexpr int kMid = 1 << (W - 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int row = d.tk + 64 * p;
    uint32_t x[2][4];
    read16<W>(x[0], raw + row * (16 * W) + 2 * W * (2 * d.c + d.hs));
    read16<W>(x[1], raw + row * (16 * W) + 2 * W * (2 * d.c + (d.hs ^ 1)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(x[i >> 1], i & 1, w0, w1);
      group_codes<W, kMid>(w0, w1, o);
      put(sm.k[q], d.off[i] + p * (64 * 128), o);
    }
    if (d.c == 0) {
      const bool ok = there[row >> 5] >> (row & 31) & 1u;
      const __half2 m = u2h(ok ? *reinterpret_cast<const uint32_t *>(raw + Raw<KH>::kMd + 4 * row) : 0u);
      const int32_t at = ok ? *reinterpret_cast<const int32_t *>(raw + Raw<KH>::kPos + 4 * row) : 0;
      const float s = __low2float(m), z = __high2float(m);
      sm.s[q][row] = s * f;
      sm.z[q][row] = fmaf(kMid, s, z) * f;
      const bool in = ok && at >= 0 && at < ctx;
      if (ok && !in) set_error(d.a->status, DKV_E_INTERNAL);
      sm.pos[q][row] = in ? at : -1;
    }
  }
}

// A block of Q: which heads and tokens its columns are.
struct Block {
  int32_t head0, i0;
};

template <int SC, bool kMany>
__global__ void __launch_bounds__(Roles<kMany>::kThreads, 1)
    k_extend_sig(const __grid_constant__ ExtendArgs a, int32_t splits, int32_t lg) {
  constexpr int KH = scheme_kh(SC), kWg = Roles<kMany>::kWg;
  constexpr int kConvWarp = Roles<kMany>::kConv, kMmaWarp = Roles<kMany>::kMma, kCopyWarp = Roles<kMany>::kCopy;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // blocks in the order (request, the longest first; layer, head; part)
  const uint32_t ui = blockIdx.x / splits, lh = static_cast<uint32_t>(a.n_layers) * a.Hkv, k = ui / lh, rest = ui - k * lh;
  const int32_t sp = static_cast<int32_t>(blockIdx.x - ui * splits);
  const int32_t li = static_cast<int32_t>(rest / a.Hkv), h = static_cast<int32_t>(rest - li * a.Hkv);
  const int32_t r = longest_first(a, static_cast<int32_t>(k));
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t acc_n = __ldg(a.acc_lens + r), ctx = __ldg(a.ctx_lens + r);
  if (acc_n == 0) return;
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t fresh = a.k_new ? acc_n : 0;
  const Tiles ts{(x.n_hi + 127) / 128, (x.n_lo + 127) / 128, (fresh + 127) / 128};
  // whole groups, as even as they go: a group's Q is staged whether it has one tile or four
  const int32_t nt = ts.count(), per = ((nt + kGroup - 1) / kGroup + splits - 1) / splits * kGroup;
  const int32_t j0 = min(nt, sp * per), n = min(nt, j0 + per) - j0;
  if (n == 0) return;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  volatile int32_t *abort = &sm.abort;
  // blocks of Q, 2^lg columns per head: hpb heads each, or (lg = 7) 128 tokens of one head
  const int32_t nb = 1 << lg;
  const int32_t hpb = min(a.G, min(128 >> lg, kHeads)), ib = lg == 7 ? (acc_n + 127) / 128 : 1;
  const int32_t nblk = (a.G + hpb - 1) / hpb * ib, cols = (hpb * nb + 31) & ~31, groups = (n + kGroup - 1) / kGroup;
  auto block_at = [&](int32_t b) { return Block{b / ib * hpb, b % ib * 128}; };
  // raw tiles: behind the blocks of Q, of which one is enough where it stays
  static_assert(kRaw * Raw<KH>::kSlot <= kTileBytes + kExtra && Raw<KH>::kSlot <= kExtra);
  const int32_t nraw = kMany ? 1 : kRaw;
  uint8_t *const raw = kMany ? sm.extra : sm.q[1];

  if (tid == 0) {
    for (int i = 0; i < kGroup; ++i) {
      mbar_init(&sm.kfull[i], kConvWarps);
      mbar_init(&sm.kempty[i], 4);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sfree[i], 4);
      mbar_init(&sm.cfull[i], kConvWarps);
      mbar_init(&sm.cempty[i], 4 * kWg);
      mbar_init(&sm.qm[i], kConvWarps);
      sm.qmax[i] = 0;
    }
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(&sm.rfull[i], 33);  // the copy warp's lanes and its first one's byte count
      mbar_init(&sm.rempty[i], kConvWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.qfull[i], kConvWarps);
      mbar_init(&sm.qempty[i], 1);
    }
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&sm.tmem, kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, abort, a.status); };
  // the same answer in every lane: the loops below hold warp-wide instructions
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };

  if (warp < kConvWarp) {
    // ================= sum warps: a thread per token
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const bool wide = (a.G & 3) == 0;  // sig_sum is 16-byte aligned, and so are four heads of it then
    uint64_t run = 0;  // a head's sums so far, over even and odd columns (one tile a warp where it passes a block's end)
    bool ok = true;
#pragma unroll 1
    for (int32_t g = 0; g < groups && ok; ++g) {
      const int32_t ng = min(kGroup, n - g * kGroup);
#pragma unroll 1
      for (int32_t b = 0; b < nblk && ok; ++b) {
        const int32_t qi = kMany ? g * nblk + b : 0;
        const Block bk = block_at(b);
        if ((kMany || g == 0) && !(ok = warp_wait(&sm.cfull[qi & 3], (qi >> 2) & 1u))) break;
        const float qf = sm.qf[qi & 3];
        const float4 *col = sm.col[qi & 3];
        const bool odd = *reinterpret_cast<const uint64_t *>(sm.odd[qi & 3]) != 0;
#pragma unroll 1
        for (int32_t t = wg; t < ng; t += kWg) {
          if (!(ok = warp_wait(&sm.kfull[t], g & 1u) && warp_wait(&sm.sfull[t], (g * nblk + b) & 1u))) break;
          fence_after();
          const float se = sm.s[t][row] * qf, ze = sm.z[t][row] * qf;
          const int32_t pos = sm.pos[t][row];  // -1: no token
          const uint64_t s2 = f2_pack(se, se), z2 = f2_pack(ze, ze);
          const Tile tl = tile_at(ts, x, fresh, j0 + g * kGroup + t);
          const int32_t tj = tl.kind == 2 ? tl.t0 + row : -1;  // index among the new tokens (held: -1)
          const bool diag = __any_sync(kFull, bk.i0 < tj), ends = ib == 1 || b % ib == ib - 1;
          int32_t cnt = 0;  // heads that are done, v: the last four
          float v[4];
          // blocks with odd columns have a copy of the loop of their own, out of
          // the usual one's way in the instruction cache
          auto columns = [&](auto which) {
            constexpr bool odd = decltype(which)::value;
#pragma unroll 1
            for (int32_t c = 0; c < cols; c += 16) {
              uint32_t u[16];
              __syncwarp();  // lanes without a token have skipped ahead
              tmem_ld16(tmem + lanes + 128 * t + c, u);
              tmem_wait16(u);
              if constexpr (odd) {
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * pow2f(-sm.d[qi & 3][c + i]));
              }
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 cv = col[(c >> 1) + i];
                float y0, y1;
                f2_unpack(f2_fma(s2, f2_pack(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                                 f2_fma(z2, f2_pack(cv.x, cv.y), f2_pack(cv.z, cv.w))), y0, y1);
                u[2 * i] = __float_as_uint(y0);
                u[2 * i + 1] = __float_as_uint(y1);
              }
              if constexpr (odd) {  // a normaliser's own rounding can put x above it: weights end at 1
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = __uint_as_float(u[i]) > 0.0f ? 0u : u[i];
              }
              if (diag) {  // rows before new token tj do not attend to it
                const int32_t skip = tj - bk.i0 - (c & (nb - 1));
#pragma unroll
                for (int i = 0; i < 16; ++i) u[i] = (i & (nb - 1)) < skip ? 0xff800000u : u[i];
              }
              uint64_t q8[2];  // eight columns each
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const uint64_t w = f2_pack(ex2(__uint_as_float(u[2 * i])), ex2(__uint_as_float(u[2 * i + 1])));
                q8[i >> 2] = i & 3 ? f2_add(q8[i >> 2], w) : w;
              }
              if (lg == 3) {
                v[0] = v[2];
                v[1] = v[3];
                v[2] = f2_sum(q8[0]);
                v[3] = f2_sum(q8[1]);
                cnt += 2;
              } else {
                run = f2_add(run, f2_add(q8[0], q8[1]));
                if (((c + 16) & (nb - 1)) != 0 || !ends) continue;
                v[0] = v[1];
                v[1] = v[2];
                v[2] = v[3];
                v[3] = f2_sum(run);
                run = 0;
                ++cnt;
              }
              if (((cnt & 3) != 0 && c + 16 < cols) || pos < 0) continue;
              // heads [base, cnt) of the block to their places; this thread alone adds to the token's sums
              const int32_t base = (cnt - 1) & ~3, most = min(cnt, min(hpb, a.G - bk.head0));
              const int64_t at = (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.cap + pos;
              if (!in_range(at, static_cast<int64_t>(a.L) * a.R * a.cap, a.status)) continue;
              float *dst = a.sig_sum + at * a.Hq + h * a.G + bk.head0 + cnt - 4;
              if (wide && most - base == 4 && tj < 0) {
                red_add4(dst, v[0], v[1], v[2], v[3]);
              } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                  if (cnt - 4 + q < base || cnt - 4 + q >= most) continue;
                  if (tj < 0) red_add(dst + q, v[q]);
                  else dst[q] = v[q];
                }
              }
            }
          };
          if (__builtin_expect(odd, 0)) columns(std::true_type{});
          else columns(std::false_type{});
          fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.sfree[t]);
            if (b == nblk - 1) mbar_arrive(&sm.kempty[t]);
          }
        }
        __syncwarp();
        if (lane == 0 && kMany) mbar_arrive(&sm.cempty[qi & 3]);
      }
    }
  } else if (warp < kMmaWarp) {
    // ================= convert warps
    const int dt = tid - 32 * kConvWarp;
    DeqCtx d{&a, dt >> 2, dt & 3, ((dt & 3) >> 1) ^ (__popc(dt >> 2 & 7) & 1), {}};
#pragma unroll
    for (int i = 0; i < 4; ++i) d.off[i] = group_at(d.tk, 4 * d.c + (i ^ (2 * d.hs)));
    const float f = a.scale * kLog2e;
    bool ok = true;
    // block b of Q into buffer qi
    auto stage = [&](int32_t b, int32_t qi) -> bool {
      const Block bk = block_at(b);
      uint4 v[2][4];
      uint32_t mx = 0, ex = 0;  // largest finite |value| of the block (bits), of the thread's columns (exponents)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int32_t cl = d.tk + 64 * p, hd = bk.head0 + (cl >> lg), i = bk.i0 + (cl & (nb - 1));
        const bool have = cl < hpb * nb && hd < a.G && i < acc_n;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((tok0 + i) * a.Hq + h * a.G + hd) * 128) + 4 * d.c;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[p][k] = have ? __ldg(src + (k ^ (2 * d.hs))) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t m2 = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          m2 = max_bf16x2(m2, v[p][k].x & 0x7fff7fffu);
          m2 = max_bf16x2(m2, v[p][k].y & 0x7fff7fffu);
          m2 = max_bf16x2(m2, v[p][k].z & 0x7fff7fffu);
          m2 = max_bf16x2(m2, v[p][k].w & 0x7fff7fffu);
        }
        uint32_t rm = max(m2 << 16, m2 & 0xffff0000u);  // bits of |value|: they order like it
        rm = max(rm, __shfl_xor_sync(kFull, rm, 1));
        rm = max(rm, __shfl_xor_sync(kFull, rm, 2));
        if (rm >= 0x7f800000u) rm = 0;  // an infinity spoils its own row alone
        mx = max(mx, rm);
        ex |= rm >> 23 << (8 * p);
      }
      mx = __reduce_max_sync(kFull, mx);
      if (lane == 0) {
        if (mx) atomicMax(&sm.qmax[qi & 3], mx);
        mbar_arrive(&sm.qm[qi & 3]);
      }
      if (!warp_wait(&sm.qm[qi & 3], (qi >> 2) & 1u)) return false;
      const int e = block_exponent(*const_cast<volatile uint32_t *>(&sm.qmax[qi & 3]));
      if (qi >= 2 && !warp_wait(&sm.qempty[qi & 1], ((qi >> 1) - 1) & 1u)) return false;
      if (qi >= 4 && !warp_wait(&sm.cempty[qi & 3], ((qi >> 2) - 1) & 1u)) return false;
      if (dt == 0) {
        sm.qf[qi & 3] = pow2f(-e);
        sm.qmax[(qi + 2) & 3] = 0;  // last used two blocks ago
      }
      {  // the columns' own shifts: by way of shared memory, the registers are full of Q
        const int s0 = row_shift(ex & 255u, e), s1 = row_shift(ex >> 8, e);
        if (d.c == 0) {
          sm.d[qi & 3][d.tk] = static_cast<int8_t>(s0);
          sm.d[qi & 3][d.tk + 64] = static_cast<int8_t>(s1);
        }
        const bool odd = __any_sync(kFull, (s0 | s1) != 0);
        if (lane == 0) sm.odd[qi & 3][warp - kConvWarp] = odd;
        __syncwarp();
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int32_t cl = d.tk + 64 * p, hd = bk.head0 + (cl >> lg), i = bk.i0 + (cl & (nb - 1));
        const bool have = cl < hpb * nb && hd < a.G && i < acc_n;
        const int shift = sm.d[qi & 3][cl];
        const float sc = pow2f(e + shift);
        const uint64_t sc2 = f2_pack(sc, sc);
        uint64_t acc = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 y = v[p][k];
          const uint64_t c04 = f2_mul(sc2, f2_pack(bf16_lo(y.x), bf16_lo(y.z))), c15 = f2_mul(sc2, f2_pack(bf16_hi(y.x), bf16_hi(y.z)));
          const uint64_t c26 = f2_mul(sc2, f2_pack(bf16_lo(y.y), bf16_lo(y.w))), c37 = f2_mul(sc2, f2_pack(bf16_hi(y.y), bf16_hi(y.w)));
          acc = f2_add(acc, f2_add(f2_add(c04, c15), f2_add(c26, c37)));
          *reinterpret_cast<uint4 *>(sm.q[qi & 1] + d.off[k] + p * (64 * 128)) =
              make_uint4(f16x2_of(c04), f16x2_of(c15), f16x2_of(c26), f16x2_of(c37));
        }
        float sum = f2_sum(acc);
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        if (d.c == 0) {
          const float ls = have ? a.lse[(tok0 + i) * a.Hq + h * a.G + hd] : -INFINITY;
          float *dst = reinterpret_cast<float *>(&sm.col[qi & 3][cl >> 1]) + (cl & 1);
          dst[0] = have ? sum * pow2f(-shift) : 0.0f;
          dst[2] = ls == -INFINITY ? -INFINITY : -ls * kLog2e;  // -inf: the column adds nothing
          if (fabsf(dst[2]) > kFar && ls != -INFINITY) sm.odd[qi & 3][warp - kConvWarp] = 1;
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sm.qfull[qi & 1]);
        mbar_arrive(&sm.cfull[qi & 3]);
      }
      return true;
    };
    if (!kMany) ok = stage(0, 0);
    int32_t st = 0;
    uint32_t ph = 0;
#pragma unroll 1
    for (int32_t g = 0; g < groups && ok; ++g) {
      const int32_t ng = min(kGroup, n - g * kGroup);
#pragma unroll 1
      for (int32_t b = 0; b < nblk && ok; ++b) {
        if (kMany) ok = stage(b, g * nblk + b);
        if (b > 0) continue;
#pragma unroll 1
        for (int32_t q = 0; q < ng && ok; ++q) {
          const Tile t = tile_at(ts, x, fresh, j0 + g * kGroup + q);
          const uint8_t *src = raw + st * Raw<KH>::kSlot;
          if (!(ok = warp_wait(&sm.rfull[st], ph))) break;
          if (g > 0 && !(ok = warp_wait(&sm.kempty[q], (g - 1) & 1u))) break;
          if (t.kind == 0) {
            convert_key<KH, KH>(d, src, sm.there[st], sm, q, f, ctx);
          } else if (t.kind == 1) {
            convert_key<KH / 2, KH>(d, src, sm.there[st], sm, q, f, ctx);
          } else {
            new_k<2, false>(d, t, tok0, h, sm, sm.k[q], q, f);
            if (d.c == 0) {
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                const int row = d.tk + 64 * p;
                sm.pos[q][row] = row < t.n ? ctx + t.t0 + row : -1;
              }
            }
          }
          fence_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sm.kfull[q]);
            mbar_arrive(&sm.rempty[st]);
          }
          if (++st == nraw) st = 0, ph ^= 1u;
        }
      }
    }
  } else if (warp >= kCopyWarp) {
    // ================= copy warps: a raw tile each (the first one alone where there is one raw tile)
    const PageGeom pg = page_geom(SC, a.P);
    const int st = warp - kCopyWarp;
    uint8_t *const slot = raw + st * Raw<KH>::kSlot;
    bool ok = st < nraw;
    Tile t{};
    PageRange g{};
    auto ahead = [&](int32_t j) {  // tile j, and the lane's page of it
      t = tile_at(ts, x, fresh, j0 + j);
      if (t.kind == 2) return;
      const bool high = t.kind == 0;
      int32_t last, rem;
      g.per = high ? a.P : 2 * a.P;
      g.M = 0xffffffffu / g.per + 1;
      split(t.t0, g.per, g.M, g.k0, rem);
      split(t.t0 + t.n - 1, g.per, g.M, last, rem);
      g.n = last - g.k0 + 1;
      g.fwd = a.fwd + x.u * a.pmax + (high ? 0 : x.p_hi) + g.k0;
      g.id = lane < g.n ? __ldg(g.fwd + lane) : -1;
    };
    if (ok && st < n) ahead(st);
    int32_t uses = 0;
#pragma unroll 1
    for (int32_t j = st; j < n && ok; j += nraw) {
      if (uses > 0 && !(ok = warp_wait(&sm.rempty[st], (uses - 1) & 1u))) break;
      if (t.kind != 2) {
        copy_keys<KH>(a, t, g, pg, slot, sm.there[st], &sm.rfull[st]);
      } else {  // new tokens are read where they are converted
        mbar_arrive(&sm.rfull[st]);
        if (lane == 0) mbar_arrive(&sm.rfull[st]);
      }
      ++uses;
      if (j + nraw < n) ahead(j + nraw);
    }
    // every copy has landed before the block leaves (bounded)
    if (uses > 0) mbar_wait(&sm.rfull[st], (uses - 1) & 1u, nullptr);
  } else if (lane == 0) {
    // ================= MMA warp, one lane
    const uint32_t id = idesc(false, 128, cols, false);
    const uint64_t dk = sw128_desc(saddr(sm.k[0]), 16, 1024), dq = sw128_desc(saddr(sm.q[0]), 16, 1024);
    constexpr uint32_t kStep = kTileBytes >> 4;
    bool ok = true;
    for (int32_t g = 0; g < groups && ok; ++g) {
      const int32_t ng = min(kGroup, n - g * kGroup);
      for (int32_t b = 0; b < nblk && ok; ++b) {
        const int32_t qi = kMany ? g * nblk + b : 0;
        if ((kMany || g == 0) && !(ok = wait(&sm.qfull[qi & 1], (qi >> 1) & 1u))) break;
        const int32_t use = g * nblk + b;  // of every tensor-memory buffer
        for (int32_t t = 0; t < ng; ++t) {
          if (b == 0 && !(ok = wait(&sm.kfull[t], g & 1u))) break;
          if (use > 0 && !(ok = wait(&sm.sfree[t], (use - 1) & 1u))) break;
          fence_after();
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // 16 channels a step
            const uint32_t o = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
            mma_ss(tmem + 128 * t, dk + t * kStep + o, dq + (qi & 1) * kStep + o, id, kk > 0 ? 1u : 0u);
          }
          mma_commit(&sm.sfull[t]);
        }
        if (ok && kMany) mma_commit(&sm.qempty[qi & 1]);
      }
    }
    // every MMA of the block done (also after an abort)
    mma_commit(&sm.done);
    mbar_wait(&sm.done, 0, nullptr);
  }
  __syncwarp();
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

template <int SC, bool kMany>
cudaError_t launch(const ExtendArgs &a, int64_t blocks, int32_t splits, int32_t lg, cudaStream_t s) {
  const int smem = static_cast<int>(kSmemBytes);
  if (cudaError_t e = cudaFuncSetAttribute(k_extend_sig<SC, kMany>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  k_extend_sig<SC, kMany><<<static_cast<unsigned>(blocks), Roles<kMany>::kThreads, smem, s>>>(a, splits, lg);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_sig(const ExtendArgs &a, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.n_layers) * a.R * a.Hkv;
  const int32_t lg = a.max_new <= 8 ? 3 : a.max_new <= 16 ? 4 : a.max_new <= 32 ? 5 : a.max_new <= 64 ? 6 : 7;
  // parts of a unit's tiles, a group each at least, up to two waves of blocks
  // (drafts of 16 requests: 70 / 52 / 57 us with one wave, two, three; a chunk
  // of 4 x 1024 tokens: 629 / 542 / 549 us)
  const int64_t tiles = (static_cast<int64_t>(a.cap) + 127) / 128 + 2;
  const int64_t splits = std::clamp<int64_t>(2 * 152 / std::max<int64_t>(units, 1), 1, (tiles + kGroup - 1) / kGroup);
  const int64_t blocks = units * splits;
  if (blocks == 0) return cudaSuccess;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const int32_t sp = static_cast<int32_t>(splits);
  const bool many = lg == 7 || a.G > std::min(128 >> lg, kHeads);  // more than one block of Q (max_new bounds every request)
  if (many)
    return a.scheme == 0 ? launch<0, true>(a, blocks, sp, lg, s) : a.scheme == 1 ? launch<1, true>(a, blocks, sp, lg, s)
                                                                                : launch<2, true>(a, blocks, sp, lg, s);
  return a.scheme == 0 ? launch<0, false>(a, blocks, sp, lg, s) : a.scheme == 1 ? launch<1, false>(a, blocks, sp, lg, s)
                                                                               : launch<2, false>(a, blocks, sp, lg, s);
}

}  // namespace dkv
