// chunk_sig.cu -- what a chunk's rows give every token's significance
// (dkv_chunk_significance), on the fifth-generation tensor cores.
//
// A position t receives, per query head q of its KV head's group,
//   sum_i p(i, t),   p(i, t) = 2^(s (q_i . k_t) - lse_i)   (s, lse in log2 units)
// recomputed from the stored lse.  S^T = K Q^T puts a position on a
// tensor-memory lane, so its sum is that of one thread in a fixed order; no
// other thread of the call adds to the same address.
//
// An item is a pair of key tiles (256 positions) of a unit (layer, request, KV
// head) against all its rows, in blocks of 128 columns: `nb` tokens of each of
// 128 / nb heads (nb: the power of two that holds the longest chunk, 16 .. 128;
// with 128 one head at a time).  Persistent blocks, one a multiprocessor, take
// items c, c + grid, ... of the requests in the order of their chunks' lengths,
// the longest first.
//   copy warp       K tiles and blocks of Q by TMA through a ring of tiles;
//     each block's -lse;
//   sum warps (2 x 4)  a warpgroup a key tile: its K from shared to tensor
//     memory once an item, then a thread per position: exponentials and sums;
//   product warp    S^T of every (block, key tile) into three
//     buffers.  With K in tensor memory a product reads 64 bytes a clock of
//     shared memory instead of 128, which leaves room for the normalisers'
//     broadcast reads.
//
// Measured (of 1951.6 TFLOP/s of bf16 products): 4 requests, 1024 tokens each
// after 8192, 32 heads over 8 (0.292 TFLOP) 259 us, 58%; 16 requests of 0 to 333
// tokens after 0 to 5001, 28 heads over 4 (49.3 GFLOP) 109 to 113 us, 23%; 16 tokens
// after 512 18 us.  Bound by the sum warps: the exponentials' unit, the
// products and the instructions' issue are each at 43 to 46% of their rates, and
// the three buffers let a warpgroup run at most two blocks ahead.  Sixteen sum
// warps or buffers of 96 columns took 271 to 327 us, a whole warp that waits
// for the products 267, 6 or 12 items a block for 4 266 to 269 (the ragged
// ones 107 and 144).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "chunk.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kSumWarps = 8, kCopyWarp = kSumWarps, kMmaWarp = kSumWarps + 1;
constexpr int kThreads = 32 * (kSumWarps + 2);
constexpr uint32_t kTmemCols = 512;  // K of warpgroup w at 64 w, S^T buffers at 128, 256, 384
constexpr int kRing = 6, kBufs = 3, kSegs = 4;
constexpr int kNl = 8;               // blocks' normalisers in flight
constexpr int kSort = 512;           // requests that are put in order

struct Seg {
  int32_t nk;              // key tiles (1 or 2); 0: the end
  int32_t key0;            // first position
  int32_t li, h, r;
  int32_t tok, n, ctx;     // the request's first token in the batch, its tokens, the positions before
  int32_t b0, b1, tb0, tb1;  // blocks: of heads, of tokens
};

struct __align__(1024) Smem {
  uint8_t ring[kRing][kTileBytes];
  float nl[kNl][128];      // -lse of a block's columns (log2 units); -inf: not a row
  uint64_t full[kRing], empty[kRing], nlfull[kNl], nlfree[kNl];
  uint64_t segfull, segfree, kready[2], kdone, sfull[kBufs], sfree[kBufs], done;
  Seg seg[kSegs];
  int32_t key[kSort], order[kSort];
  uint32_t tmem;
  int32_t abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// (checked build) entries of sig_sum
__device__ __forceinline__ int64_t sums_of(const ChunkArgs &a) { return static_cast<int64_t>(a.L) * a.R * a.cap * a.Hq; }

// Requests by the length of their chunks, the longest first (ties: the first
// one), when there are not more than the order has room for.
__device__ __forceinline__ void sort_requests(const ChunkArgs &a, Smem &sm) {
  if (a.R > kSort) return;
  for (int32_t i = threadIdx.x; i < a.R; i += kThreads) sm.key[i] = __ldg(a.new_lens + i);
  __syncthreads();
  for (int32_t i = threadIdx.x; i < a.R; i += kThreads) {
    const int32_t mine = sm.key[i];
    int32_t rank = 0;
    for (int32_t j = 0; j < a.R; ++j) rank += sm.key[j] > mine || (sm.key[j] == mine && j < i);
    sm.order[rank] = i;
  }
}

// kWide: blocks of 128 tokens of one head; else all tokens of several heads are in one block.
template <bool kWide>
__global__ void __launch_bounds__(kThreads, 1)
    k_chunk_sig(const __grid_constant__ ChunkArgs a, const __grid_constant__ CUtensorMap qmap,
                const __grid_constant__ CUtensorMap kmap, int32_t tokens) {
  const int32_t nb = kWide ? 128 : tokens;
  extern __shared__ unsigned char smem_raw[];
  // aligned by an offset, not by an integer address: the compiler then knows that these are shared accesses
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int64_t unused;
  if (!chunk_lens(a, 0, unused)) return;  // before any allocation
  volatile int32_t *abort = &sm.abort;
  if (tid == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < kNl; ++i) {
      mbar_init(&sm.nlfull[i], 1);
      mbar_init(&sm.nlfree[i], kSumWarps);
    }
    mbar_init(&sm.segfull, 1);
    mbar_init(&sm.segfree, kSumWarps + 1);
    for (int i = 0; i < 2; ++i) mbar_init(&sm.kready[i], 4);
    mbar_init(&sm.kdone, 1);
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sfree[i], 4);
    }
    mbar_init(&sm.done, 1);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  sort_requests(a, sm);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  const int32_t G = a.G, hb = 128 / nb, nhb = (G + hb - 1) / hb;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, abort, a.status); };
  // the same answer in every lane: the loops below hold warp-wide instructions
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };

  if (warp == kCopyWarp) {
    // ================= copies
    const int64_t units = static_cast<int64_t>(a.n_layers) * a.Hkv;
    const int32_t npg = 128 / a.B;
    auto request = [&](int32_t k) { return a.R <= kSort ? sm.order[k] : k; };
    auto pairs_of = [&](int32_t r) {
      const int32_t n = __ldg(a.new_lens + r);
      return n > 0 ? (__ldg(a.ctx_lens + r) + n - 1) / 256 + 1 : 0;
    };
    int64_t all = 0;
    for (int32_t k0 = 0; k0 < a.R; k0 += 32) {
      int64_t x = k0 + lane < a.R ? pairs_of(k0 + lane) : 0;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
      all += x;
    }
    // heads apart where there are few pairs: four items a block if that is to be had
    const int64_t grid = gridDim.x;
    const int32_t parts = static_cast<int32_t>(min(static_cast<int64_t>(nhb), max(int64_t{1}, (4 * grid + all * units - 1) / (all * units))));
    const int32_t hpp = (nhb + parts - 1) / parts, np = (nhb + hpp - 1) / hpp;
    const int64_t per = units * np;  // items of a pair
    int32_t c = 0, nq = 0, s = 0, k0 = 0;
    int64_t before = 0;  // pairs of the requests before the k0-th
    bool ok = true;
    for (int64_t item = blockIdx.x;; item += grid, ++s) {
      // the request that holds the item: 32 at a time
      Seg g{};
      int32_t rk = -1, at = 0;
      while (k0 < a.R) {
        const int32_t r = k0 + lane < a.R ? request(k0 + lane) : 0, mine = k0 + lane < a.R ? pairs_of(r) : 0;
        int32_t incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int32_t y = __shfl_up_sync(kFull, incl, o);
          if (lane >= o) incl += y;
        }
        const uint32_t m = __ballot_sync(kFull, item < (before + incl) * per);
        if (m) {
          const int src = __ffs(m) - 1;
          rk = __shfl_sync(kFull, r, src);
          const int64_t in = item - (before + __shfl_sync(kFull, incl - mine, src)) * per;
          // within a request: unit, part of the heads, pair
          const int32_t pairs = __shfl_sync(kFull, mine, src);
          const int64_t up = in / pairs;
          at = static_cast<int32_t>(in - up * pairs);
          const int32_t unit = static_cast<int32_t>(up / np), part = static_cast<int32_t>(up - static_cast<int64_t>(unit) * np);
          g.li = unit / a.Hkv;
          g.h = unit - g.li * a.Hkv;
          g.b0 = part * hpp;
          g.b1 = min(nhb, g.b0 + hpp);
          break;
        }
        before += __shfl_sync(kFull, incl, 31);
        k0 += 32;
      }
      if (rk >= 0) {
        g.r = rk;
        g.n = __ldg(a.new_lens + rk);
        g.ctx = __ldg(a.ctx_lens + rk);
        g.key0 = at * 256;
        g.nk = g.key0 + 128 < g.ctx + g.n ? 2 : 1;
        int64_t t = 0;
        for (int32_t i = lane; i < rk; i += 32) t += __ldg(a.new_lens + i);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(kFull, t, o);
        g.tok = static_cast<int32_t>(t);
        g.tb0 = max(0, g.key0 - g.ctx) / nb;
        g.tb1 = (g.n + nb - 1) / nb;
      }
      // every role has read the segment before
      if (s > 0 && !(ok = warp_wait(&sm.segfree, (s - 1) & 1u))) break;
      if (lane == 0) {
        sm.seg[s % kSegs] = g;
        mbar_arrive(&sm.segfull);
      }
      __syncwarp();
      if (g.nk == 0) break;
      const int64_t base = (static_cast<int64_t>(a.layer0) + g.li) * a.F;
      auto slot_free = [&] { return c < kRing || (ok = warp_wait(&sm.empty[c % kRing], (c / kRing - 1) & 1u)); };
      for (int32_t k = 0; k < g.nk && ok; ++k) {  // lane 2 j (+ 1): channels 0 .. 63 (64 ..) of page j
        const int32_t j = (g.key0 / 128 + k) * npg + (lane >> 1);
        int32_t id = -1;
        if ((lane >> 1) < npg && j * a.B < g.ctx + g.n) id = max(chunk_page(a, g.r, j), 0);
        const uint32_t boxes = __popc(__ballot_sync(kFull, id >= 0));
        if (!slot_free()) break;
        uint64_t *bar = &sm.full[c % kRing];
        if (lane == 0) mbar_expect_tx(bar, boxes * a.B * 128);
        __syncwarp();
        int32_t at = static_cast<int32_t>((base + id) * a.B);
        if (id >= 0 && !in_range(at, static_cast<int64_t>(a.L) * a.F * a.B + 1 - a.B, a.status)) at = 0;
        if (id >= 0)
          copy_box(sm.ring[c % kRing] + (lane & 1) * kBox + (lane >> 1) * a.B * 128, &kmap, (lane & 1) * 64, g.h, at, bar);
        ++c;
      }
      for (int32_t b = g.b0; b < g.b1 && ok; ++b)
        for (int32_t tb = g.tb0; tb < g.tb1 && ok; ++tb, ++nq) {
          const int32_t tok0 = static_cast<int32_t>(static_cast<int64_t>(g.li) * a.T + g.tok + tb * nb);
          float e[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t col = lane + 32 * i, hq = b * hb + col / nb, t = col % nb;
            e[i] = -INFINITY;
            if (hq < G && tb * nb + t < g.n && in_range(static_cast<int64_t>(tok0) + t, a.n_layers * a.T, a.status)) e[i] = __ldg(a.lse + (static_cast<int64_t>(tok0) + t) * a.Hq + g.h * G + hq);
          }
          if (!slot_free()) break;
          if (lane == 0) {
            uint64_t *bar = &sm.full[c % kRing];
            mbar_expect_tx(bar, kTileBytes);
            copy_box(sm.ring[c % kRing], &qmap, 0, tok0, g.h * G + b * hb, bar);
            copy_box(sm.ring[c % kRing] + kBox, &qmap, 64, tok0, g.h * G + b * hb, bar);
          }
          __syncwarp();
          ++c;
          const int q = nq % kNl;
          if (nq >= kNl && !(ok = warp_wait(&sm.nlfree[q], (nq / kNl - 1) & 1u))) break;
#pragma unroll
          for (int i = 0; i < 4; ++i) sm.nl[q][lane + 32 * i] = e[i] == -INFINITY ? -INFINITY : -e[i] * kLog2e;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.nlfull[q]);
        }
      if (!ok) break;
    }
    // The products have waited for every copy; where a wait gave up, the copies issued land before the block
    // leaves (bounded).
    if (lane == 0 && !ok)
      for (int32_t i = max(0, c - kRing); i < c; ++i) mbar_wait(&sm.full[i % kRing], (i / kRing) & 1u, nullptr);
  } else if (warp == kMmaWarp) {
    // ================= products: one lane waits and issues
    if (elect_one()) {
      constexpr uint32_t kStep = kTileBytes >> 4;
      const uint64_t dq = sw128_desc(saddr(sm.ring[0]), 16, 1024);
      int32_t c = 0, gb = 0;
      bool ok = true;
      for (int32_t s = 0; ok; ++s) {
        if (!(ok = wait(&sm.segfull, s & 1u))) break;
        const int32_t nk = sm.seg[s % kSegs].nk;
        const int32_t blocks = (sm.seg[s % kSegs].b1 - sm.seg[s % kSegs].b0) * (sm.seg[s % kSegs].tb1 - sm.seg[s % kSegs].tb0);
        mbar_arrive(&sm.segfree);
        if (nk == 0) break;
        for (int32_t k = 0; k < 2 && ok; ++k) {  // K is in tensor memory: its slot is free
          if (!(ok = wait(&sm.kready[k], s & 1u))) break;
          if (k < nk) mbar_arrive(&sm.empty[c++ % kRing]);
        }
        for (int32_t q = 0; q < blocks && ok; ++q, ++c) {
          const int32_t slot = c % kRing;
          if (!(ok = wait(&sm.full[slot], (c / kRing) & 1u))) break;
          for (int32_t k = 0; k < nk; ++k, ++gb) {
            const int buf = gb % kBufs;
            if (gb >= kBufs && !(ok = wait(&sm.sfree[buf], (gb / kBufs - 1) & 1u))) break;
            fence_after();
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + 128 * (1 + buf), tmem + 64 * k + 8 * kk,
                     dq + slot * kStep + (((kk >> 2) * kBox + (kk & 3) * 32) >> 4), idesc(true, 128, 128, false),
                     kk > 0 ? 1u : 0u);
            mma_commit(&sm.sfull[buf]);
            if (k == nk - 1) mma_commit(&sm.empty[slot]);
          }
        }
        if (ok) mma_commit(&sm.kdone);
      }
      // every product done (also after an abort)
      mma_commit(&sm.done);
      mbar_wait(&sm.done, 0, nullptr);
    }
  } else {
    // ================= sum warps: a thread per position
    const int wg = warp >> 2, row = tid & 127;
    const float sl2 = a.scale * kLog2e;  // logits in log2 units
    const uint64_t s2 = f2_pack(sl2, sl2);
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    int32_t c = 0, gb = 0, nq = 0;
    bool ok = true;
    for (int32_t s = 0; ok; ++s) {
      if (!(ok = warp_wait(&sm.segfull, s & 1u))) break;
      const Seg g = sm.seg[s % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.segfree);
      if (g.nk == 0) break;
      const int32_t blocks = (g.b1 - g.b0) * (g.tb1 - g.tb0);
      const int32_t key = g.key0 + 128 * wg + row;
      // the products of the segment before have read their K.  A warpgroup without a tile waits too, and says so in
      // kready: were this segment's products complete before it has seen the last one's, it would take the phase of
      // kdone for the one to come and wait on.
      if (s > 0 && !(ok = warp_wait(&sm.kdone, (s - 1) & 1u))) break;
      fence_after();
      if (wg < g.nk) {
        // ---- K to tensor memory
        const int32_t kc = c + wg;
        if (!(ok = warp_wait(&sm.full[kc % kRing], (kc / kRing) & 1u))) break;
        const uint8_t *src = sm.ring[kc % kRing] + row * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 32 channels: 16 columns
          uint32_t x[16];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4 *>(x + 4 * e) =
                *reinterpret_cast<const uint4 *>(src + (i >> 1) * kBox + 16 * (((i & 1) * 4 + e) ^ (row & 7)));
          tmem_st16(lanes + 64 * wg + 16 * i, x);
        }
        tmem_wait_st();
        fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.kready[wg]);
      c += g.nk + blocks;
      float *dst = a.sig_sum + ((static_cast<int64_t>(a.layer0) + g.li) * a.R * a.cap + static_cast<int64_t>(g.r) * a.cap + key) * a.Hq + g.h * G;
      const bool there = key < g.ctx + g.n, held = key < g.ctx;
      float acc = 0.0f;
      for (int32_t b = g.b0; b < g.b1 && ok; ++b)
        for (int32_t tb = g.tb0; tb < g.tb1 && ok; ++tb, ++nq) {
          const int q = nq % kNl;
          if (!(ok = warp_wait(&sm.nlfull[q], (nq / kNl) & 1u))) break;  // also without a tile: nlfree counts every warp
          if (wg < g.nk) {
            const int32_t gi = gb + wg, buf = gi % kBufs;
            if (!(ok = warp_wait(&sm.sfull[buf], (gi / kBufs) & 1u))) break;
            fence_after();
            const uint32_t src = lanes + 128 * (1 + buf);
            const float4 *nl = reinterpret_cast<const float4 *>(sm.nl[q]);
            // tokens of the block that the position receives from: lo <= t < hi
            const int32_t lo = key - g.ctx - tb * nb, hi = g.n - tb * nb;
            const bool masked = hi < nb || __any_sync(kFull, lo > 0);
            // weights of the tile's columns 16 k .. + 15 (v) to their sum; kMask: of tokens outside [lo, hi) none
            auto sum16 = [&](const uint32_t *v, int k, auto mask) {
              uint64_t t2[2] = {0, 0};
              const int32_t t0 = (16 * k) & (nb - 1);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float4 z = nl[4 * k + e];
                float y[4];
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1])), s2, f2_pack(z.x, z.y)), y[0], y[1]);
                f2_unpack(f2_fma(f2_pack(__uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3])), s2, f2_pack(z.z, z.w)), y[2], y[3]);
                if constexpr (decltype(mask)::value) {
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    if (t0 + 4 * e + j < lo || t0 + 4 * e + j >= hi) y[j] = -INFINITY;
                }
                t2[0] = f2_add(t2[0], f2_pack(ex2(y[0]), ex2(y[1])));
                t2[1] = f2_add(t2[1], f2_pack(ex2(y[2]), ex2(y[3])));
              }
              return f2_add(t2[0], t2[1]);
            };
            auto flush = [&](int32_t hq) {  // a head's last columns are in
              if (there && hq < G && in_range(key, a.cap, a.status) && in_range(dst + hq - a.sig_sum, sums_of(a), a.status)) {
                if (held) red_add(dst + hq, acc);
                else dst[hq] = acc;
              }
              acc = 0.0f;
            };
            auto tile = [&](auto mask) {
              uint32_t u[2][32];
              tmem_ld32(src, u[0]);
              tmem_wait32(u[0]);
              [[maybe_unused]] uint64_t t2 = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (i < 3) tmem_ld32(src + 32 * (i + 1), u[(i + 1) & 1]);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                  const uint64_t x = sum16(&u[i & 1][16 * half], 2 * i + half, mask);
                  if constexpr (kWide) {
                    t2 = f2_add(t2, x);
                  } else {
                    acc += f2_sum(x);
                    if (((32 * i + 16 * half + 16) & (nb - 1)) == 0) flush(b * hb + (32 * i + 16 * half) / nb);
                  }
                }
                if (i < 3) tmem_wait32(u[(i + 1) & 1]);
              }
              if constexpr (kWide) acc += f2_sum(t2);
            };
            if (masked) tile(std::true_type{});
            else tile(std::false_type{});
            if constexpr (kWide) {
              if (tb == g.tb1 - 1) flush(b);
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.sfree[buf]);
          }
          gb += g.nk;
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.nlfree[q]);
        }
    }
  }

  // ---- teardown: copies and products are complete (bounded waits above)
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    tmem_free(tmem, kTmemCols);
  }
}

}  // namespace

cudaError_t launch_chunk_sig(const ChunkArgs &a, cudaStream_t s) {
  int32_t nb = 16;
  while (nb < 128 && nb < a.max_new) nb *= 2;
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  alignas(64) CUtensorMap qmap, kmap;
  if ((e = chunk_map(&qmap, a.q, a.n_layers * a.T, a.q_stride, a.Hq, 128, nb, 128 / nb)) != cudaSuccess) return e;
  if ((e = chunk_map(&kmap, a.k, a.Hkv, 128, static_cast<int64_t>(a.L) * a.F * a.B, a.Hkv * int64_t{128}, 1, a.B)) != cudaSuccess)
    return e;
  auto *k = nb == 128 ? k_chunk_sig<true> : k_chunk_sig<false>;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes))) != cudaSuccess)
    return e;
  k<<<sms, kThreads, kSmemBytes, s>>>(a, qmap, kmap, nb);
  return cudaGetLastError();
}

}  // namespace dkv
