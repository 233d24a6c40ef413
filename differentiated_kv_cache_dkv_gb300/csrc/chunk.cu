// chunk.cu -- attention of a chunk of new tokens a request over bf16 pages
// (dkv_chunk_attention), on the fifth-generation tensor cores.
//
// A row is one (new token i, query head g of the KV head's group), numbered
// i G + g within its unit (layer, request, KV head); with that packing the
// heads of a group share every tile of K and V.  A row tile is tpt = 128 / G
// whole tokens, an item two row tiles (or one, when no more rows are left) of
// a unit against its keys, in key tiles of 128 positions.  Three launches:
//   k_chunk_append  stores the new tokens' K and V in their pages; block 0
//     meanwhile plans: tokens, items and key tiles of each request, and which
//     of them each block of the attention takes.
//   k_chunk         one block a multiprocessor.  Whole items first, block c
//     taking items c, c + grid, ... (neighbours read the same K and V at the
//     same time, which keeps them in L2), as many waves as leave every block at
//     or below the mean; the rest of the key tiles, laid end to end, is cut so
//     that all blocks end up with the same number.  Items that are cut leave
//     partial results.
//   k_chunk_join    joins those, each item's by several blocks.
// The roles of a block, pipelined through mbarriers:
//   copy warp       Q, K and V by TMA, a lane a page, through a ring of tiles;
//   product warps (2)  S = Q K^T and O += P V of a warpgroup each, P read from
//     tensor memory; one warpgroup's products run while the other is in its
//     softmax;
//   softmax warps (2 x 4)  a thread per row: P = 2^(x - m) in bf16 into the
//     columns of S, the running sum.
// With two row tiles the warpgroups take one each and share every key tile;
// with one they take every other key tile of it and join their results.  Up to
// 16 rows lie four times in their row tile, once in each warp's 32 lanes of
// tensor memory, and every warp weighs a quarter of a key tile's columns: eight
// softmaxes over keys of their own, joined at the end (one warp alone would
// take 3000 cycles a tile: 64 single tokens 314 us, then 273).
//
// The reference m of a row is the maximum of its first 32 columns, rounded up to a whole
// number (log2 units), and moves only when the sum of a tile's weights (of 32
// columns of it in the careful body) passes 2^13: weights and outputs in
// progress have fp32's exponent, so nothing is lost by a reference that is not
// the maximum, and the usual tile needs no maximum at all.  A row's weights then
// add up to at most 2^15 a tile, 2^8 cap: that times the largest value has to
// stay below 2^128.  P waits in registers until the test: the careful body then
// starts again from S.  What a row does not see is taken out of S before.
// With up to 16 rows every quarter's maximum is taken, and the reference moves
// when it lies more than 8 above.
//
// Measured (a whole call, its append included; of 1951.6 TFLOP/s of bf16
// products and 6773 GB/s of copies measured on the same kind of GPU):
//   4 requests, 1024 tokens each after 16384, 32 heads over 8 (1.13 TFLOP):
//     808 us, 72%.  A key tile takes 3200 cycles; its products alone, at the
//     full rate, 2048.  S = Q K^T reads both operands from shared memory, 128
//     bytes a clock, which is all there is, beside TMA's writes.
//   4 prompts of 2048 from their start (137 GFLOP): 167 us, 42%.  An item has
//     8.5 key tiles there, and between items 4700 cycles pass in which outputs
//     leave and the next first softmax has no product beside it; append 14 us.
//   16 requests, 0 to 333 tokens after 0 to 5001, 28 heads over 4 (98.7 GFLOP):
//     122 us, 41%: the same; append 8 us.
//   64 single tokens after 2047 to 8191 (1.34 GB): 270 us, 73% of the copies'
//     rate: five tiles of 32 KB a multiprocessor in flight, four of them 294 us,
//     three 383; append 13 us.
//   1 request, 16 tokens after 512: 32 us, three launches and a chain of waits.
// k_chunk has 168 registers a thread and spills 52 bytes.
#include <algorithm>
#include <cmath>
#include <cstddef>
#include <type_traits>

#include "chunk.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kBlocks = 152;        // most blocks of the attention: one a multiprocessor
constexpr int kStart = 3;           // what an item costs beside its key tiles, in key tiles: Q, the first S, the outputs
constexpr int kMaxWaves = 64;       // of whole items; the plan looks at each
constexpr int kSmemReqs = 256;      // requests, and items a unit of them, that the plan keeps in shared memory
constexpr int kSmemItems = 1024;

// Costs are in key tiles; an item's are its key tiles' and kStart before them.
struct PlanHeader {
  int64_t cut0;    // cost of the whole items that the waves take
  int32_t waves;
  int32_t ok;      // lengths valid
  int32_t pad[12];
};
struct ReqPlan {
  int64_t tile0;       // cost of the requests before
  int32_t tok0, rt0;   // tokens, items a unit of the requests before
  int32_t items;       // items a unit
  int32_t tiles;       // cost a unit
  int32_t ctx, n;
};
// An item that several blocks have a part of.
struct CutItem {
  int64_t begin, end;   // its cost lies there, key tiles behind the first kStart
  int32_t slot;         // of the first part's results (later blocks': twice their number)
  int32_t li, h, tok;   // as in Seg
  int32_t n, pad;       // n = 0: there is none
};
struct PlanPtrs {
  PlanHeader *hdr;
  ReqPlan *req;    // [R]
  int32_t *pre;    // [items a unit of all requests]: cost of the request's items before
  int64_t *cut;    // [grid + 1]: where each block's share of the cut tiles starts
  CutItem *item;   // [grid]: the cut item whose first part is the block's
  float4 *o;       // [2 grid][32][rows] partial results, four channels each
  float2 *ml;      // [2 grid][rows]: reference and sum
};

struct ChunkLayout {
  size_t req, pre, cut, item, ml, o, bytes;
  int32_t tpt, tpi, rows;  // tokens a row tile, an item; rows of a partial result
};

// Items a unit of all requests, at most.
__host__ __device__ __forceinline__ int64_t items_most(const ChunkArgs &a, int32_t tpi) { return a.T / tpi + a.R + 1; }

// (checked build) rows of the outputs
__device__ __forceinline__ int64_t outs_of(const ChunkArgs &a) { return static_cast<int64_t>(a.n_layers) * a.T * a.Hq; }

__host__ ChunkLayout chunk_layout(const ChunkArgs &a) {
  ChunkLayout w{};
  w.tpt = 128 / a.G;
  w.tpi = 2 * w.tpt;
  w.rows = std::min(w.tpi, a.max_new) * a.G;
  size_t x = align256(sizeof(PlanHeader));
  w.req = x; x = align256(x + sizeof(ReqPlan) * static_cast<size_t>(a.R));
  w.pre = x; x = align256(x + 4 * static_cast<size_t>(items_most(a, w.tpi)));
  w.cut = x; x = align256(x + 8 * (kBlocks + 1));
  w.item = x; x = align256(x + sizeof(CutItem) * kBlocks);
  w.ml = x;  x = align256(x + sizeof(float2) * 2 * kBlocks * static_cast<size_t>(w.rows));
  w.o = x;   x = align256(x + 512 * 2 * kBlocks * static_cast<size_t>(w.rows));
  w.bytes = x;
  return w;
}

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

// Exclusive prefix sum over the block; `total` gets the sum.
template <class T>
__device__ __forceinline__ T block_scan(T x, T *sm, T &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = incl;
  __syncthreads();
  T before = 0;
  total = 0;
  for (int w = 0; w < kAppendThreads / 32; ++w) {
    if (w < warp) before += sm[w];
    total += sm[w];
  }
  return before + incl - x;
}

// The request of item i: the last whose first item (rt0 U1) is at most i, among those that have items.
template <class F>
__device__ __forceinline__ int32_t find_req(int32_t R, F first, int64_t i) {
  int32_t lo = 0, hi = R - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (first(mid) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int32_t item_cost(const PlanPtrs &p, const ReqPlan &q, int32_t j) {
  return (j + 1 < q.items ? p.pre[q.rt0 + j + 1] : q.tiles) - p.pre[q.rt0 + j];
}

// Block 0: what every block of the attention takes.
__device__ void plan(const ChunkArgs &a, const PlanPtrs &p, int32_t tpi, int32_t grid) {
  __shared__ int64_t sm64[kAppendThreads / 32];
  __shared__ ReqPlan req_sm[kSmemReqs];
  __shared__ int32_t pre_sm[kSmemItems];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t U1 = static_cast<int64_t>(a.n_layers) * a.Hkv;
  // read again and again: from shared memory where there is room
  ReqPlan *req = a.R <= kSmemReqs ? req_sm : p.req;
  for (int32_t c = tid; c < grid; c += kAppendThreads) p.item[c].n = 0;
  // tokens and items before each request
  int64_t tok = 0, rts = 0;
  for (int32_t r0 = 0; r0 < a.R; r0 += kAppendThreads) {
    const int32_t r = r0 + tid;
    const int64_t n = r < a.R ? __ldg(a.new_lens + r) : 0, it = (n + tpi - 1) / tpi;
    int64_t t1, t2;
    const int64_t tb = block_scan(n, sm64, t1), ib = block_scan(it, sm64, t2);
    if (r < a.R) {
      ReqPlan q;
      q.tile0 = 0;
      q.tok0 = static_cast<int32_t>(tok + tb);
      q.rt0 = static_cast<int32_t>(rts + ib);
      q.items = static_cast<int32_t>(it);
      q.tiles = 0;
      q.ctx = __ldg(a.ctx_lens + r);
      q.n = static_cast<int32_t>(n);
      req[r] = q;
    }
    tok += t1;
    rts += t2;
  }
  int32_t *pre = rts <= kSmemItems ? pre_sm : p.pre;
  __syncthreads();
  // cost of each item: a warp a request
  for (int32_t r = warp; r < a.R; r += kAppendThreads / 32) {
    const ReqPlan q = req[r];
    int32_t sum = 0;
    for (int32_t j0 = 0; j0 < q.items; j0 += 32) {
      const int32_t j = j0 + lane;
      const int32_t t = j < q.items ? static_cast<int32_t>((q.ctx + min(static_cast<int64_t>(q.n), (j + 1) * static_cast<int64_t>(tpi)) + 127) / 128) + kStart : 0;
      int32_t incl = t;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      if (j < q.items && in_range(q.rt0 + j, items_most(a, tpi), a.status)) pre[q.rt0 + j] = sum + incl - t;
      sum += __shfl_sync(kFull, incl, 31);
    }
    if (lane == 0) req[r].tiles = sum;
  }
  __syncthreads();
  int64_t W = 0;
  for (int32_t r0 = 0; r0 < a.R; r0 += kAppendThreads) {
    const int32_t r = r0 + tid;
    const int64_t s = r < a.R ? req[r].tiles * U1 : 0;
    int64_t t1;
    const int64_t b = block_scan(s, sm64, t1);
    if (r < a.R) req[r].tile0 = W + b;
    W += t1;
  }
  __syncthreads();
  if (req == req_sm)
    for (int32_t r = tid; r < a.R; r += kAppendThreads) p.req[r] = req[r];
  if (pre == pre_sm && in_range(rts, items_most(a, tpi) + 1, a.status))
    for (int32_t i = tid; i < static_cast<int32_t>(rts); i += kAppendThreads) p.pre[i] = pre[i];
  // waves of whole items, while no block gets more than the mean
  const int64_t items = rts * U1, target = (W + grid - 1) / grid;
  auto first = [&](int32_t r) { return req[r].rt0 * U1; };
  auto tiles_of = [&](const ReqPlan &q, int32_t j) {
    return (j + 1 < q.items ? pre[q.rt0 + j + 1] : q.tiles) - pre[q.rt0 + j];
  };
  int64_t mine = 0;
  int32_t waves = 0;
  for (; waves < kMaxWaves && (waves + 1) * static_cast<int64_t>(grid) <= items; ++waves) {
    int64_t d = mine;
    if (tid < grid) {
      const int64_t i = waves * static_cast<int64_t>(grid) + tid;
      const ReqPlan &q = req[find_req(a.R, first, i)];
      d += tiles_of(q, static_cast<int32_t>((i - q.rt0 * U1) % q.items));
    }
    if (__syncthreads_or(d > target)) break;
    mine = d;
  }
  // the rest, so that every block ends at the mean
  int64_t cut0 = W;
  if (waves * static_cast<int64_t>(grid) < items) {
    const int64_t i = waves * static_cast<int64_t>(grid);
    const ReqPlan &q = req[find_req(a.R, first, i)];
    const int64_t k = i - q.rt0 * U1;
    cut0 = q.tile0 + k / q.items * q.tiles + pre[q.rt0 + static_cast<int32_t>(k % q.items)];
  }
  int64_t all;
  const int64_t b = block_scan(tid < grid ? target - mine : 0, sm64, all);
  if (tid < grid) p.cut[tid] = min(W, cut0 + b);
  if (tid == 0) {
    p.cut[grid] = W;
    *p.hdr = PlanHeader{cut0, waves, 1, {}};
  }
}

// Block 0 plans; block 1 + b stores tokens [16 b', ...) of a layer, a lane per 16 bytes.
__global__ void __launch_bounds__(kAppendThreads)
    k_chunk_append(const __grid_constant__ ChunkArgs a, const PlanPtrs p, int32_t tpi, int32_t grid) {
  let_next_launch_start();
  __shared__ int32_t req_s[kAppendTokens], pos_s[kAppendTokens];
  const uint32_t per = static_cast<uint32_t>((a.T + kAppendTokens - 1) / kAppendTokens);
  const uint32_t b = blockIdx.x == 0 ? 0 : blockIdx.x - 1;
  const int32_t li = static_cast<int32_t>(b / per);
  const int64_t t0 = static_cast<int64_t>(b % per) * kAppendTokens;
  int64_t unused;
  if (!chunk_lens(a, 0, unused)) {
    if (blockIdx.x == 0 && threadIdx.x == 0) p.hdr->ok = 0;
    return;
  }
  if (blockIdx.x == 0) {
    plan(a, p, tpi, grid);
    return;
  }
  const int32_t n = static_cast<int32_t>(min(a.T - t0, static_cast<int64_t>(kAppendTokens)));
  if (threadIdx.x < 32) {  // requests of the block's tokens
    const int lane = threadIdx.x;
    int64_t before = 0;
    int32_t done = 0;
    for (int32_t r0 = 0; r0 < a.R && done < n; r0 += 32) {
      const int32_t r = r0 + lane, m = r < a.R ? __ldg(a.new_lens + r) : 0;
      int64_t incl = m;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
      }
      const int64_t lo = before + incl - m, hi = before + incl;  // this request's tokens
      for (int64_t t = max(lo, t0); t < min(hi, t0 + n); ++t) {
        req_s[t - t0] = r;
        pos_s[t - t0] = static_cast<int32_t>(__ldg(a.ctx_lens + r) + t - lo);
      }
      before += __shfl_sync(kFull, incl, 31);
      done = static_cast<int32_t>(min(before - t0, static_cast<int64_t>(n)));
    }
  }
  __syncthreads();
  const int32_t units = a.Hkv * 16;  // 16-byte units of a token's K (or V) rows
  bool bad = false;
  for (int32_t i = threadIdx.x; i < n * units; i += kAppendThreads) {
    const int32_t t = i / units, c = i - t * units, pos = pos_s[t];
    if (!in_range(req_s[t], a.R, a.status) || !in_range(pos, a.cap, a.status) || !in_range(t0 + t, a.T, a.status)) continue;
    const int32_t id = chunk_page(a, req_s[t], pos / a.B);
    if (id < 0) continue;
    const int64_t from = (static_cast<int64_t>(li) * a.T + t0 + t) * a.kv_stride + c * 8;
    const int64_t to = (((static_cast<int64_t>(a.layer0) + li) * a.F + id) * a.B + pos % a.B) * (a.Hkv * int64_t{128}) + c * 8;
    if (!in_range(to, static_cast<int64_t>(a.L) * a.F * a.B * a.Hkv * 128 - 7, a.status)) continue;
    uint4 x[2];
    x[0] = *reinterpret_cast<const uint4 *>(a.k_new + from);
    x[1] = *reinterpret_cast<const uint4 *>(a.v_new + from);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      uint4 &y = x[kv];
      if (!(finite2(y.x) && finite2(y.y) && finite2(y.z) && finite2(y.w))) {
        bad = true;
        y = make_uint4(finite_only(y.x), finite_only(y.y), finite_only(y.z), finite_only(y.w));
      }
      *reinterpret_cast<uint4 *>((kv ? a.v : a.k) + to) = y;
    }
  }
  if (bad) set_error(a.status, DKV_E_RANGE);
}

// --------------------------------------------------------------- attention --

constexpr int kSoftWarps = 8, kCopyWarp = kSoftWarps, kMmaWarp = kSoftWarps + 1;
constexpr int kThreads = 32 * (kSoftWarps + 3);
constexpr uint32_t kTmemCols = 512;  // S (and P) of warpgroup w at 128 w, O at 256 + 128 w
constexpr int kRing = 5;             // K and V tiles in flight
constexpr int kSegs = 4;
constexpr float kMost = 0x1p13f;     // sum of a tile's weights that moves the reference
constexpr float kFar = 0x1p20f;      // references beyond it: logits are rounded before it is taken off

// What a block does next: key tiles [t0, t0 + nt) of an item.
struct Seg {
  int32_t nt;            // 0: the end
  int32_t t0;
  int32_t slot;          // of the partial results, -1: the whole item
  int32_t li, h, r;
  int32_t tok, i0, n;    // the item's first token in the batch and in the request, its tokens
  int32_t ctx;
};

struct __align__(1024) Smem {
  uint8_t q[2][kTileBytes];        // row tiles; then the second warpgroup's outputs, by column
  uint8_t ring[kRing][kTileBytes];
  uint64_t qfull, qfree, joined, qjoin, full[kRing], empty[kRing];
  uint64_t sfull[2], pready[2], odone[2], ofree[2], turn[2], ojoin, done[2];
  Seg seg[kSegs];
  float2 ml[128];                  // the second warpgroup's references and sums; [8][16] of eight warps
  uint32_t tmem;
  int32_t abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Key tiles that lie in the first x of an item's cost.
__device__ __forceinline__ int32_t tiles_in(int64_t x) { return static_cast<int32_t>(max(x - kStart, int64_t{0})); }

// Block c's segment number s: whole items c, c + grid, ..., then its share of
// the cut rest, from w on (w: where the next of those starts).
__device__ __forceinline__ Seg next_seg(const ChunkArgs &a, const PlanPtrs &p, int32_t waves, int64_t cut0, int32_t tpi,
                                        int32_t grid, int32_t s, int64_t &w) {
  const int64_t U1 = static_cast<int64_t>(a.n_layers) * a.Hkv;
  Seg g{};
  CutItem cut{};
  bool first = false;  // a cut item whose first part this is
  const int32_t c = blockIdx.x;
  int64_t k;  // item within the request
  ReqPlan q;
  int32_t r;
  if (s < waves) {
    const int64_t i = s * static_cast<int64_t>(grid) + c;
    r = find_req(a.R, [&](int32_t x) { return p.req[x].rt0 * U1; }, i);
    q = p.req[r];
    k = i - q.rt0 * U1;
    g.t0 = 0;
    g.nt = item_cost(p, q, static_cast<int32_t>(k % q.items)) - kStart;
    g.slot = -1;
  } else {
    const int64_t w0 = p.cut[c], w1 = p.cut[c + 1];
    if (w >= w1) return g;
    r = find_req(a.R, [&](int32_t x) { return p.req[x].tile0; }, w);
    q = p.req[r];
    const int64_t unit = (w - q.tile0) / q.tiles, in = (w - q.tile0) - unit * q.tiles;
    const int32_t j = find_req(q.items, [&](int32_t x) { return static_cast<int64_t>(p.pre[q.rt0 + x]); }, in);
    k = unit * q.items + j;
    const int32_t all = item_cost(p, q, j);
    const int64_t begin = w - (in - p.pre[q.rt0 + j]), end = begin + all, w2 = min(w1, end);
    g.t0 = tiles_in(w - begin);
    g.nt = tiles_in(w2 - begin) - g.t0;
    if (g.nt == 0) return g;  // the block's share ends before the item's first tile
    g.slot = g.nt == all - kStart ? -1 : 2 * c + (w == w0 ? 0 : 1);
    first = g.slot >= 0 && g.t0 == 0;
    cut = CutItem{begin, end, g.slot, 0, 0, 0, 0, 0};
    w = w2;
  }
  const int32_t unit = static_cast<int32_t>(k / q.items), j = static_cast<int32_t>(k - static_cast<int64_t>(unit) * q.items);
  g.li = unit / a.Hkv;
  g.h = unit - g.li * a.Hkv;
  g.r = r;
  g.i0 = j * tpi;
  g.n = min(tpi, q.n - g.i0);
  g.tok = q.tok0 + g.i0;
  g.ctx = q.ctx;
  if (!in_range(g.li, a.n_layers, a.status) || !in_range(g.tok, a.T + 1 - g.n, a.status) ||
      !in_range(g.slot + 1, 2 * grid + 1, a.status) || !in_range(g.ctx, a.cap + 1 - g.i0 - g.n, a.status))
    return Seg{};
  if (first && (threadIdx.x & 31) == 0) {
    cut.li = g.li;
    cut.h = g.h;
    cut.tok = g.tok;
    cut.n = g.n;
    p.item[c] = cut;
  }
  return g;
}

// Columns of 32 that a row keeps: the first `lim`.
__device__ __forceinline__ void keep_columns(uint32_t (&u)[32], int32_t lim) {
  const uint32_t m = lim >= 32 ? ~0u : (lim <= 0 ? 0u : (1u << lim) - 1u);
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (!(m >> i & 1u)) u[i] = 0xff800000u;
}

// The maximum of 32 values.
__device__ __forceinline__ float max32(const uint32_t (&u)[32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 16; ++i) m[i & 3] = max3(m[i & 3], __uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// Weights of 32 logits in bf16 (w) and what the rounding left of them (u);
// returns their sum, even and odd columns.  The logit is rounded before the
// reference is taken off, so that what is left of the largest is at most 2^8
// whatever their size (not as packed pairs: those two operations came out as
// one, without the rounding).
__device__ __forceinline__ uint64_t weigh_rounded(uint32_t (&u)[32], uint32_t *w, float sl2, float mo) {
  uint64_t t2[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float p0 = ex2(__fsub_rn(__fmul_rn(__uint_as_float(u[2 * e]), sl2), mo));
    const float p1 = ex2(__fsub_rn(__fmul_rn(__uint_as_float(u[2 * e + 1]), sl2), mo));
    t2[e & 1] = f2_add(t2[e & 1], f2_pack(p0, p1));
    w[e] = bf16x2_rn(p0, p1);
    u[e] = bf16x2_rest(p0, p1, w[e]);
  }
  return f2_add(t2[0], t2[1]);
}

// ... of the usual tile: one multiply-add a logit, bf16 weights alone.
__device__ __forceinline__ uint64_t weigh(const uint32_t (&u)[32], uint32_t *w, uint64_t sl2x2, uint64_t nm2) {
  uint64_t t2[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    float y0, y1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), sl2x2, nm2), y0, y1);
    const float p0 = ex2(y0), p1 = ex2(y1);
    t2[e & 1] = f2_add(t2[e & 1], f2_pack(p0, p1));
    w[e] = bf16x2_rn(p0, p1);
  }
  return f2_add(t2[0], t2[1]);
}

// 32 bf16 weights times a power of two.
__device__ __forceinline__ void scale_weights(uint32_t at, float f) {
  uint32_t x[16];
  tmem_ld16(at, x);
  tmem_wait16(x);
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = bf16x2_rn(bf16_lo(x[e]) * f, bf16_hi(x[e]) * f);
  tmem_st16(at, x);
  tmem_wait_st();
}

// Two 16-byte words a lane (one row), exchanged within two lanes: then e0 is of
// the even lane's row and e1 of the odd one's, the even lane's half first.
__device__ __forceinline__ void transpose2(uint4 &e0, uint4 &e1) {
  const bool b = threadIdx.x & 1;
  uint4 t = b ? e0 : e1;
  t.x = __shfl_xor_sync(kFull, t.x, 1);
  t.y = __shfl_xor_sync(kFull, t.y, 1);
  t.z = __shfl_xor_sync(kFull, t.z, 1);
  t.w = __shfl_xor_sync(kFull, t.w, 1);
  if (b) e0 = t;
  else e1 = t;
}

// This thread's row of O times f.  (The products into O were complete when S was.)
__device__ __forceinline__ void scale_row(uint32_t o, float f) {
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t x[16];
    tmem_ld16(o + 16 * c, x);
    tmem_wait16(x);
#pragma unroll
    for (int e = 0; e < 16; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
    tmem_st16(o + 16 * c, x);
  }
  tmem_wait_st();
}

__global__ void __launch_bounds__(kThreads, 1)
    k_chunk(const __grid_constant__ ChunkArgs a, const PlanPtrs p, const __grid_constant__ CUtensorMap qmap,
            const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
            const __grid_constant__ CUtensorMap qmap4, int32_t tpt, int32_t tpq, int32_t rows) {
  extern __shared__ unsigned char smem_raw[];
  // aligned by an offset, not by an integer address: the compiler then knows that these are shared accesses
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int32_t *abort = &sm.abort;
  if (tid == 0) {
    mbar_init(&sm.qfull, 1);
    mbar_init(&sm.qfree, 2 + kSoftWarps);
    mbar_init(&sm.joined, kSoftWarps);
    mbar_init(&sm.qjoin, kSoftWarps);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.done[i], 1);
      mbar_init(&sm.turn[i], 1);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.pready[i], 4);
      mbar_init(&sm.odone[i], 1);
      mbar_init(&sm.ofree[i], 4);
    }
    mbar_init(&sm.ojoin, 4);
    sm.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sm.tmem;
  after_launch_before();
  let_next_launch_start();
  const bool valid = *reinterpret_cast<volatile int32_t *>(&p.hdr->ok) != 0;
  const int32_t tpi = 2 * tpt, G = a.G;
  auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, abort, a.status); };
  // the same answer in every lane: the loops below hold warp-wide instructions
  auto warp_wait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(kFull, wait(bar, parity)) != 0; };

  if (!valid) {
    // nothing to do: the lengths have been reported
  } else if (warp == kCopyWarp) {
    // ================= copies: a segment's first K and V tiles, its Q, the others
    asm volatile("fence.proxy.async;" ::: "memory");  // the copies read what the launch before stored
    const int32_t waves = p.hdr->waves, grid = gridDim.x, npg = 128 / a.B;
    const int64_t cut0 = p.hdr->cut0;
    int64_t w = p.cut[blockIdx.x];
    int32_t c = 0, joins = 0;  // tiles of K or V copied, segments whose warpgroups joined
    bool ok = true, joining = false;
    int32_t s = 0;
    for (; ok; ++s) {
      const Seg g = next_seg(a, p, waves, cut0, tpi, grid, s, w);
      const int32_t end = g.ctx + g.i0 + g.n;  // positions the item's last row attends
      const int32_t *row = a.table + static_cast<int64_t>(g.r) * a.tmax;
      const int64_t base = (static_cast<int64_t>(a.layer0) + g.li) * a.F;
      // lane 2 k (+ 1): channels 0 .. 63 (64 ..) of the tile's page k
      auto page_of = [&](int32_t t) {
        const int32_t j = t * npg + (lane >> 1);
        if ((lane >> 1) >= npg || j * a.B >= end) return -1;
        const int32_t id = __ldg(row + j);
        if (id >= 0 && id < a.F) return id;
        set_error(a.status, DKV_E_INTERNAL);
        return 0;
      };
      auto copy_tile = [&](int32_t t, int32_t id) {
        const uint32_t boxes = __popc(__ballot_sync(kFull, id >= 0));
        int32_t at = static_cast<int32_t>((base + id) * a.B);
        if (id >= 0 && !in_range(at, static_cast<int64_t>(a.L) * a.F * a.B + 1 - a.B, a.status)) at = 0;
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int32_t slot = c % kRing;
          if (c >= kRing && !(ok = warp_wait(&sm.empty[slot], (c / kRing - 1) & 1u))) return;
          if (lane == 0) mbar_expect_tx(&sm.full[slot], boxes * a.B * 128);
          __syncwarp();
          if (id >= 0)
            copy_box(sm.ring[slot] + (lane & 1) * kBox + (lane >> 1) * a.B * 128, kv ? &vmap : &kmap, (lane & 1) * 64, g.h, at,
                     &sm.full[slot]);
          ++c;
        }
      };
      int32_t id = 0;
      if (g.nt > 0) {
        id = page_of(g.t0);
        copy_tile(g.t0, id);
        if (!ok) break;
        id = g.nt > 1 ? page_of(g.t0 + 1) : -1;
      }
      // Q when the products of the segment before have read theirs, every warp has read what the segment is
      // (so that none of them misses a phase of qfull) and its outputs have left the place
      if (s > 0 && !(ok = warp_wait(&sm.qfree, (s - 1) & 1u))) break;
      if (joining) {
        if (!(ok = warp_wait(&sm.joined, joins & 1u))) break;
        ++joins;
      }
      if (lane == 0) {
        sm.seg[s % kSegs] = g;
        if (g.nt > 0) {
          const int32_t at = static_cast<int32_t>(g.li * a.T + g.tok);
          if (g.n <= tpq) {
            mbar_expect_tx(&sm.qfull, 4 * 2 * tpq * G * 128);
            for (int t = 0; t < 4; ++t)
              for (int half = 0; half < 2; ++half)
                copy_box(sm.q[0] + half * kBox + 32 * t * 128, &qmap4, half * 64, g.h * G, at, &sm.qfull);
          } else {
            const int tiles = g.n > tpt ? 2 : 1;
            mbar_expect_tx(&sm.qfull, tiles * 2 * tpt * G * 128);
            for (int t = 0; t < tiles; ++t)
              for (int half = 0; half < 2; ++half)
                copy_box(sm.q[t] + half * kBox, &qmap, half * 64, g.h * G, at + t * tpt, &sm.qfull);
          }
        } else {
          mbar_arrive(&sm.qfull);
        }
      }
      __syncwarp();
      if (g.nt == 0) break;
      joining = g.n <= tpq || (g.n <= tpt && g.nt > 1);
      for (int32_t t = 1; t < g.nt && ok; ++t) {
        const int32_t now = id;
        id = t + 1 < g.nt ? page_of(g.t0 + t + 1) : -1;
        copy_tile(g.t0 + t, now);
      }
    }
    // The products have waited for every copy; where a wait gave up, the copies issued land before the block
    // leaves (bounded).
    if (lane == 0 && !ok) {
      if (s > 0) mbar_wait(&sm.qfull, (s - 1) & 1u, nullptr);
      for (int32_t i = max(0, c - kRing); i < c; ++i) mbar_wait(&sm.full[i % kRing], (i / kRing) & 1u, nullptr);
    }
  } else if (warp >= kMmaWarp) {
    // ================= products: a warp waits, one lane issues.  With two row tiles each of the two warps has a
    // warpgroup's products, and while one waits, the other's keep the tensor cores busy.  With one the first
    // warp has both, in turn.  Both warps see every tile of the ring land, in order, and a slot is free when
    // both are done with it: a warp that skipped some could take a phase of a barrier for a later one.
    const int me = warp - kMmaWarp;
    constexpr uint32_t kStep = kTileBytes >> 4;
    const uint64_t dq = sw128_desc(saddr(sm.q[0]), 16, 1024), dk = sw128_desc(saddr(sm.ring[0]), 16, 1024);
    const uint64_t dv = sw128_desc(saddr(sm.ring[0]), kBox, 1024);
    int32_t base = 0, np[2] = {0, 0}, nseg[2] = {0, 0};  // tiles so far; P taken, segments by warpgroup
    int32_t turns = 0;                                   // tiles of two row tiles so far
    bool ok = true, by_two = false;                      // the second warpgroup's last products: the second warp's
    for (int32_t s = 0; ok; ++s) {
      if (!(ok = warp_wait(&sm.qfull, s & 1u))) break;
      const int32_t nt = sm.seg[s % kSegs].nt;
      if (nt == 0) break;
      const bool two = sm.seg[s % kSegs].n > tpt;
      if (!two && me == 1) {  // sees the tiles only
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.qfree);
        for (int32_t i = 2 * base; i < 2 * (base + nt) && ok; ++i) {
          if (!(ok = warp_wait(&sm.full[i % kRing], (i / kRing) & 1u))) break;
          if (lane == 0) mbar_arrive(&sm.empty[i % kRing]);
        }
      } else {
        auto scores = [&](int32_t t) {
          const int wg = two ? me : t & 1;
          const int32_t i = 2 * (base + t), slot = i % kRing;
          if (!(ok = warp_wait(&sm.full[slot], (i / kRing) & 1u))) return;
          // the other warp's products into this warpgroup's columns, of the segment before, are complete
          if (wg == 1 && t < 2 && nseg[1] > 0 && by_two != two && (two ? t == 0 : t == 1) &&
              !(ok = warp_wait(&sm.odone[1], (nseg[1] - 1) & 1u)))
            return;
          fence_after();
          if (elect_one()) {
            const uint64_t da = dq + (two && me ? kStep : 0), db = dk + slot * kStep;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t o = ((kk >> 2) * kBox + (kk & 3) * 32) >> 4;
              mma_ss(tmem + 128 * wg, da + o, db + o, idesc(true, 128, 128, false), kk > 0 ? 1u : 0u);
            }
            mma_commit(&sm.sfull[wg]);
            mma_commit(&sm.empty[slot]);
            if (t == nt - 1) mma_commit(&sm.qfree);
          }
          __syncwarp();
        };
        const int32_t ahead = two ? 1 : 2;  // tiles whose S is issued before the first P is waited for
        // Products go in turn, PV and S of one warpgroup, then of the other.  Mixed, they would end together,
        // and both warpgroups would be in their softmax at the same time, with the tensor cores idle (a late
        // chunk: 1016 us mixed).
        auto other_turn = [&] {
          if (two && lane == 0) mbar_arrive(&sm.turn[me ^ 1]);
        };
        scores(0);
        if (me == 1) other_turn();
        if (!two && ok && nt > 1) scores(1);
        for (int32_t t = 0; t < nt && ok; ++t) {
          const int wg = two ? me : t & 1;
          const int32_t i = 2 * (base + t) + 1, slot = i % kRing;
          if (!(ok = warp_wait(&sm.full[slot], (i / kRing) & 1u))) break;
          // O of the segment before has been read
          if (t < ahead && nseg[wg] > 0 && !(ok = warp_wait(&sm.ofree[wg], (nseg[wg] - 1) & 1u))) break;
          const int32_t taken = np[wg] + (two ? t : t >> 1);
          if (!(ok = warp_wait(&sm.pready[wg], taken & 1u))) break;
          if (two && !(ok = warp_wait(&sm.turn[me], (turns + t) & 1u))) break;
          fence_after();
          if (elect_one()) {
            const uint64_t db = dv + slot * kStep;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_ts(tmem + 256 + 128 * wg, tmem + 128 * wg + 32 * (kk >> 1) + 8 * (kk & 1), db + ((kk * 2048) >> 4),
                     idesc(true, 128, 128, true), t < ahead && kk == 0 ? 0u : 1u);
            if (!two) {  // the weights' second halves
#pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                mma_ts(tmem + 256 + 128 * wg, tmem + 128 * wg + 32 * (kk >> 1) + 16 + 8 * (kk & 1), db + ((kk * 2048) >> 4),
                       idesc(true, 128, 128, true), 1u);
            }
            if (t + ahead >= nt) mma_commit(&sm.odone[wg]);
            mma_commit(&sm.empty[slot]);
          }
          __syncwarp();
          if (t + ahead < nt) scores(t + ahead);
          if (me == 0 || t + 1 < nt) other_turn();
        }
        if (two) turns += nt;
      }
      np[0] += two ? nt : (nt + 1) / 2;
      np[1] += two ? nt : nt / 2;
      ++nseg[0];
      if (two || nt > 1) {
        ++nseg[1];
        by_two = two;
      }
      base += nt;
    }
    // every product of this warp done (also after an abort)
    if (elect_one()) mma_commit(&sm.done[me]);
    __syncwarp();
    mbar_wait(&sm.done[me], 0, nullptr);
  } else {
    // ================= softmax warps: a thread per row
    const int wg = warp >> 2, row = tid & 127;
    const float sl2 = a.scale * kLog2e;  // logits in log2 units
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t ts_s = tmem + lanes + 128 * wg, ts_o = tmem + lanes + 256 + 128 * wg;
    int32_t base = 0, ns = 0, nseg = 0, joins = 0, qjoins = 0;
    bool ok = true;
    for (int32_t s = 0; ok; ++s) {
      if (!(ok = warp_wait(&sm.qfull, s & 1u))) break;
      // read where it is needed: every register counts in the loop over the tiles
      const Seg &g = sm.seg[s % kSegs];
      const int32_t nt = g.nt;
      const bool two = g.n > tpt;
      const bool four = g.n <= tpq;                   // the rows lie four times in the row tile
      const int32_t rt = (four ? lane : row) / G;     // token of the row tile
      const int32_t i = (two && wg ? tpt : 0) + rt;   // token of the item
      const bool live = rt < (four ? tpq : tpt) && i < g.n;
      // of the segment's first key tile: columns this row keeps, positions the item has
      const int32_t lim0 = g.ctx + g.i0 + i + 1 - 128 * g.t0, end0 = g.ctx + g.i0 + g.n - 128 * g.t0;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.qfree);
      if (nt == 0) break;
      const bool some = __any_sync(kFull, live);
      float m = live ? -INFINITY : 0.0f;
      uint64_t l2 = 0;  // running sum, even and odd columns
      bool started = false;
      for (int32_t t = two ? 0 : wg; t < nt && ok; t += two ? 1 : 2, ++ns) {
        if (!(ok = warp_wait(&sm.sfull[wg], ns & 1u))) break;
        fence_after();
        if (four) {
          const int q = warp & 3;  // this warp's columns: 32 q .. + 31
          const int32_t lim = live ? lim0 - 128 * t - 32 * q : 32;
          uint32_t u[32], w[16];
          tmem_ld32(ts_s + 32 * q, u);
          tmem_wait32(u);
          if (__any_sync(kFull, lim < 32)) keep_columns(u, lim);
          const float top = ceilf(max32(u) * sl2), mn = live && top > m + 8.0f ? top : m;
          const float f = mn == m ? 1.0f : ex2(m - mn);
          if (started && __any_sync(kFull, f != 1.0f)) scale_row(ts_o, f);
          l2 = f2_mul(l2, f2_pack(f, f));
          m = mn;
          l2 = f2_add(l2, weigh_rounded(u, w, sl2, m == -INFINITY ? 0.0f : m));
          uint32_t zero[16] = {};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (c == q) {
              tmem_st16(ts_s + 32 * c, w);
              tmem_st16(ts_s + 32 * c + 16, u);
            } else {
              tmem_st16(ts_s + 32 * c, zero);
              tmem_st16(ts_s + 32 * c + 16, zero);
            }
          }
        } else if (some) {
          const int32_t lim = live ? lim0 - 128 * t : 128;
          if (__any_sync(kFull, lim < 128)) {
            // the item's last tiles: what a row does not see leaves S before the usual code reads it
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              if (__all_sync(kFull, lim >= 32 * c + 32)) continue;
              uint32_t u[32];
              tmem_ld32(ts_s + 32 * c, u);
              tmem_wait32(u);
              keep_columns(u, lim - 32 * c);
              tmem_st16(ts_s + 32 * c, u);
              tmem_st16(ts_s + 32 * c + 16, u + 16);
            }
            tmem_wait_st();
          }
          if (__any_sync(kFull, live && m == -INFINITY)) {  // rows start: their first columns set the reference
            uint32_t u[32];
            tmem_ld32(ts_s, u);
            tmem_wait32(u);
            const float top = ceilf(max32(u) * sl2);
            if (m == -INFINITY) m = top;
          }
          uint64_t sum = 0;
          bool slow = true;
          const bool near = two && !__any_sync(kFull, live && !(fabsf(m) < kFar));
          // P of 32 columns takes the first 16 of their columns of S
          if (near) {
            const uint64_t nm2 = f2_pack(-m, -m);
            // without a branch, and P in registers until the tile's sum is known: a test for every 32 columns made
            // the tile 1560 cycles of 1000, masks where they are needed 1370 (and a masked tile in the loop below took
            // 2800)
            uint32_t u0[32], u1[32], w[64];
            // columns 32 c .. + 31 in u, the next ones on their way to v
            auto chunk = [&](auto which, uint32_t(&u)[32], uint32_t(&v)[32]) {
              constexpr int c = decltype(which)::value;
              if constexpr (c < 3) tmem_ld32(ts_s + 32 * (c + 1), v);
              sum = f2_add(sum, weigh(u, w + 16 * c, sl2x2, nm2));
              if constexpr (c < 3) tmem_wait32(v);
            };
            tmem_ld32(ts_s, u0);
            tmem_wait32(u0);
            chunk(std::integral_constant<int, 0>{}, u0, u1);
            chunk(std::integral_constant<int, 1>{}, u1, u0);
            chunk(std::integral_constant<int, 2>{}, u0, u1);
            chunk(std::integral_constant<int, 3>{}, u1, u0);
            if (__builtin_expect(!__any_sync(kFull, live && !(f2_sum(sum) <= kMost)), 1)) {
#pragma unroll
              for (int c = 0; c < 4; ++c) tmem_st16(ts_s + 32 * c, w + 16 * c);
              slow = false;
            } else {
              sum = 0;
            }
          }
          if (__builtin_expect(slow, 0)) {
            // in a short loop: this code runs seldom with two row tiles, and what is not in the instruction cache
            // costs more than it does
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t u[32], w[16];
              auto load = [&] {
                tmem_ld32(ts_s + 32 * c, u);
                tmem_wait32(u);
              };
              load();
              const float mo = m == -INFINITY ? 0.0f : m;
              uint64_t x = near ? weigh(u, w, sl2x2, f2_pack(-mo, -mo)) : weigh_rounded(u, w, sl2, mo);
              if (__any_sync(kFull, live && !(f2_sum(x) <= kMost))) {
                // the reference moves: outputs in progress, sums and the tile's earlier weights follow
                load();
                const float top = ceilf(max32(u) * sl2), mn = live && top > m ? top : m;
                const float f = mn == m ? 1.0f : ex2(m - mn);
                for (int k = 0; k < c; ++k) {
                  scale_weights(ts_s + 32 * k, f);
                  if (!two) scale_weights(ts_s + 32 * k + 16, f);
                }
                if (started) scale_row(ts_o, f);
                l2 = f2_mul(l2, f2_pack(f, f));
                sum = f2_mul(sum, f2_pack(f, f));
                m = mn;
                x = weigh_rounded(u, w, sl2, m == -INFINITY ? 0.0f : m);
              }
              sum = f2_add(sum, x);
              tmem_st16(ts_s + 32 * c, w);
              if (!two) tmem_st16(ts_s + 32 * c + 16, u);  // what the rounding left of the weights
            }
          }
          l2 = f2_add(l2, sum);
        }
        started = true;
        // rows of V behind the item's last position hold anything: zeros, as 0 times anything is not 0
        const int32_t end = end0 - 128 * t;
        if (end < 128) {
          const int32_t vi = 2 * (base + t) + 1, slot = vi % kRing;
          if (!(ok = warp_wait(&sm.full[slot], (vi / kRing) & 1u))) break;
          if (row >= end) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              *reinterpret_cast<uint4 *>(sm.ring[slot] + (e >> 3) * kBox + row * 128 + (e & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_async();
        }
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.pready[wg]);
      }
      if (!ok) break;
      // ---- the segment's results
      if (four) {
        // a warp's rows go to shared memory, [warp][column][16 rows]; then a thread joins eight columns of a row
        float *ox = reinterpret_cast<float *>(sm.q[0]) + warp * (128 * 16);
        if (started) {
          if (!(ok = warp_wait(&sm.odone[wg], nseg & 1u))) break;
          ++nseg;
          fence_after();
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t u[32];
            tmem_ld32(ts_o + 32 * c, u);
            tmem_wait32(u);
            if (live) {
#pragma unroll
              for (int e = 0; e < 32; ++e) ox[(32 * c + e) * 16 + lane] = __uint_as_float(u[e]);
            }
          }
        }
        if (lane < 16) sm.ml[warp * 16 + lane] = make_float2(m, f2_sum(l2));
        fence_before();
        __syncwarp();
        if (lane == 0) {
          if (started) mbar_arrive(&sm.ofree[wg]);
          mbar_arrive(&sm.qjoin);
        }
        if (!(ok = warp_wait(&sm.qjoin, qjoins & 1u))) break;
        ++qjoins;
        const int32_t jr = tid & 15, col = 8 * (tid >> 4);
        if (jr < g.n * G) {
          float mm = -INFINITY, l = 0.0f, x[8] = {};
#pragma unroll
          for (int w = 0; w < kSoftWarps; ++w) mm = fmaxf(mm, sm.ml[w * 16 + jr].x);
#pragma unroll
          for (int w = 0; w < kSoftWarps; ++w) {
            const float2 y = sm.ml[w * 16 + jr];
            if (y.x == -INFINITY) continue;  // nothing of the row was this warp's
            const float f = y.x == mm ? 1.0f : ex2(y.x - mm);
            l += y.y * f;
            const float *o = reinterpret_cast<const float *>(sm.q[0]) + (w * 128 + col) * 16 + jr;
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] += o[16 * e] * f;
          }
          const int64_t at = (static_cast<int64_t>(g.li) * a.T + g.tok + jr / G) * a.Hq + g.h * G + jr % G;
          if (!in_range(at, outs_of(a), a.status) || !in_range(jr, rows, a.status)) {
          } else if (g.slot < 0) {
            const float inv = 1.0f / l;
            *reinterpret_cast<uint4 *>(a.out + at * 128 + col) =
                make_uint4(bf16x2_rn(x[0] * inv, x[1] * inv), bf16x2_rn(x[2] * inv, x[3] * inv),
                           bf16x2_rn(x[4] * inv, x[5] * inv), bf16x2_rn(x[6] * inv, x[7] * inv));
            if (a.lse && col == 0) a.lse[at] = (mm + log2f(l)) * 0.693147180559945309f;
          } else {
            const int64_t part = static_cast<int64_t>(g.slot) * 32 + (col >> 2);
            p.o[part * rows + jr] = make_float4(x[0], x[1], x[2], x[3]);
            p.o[(part + 1) * rows + jr] = make_float4(x[4], x[5], x[6], x[7]);
            if (col == 0) p.ml[static_cast<int64_t>(g.slot) * rows + jr] = make_float2(mm, l);
          }
        }
        fence_async();  // the next Q is copied where these reads were
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.joined);
        base += nt;
        continue;
      }
      const bool join = !two && nt > 1;
      float l = f2_sum(l2);
      const int64_t at = (static_cast<int64_t>(g.li) * a.T + g.tok + i) * a.Hq + g.h * G + (row - rt * G);
      const int32_t prow = (two && wg ? tpt * G : 0) + row;  // of a partial result
      // where the two rows of this lane's pair go (-1: not a row)
      const int64_t to0 = __shfl_sync(kFull, live ? at : -1, lane & ~1), to1 = __shfl_sync(kFull, live ? at : -1, lane | 1);
      if (started) {
        if (!(ok = warp_wait(&sm.odone[wg], nseg & 1u))) break;
        ++nseg;
        fence_after();
        float *ox = reinterpret_cast<float *>(sm.q[0]);  // [column][row]
        float f0 = 1.0f, f1 = 0.0f;
        if (join && wg == 0) {
          if (!(ok = warp_wait(&sm.ojoin, joins & 1u))) break;
          const float2 x = sm.ml[row];
          const float mm = fmaxf(m, x.x);
          f0 = m == mm ? 1.0f : ex2(m - mm);
          f1 = x.x == mm ? 1.0f : ex2(x.x - mm);
          l = l * f0 + x.y * f1;
          m = mm;
        }
        const float inv = g.slot < 0 ? 1.0f / l : 1.0f;
        f0 *= inv;
        f1 *= inv;
        // loops of a few instructions: this code runs once an item, and fetching it costs as much as what it does (all
        // columns in two bodies of two steps each: a first chunk 203 us of 197)
        if (some) {
          if (join && wg == 1) {
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              uint32_t u[16];
              tmem_ld16(ts_o + 16 * c, u);
              tmem_wait16(u);
#pragma unroll
              for (int e = 0; e < 16; ++e) ox[(16 * c + e) * 128 + row] = __uint_as_float(u[e]);
            }
          } else {
            uint16_t *dst0 = a.out + (to0 * 128 + 8 * (lane & 1)), *dst1 = a.out + (to1 * 128 + 8 * (lane & 1));
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t u[32];
              tmem_ld32(ts_o + 32 * c, u);
              tmem_wait32(u);
              float x[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(u[e]) * f0;
              if (join) {
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] += ox[(32 * c + e) * 128 + row] * f1;
              }
              if (g.slot < 0) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  uint4 y[2];
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const float *z = x + 16 * k + 8 * e;
                    y[e] = make_uint4(bf16x2_rn(z[0], z[1]), bf16x2_rn(z[2], z[3]), bf16x2_rn(z[4], z[5]), bf16x2_rn(z[6], z[7]));
                  }
                  transpose2(y[0], y[1]);  // two lanes write 32 bytes of a row
                  if (to0 >= 0 && in_range(to0, outs_of(a), a.status)) *reinterpret_cast<uint4 *>(dst0 + 32 * c + 16 * k) = y[0];
                  if (to1 >= 0 && in_range(to1, outs_of(a), a.status)) *reinterpret_cast<uint4 *>(dst1 + 32 * c + 16 * k) = y[1];
                }
              } else if (live && in_range(prow, rows, a.status)) {
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  p.o[(static_cast<int64_t>(g.slot) * 32 + 8 * c + e) * rows + prow] =
                      make_float4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
              }
            }
          }
          if (join && wg == 1) sm.ml[row] = make_float2(m, l);
          else if (live && g.slot >= 0 && in_range(prow, rows, a.status)) p.ml[static_cast<int64_t>(g.slot) * rows + prow] = make_float2(m, l);
          else if (live && g.slot < 0 && a.lse && in_range(at, outs_of(a), a.status)) a.lse[at] = (m + log2f(l)) * 0.693147180559945309f;
        }
        fence_before();
        if (join) fence_async();  // the next Q is copied where these reads (and the other's writes) were
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.ofree[wg]);
          if (join && wg == 1) mbar_arrive(&sm.ojoin);
          if (join) mbar_arrive(&sm.joined);
        }
        if (join) ++joins;
      }
      base += nt;
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

// ------------------------------------------------------------------- join --

constexpr int kJoinWarps = 8, kJoinShares = 4;

// Block c kJoinShares + s: a share of the rows of the cut item whose first part is block c's, out of its parts' results.
// (In the attention itself, by the block that ended last, they took 20 us behind the last tile: a first chunk 197 us of 167.)
__global__ void __launch_bounds__(32 * kJoinWarps)
    k_chunk_join(const __grid_constant__ ChunkArgs a, const PlanPtrs p, int32_t grid, int32_t rows) {
  __shared__ int32_t slots[kBlocks], parts_s;
  const int32_t c = blockIdx.x / kJoinShares, share = blockIdx.x % kJoinShares;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.G;
  after_launch_before();
  if (!p.hdr->ok) return;
  const CutItem g = p.item[c];
  if (4 * ((g.n * G + 7) / 8) <= kJoinWarps * share) return;
  if (warp == 0) {
    int32_t parts = 1;
    if (lane == 0) slots[0] = g.slot;
    for (int32_t b0 = c + 1; b0 < grid; b0 += 32) {
      const int32_t b = b0 + lane;
      const int64_t x0 = b < grid ? p.cut[b] : g.end, x1 = b < grid ? p.cut[b + 1] : g.end;
      const bool has = x1 > x0 && x0 < g.end;
      const uint32_t m = __ballot_sync(kFull, has);
      if (has && in_range(parts + __popc(m & ((1u << lane) - 1u)), kBlocks, a.status)) slots[parts + __popc(m & ((1u << lane) - 1u))] = 2 * b;
      parts += __popc(m);
      if (__any_sync(kFull, x0 >= g.end)) break;
    }
    if (lane == 0) parts_s = parts;
  }
  __syncthreads();
  const int32_t parts = parts_s;
  // a warp takes eight rows of 32 channels, a thread eight channels of a row; nk such groups and np parts at a time
  const int32_t nr = g.n * G, all = kJoinWarps * kJoinShares, groups = 4 * ((nr + 7) / 8);
  auto join_parts = [&](auto nk_of, auto np_of) {
    constexpr int nk = decltype(nk_of)::value, np = decltype(np_of)::value;
    for (int32_t k0 = kJoinWarps * share + warp; k0 < groups; k0 += nk * all) {
      float mm[nk], l[nk], x[nk][8];
#pragma unroll
      for (int k = 0; k < nk; ++k) {
        mm[k] = -INFINITY;
        l[k] = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[k][e] = 0.0f;
      }
      auto row_of = [&](int k) { return 8 * ((k0 + k * all) >> 2) + (lane >> 2); };
      auto unit_of = [&](int k) { return 8 * ((k0 + k * all) & 3) + 2 * (lane & 3); };
#pragma unroll 1
      for (int32_t i0 = 0; i0 < parts; i0 += np) {
        float2 y[nk][np];
        float4 u[nk][np], v[nk][np];
#pragma unroll
        for (int i = 0; i < np; ++i) {
          const bool is = i0 + i < parts;
          const int64_t slot = is ? slots[i0 + i] : 0;
#pragma unroll
          for (int k = 0; k < nk; ++k) {
            y[k][i].x = -INFINITY;
            if (!is || row_of(k) >= nr) continue;
            if (!in_range(slot, 2 * grid, a.status) || !in_range(row_of(k), rows, a.status)) continue;
            y[k][i] = __ldcg(p.ml + slot * rows + row_of(k));
            u[k][i] = __ldcg(p.o + (slot * 32 + unit_of(k)) * rows + row_of(k));
            v[k][i] = __ldcg(p.o + (slot * 32 + unit_of(k) + 1) * rows + row_of(k));
          }
        }
#pragma unroll
        for (int k = 0; k < nk; ++k) {
          float mn = mm[k];
#pragma unroll
          for (int i = 0; i < np; ++i) mn = fmaxf(mn, y[k][i].x);
          if (mn == -INFINITY) continue;
          const float f = mm[k] == mn ? 1.0f : ex2(mm[k] - mn);
          mm[k] = mn;
          l[k] *= f;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[k][e] *= f;
#pragma unroll
          for (int i = 0; i < np; ++i) {
            if (y[k][i].x == -INFINITY) continue;  // every tile of that part lies behind the row, or there is none
            const float f1 = y[k][i].x == mn ? 1.0f : ex2(y[k][i].x - mn);
            l[k] += y[k][i].y * f1;
            x[k][0] += u[k][i].x * f1;
            x[k][1] += u[k][i].y * f1;
            x[k][2] += u[k][i].z * f1;
            x[k][3] += u[k][i].w * f1;
            x[k][4] += v[k][i].x * f1;
            x[k][5] += v[k][i].y * f1;
            x[k][6] += v[k][i].z * f1;
            x[k][7] += v[k][i].w * f1;
          }
        }
      }
#pragma unroll
      for (int k = 0; k < nk; ++k) {
        const int32_t jr = row_of(k), unit = unit_of(k);
        if (jr >= nr) continue;
        const float inv = 1.0f / l[k];
        const int64_t at = (static_cast<int64_t>(g.li) * a.T + g.tok + jr / G) * a.Hq + g.h * G + jr % G;
        if (!in_range(at, outs_of(a), a.status)) continue;
        *reinterpret_cast<uint4 *>(a.out + at * 128 + 4 * unit) =
            make_uint4(bf16x2_rn(x[k][0] * inv, x[k][1] * inv), bf16x2_rn(x[k][2] * inv, x[k][3] * inv),
                       bf16x2_rn(x[k][4] * inv, x[k][5] * inv), bf16x2_rn(x[k][6] * inv, x[k][7] * inv));
        if (a.lse && unit == 0) a.lse[at] = (mm[k] + log2f(l[k])) * 0.693147180559945309f;
      }
    }
  };
  // few rows have many parts, many rows mostly two
  if (groups <= all) join_parts(std::integral_constant<int, 1>{}, std::integral_constant<int, 4>{});
  else join_parts(std::integral_constant<int, 2>{}, std::integral_constant<int, 2>{});
}

}  // namespace

size_t chunk_workspace(const ChunkArgs &a) { return chunk_layout(a).bytes; }

cudaError_t launch_chunk(const ChunkArgs &a, void *ws, cudaStream_t s) {
  const ChunkLayout w = chunk_layout(a);
  uint8_t *b = static_cast<uint8_t *>(ws);
  const PlanPtrs p{reinterpret_cast<PlanHeader *>(b), reinterpret_cast<ReqPlan *>(b + w.req),
                   reinterpret_cast<int32_t *>(b + w.pre), reinterpret_cast<int64_t *>(b + w.cut),
                   reinterpret_cast<CutItem *>(b + w.item), reinterpret_cast<float4 *>(b + w.o),
                   reinterpret_cast<float2 *>(b + w.ml)};
  int dev = 0, sms = 0;
  cudaError_t e;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
  const int grid = std::max(1, std::min(sms, kBlocks));
  alignas(64) CUtensorMap qmap, kmap, vmap;
  if ((e = chunk_map(&qmap, a.q, a.Hq, 128, a.n_layers * a.T, a.q_stride, a.G, w.tpt)) != cudaSuccess) return e;
  const int64_t rows = static_cast<int64_t>(a.L) * a.F * a.B, stride = a.Hkv * int64_t{128};
  if ((e = chunk_map(&kmap, a.k, a.Hkv, 128, rows, stride, 1, a.B)) != cudaSuccess) return e;
  if ((e = chunk_map(&vmap, a.v, a.Hkv, 128, rows, stride, 1, a.B)) != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(k_chunk, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmemBytes))) != cudaSuccess)
    return e;
  const int32_t tpq = 16 / a.G;  // tokens whose rows lie four times in a row tile
  alignas(64) CUtensorMap qmap4;
  if ((e = chunk_map(&qmap4, a.q, a.Hq, 128, a.n_layers * a.T, a.q_stride, a.G, std::max(tpq, 1))) != cudaSuccess) return e;
  const int64_t copies = a.k_new ? a.n_layers * ((a.T + kAppendTokens - 1) / kAppendTokens) : 0;
  k_chunk_append<<<static_cast<unsigned>(1 + copies), kAppendThreads, 0, s>>>(a, p, w.tpi, grid);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if ((e = launch_after(k_chunk, dim3(grid), kThreads, kSmemBytes, s, a, p, qmap, kmap, vmap, qmap4, w.tpt, tpq, w.rows)) != cudaSuccess)
    return e;
  return launch_after(k_chunk_join, dim3(kJoinShares * grid), 32 * kJoinWarps, 0, s, a, p, grid, w.rows);
}

}  // namespace dkv
