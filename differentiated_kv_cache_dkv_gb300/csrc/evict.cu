// evict.cu -- eviction of a unit's least attended tokens (dkv_evict).
//
// DiffKV (arXiv 2412.03131) prunes by a threshold on the average attention a
// token has received; a pool that runs out needs a bound on the tokens
// instead.  Of a unit's held tokens those with the K largest weights w(p)
// stay, K the budget: a selection, no sort.
//
//   k_evict_plan   a block per unit: the weights become 32-bit keys in the
//     order of the floats (in shared memory), counting passes of 11 bits
//     find the K-th largest key T and how many equal to it stay; the position
//     of the last of those decides between equals.  Survivors and evicted are
//     counted against headers and slots, pages against the reverse table.
//     Leaves the survivors' counts, the slots that stay and the evicted
//     positions as bits.
//   k_evict_scan   one block: freed pages of the units before each (prefix
//     sum), the first error.  After an error nothing is changed.
//   k_evict_apply  a block for 4096 positions of a unit: prefix counts over the
//     slots that stay give every mover its hole; the moves, a group of lanes
//     each; the cleared slots, the rows of the evicted, the tables, the ring
//     and its tail.
//
// Floor: the significance (4 Hq bytes a position), slots and classes, and the
// moved tokens' bytes.  What bounds it is latency: a unit's passes follow one
// another (weights, counts, slots; then ranks, moves, tables), with 65% (plan)
// and 53% (apply) of the warps' places taken.  Measured, with a copy that puts
// the state back: 8 layers of 16 requests of 2048 to 8192 positions, 8 KV heads,
// half evicted (0.5 GB) 281 us, 26% of 6773 GB/s; 28 layers of 7 requests, 4 KV
// heads, 85% kept (99 MB) 123 to 136 us, 12%; one layer of 4 requests of 512 46
// to 59 us.  Four positions in flight a thread in three blocks a multiprocessor
// (40 registers, 20 bytes spilled): eight in two 294 us, four in four 322 (more
// spilled); 256 threads a block 305 to 342, 1024 327.  Five apply blocks a
// multiprocessor (48 registers, 16 bytes spilled): four 284, six 333 us; 256 or
// 1024 moves listed at a time 291 to 293; a block for 2048 positions 302.
//   Equal weights at the border are settled by one warp that walks the
// positions: one unit of 8192 positions, halved, 67 us with distinct sums, 63
// with equal ones, 97 with three values; of 262 000 positions 790, 1760, 2510.
#include <cuda_runtime.h>

#include <algorithm>

#include "dkv_internal.cuh"

namespace dkv {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBins = 2048;   // of a counting pass
constexpr int kPlanThreads = 512, kScanThreads = 1024, kApplyThreads = 256;
constexpr int kMoves = 512;   // moves a block lists at a time
constexpr int kIds = 1024;    // page ids of a list that a block keeps in shared memory

// Order of the floats as unsigned numbers; 0 is left for "not held" and the
// largest for the protected; a NaN is below every number.
__device__ __forceinline__ uint32_t order_key(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);  // -0 counts as 0
  if (x != x) return 1u;
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// The larger one; NaN where one is NaN.
__device__ __forceinline__ float nan_max(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Sum over the block, to every thread; `sm` holds one int a warp.
__device__ __forceinline__ int32_t block_sum(int32_t x, int32_t *sm) {
  x = __reduce_add_sync(kFull, x);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
  __syncthreads();
  int32_t t = 0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += sm[w];
  return t;
}

// A unit of the tables: its request, head, and where its rows start.
struct Place {
  int32_t r, h;
  int64_t row;  // index of position 0 in [L][R * cap]
};
__device__ __forceinline__ Place place_of(const EvictArgs &a, int32_t u) {
  const uint32_t lr = static_cast<uint32_t>(u) / a.Hkv;
  Place p;
  p.h = static_cast<int32_t>(static_cast<uint32_t>(u) - lr * a.Hkv);
  p.r = static_cast<int32_t>(lr % a.R);
  p.row = static_cast<int64_t>(lr) * a.cap;
  return p;
}

// Positions of all layers and requests.
__device__ __forceinline__ int64_t rows_of(const EvictArgs &a) { return static_cast<int64_t>(a.L) * a.R * a.cap; }

// Words of the slot bitmaps: the high list's, then the low list's.
__device__ __forceinline__ int32_t words_of(int32_t n) { return (n + 31) >> 5; }

__global__ void __launch_bounds__(kPlanThreads, 3) k_evict_plan(const __grid_constant__ EvictArgs a) {
  let_next_launch_start();
  extern __shared__ uint32_t dyn[];
  __shared__ int32_t sm[kPlanThreads / 32];
  __shared__ uint32_t hist[kBins];
  __shared__ int32_t pick_s[3], bad_s;
  const int32_t u = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const Place pl = place_of(a, u);
  const int32_t ctx = __ldg(a.ctx_lens + pl.r), budget = __ldg(a.budgets + pl.r);
  const int4 hd = *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * static_cast<int64_t>(u));
  const int32_t n_hi = hd.x, n_lo = hd.y;
  int32_t err = 0;
  if (ctx < 0 || ctx > a.cap) err = DKV_E_LENS;
  else if (n_hi < 0 || n_lo < 0 || static_cast<int64_t>(n_hi) + n_lo > ctx || hd.z != (n_hi + a.P - 1) / a.P ||
           hd.w != (n_lo + 2 * a.P - 1) / (2 * a.P) || hd.z + hd.w > a.pmax)
    err = DKV_E_INTERNAL;
  if constexpr (kChecked) {  // words of the bitmaps, rows of the unit
    if (!err && !(in_range(words_of(n_hi) + words_of(n_lo), a.cap / 32 + 3, a.status) && in_range(pl.row + ctx, rows_of(a) + 1, a.status)))
      err = DKV_E_INTERNAL;
  }
  if (err || budget < 0 || n_hi + n_lo <= budget) {
    if (tid == 0) a.unit[u] = EvictUnit{-1, -1, 0, err};
    return;
  }
  const int32_t held = n_hi + n_lo, wh = words_of(n_hi), words = wh + words_of(n_lo);
  uint32_t *stay = dyn, *gone = dyn + words, *high = dyn + 2 * (a.cap / 32 + 2);  // high: positions of the high class
  uint32_t *key = a.cap > kEvictKeys ? a.keys + static_cast<int64_t>(u) * a.cap : high + (a.cap / 32 + 1);
  for (int32_t i = tid; i < 2 * words; i += kPlanThreads) dyn[i] = 0;
  if (tid == 0) bad_s = 0;
  for (int i = tid; i < kBins; i += kPlanThreads) hist[i] = 0;
  // pages and their reverse entries: a thread's first one on its way through all that follows
  const int32_t pages = hd.z + hd.w;
  auto page_of = [&](int32_t j) { return a.fwd[static_cast<int64_t>(u) * a.pmax + j]; };
  const int32_t id0 = tid < pages ? page_of(tid) : -1;
  const bool in0 = id0 >= 0 && id0 < a.F;
  const int32_t ru0 = in0 ? a.rev_unit[id0] : -1, ri0 = in0 ? a.rev_idx[id0] : -1;
  __syncthreads();

  // keys, the first counting pass, and what the classes say is held
  int32_t hi = 0, lo = 0, safe = 0;
  const uint8_t *cls = a.classes + pl.row * a.Hkv + pl.h;
  const int32_t G = a.G;
  const bool quad = (G & 3) == 0 && (a.Hq & 3) == 0;  // then a token's scores are whole 16-byte words
  const float *sig = a.sig_sum + pl.row * a.Hq + pl.h * G;
  const int32_t *cnt = a.sig_cnt ? a.sig_cnt + static_cast<int64_t>(pl.r) * a.cap : nullptr;
  constexpr int kEach = 4;  // positions a thread has in flight; the scores of positions without a token are read too
  for (int32_t p0 = tid; p0 - tid < ctx; p0 += kEach * kPlanThreads) {
    int32_t c[kEach];
    float w[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int32_t p = min(p0 + e * kPlanThreads, ctx - 1);
      c[e] = cls[static_cast<int64_t>(p) * a.Hkv];
      const float *x = sig + static_cast<int64_t>(p) * a.Hq;
      // a token's scores one after the other: they share sectors, which stay in the first-level cache
      if (quad) {
        float4 y = __ldg(reinterpret_cast<const float4 *>(x));
        w[e] = nan_max(nan_max(y.x, y.y), nan_max(y.z, y.w));
        for (int g = 4; g < G; g += 4) {
          y = __ldg(reinterpret_cast<const float4 *>(x + g));
          w[e] = nan_max(w[e], nan_max(nan_max(y.x, y.y), nan_max(y.z, y.w)));
        }
      } else {
        w[e] = __ldg(x);
#pragma unroll 4
        for (int g = 1; g < G; ++g) w[e] = nan_max(w[e], __ldg(x + g));
      }
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int32_t p = p0 + e * kPlanThreads;
      const uint32_t m = __ballot_sync(kFull, c[e] == DKV_CLASS_K8V4);  // of the positions behind the last nothing is read
      if (p >= ctx) continue;
      if (lane == 0) high[p >> 5] = m;
      uint32_t k = 0;
      if (c[e]) {
        const bool s = p < a.sinks || p >= static_cast<int64_t>(ctx) - a.window;
        if (c[e] > DKV_CLASS_K8V4) bad_s = 1;
        hi += c[e] == DKV_CLASS_K8V4;
        lo += c[e] == DKV_CLASS_K4V2;
        safe += s;
        if (cnt) w[e] = __fdiv_rn(w[e], static_cast<float>(__ldg(cnt + p)));
        k = s ? 0xffffffffu : order_key(w[e]);
        atomicAdd(hist + (k >> 21), 1u);
      }
      key[p] = k;
    }
  }
  // the first slots are on their way while the threshold is found
  const int32_t *slots = a.slot_of + pl.row * a.Hkv + pl.h;
  int32_t slot[kEach];
#pragma unroll
  for (int e = 0; e < kEach; ++e) slot[e] = slots[static_cast<int64_t>(min(tid + e * kPlanThreads, ctx - 1)) * a.Hkv];
  hi = block_sum(hi, sm);
  lo = block_sum(lo, sm);
  safe = block_sum(safe, sm);
  if (hi != n_hi || lo != n_lo || bad_s) err = DKV_E_INTERNAL;
  const int32_t K = max(budget, safe);
  if (err || K >= held) {  // block-wide alike
    if (tid == 0) a.unit[u] = EvictUnit{-1, -1, 0, err};
    return;
  }

  // T: the K-th largest key; `left`: how many of the keys equal to it (as far as it is known) stay
  uint32_t T = 0xffffffffu, known = 0xffffffffu;
  int32_t left = 0, ties = 0;
  __syncthreads();
  if (K > 0) {
    T = known = 0;
    left = K;
    ties = left + 1;
    for (int shift = 21; ties > left && known != 0xffffffffu; shift -= shift > 11 ? 11 : shift) {
      const uint32_t digit = known ? (shift ? 0x7ffu : 0x3ffu) : 0x7ffu;
      if (known) {
        for (int i = tid; i < kBins; i += kPlanThreads) hist[i] = 0;
        __syncthreads();
        for (int32_t p = tid; p < ctx; p += kPlanThreads) {
          const uint32_t k = key[p];
          if (k && (k & known) == T) atomicAdd(hist + (k >> shift & digit), 1u);
        }
        __syncthreads();
      }
      // thread i: bins from 2047 - 4 i down
      int32_t n[kBins / kPlanThreads], sum = 0;
#pragma unroll
      for (int j = 0; j < kBins / kPlanThreads; ++j) sum += n[j] = static_cast<int32_t>(hist[kBins - 1 - (kBins / kPlanThreads) * tid - j]);
      int32_t above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t x = __shfl_up_sync(kFull, above, o);
        if (lane >= o) above += x;
      }
      if (lane == 31) sm[tid >> 5] = above;
      __syncthreads();
      above -= sum;
      for (int w = 0; w < (tid >> 5); ++w) above += sm[w];
      if (above < left && above + sum >= left) {
        int j = 0;
        while (above + n[j] < left) above += n[j++];
        pick_s[0] = kBins - 1 - (kBins / kPlanThreads) * tid - j;
        pick_s[1] = left - above;
        pick_s[2] = n[j];
      }
      __syncthreads();
      T |= static_cast<uint32_t>(pick_s[0]) << shift;
      left = pick_s[1];
      ties = pick_s[2];
      known |= digit << shift;
      __syncthreads();
    }
  }
  // of more equals than may stay the lowest positions do: up to the left-th
  if (ties > left) {
    if (tid < 32) {
      int32_t seen = 0, cut = -1;
      for (int32_t p = lane; p - lane < ctx; p += 32) {
        uint32_t m = __ballot_sync(kFull, p < ctx && key[p] && (key[p] & known) == T);
        if (seen + __popc(m) >= left) {
          while (seen + 1 < left) {
            m &= m - 1u;
            ++seen;
          }
          cut = p - lane + __ffs(m) - 1;
          break;
        }
        seen += __popc(m);
      }
      if (lane == 0) pick_s[0] = cut;
    }
    __syncthreads();
  } else {
    if (tid == 0) pick_s[0] = left > 0 ? ctx : -1;
    __syncthreads();
  }
  const int32_t cut = pick_s[0];

  // survivors and evicted, by slot and by position
  uint32_t *gone_pos = a.gone + static_cast<int64_t>(u) * ((a.cap + 31) / 32);
  bool bad = false;
  for (int32_t p0 = tid; p0 - tid < ctx; p0 += kEach * kPlanThreads) {
    if (p0 != tid) {
#pragma unroll
      for (int e = 0; e < kEach; ++e) slot[e] = slots[static_cast<int64_t>(min(p0 + e * kPlanThreads, ctx - 1)) * a.Hkv];
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int32_t p = p0 + e * kPlanThreads, s = slot[e];
      bool out = false;
      const uint32_t k = p < ctx ? key[p] : 0;
      if (k) {
        const bool hi_cls = high[p >> 5] >> (p & 31) & 1u;
        out = !((k & known) > T || ((k & known) == T && p <= cut));
        if (s < 0 || s >= (hi_cls ? n_hi : n_lo)) {
          bad = true;
        } else {
          const uint32_t bit = 1u << (s & 31);
          bad |= (atomicOr((out ? gone : stay) + (hi_cls ? 0 : wh) + (s >> 5), bit) & bit) != 0;
        }
      }
      const uint32_t m = __ballot_sync(kFull, out);
      if (lane == 0 && p < ctx) gone_pos[p >> 5] = m;
    }
  }
  if (bad) bad_s = 1;
  __syncthreads();
  int32_t all = 0, kh = 0, kl = 0;
  for (int32_t i = tid; i < words; i += kPlanThreads) {
    all += __popc(stay[i] | gone[i]);
    if (i < wh) kh += __popc(stay[i]);
    else kl += __popc(stay[i]);
  }
  all = block_sum(all, sm);
  kh = block_sum(kh, sm);
  kl = block_sum(kl, sm);
  bool wrong = all != held || (tid < pages && (ru0 != a.unit_base + u || ri0 != tid || !in0));
  for (int32_t j = tid + kPlanThreads; j < pages; j += kPlanThreads) {
    const int32_t id = page_of(j);
    if (id < 0 || id >= a.F || a.rev_unit[id] != a.unit_base + u || a.rev_idx[id] != j) wrong = true;
  }
  uint32_t *stay_out = a.stay + static_cast<int64_t>(u) * (a.cap / 32 + 2);
  for (int32_t i = tid; i < words; i += kPlanThreads) stay_out[i] = stay[i];
  if (wrong) bad_s = 1;
  __syncthreads();
  if (tid == 0) {
    const int32_t freed = hd.z + hd.w - (kh + a.P - 1) / a.P - (kl + 2 * a.P - 1) / (2 * a.P);
    a.unit[u] = bad_s ? EvictUnit{-1, -1, 0, DKV_E_INTERNAL} : EvictUnit{kh, kl, freed, 0};
  }
}

__global__ void __launch_bounds__(kScanThreads) k_evict_scan(const __grid_constant__ EvictArgs a) {
  __shared__ int64_t wsum[kScanThreads / 32];
  __shared__ unsigned long long err_s;
  let_next_launch_start();
  after_launch_before();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t per = (a.U + kScanThreads - 1) / kScanThreads, u0 = tid * per, u1 = min(a.U, u0 + per);
  if (tid == 0) err_s = ~0ull;
  __syncthreads();
  int64_t sum = 0;
  unsigned long long e = ~0ull;
  for (int64_t u = u0; u < u1; ++u) {
    const int4 x = *reinterpret_cast<const int4 *>(a.unit + u);
    sum += x.z;
    if (x.w && e == ~0ull) e = static_cast<unsigned long long>(u) << 8 | static_cast<unsigned>(-x.w);
  }
  if (e != ~0ull) atomicMin(&err_s, e);
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int64_t before = incl - sum, total = 0;
  for (int w = 0; w < kScanThreads / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  for (int64_t u = u0; u < u1; ++u) {
    a.off[u] = before;
    before += a.unit[u].freed;
  }
  if (tid == 0) {
    const uint64_t head = a.cursors[0], tail = a.cursors[1];
    int32_t err = err_s == ~0ull ? 0 : -static_cast<int32_t>(err_s & 0xffu);
    if (!err && (tail < head || tail - head + static_cast<uint64_t>(total) > static_cast<uint64_t>(a.F)))
      err = DKV_E_INTERNAL;
    a.ws->err = err;
    a.ws->tail = tail;
    a.ws->freed = total;
    if (err) set_error(a.status, err);
  }
}

// One list of a unit, as a block sees it: its pages' ids, slots a page.
struct List {
  const int32_t *ids;
  int32_t pages, per, ku, vu;  // pages; slots a page; 16-byte units of K and of V a slot
  float inv;
};
// Where a slot lies: page id and slot of the page.
__device__ __forceinline__ int2 slot_at(const EvictArgs &a, const List &l, int32_t s) {
  // s below 2^18: the quotient is exact, the product's error is below half of 1 / per
  const int32_t j = static_cast<int32_t>((static_cast<float>(s) + 0.5f) * l.inv);
  if (!in_range(j, l.pages, a.status)) return make_int2(-1, 0);
  return make_int2(l.ids[j], s - j * l.per);
}
// (checked build) a place that slot_at gave lies in the pool
__device__ __forceinline__ bool in_pool(const EvictArgs &a, const List &l, int2 s) {
  return in_range(s.x, a.F, a.status) && in_range(s.y, l.per, a.status);
}

// What lane j of a slot's lanes carries: a 16-byte unit of K or V, the
// metadata (8 bytes), the position (4) or nothing, `off` bytes into the page
// plus `step` a slot.
struct LanePart {
  int32_t bytes, off, step;
};
__device__ __forceinline__ LanePart lane_part(const EvictArgs &a, const List &l, int32_t j) {
  if (j < l.ku) return {16, 16 * j, 16 * l.ku};
  j -= l.ku;
  if (j < l.vu) return {16, static_cast<int32_t>(a.pg.vbase) + 16 * j, 16 * l.vu};
  j -= l.vu;
  if (j == 0) return {8, static_cast<int32_t>(a.pg.meta), 8};
  return {j == 1 ? 4 : 0, static_cast<int32_t>(a.pg.pos), 4};
}

// Slots src[0 .. n) of a list to dst[0 .. n), kLanes lanes a move, and the
// index entries (to_slot) that go with the positions.
template <int kLanes>
__device__ __forceinline__ void move_slots(const EvictArgs &a, const List &l, const int2 *src, const int2 *dst,
                                           const int32_t *to_slot, int32_t n, int32_t *slots, int32_t ctx) {
  const LanePart part = lane_part(a, l, threadIdx.x % kLanes);
  if (part.bytes == 0) return;
  constexpr int kGroups = kApplyThreads / kLanes, kEach = 4;
  uint8_t *base = a.pages + part.off;
  auto at = [&](int2 s) { return base + (s.x * a.pg.bytes + s.y * part.step); };
  for (int32_t m0 = threadIdx.x / kLanes; m0 < n; m0 += kGroups * kEach) {
    uint4 x[kEach];
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int2 from = src[min(m0 + e * kGroups, n - 1)];
      if (!in_pool(a, l, from)) continue;
      const uint8_t *f = at(from);
      if (part.bytes == 16) x[e] = __ldcs(reinterpret_cast<const uint4 *>(f));
      else if (part.bytes == 8) *reinterpret_cast<uint2 *>(&x[e]) = *reinterpret_cast<const uint2 *>(f);
      else x[e].x = *reinterpret_cast<const uint32_t *>(f);
    }
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
      const int32_t m = m0 + e * kGroups;
      if (m >= n) break;
      if (!in_pool(a, l, dst[m])) continue;
      uint8_t *t = at(dst[m]);
      if (part.bytes == 16) {
        *reinterpret_cast<uint4 *>(t) = x[e];
      } else if (part.bytes == 8) {
        *reinterpret_cast<uint2 *>(t) = make_uint2(x[e].x, x[e].y);
      } else {
        *reinterpret_cast<uint32_t *>(t) = x[e].x;
        if (x[e].x < static_cast<uint32_t>(ctx)) slots[static_cast<int64_t>(x[e].x) * a.Hkv] = to_slot[m];
        else set_error(a.status, DKV_E_INTERNAL);
      }
    }
  }
}

// `slices` blocks a unit: each a share of the evicted positions and of the
// moves; the last one to end, which finds all moves done, clears the vacated
// slots and writes the tables.
__global__ void __launch_bounds__(kApplyThreads, 5) k_evict_apply(const __grid_constant__ EvictArgs a, int32_t slices) {
  after_launch_before();
  extern __shared__ uint32_t dyn[];
  __shared__ int2 src[kMoves], dst[kMoves];
  __shared__ int32_t to_slot[kMoves], ids[kIds];
  __shared__ int32_t wsum[kApplyThreads / 32];
  __shared__ int32_t last_s;
  if (a.ws->err) return;
  // every block starts from the workspace's tail; the ring's own moves in the launch that fills it
  if (blockIdx.x == 0 && threadIdx.x == 0) a.cursors[1] = a.ws->tail + static_cast<uint64_t>(a.ws->freed);
  const int32_t u = blockIdx.x / slices, slice = blockIdx.x - u * slices, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const EvictUnit un = a.unit[u];
  if (un.keep_hi < 0) return;
  const Place pl = place_of(a, u);
  const int32_t ctx = __ldg(a.ctx_lens + pl.r);
  const int4 hd = *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * static_cast<int64_t>(u));
  const int32_t wh = words_of(hd.x), words = wh + words_of(hd.y);
  if (!in_range(words, a.cap / 32 + 3, a.status)) return;
  uint32_t *stay = dyn, *rank = dyn + words;  // slots that stay, and how many of them before a word
  const uint32_t *stay_in = a.stay + static_cast<int64_t>(u) * (a.cap / 32 + 2);
  for (int32_t i = tid; i < words; i += kApplyThreads) stay[i] = __ldg(stay_in + i);
  // the evicted leave the rows
  uint8_t *cls = a.classes + pl.row * a.Hkv + pl.h;
  int32_t *slots = a.slot_of + pl.row * a.Hkv + pl.h;
  const uint32_t *gone_pos = a.gone + static_cast<int64_t>(u) * ((a.cap + 31) / 32);
  for (int32_t p = slice * kApplyThreads + tid; p < ctx; p += slices * kApplyThreads)
    if (__ldg(gone_pos + (p >> 5)) >> (p & 31) & 1u && in_range(pl.row + p, rows_of(a), a.status)) {
      cls[static_cast<int64_t>(p) * a.Hkv] = DKV_CLASS_PRUNE;
      slots[static_cast<int64_t>(p) * a.Hkv] = -1;
    }
  __syncthreads();
  {
    const int32_t per = (words + kApplyThreads - 1) / kApplyThreads, i0 = min(words, tid * per), i1 = min(words, i0 + per);
    int32_t sum = 0;
    for (int32_t i = i0; i < i1; ++i) sum += __popc(stay[i]);
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t x = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) wsum[warp] = incl;
    __syncthreads();
    int32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    for (int32_t i = i0; i < i1; ++i) {
      rank[i] = before;
      before += __popc(stay[i]);
    }
    __syncthreads();
  }
  int32_t *row = a.fwd + static_cast<int64_t>(u) * a.pmax;
  auto list_of = [&](bool high) {
    const int32_t per = high ? a.P : 2 * a.P;
    return List{row + (high ? 0 : hd.z), high ? hd.z : hd.w, per, high ? a.pg.kh : a.pg.kh >> 1, high ? a.pg.vh : a.pg.vh >> 1,
                1.0f / static_cast<float>(per)};
  };
  for (int i = 0; i < 2; ++i) {
    const bool high = i == 0;
    const int32_t n = high ? hd.x : hd.y, keep = high ? un.keep_hi : un.keep_lo, w0 = high ? 0 : wh;
    if (keep == n) continue;
    const int32_t base = high ? 0 : un.keep_hi;  // survivors of the lists before
    const uint32_t *st = stay + w0, *rk = rank + w0;
    // survivors in slots below keep; as many movers as holes
    const int32_t b_keep = static_cast<int32_t>(rk[keep >> 5]) - base + __popc(st[keep >> 5] & ((1u << (keep & 31)) - 1u));
    const int32_t moves = keep - b_keep;
    if (slice * kMoves >= moves) continue;
    List l = list_of(high);
    const int32_t pages = high ? hd.z : hd.w;
    if (pages <= kIds) {
      for (int32_t j = tid; j < pages; j += kApplyThreads) ids[j] = l.ids[j];
      l.ids = ids;
      __syncthreads();
    }
    for (int32_t m0 = slice * kMoves; m0 < moves; m0 += slices * kMoves) {
      const int32_t nm = min(kMoves, moves - m0);
      for (int32_t w = tid; w < words_of(n); w += kApplyThreads) {
        const int32_t s0 = 32 * w, before = static_cast<int32_t>(rk[w]) - base;
        const uint32_t low = keep >= s0 + 32 ? ~0u : (keep <= s0 ? 0u : (1u << (keep - s0)) - 1u);  // slots below keep
        uint32_t hole = ~st[w] & low, mover = st[w] & ~low;
        int32_t m = s0 - before - m0;
        if (m < nm && m + 32 > 0)
          for (; hole; hole &= hole - 1u, ++m)
            if (m >= 0 && m < nm) {
              to_slot[m] = s0 + __ffs(hole) - 1;
              dst[m] = slot_at(a, l, to_slot[m]);
            }
        m = before + __popc(st[w] & low) - b_keep - m0;
        if (m < nm && m + 32 > 0)
          for (; mover; mover &= mover - 1u, ++m)
            if (m >= 0 && m < nm) src[m] = slot_at(a, l, s0 + __ffs(mover) - 1);
      }
      __syncthreads();
      if (high) move_slots<16>(a, l, src, dst, to_slot, nm, slots, ctx);
      else move_slots<8>(a, l, src, dst, to_slot, nm, slots, ctx);
      __syncthreads();
    }
    __syncthreads();
  }
  // the last block of the unit goes on
  if (slices > 1) {
    __threadfence();
    __syncthreads();
    if (tid == 0) last_s = atomicAdd(&a.unit[u].pad, 1) == slices - 1;
    __syncthreads();
    if (!last_s) return;
    __threadfence();
  }
  // vacated slots of the last kept page of each list
  for (int i = 0; i < 2; ++i) {
    const bool high = i == 0;
    const int32_t n = high ? hd.x : hd.y, keep = high ? un.keep_hi : un.keep_lo;
    const List l = list_of(high);
    const int32_t end = min(n, (keep + l.per - 1) / l.per * l.per), lanes = high ? 16 : 8;
    for (int32_t k = tid; k < (end - keep) * lanes; k += kApplyThreads) {
      const LanePart part = lane_part(a, l, k % lanes);
      const int2 at = slot_at(a, l, keep + k / lanes);
      if (!in_pool(a, l, at)) continue;
      uint8_t *t = a.pages + part.off + (at.x * a.pg.bytes + at.y * part.step);
      if (part.bytes == 16) *reinterpret_cast<uint4 *>(t) = make_uint4(0, 0, 0, 0);
      else if (part.bytes == 8) *reinterpret_cast<uint2 *>(t) = make_uint2(0, 0);
      else if (part.bytes == 4) *reinterpret_cast<int32_t *>(t) = -1;
    }
  }
  __syncthreads();

  // surplus pages to the ring, in the order of the row
  const int32_t need_hi = (un.keep_hi + a.P - 1) / a.P, need_lo = (un.keep_lo + 2 * a.P - 1) / (2 * a.P);
  const uint64_t F = static_cast<uint64_t>(a.F), at0 = (a.ws->tail + static_cast<uint64_t>(a.off[u])) % F;
  const int32_t fh = hd.z - need_hi;
  for (int32_t i = tid; i < un.freed; i += kApplyThreads) {
    const int32_t id = i < fh ? row[need_hi + i] : row[hd.z + need_lo + i - fh];
    uint64_t at = at0 + i;
    if (at >= F) at -= F;
    if (!in_range(static_cast<int64_t>(at), a.F, a.status) || !in_range(id, a.F, a.status)) continue;
    a.free_list[at] = id;
    a.rev_unit[id] = -1;
    a.rev_idx[id] = -1;
    a.page_cls[id] = 0;
  }
  __syncthreads();
  // the kept low pages follow the kept high ones
  if (fh > 0) {
    for (int32_t i0 = 0; i0 < need_lo; i0 += kApplyThreads) {
      const int32_t i = i0 + tid, id = i < need_lo ? row[hd.z + i] : 0;
      __syncthreads();
      if (i < need_lo && in_range(id, a.F, a.status) && in_range(need_hi + i, a.pmax, a.status)) {
        row[need_hi + i] = id;
        a.rev_idx[id] = need_hi + i;
      }
      __syncthreads();
    }
  }
  for (int32_t i = need_hi + need_lo + tid; i < hd.z + hd.w; i += kApplyThreads)
    if (in_range(i, a.pmax, a.status)) row[i] = -1;
  if (tid == 0)
    *reinterpret_cast<int4 *>(a.unit_hdr + 4 * static_cast<int64_t>(u)) = make_int4(un.keep_hi, un.keep_lo, need_hi, need_lo);
}

}  // namespace

// Dynamic shared memory of the apply and of the plan kernel.
static constexpr size_t apply_bytes(int32_t cap) { return 8 * static_cast<size_t>(cap / 32 + 2); }
static constexpr size_t plan_bytes(int32_t cap) {
  return apply_bytes(cap) + 4 * static_cast<size_t>(cap / 32 + 1) + (cap > kEvictKeys ? 0 : 4 * static_cast<size_t>(cap));
}

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  const size_t maps = apply_bytes(a.cap), plan = plan_bytes(a.cap);
  // blocks a unit: one for 4096 positions
  const int32_t slices = static_cast<int32_t>(std::min<int64_t>((a.cap + 4095) / 4096, std::max<int64_t>(1, INT32_MAX / a.U)));
  // the limits are the kernels', not the call's: always what any cap needs, as another thread's call may come between
  constexpr int most_plan = static_cast<int>(std::max(plan_bytes(kEvictKeys), plan_bytes(kEvictCap)));
  constexpr int most_apply = static_cast<int>(apply_bytes(kEvictCap));
  if (cudaError_t e = cudaFuncSetAttribute(k_evict_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, most_plan)) return e;
  if (cudaError_t e = cudaFuncSetAttribute(k_evict_apply, cudaFuncAttributeMaxDynamicSharedMemorySize, most_apply)) return e;
  k_evict_plan<<<static_cast<unsigned>(a.U), kPlanThreads, plan, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (cudaError_t e = launch_after(k_evict_scan, 1, kScanThreads, 0, s, a)) return e;
  return launch_after(k_evict_apply, static_cast<unsigned>(a.U * slices), kApplyThreads, maps, s, a, slices);
}

}  // namespace dkv
