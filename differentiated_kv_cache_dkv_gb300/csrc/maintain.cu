// maintain.cu -- page operations of a pool that serves many requests:
// dkv_fork (copy requests), dkv_release (free requests), dkv_defrag (move the
// live pages to the lowest ids).
//
// DiffKV (arXiv 2412.03131), "What carries the argument" and abstract: the
// on-GPU memory manager allocates and recycles pages through a circular free
// list in one coordinated step.  The pages describe the allocation; these are
// the other steps of a pool's life, with the same prefix-sum placement.
//
// An operation is two or three launches in stream order: a plan kernel
// checks everything and leaves one partial sum per block, the next kernel
// adds up the partial sums itself (each block reads all of them: at most a
// few thousand 16-byte entries from L2, less than a look-back's waits or a
// launch would take), stops if any check failed or the pages do not suffice,
// and places its block's share.  Nothing is written to the pool before every
// check of the call has passed, which makes the calls all-or-nothing.
//   fork     k_list_plan, k_list_place (tables, copy list), k_fork_copy
//   release  k_list_plan, k_list_place
//   defrag   k_defrag_plan, k_defrag_list, k_defrag_move
// Small calls run their steps in one launch (k_small).
//
// Measured: 8 prompts of 2048 .. 6144 tokens in 32 layers forked 521 us for
// 2.88 GB, 5.5 TB/s, 82% of the measured copy rate (the copies alone 87%); a
// 28-layer pool of 0.83 GB moved 157 us, 5.3 TB/s, 79%; 8 requests of 32 layers
// released 27 us, for 400,000 pages whose entries lie scattered: the latency of
// two kernels' dependent loads and 1.2 million 32-byte sectors; the calls on
// one small request 10 to 14 us of dependent loads.  (The calls alone: a timing
// that puts the tables back before every pass adds 5 to 12 us.)
#include <cuda_runtime.h>

#include <algorithm>

#include "dkv_internal.cuh"

namespace dkv {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr unsigned kFull = 0xffffffffu;

// Sum of x over the block (all threads get it).  `sm` holds kWarps values.
__device__ __forceinline__ int64_t block_sum(int64_t x, int64_t *sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = x;
  __syncthreads();
  int64_t t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += sm[w];
  return t;
}

// A list unit (l, k, h) of request list q: its index in the tables.
__device__ __forceinline__ int64_t list_unit(const PageOpArgs &a, int64_t v, const int32_t *q, int32_t &k) {
  // v < 2^31: 32-bit divisions
  const uint32_t lk = static_cast<uint32_t>(v) / a.Hkv, l = lk / a.n;
  k = static_cast<int32_t>(lk - l * a.n);
  const int32_t r = __ldg(q + k);
  if (r < 0 || r >= a.R) return -1;
  return (static_cast<int64_t>(l) * a.R + r) * a.Hkv + static_cast<int32_t>(static_cast<uint32_t>(v) - lk * a.Hkv);
}

// Pages of a unit from its header; -1 when the header contradicts itself.
__device__ __forceinline__ int32_t unit_pages(const PageOpArgs &a, const int4 &h) {
  if (h.x < 0 || h.y < 0 || h.z != (static_cast<int64_t>(h.x) + a.P - 1) / a.P ||
      h.w != (static_cast<int64_t>(h.y) + 2 * a.P - 1) / (2 * a.P) || h.z + h.w > a.pmax)
    return -1;
  return h.z + h.w;
}

// The request lists themselves (one block): no request may be named twice as
// a destination (fork) or at all (release), nor be both source and
// destination.  `bits` has room for R bits twice.
__device__ int32_t check_lists(const PageOpArgs &a, uint32_t *bits) {
  const int32_t words = (a.R + 31) / 32;
  for (int32_t i = threadIdx.x; i < 2 * words; i += kThreads) bits[i] = 0;
  __syncthreads();
  int32_t bad = 0;
  const int32_t *once = a.dst ? a.dst : a.src;
  for (int32_t k = threadIdx.x; k < a.n; k += kThreads) {
    const int32_t r = __ldg(once + k);
    if (r < 0 || r >= a.R) bad = 1;
    else if (atomicOr(bits + (r >> 5), 1u << (r & 31)) >> (r & 31) & 1u) bad = 1;
  }
  __syncthreads();
  if (a.dst) {
    for (int32_t k = threadIdx.x; k < a.n; k += kThreads) {
      const int32_t r = __ldg(a.src + k);
      if (r < 0 || r >= a.R || (bits[r >> 5] >> (r & 31) & 1u)) bad = 1;
      // the context whose rows are copied must lie in the request's rows
      else if (a.ctx_lens && (__ldg(a.ctx_lens + r) < 0 || __ldg(a.ctx_lens + r) > a.cap)) bad |= 2;
    }
  }
  bad = __syncthreads_or(bad & 1) ? 1 : (__syncthreads_or(bad & 2) ? 2 : 0);
  return bad == 1 ? DKV_E_INTERNAL : (bad == 2 ? DKV_E_LENS : 0);
}

// ---------------------------------------------------------- fork, release --

// One warp per list unit, a.upb units a block: header, page ids and reverse
// entries agree, destinations (for a fork) are empty; part[block] = {pages of
// the block's units, error}.  The loads of a unit depend on each other (request,
// header, ids, reverse entries), so a warp takes one unit where the blocks
// allow it, and 128 pages of it at a time.
template <bool kFork>
__device__ __forceinline__ void list_plan(const PageOpArgs &a) {
  extern __shared__ uint32_t bits[];
  __shared__ int64_t sm[kWarps];
  __shared__ int32_t err_s;
  if (threadIdx.x == 0) err_s = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t sum = 0;
  int32_t err = 0;
  for (int i = warp; i < a.upb; i += kWarps) {
    const int64_t v = static_cast<int64_t>(blockIdx.x) * a.upb + i;
    if (v >= a.V) break;
    int32_t k, d = 0;
    const int64_t u = list_unit(a, v, a.src, k);
    if (u >= 0) {
      d = unit_pages(a, *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * u));
      if (d < 0) err = DKV_E_INTERNAL;
      for (int32_t j0 = lane; j0 < d; j0 += 128) {
        int32_t id[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t j = j0 + 32 * e;
          id[e] = j < d ? a.fwd[u * a.pmax + j] : 0;
          if (id[e] < 0 || id[e] >= a.F) {
            err = DKV_E_INTERNAL;
            id[e] = 0;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t j = j0 + 32 * e;
          if (!in_range(id[e], a.F, a.status)) continue;
          const bool same = a.rev_unit[id[e]] == a.unit_base + u && a.rev_idx[id[e]] == j;
          if (j < d && !same) err = DKV_E_INTERNAL;
        }
      }
    } else {
      err = DKV_E_INTERNAL;
    }
    if (kFork) {
      const int64_t w = list_unit(a, v, a.dst, k);
      if (w < 0) {
        err = DKV_E_INTERNAL;
      } else {
        const int4 h = *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * w);
        if (h.x | h.y | h.z | h.w) err = DKV_E_INTERNAL;
      }
    }
    if (lane == 0) sum += max(d, 0);
  }
  if (blockIdx.x == gridDim.x - 1) {  // in a small call a block without units
    const int32_t e = check_lists(a, bits);
    if (e) err = e;
    if (threadIdx.x == 0) {  // the cursors before the call: the next kernel moves them
      a.ws->head = a.cursors[0];
      a.ws->tail = a.cursors[1];
    }
  }
  if (err) atomicCAS(&err_s, 0, err);
  sum = block_sum(sum, sm);
  if (threadIdx.x == 0) a.part[blockIdx.x] = make_longlong2(sum, err_s);
}

// A place of the ring: x < 2 F.
__device__ __forceinline__ int64_t ring(int64_t x, int64_t F) { return x < F ? x : x - F; }

// Sum of the plan's partial sums before this block and of all, and the first
// error in block order.  Every thread of the block calls it.
__device__ __forceinline__ int32_t plan_totals(const longlong2 *part, int32_t nparts, int64_t *sm, int64_t &before,
                                               int64_t &total) {
  int64_t b = 0, t = 0, e = INT64_MAX;
  if (nparts <= 32) {  // every warp for itself
    const int32_t i = threadIdx.x & 31;
    if (i < nparts) {
      const longlong2 p = part[i];
      t = p.x;
      if (i < static_cast<int32_t>(blockIdx.x)) b = p.x;
      if (p.y) e = (static_cast<int64_t>(i) << 8) - p.y;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b += __shfl_xor_sync(kFull, b, o);
      t += __shfl_xor_sync(kFull, t, o);
      e = min(e, __shfl_xor_sync(kFull, e, o));
    }
    before = b;
    total = t;
    return e == INT64_MAX ? 0 : -static_cast<int32_t>(e & 0xff);
  }
  for (int32_t i = threadIdx.x; i < nparts; i += kThreads) {
    const longlong2 p = part[i];
    t += p.x;
    if (i < static_cast<int32_t>(blockIdx.x)) b += p.x;
    if (p.y && e == INT64_MAX) e = (static_cast<int64_t>(i) << 8) - p.y;  // -p.y is 1 .. 7
  }
  before = block_sum(b, sm);
  total = block_sum(t, sm);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) e = min(e, __shfl_xor_sync(kFull, e, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = e;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) e = min(e, sm[w]);
  return e == INT64_MAX ? 0 : -static_cast<int32_t>(e & 0xff);
}

// Same blocks as the plan: places the block's units after the sum of the
// blocks before.  Fork: new page ids into the destination's tables, (old,
// new) into the copy list.  Release: ids into the ring, tables cleared.
template <bool kFork>
__device__ __forceinline__ void list_place(const PageOpArgs &a, int32_t nparts) {
  __shared__ int64_t sm[kWarps];
  __shared__ int32_t d_s[kMaxPlanUnits];
  int64_t before, total;
  int32_t err = plan_totals(a.part, nparts, sm, before, total);
  const uint64_t head = a.ws->head, tail = a.ws->tail;
  const int64_t free = static_cast<int64_t>(tail - head);
  if (!err && (free < 0 || free > a.F || (!kFork && free + total > a.F))) err = DKV_E_INTERNAL;
  if (!err && kFork && total > free) err = DKV_E_NOMEM;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.ws->total = err ? -1 : total;
    if (err) set_error(a.status, err);
    else a.cursors[kFork ? 0 : 1] = (kFork ? head : tail) + total;
  }
  if (err) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t v0 = static_cast<int64_t>(blockIdx.x) * a.upb;
  for (int i = threadIdx.x; i < a.upb; i += kThreads) {
    int32_t k, d = 0;
    if (v0 + i < a.V) {
      const int64_t u = list_unit(a, v0 + i, a.src, k);
      const int4 h = *reinterpret_cast<const int4 *>(a.unit_hdr + 4 * u);
      d = h.z + h.w;
    }
    d_s[i] = d;
  }
  __syncthreads();
  const int64_t at0 = static_cast<int64_t>(((kFork ? head : tail) + before) % static_cast<uint64_t>(a.F));
  for (int i = warp; i < a.upb; i += kWarps) {
    if (v0 + i >= a.V) break;
    int64_t off = 0;
    for (int j = lane; j < i; j += 32) off += d_s[j];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) off += __shfl_xor_sync(kFull, off, o);
    const int32_t d = d_s[i];
    int32_t k;
    const int64_t u = list_unit(a, v0 + i, a.src, k);
    int4 *hdr = reinterpret_cast<int4 *>(a.unit_hdr);
    if (kFork) {
      const int64_t w = list_unit(a, v0 + i, a.dst, k);
      const int4 h = hdr[u];
      for (int32_t j0 = lane; j0 < d; j0 += 128) {
        int32_t id[4], old[4];  // the loads before the stores, which might alias for all the compiler knows
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t j = j0 + 32 * e;
          if (j >= d || !in_range(at0 + off + j, 2 * a.F, a.status)) break;
          id[e] = a.free_list[ring(at0 + off + j, a.F)];
          old[e] = a.fwd[u * a.pmax + j];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t j = j0 + 32 * e;
          if (j >= d || !in_range(before + off + j, a.F, a.status)) break;
          const bool ok = id[e] >= 0 && id[e] < a.F;
          a.list[before + off + j] = ok ? make_int2(old[e], id[e]) : make_int2(-1, -1);
          if (!ok) {  // the ring is not what the contract says: skip the page
            set_error(a.status, DKV_E_INTERNAL);
            continue;
          }
          a.fwd[w * a.pmax + j] = id[e];
          a.rev_unit[id[e]] = static_cast<int32_t>(a.unit_base + w);
          a.rev_idx[id[e]] = j;
          a.page_cls[id[e]] = j < h.z ? DKV_CLASS_K8V4 : DKV_CLASS_K4V2;
        }
      }
      for (int32_t j = d + lane; j < a.pmax; j += 32) a.fwd[w * a.pmax + j] = -1;
      if (lane == 0) hdr[w] = h;
    } else {
      for (int32_t j0 = lane; j0 < d; j0 += 128) {
        int32_t id[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) id[e] = j0 + 32 * e < d ? a.fwd[u * a.pmax + j0 + 32 * e] : 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t j = j0 + 32 * e;
          if (j >= d || !in_range(at0 + off + j, 2 * a.F, a.status) || !in_range(id[e], a.F, a.status)) break;
          a.free_list[ring(at0 + off + j, a.F)] = id[e];
          a.rev_unit[id[e]] = -1;
          a.rev_idx[id[e]] = -1;
          a.page_cls[id[e]] = 0;
          a.fwd[u * a.pmax + j] = -1;
        }
      }
      if (lane == 0) hdr[u] = make_int4(0, 0, 0, 0);
    }
  }
}

// ------------------------------------------------------------------ copies --

constexpr int kUnroll = 8;  // 16-byte loads in flight per lane

// One warp copies n 16-byte words.
__device__ __forceinline__ void warp_copy(uint4 *dst, const uint4 *src, int32_t n, int lane) {
  for (int32_t c = lane; c < n; c += 32 * kUnroll) {
    uint4 x[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (c + 32 * i < n) x[i] = __ldcs(src + c + 32 * i);
#pragma unroll
    for (int i = 0; i < kUnroll; ++i)
      if (c + 32 * i < n) __stcs(dst + c + 32 * i, x[i]);
  }
}

constexpr int64_t kRowPiece = 4096;  // bytes of a row array one warp copies

// Piece p of the rows [0, ctx) of one (layer, fork) in an array with `row`
// bytes a position; `base` is the array at that layer.
__device__ __forceinline__ void copy_rows(uint8_t *base, const PageOpArgs &a, int32_t src, int32_t dst, int64_t row,
                                          int64_t p, int lane) {
  const int64_t bytes = __ldg(a.ctx_lens + src) * row, o = p * kRowPiece;
  if (o >= bytes || !in_range(bytes, a.cap * row + 1, a.status) || !in_range(dst, a.R, a.status)) return;
  const uint8_t *s = base + src * (a.cap * row) + o;
  uint8_t *d = base + dst * (a.cap * row) + o;
  const int64_t n = min(bytes - o, kRowPiece);
  warp_copy(reinterpret_cast<uint4 *>(d), reinterpret_cast<const uint4 *>(s), static_cast<int32_t>(n / 16), lane);
  for (int64_t c = (n & ~int64_t(15)) + lane; c < n; c += 32) d[c] = s[c];
}

// A warp per page of the copy list, then a warp per piece of the row arrays.
__device__ __forceinline__ void fork_copy(const PageOpArgs &a) {
  const int64_t total = a.ws->total;
  if (total < 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t b = a.page_bytes;
  for (int64_t j = warp; j < total; j += step) {
    const int2 p = a.list[j];
    if (p.x < 0 || !in_range(p.x, a.F, a.status) || !in_range(p.y, a.F, a.status)) continue;
    warp_copy(reinterpret_cast<uint4 *>(a.pages + p.y * b), reinterpret_cast<const uint4 *>(a.pages + p.x * b),
              static_cast<int32_t>(b / 16), lane);
  }
  if (!a.ctx_lens) return;
  // row pieces of one (layer, fork): classes, slots, significance, counts
  const int64_t row[4] = {a.classes ? a.Hkv : 0, a.slot_of ? int64_t{4} * a.Hkv : 0,
                          a.sig_sum ? int64_t{4} * a.Hq : 0, a.sig_cnt ? 4 : 0};
  int64_t per = 0, np[4];
  for (int i = 0; i < 4; ++i) per += np[i] = (a.cap * row[i] + kRowPiece - 1) / kRowPiece;
  uint8_t *base[4] = {a.classes, reinterpret_cast<uint8_t *>(a.slot_of), reinterpret_cast<uint8_t *>(a.sig_sum),
                      reinterpret_cast<uint8_t *>(a.sig_cnt)};
  for (int64_t j = warp; j < per * a.L * a.n; j += step) {
    int64_t p = j % per;
    const int64_t lk = j / per;
    const int32_t k = static_cast<int32_t>(lk % a.n), l = static_cast<int32_t>(lk / a.n);
    int i = 0;
    while (p >= np[i]) p -= np[i++];
    if (i == 3 && l != 0) continue;  // the counts are shared by the layers
    copy_rows(base[i] + l * (static_cast<int64_t>(a.R) * a.cap * row[i]), a, __ldg(a.src + k), __ldg(a.dst + k),
              row[i], p, lane);
  }
}

// ------------------------------------------------------------------ defrag --

// kDefragPages page ids a block: free pages below n (the live count) and live
// pages at or above it are counted; what the tables say of each live page is
// checked.  part = {holes, movers << 1 | error}.
__device__ __forceinline__ void defrag_plan(const PageOpArgs &a) {
  __shared__ int64_t sm[kWarps];
  __shared__ int32_t err_s;
  if (threadIdx.x == 0) err_s = 0;
  __syncthreads();
  const uint64_t head = a.cursors[0], tail = a.cursors[1];
  const int64_t n = a.F - static_cast<int64_t>(tail - head);
  const bool ok = tail >= head && n >= 0;
  int64_t holes = 0, movers = 0;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kDefragPages;
  constexpr int kEach = kDefragPages / kThreads;
  int32_t u[kEach], j[kEach], c[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t p = p0 + threadIdx.x + i * kThreads;
    const bool in = p < a.F;
    u[i] = in ? a.rev_unit[p] : -1;
    j[i] = in ? a.rev_idx[p] : 0;
    c[i] = in ? a.page_cls[p] : 0;
  }
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t p = p0 + threadIdx.x + i * kThreads, t = u[i] - a.unit_base;
    bool good = ok && (c[i] == 0) == (u[i] < 0);
    if (c[i] != 0) good = good && t >= 0 && t < a.U && j[i] >= 0 && j[i] < a.pmax && a.fwd[t * a.pmax + j[i]] == p;
    if (p >= a.F) continue;
    bad |= !good;
    if (c[i] == 0 && p < n) ++holes;
    if (c[i] != 0 && p >= n) ++movers;
  }
  if (bad) err_s = 1;
  holes = block_sum(holes, sm);
  movers = block_sum(movers, sm);
  if (threadIdx.x == 0) {
    a.part[blockIdx.x] = make_longlong2(holes, (movers << 1) | err_s);
    if (blockIdx.x == 0) {
      a.ws->head = head;
      a.ws->tail = tail;
    }
  }
}

// Same blocks: the block's holes and movers go to the lists at the ranks the
// sums before give, in ascending order of id.
__device__ __forceinline__ void defrag_list(const PageOpArgs &a, int32_t nparts) {
  __shared__ int64_t sm[kWarps];
  __shared__ int32_t wsum[2][kWarps];
  int64_t hb = 0, ht = 0, mb = 0, mt = 0, bad = 0;
  for (int32_t i = threadIdx.x; i < nparts; i += kThreads) {
    const longlong2 p = a.part[i];
    ht += p.x;
    mt += p.y >> 1;
    bad += p.y & 1;
    if (i < static_cast<int32_t>(blockIdx.x)) {
      hb += p.x;
      mb += p.y >> 1;
    }
  }
  ht = block_sum(ht, sm);
  mt = block_sum(mt, sm);
  bad = block_sum(bad, sm);
  hb = block_sum(hb, sm);
  mb = block_sum(mb, sm);
  const bool fail = bad != 0 || ht != mt;
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.ws->total = fail ? -1 : mt;
    if (fail) set_error(a.status, DKV_E_INTERNAL);
  }
  if (fail) return;
  const int64_t n = a.F - static_cast<int64_t>(a.ws->tail - a.ws->head);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t p0 = static_cast<int64_t>(blockIdx.x) * kDefragPages;
  for (int i0 = 0; i0 < kDefragPages && p0 + i0 < a.F; i0 += kThreads) {
    const int64_t p = p0 + i0 + threadIdx.x;
    const bool live = p < a.F && a.page_cls[p] != 0;
    const bool hole = p < a.F && p < n && !live, mover = p >= n && live;
    const uint32_t hm = __ballot_sync(kFull, hole), mm = __ballot_sync(kFull, mover);
    if (lane == 0) {
      wsum[0][warp] = __popc(hm);
      wsum[1][warp] = __popc(mm);
    }
    __syncthreads();
    int64_t h = hb, m = mb;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        h += wsum[0][w];
        m += wsum[1][w];
      }
      hb += wsum[0][w];
      mb += wsum[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    if (hole && in_range(h + __popc(hm & below), a.F, a.status)) a.list[h + __popc(hm & below)].y = static_cast<int32_t>(p);
    if (mover && in_range(m + __popc(mm & below), a.F, a.status))
      a.list[m + __popc(mm & below)].x = static_cast<int32_t>(p);
    __syncthreads();
  }
}

// A warp per move: the page's bytes, its reverse entry and class, the owner's
// forward entry; then the free list and the cursors.  Sources (ids >= n) and
// destinations (ids < n) are disjoint, so the order of the moves is free.
__device__ __forceinline__ void defrag_move(const PageOpArgs &a) {
  const int64_t total = a.ws->total;
  if (total < 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t b = a.page_bytes;
  for (int64_t j = warp; j < total; j += step) {
    const int2 p = a.list[j];  // x: the page that moves, y: where to
    if (!in_range(p.x, a.F, a.status) || !in_range(p.y, a.F, a.status)) continue;
    if (lane == 0) {
      const int32_t u = a.rev_unit[p.x], k = a.rev_idx[p.x];
      a.rev_unit[p.y] = u;
      a.rev_idx[p.y] = k;
      a.page_cls[p.y] = a.page_cls[p.x];
      a.fwd[(u - a.unit_base) * a.pmax + k] = p.y;
      a.rev_unit[p.x] = -1;
      a.rev_idx[p.x] = -1;
      a.page_cls[p.x] = 0;
    }
    warp_copy(reinterpret_cast<uint4 *>(a.pages + p.y * b), reinterpret_cast<const uint4 *>(a.pages + p.x * b),
              static_cast<int32_t>(b / 16), lane);
  }
  const uint64_t head = a.ws->head, tail = a.ws->tail, F = static_cast<uint64_t>(a.F);
  const uint64_t n = F - (tail - head);
  for (int64_t i = n + blockIdx.x * kThreads + threadIdx.x; i < a.F; i += static_cast<int64_t>(gridDim.x) * kThreads)
    a.free_list[i] = static_cast<int32_t>(i);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    const uint64_t h = head + (n + F - head % F) % F;  // the next value that is n mod F
    a.cursors[0] = h;
    a.cursors[1] = h + (F - n);
  }
}

// ----------------------------------------------------------------- launches --

template <bool kFork>
__global__ void __launch_bounds__(kThreads) k_list_plan(const __grid_constant__ PageOpArgs a) {
  let_next_launch_start();
  list_plan<kFork>(a);
}
template <bool kFork>
__global__ void __launch_bounds__(kThreads) k_list_place(const __grid_constant__ PageOpArgs a, int32_t nparts) {
  let_next_launch_start();
  after_launch_before();
  list_place<kFork>(a, nparts);
}
__global__ void __launch_bounds__(kThreads) k_fork_copy(const __grid_constant__ PageOpArgs a) {
  after_launch_before();
  fork_copy(a);
}
__global__ void __launch_bounds__(kThreads) k_defrag_plan(const __grid_constant__ PageOpArgs a) {
  let_next_launch_start();
  defrag_plan(a);
}
__global__ void __launch_bounds__(kThreads) k_defrag_list(const __grid_constant__ PageOpArgs a, int32_t nparts) {
  let_next_launch_start();
  after_launch_before();
  defrag_list(a, nparts);
}
__global__ void __launch_bounds__(kThreads) k_defrag_move(const __grid_constant__ PageOpArgs a) {
  after_launch_before();
  defrag_move(a);
}

// The steps of a small call in one launch: a cluster of kCluster blocks, whose
// barrier (hardware's, so every block is there) stands for the launches' order.
constexpr int kCluster = 8;

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

enum Op { kForkOp, kReleaseOp, kDefragOp };
template <int kOp>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) k_small(const __grid_constant__ PageOpArgs a) {
  if (kOp == kDefragOp) defrag_plan(a);
  else list_plan<kOp == kForkOp>(a);
  __threadfence();
  cluster_sync();
  if (kOp == kDefragOp) defrag_list(a, kCluster);
  else list_place<kOp == kForkOp>(a, kCluster);
  if (kOp == kReleaseOp) return;
  __threadfence();
  cluster_sync();
  if (kOp == kForkOp) fork_copy(a);
  else defrag_move(a);
}

int copy_grid(int64_t warps, int sms) {
  // Many short-lived blocks, a few pages a warp: 8 / 64 / 128 / 512 blocks a
  // multiprocessor take 547 / 530 / 524 / 580 us (8 prompts of 32 layers forked)
  // and 172 / 162 / 164 / 174 us (a 60% live pool packed).
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((warps + kWarps - 1) / kWarps, int64_t{sms} * 96)));
}

}  // namespace

// Up to 64 list units (or 8192 pages to look through) and 4 MB of copies eight
// blocks do as fast as the launches that more of them would take.
constexpr int64_t kSmallBytes = 4 << 20;

cudaError_t launch_fork(const PageOpArgs &a, int sms, cudaStream_t s) {
  const int32_t parts = static_cast<int32_t>((a.V + a.upb - 1) / a.upb);
  const size_t bits = 8 * static_cast<size_t>((a.R + 31) / 32);
  const int64_t rows = a.ctx_lens ? static_cast<int64_t>(a.L) * a.n * a.cap : 0;
  if (parts <= kCluster && a.V * a.pmax * a.page_bytes + rows * (int64_t{5} * a.Hkv + int64_t{4} * a.Hq + 4) <= kSmallBytes) {
    k_small<kForkOp><<<kCluster, kThreads, bits, s>>>(a);
    return cudaGetLastError();
  }
  k_list_plan<true><<<parts, kThreads, bits, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (cudaError_t e = launch_after(k_list_place<true>, dim3(parts), kThreads, 0, s, a, parts)) return e;
  return launch_after(k_fork_copy, dim3(copy_grid(a.V * a.pmax + rows / 16 + 1, sms)), kThreads, 0, s, a);
}

cudaError_t launch_release(const PageOpArgs &a, cudaStream_t s) {
  const int32_t parts = static_cast<int32_t>((a.V + a.upb - 1) / a.upb);
  const size_t bits = 8 * static_cast<size_t>((a.R + 31) / 32);
  if (parts <= kCluster) {
    k_small<kReleaseOp><<<kCluster, kThreads, bits, s>>>(a);
    return cudaGetLastError();
  }
  k_list_plan<false><<<parts, kThreads, bits, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  return launch_after(k_list_place<false>, dim3(parts), kThreads, 0, s, a, parts);
}

cudaError_t launch_defrag(const PageOpArgs &a, int sms, cudaStream_t s) {
  const int32_t parts = static_cast<int32_t>((a.F + kDefragPages - 1) / kDefragPages);
  if (parts <= kCluster && a.F * a.page_bytes <= kSmallBytes) {
    k_small<kDefragOp><<<kCluster, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  k_defrag_plan<<<parts, kThreads, 0, s>>>(a);
  if (cudaError_t e = cudaGetLastError()) return e;
  if (cudaError_t e = launch_after(k_defrag_list, dim3(parts), kThreads, 0, s, a, parts)) return e;
  return launch_after(k_defrag_move, dim3(copy_grid(a.F, sms)), kThreads, 0, s, a);
}

}  // namespace dkv
