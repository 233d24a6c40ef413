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
// two registers and its sums plain additions of one thread in a fixed order
// (no atomics).  A block takes a contiguous range of one unit's token tiles,
// four tiles (a group) at a time, K converted once and resident, and streams
// the rows of Q past them in blocks of 128 columns: `nb` columns per head, as
// many heads as fit (a draft of eight tokens: 16 columns for each of four
// heads), so every 16 columns belong to one head.
//   convert warps (8)  K tiles as in the attention (codes less their middle,
//     fp16); Q blocks as fp16 times one power of two per block, with the sums
//     of their rows and -lse (log2) per column;
//   MMA warp           S^T of every (block, tile) into four tensor-memory
//     buffers, one per tile of the group;
//   sum warps (2 x 4)  a thread per token, tiles w and w + 2 of the group.
#include <algorithm>
#include <cmath>

#include "token_tiles.cuh"

namespace dkv {

namespace {

using namespace tc;

constexpr int kSumWarps = 8, kConvWarps = 8;
constexpr int kMmaWarp = kSumWarps + kConvWarps;
constexpr int kThreads = 32 * (kMmaWarp + 1);
constexpr uint32_t kTmemCols = 512;
constexpr int kGroup = 4;    // token tiles resident at once
constexpr int kMaxAcc = 8;   // heads whose sums wait in shared memory for one joint update

struct __align__(1024) Smem {
  uint8_t k[kGroup][kTileBytes];
  uint8_t q[2][kTileBytes];
  float s[2 * kGroup][128], z[2 * kGroup][128];  // by parity of the group
  int32_t pos[2 * kGroup][128];                  // -1: not a token
  float4 col[4][64];                             // per column pair: row sums of Q, -lse (log2)
  float acc[kGroup][kMaxAcc][128];
  uint64_t kfull[kGroup], kempty[kGroup], mfull[2 * kGroup], sfull[kGroup], sfree[kGroup];
  uint64_t qfull[2], qempty[2], cfull[4], qm[4], done;
  uint32_t qmax[4];
  float qf[4];  // 2^-e of the block's Q
  uint32_t tmem;
  int32_t abort;
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

// Tokens tk and tk + 64 of a tile: K codes, scale and zero, position.
struct Key {
  uint32_t k[2][2][4];
  uint32_t md[2];
  int32_t pos[2];
};

template <int KW>
__device__ __forceinline__ void fetch_key(const DeqCtx &d, const Where<2> &w, Key &h, int32_t posoff) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const bool ok = w.id[p] >= 0 && w.id[p] < d.a->F;
    const uint8_t *pg = d.a->pages + (ok ? w.id[p] : 0) * d.bytes;
    const uint8_t *src = pg + w.slot[p] * (16 * KW) + d.c * (4 * KW);
    load16<KW>(h.k[p][0], src + d.hs * (2 * KW));
    load16<KW>(h.k[p][1], src + (d.hs ^ 1) * (2 * KW));
    h.md[p] = __ldg(reinterpret_cast<const uint32_t *>(pg + d.meta + 8 * w.slot[p]));
    h.pos[p] = ok ? __ldg(reinterpret_cast<const int32_t *>(pg + posoff + 4 * w.slot[p])) : -1;
    if (!ok && w.id[p] != -1) set_error(d.a->status, DKV_E_INTERNAL);
  }
}

template <int W>
__device__ __forceinline__ void convert_key(const DeqCtx &d, const Where<2> &w, const Key &h, Smem &sm, uint8_t *dst,
                                            int slot, float f, int32_t ctx) {
  constexpr int kMid = 1 << (W - 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t w0, w1;
      __half2 o[4];
      group_of<W>(h.k[p][i >> 1], i & 1, w0, w1);
      group_codes<W, kMid>(w0, w1, o);
      put(dst, d.off[i] + p * (64 * 128), o);
    }
    if (d.c == 0) {
      const int row = d.tk + 64 * p;
      const __half2 m = u2h(h.md[p]);
      const float s = __low2float(m), z = __high2float(m);
      sm.s[slot][row] = s * f;
      sm.z[slot][row] = fmaf(kMid, s, z) * f;
      const bool bad = h.pos[p] >= ctx || h.pos[p] < 0;
      if (bad && w.id[p] >= 0 && w.id[p] < d.a->F) set_error(d.a->status, DKV_E_INTERNAL);
      sm.pos[slot][row] = bad ? -1 : h.pos[p];
    }
  }
}

// A block of Q: which heads and tokens its columns are.
struct Block {
  int32_t head0, i0;
};

template <int SC>
__global__ void __launch_bounds__(kThreads, 1)
    k_extend_sig(const __grid_constant__ ExtendArgs a, int32_t splits, int32_t nb) {
  constexpr int KH = scheme_kh(SC);
  extern __shared__ __align__(16) unsigned char smem_raw[];
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + (-saddr(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ui = blockIdx.x / splits, rh = ui / a.Hkv;  // unit, (layer, request)
  const int32_t sp = static_cast<int32_t>(blockIdx.x - ui * splits), h = static_cast<int32_t>(ui - rh * a.Hkv);
  const int32_t li = static_cast<int32_t>(rh / a.R), r = static_cast<int32_t>(rh - li * a.R);
  int64_t before;
  if (!lens_valid(a, r, before)) return;
  const int32_t acc_n = __ldg(a.acc_lens + r), ctx = __ldg(a.ctx_lens + r);
  if (acc_n == 0) return;
  const Unit x = load_unit(a, (static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.Hkv + h);
  const int32_t fresh = a.k_new ? acc_n : 0;
  const Tiles ts{(x.n_hi + 127) / 128, (x.n_lo + 127) / 128, (fresh + 127) / 128};
  const int32_t nt = ts.count(), per = (nt + splits - 1) / splits;
  const int32_t j0 = min(nt, sp * per), n = min(nt, j0 + per) - j0;
  if (n == 0) return;
  const int64_t tok0 = static_cast<int64_t>(li) * a.T + before;
  volatile int32_t *abort = &sm.abort;
  // blocks of Q: hpb heads each, or (nb = 128) 128 tokens of one head
  const int32_t hpb = min(a.G, 128 / nb), ib = nb == 128 ? (acc_n + 127) / 128 : 1;
  const int32_t nblk = (a.G + hpb - 1) / hpb * ib, cols = hpb * nb, groups = (n + kGroup - 1) / kGroup;
  auto block_at = [&](int32_t b) { return Block{b / ib * hpb, b % ib * 128}; };

  if (tid == 0) {
    for (int i = 0; i < kGroup; ++i) {
      mbar_init(&sm.kfull[i], kConvWarps);
      mbar_init(&sm.kempty[i], 1);
      mbar_init(&sm.sfull[i], 1);
      mbar_init(&sm.sfree[i], kSumWarps / 2);
      mbar_init(&sm.cfull[i], kConvWarps);
      mbar_init(&sm.qm[i], kConvWarps);
      sm.qmax[i] = 0;
    }
    for (int i = 0; i < 2 * kGroup; ++i) mbar_init(&sm.mfull[i], kConvWarps);
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

  if (warp < kSumWarps) {
    // ================= sum warps: a thread per token
    const int wg = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const bool joint = a.G <= kMaxAcc;  // the heads' sums wait for one update of the token's row
    float s[2], z[2], run[2] = {0.0f, 0.0f};
    int32_t pos[2], tj[2];  // position; index among the new tokens (held: -1)
    bool ok = true;
    for (int32_t g = 0; g < groups && ok; ++g) {
      const int32_t ng = min(kGroup, n - g * kGroup);
      for (int32_t b = 0; b < nblk && ok; ++b) {
        const int32_t qi = nblk == 1 ? 0 : g * nblk + b;
        const Block bk = block_at(b);
        if ((nblk > 1 || g == 0) && !(ok = warp_wait(&sm.cfull[qi & 3], (qi >> 2) & 1u))) break;
        const float qf = sm.qf[qi & 3];
        const float4 *col = sm.col[qi & 3];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int t = wg + 2 * e;
          if (t >= ng || !ok) continue;
          if (b == 0) {
            const int ms = (g & 1) * kGroup + t;
            if (!(ok = warp_wait(&sm.mfull[ms], (g >> 1) & 1u))) continue;
            s[e] = sm.s[ms][row];
            z[e] = sm.z[ms][row];
            pos[e] = sm.pos[ms][row];
            const Tile tl = tile_at(ts, x, fresh, j0 + g * kGroup + t);
            tj[e] = tl.kind == 2 ? tl.t0 + row : -1;
          }
          // the row that the sums are added to, early
          const bool last = b == nblk - 1;
          float *dst = a.sig_sum + ((static_cast<int64_t>(a.layer0 + li) * a.R + r) * a.cap + max(pos[e], 0)) * a.Hq +
                       h * a.G;
          float old[kMaxAcc];
          if (last && joint) {
#pragma unroll
            for (int q = 0; q < kMaxAcc; ++q) old[q] = q < a.G && pos[e] >= 0 && tj[e] < 0 ? dst[q] : 0.0f;
          }
          if (!(ok = warp_wait(&sm.sfull[t], (g * nblk + b) & 1u))) continue;
          fence_after();
          const float se = s[e] * qf, ze = z[e] * qf;
          const uint64_t s2 = f2_pack(se, se), z2 = f2_pack(ze, ze);
          const bool diag = __any_sync(kFull, tj[e] >= 0 && bk.i0 < tj[e]);
#pragma unroll 1
          for (int32_t c = 0; c < cols; c += 16) {
            uint32_t u[16];
            tmem_ld16(tmem + lanes + 128 * t + c, u);
            tmem_wait16(u);
            uint64_t sum[2] = {0, 0};
            // new token tj: rows before it do not attend to it
            const int32_t skip = diag ? tj[e] - (bk.i0 + c % nb) : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 cv = col[(c >> 1) + i];
              float y0, y1;
              f2_unpack(f2_fma(s2, f2_pack(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])),
                               f2_fma(z2, f2_pack(cv.x, cv.y), f2_pack(cv.z, cv.w))), y0, y1);
              y0 = ex2(y0);
              y1 = ex2(y1);
              if (diag) {
                y0 = 2 * i < skip ? 0.0f : y0;
                y1 = 2 * i + 1 < skip ? 0.0f : y1;
              }
              sum[i & 1] = f2_add(sum[i & 1], f2_pack(y0, y1));
            }
            float a0, a1;
            f2_unpack(f2_add(sum[0], sum[1]), a0, a1);
            run[e] += a0 + a1;
            if ((c + 16) % nb == 0 && (nb < 128 || b % ib == ib - 1)) {  // the head is done
              const int32_t hd = bk.head0 + c / nb;
              if (joint) {
                if (hd < a.G) sm.acc[t][hd][row] = run[e];
              } else if (hd < a.G && pos[e] >= 0) {
                dst[hd] = tj[e] < 0 ? dst[hd] + run[e] : run[e];
              }
              run[e] = 0.0f;
            }
          }
          fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.sfree[t]);
          if (last && joint && pos[e] >= 0) {
            float v[kMaxAcc];
#pragma unroll
            for (int q = 0; q < kMaxAcc; ++q) v[q] = q < a.G ? old[q] + sm.acc[t][q][row] : 0.0f;
            if ((a.G & 3) == 0) {  // 16-byte aligned: Hq is a multiple of 4 as well
              *reinterpret_cast<float4 *>(dst) = make_float4(v[0], v[1], v[2], v[3]);
              if (a.G == 8) *reinterpret_cast<float4 *>(dst + 4) = make_float4(v[4], v[5], v[6], v[7]);
            } else {
#pragma unroll
              for (int q = 0; q < kMaxAcc; ++q)
                if (q < a.G) dst[q] = v[q];
            }
          }
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ================= convert warps
    const int dt = tid - 32 * kSumWarps;
    const PageGeom pg = page_geom(SC, a.P);
    DeqCtx d{&a, x, 0xffffffffu / a.P + 1, 0xffffffffu / (2 * a.P) + 1, static_cast<int32_t>(pg.bytes),
             static_cast<uint32_t>(pg.vbase), static_cast<uint32_t>(pg.meta), dt >> 2, dt & 3, (dt & 3) >> 1, {}};
#pragma unroll
    for (int i = 0; i < 4; ++i) d.off[i] = group_at(d.tk, 4 * d.c + (i ^ (2 * d.hs)));
    const float f = a.scale * kLog2e;
    const int32_t posoff = static_cast<int32_t>(pg.pos);
    Key key;
    Where<2> w0, w1;
    bool ok = true;
    Tile t{}, tn{};
    auto load = [&] {
      if (t.kind == 0) fetch_key<KH>(d, w0, key, posoff);
      else if (t.kind == 1) fetch_key<KH / 2>(d, w0, key, posoff);
    };
    // block b of Q into buffer qi
    auto stage = [&](int32_t b, int32_t qi) -> bool {
      const Block bk = block_at(b);
      if (qi >= 2 && !warp_wait(&sm.qempty[qi & 1], ((qi >> 1) - 1) & 1u)) return false;
      uint4 v[2][4];
      uint32_t mx = 0;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int32_t cl = d.tk + 64 * p, hd = bk.head0 + cl / nb, i = bk.i0 + cl % nb;
        const bool have = cl < cols && hd < a.G && i < acc_n;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + ((tok0 + i) * a.Hq + h * a.G + hd) * 128) + 4 * d.c;
        uint32_t rm = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[p][k] = have ? __ldg(src + (k ^ (2 * d.hs))) : make_uint4(0, 0, 0, 0);
          const uint32_t *w = reinterpret_cast<const uint32_t *>(&v[p][k]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            rm = max(rm, max((w[q] << 16) & 0x7fffffffu, w[q] & 0x7fff0000u));  // bits of |value|: they order like it
        }
        rm = max(rm, __shfl_xor_sync(kFull, rm, 1));
        rm = max(rm, __shfl_xor_sync(kFull, rm, 2));
        if (rm < 0x7f800000u) mx = max(mx, rm);  // a row that is not finite spoils itself alone
      }
      mx = __reduce_max_sync(kFull, mx);
      if (lane == 0) {
        if (mx) atomicMax(&sm.qmax[qi & 3], mx);
        mbar_arrive(&sm.qm[qi & 3]);
      }
      if (!warp_wait(&sm.qm[qi & 3], (qi >> 2) & 1u)) return false;
      const int e = lift_exponent(*const_cast<volatile uint32_t *>(&sm.qmax[qi & 3]));
      const float sc = pow2f(e);
      if (dt == 0) {
        sm.qf[qi & 3] = pow2f(-e);
        sm.qmax[(qi + 2) & 3] = 0;  // last used two blocks ago
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int32_t cl = d.tk + 64 * p, hd = bk.head0 + cl / nb, i = bk.i0 + cl % nb;
        const bool have = cl < cols && hd < a.G && i < acc_n;
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 y = v[p][k];
          const float c0 = bf16_lo(y.x) * sc, c1 = bf16_hi(y.x) * sc, c2 = bf16_lo(y.y) * sc, c3 = bf16_hi(y.y) * sc;
          const float c4 = bf16_lo(y.z) * sc, c5 = bf16_hi(y.z) * sc, c6 = bf16_lo(y.w) * sc, c7 = bf16_hi(y.w) * sc;
          sum += ((c0 + c1) + (c2 + c3)) + ((c4 + c5) + (c6 + c7));
          *reinterpret_cast<uint4 *>(sm.q[qi & 1] + d.off[k] + p * (64 * 128)) =
              make_uint4(f16x2_rn(c0, c4), f16x2_rn(c1, c5), f16x2_rn(c2, c6), f16x2_rn(c3, c7));
        }
        sum += __shfl_xor_sync(kFull, sum, 1);
        sum += __shfl_xor_sync(kFull, sum, 2);
        if (d.c == 0) {
          const float ls = have ? a.lse[(tok0 + i) * a.Hq + h * a.G + hd] : -INFINITY;
          float *dst = reinterpret_cast<float *>(&sm.col[qi & 3][cl >> 1]) + (cl & 1);
          dst[0] = have ? sum : 0.0f;
          dst[2] = ls == -INFINITY ? -INFINITY : -ls * kLog2e;  // -inf: the column adds nothing
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
    t = tile_at(ts, x, fresh, j0);
    locate(d, t, w0);
    load();
    if (n > 1) {
      tn = tile_at(ts, x, fresh, j0 + 1);
      locate(d, tn, w1);
    }
#pragma unroll 1
    for (int32_t g = 0; g < groups && ok; ++g) {
      if (nblk > 1 || g == 0) ok = stage(0, g * nblk);
      const int32_t ng = min(kGroup, n - g * kGroup);
#pragma unroll 1
      for (int32_t q = 0; q < ng && ok; ++q) {
        const int32_t j = g * kGroup + q;
        const int ms = (g & 1) * kGroup + q;
        if (g > 0 && !(ok = warp_wait(&sm.kempty[q], (g - 1) & 1u))) break;
        if (t.kind == 0) {
          convert_key<KH>(d, w0, key, sm, sm.k[q], ms, f, ctx);
        } else if (t.kind == 1) {
          convert_key<KH / 2>(d, w0, key, sm, sm.k[q], ms, f, ctx);
        } else {
          new_k<2, false>(d, t, tok0, h, sm, sm.k[q], ms, f);
          if (d.c == 0) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const int row = d.tk + 64 * p;
              sm.pos[ms][row] = row < t.n ? ctx + t.t0 + row : -1;
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.kfull[q]);
          mbar_arrive(&sm.mfull[ms]);
        }
        if (j + 1 < n) {
          t = tn;
          w0 = w1;
          load();
        }
        if (j + 2 < n) {
          tn = tile_at(ts, x, fresh, j0 + j + 2);
          locate(d, tn, w1);
        }
      }
#pragma unroll 1
      for (int32_t b = 1; b < nblk && ok; ++b) ok = stage(b, g * nblk + b);
    }
  } else if (lane == 0) {
    // ================= MMA warp, one lane
    const uint32_t id = idesc(false, 128, cols, false);
    const uint64_t dk = sw128_desc(saddr(sm.k[0]), 16, 1024), dq = sw128_desc(saddr(sm.q[0]), 16, 1024);
    constexpr uint32_t kStep = kTileBytes >> 4;
    bool ok = true;
    for (int32_t g = 0; g < groups && ok; ++g) {
      const int32_t ng = min(kGroup, n - g * kGroup);
      for (int32_t b = 0; b < nblk && ok; ++b) {
        const int32_t qi = nblk == 1 ? 0 : g * nblk + b;
        if ((nblk > 1 || g == 0) && !(ok = wait(&sm.qfull[qi & 1], (qi >> 1) & 1u))) break;
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
          if (b == nblk - 1) mma_commit(&sm.kempty[t]);
        }
        if (ok && nblk > 1) mma_commit(&sm.qempty[qi & 1]);
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

template <int SC>
cudaError_t launch(const ExtendArgs &a, int64_t blocks, int32_t splits, int32_t nb, cudaStream_t s) {
  const int smem = static_cast<int>(kSmemBytes);
  if (cudaError_t e = cudaFuncSetAttribute(k_extend_sig<SC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) return e;
  k_extend_sig<SC><<<static_cast<unsigned>(blocks), kThreads, smem, s>>>(a, splits, nb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_extend_sig(const ExtendArgs &a, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(a.n_layers) * a.R * a.Hkv;
  const int32_t nb = a.max_new <= 16 ? 16 : a.max_new <= 32 ? 32 : a.max_new <= 64 ? 64 : 128;
  // runs of a unit's tiles, until every SM has a few blocks of at least one group
  const int64_t tiles = (static_cast<int64_t>(a.cap) + 127) / 128 + 2;
  int64_t splits = 1;
  while (units * splits < 4 * 152 && splits * 2 * kGroup <= tiles) splits *= 2;
  const int64_t blocks = units * splits;
  if (blocks == 0 || a.max_new == 0) return cudaSuccess;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const int32_t sp = static_cast<int32_t>(splits);
  return a.scheme == 0 ? launch<0>(a, blocks, sp, nb, s) : a.scheme == 1 ? launch<1>(a, blocks, sp, nb, s)
                                                                       : launch<2>(a, blocks, sp, nb, s);
}

}  // namespace dkv
