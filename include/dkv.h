/*
 * dkv.h -- libdkv: differentiated KV-cache compaction on one GB300 (sm_103a).
 *
 * Method: "DiffKV: Differentiated Memory Management for Large Language Models
 * with Parallel KV Compaction" (arXiv 2412.03131), as summarised on its Pith
 * review page.  For every (layer, request, KV head) -- a "unit" -- the library
 *   1. scores each token by the average attention it has received from later
 *      tokens, max-aggregated over the GQA query heads of the KV head
 *      ("What carries the argument"; Referee Report, major comment 2 on
 *      Section 4 / Algorithm 1);
 *   2. classifies it against alpha_h/N and alpha_l/N into K8V4 (keys 8-bit,
 *      values 4-bit), K4V2 or pruned ("Core claim");
 *   3. hands every unit a disjoint contiguous run of page ids from a circular
 *      free page list through a parallel prefix sum over the units' page
 *      demands, and fills the bidirectional page table ("What carries the
 *      argument"; abstract: "on-GPU memory manager that compacts fragmented
 *      free memory list into contiguous regions in parallel");
 *   4. quantises the surviving tokens per token (asymmetric min/max over the
 *      128 channels of a head, fp16 scale and zero, fp32 round-half-to-even)
 *      and packs them into unified pages ("Core claim": unified pages).
 *
 * Conventions shared by every call
 *   - Every data pointer is a DEVICE pointer, allocated and owned by the
 *     caller.  The library allocates no device memory; dkv_compact takes a
 *     caller-provided workspace sized by dkv_workspace_size.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Calls are asynchronous on that stream unless stated.
 *   - Return value: DKV_OK or a negative code.  A *synchronous* error (bad
 *     argument: DKV_E_INVAL; a CUDA launch failure: DKV_E_CUDA) means nothing
 *     was enqueued.  Conditions found on the device (DKV_E_NOMEM,
 *     DKV_E_RANGE, DKV_E_TIMEOUT, DKV_E_LENS, DKV_E_INTERNAL) are recorded in
 *     the pool's device status word and read with dkv_get_status.  A call
 *     that ends in a device-side error changes neither the cursors, nor the
 *     forward and reverse tables, nor any live page: it is all-or-nothing
 *     (pages that were free may have been scribbled and stay free).
 *   - Calls on one pool must be ordered on one stream (or synchronised by the
 *     caller); two calls on one pool in flight at once race.
 *
 * Unit order is layer-major: u = (l * R + r) * Hkv + h.  One call over L
 * layers gives bit-identical results to L one-layer calls made in layer
 * order with unit_base = l * R * Hkv and tables offset by the same unit count.
 *
 * Precision schemes (dkv_pool.scheme).  The review's free-parameter list
 * compares K8V4, K4V8, K8V2, K4V2, K2V4 and K4V1 (its Section 7.2) and keeps
 * K8V4-K4V2.  A scheme pairs a high class (K at kh bits, V at vh bits) with a
 * low class at half of each, so a low token takes exactly half a high
 * token's code bytes:
 *     DKV_SCHEME_K8V4_K4V2 (0, the default)   kh = 8, vh = 4
 *     DKV_SCHEME_K8V2_K4V1 (1)                kh = 8, vh = 2
 *     DKV_SCHEME_K4V8_K2V4 (2)                kh = 4, vh = 8
 * DKV_CLASS_K8V4 / DKV_CLASS_K4V2 below name the high / low class of
 * whichever scheme the pool uses.
 *
 * Unified page layout (P even; C = 16 (kh + vh) P bytes of codes; page bytes
 * C + 24 P: 216 P for schemes 0 and 2, 184 P for scheme 1).  A high page
 * holds P tokens, a low page 2P tokens:
 *     [0, 16 kh P)     K codes: high slot s at 16 kh s, low slot s at 8 kh s
 *     [16 kh P, C)     V codes: high slot s at 16 kh P + 16 vh s, low slot s
 *                      at 16 kh P + 8 vh s
 *     [C, C + 16P)     per slot s at C + 8 s: fp16 k_scale, k_zero, v_scale,
 *                      v_zero
 *     [C + 16P, C + 24P)  per slot s at C + 16P + 4 s: int32 token position
 * For scheme 0 that is K codes [0, 128P), V codes [128P, 192P), metadata at
 * 192P, positions at 208P.  Sub-byte codes pack lowest channel in the lowest
 * bits.  Slots fill in rank order (ascending position); unused slots,
 * including slots P..2P-1 of a high page, hold zero codes, zero metadata and
 * position -1.
 *
 * Quantiser per token row x[0..127] and bit width b (n = 2^b - 1):
 *     mn = min x, mx = max x (a zero extreme taken as +0); any non-finite x
 *     or |x| > 65504 is DKV_E_RANGE
 *     s16 = fp16_rn((mx - mn) / n), set to 2^-24 if it is 0 while mx > mn,
 *           and to 65504 if it is infinite (1-bit codes of a span > 65519)
 *     z16 = fp16_rn(mn);  s = (float)s16, z = (float)z16
 *     q   = s == 0 ? 0 : clamp(rint_even((x - z) / s), 0, n)   (fp32 ops)
 *     x'  = fma((float)q, s, z)                               (dequantised)
 */
#ifndef DKV_H
#define DKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DKV_OK 0
#define DKV_E_INVAL (-1)    /* sync: invalid argument; nothing enqueued */
#define DKV_E_NOMEM (-2)    /* device: total page demand > free pages */
#define DKV_E_RANGE (-3)    /* device: a K/V value to quantise is non-finite or > 65504 */
#define DKV_E_TIMEOUT (-4)  /* device: a bounded wait of the page scan gave up */
#define DKV_E_INTERNAL (-5) /* device: an internal consistency check failed */
#define DKV_E_CUDA (-6)     /* sync: a CUDA call failed while enqueuing */
#define DKV_E_LENS (-7)     /* device: lens[] disagree with T or max_len */

/* Token classes written to dkv_batch.classes and dkv_pool.page_cls (high /
 * low class of the pool's scheme; the names are those of scheme 0). */
#define DKV_CLASS_PRUNE 0
#define DKV_CLASS_K4V2 1
#define DKV_CLASS_K8V4 2

/* Precision schemes (dkv_pool.scheme). */
#define DKV_SCHEME_K8V4_K4V2 0
#define DKV_SCHEME_K8V2_K4V1 1
#define DKV_SCHEME_K4V8_K2V4 2

#define DKV_HEAD_DIM 128

/* One batch of prefill tokens.  T = sum(lens) tokens per layer and KV head. */
typedef struct dkv_batch {
  int32_t L, R, Hq, Hkv, D;  /* layers, requests, query heads, KV heads, D = 128 */
  int32_t max_len;           /* host-side upper bound on every lens[r] */
  int64_t T;                 /* total tokens of the batch (sum of lens) */
  int64_t unit_base;         /* global id of unit 0 of this call, stored in rev_unit */
  const void *k;             /* bf16 [L][T][Hkv][128], 16-byte aligned */
  const void *v;             /* bf16 [L][T][Hkv][128], 16-byte aligned */
  const float *sig_sum;      /* fp32 [L][T][Hq]: summed attention each token received */
  const int32_t *sig_cnt;    /* int32 [T]: how many scores were summed (N - i in prefill) */
  const int32_t *lens;       /* int32 [R]: tokens of each request, device memory */
  uint8_t *classes;          /* out: uint8 [L][T][Hkv], DKV_CLASS_* per token row */
} dkv_batch;

typedef struct dkv_params {
  float alpha_h;             /* K8V4 threshold alpha_h / N */
  float alpha_l;             /* K4V2 threshold alpha_l / N; 0 <= alpha_l <= alpha_h */
  int32_t spin_limit;        /* polls of one predecessor in the scan look-back before
                                DKV_E_TIMEOUT; 0 gives up at once (any call with
                                more than one scan partition then times out);
                                negative = library default (about a second) */
  int32_t reserved;          /* must be 0 */
  void *profiler;            /* nullable dkv_profiler*: per-kernel event timing */
} dkv_params;

/* The page pool: circular free list, cursors, reverse table and pages. */
typedef struct dkv_pool {
  int64_t F;                 /* pages; 1 <= F <= 2^31 - 1 */
  int32_t P;                 /* high-class tokens per page (low-class pages hold 2P); even */
  int32_t scheme;            /* DKV_SCHEME_*: bit widths and page layout (0 = K8V4/K4V2) */
  int32_t *free_list;        /* int32 [F]: ring of free page ids, slots [head, tail) mod F */
  uint64_t *cursors;         /* uint64 [2]: {head, tail}, monotone; free = tail - head */
  int32_t *rev_unit;         /* int32 [F]: owning global unit id, -1 if free */
  int32_t *rev_idx;          /* int32 [F]: index in the owner's forward row, -1 if free */
  uint8_t *page_cls;         /* uint8 [F]: 0 free, 1 K4V2 page, 2 K8V4 page */
  uint8_t *pages;            /* uint8 [F][dkv_page_bytes], 16-byte aligned */
  int32_t *status;           /* int32 [1]: first device-side error since last read */
} dkv_pool;

/* Forward page table of the units of one call. */
typedef struct dkv_tables {
  int32_t *fwd;              /* int32 [U][pmax]: page ids, K8V4 pages first; -1 past demand */
  int32_t pmax;              /* >= ceil(max_len / P) + 1 */
  int32_t reserved;
  int32_t *unit_hdr;         /* int32 [U][4]: {n_k8v4, n_k4v2, pages_k8v4, pages_k4v2} */
} dkv_tables;

/* Bytes of one unified page of the given scheme and P (host only):
 * (16 (kh + vh) + 24) P.  DKV_E_INVAL for an unknown scheme or P not even
 * and positive. */
int32_t dkv_page_bytes(int32_t scheme, int32_t P, int64_t *bytes);

/* Workspace bytes dkv_compact needs for this batch shape (host only; reads
 * L, R, Hkv, T and max_len of `b`).  Returns DKV_OK or DKV_E_INVAL. */
int32_t dkv_workspace_size(const dkv_batch *b, size_t *bytes);

/* Reset a pool: free_list[i] = i, head = 0, tail = F, rev_* = -1,
 * page_cls = 0, status = 0.  Page contents are left as they are. */
int32_t dkv_init_pool(const dkv_pool *pool, void *stream);

/* Prefill compaction of one batch (steps 1-4 above), asynchronous.
 * workspace: device, 256-byte aligned, >= dkv_workspace_size bytes; its
 * contents need no initialisation and are scratch after the call.
 * On success: classes written; for every unit u, fwd[u][0 .. d_u) holds the
 * page ids taken from free-list slots [head + off_u, head + off_u + d_u) mod F
 * (off_u = exclusive prefix sum of d_u = ceil(n_k8v4 / P) + ceil(n_k4v2 / 2P)),
 * rev_unit / rev_idx / page_cls describe those pages, the pages hold the
 * packed tokens, and head advanced by sum(d_u).
 * One part of the work, clearing the unused slot halves of the new K8V4
 * pages, runs on a library-owned second stream of the current device: it is
 * forked from `stream` after the page scan and joined back before the
 * commit, so the call's effects are ordered on `stream` as if it ran there
 * alone (under stream capture it becomes a fork and a join of the graph).
 * The first call in a CUDA context creates that stream and two events, kept
 * for that context until process exit (a context made after cudaDeviceReset
 * gets its own); make that first call before any stream capture.  Calls from
 * several host threads are safe (the fork and join are enqueued under a
 * lock). */
int32_t dkv_compact(const dkv_batch *b, const dkv_params *p, const dkv_pool *pool,
                    const dkv_tables *t, void *workspace, size_t workspace_bytes,
                    void *stream);

/* dkv_compact without a caller workspace, for callers that cannot allocate
 * device memory (no counterpart in the paper).  Same arguments, results and
 * errors as dkv_compact; the scratch is a library-owned __device__ array of
 * DKV_NOALLOC_SCRATCH_BYTES that every GPU loading the library holds until
 * process exit.  A batch whose dkv_workspace_size exceeds that limit is
 * rejected with DKV_E_INVAL before anything is enqueued (the Llama-3-8B-shaped
 * batch of 32 layers x 16 x 4096 tokens needs about 12.5 MiB).  Every call
 * resolves the array's device address in the current context
 * (cudaGetSymbolAddress, which loads the library's module on first use); make
 * the first call on a device before any stream capture.  The array is shared by all calls on a device and keeps the last call's contents
 * (nothing in it needs to start at zero): calls that overlap on the GPU race,
 * so order them on one stream.  Allocates no device memory (the first call
 * on a device creates dkv_compact's second stream and its events). */
#define DKV_NOALLOC_SCRATCH_BYTES (16u << 20)
int32_t dkv_compact_noalloc(const dkv_batch *b, const dkv_params *p, const dkv_pool *pool,
                            const dkv_tables *t, void *stream);

/* Dequantise one page: k_out, v_out fp32 [2P][128], pos_out int32 [2P]
 * (device).  Slots the page class does not have, unused slots and free pages
 * decode to 0 with position -1.  page_id outside [0, F) is DKV_E_INVAL. */
int32_t dkv_dequant_page(const dkv_pool *pool, int32_t page_id, float *k_out, float *v_out,
                         int32_t *pos_out, void *stream);

/* Dequantise n pages whose ids are in device memory page_ids[n]; outputs are
 * [n][2P][128] and [n][2P].  An id outside [0, F) decodes as a free page. */
int32_t dkv_dequant_pages(const dkv_pool *pool, const int32_t *page_ids, int32_t n,
                          float *k_out, float *v_out, int32_t *pos_out, void *stream);

/* ------------------------------------------------------------------------
 * Generation (decode) step.  DiffKV review, Referee Report, major comment 2
 * (Algorithm 1 classifies tokens as they age in the generation phase;
 * demotion and pruning are irreversible), with "What carries the argument"
 * and "Core claim" for classes, unified pages and the page allocator.
 *
 * The context axis of a decode batch is capacity-strided: position i of
 * request r is token row r * cap + i of sig_sum, sig_cnt, classes and
 * slot_of.  Units, pages and tables are those of dkv_compact (a prefill with
 * tables of the same pmax leaves a valid starting state).
 *
 * One step, with N = ctx_lens[r] + new_lens[r]:
 *   - every live token's class becomes min(old class, classify(score, N));
 *     the new token (position ctx_lens[r], when new_lens[r] = 1) is
 *     classified as in prefill;
 *   - per unit, each list (K8V4 slots, K4V2 slots) drops its removed tokens;
 *     with `keep` survivors, those in slots >= keep move, in ascending slot
 *     order, into the holes below keep, in ascending order (bytes copied);
 *   - tokens demoted K8V4 -> K4V2 are appended to the K4V2 list in ascending
 *     position order, requantised (4-bit K, 2-bit V, the quantiser above)
 *     from their dequantised values x = fma(q, s, z); then the new token is
 *     appended to its list (a pruned new token is dropped);
 *   - each list keeps its first min(have, need) pages, need = ceil(n / P)
 *     (K8V4) or ceil(n / 2P) (K4V2); new pages come from free-list slots
 *     head + off_u + k (mod F), off_u the exclusive prefix sum over units of
 *     their new pages, a unit's K8V4 pages first; surplus pages are appended
 *     at the tail in (unit, list, page index) order with rev -1, class 0;
 *   - unused slots of the kept pages are cleared; head and tail advance by
 *     the new and freed page counts; fwd / rev / page_cls / unit_hdr follow.
 * ------------------------------------------------------------------------ */
typedef struct dkv_decode_batch {
  int32_t L, R, Hq, Hkv, D;  /* as dkv_batch; D = 128 */
  int32_t cap;               /* positions reserved per request; a multiple of 16 */
  int64_t unit_base;         /* global id of unit 0 of this call */
  const void *k_new;         /* bf16 [L][R][Hkv][128]: each request's new token (16-byte aligned) */
  const void *v_new;         /* bf16 [L][R][Hkv][128] */
  const float *sig_sum;      /* fp32 [L][R * cap][Hq] (16-byte aligned) */
  const int32_t *sig_cnt;    /* int32 [R * cap]: scores summed for each position */
  const int32_t *ctx_lens;   /* int32 [R]: positions 0 .. ctx-1 are held; device memory */
  const int32_t *new_lens;   /* int32 [R]: 0 or 1 new token at position ctx */
  uint8_t *classes;          /* in/out uint8 [L][R * cap][Hkv] (16-byte aligned): DKV_CLASS_* of
                                positions < ctx (+ the new one after the step); other bytes are
                                not read except the new position's, which the step overwrites */
  int32_t *slot_of;          /* in/out int32 [L][R * cap][Hkv]: slot of each held token in its
                                class list, -1 when pruned; built by dkv_decode_index and
                                maintained by dkv_decode_step */
  int32_t window;            /* W >= 0: the recent window, positions [N - W, N) after the step
                                (the review's Algorithm 1 keeps the W most recent tokens at high
                                precision).  The new token enters as K8V4 when W >= 1 (and is
                                classified when W = 0); held tokens in the window keep their class */
  int32_t mode;              /* 0: every older held token is re-scored (the semantics above);
                                1: only the token the new one pushes out of the window, position
                                ctx - W, is classified, once (Algorithm 1's candidate) */
} dkv_decode_batch;

/* Workspace bytes of dkv_decode_step for this shape (host only). */
int32_t dkv_decode_workspace_size(const dkv_decode_batch *b, size_t *bytes);

/* Derive classes and slot_of of positions 0 .. ctx_lens[r]-1 from the pages
 * and tables (after a prefill, or to rebuild them).  Reads the shape,
 * ctx_lens, the tables and the pages; k_new, v_new, sig_sum, sig_cnt and
 * new_lens are not used (may be NULL).  Every byte of classes
 * and every entry of slot_of is first reset (0 and -1), then each used slot
 * of each unit's lists writes its position's class and slot.  A position or
 * page id out of range in the pages is reported as DKV_E_INTERNAL in the
 * status word.  Asynchronous; allocates nothing. */
int32_t dkv_decode_index(const dkv_decode_batch *b, const dkv_pool *pool, const dkv_tables *t,
                         void *stream);

/* One generation step (semantics above), asynchronous.  workspace: device,
 * 256-byte aligned, >= dkv_decode_workspace_size bytes, scratch.  The caller
 * advances ctx_lens by new_lens after a successful step.  A bad shape, cap
 * not a multiple of 16, window < 0 or mode not 0 or 1 is DKV_E_INVAL before
 * anything is enqueued.  Device-side errors
 * (read with dkv_get_status): DKV_E_LENS (ctx + new > cap, new not 0 or 1, a
 * list needing more than pmax pages), DKV_E_RANGE (a kept new token with a
 * non-finite value or one above 65504), DKV_E_NOMEM (new pages > free
 * pages), DKV_E_TIMEOUT (scan wait), DKV_E_INTERNAL (classes, headers,
 * slot_of or pages contradict one another).  On LENS, RANGE, NOMEM and
 * TIMEOUT, and on INTERNAL found before any page is touched, the step
 * changes nothing (classes restored); INTERNAL found while moving slots
 * leaves the state undefined.  With dkv_params.profiler the five intervals
 * are: counter reset, reclassification (or the candidate kernel in mode 1),
 * page scan, apply, requantisation of the demoted tokens. */
int32_t dkv_decode_step(const dkv_decode_batch *b, const dkv_params *p, const dkv_pool *pool,
                        const dkv_tables *t, void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Decode attention over the unified pages.
 *
 * DiffKV (arXiv 2412.03131), Figure 7 and section 6.1: the generation step's
 * attention reads the mixed-precision unified pages.  The pages do not print
 * that kernel; this is plain scaled dot-product attention.  For query head q
 * of request r in layer l (unit (l, r, q / G), G = Hq / Hkv) the attended
 * tokens are every used slot of the unit's high- and low-class lists (the
 * pool's bit-width scheme: K8V4/K4V2, K8V2/K4V1 or K4V8/K2V4), with K and V
 * the dequantised values fma(code, scale, zero) that dkv_dequant_page gives,
 * plus the step's new token (its bf16 K and V, position ctx_lens[r]) when
 * k_new is given and new_lens[r] = 1:
 *   out = sum_t p_t v_t,   p = softmax_t(scale * (q . k_t)).
 * An empty attended set gives a zero output.  With sig_sum given, each
 * attended held token's significance row receives its probability
 * (sig_sum[l][r * cap + pos][q] += p_t) and the new token's row is set to
 * its p; this is the score whose average decides the classes (Pith review,
 * "What carries the argument").  Counts (sig_cnt) are the caller's: +1 for
 * every held position, 1 for the new token.
 * Computed in fp32 (logits from the codes: scale_k (q . c) + zero_k (sum q)).
 * ------------------------------------------------------------------------ */
typedef struct dkv_attn_batch {
  int32_t L, R, Hq, Hkv;     /* the tables' shape, as in dkv_decode_batch; 1 <= Hq / Hkv <= 8 */
  int32_t cap;               /* positions per request (sig_sum rows); ctx + new <= cap */
  int32_t layer0, n_layers;  /* attend layers [layer0, layer0 + n_layers) of the tables */
  const void *q;             /* bf16 [n_layers][R][Hq][128], 16-byte aligned */
  const void *k_new;         /* bf16 [n_layers][R][Hkv][128] or NULL (no new token), 16-byte aligned */
  const void *v_new;         /* bf16, as k_new (NULL exactly when k_new is) */
  const int32_t *new_lens;   /* int32 [R], 0 or 1 (read only with k_new) */
  const int32_t *ctx_lens;   /* int32 [R]: tokens held before the step (the new token's position) */
  float scale;               /* softmax scale, finite */
  float *out;                /* out fp32 [n_layers][R][Hq][128] */
  float *sig_sum;            /* NULL, or in/out fp32 [L][R * cap][Hq] */
} dkv_attn_batch;

/* Decode attention (above), asynchronous; allocates nothing.  The pool and
 * tables are read only.  Synchronous DKV_E_INVAL: a bad shape or pointer,
 * G outside 1..8, or a shape whose per-block shared memory does not fit 220 KB
 * (218 KB for G above 4) even with a cluster of 8 blocks per unit (a block
 * holds 2 page buffers of 216 P bytes per warp, 6 warps for G <= 4 and 8 above,
 * plus its share of the unit's logits and positions, (cap + 1) (4 G + 4) / S
 * bytes; S is the smallest cluster that fits, preferring two blocks per SM).
 * Device-side errors (pool status word): DKV_E_LENS (a new token at ctx >= cap:
 * attended without it), DKV_E_INTERNAL (a unit header, page id or stored
 * position that contradicts the tables: that unit or token is left out). */
int32_t dkv_decode_attention(const dkv_attn_batch *b, const dkv_pool *pool, const dkv_tables *t, void *stream);

/* ------------------------------------------------------------------------
 * Prefill attention that produces the significance inputs of compaction.
 *
 * DiffKV (arXiv 2412.03131), Pith review, "What carries the argument": a
 * token's significance is the average attention it receives from the tokens
 * after it; Referee Report, major comment 2: the average is over the N - i
 * scores token i receives.  For every layer, request and query head q (KV head
 * q / G), query i attends causally over keys 0 .. i of its request:
 *   out_i = sum_{j <= i} p(i, j) v_j,   p(i, .) = softmax_j(scale * q_i . k_j),
 * and the call writes sig_sum[l][t(j)][q] = sum_{i >= j} p(i, j) and
 * sig_cnt[t(j)] = N - j: the inputs dkv_compact classifies.  Computed on the
 * tensor cores (tcgen05): bf16 x bf16 products exact, fp32 accumulation; the
 * significance sums add the fp32 probabilities, the outputs use p rounded to
 * bf16 for the P V product.
 * ------------------------------------------------------------------------ */
typedef struct dkv_prefill_batch {
  int32_t L, R, Hq, Hkv;     /* 1 <= Hq / Hkv */
  int32_t max_len;           /* >= every lens[r] */
  int32_t reserved;
  int64_t T;                 /* sum of lens */
  const void *q;             /* bf16 [L][T][Hq][128], 16-byte aligned */
  const void *k;             /* bf16 [L][T][Hkv][128], 16-byte aligned (the dkv_batch layout) */
  const void *v;             /* bf16 [L][T][Hkv][128], 16-byte aligned; |v| <= 65504 */
  const int32_t *lens;       /* int32 [R] */
  float scale;               /* softmax scale, finite */
  float *out;                /* out fp32 [L][T][Hq][128] */
  float *sig_sum;            /* out fp32 [L][T][Hq] (overwritten) */
  int32_t *sig_cnt;          /* out int32 [T] (overwritten) */
} dkv_prefill_batch;

/* Prefill attention (above), asynchronous; allocates nothing.  Synchronous
 * DKV_E_INVAL for a bad shape or pointer.  Device-side (pool status word;
 * only `pool->status` is used): DKV_E_LENS when a length is negative or above
 * max_len, or the lengths do not add up to T; every block checks all of them
 * before it reads or writes anything, so out and sig_cnt are then left as
 * they were (sig_sum is zeroed first, in any case).  Significance sums are
 * added across query tiles by fp32 atomics, so their last bits depend on the
 * order. */
int32_t dkv_prefill_attention(const dkv_prefill_batch *b, const dkv_pool *pool, void *stream);

/* ------------------------------------------------------------------------
 * Attention of several new tokens a request over the unified pages: drafted
 * tokens to verify, the next turn of a conversation, a chunk of a prompt.
 *
 * dkv_decode_attention's definition for new_lens[r] >= 0 query tokens instead
 * of one.  The batch's T = sum(new_lens) tokens are packed request after
 * request; token i of request r stands at position ctx_lens[r] + i.  For
 * query head q of that token (unit (l, r, q / G)) the attended tokens are
 * every used slot of the unit's high- and low-class lists, with K and V the
 * dequantised values fma(code, scale, zero), and, when k_new is given, the
 * request's new tokens 0 .. i (bf16 K and V):
 *   x_t = scale * (q . k_t),  out = sum_t exp(x_t - lse) v_t,
 *   lse = log sum_t exp(x_t).
 * A row that attends nothing gives a zero output and lse = -inf.  The pages
 * are not changed: tokens that are kept enter the cache through
 * dkv_decode_step.
 *
 * Precision: logits, references, sums, outputs in progress and the
 * significance are fp32, the products' operands 16 bits.  Of K the codes enter
 * exactly; a query value keeps its 8 bits down to 2^-19 of its row's largest;
 * held V is rounded to fp16 (and held at +-65504), the weights against it to
 * fp16 (none below 2^-32 of the row's largest); weights against the new tokens
 * are the sum of two bf16 values; out is bf16.  dkv_decode_attention keeps
 * weights and V to more bits and writes fp32.
 * Range: queries and new keys of any finite size; a row depends on no other
 * row's query.  Logits count as fp32 does: beyond 2^24 the largest alone is
 * left, and one that passes fp32's range spoils its row.  New values up to
 * 2^100.  A query that is not finite spoils its own row alone.
 *
 * dkv_extend_significance adds to sig_sum what dkv_decode_attention's
 * significance update adds, for the first acc_lens[r] new tokens of each
 * request (drafts that were rejected leave no trace): with p(i, t) =
 * exp(x_t - lse) recomputed from the lse of dkv_extend_attention,
 *   sig_sum[l][r * cap + pos(t)][q] += sum_{i < acc} p(i, t)   held token t,
 *   sig_sum[l][r * cap + ctx + j][q] = sum_{j <= i < acc} p(i, j)  new j < acc
 * (the new tokens' rows when k_new is given).  Each sum is formed by one
 * thread in a fixed order, so equal inputs give equal bits.  Counts (sig_cnt)
 * are the caller's: + acc_lens[r] for every held position, acc_lens[r] - j
 * for new token j.  lse rounded to fp32 is all that is left of a row: where
 * |lse| passes 2^20 its p are 0 or 1 by that rounding; p below 2^-126 are 0.
 * ------------------------------------------------------------------------ */
typedef struct dkv_extend_batch {
  int32_t L, R, Hq, Hkv;     /* the tables' shape, as in dkv_decode_batch; 1 <= Hq / Hkv <= 128 */
  int32_t cap;               /* positions per request (sig_sum rows); ctx + new <= cap */
  int32_t layer0, n_layers;  /* attend layers [layer0, layer0 + n_layers) of the tables */
  int32_t max_new;           /* >= every new_lens[r]; the work is divided by it, so that exact is fastest */
  int64_t T;                 /* sum of new_lens */
  const void *q;             /* bf16 [n_layers][T][Hq][128], 16-byte aligned */
  const void *k_new;         /* bf16 [n_layers][T][Hkv][128], finite, or NULL; 16-byte aligned */
  const void *v_new;         /* bf16, as k_new (NULL exactly when k_new is; not read by
                                dkv_extend_significance) */
  const int32_t *new_lens;   /* int32 [R], device */
  const int32_t *ctx_lens;   /* int32 [R], device */
  float scale;               /* softmax scale, finite */
  void *out;                 /* out bf16 [n_layers][T][Hq][128], 16-byte aligned (attention only) */
  float *lse;                /* fp32 [n_layers][T][Hq], natural log: out of the attention (may be
                                NULL there), in of the significance */
} dkv_extend_batch;

/* Workspace bytes of dkv_extend_attention (host only; may be 0). */
int32_t dkv_extend_workspace_size(const dkv_extend_batch *b, const dkv_pool *pool, const dkv_tables *t,
                                  size_t *bytes);

/* Attention of several new tokens (above), asynchronous; allocates nothing.
 * workspace: device, 256-byte aligned, >= dkv_extend_workspace_size bytes
 * (NULL when that is 0), scratch: calls that may overlap on the GPU (two
 * streams, two captured graphs) need one each.  The size grows with T, and
 * not otherwise in one order: ask for each shape.  Pool and tables are read
 * only.  T = 0, R = 0 or n_layers = 0 is DKV_OK with nothing launched (the
 * lengths are not looked at).  Synchronous DKV_E_INVAL: a bad shape, pointer
 * or workspace.
 * Device-side (pool status word): DKV_E_LENS when a new_lens[r] is outside
 * [0, max_new], ctx_lens[r] + new_lens[r] is outside [0, cap] or the lengths do not add up to T:
 * nothing is written then; DKV_E_RANGE for a new K or V value that is not
 * finite (taken as 0); DKV_E_INTERNAL for a unit header or page id that
 * contradicts the tables (that unit's lists or that page's tokens are left out);
 * DKV_E_TIMEOUT when a bounded wait gave up (outputs undefined). */
int32_t dkv_extend_attention(const dkv_extend_batch *b, const dkv_pool *pool, const dkv_tables *t,
                             void *workspace, size_t workspace_bytes, void *stream);

/* Significance of the accepted new tokens (above), asynchronous; needs no
 * workspace and allocates nothing.  acc_lens: int32 [R], device, 0 <= acc <=
 * new; sig_sum: in/out fp32 [L][R * cap][Hq], 16-byte aligned.  A row whose
 * lse is -inf adds nothing.  Errors as dkv_extend_attention; DKV_E_LENS also
 * for an acc_lens[r] outside [0, new_lens[r]], DKV_E_INTERNAL also for a
 * stored position outside [0, ctx_lens[r]) (that token is left out). */
int32_t dkv_extend_significance(const dkv_extend_batch *b, const int32_t *acc_lens, float *sig_sum,
                                const dkv_pool *pool, const dkv_tables *t, void *stream);

/* ------------------------------------------------------------------------
 * A prompt that arrives in chunks.  Its tokens can be classified when the last
 * chunk is there: the score of a token averages over every token after it.
 * Until then the earlier chunks' K and V are held as they are, in bf16 pages
 * of their own, and each chunk attends to them and gives them significance;
 * after the last one sig_sum holds what one dkv_prefill_attention over the
 * whole prompt would have left, and dkv_compact takes the prompt over.
 *
 * Position p of request r lies in slot p mod B of page table[r][p / B], the
 * same page in every layer.  A page may stand in several requests' rows (a
 * shared prefix); a page that receives new tokens must stand in one.  Where a
 * request's pages follow one another, their K and V rows are dkv_batch's k and
 * v of one request and layer as they lie.
 *
 * dkv_chunk_attention: the batch's T = sum(new_lens) tokens are packed request
 * after request; token i of request r stands at position ctx_lens[r] + i.
 * With k_new given, the new tokens' K and V are first stored in their places.
 * Then, for query head q of that token (KV head q / G, G = Hq / Hkv), over the
 * positions t = 0 .. ctx_lens[r] + i:
 *   x_t = scale * (q . k_t),  out = sum_t exp(x_t - lse) v_t,
 *   lse = log sum_t exp(x_t).
 * new_lens[r] = 1 is a generation step over the unquantised cache.
 *
 * Precision: products of bf16 values added in fp32; references, sums and
 * outputs in progress are fp32; out is bf16.  A request's new tokens
 * are worked on 2 (128 / G) at a time; their weights enter the second product
 * rounded to bf16, and where only 128 / G or fewer are left (short chunks,
 * single tokens), as the sum of two bf16 values.
 * Range: queries and keys of any finite size; a query that is not finite, or a
 * logit that passes fp32's range, spoils its row; values up to 2^100, or
 * 2^120 / cap where that is less.  Slots of a page behind a request's
 * last token may hold anything; the tokens before it are finite (one that is
 * not may spoil the rows before it too).
 *
 * dkv_chunk_significance adds what those rows give: with p(i, t) =
 * exp(x_t - lse) recomputed from the lse of dkv_chunk_attention,
 *   sig_sum[l][r * cap + t][q] += sum_i p(i, t)         t < ctx_lens[r],
 *   sig_sum[l][r * cap + ctx + j][q] = sum_{i >= j} p(i, ctx + j)   new j.
 * Each sum is formed in a fixed order: equal inputs give equal bits.  Counts
 * (sig_cnt) are the caller's: + new_lens[r] for every held position,
 * new_lens[r] - j for new token j.  A row whose lse is -inf adds nothing; p
 * below 2^-126 are 0.  Queries are finite here: one that is not spoils its
 * head's sums.
 * ------------------------------------------------------------------------ */
typedef struct dkv_chunk_pages {
  int64_t F;                 /* pages; 1 <= F */
  int32_t B;                 /* tokens a page: 8, 16, 32, 64 or 128 */
  int32_t tmax;              /* entries of a request's row of the table; tmax * B >= cap */
  void *k, *v;               /* bf16 [L][F][B][Hkv][128], 16-byte aligned */
  const int32_t *table;      /* int32 [R][tmax], device; entries behind a request's last token are not read */
} dkv_chunk_pages;

typedef struct dkv_chunk_batch {
  int32_t L, R, Hq, Hkv;     /* the pages' layers, requests, heads; L, R <= 65535, Hq <= 128.  L F B, R tmax,
                                n_layers T and n_layers R Hkv stay below 2^31 */
  int32_t cap;               /* positions per request (sig_sum rows); ctx + new <= cap */
  int32_t layer0, n_layers;  /* attend layers [layer0, layer0 + n_layers) of the pages */
  int32_t max_new;           /* >= every new_lens[r]; exact is fastest.  A chunk's work, n G / 256 * (cap / 128 + 4)
                                with n = min(max_new, T), has to stay below 2^31: split a larger one */
  int64_t T;                 /* sum of new_lens */
  int64_t q_stride, kv_stride; /* elements from one token's row of q (of k_new and v_new) to the next, a
                                multiple of 8, at most 2^32; 0: Hq * 128 (Hkv * 128).  Layers follow T rows later */
  const void *q;             /* bf16 [n_layers][T][Hq][128], 16-byte aligned */
  const void *k_new;         /* bf16 [n_layers][T][Hkv][128], 16-byte aligned, or NULL: the pages hold the new
                                tokens already (not read by dkv_chunk_significance) */
  const void *v_new;         /* bf16, as k_new (NULL exactly when k_new is) */
  const int32_t *new_lens;   /* int32 [R], device */
  const int32_t *ctx_lens;   /* int32 [R], device */
  float scale;               /* softmax scale, finite, > 0 */
  void *out;                 /* out bf16 [n_layers][T][Hq][128], 16-byte aligned (attention only) */
  float *lse;                /* fp32 [n_layers][T][Hq], natural log: out of the attention (may be
                                NULL there), in of the significance */
} dkv_chunk_batch;

/* Workspace bytes of dkv_chunk_attention (host only). */
int32_t dkv_chunk_workspace_size(const dkv_chunk_batch *b, const dkv_chunk_pages *pages, size_t *bytes);

/* Chunk attention (above), asynchronous; allocates nothing.  workspace:
 * device, 256-byte aligned, >= dkv_chunk_workspace_size bytes, scratch: calls
 * that may overlap on the GPU (two streams, two captured graphs) need one
 * each.  Of the pool only `status` is used.  T = 0, R = 0 or n_layers = 0 is
 * DKV_OK with nothing launched (the lengths are not looked at).  Synchronous
 * DKV_E_INVAL: a bad shape, pointer or workspace.  Device-side: DKV_E_LENS
 * when a new_lens[r] is outside [0, max_new], ctx_lens[r] + new_lens[r] is
 * outside [0, cap] or the lengths do not add up to T: nothing is written then;
 * DKV_E_RANGE for a new K or V value that is not finite (stored and taken as
 * 0); DKV_E_INTERNAL for a page id outside [0, F): nothing is stored for it
 * and page 0 is read in its place, which leaves that request's outputs without
 * meaning and the others as they are; DKV_E_TIMEOUT when a bounded wait gave
 * up (outputs undefined). */
int32_t dkv_chunk_attention(const dkv_chunk_batch *b, const dkv_chunk_pages *pages, const dkv_pool *pool,
                            void *workspace, size_t workspace_bytes, void *stream);

/* Significance of those rows (above), asynchronous; needs no workspace and
 * allocates nothing.  K is read from the pages, the new tokens' too.  sig_sum:
 * in/out fp32 [L][R * cap][Hq], 16-byte aligned.  Errors as
 * dkv_chunk_attention; a page id outside [0, F) leaves the sums of that page's
 * tokens without meaning. */
int32_t dkv_chunk_significance(const dkv_chunk_batch *b, const dkv_chunk_pages *pages, float *sig_sum,
                               const dkv_pool *pool, void *stream);

/* ------------------------------------------------------------------------
 * Page operations of a pool that serves many requests: a request is forked,
 * requests leave, a fragmented pool is packed.  All three are all-or-nothing:
 * on a device-side error (status word) nothing has changed.  (One exception:
 * the entries of the free list are trusted; an id outside [0, F) in it is
 * reported as DKV_E_INTERNAL by the fork that draws it, which leaves that page
 * out.)  n = 0 is DKV_OK with nothing launched.
 *
 * They share one workspace (device, 256-byte aligned, at least
 * dkv_page_ops_workspace_size bytes for the tables' U units, scratch).
 * Requests are named by device lists; "list units" of requests q[0..n) are
 * the units (l, q[k], h) in the order (l, k, h), so a call over L layers
 * equals L one-layer calls (unit_base and table offsets as in dkv_compact).
 * ------------------------------------------------------------------------ */
int32_t dkv_page_ops_workspace_size(const dkv_pool *pool, int64_t U, size_t *bytes);

typedef struct dkv_fork_batch {
  int32_t L, R, Hq, Hkv;     /* the tables' shape; R <= 65535; Hq is read with sig_sum only */
  int32_t cap;               /* positions per request; a multiple of 16 */
  int32_t n;                 /* forks */
  int64_t unit_base;         /* global id of unit 0 of the tables */
  const int32_t *src, *dst;  /* int32 [n], device: request dst[k] becomes a copy of src[k] */
  const int32_t *ctx_lens;   /* int32 [R], device: positions held (read for the rows below; NULL
                                exactly when all four are) */
  uint8_t *classes;          /* NULL or in/out [L][R * cap][Hkv], as in dkv_decode_batch */
  int32_t *slot_of;          /* NULL or in/out [L][R * cap][Hkv] */
  float *sig_sum;            /* NULL or in/out [L][R * cap][Hq] */
  int32_t *sig_cnt;          /* NULL or in/out [R * cap] */
} dkv_fork_batch;

/* Fork requests, asynchronous.  A page has one owner and a generation step
 * moves and requantises tokens in place, so a fork copies: the d_v pages of
 * source list unit v are copied to the pages of free-list slots
 * [head + off_v, head + off_v + d_v) mod F (off_v the exclusive prefix sum of
 * d_v over the list units), in their order; the destination's forward row,
 * header, rev_unit, rev_idx and page_cls follow, and head advances by the
 * sum.  Of each given row array the rows of positions [0, ctx_lens[src]) are
 * copied to the destination request (16-byte aligned arrays); later rows stay
 * as they were, and the caller sets ctx_lens[dst].  One source may be forked several times.  Device-side
 * errors: DKV_E_NOMEM (pages), DKV_E_INTERNAL (a request index out of range, a destination named
 * twice, that is also a source, or whose units still hold pages; headers or page ids that contradict the
 * tables), DKV_E_LENS (ctx_lens[src] outside [0, cap]). */
int32_t dkv_fork(const dkv_fork_batch *b, const dkv_pool *pool, const dkv_tables *t, void *workspace,
                 size_t workspace_bytes, void *stream);

typedef struct dkv_release_batch {
  int32_t L, R, Hkv;         /* the tables' shape; R <= 65535 */
  int32_t n;                 /* requests that leave */
  int64_t unit_base;         /* global id of unit 0 of the tables */
  const int32_t *reqs;       /* int32 [n], device */
} dkv_release_batch;

/* Release requests, asynchronous: the pages of the list units are appended
 * at the free list's tail in (list unit, page index) order with rev_unit =
 * rev_idx = -1 and page_cls 0, their forward rows become -1 and their headers
 * 0, and tail advances by the count.  Page contents, classes, slots and
 * significance rows stay as they were.  A request without pages releases
 * none.  Device-side: DKV_E_INTERNAL (a request out of range or named twice;
 * a header, page id or reverse entry that contradicts the tables). */
int32_t dkv_release(const dkv_release_batch *b, const dkv_pool *pool, const dkv_tables *t, void *workspace,
                    size_t workspace_bytes, void *stream);

/* Pack the pool, asynchronous: with n = F - (tail - head) pages live, the
 * live pages with ids >= n move into the free ids below n, ascending into
 * ascending, so that the live pages are exactly [0, n).  Contents, rev_unit,
 * rev_idx, page_cls and the owners' forward entries follow.  The free list becomes
 * the ids [n, F) in order, at slots of the same numbers: head advances to the
 * next value that is n mod F and tail = head + F - n (both stay monotone),
 * so the memory of [n, F) can be handed back.  `t` holds all U units that
 * own pages of the pool (global ids [unit_base, unit_base + U)).
 * Device-side: DKV_E_INTERNAL (page classes, reverse entries, forward rows
 * and cursors contradict one another). */
int32_t dkv_defrag(const dkv_pool *pool, const dkv_tables *t, int64_t U, int64_t unit_base, void *workspace,
                   size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Eviction by accumulated attention.  The classes come from thresholds
 * alpha / N, so they do not bound what a unit holds; when a pool runs out, or a
 * request has a budget, the tokens that received the least attention go.
 *
 * A unit (l, r, h) of a request with budgets[r] >= 0 keeps of the tokens it
 * holds (classes != 0, position < ctx_lens[r]) those at the first `sinks`
 * positions and the last `window` positions [ctx - window, ctx), and of the
 * others the budgets[r] - (those) with the largest weight
 *   w(p) = max over the group's query heads of sig_sum[l][r * cap + p][q],
 * divided by sig_cnt[r * cap + p] (in fp32) where sig_cnt is given; of equal
 * weights the lowest position stays first; a weight that is NaN goes first.
 * A negative budget leaves the request alone, as does one that its units do
 * not pass.
 *
 * Lists close as in dkv_decode_step: with `keep` survivors of a list, those in
 * slots >= keep move, in ascending slot order, into the holes below keep, in
 * ascending order (bytes copied); each list keeps its first need = ceil(keep /
 * P) (low: / 2P) pages and the others are appended at the free list's tail in
 * (unit, list, page index) order with rev -1 and class 0; the vacated slots of
 * the kept pages are cleared; classes (0) and slot_of (-1) of the evicted,
 * slot_of of the moved, fwd, rev_idx, unit_hdr and the tail follow.  Freed pages
 * keep their contents.
 * ------------------------------------------------------------------------ */
typedef struct dkv_evict_batch {
  int32_t L, R, Hq, Hkv;     /* the tables' shape; R <= 65535 */
  int32_t cap;               /* positions per request, as in dkv_decode_batch; a multiple of 16, <= 2^18 */
  int32_t sinks, window;     /* >= 0 */
  int32_t reserved;          /* must be 0 */
  int64_t unit_base;         /* global id of unit 0 of the tables */
  const int32_t *budgets;    /* int32 [R], device: most tokens a unit of the request keeps; < 0: all */
  const int32_t *ctx_lens;   /* int32 [R], device: positions held */
  const float *sig_sum;      /* fp32 [L][R * cap][Hq], 16-byte aligned */
  const int32_t *sig_cnt;    /* int32 [R * cap], or NULL: the sums themselves are compared */
  uint8_t *classes;          /* in/out uint8 [L][R * cap][Hkv], as in dkv_decode_batch */
  int32_t *slot_of;          /* in/out int32 [L][R * cap][Hkv] */
} dkv_evict_batch;

/* Workspace bytes of dkv_evict (host only). */
int32_t dkv_evict_workspace_size(const dkv_evict_batch *b, const dkv_pool *pool, const dkv_tables *t, size_t *bytes);

/* Evict (above), asynchronous; allocates nothing.  workspace: device, 256-byte
 * aligned, >= dkv_evict_workspace_size bytes, scratch: calls on different pools
 * that may overlap on the GPU need one each (calls on one pool are ordered by
 * the caller, as all that change it).  Synchronous
 * DKV_E_INVAL: a bad shape, pointer or workspace.  All-or-nothing: on a
 * device-side error (status word) nothing has changed: DKV_E_LENS (a
 * ctx_lens[r] outside [0, cap]), DKV_E_INTERNAL (headers, classes, slots, page
 * ids, reverse entries or cursors that contradict one another).  The position
 * that a moved token's page slot holds is not compared with slot_of before: one
 * outside [0, ctx_lens[r]) is reported (DKV_E_INTERNAL) while the token is moved
 * and no slot_of is written for it.  A unit that its budget leaves as it is is
 * not looked into beyond its header. */
int32_t dkv_evict(const dkv_evict_batch *b, const dkv_pool *pool, const dkv_tables *t, void *workspace,
                  size_t workspace_bytes, void *stream);

/* Synchronise `stream`, return the pool's device status word (DKV_OK or the
 * first device-side error since the last read) and clear it. */
int32_t dkv_get_status(const dkv_pool *pool, void *stream);

/* Per-kernel timing of dkv_compact with CUDA events.  A profiler holds
 * events for up to max_calls calls; every dkv_compact given it (through
 * dkv_params.profiler) records its kernels into the next call slot.
 * dkv_profiler_read synchronises and writes, for each recorded call c and
 * kernel k, ms[c * DKV_PROFILE_KERNELS + k]; it returns the number of calls
 * recorded and starts a new recording. */
#define DKV_PROFILE_KERNELS 5 /* prep, classify, page scan, quantise+scatter, commit */
int32_t dkv_profiler_create(int32_t max_calls, void **profiler);
int32_t dkv_profiler_read(void *profiler, float *ms, int32_t capacity_calls);
int32_t dkv_profiler_destroy(void *profiler);

const char *dkv_status_string(int32_t code);

/* Text of the CUDA error behind the calling thread's last DKV_E_CUDA
 * ("no error" if there was none). */
const char *dkv_last_cuda_error(void);
int32_t dkv_version(void);

/* How the library was built: DKV_BUILD_CHECKED is set in the bounds-checked
 * build (lib/libdkv_checked.so, compiled with -DDKV_CHECKED).  There every
 * page id, free-list index and page-list index that a kernel takes from the
 * tables is checked before it is used; a value outside its range records
 * DKV_E_INTERNAL in the pool status and the access is skipped (the kernel
 * does not trap).  The pool contents after such an error are unspecified.
 * The normal build keeps the checks that cost nothing measurable (page ids
 * read from the forward table or the free list before a page is touched). */
#define DKV_BUILD_CHECKED 1
int32_t dkv_build_flags(void);

#ifdef __cplusplus
}
#endif
#endif /* DKV_H */
