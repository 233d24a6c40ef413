// tensor_ops.cuh -- mbarrier, tensor-memory and tcgen05 helpers, and the
// conversion of page codes to 16-bit operands, shared by the kernels of the
// multi-token attention (extend.cu, extend_sig.cu).
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dkv_internal.cuh"

namespace dkv {
namespace tc {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr uint32_t kBox = 128 * 128;      // one operand box: 128 rows of 64 16-bit values (16 KB)
constexpr uint32_t kTileBytes = 2 * kBox;  // 128 rows of 128
constexpr uint64_t kWaitNs = 1000000000ull;
constexpr uint32_t kWaitPolls = 1u << 26;

__device__ __forceinline__ uint32_t saddr(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(saddr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.shared::cta.b64 st, [%0]; }" ::"r"(saddr(bar)) : "memory");
}

// Arrive and expect `bytes` of copies.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("{ .reg .b64 st; mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1; }" ::"r"(saddr(bar)),
               "r"(bytes)
               : "memory");
}

// Bulk copy of n bytes (a multiple of 16, as both addresses) to shared memory.
__device__ __forceinline__ void copy_bulk(void *dst, const void *src, uint32_t n, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(saddr(dst)),
               "l"(src), "r"(n), "r"(saddr(bar))
               : "memory");
}

// Four bytes to shared memory, asynchronously; arrive_async arrives when this
// thread's copies so far have landed.
__device__ __forceinline__ void copy_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(saddr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void arrive_async(uint64_t *bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t addr, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
      : "=r"(done)
      : "r"(addr), "r"(parity)
      : "memory");
  return done != 0;
}

// Bounded wait for the phase of the given parity: false after about kWaitNs,
// or as soon as *abort (when given) is set by another thread.  The loop is out
// of line: the kernels have a dozen waits, and their code has to fit the
// instruction cache.
static __device__ __noinline__ bool mbar_wait_loop(uint32_t addr, uint32_t parity, const volatile int32_t *abort) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try(addr, parity)) return true;
    if ((i & 63) == 63) {
      if (abort && *abort) return false;
      const uint64_t t = global_ns();
      if (t0 == 0) t0 = t;
      else if (t - t0 > kWaitNs) return false;
    }
  }
  return false;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, const volatile int32_t *abort) {
  const uint32_t addr = saddr(bar);
  return mbar_try(addr, parity) || mbar_wait_loop(addr, parity, abort);
}

// A wait that gives up records the timeout once and makes everyone stop.
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, volatile int32_t *abort,
                                              int32_t *status) {
  if (mbar_wait(bar, parity, abort)) return true;
  if (!*abort) {
    *abort = 1;
    set_error(status, DKV_E_TIMEOUT);
  }
  return false;
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// generic writes to shared memory become visible to the tensor cores
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Shared-memory matrix descriptor of a 128-byte-swizzled operand: start
// address, leading and stride byte offsets (16-byte units), descriptor
// version 1, swizzle mode 2 (128 bytes); tiles are 1024-byte aligned.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3fffu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3fffu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3fffu) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B both fp16
// or both bf16, A K-major, B K-major or MN-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int M, int N, bool b_mn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

constexpr uint32_t kAMn = 1u << 15;  // ... with A MN-major

// D[tmem] (+)= A[smem] B[smem].
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

// D[tmem] (+)= A[tmem] B[smem]: A's rows are lanes, two 16-bit values a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{ .reg .pred p; setp.ne.b32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

// The barrier receives one arrival when every MMA this thread issued so far
// has completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar))
               : "memory");
}

__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols) {  // one warp
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(saddr(dst)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {  // the same warp
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}

// 32 consecutive 32-bit columns of this thread's lane (no wait).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t *r) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait4(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]) : : "memory");
}
// Loads done: the registers they filled pass through, so that nothing reads
// them earlier.
__device__ __forceinline__ void tmem_wait32(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
        "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
        "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
        "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :
      : "memory");
}
__device__ __forceinline__ void tmem_wait16(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x by the special-function unit (relative error about 2^-22; results below
// 2^-126 flush to zero).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs: one instruction, each half rounded like the scalar one.
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t r, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(r));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float f2_sum(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Additions to global memory without their results (16-byte aligned for four).
__device__ __forceinline__ void red_add(float *p, float x) {
  asm volatile("red.global.add.f32 [%0], %1;" ::"l"(p), "f"(x) : "memory");
}
__device__ __forceinline__ void red_add4(float *p, float x, float y, float z, float w) {
  asm volatile("red.global.v4.f32.add [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(x), "f"(y), "f"(z), "f"(w) : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Two fp32 values rounded to nearest even into one register, `lo` in the low half.
__device__ __forceinline__ uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of(uint64_t a) {
  float lo, hi;
  f2_unpack(a, lo, hi);
  return f16x2_rn(lo, hi);
}
__device__ __forceinline__ uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// What bf16x2_rn(lo, hi) = w left of the two values, as bf16.
__device__ __forceinline__ uint32_t bf16x2_rest(float lo, float hi, uint32_t w) {
  return bf16x2_rn(lo - bf16_lo(w), hi - bf16_hi(w));
}
__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

__device__ __forceinline__ uint32_t h2u(__half2 x) { return *reinterpret_cast<uint32_t *>(&x); }
__device__ __forceinline__ __half2 u2h(uint32_t x) { return *reinterpret_cast<__half2 *>(&x); }

// ------------------------------------------------------------- page codes --
//
// Operand rows hold their 128 channels in groups of eight, each group in the
// order 0 4 1 5 2 6 3 7: with it the two codes of a 16-bit pair of a 4-bit
// group lie 16 bits apart in the page's own word, and one masked word gives
// a pair.  A code c at bit k of a half under the exponent of 1024 reads as
// 1024 + 2^k c, and one half-precision multiply-add (exact: |result| <= 255)
// makes it c - mid.

// fp16 bits of a value that fp16 holds exactly in its normal range (compile
// time: a conversion in the loop would cost as much as the codes').
__host__ __device__ constexpr uint32_t half_bits(double x) {
  if (x == 0.0) return 0;
  const uint32_t sign = x < 0 ? 0x8000u : 0u;
  double a = x < 0 ? -x : x;
  int e = 15;
  while (a >= 2.0) a /= 2.0, ++e;
  while (a < 1.0) a *= 2.0, --e;
  return sign | static_cast<uint32_t>(e) << 10 | static_cast<uint32_t>((a - 1.0) * 1024.0);
}
__host__ __device__ constexpr uint32_t half_pair(double lo, double hi) { return half_bits(lo) | half_bits(hi) << 16; }

// Codes of one group (8 channels, W bits each, in `w0`, for W = 8 also `w1`)
// as four fp16 pairs, minus MID.
template <int W, int MID>
__device__ __forceinline__ void group_codes(uint32_t w0, uint32_t w1, __half2 (&o)[4]) {
  constexpr uint32_t kExp = 0x64006400u;
  if constexpr (W == 8) {
    constexpr uint32_t b = half_pair(-1024.0 - MID, -1024.0 - MID);
    const uint32_t p01 = __byte_perm(w0, w1, 0x5140), p23 = __byte_perm(w0, w1, 0x7362);
    o[0] = __hadd2(u2h(__byte_perm(p01, kExp, 0x7170)), u2h(b));
    o[1] = __hadd2(u2h(__byte_perm(p01, kExp, 0x7372)), u2h(b));
    o[2] = __hadd2(u2h(__byte_perm(p23, kExp, 0x7170)), u2h(b));
    o[3] = __hadd2(u2h(__byte_perm(p23, kExp, 0x7372)), u2h(b));
  } else if constexpr (W == 4) {
    constexpr uint32_t b0 = half_pair(-1024.0 - MID, -1024.0 - MID), b1 = half_pair(-64.0 - MID, -64.0 - MID);
    constexpr uint32_t q = half_pair(0.0625, 0.0625);
    const uint32_t y = w0 >> 8;
    o[0] = __hadd2(u2h((w0 & 0x000f000fu) | kExp), u2h(b0));
    o[1] = __hfma2(u2h((w0 & 0x00f000f0u) | kExp), u2h(q), u2h(b1));
    o[2] = __hadd2(u2h((y & 0x000f000fu) | kExp), u2h(b0));
    o[3] = __hfma2(u2h((y & 0x00f000f0u) | kExp), u2h(q), u2h(b1));
  } else if constexpr (W == 2) {  // the low 16 bits
    constexpr uint32_t q[4] = {half_pair(1.0, 1.0), half_pair(0.25, 0.25), half_pair(0.0625, 0.0625),
                               half_pair(0.015625, 0.015625)};
    constexpr uint32_t b[4] = {half_pair(-1024.0 - MID, -1024.0 - MID), half_pair(-256.0 - MID, -256.0 - MID),
                               half_pair(-64.0 - MID, -64.0 - MID), half_pair(-16.0 - MID, -16.0 - MID)};
    const uint32_t y = __byte_perm(w0, 0, 0x4140);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = __hfma2(u2h((y & (0x00030003u << (2 * k))) | kExp), u2h(q[k]), u2h(b[k]));
  } else {  // W == 1: the low 8 bits
    constexpr uint32_t q[4] = {half_pair(1.0, 0.0625), half_pair(0.5, 0.03125), half_pair(0.25, 0.015625),
                               half_pair(0.125, 0.0078125)};
    constexpr uint32_t b[4] = {half_pair(-1024.0 - MID, -64.0 - MID), half_pair(-512.0 - MID, -32.0 - MID),
                               half_pair(-256.0 - MID, -16.0 - MID), half_pair(-128.0 - MID, -8.0 - MID)};
    const uint32_t y = __byte_perm(w0, 0, 0x4040);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      o[k] = __hfma2(u2h((y & ((1u << k) | (0x100000u << k))) | kExp), u2h(q[k]), u2h(b[k]));
  }
}

// Words of group g (0 or 1) of those 16 channels.
template <int W>
__device__ __forceinline__ void group_of(const uint32_t (&x)[4], int g, uint32_t &w0, uint32_t &w1) {
  w1 = 0;
  if constexpr (W == 8) w0 = x[2 * g], w1 = x[2 * g + 1];
  else if constexpr (W == 4) w0 = x[g];
  else if constexpr (W == 2) w0 = x[0] >> (16 * g);
  else w0 = x[0] >> (8 * g);
}

// Channels (2 i, 2 i + 1 ...) of a group in operand order from eight bf16 in
// channel order (four words): pairs (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ void group_bf16(const uint4 &v, uint32_t (&o)[4]) {
  o[0] = __byte_perm(v.x, v.z, 0x5410);
  o[1] = __byte_perm(v.x, v.z, 0x7632);
  o[2] = __byte_perm(v.y, v.w, 0x5410);
  o[3] = __byte_perm(v.y, v.w, 0x7632);
}

// Byte offset of group gi (0 .. 15) of operand row `row` in a 128-row tile
// (two boxes of 64 channels, 128-byte swizzle).
__device__ __forceinline__ uint32_t group_at(int row, int gi) {
  return (gi >> 3) * kBox + row * 128 + (((gi & 7) ^ (row & 7)) << 4);
}

// ------------------------------------------------------------------- units --

// Every length in range and their sum T; `before` gets the tokens of the
// requests before r.  Warp 0 works, every thread of the block calls it.
__device__ __forceinline__ bool lens_valid(const ExtendArgs &a, int32_t r, int64_t &before) {
  __shared__ int64_t before_s;
  __shared__ int32_t ok_s;
  if (threadIdx.x < 32) {
    int64_t b = 0, t = 0;
    int bad = 0;
    for (int32_t i = threadIdx.x; i < a.R; i += 32) {
      const int32_t n = __ldg(a.new_lens + i), c = __ldg(a.ctx_lens + i);
      if (n < 0 || n > a.max_new || c < 0 || static_cast<int64_t>(c) + n > a.cap) bad = 1;
      if (a.acc_lens && (__ldg(a.acc_lens + i) < 0 || __ldg(a.acc_lens + i) > n)) bad = 1;
      t += n;
      if (i < r) b += n;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      b += __shfl_xor_sync(kFull, b, o);
      t += __shfl_xor_sync(kFull, t, o);
      bad |= __shfl_xor_sync(kFull, bad, o);
    }
    if (threadIdx.x == 0) {
      before_s = b;
      ok_s = !bad && t == a.T;
      if (!ok_s) set_error(a.status, DKV_E_LENS);
    }
  }
  __syncthreads();
  before = before_s;
  return ok_s != 0;
}

// Lets k_extend_merge's blocks start while the attention's last ones run (they
// wait for its end: only the launch overlaps).
__device__ __forceinline__ void let_merge_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// The request with the k-th most tokens, held and new (ties: the first one), or k itself when
// there are more requests than that is worth.  Every block asks, all its threads.
constexpr int32_t kOrder = 512;
__device__ __forceinline__ int32_t longest_first(const ExtendArgs &a, int32_t k) {
  __shared__ __align__(16) int32_t len[kOrder];
  __shared__ int32_t pick;
  if (a.R == 1 || a.R > kOrder) return k;
  const int32_t tid = threadIdx.x, n4 = (a.R + 3) / 4;
  if (tid == 0) pick = k;
  for (int32_t i = tid; i < 4 * n4; i += blockDim.x) {
    // lengths that are not valid yet may wrap: any order will do for them
    len[i] = i < a.R ? static_cast<int32_t>(static_cast<uint32_t>(__ldg(a.ctx_lens + i)) + __ldg(a.new_lens + i)) : INT32_MIN;
  }
  __syncthreads();
  for (int32_t i = tid; i < a.R; i += blockDim.x) {
    const int32_t mine = len[i];
    int32_t rank = 0;
    for (int32_t j = 0; j < n4; ++j) {
      const int4 x = *reinterpret_cast<const int4 *>(len + 4 * j);
      rank += (x.x > mine || (x.x == mine && 4 * j < i)) + (x.y > mine || (x.y == mine && 4 * j + 1 < i)) +
              (x.z > mine || (x.z == mine && 4 * j + 2 < i)) + (x.w > mine || (x.w == mine && 4 * j + 3 < i));
    }
    if (rank == k) pick = i;
  }
  __syncthreads();
  return static_cast<int32_t>(__reduce_max_sync(kFull, static_cast<uint32_t>(pick)));  // into a uniform register
}

// The lists of a unit (empty when its header contradicts itself).
struct Unit {
  int64_t u;  // index in the tables
  int32_t n_hi, n_lo, p_hi;
};

__device__ __forceinline__ Unit load_unit(const ExtendArgs &a, int64_t u) {
  const int4 h = __ldg(reinterpret_cast<const int4 *>(a.unit_hdr + 4 * u));
  Unit x{u, h.x, h.y, h.z};
  if (h.x < 0 || h.y < 0 || h.z != (static_cast<int64_t>(h.x) + a.P - 1) / a.P ||
      h.w != (static_cast<int64_t>(h.y) + 2 * a.P - 1) / (2 * a.P) || h.z + h.w > a.pmax) {
    set_error(a.status, DKV_E_INTERNAL);
    x.n_hi = x.n_lo = x.p_hi = 0;
  }
  return x;
}

// Token tiles: 128 tokens of one kind, the high list's, then the low list's,
// then the new tokens'.
struct Tiles {
  int32_t hi, lo, fresh;
  __device__ __forceinline__ int32_t count() const { return hi + lo + fresh; }
};

}  // namespace tc
}  // namespace dkv
