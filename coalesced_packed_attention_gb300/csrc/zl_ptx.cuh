// Thin inline-PTX wrappers for sm_103a: mbarriers, TMA tensor loads, tcgen05 (TMEM
// allocation, MMA, commit, TMEM load/store) and the two shared-memory matrix
// descriptor / instruction descriptor encodings the kernels use.
#pragma once
#include <cuda.h>
#include <stdint.h>

namespace zl {

// Spin budget of every bounded wait, in SM clock cycles (~0.5 s at 2 GHz).  A wait
// that runs out records ZL_ERR_TIMEOUT in the plan's status word and the kernel
// leaves its loops instead of hanging the GPU.
constexpr long long kWaitLimitCycles = 1000000000LL;

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ------------------------------------------------------------------ mbarrier
__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Wait until the phase with the given parity has completed; false after the budget.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (clock64() - t0 > kWaitLimitCycles) return false;
  }
  return true;
}

// ------------------------------------------------------------------ TMA
__device__ __forceinline__ void tma_prefetch_desc(const void* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// 3-D tiled load (coordinates innermost first) completing on an mbarrier.
__device__ __forceinline__ void tma_load_3d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}

// Orders this thread's generic-proxy shared-memory writes before later async-proxy
// (tensor core, bulk copy) accesses of the same bytes.
__device__ __forceinline__ void fence_proxy_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// Zero rows [first_row, 128) of a [128 rows, D] bf16 tile held as D/64 boxes of 128 rows
// x 128 bytes (the 128-byte swizzle permutes 16-byte chunks within a row, so a row stays
// within its own 128 bytes); the 32 lanes of a warp share the stores.  Callers then
// fence (fence_proxy_async_smem) and __syncwarp before a product reads the tile.  Used
// on the ragged last block of an item, whose rows past the item are other tokens of the
// packed tensor: a zero weight times a non-finite value there would be NaN.
template <int D>
__device__ __forceinline__ void zero_tile_rows(uint32_t tile, int first_row, int lane) {
  const int n = (128 - first_row) * 8;  // 16-byte chunks per box
#pragma unroll
  for (int b = 0; b < D / 64; ++b)
    for (int i = lane; i < n; i += 32)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + b * 16384 + first_row * 128 + i * 16),
                   "r"(0u)
                   : "memory");
}

// ------------------------------------------------------------------ tcgen05
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)),
               "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T-ish per the descriptors; accumulate != 0 keeps D.
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Same with the A operand read from TMEM (lane = row, two bf16 per 32-bit column).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive (once) on an mbarrier when every MMA issued so far by this thread is done.
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   smem_u32(bar))
               : "memory");
}

// The same three, executed by a whole warp whose control flow and operands are
// warp-uniform: elect.sync picks one lane (the same lane every time for a full warp) and
// only that lane executes the product or the commit, under a predicate rather than a
// branch, so the issuing loop stays convergent.
__device__ __forceinline__ void mma_ss_w(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts_w(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_commit_w(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}

#define ZL_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                 "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define ZL_W8(i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                 "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])

// 32 lanes x 32 consecutive 32-bit columns: thread t of the warp gets row (lane base + t).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : ZL_R8(0), ZL_R8(8), ZL_R8(16), ZL_R8(24)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      ZL_W8(0), ZL_W8(8)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      ZL_W8(0), ZL_W8(8), ZL_W8(16), ZL_W8(24)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptor, 128-byte swizzle (the layout TMA writes with
// CU_TENSOR_MAP_SWIZZLE_128B into a 1024-byte aligned buffer).
//   K-major operand : rows of 128 B (64 bf16 of K), 8-row groups sbo = 1024 B apart;
//                     a K step inside the 128-byte row advances the start address.
//   MN-major operand: 64 MN elements per 128-byte row, K rows 128 B apart, 8-row K
//                     groups sbo apart, 64-element MN groups lbo apart.
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((sbo >> 4) & 0x3FFFu) << 32;
  d |= (uint64_t)1 << 46;  // descriptor version for tcgen05
  d |= (uint64_t)2 << 61;  // swizzle mode: 128 B
  return d;
}

// The same descriptor advanced by `bytes` (a multiple of 16): the start address is
// the low 14-bit field and a shared-memory address stays below 256 KB, so a plain add
// never carries into the next field.
__device__ __forceinline__ uint64_t sdesc_add(uint64_t desc, uint32_t bytes) { return desc + (bytes >> 4); }
// Low and high 32-bit words of sdesc_sw128 with SBO = 1024 B: every such descriptor
// shares the high word, so an issuer can keep only low words (start | LBO) and join.
__device__ __forceinline__ uint32_t sdesc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | (((lbo >> 4) & 0x3FFFu) << 16);
}
constexpr uint32_t kSdescHi1024 = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint64_t sdesc_join(uint32_t lo) { return ((uint64_t)kSdescHi1024 << 32) | lo; }

// Instruction descriptor of tcgen05.mma kind::f16: bf16 A and B, fp32 D, M x N tile.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn_major, bool b_mn_major) {
  return (1u << 4)                                 // D format: f32
         | (1u << 7)                               // A format: bf16
         | (1u << 10)                              // B format: bf16
         | ((a_mn_major ? 1u : 0u) << 15)          // A major-ness
         | ((b_mn_major ? 1u : 0u) << 16)          // B major-ness
         | ((uint32_t)(N >> 3) << 17)              // N / 8
         | ((uint32_t)(M >> 4) << 24);             // M / 16
}

// Four or eight K steps of one product in a row, under one election: a step's operands are the first's plus kA (A) and
// kB (B), and from the fifth on kA4 and kB4 more; a TMEM operand in columns, descriptors (low words) in 16 bytes.
// `accumulate` says whether the first step adds to what is there.  (Step by step, an election and a predicate each, the
// issuing warp was what the tensor core waited for: forward of 4109 tokens, 24/8 heads, d = 64, 33.3 against 31.6 us.)
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ts8_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 4 * %6 + %7;\n\tadd.u32 y, %2, 4 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 5 * %6 + %7;\n\tadd.u32 y, %2, 5 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 6 * %6 + %7;\n\tadd.u32 y, %2, 6 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 7 * %6 + %7;\n\tadd.u32 y, %2, 7 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4)
      : "memory");
}
// The same, and a commit to `bar`.
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ts8_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 4 * %6 + %7;\n\tadd.u32 y, %2, 4 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 5 * %6 + %7;\n\tadd.u32 y, %2, 5 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 6 * %6 + %7;\n\tadd.u32 y, %2, 6 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "add.u32 x, %1, 7 * %6 + %7;\n\tadd.u32 y, %2, 7 * %8 + %9;\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], b, %4, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4), "r"(smem_u32(bar))
      : "memory");
}
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ss8_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 4 * %6 + %7;\n\tadd.u32 y, %2, 4 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 5 * %6 + %7;\n\tadd.u32 y, %2, 5 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 6 * %6 + %7;\n\tadd.u32 y, %2, 6 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 7 * %6 + %7;\n\tadd.u32 y, %2, 7 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4)
      : "memory");
}
// The same, and a commit to `bar`.
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ss8_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 4 * %6 + %7;\n\tadd.u32 y, %2, 4 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 5 * %6 + %7;\n\tadd.u32 y, %2, 5 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 6 * %6 + %7;\n\tadd.u32 y, %2, 6 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 7 * %6 + %7;\n\tadd.u32 y, %2, 7 * %8 + %9;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4), "r"(smem_u32(bar))
      : "memory");
}
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ss4_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4)
      : "memory");
}
// The same, and a commit to `bar`.
template <int kA, int kA4, int kB, int kB4>
__device__ __forceinline__ void mma_ss4_w(uint32_t d_tmem, uint32_t a, uint32_t b_lo, uint32_t idesc, uint32_t accumulate, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b32 x, y;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, 0, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
      "add.u32 x, %1, 0 * %6;\n\tadd.u32 y, %2, 0 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t"
      "add.u32 x, %1, 1 * %6;\n\tadd.u32 y, %2, 1 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 2 * %6;\n\tadd.u32 y, %2, 2 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "add.u32 x, %1, 3 * %6;\n\tadd.u32 y, %2, 3 * %8;\n\tmov.b64 a, {x, %3};\n\tmov.b64 b, {y, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, t;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t}" ::"r"(d_tmem),
      "r"(a), "r"(b_lo), "r"(kSdescHi1024), "r"(idesc), "r"(accumulate), "n"(kA), "n"(kA4), "n"(kB), "n"(kB4), "r"(smem_u32(bar))
      : "memory");
}

// ------------------------------------------------------------------ math
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// max of three (one instruction on sm_100 and later)
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Two-wide fp32 arithmetic (one instruction per pair on sm_100 and later; each lane
// rounds exactly like the scalar operation)
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

}  // namespace zl
