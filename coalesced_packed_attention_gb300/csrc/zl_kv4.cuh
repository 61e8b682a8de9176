// Key-value cache in 4 bits: geometry, checks of arguments, and what its kernels share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/zl.h"
#include "zl_causal.h"

namespace zl {

constexpr int kKv4Slots = 16;  // slots of a tile

// The cache as kernels take it.
struct Kv4 {
  uint8_t* data;
  const int32_t* pages;
  const int32_t* lens;
  int32_t* status;
  int64_t n_pages;
  int32_t n_seqs, heads, max_pages, page_shift;
};

inline bool kv4_aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline zl_status kv4_check(const zl_kv4_cache* c, Kv4* out) {
  if (!c) return ZL_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return ZL_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128 && c->page != 256) return ZL_ERR_UNSUPPORTED;
  if (c->n_seqs < 0 || c->n_seqs > (1 << 20) || c->n_kv_heads < 1 || c->n_kv_heads > 1024 || c->max_pages < 0 ||
      c->n_pages < 0 || c->n_pages > INT32_MAX || (int64_t)c->max_pages * c->page >= 1 << 30 ||
      (int64_t)c->max_pages * (c->page / 16) * c->n_kv_heads > INT32_MAX ||  // a sequence's tiles are numbered
      c->n_pages * c->n_kv_heads * (c->page / 16) >= 1 << 28)  // of 1152 bytes and more: 309 GB
    return ZL_ERR_INVALID_ARG;
  if (c->n_seqs > 0 && (!c->lens || (c->max_pages > 0 && !c->pages) || (c->n_pages > 0 && !c->data))) return ZL_ERR_INVALID_ARG;
  if (!kv4_aligned(c->data, 16) || !kv4_aligned(c->pages, 4) || !kv4_aligned(c->lens, 4) || !kv4_aligned(c->status, 4))
    return ZL_ERR_ALIGN;
  int shift = 0;
  while ((1 << shift) < c->page) ++shift;
  *out = {static_cast<uint8_t*>(c->data), c->pages,      c->lens,      c->status, c->n_pages,
          c->n_seqs,                      c->n_kv_heads, c->max_pages, shift};
  return ZL_OK;
}

// Rows of bf16 [tokens, heads, d] with a token stride.
inline zl_status kv4_check_rows(const void* p, int64_t stride, int64_t row) {
  if (!p || stride < row) return ZL_ERR_INVALID_ARG;
  return kv4_aligned(p, 16) && stride % 8 == 0 ? ZL_OK : ZL_ERR_ALIGN;
}

// Inputs of the kernels below may be written by the kernel before them while they are being set up: plain loads.
__device__ __forceinline__ void kv4_report(const Kv4& c, int32_t bit) {
  if (c.status) atomicOr(c.status, bit);
}
__device__ __forceinline__ int kv4_len(const Kv4& c, int b) {
  const int m = c.lens[b], most = c.max_pages << c.page_shift;
  if (m >= 0 && m <= most) return m;
  kv4_report(c, ZL_KV4_BAD_LEN);
  return m < 0 ? 0 : most;
}
// New tokens of a sequence: first and count; none where its range does not fit.
__device__ __forceinline__ int kv4_new(const Kv4& c, const int32_t* starts, int64_t n_tokens, int max_new, int b, int* first) {
  if (!starts) {
    *first = b;
    return 1;
  }
  const int64_t lo = starts[b], hi = starts[b + 1];
  *first = (int)lo;
  if (lo >= 0 && hi >= lo && hi <= n_tokens && hi - lo <= max_new) return (int)(hi - lo);
  kv4_report(c, ZL_KV4_BAD_STARTS);
  return 0;
}
// Number of a slot's tile in `data` (they are less than 2^28), or kKv4None where its page is none of the cache's.
constexpr uint32_t kKv4None = 0xFFFFFFFFu;
__device__ __forceinline__ uint32_t kv4_place(const Kv4& c, int b, int h, int slot) {
  const uint32_t page = c.pages[(int64_t)b * c.max_pages + (slot >> c.page_shift)];
  const int shift = c.page_shift - 4;
  return page < (uint32_t)c.n_pages ? ((page * c.heads + h) << shift) + ((slot >> 4) & ((1 << shift) - 1)) : kKv4None;
}
// The tile itself, or null.
template <int D>
__device__ __forceinline__ uint8_t* kv4_tile(const Kv4& c, int b, int h, int slot) {
  const uint32_t place = kv4_place(c, b, h, slot);
  return place == kKv4None ? nullptr : c.data + (uint64_t)place * (18 * D);
}

// Four codes of two channels each -> four pairs of fp16.
__device__ __forceinline__ void kv4_decode(uint32_t codes, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(codes));
}
__device__ __forceinline__ uint32_t kv4_mul(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}
// A scale's bits are those of an fp16 number from its exponent on: two of them, low and high half.
__device__ __forceinline__ uint32_t kv4_scale2(uint32_t lo, uint32_t hi) { return (lo << 7) | (hi << 23); }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; what each wrote before it, to shared or global memory, the others see after it.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();  // .aligned: the warp's lanes come together, also from branches
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix sum over a block's threads, and the total; warp_sums: one number a warp in shared memory.
template <int kThreads>
__device__ __forceinline__ int64_t kv4_scan(int64_t mine, int64_t* total, int64_t* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += warp_sums[i];
    all += warp_sums[i];
  }
  __syncthreads();
  *total = all;
  return before + x - mine;
}

}  // namespace zl
