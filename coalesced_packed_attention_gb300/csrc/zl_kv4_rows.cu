// Rows of the 4-bit cache: new keys and values in, all of a sequence's out.
//
// In: a block of 16 channels has the scale s nearest to max|x| / 6 (five bits of exponent, three of mantissa) and each
// channel the code nearest to |x| / s, ties to even.  Every step is exact or correctly rounded: the quotients of bf16 numbers
// by 6 or by a four-bit s are at least 2^-14 (relative) away from the borders that they do not hit, far more than
// a division's 2^-24, so the codes are those of exact arithmetic.
// Out: code * s has six bits at most, exact in fp16 and bf16.
// Both move bytes: a thread takes 8 channels (16 bytes of bf16, 4 of codes), two threads share a scale.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "zl_internal.h"
#include "zl_kv4.cuh"
#include "zl_overlap.cuh"

namespace zl {
namespace {

constexpr int kRowThreads = 256;
constexpr int kWriteTokens = 4;  // tokens a block takes at a time

struct WriteParams {
  Kv4 c;
  const __nv_bfloat16* x[2];  // keys, values
  int64_t stride[2];
  const int32_t* starts;
  const int32_t* positions;
  int32_t* slot_positions;
  int64_t n_tokens;
};

// Bits of the scale of a block whose largest magnitude is amax.
__device__ __forceinline__ uint32_t scale_bits(float amax) {
  const float q = __fdiv_rn(amax, 6.f);
  if (q < 0x1p-14f) return (uint32_t)__float2int_rn(q * 0x1p17f);  // steps of 2^-17; 8 of them are the first normal number
  const uint32_t b = __float_as_uint(q);
  const uint32_t r = ((b + 0x7FFFFu + ((b >> 20) & 1)) >> 20) - ((127 - 15) << 3);  // three bits of mantissa, ties to even
  return r < 224 ? r : 224;                                                         // 2^13
}

__device__ __forceinline__ float scale_value(uint32_t bits) { return __half2float(__ushort_as_half((unsigned short)(bits << 7))); }

__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint32_t o;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tmov.b32 %0, {t, 0, 0, 0};\n\t}" : "=r"(o) : "f"(lo), "f"(hi));
  return o;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) zl_kv4_write_kernel(const WriteParams p) {
  __shared__ int s_seq[kWriteTokens], s_slot[kWriteTokens];
  let_next_start();
  wait_for_previous();
  const int64_t t0 = (int64_t)blockIdx.x * kWriteTokens;
  if (threadIdx.x < kWriteTokens) {
    const int64_t t = t0 + threadIdx.x;
    int seq = -1, slot = -1;
    if (t < p.n_tokens) {
      int lo = (int)t;
      if (p.starts) {  // the last sequence that starts at or before the token
        int hi = p.c.n_seqs;
        lo = 0;
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (p.starts[mid] <= t) lo = mid;
          else hi = mid;
        }
      }
      int first = 0;
      const int n = kv4_new(p.c, p.starts, p.n_tokens, INT32_MAX, lo, &first);
      if (t >= first && t - first < n) {
        seq = lo;
        slot = kv4_len(p.c, lo) - n + (int)(t - first);
      }
    }
    s_seq[threadIdx.x] = seq;
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();
  const int per_row = p.c.heads * (D / 8);  // threads of a token's keys or values
  const int units = kWriteTokens * 2 * per_row;
  // two threads of a scale are neighbours: per_row is even and 256 is
#pragma unroll 2
  for (int base = 0; base < units; base += kRowThreads) {
    const int u = base + threadIdx.x;
    const int tok = u / (2 * per_row), rest = u - tok * 2 * per_row;
    const int which = rest >= per_row, e = rest - which * per_row;
    const int h = e / (D / 8), c8 = e % (D / 8);
    const int seq = u < units ? s_seq[tok] : -1, slot = u < units ? s_slot[tok] : -1;
    const bool there = seq >= 0 && slot >= 0;
    uint4 raw = make_uint4(0, 0, 0, 0);
    uint8_t* tile = nullptr;
    if (there) {
      raw = *reinterpret_cast<const uint4*>((which ? p.x[1] : p.x[0]) + (t0 + tok) * (which ? p.stride[1] : p.stride[0]) + h * D + c8 * 8);
      tile = kv4_tile<D>(p.c, seq, h, slot);
      if (!tile) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    }
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8], amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
      amax = fmaxf(amax, fabsf(x[i]));  // of a number and NaN the number
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    if (!tile) continue;
    const uint32_t sb = scale_bits(amax);
    const float s = scale_value(sb);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float y[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float v = x[2 * i + j];
        y[j] = v == v && sb ? __fdiv_rn(v, s) : 0.f;
      }
      codes |= encode2(y[0], y[1]) << (8 * i);
    }
    const int row = slot & 15;
    *reinterpret_cast<uint32_t*>(tile + which * 8 * D + row * (D / 2) + c8 * 4) = codes;
    if (!(c8 & 1)) tile[16 * D + which * D + row * (D / 16) + c8 / 2] = (uint8_t)sb;
  }
  if (p.slot_positions) {
    for (int u = threadIdx.x; u < kWriteTokens * p.c.heads; u += kRowThreads) {
      const int tok = u / p.c.heads, h = u % p.c.heads;
      if (s_seq[tok] >= 0 && s_slot[tok] >= 0) {
        const int64_t slots = (int64_t)p.c.max_pages << p.c.page_shift;
        p.slot_positions[((int64_t)s_seq[tok] * p.c.heads + h) * slots + s_slot[tok]] = p.positions[t0 + tok];
      }
    }
  }
}

struct ReadParams {
  Kv4 c;
  __nv_bfloat16* out[2];
  int64_t stride[2];
  const int64_t* row_starts;
  int64_t n_rows;
};

__device__ __forceinline__ uint32_t to_bf16x2(uint32_t half2_bits) {
  __half2 h;
  memcpy(&h, &half2_bits, 4);
  const float2 f = __half22float2(h);
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
  uint32_t o;
  memcpy(&o, &b, 4);
  return o;
}

// A block takes a run of the 16-slot tiles of all sequences, every head of a tile.
template <int D>
__global__ void __launch_bounds__(kRowThreads) zl_kv4_read_kernel(const ReadParams p) {
  __shared__ int64_t warp_sums[kRowThreads / 32];
  __shared__ int64_t s_before;
  __shared__ int s_seq;
  let_next_start();
  wait_for_previous();
  // tiles of all sequences in a row, dealt out evenly
  const int n = p.c.n_seqs, per = (n + kRowThreads - 1) / kRowThreads;
  const int b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);
  int64_t mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += (kv4_len(p.c, b) + kKv4Slots - 1) / kKv4Slots;
  int64_t before = kv4_scan<kRowThreads>(mine, &total, warp_sums);
  int64_t at = total * blockIdx.x / gridDim.x;
  const int64_t end = total * (blockIdx.x + 1) / gridDim.x;
  if (at >= end) return;
  if (at >= before && at < before + mine) {
    int b = b0;
    for (;; ++b) {
      const int tiles = (kv4_len(p.c, b) + kKv4Slots - 1) / kKv4Slots;
      if (at < before + tiles) break;
      before += tiles;
    }
    s_seq = b;
    s_before = before;
  }
  __syncthreads();
  int seq = s_seq, tile = (int)(at - s_before), len = kv4_len(p.c, seq);
  const int units = p.c.heads * kKv4Slots * 2 * (D / 8);
  for (; at < end; ++at, ++tile) {
    while (tile * kKv4Slots >= len) {  // the next sequence that holds a slot
      if (++seq >= n) return;
      tile = 0;
      len = kv4_len(p.c, seq);
    }
    const int64_t row0 = p.row_starts[seq];
    if (row0 < 0 || row0 > p.n_rows - len) {
      if (threadIdx.x == 0) kv4_report(p.c, ZL_KV4_BAD_STARTS);
      continue;
    }
    const int rows = min(kKv4Slots, len - tile * kKv4Slots);
    const uint8_t* src0 = kv4_tile<D>(p.c, seq, 0, tile * kKv4Slots);
    if (!src0 && threadIdx.x == 0) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    const int64_t head_step = (int64_t)(18 * D) << (p.c.page_shift - 4);
    // a warp writes 512 contiguous bytes of a row: threads run over channels, heads, slots, then keys and values
#pragma unroll 4
    for (int u = threadIdx.x; u < units; u += kRowThreads) {
      const int c8 = u % (D / 8), hr = u / (D / 8);
      const int h = hr % p.c.heads, rw = hr / p.c.heads;
      const int row = rw & 15, which = rw >> 4;
      if (row >= rows) continue;
      uint4 o = make_uint4(0, 0, 0, 0);
      if (src0) {
        const uint8_t* src = src0 + h * head_step;
        const uint32_t codes = *reinterpret_cast<const uint32_t*>(src + which * 8 * D + row * (D / 2) + c8 * 4);
        const uint32_t sb = src[16 * D + which * D + row * (D / 16) + c8 / 2];
        const uint32_t s2 = kv4_scale2(sb, sb);
        uint32_t v[4];
        kv4_decode(codes, v);
        o = make_uint4(to_bf16x2(kv4_mul(v[0], s2)), to_bf16x2(kv4_mul(v[1], s2)), to_bf16x2(kv4_mul(v[2], s2)),
                       to_bf16x2(kv4_mul(v[3], s2)));
      }
      __nv_bfloat16* dst = which ? p.out[1] : p.out[0];
      *reinterpret_cast<uint4*>(dst + (row0 + tile * kKv4Slots + row) * (which ? p.stride[1] : p.stride[0]) + h * D + c8 * 8) = o;
    }
  }
}

}  // namespace
}  // namespace zl

using namespace zl;

extern "C" zl_status zl_kv4_write(const zl_kv4_cache* cache, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                                  int64_t n_tokens, const int32_t* starts, const int32_t* positions,
                                  int32_t* slot_positions, void* stream) {
  NvtxRange range("zl_kv4_write");
  WriteParams p{};
  zl_status s = kv4_check(cache, &p.c);
  if (s != ZL_OK) return s;
  if (n_tokens < 0 || n_tokens > INT32_MAX || (!positions) != (!slot_positions)) return ZL_ERR_INVALID_ARG;
  if (!starts && n_tokens != cache->n_seqs) return ZL_ERR_INVALID_ARG;
  if (n_tokens == 0 || cache->n_seqs == 0) return ZL_OK;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
  if ((s = kv4_check_rows(k, k_stride, row)) != ZL_OK || (s = kv4_check_rows(v, v_stride, row)) != ZL_OK) return s;
  if (!kv4_aligned(starts, 4) || !kv4_aligned(positions, 4) || !kv4_aligned(slot_positions, 4)) return ZL_ERR_ALIGN;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.starts = starts;
  p.positions = positions;
  p.slot_positions = slot_positions;
  p.n_tokens = n_tokens;
  const unsigned blocks = (unsigned)((n_tokens + kWriteTokens - 1) / kWriteTokens);
  const auto kernel = cache->head_dim == 128 ? zl_kv4_write_kernel<128> : zl_kv4_write_kernel<64>;
  return launch_overlapped(kernel, blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream), p) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

extern "C" zl_status zl_kv4_read(const zl_kv4_cache* cache, void* k_out, int64_t k_stride, void* v_out, int64_t v_stride,
                                 int64_t n_rows, const int64_t* row_starts, void* stream) {
  NvtxRange range("zl_kv4_read");
  ReadParams p{};
  zl_status s = kv4_check(cache, &p.c);
  if (s != ZL_OK) return s;
  if (n_rows < 0 || n_rows > INT64_MAX / 2) return ZL_ERR_INVALID_ARG;
  if (n_rows == 0 || cache->n_seqs == 0) return ZL_OK;
  const int64_t row = (int64_t)cache->n_kv_heads * cache->head_dim;
  if ((s = kv4_check_rows(k_out, k_stride, row)) != ZL_OK || (s = kv4_check_rows(v_out, v_stride, row)) != ZL_OK) return s;
  if (!row_starts) return ZL_ERR_INVALID_ARG;
  if (!kv4_aligned(row_starts, 8)) return ZL_ERR_ALIGN;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  p.out[0] = static_cast<__nv_bfloat16*>(k_out);
  p.out[1] = static_cast<__nv_bfloat16*>(v_out);
  p.stride[0] = k_stride;
  p.stride[1] = v_stride;
  p.row_starts = row_starts;
  p.n_rows = n_rows;
  const auto kernel = cache->head_dim == 128 ? zl_kv4_read_kernel<128> : zl_kv4_read_kernel<64>;
  static PerDeviceInt resident[2];
  int per_sm = 0;
  cudaError_t e = resident[cache->head_dim == 128].get(&per_sm, [&](int, int* out) {
    const cudaError_t r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kernel, kRowThreads, 0);
    if (*out < 1) *out = 1;
    return r;
  });
  if (e != cudaSuccess) return ZL_ERR_CUDA;
  // no more blocks than the rows asked for have tiles
  const int64_t tiles = n_rows / kKv4Slots + cache->n_seqs;
  const int64_t blocks = (int64_t)sms * per_sm < tiles ? (int64_t)sms * per_sm : tiles;
  e = launch_overlapped(kernel, (unsigned)blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
