// Rows of the 4-bit cache: new keys and values in, all of a sequence's out.
//
// In: a block of 16 channels has the scale s nearest to max|x| / 6 (five bits of exponent, three of mantissa) and each
// channel the code nearest to |x| / s, ties to even.  The codes are those of exact arithmetic: quotients of bf16
// numbers by 6 or by a four-bit s either hit a border between two codes (scales) or miss it by 2^-11 and more, so a
// product with the reciprocal, off by 2^-20 at most, rounded to a multiple of 2^-16, is on the right side, or on the
// border, where the conversion's own ties to even decide.  (IEEE divisions took two thirds of the time.)
// Out: code * s has six bits at most, exact in fp16 and bf16.
// Both move bytes: a thread takes 8 channels (16 bytes of bf16, 4 of codes), two threads share a scale, and has several
// loads under way.  Measured at 8 heads, d = 128: 14 336 tokens in 21 us (75 MB, 3.6 TB/s: the arithmetic of the codes
// and one wave of blocks), 4 x 16 384 slots out in 58 us (344 MB, 5.9 TB/s, 0.89 of a copy).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "zl_internal.h"
#include "zl_kv4.cuh"
#include "zl_overlap.cuh"
#include "zl_ptx.cuh"

namespace zl {
namespace {

constexpr int kRowThreads = 256;
constexpr int kWriteTokens = 32;  // tokens a block takes at most: a lane each looks up where one goes
constexpr int kWriteLoads = 4;    // units of 8 channels that a thread has under way

struct WriteParams {
  Kv4 c;
  const __nv_bfloat16* x[2];  // keys, values
  int64_t stride[2];
  const int32_t* starts;
  const int32_t* positions;
  int32_t* slot_positions;
  int64_t n_tokens;
  int32_t per_block;  // tokens of a block
};

// Bits of the scale of a block whose largest magnitude is amax.
__device__ __forceinline__ uint32_t scale_bits(float amax) {
  // a sixth, to the multiple of 2^-15 of its power of two that it is meant to be, if there is one
  const uint32_t b = (__float_as_uint(amax * (1.f / 6.f)) + 0x80u) & 0xFFFFFF00u;
  const float q = __uint_as_float(b);
  if (q < 0x1p-14f) return (uint32_t)__float2int_rn(q * 0x1p17f);  // steps of 2^-17; 8 of them are the first normal number
  const uint32_t r = ((b + 0x7FFFFu + ((b >> 20) & 1)) >> 20) - ((127 - 15) << 3);  // three bits of mantissa, ties to even
  return r < 224 ? r : 224;                                                         // 2^13
}

// Eight numbers' codes; inv: 1 / s, to an ulp or two.
__device__ __forceinline__ uint32_t encode8(const uint32_t (&w)[4], float inv) {
  // at 192 numbers are 2^-16 apart
  const float2 inv2 = make_float2(inv, inv), up = make_float2(192.f, 192.f), down = make_float2(-192.f, -192.f);
  float2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y[i] = add2(fma2(make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)), inv2, up), down);
  uint32_t o;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\tmov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(o)
      : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
  return o;
}

// Largest magnitudes of a block of 16, as bf16 bits: this thread's 8 numbers and its neighbour's; above 0x7F80 where
// one is NaN.
__device__ __forceinline__ uint32_t abs_max(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}
__device__ __forceinline__ uint32_t block_max(const uint32_t (&w)[4]) {
  uint32_t m = abs_max(abs_max(w[0], w[1]), abs_max(w[2], w[3]));
  m = abs_max(m, m >> 16) & 0x7FFFu;
  return max(m, __shfl_xor_sync(0xffffffffu, m, 1));
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <int D>
__global__ void __launch_bounds__(kRowThreads) zl_kv4_write_kernel(const WriteParams p) {
  __shared__ int s_seq[kWriteTokens], s_slot[kWriteTokens];
  __shared__ uint8_t* s_codes[kWriteTokens];  // the token's row in its tile of the first head: codes and scales, or null
  __shared__ uint8_t* s_scales[kWriteTokens];
  let_next_start();
  wait_for_previous();
  const int64_t t0 = (int64_t)blockIdx.x * p.per_block;
  const int tokens = (int)min((int64_t)p.per_block, p.n_tokens - t0);
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    const int64_t t = t0 + lane;
    int b = (int)t0;
    if (p.starts) {  // the last sequence that starts at or before the block's first token, 32 ways at a time
      int lo = 0, hi = p.c.n_seqs;
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32, at = lo + lane * step;
        const int before = __popc(__ballot_sync(0xffffffffu, at < hi && p.starts[min(at, hi - 1)] <= t0));
        lo += max(0, before - 1) * step;
        hi = min(hi, lo + step);
      }
      b = lo;
    }
    int seq = -1, slot = -1;
    if (lane < tokens) {
      if (!p.starts) b = (int)t;
      else
        while (b + 1 < p.c.n_seqs && p.starts[b + 1] <= t) ++b;
      int first = 0;
      const int n = kv4_new(p.c, p.starts, p.n_tokens, INT32_MAX, b, &first);
      if (t >= first && t - first < n) {
        seq = b;
        slot = kv4_len(p.c, b) - n + (int)(t - first);
      }
    }
    s_seq[lane] = seq;
    s_slot[lane] = slot;
    uint8_t* tile = slot >= 0 ? kv4_tile<D>(p.c, seq, 0, slot) : nullptr;
    if (slot >= 0 && !tile) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    s_codes[lane] = tile ? tile + (slot & 15) * (D / 2) : nullptr;
    s_scales[lane] = tile + 16 * D + (slot & 15) * (D / 16);
  }
  __syncthreads();
  // A thread keeps to one column: 8 channels of a head's key or value; where a token has fewer than the block has
  // threads, several tokens side by side.  The two threads of a scale are neighbours: columns come by the 16.
  const int per_row = p.c.heads * (D / 8), columns = 2 * per_row;
  const int wide = min(columns, kRowThreads), side = kRowThreads / wide;
  const int head_step = (18 * D) << (p.c.page_shift - 4);
  for (int c0 = 0; c0 < columns; c0 += wide) {
    const int c = c0 + threadIdx.x % wide, tok0 = threadIdx.x / wide;
    const bool mine = c < columns && tok0 < side;
    const int which = c >= per_row, e = c - which * per_row, h = e / (D / 8), c8 = e % (D / 8);
    const int64_t stride = which ? p.stride[1] : p.stride[0];
    const __nv_bfloat16* src = (which ? p.x[1] : p.x[0]) + t0 * stride + h * D + c8 * 8;
    const int codes_at = h * head_step + which * 8 * D + c8 * 4, scale_at = h * head_step + which * D + c8 / 2;
    for (int i0 = 0; i0 < tokens; i0 += side * kWriteLoads) {
      uint32_t w[kWriteLoads][4];
      uint8_t* codes[kWriteLoads];
#pragma unroll
      for (int y = 0; y < kWriteLoads; ++y) {
        const int tok = i0 + y * side + tok0;
        codes[y] = mine && tok < tokens ? s_codes[tok] : nullptr;
        const uint4 raw = codes[y] ? *reinterpret_cast<const uint4*>(src + tok * stride) : make_uint4(0, 0, 0, 0);
        w[y][0] = raw.x; w[y][1] = raw.y; w[y][2] = raw.z; w[y][3] = raw.w;
      }
      uint32_t m[kWriteLoads], most = 0;
#pragma unroll
      for (int y = 0; y < kWriteLoads; ++y) most = max(most, m[y] = block_max(w[y]));
      if (__any_sync(0xffffffffu, most > 0x7F80u)) {  // NaN is held as 0
#pragma unroll
        for (int y = 0; y < kWriteLoads; ++y) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if ((w[y][i] & 0x7FFFu) > 0x7F80u) w[y][i] &= 0xFFFF0000u;
            if ((w[y][i] & 0x7FFF0000u) > 0x7F800000u) w[y][i] &= 0xFFFFu;
          }
          m[y] = block_max(w[y]);
        }
      }
#pragma unroll
      for (int y = 0; y < kWriteLoads; ++y) {
        const uint32_t sb = scale_bits(__uint_as_float(m[y] << 16));
        const float s = __half2float(__ushort_as_half((unsigned short)(sb << 7)));
        if (codes[y]) {
          // scale 0: every channel is 0
          *reinterpret_cast<uint32_t*>(codes[y] + codes_at) = sb ? encode8(w[y], reciprocal(s)) : 0;
          if (!(c8 & 1)) s_scales[i0 + y * side + tok0][scale_at] = (uint8_t)sb;
        }
      }
    }
  }
  if (p.slot_positions) {
    const int64_t slots = (int64_t)p.c.max_pages << p.c.page_shift;
    for (int u = threadIdx.x; u < tokens * p.c.heads; u += kRowThreads) {
      const int tok = u / p.c.heads, h = u % p.c.heads;
      if (s_slot[tok] >= 0) p.slot_positions[((int64_t)s_seq[tok] * p.c.heads + h) * slots + s_slot[tok]] = p.positions[t0 + tok];
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

// The 16-slot tiles of all sequences' heads in a row (a tile's heads side by side, as their rows are), dealt out evenly
// over the blocks; a warp takes one at a time, all its loads under way together.
template <int D>
__global__ void __launch_bounds__(kRowThreads) zl_kv4_read_kernel(const ReadParams p) {
  __shared__ int64_t warp_sums[kRowThreads / 32];
  __shared__ int64_t s_before;
  __shared__ int s_seq;
  let_next_start();
  wait_for_previous();
  const int n = p.c.n_seqs, per = (n + kRowThreads - 1) / kRowThreads;
  const int b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);
  int64_t mine = 0, total;
  for (int b = b0; b < b1; ++b) mine += (kv4_len(p.c, b) + kKv4Slots - 1) / kKv4Slots;
  int64_t before = kv4_scan<kRowThreads>(mine, &total, warp_sums);
  const int64_t begin = total * p.c.heads * blockIdx.x / gridDim.x, end = total * p.c.heads * (blockIdx.x + 1) / gridDim.x;
  if (begin >= end) return;
  const int64_t begin_tile = begin / p.c.heads;
  if (begin_tile >= before && begin_tile < before + mine) {
    int b = b0;
    for (;; ++b) {
      const int tiles = (kv4_len(p.c, b) + kKv4Slots - 1) / kKv4Slots;
      if (begin_tile < before + tiles) break;
      before += tiles;
    }
    s_seq = b;
    s_before = before;
  }
  __syncthreads();
  int seq = s_seq, len = kv4_len(p.c, seq);
  int64_t seq_begin = s_before * p.c.heads;  // first tile and head of the sequence
  const int lane = threadIdx.x & 31;
  for (int64_t at = begin + (threadIdx.x >> 5); at < end; at += kRowThreads / 32) {
    int64_t seq_size = (int64_t)((len + kKv4Slots - 1) / kKv4Slots) * p.c.heads;
    while (at - seq_begin >= seq_size) {  // a later sequence
      if (++seq >= n) return;
      seq_begin += seq_size;
      len = kv4_len(p.c, seq);
      seq_size = (int64_t)((len + kKv4Slots - 1) / kKv4Slots) * p.c.heads;
    }
    const int off = (int)(at - seq_begin), tile = off / p.c.heads, h = off - tile * p.c.heads;
    const int64_t row0 = p.row_starts[seq];
    const uint8_t* src = kv4_tile<D>(p.c, seq, h, tile * kKv4Slots);
    if (row0 < 0 || row0 > p.n_rows - len) {
      if (lane == 0) kv4_report(p.c, ZL_KV4_BAD_STARTS);
      continue;
    }
    if (!src && lane == 0) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    const int rows = min(kKv4Slots, len - tile * kKv4Slots);
    constexpr int kPerRow = D / 8, kRowsAtOnce = 32 / kPerRow, kLoads = kKv4Slots / kRowsAtOnce;
    const int c8 = lane % kPerRow, r0 = lane / kPerRow;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint32_t codes[kLoads], sb[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int row = r0 + i * kRowsAtOnce;
        codes[i] = sb[i] = 0;
        if (src) {  // a tile is there as a whole
          codes[i] = *reinterpret_cast<const uint32_t*>(src + which * 8 * D + row * (D / 2) + c8 * 4);
          sb[i] = src[16 * D + which * D + row * (D / 16) + c8 / 2];
        }
      }
      const int64_t stride = which ? p.stride[1] : p.stride[0];
      __nv_bfloat16* dst = (which ? p.out[1] : p.out[0]) + (row0 + tile * kKv4Slots + r0) * stride + h * D + c8 * 8;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        uint32_t v[4];
        kv4_decode(codes[i], v);
        const uint32_t s2 = kv4_scale2(sb[i], sb[i]);
        const uint4 o = make_uint4(to_bf16x2(kv4_mul(v[0], s2)), to_bf16x2(kv4_mul(v[1], s2)), to_bf16x2(kv4_mul(v[2], s2)),
                                   to_bf16x2(kv4_mul(v[3], s2)));
        if (r0 + i * kRowsAtOnce < rows) *reinterpret_cast<uint4*>(dst + i * kRowsAtOnce * stride) = o;
      }
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
  if (n_tokens < 0 || n_tokens > INT32_MAX) return ZL_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!positions) != (!slot_positions)) return ZL_ERR_INVALID_ARG;  // none of no tokens
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
  // as few tokens a block as give every SM four blocks
  const int64_t even = (n_tokens + 4 * sms - 1) / (4 * sms);
  p.per_block = (int32_t)(even < kWriteTokens ? even : kWriteTokens);
  const unsigned blocks = (unsigned)((n_tokens + p.per_block - 1) / p.per_block);
  const auto kernel = cache->head_dim == 128 ? zl_kv4_write_kernel<128> : zl_kv4_write_kernel<64>;
  const cudaError_t e = launch_overlapped(kernel, blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
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
  // no more warps than the rows asked for have tiles
  const int64_t most = ((n_rows / kKv4Slots + cache->n_seqs) * cache->n_kv_heads + kRowThreads / 32 - 1) / (kRowThreads / 32);
  const int64_t blocks = (int64_t)sms * per_sm < most ? (int64_t)sms * per_sm : most;
  e = launch_overlapped(kernel, (unsigned)blocks, kRowThreads, 0, static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
