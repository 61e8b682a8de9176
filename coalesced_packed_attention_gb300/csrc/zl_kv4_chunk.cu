// Attention of many rows over the 4-bit cache: chunks of prompts, drafted tokens of large groups.
//
// With many rows (tokens x group) a key head, forming fp16 operands from codes for every 16 rows is what a pass over
// the cache costs (zl_kv4_attn.cu, which also has the rule between the two).  Here it is done once for 128 rows: eight
// warps turn a block of 128 slots into fp16 tiles in shared memory (exact: code * scale has six bits), and the tensor
// core takes them as tcgen05 operands,
//   S = Q K^T (both from shared memory),  O += P V (P from tensor memory, V channel-major),
// with 128 rows to a tile and S, P and O in tensor memory; one warpgroup does the softmax, a thread a row.
//
// Per block of 128 slots the tensor core works 1024 cycles (d = 128), the exponentials of 128 rows take 1024, and
// shared memory moves 178 KB (codes in and out 18 + 18, tiles in 64, operands out 96): 1400 cycles.  Measured, a block
// takes some 3500 (128 rows over 16 x 4096 slots of 8 key heads, d = 128: 67 us, 27 blocks an SM; 16-row passes 165;
// rows read back and causal attention 110): the chain S -> maximum -> exponentials -> P -> P V of the one warpgroup
// that a tile of 128 rows has, each step some 400 to 1200 cycles with its waits.  The scores kept in 208 registers a
// thread between maximum and exponentials, with the next block's keys formed ahead of this block's values, took as long
// (67 us).  Rows that a tile lacks cost nothing in the softmax (their warps pass by) and the same in the products.
// Order: S of a block is issued ahead of P V of the one before it, so that the softmax always has scores to work on;
// two buffers each of S, P, K and V, three of codes.
// Roles (448 threads, one block an SM): warps 0-3 softmax and output (thread = row = TMEM lane), 4-11 operands, 12
// products, 13 copies.  TMEM (512 columns): S [0,128) [128,256), O [256,256+d), P [384,448) [448,512).
// Items, cuts and the join are those of the other kernel, with tiles of 128 rows and units of 128 slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "zl_internal.h"
#include "zl_kv4_attn.cuh"
#include "zl_overlap.cuh"

namespace zl {
namespace {

constexpr int kThreads = 448, kUnit = 128, kItemCost = 2;
constexpr int kOperandWarps = 8;
constexpr int kCodeStages = 3, kStages = 2;
constexpr int kTileSlots = kUnit / kKv4Slots;  // tiles of a unit

template <int D>
struct Layout {
  static constexpr int kBox = 128 * 128;      // 128 rows x 128 bytes: 64 channels, swizzled
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kCodes = kTileSlots * 18 * D;
  static constexpr int kQ = 0, kK = kQ + kTile, kV = kK + kStages * kTile;
  static constexpr int kC = kV + kStages * kTile;
  static constexpr int kF = kC + kCodeStages * kCodes;  // [row] factor of a row's scores
  static constexpr int kBytes = kF + 128 * 4;
  // one block an SM: two would contend for tensor memory
  static constexpr int kSmem = (kBytes > 120 * 1024 ? kBytes : 120 * 1024) + 1024;  // to begin at a multiple of 1024
};

// Instruction descriptor of kind::f16 with fp16 A and B, fp32 D, M = 128.
constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) zl_kv4_chunk_kernel(const AttnParams p) {
  using L = Layout<D>;
  using W = Walk<kChunkRows, kUnit, kItemCost>;
  extern __shared__ __align__(1024) uint8_t smem_base[];
  uint8_t* smem = smem_base + (1024 - (smem_u32(smem_base) & 1023)) % 1024;  // what the swizzle wants
  __shared__ uint64_t bars[2 * kCodeStages + 4 * kStages + 2 + 5 + 1];
  __shared__ int64_t warp_sums[kThreads / 32];
  __shared__ int64_t s_before;
  __shared__ int s_seq;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  __shared__ uint32_t have_codes[kCodeStages], have_keys[4];  // which tiles of a unit are there: by stage of codes, by unit
  uint64_t* codes_full = bars;                       // [3]
  uint64_t* codes_empty = codes_full + kCodeStages;  // [3]
  uint64_t* k_full = codes_empty + kCodeStages;      // [2] each
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* q_full = v_empty + kStages;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;  // [2]
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* pv_done = p_full + 2;
  uint64_t* drained = pv_done + 1;
  float* row_factor = reinterpret_cast<float*>(smem + L::kF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kCodeStages; ++i) {
      mbar_init(codes_full + i, 1);
      mbar_init(codes_empty + i, kOperandWarps);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(k_full + i, kOperandWarps);
      mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, kOperandWarps);
      mbar_init(v_empty + i, 1);
    }
    mbar_init(q_full, kOperandWarps);
    mbar_init(q_empty, 1 + 4);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4);
    }
    mbar_init(pv_done, 1);
    mbar_init(drained, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  let_next_start();
  wait_for_previous();
  W seg;
  int64_t each;
  if (!first_segment_of<kThreads, 1 + kItemCost>(p, warp_sums, &s_before, &s_seq, seg, &each)) return;
  if (warp == 12) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // Bounded wait of a whole warp; on expiry every role leaves its loop.
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t a = smem_u32(bar);
    bool ok = mbar_try_wait(a, parity);
    if (!ok) {
      const long long t0 = clock64();
      while (!(ok = mbar_try_wait(a, parity)) && !abort_flag) {
        if (clock64() - t0 > kWaitLimitCycles) {
          abort_flag = 1;
          kv4_report(p.c, ZL_KV4_TIMEOUT);
        }
      }
    }
    return __all_sync(0xffffffffu, ok) != 0;
  };
  auto arrive = [&](uint64_t* bar) {  // of a warp, once all its lanes are here
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };

  if (warp == 13) {
    // ------------------------------------------------------------ copies: the tiles of a unit, one a lane
    uint32_t it = 0;
    bool ok = true;
    for (; !seg.done() && ok; seg.next(p)) {
      for (int x = seg.a; x < seg.e; ++x, ++it) {
        const int slot = x * kUnit + lane * kKv4Slots;
        uint32_t place = kKv4None;
        if (lane < kTileSlots && slot < seg.m) {
          place = kv4_place(p.c, seg.seq, seg.head, slot);
          if (place == kKv4None) kv4_report(p.c, ZL_KV4_BAD_PAGE);
        }
        const uint32_t have = __ballot_sync(0xffffffffu, place != kKv4None);
        const uint32_t st = it % kCodeStages;
        if (!(ok = wait(codes_empty + st, (it / kCodeStages & 1) ^ 1))) break;
        if (lane == 0) {
          have_codes[st] = have;
          mbar_arrive_expect_tx(codes_full + st, __popc(have) * 18 * D);
        }
        __syncwarp();
        if (place != kKv4None) {
          const uint32_t dst = smem_u32(smem + L::kC + st * L::kCodes + lane * 18 * D);
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                       "l"(p.c.data + (uint64_t)place * (18 * D)), "r"(18 * D), "r"(smem_u32(codes_full + st))
                       : "memory");
        }
      }
    }
    if (abort_flag)  // the copies in flight land before the block's shared memory goes back (a bounded wait each)
      for (uint32_t i = 1; i <= kCodeStages && i <= it; ++i)
        mbar_wait(codes_full + (it - i) % kCodeStages, (it - i) / kCodeStages & 1);
  } else if (warp == 12) {
    // ------------------------------------------------------------ products
    // The whole warp runs the loop; one elected lane executes each product and commit.
    constexpr uint32_t kIdS = idesc_f16(128, false), kIdPV = idesc_f16(D, true);
    constexpr int kNextBox = L::kBox / 16 - 4 * 2;  // K steps 0-3 lie in the first box, 4-7 in the second
    const uint32_t dQ = sdesc_lo(smem_u32(smem + L::kQ), 16), dK = sdesc_lo(smem_u32(smem + L::kK), 16);
    const uint32_t dV = sdesc_lo(smem_u32(smem + L::kV), L::kBox);
    uint32_t it = 0, segs = 0;
    bool ok = true, pend = false, pend_first = false;
    auto weigh = [&]() {  // P V of the unit before `it`
      const uint32_t i = it - 1, st = i % kStages;
      if (!wait(v_full + st, i / kStages & 1) || !wait(p_full + (i & 1), i / 2 & 1)) return false;
      tc_fence_after();
      mma_ts8_w<8, 0, 128, 0>(tmem + 256, tmem + 384 + 64 * (i & 1), dV + ((st * L::kTile) >> 4), kIdPV, pend_first ? 0u : 1u);
      mma_commit_w(v_empty + st);
      mma_commit_w(pv_done);
      return true;
    };
    for (; !seg.done() && ok; seg.next(p), ++segs) {
      for (int x = seg.a; x < seg.e; ++x) {
        const uint32_t st = it % kStages;
        if (!wait(k_full + st, it / kStages & 1) || (x == seg.a && !wait(q_full, segs & 1))) { ok = false; break; }
        tc_fence_after();
        const uint32_t dk = dK + ((st * L::kTile) >> 4);
        if constexpr (D == 128) mma_ss8_w<2, kNextBox, 2, kNextBox>(tmem + 128 * (it & 1), dQ, dk, kIdS, 0u);
        else mma_ss4_w<2, 0, 2, 0>(tmem + 128 * (it & 1), dQ, dk, kIdS, 0u);
        mma_commit_w(s_full + (it & 1));
        mma_commit_w(k_empty + st);
        if (x == seg.e - 1) mma_commit_w(q_empty);
        if (pend && !weigh()) { ok = false; break; }
        pend = true;
        pend_first = x == seg.a;
        ++it;
      }
    }
    if (ok && pend) weigh();
    // every product has ended before the block's memory goes back
    mma_commit_w(drained);
    mbar_wait(drained, 0);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ operands
    const int dt = threadIdx.x - 128;  // 0 .. 255
    uint32_t it = 0, segs = 0;
    bool ok = true;
    for (; !seg.done() && ok; seg.next(p), ++segs) {
      // queries: two threads a row, scaled by a power of two so that the row's largest is below 2
      if (!(ok = wait(q_empty, (segs & 1) ^ 1))) break;
      {
        const int r = dt >> 1, half = dt & 1, row = seg.tile * kChunkRows + r;
        constexpr int kLoads = D / 16;  // of 8 channels
        uint4 raw[kLoads];
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raw[i] = make_uint4(0, 0, 0, 0);
        if (row < seg.n * p.group) {
          const int tok = row / p.group;
          const int64_t head_at = (int64_t)(seg.head * p.group + row - tok * p.group) * D + half * (D / 2);
          const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(seg.first + tok) * p.q_stride + head_at);
#pragma unroll
          for (int i = 0; i < kLoads; ++i) raw[i] = src[i];
        }
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
          for (int y = 0; y < 4; ++y) top = max(top, max(w[y] & 0x7FFF0000u, (w[y] << 16) & 0x7FFF0000u));
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        const int ex = max(1, min(253, (int)(top >> 23)));  // 2^(ex - 127): the row's size
        const float down = __uint_as_float((uint32_t)(254 - ex) << 23), up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
          uint32_t o[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const __half2 h = __floats2half2_rn(__uint_as_float(w[y] << 16) * down, __uint_as_float(w[y] & 0xFFFF0000u) * down);
            memcpy(&o[y], &h, 4);
          }
          const int box = D == 128 ? half : 0, chunk = D == 128 ? i : half * kLoads + i;
          *reinterpret_cast<uint4*>(smem + L::kQ + box * L::kBox + r * 128 + ((chunk ^ (r & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
        if (half == 0) row_factor[r] = fmaxf(up * p.scale_log2, 0x1p-126f);  // not 0, which -inf is multiplied by
        fence_proxy_async_smem();
        arrive(q_full);
      }
      // A unit's keys or values: a lane takes 32 channels of a slot, neighbours the rest of it.  Lanes of the upper
      // channels begin with their third chunk, so that eight lanes' stores meet all banks.
      auto convert = [&](const uint8_t* codes, uint8_t* tile, int which, int valid, uint32_t have) {
        constexpr int kParts = D / 32;  // lanes a slot
#pragma unroll
        for (int y = 0; y < kParts / 2; ++y) {
          const int u = dt + 256 * y, key = u / kParts, part = u % kParts;
          const uint8_t* src = codes + (key >> 4) * 18 * D;
          const uint4 raw = *reinterpret_cast<const uint4*>(src + which * 8 * D + (key & 15) * (D / 2) + part * 16);
          uint32_t s0 = src[(16 + which) * D + (key & 15) * (D / 16) + 2 * part];
          uint32_t s1 = src[(16 + which) * D + (key & 15) * (D / 16) + 2 * part + 1];
          // what lies in slots past the end may be no number: as values they are 0 (their weights are, too)
          if (key >= valid || !((have >> (key >> 4)) & 1)) s0 = s1 = 0;
          const bool upper = part >= 2;
          const uint32_t w[4] = {upper ? raw.z : raw.x, upper ? raw.w : raw.y, upper ? raw.x : raw.z, upper ? raw.y : raw.w};
          const uint32_t sa = kv4_scale2(s0, s0), sb = kv4_scale2(s1, s1);
          uint8_t* dst = tile + (part >> 1) * L::kBox + key * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[4];
            kv4_decode(w[i], v);
            const uint32_t s = (i < 2) != upper ? sa : sb;
            const int chunk = ((part & 1) * 4 + (i ^ (upper ? 2 : 0))) ^ (key & 7);
            *reinterpret_cast<uint4*>(dst + (chunk << 4)) =
                make_uint4(kv4_mul(v[0], s), kv4_mul(v[1], s), kv4_mul(v[2], s), kv4_mul(v[3], s));
          }
        }
        fence_proxy_async_smem();
      };
      for (int x = seg.a; x < seg.e; ++x, ++it) {
        const uint32_t cs = it % kCodeStages, st = it % kStages;
        if (!wait(codes_full + cs, it / kCodeStages & 1) || !wait(k_empty + st, (it / kStages & 1) ^ 1)) { ok = false; break; }
        const uint8_t* codes = smem + L::kC + cs * L::kCodes;
        const uint32_t have = have_codes[cs];
        const int valid = seg.m - x * kUnit;
        if (dt == 0) have_keys[it & 3] = have;
        convert(codes, smem + L::kK + st * L::kTile, 0, valid, have);
        arrive(k_full + st);
        if (!wait(v_empty + st, (it / kStages & 1) ^ 1)) { ok = false; break; }
        convert(codes, smem + L::kV + st * L::kTile, 1, valid, have);
        arrive(v_full + st);
        if (lane == 0) mbar_arrive(codes_empty + cs);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, output: thread = row
    const int r = threadIdx.x;
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    uint32_t it = 0, segs = 0;
    bool ok = true, first_segment = true;
    for (; !seg.done() && ok; seg.next(p), ++segs) {
      const int row0 = seg.tile * kChunkRows, rows = seg.n * p.group, row = row0 + r, tok = row / p.group;
      const bool active = row0 + warp * 32 < rows;  // a warp with a row
      if (!(ok = wait(q_full, segs & 1))) break;
      const float f = row_factor[r];
      arrive(q_empty);
      const int last = seg.m - seg.n + tok;                                 // the last slot that this row sees
      const int full = seg.m - seg.n + (row0 + warp * 32) / p.group;        // slots up to here are seen by the warp's rows
      float ref = kLow;
      float2 sum = make_float2(0.f, 0.f);
      for (int x = seg.a; x < seg.e; ++x, ++it) {
        const uint32_t b = it & 1;
        if (!(ok = wait(s_full + b, it / 2 & 1))) break;
        tc_fence_after();
        bool grow = false;
        float most = ref;
        uint32_t u[2][32];
        const int slot0 = x * kUnit;
        const uint32_t tS = tmem + lane_base + 128 * b, tP = tmem + lane_base + 384 + 64 * b;
        uint32_t have = 0xFF;
        bool plain = true;
        if (active) {
          have = have_keys[it & 3];
          plain = have == 0xFF && slot0 + kUnit - 1 <= full;
          // slots that a row does not see, or that are not there, are -inf
          auto load = [&](int half) {
            tmem_ld32(tS + 64 * half, u[0]);
            tmem_ld32(tS + 64 * half + 32, u[1]);
            tmem_ld_wait();
            if (!plain)
#pragma unroll
              for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const int at = 64 * half + 32 * c + e;
                  if (slot0 + at > last || !((have >> (at >> 4)) & 1)) u[c][e] = 0xFF800000u;
                }
          };
          float top = -INFINITY;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            load(half);
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int e = 0; e < 32; e += 2) top = max3(top, __uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1]));
          }
          top *= f;
          grow = top > ref + lag_of(ref);
          most = fmaxf(ref, reference_of(top));
        }
        // O is whole up to the unit before (within the segment; at its end the last one was waited for)
        if (x > seg.a && !(ok = wait(pv_done, (it - 1) & 1))) break;
        if (active) {
          tc_fence_after();
          if (__any_sync(0xffffffffu, grow)) {
            const float down = ex2(ref - most);
            ref = most;
            sum = mul2(sum, make_float2(down, down));
            if (x > seg.a) {
              uint32_t o[32];
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                tmem_ld32(tmem + lane_base + 256 + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * down);
                tmem_st32(tmem + lane_base + 256 + c, o);
              }
            }
          }
          const float2 f2 = make_float2(f, f), low = make_float2(-ref, -ref);
          // the upper half's scores are still here
#pragma unroll
          for (int half = 1; half >= 0; --half) {
            if (half == 0) {
              tmem_ld32(tS, u[0]);
              tmem_ld32(tS + 32, u[1]);
              tmem_ld_wait();
              if (!plain)
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    const int at = 32 * c + e;
                    if (slot0 + at > last || !((have >> (at >> 4)) & 1)) u[c][e] = 0xFF800000u;
                  }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t w[16];
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float2 y = fma2(make_float2(__uint_as_float(u[c][e]), __uint_as_float(u[c][e + 1])), f2, low);
                const float2 v = make_float2(ex2(y.x), ex2(y.y));
                sum = add2(sum, v);
                const __half2 h = __floats2half2_rn(v.x, v.y);
                memcpy(&w[e / 2], &h, 4);
              }
              tmem_st16(tP + 32 * half + 16 * c, w);
            }
          }
          tmem_st_wait();
          tc_fence_before();
        }
        arrive(p_full + b);
      }
      if (!ok) break;
      if (!(ok = wait(pv_done, (it - 1) & 1))) break;
      const bool whole = seg.a == 0 && seg.e == seg.chunks;
      const int part = 2 * blockIdx.x + (first_segment ? 0 : 1);
      if (active) {
        tc_fence_after();
        const float l = sum.x + sum.y;
        const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
        const int64_t at = (int64_t)(seg.first + tok) * p.q_heads + seg.head * p.group + (row - tok * p.group);
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          uint32_t o[32];
          __syncwarp();  // lanes without a row have gone ahead
          tmem_ld32(tmem + lane_base + 256 + c, o);
          tmem_ld_wait();
          if (row >= rows) continue;
          if (l == 0.f) {  // no slot: 0 x what is not finite must not show
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0;
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                w[y] = pack_bf16(__uint_as_float(o[e + 2 * y]) * inv, __uint_as_float(o[e + 2 * y + 1]) * inv);
              *reinterpret_cast<uint4*>(p.o + at * D + c + e) = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(p.part_o + ((int64_t)part * kChunkRows + r) * D + c + e) =
                  make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
        }
        if (row < rows) {
          if (whole) p.lse[at] = natural_lse(ref, l);
          else p.part_ml[(int64_t)part * kChunkRows + r] = make_float2(ref, l);
        }
        tc_fence_before();
      }
      if (threadIdx.x == 0) describe(p, seg, part, row0, rows, each);
      first_segment = false;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
cudaError_t launch(const AttnParams& p, int blocks, cudaStream_t stream) {
  const auto kernel = zl_kv4_chunk_kernel<D>;
  static PerDeviceOnce once;
  const cudaError_t e = once.run(
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kSmem); });
  if (e != cudaSuccess) return e;
  return launch_overlapped(kernel, blocks, kThreads, Layout<D>::kSmem, stream, p);
}

}  // namespace

cudaError_t launch_kv4_chunk(int head_dim, const AttnParams& p, int blocks, cudaStream_t stream) {
  return head_dim == 128 ? launch<128>(p, blocks, stream) : launch<64>(p, blocks, stream);
}

}  // namespace zl
