// Attention of new tokens over the 4-bit cache.
//
// With the group's query heads of all new tokens as rows r of one key head:
//   S[key, r] = scale K Q^T,  P = exp(S - max),  O^T[channel, r] = V^T P,  LSE = max + log sum P,
// one pass over the keys with the running maximum and sum of a softmax.  Bound by the cache's bytes, 1.125 d a slot and
// key head: at the copy rate an SM has 6 cycles (d = 128) for a slot, in which it has to turn 256 codes into fp16 and
// to multiply them.  So codes become operands in registers, where the matrix instructions take them:
//  - K is the A operand (16 keys x 16 channels) of m16n8k16, rows the 8 columns: a warp's products serve 8 rows at no
//    waste for small groups.  The sum over channels has any order, so lane t of a quad takes the quarter t of the
//    channels, 16 bytes of a row, and two scales serve it.
//  - S^T's accumulator becomes P's operand by one 8 x 8 transposition (movmatrix) each 8 keys.
//  - V is the A operand V^T (16 channels x 16 keys).  Its pairs run over keys: two keys' bytes become bytes of pairs
//    with four logic instructions for 16 codes, before they are turned into fp16.  Lane g takes the g-th eighth of the
//    channels, so one scale a key serves it.
//  - code * scale is exact in fp16; Q is scaled by a power of two a row so that fp16 holds its bf16 digits.
// Every warp streams runs of 32 slots of its own through shared memory (bulk copies, a ring of stages, no other warp in
// between); 4 warps of a block share a (sequence, key head, row tile) and join at its end.
// The slots of all items lie in a row that is dealt out evenly over the blocks, whatever the lengths: a block writes
// what it holds alone; items cut between blocks leave parts (O, max, sum) that a second launch joins in order.  Short
// items go to a block or a cluster of blocks each instead, which joins them itself.
// Measured, 32/8 heads, d = 128: 64 single tokens behind 1 to 16 384 slots 86 us (436 MB, 5.1 TB/s; the loads without
// arithmetic 69 us), one behind 131 071 slots 34 us and 6 for its join (151 MB).  What is above the loads is arithmetic
// that they do not hide: some 595 instructions for 32 slots, 256 of them conversions and products at half rate.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "zl_internal.h"
#include "zl_kv4_attn.cuh"
#include "zl_overlap.cuh"

namespace zl {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kUnit = 32;          // slots of a unit: two tiles
constexpr int kItemCost = 8;       // units: 64 single tokens over 15 to 16 384 slots took 98 us at 4, 87 at 8 and 12, 90 at 20
constexpr int kMaxCluster = 8;
constexpr int kMaxBlocks = 640;    // blocks of a launch at most: what the workspace has room for
constexpr uint32_t kTwice = 0x00800080u;  // a scale's bits times this: the scale in both halves (the multiplier has time)

// ---------------------------------------------------------------- pieces of a product
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The first product of a sum.
__device__ __forceinline__ void mma16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t o;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(o) : "r"(x));
  return o;
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  uint32_t o;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(o) : "f"(hi), "f"(lo));
  return o;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// Numbers of the same place in another block of the cluster.
__device__ __forceinline__ uint32_t peer_address(const void* mine, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  return a;
}
__device__ __forceinline__ float peer1(const float* mine, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_address(mine, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float2 peer2(const float2* mine, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_address(mine, rank)) : "memory");
  return v;
}
__device__ __forceinline__ float4 peer4(const float* mine, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(peer_address(mine, rank))
               : "memory");
  return v;
}

// weights_out of slots [s0, s1) of an item whose rows are all this block's: scores that it has just written, four slots
// a thread.
__device__ __forceinline__ void add_weights(const AttnParams& p, int seq, int head, int m, int n, int rows, int s0, int s1,
                                            const float* row_lse) {
  const int64_t slots = (int64_t)p.c.max_pages << p.c.page_shift, pair = (int64_t)seq * p.c.heads + head;
  const float* x = p.scores + pair * p.score_rows * slots;
  for (int s = s0 + 4 * threadIdx.x; s < s1; s += 4 * kThreads) {
    float w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = p.w_in && s + i < m - n ? p.decay * p.w_in[pair * slots + s + i] : 0.f;
#pragma unroll 4
    for (int r = 0; r < rows; ++r) {
      // slots of the table past the last one are the workspace's, too
      const float4 v = *reinterpret_cast<const float4*>(x + r * slots + s);
      const float l = row_lse[r];
      if (l == INFINITY) continue;
      w[0] += ex2(v.x - l);
      w[1] += ex2(v.y - l);
      w[2] += ex2(v.z - l);
      w[3] += ex2(v.w - l);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (s + i < s1) p.w_out[pair * slots + s + i] = w[i];
  }
}

// ---------------------------------------------------------------- the kernel
template <int D, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStageBytes = 2 * 18 * D;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kPitch = D + 4;  // floats of a row in the join's buffer
  static constexpr int kRing = kWarps * kStages * kStageBytes;
  static constexpr int kJoin = kWarps * kRows * kPitch * 4;
  static constexpr int kSmem = kRing + kJoin + kWarps * kRows * 8;
  static constexpr int kBlocks = NT == 1 || D == 64 ? 4 : 2;  // an SM's, by registers and shared memory
};

// kCluster: a cluster takes one item, each of its blocks an equal part of the units, and joins it through its blocks'
// shared memory: no second launch.  Else the items' units are dealt out evenly.  (The rule between them: cluster_of.)
template <int D, int NT, bool kScores, bool kCluster>
__global__ void __launch_bounds__(kThreads, Shape<D, NT>::kBlocks) zl_kv4_attn_kernel(const AttnParams p) {
  using S = Shape<D, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t bars[kWarps * S::kStages];
  __shared__ int64_t warp_sums[kWarps];
  __shared__ int64_t s_before;
  __shared__ int s_seq;
  __shared__ float2 block_ml[kCluster ? S::kRows : 1];
  __shared__ float row_lse[kCluster && kScores ? S::kRows : 1];  // of the rows that this block put together, then of all; base 2
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  float* join = reinterpret_cast<float*>(smem + S::kRing);
  float2* join_ml = reinterpret_cast<float2*>(smem + S::kRing + S::kJoin);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * S::kStages; ++i) mbar_init(&bars[i], 1);
    fence_mbar_init();
  }
  __syncthreads();  // every warp loads on barriers of its own, which it may do at once
  let_next_start();
  wait_for_previous();

  using W = Walk<S::kRows, kUnit, kItemCost>;
  W cons;
  int64_t each = 0;
  const uint32_t cluster = kCluster ? cluster_size() : 1;
  if constexpr (kCluster) {
    const int item = blockIdx.x / cluster, pair = item / p.max_tiles;
    cons.tile = item - pair * p.max_tiles;
    cons.seq = pair / p.c.heads;
    cons.head = pair - cons.seq * p.c.heads;
    cons.left = 0;
    cons.load(p);
    if (cons.tile >= cons.row_tiles) {  // all of the cluster
      if (kScores && p.own_weights) {
        const int64_t at = (int64_t)item * ((int64_t)p.c.max_pages << p.c.page_shift);
        for (int s = cluster_rank() * kThreads + threadIdx.x; s < cons.m; s += cluster * kThreads)
          p.w_out[at + s] = p.w_in ? p.decay * p.w_in[at + s] : 0.f;
      }
      return;
    }
    const int per = (cons.chunks + (int)cluster - 1) / (int)cluster;
    cons.a = min(cons.chunks, per * (int)cluster_rank());
    cons.e = min(cons.chunks, cons.a + per);
  } else if (!first_segment_of<kThreads, kWarps + kItemCost>(p, warp_sums, &s_before, &s_seq, cons, &each)) {
    return;
  }

  // Loading: a warp looks up the places of its next 32 units at once, one a lane, and issues them one by one.
  W prod = cons;
  int prod_x = prod.a + warp;         // the next unit to look up
  uint32_t tile0 = kKv4None, tile1 = kKv4None;  // the two tiles of a lane's unit
  int batch = 0, batch_end = 0;       // units looked up and not yet issued: lanes [batch, batch_end)
  bool any_bad = false;               // a page of this run is none of the cache's
  auto look_up = [&]() {
    batch = batch_end = 0;
    while (prod_x >= prod.e) {  // to the next segment that has a unit for this warp
      prod.next(p);
      if (prod.done()) return;
      prod_x = prod.a + warp;
    }
    const int x = prod_x + kWarps * lane, slot = x * kUnit;
    bool bad = false;
    auto place = [&](int at) {
      if (x >= prod.e || at >= prod.m) return kKv4None;
      const uint32_t tile = kv4_place(p.c, prod.seq, prod.head, at);
      bad |= tile == kKv4None;
      return tile;
    };
    tile0 = place(slot);
    tile1 = place(slot + kKv4Slots);
    if (bad) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    any_bad |= __any_sync(0xffffffffu, bad);
    batch_end = min(32, (prod.e - prod_x + kWarps - 1) / kWarps);
    prod_x += 32 * kWarps;
  };
  uint8_t* ring = smem + warp * S::kStages * S::kStageBytes;
  uint64_t* bar = bars + warp * S::kStages;
  uint32_t phases = 0;  // parity of each stage's next wait
  int fill = 0, drain = 0, in_flight = 0;
  auto produce = [&]() {
    if (batch == batch_end) {
      look_up();
      if (batch == batch_end) return;
    }
    const uint32_t t0 = __shfl_sync(0xffffffffu, tile0, batch), t1 = __shfl_sync(0xffffffffu, tile1, batch);
    ++batch;
    if (lane == 0) {
      const uint32_t dst = smem_u32(ring + fill * S::kStageBytes), b = smem_u32(&bar[fill]);
      if (t0 != kKv4None && t1 == t0 + 1) {
        mbar_arrive_expect_tx(&bar[fill], 36 * D);
        bulk_load(dst, p.c.data + (uint64_t)t0 * (18 * D), 36 * D, b);
      } else {
        mbar_arrive_expect_tx(&bar[fill], (t0 != kKv4None ? 18 * D : 0) + (t1 != kKv4None ? 18 * D : 0));
        if (t0 != kKv4None) bulk_load(dst, p.c.data + (uint64_t)t0 * (18 * D), 18 * D, b);
        if (t1 != kKv4None) bulk_load(dst + 18 * D, p.c.data + (uint64_t)t1 * (18 * D), 18 * D, b);
      }
    }
    fill = (fill + 1) % S::kStages;
    ++in_flight;
  };
#pragma unroll
  for (int i = 0; i < S::kStages; ++i) produce();

  // rows of a lane's keys in a tile: the pairs of odd lanes are swapped, so that a load of four keys' values meets both
  // halves of the banks
  const int key0 = (g & ~1) | ((g & 1) ^ ((g >> 1) & 1));  // row g of a product; row g + 8 is key0 + 8
  const int ka = 2 * t + (t & 1), kb = 2 * t + 1 - (t & 1);
  // where a lane reads in a tile: codes and scales of its keys' K (8 keys on: half of them further), and of its V
  const int k_at = key0 * (D / 2) + t * (D / 8), ks_at = 16 * D + key0 * (D / 16) + t * (D / 64);
  const int va_at = 8 * D + ka * (D / 2) + g * (D / 16), vb_at = 8 * D + kb * (D / 2) + g * (D / 16);
  const int vsa_at = 17 * D + ka * (D / 16) + g * D / 128, vsb_at = 17 * D + kb * (D / 16) + g * D / 128;
  bool first_segment = true, alive = true;
  // (a cluster's block joins with no units, too)
  for (bool more = kCluster || !cons.done(); more; cons.next(p), more = !cons.done()) {
    const int head = cons.head, row0 = cons.tile * S::kRows;
    const int rows = cons.n * p.group;
    // queries: lane (g, t) holds quarter t of the channels of row g of every 8
    uint32_t qf[NT][D / 16][2];
    float2 f[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int r = row0 + 8 * j + g;
      uint4 raw[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw[i] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        const int tok = r / p.group;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (int64_t)(cons.first + tok) * p.q_stride +
                                                          (int64_t)(head * p.group + r - tok * p.group) * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < D / 32; ++i) raw[i] = src[i];
      }
      uint32_t top = 0;  // the largest magnitude's bits
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          top = max(top, w[x] & 0x7FFF0000u);
          top = max(top, (w[x] << 16) & 0x7FFF0000u);
        }
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int ex = max(1, min(253, (int)(top >> 23)));  // 2^(ex - 127): the row's size
      const float down = __uint_as_float((uint32_t)(254 - ex) << 23), up = __uint_as_float((uint32_t)ex << 23);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int x = 0; x < 4; ++x)  // four channels are a step's
          qf[j][2 * i + x / 2][x & 1] = pack_half(__uint_as_float(w[x] << 16) * down, __uint_as_float(w[x] & 0xFFFF0000u) * down);
      }
      const float mine = fmaxf(up * p.scale_log2, 0x1p-126f);  // not 0, which -inf is multiplied by
      f[j] = make_float2(__shfl_sync(0xffffffffu, mine, 8 * t), __shfl_sync(0xffffffffu, mine, 8 * t + 4));
    }
    float acc[D / 16][NT][4];
    float2 ref[NT], sum[NT];  // of a lane's two rows of every 8
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      ref[j] = make_float2(kLow, kLow);
      sum[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) acc[i][j][0] = acc[i][j][1] = acc[i][j][2] = acc[i][j][3] = 0.f;
    }
    const int full = cons.m - cons.n + row0 / p.group;  // slots up to here are seen by every row

    for (int x = cons.a + warp; x < cons.e; x += kWarps) {
      if (!alive) continue;
      const uint8_t* stage = ring + drain * S::kStageBytes;
      alive = __all_sync(0xffffffffu, mbar_wait(&bar[drain], (phases >> drain) & 1));
      if (!alive) {
        if (lane == 0) kv4_report(p.c, ZL_KV4_TIMEOUT);
        continue;
      }
      phases ^= 1u << drain;
      drain = (drain + 1) % S::kStages;
      --in_flight;
      const int slot0 = x * kUnit;
      const bool plain = slot0 + kUnit - 1 <= full && !any_bad;
      bool have[2] = {true, true};
      if (!plain)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = slot0 + i * kKv4Slots;
          have[i] = at < cons.m && kv4_place(p.c, cons.seq, 0, at) != kKv4None;
        }
      float s[2][NT][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* tile = stage + i * 18 * D;
        uint32_t ca[D / 32], cb[D / 32], sa[2], sb[2];
        if constexpr (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(tile + k_at), b = *reinterpret_cast<const uint4*>(tile + k_at + 512);
          ca[0] = a.x; ca[1] = a.y; ca[2] = a.z; ca[3] = a.w;
          cb[0] = b.x; cb[1] = b.y; cb[2] = b.z; cb[3] = b.w;
          const uint8_t* at = tile + ks_at;
          sa[0] = at[0] * kTwice; sa[1] = at[1] * kTwice; sb[0] = at[64] * kTwice; sb[1] = at[65] * kTwice;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(tile + k_at), b = *reinterpret_cast<const uint2*>(tile + k_at + 256);
          ca[0] = a.x; ca[1] = a.y;
          cb[0] = b.x; cb[1] = b.y;
          sa[0] = sa[1] = tile[ks_at] * kTwice;
          sb[0] = sb[1] = tile[ks_at + 32] * kTwice;
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {  // a word: 8 channels, two steps
          uint32_t a[4], b[4];
          kv4_decode(ca[w], a);
          kv4_decode(cb[w], b);
          const uint32_t s2a = sa[w / 2], s2b = sb[w / 2];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            a[y] = kv4_mul(a[y], s2a);
            b[y] = kv4_mul(b[y], s2b);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int j = 0; j < NT; ++j)
            {
              if (w == 0 && y == 0) mma16_first(s[i][j], a[0], b[0], a[1], b[1], qf[j][0][0], qf[j][0][1]);
              else mma16(s[i][j], a[2 * y], b[2 * y], a[2 * y + 1], b[2 * y + 1], qf[j][2 * w + y][0], qf[j][2 * w + y][1]);
            }
        }
      }
      // slots that a row does not see, or that are not there, are -inf; the products' sums become base-2 scores by f
      if (!plain) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int last = cons.m - cons.n + (row0 + 8 * j + 2 * t + y) / p.group - slot0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!have[i] || i * 16 + key0 > last) s[i][j][y] = -INFINITY;
              if (!have[i] || i * 16 + key0 + 8 > last) s[i][j][y + 2] = -INFINITY;
            }
          }
      }
      if constexpr (kScores) {
        const int64_t slots = (int64_t)p.c.max_pages << p.c.page_shift;
        float* dst = p.scores + (((int64_t)cons.seq * p.c.heads + head) * p.score_rows + row0 + 2 * t) * slots + slot0 + key0;
        const int left = cons.m - slot0 - key0, rows_left = rows - row0 - 2 * t;
#pragma unroll
        for (int j = 0; j < NT; ++j, dst += 8 * slots) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float2 x2 = mul2(make_float2(s[i][j][2 * y], s[i][j][2 * y + 1]), f[j]);
              const bool in = 16 * i + 8 * y < left;
              if (in && 8 * j < rows_left) dst[16 * i + 8 * y] = x2.x;
              if (in && 8 * j + 1 < rows_left) dst[slots + 16 * i + 8 * y] = x2.y;
            }
        }
      }
      float2 top[NT];
      bool grow = false;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        top[j] = mul2(make_float2(max3(fmaxf(s[0][j][0], s[0][j][2]), s[1][j][0], s[1][j][2]),
                                  max3(fmaxf(s[0][j][1], s[0][j][3]), s[1][j][1], s[1][j][3])),
                      f[j]);
        const float2 most = add2(ref[j], make_float2(lag_of(ref[j].x), lag_of(ref[j].y)));
        grow |= top[j].x > most.x || top[j].y > most.y;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float2 m = top[j];
#pragma unroll
          for (int x2 = 4; x2 < 32; x2 <<= 1) {
            m.x = fmaxf(m.x, __shfl_xor_sync(0xffffffffu, m.x, x2));
            m.y = fmaxf(m.y, __shfl_xor_sync(0xffffffffu, m.y, x2));
          }
          m = make_float2(fmaxf(reference_of(m.x), ref[j].x), fmaxf(reference_of(m.y), ref[j].y));
          const float2 down = make_float2(ex2(ref[j].x - m.x), ex2(ref[j].y - m.y));
          ref[j] = m;
          sum[j] = mul2(sum[j], down);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[i][j][0] *= down.x;
            acc[i][j][1] *= down.y;
            acc[i][j][2] *= down.x;
            acc[i][j][3] *= down.y;
          }
        }
      }
      uint32_t pb[2][NT][2];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 low = make_float2(-ref[j].x, -ref[j].y);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 e0 = fma2(make_float2(s[i][j][0], s[i][j][1]), f[j], low);
          const float2 e1 = fma2(make_float2(s[i][j][2], s[i][j][3]), f[j], low);
          const float2 p0 = make_float2(ex2(e0.x), ex2(e0.y)), p1 = make_float2(ex2(e1.x), ex2(e1.y));
          sum[j] = add2(sum[j], add2(p0, p1));
          pb[i][j][0] = transpose8(pack_half(p0.x, p0.y));
          pb[i][j][1] = transpose8(pack_half(p1.x, p1.y));
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* tile = stage + i * 18 * D;
        const int keys[4] = {ka, kb, ka + 8, kb + 8};
        uint32_t v[4][D / 64], sc[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          if constexpr (D == 128) {
            const uint2 w = *reinterpret_cast<const uint2*>(tile + (y & 1 ? vb_at : va_at) + (y / 2) * 512);
            v[y][0] = w.x;
            v[y][1] = w.y;
            sc[y] = tile[(y & 1 ? vsb_at : vsa_at) + (y / 2) * 64];
          } else {
            v[y][0] = *reinterpret_cast<const uint32_t*>(tile + (y & 1 ? vb_at : va_at) + (y / 2) * 256);
            sc[y] = tile[(y & 1 ? vsb_at : vsa_at) + (y / 2) * 32];
          }
        }
        if (!plain) {
          // what lies in slots past the end may be no number: 0 times it is not 0
#pragma unroll
          for (int y = 0; y < 4; ++y)
            if (!have[i] || slot0 + i * 16 + keys[y] >= cons.m) sc[y] = 0;
        }
        const uint32_t s01 = __byte_perm(sc[0], sc[1], 0x1410) << 7, s23 = __byte_perm(sc[2], sc[3], 0x1410) << 7;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
          uint32_t a0[4], a1[4], a2[4], a3[4];
          kv4_decode((v[0][w] & 0x0F0F0F0Fu) | ((v[1][w] << 4) & 0xF0F0F0F0u), a0);
          kv4_decode(((v[0][w] >> 4) & 0x0F0F0F0Fu) | (v[1][w] & 0xF0F0F0F0u), a1);
          kv4_decode((v[2][w] & 0x0F0F0F0Fu) | ((v[3][w] << 4) & 0xF0F0F0F0u), a2);
          kv4_decode(((v[2][w] >> 4) & 0x0F0F0F0Fu) | (v[3][w] & 0xF0F0F0F0u), a3);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            a0[y] = kv4_mul(a0[y], s01);
            a1[y] = kv4_mul(a1[y], s01);
            a2[y] = kv4_mul(a2[y], s23);
            a3[y] = kv4_mul(a3[y], s23);
#pragma unroll
            for (int j = 0; j < NT; ++j) mma16(acc[4 * w + y][j], a0[y], a1[y], a2[y], a3[y], pb[i][j][0], pb[i][j][1]);
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      produce();
    }

    // the warps' parts of the segment become one
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float all = y ? sum[j].y : sum[j].x;
#pragma unroll
        for (int x2 = 4; x2 < 32; x2 <<= 1) all += __shfl_xor_sync(0xffffffffu, all, x2);
        const int row = 8 * j + 2 * t + y;
        if (g == 0) join_ml[warp * S::kRows + row] = make_float2(y ? ref[j].y : ref[j].x, all);
        float* dst = join + (warp * S::kRows + row) * S::kPitch + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; i += 2)
          *reinterpret_cast<float4*>(dst + 2 * i) =
              make_float4(acc[i][j][y], acc[i][j][y + 2], acc[i + 1][j][y], acc[i + 1][j][y + 2]);
      }
    __syncthreads();
    const bool whole = kCluster || (cons.a == 0 && cons.e == cons.chunks);
    const int part = 2 * blockIdx.x + (first_segment ? 0 : 1);
    constexpr int kLanes = D / 4;  // threads of a row
    const int c4 = threadIdx.x % kLanes;
    auto store = [&](int r, float m, float l, const float4& o) {
      const int tok = (row0 + r) / p.group;
      const int64_t at = (int64_t)(cons.first + tok) * p.q_heads + head * p.group + (row0 + r - tok * p.group);
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      *reinterpret_cast<uint2*>(p.o + at * D + 4 * c4) =
          make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
      if (c4 == 0) {
        const float lse = natural_lse(m, l);
        p.lse[at] = lse;
        // rows that see nothing: 2^(-inf) each
        if constexpr (kCluster && kScores) row_lse[r] = lse == -INFINITY ? INFINITY : lse * kLog2e;
      }
    };
    for (int r = threadIdx.x / kLanes; r < S::kRows && row0 + r < rows; r += kThreads / kLanes) {
      float m = kLow, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, join_ml[w * S::kRows + r].x);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = join_ml[w * S::kRows + r];
        const float k = ex2(ml.x - m);
        const float4 x = *reinterpret_cast<const float4*>(join + (w * S::kRows + r) * S::kPitch + 4 * c4);
        l = fmaf(ml.y, k, l);
        o = make_float4(fmaf(x.x, k, o.x), fmaf(x.y, k, o.y), fmaf(x.z, k, o.z), fmaf(x.w, k, o.w));
      }
      if (kCluster && cluster > 1) {  // the first warp's place is this thread's own
        *reinterpret_cast<float4*>(join + r * S::kPitch + 4 * c4) = o;
        if (c4 == 0) block_ml[r] = make_float2(m, l);
      } else if (whole) {
        store(r, m, l, o);
      } else {
        *reinterpret_cast<float4*>(p.part_o + ((int64_t)part * S::kRows + r) * D + 4 * c4) = o;
        if (c4 == 0) p.part_ml[(int64_t)part * S::kRows + r] = make_float2(m, l);
      }
    }
    if constexpr (kCluster) {
      if (cluster > 1) {
        __syncwarp();
        cluster_sync();
        // the blocks' parts become one, in order; a row's are put together by one block
        for (int r = cluster_rank() + cluster * (threadIdx.x / kLanes); r < S::kRows && row0 + r < rows;
             r += cluster * (kThreads / kLanes)) {
          float2 ml[kMaxCluster];
          float4 x[kMaxCluster];
#pragma unroll
          for (uint32_t i = 0; i < kMaxCluster; ++i) {
            const uint32_t from = min(i, cluster - 1);
            ml[i] = peer2(&block_ml[r], from);
            x[i] = peer4(join + r * S::kPitch + 4 * c4, from);
          }
          float m = kLow, l = 0.f;
          float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (uint32_t i = 0; i < kMaxCluster; ++i) m = fmaxf(m, ml[i].x);
#pragma unroll
          for (uint32_t i = 0; i < kMaxCluster; ++i) {
            if (i >= cluster) break;
            const float k = ex2(ml[i].x - m);
            l = fmaf(ml[i].y, k, l);
            o = make_float4(fmaf(x[i].x, k, o.x), fmaf(x[i].y, k, o.y), fmaf(x[i].z, k, o.z), fmaf(x[i].w, k, o.w));
          }
          store(r, m, l, o);
        }
        __syncwarp();
        cluster_sync();  // no block may end while another reads its shared memory
      }
      if constexpr (kScores)
        if (p.own_weights) {
          if (cluster > 1) {
            const int r = threadIdx.x;
            float mine = 0.f;
            if (r < S::kRows) mine = peer1(&row_lse[r], r % cluster);
            cluster_sync();
            if (r < S::kRows) row_lse[r] = mine;
          }
          __syncthreads();
          add_weights(p, cons.seq, head, cons.m, cons.n, rows, cons.a * kUnit, min(cons.m, cons.e * kUnit), row_lse);
        }
    } else if (threadIdx.x == 0) {
      describe(p, cons, part, row0, rows, each);
    }
    first_segment = false;
    __syncthreads();  // the join's buffer has been read
  }
  // copies still under way (after a wait that gave up): none may land in memory that is no longer this block's
  while (in_flight > 0) {
    mbar_wait(&bar[drain], (phases >> drain) & 1);
    phases ^= 1u << drain;
    drain = (drain + 1) % S::kStages;
    --in_flight;
  }
}

// ---------------------------------------------------------------- joining cut items
// kSplit: a block a row, its 8 warps share the parts (few items, each cut many times: 76 parts of a sequence of 131 071 slots
// took one warp a row 39 us); else a block 8 rows, a warp a row.
template <int D, int kRows, bool kSplit>
__global__ void __launch_bounds__(256) zl_kv4_join_kernel(const AttnParams p) {
  constexpr int kPer = D / 32;
  __shared__ float s_o[8][kSplit ? D : 1];
  __shared__ float2 s_ml[8];
  let_next_start();
  wait_for_previous();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = kSplit ? blockIdx.y : blockIdx.y * 8 + warp;
  const Cut c = p.cuts[blockIdx.x];
  if (p.by_item) {  // items without rows were not described
    const int b = blockIdx.x / (p.c.heads * p.max_tiles);
    int first;
    const int n = kv4_new(p.c, p.starts, p.n_tokens, p.max_new, b, &first);
    if ((int)(blockIdx.x % p.max_tiles) * kRows + r >= n * p.group) return;
  }
  if (c.parts == 0 || c.row0 + r >= c.rows) return;
  const int first_block = c.which >> 1;
  float m = kLow, l = 0.f, o[kPer] = {};
  auto add = [&](float m2, float l2, const float (&o2)[kPer]) {
    const float top = fmaxf(m, m2), k1 = ex2(m - top), k2 = ex2(m2 - top);
    m = top;
    l = l * k1 + l2 * k2;
#pragma unroll
    for (int x = 0; x < kPer; ++x) o[x] = o[x] * k1 + o2[x] * k2;
  };
  // parts in batches, whose loads are under way together
  constexpr int kBatch = 8, kStep = kSplit ? 8 : 1;
  for (int i0 = kSplit ? warp : 0; i0 < c.parts; i0 += kBatch * kStep) {
    float2 ml[kBatch];
    float o2[kBatch][kPer];
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const int i = min(i0 + y * kStep, c.parts - 1);
      const int64_t at = (int64_t)(i == 0 ? c.which : 2 * (first_block + i)) * kRows + r;
      ml[y] = p.part_ml[at];
      const float* src = p.part_o + at * D + lane * kPer;
      if constexpr (kPer == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        o2[y][0] = v.x; o2[y][1] = v.y; o2[y][2] = v.z; o2[y][3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        o2[y][0] = v.x; o2[y][1] = v.y;
      }
    }
#pragma unroll
    for (int y = 0; y < kBatch; ++y)
      if (i0 + y * kStep < c.parts) add(ml[y].x, ml[y].y, o2[y]);
  }
  if constexpr (kSplit) {
#pragma unroll
    for (int x = 0; x < kPer; ++x) s_o[warp][lane * kPer + x] = o[x];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      float o2[kPer];
#pragma unroll
      for (int x = 0; x < kPer; ++x) o2[x] = s_o[w][lane * kPer + x];
      add(s_ml[w].x, s_ml[w].y, o2);
    }
  }
  const int tok = (c.row0 + r) / p.group;
  const int64_t at = (int64_t)(c.token0 + tok) * p.q_heads + c.head0 + (c.row0 + r - tok * p.group);
  const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + at * D + lane * kPer);
#pragma unroll
  for (int x = 0; x < kPer; x += 2) dst[x / 2] = pack_bf16(o[x] * inv, o[x + 1] * inv);
  if (lane == 0) p.lse[at] = natural_lse(m, l);
}

// ---------------------------------------------------------------- accumulated weights
// weights_out[slot] = decay weights[slot] + sum over rows of 2^(score - lse).  A row's scores lie side by side; a thread
// takes kPer slots and has kBatch rows' loads under way at a time: four slots where rows are few, one where they are many
// and slots would not fill the SMs (48 rows over 17 000 slots and 8 heads, out of L2: 21 us with four, 10 with one; 4
// rows over 48 x 2049 slots and 8 heads 7 us).
constexpr int kWeightThreads = 128;
template <int kPer, int kBatch>
__global__ void __launch_bounds__(kWeightThreads) zl_kv4_weights_kernel(const AttnParams p) {
  let_next_start();
  wait_for_previous();
  const int b = blockIdx.z, h = blockIdx.y, s0 = blockIdx.x * kWeightThreads * kPer, s = s0 + kPer * threadIdx.x;
  extern __shared__ float lse2[];  // base-2 LSE of every row; of rows that see nothing +inf: 2^(-inf) each
  const int m = kv4_len(p.c, b);
  int first = 0;
  const int n = kv4_new(p.c, p.starts, p.n_tokens, p.max_new, b, &first), rows = n * p.group;
  if (s0 >= m) return;
  const int64_t slots = (int64_t)p.c.max_pages << p.c.page_shift, at = ((int64_t)b * p.c.heads + h) * slots + s;
  const float* x = p.scores + ((int64_t)b * p.c.heads + h) * p.score_rows * slots + s;
  float v[kBatch][kPer], w[kPer];
  auto load = [&](int r0) {  // slots of the table past the last one are the workspace's, too
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const float* from = x + (int64_t)min(r0 + y, p.score_rows - 1) * slots;
      if constexpr (kPer == 4) {
        const float4 f = *reinterpret_cast<const float4*>(from);
        v[y][0] = f.x; v[y][1] = f.y; v[y][2] = f.z; v[y][3] = f.w;
      } else {
        v[y][0] = *from;
      }
    }
  };
  const bool in = s < m;
  if (in) load(0);
#pragma unroll
  for (int i = 0; i < kPer; ++i) w[i] = p.w_in && s + i < m - n ? p.decay * p.w_in[at + i] : 0.f;
  for (int r = threadIdx.x; r < rows; r += kWeightThreads) {
    const int tok = r / p.group;
    const float l = p.lse[(int64_t)(first + tok) * p.q_heads + h * p.group + r - tok * p.group];
    lse2[r] = l == -INFINITY ? INFINITY : l * kLog2e;
  }
  __syncthreads();
  if (!in) return;
  for (int r0 = 0; r0 < rows; r0 += kBatch) {
    if (r0 > 0) load(r0);
#pragma unroll
    for (int y = 0; y < kBatch; ++y) {
      const float l = r0 + y < rows ? lse2[r0 + y] : INFINITY;
#pragma unroll
      for (int i = 0; i < kPer; ++i) w[i] += l == INFINITY ? 0.f : ex2(v[y][i] - l);
    }
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (s + i < m) p.w_out[at + i] = w[i];
}

// ---------------------------------------------------------------- host
int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

// 8-row columns of a warp's products: one where a key head has no more rows, else two, and as many passes over the
// cache as the rows need.  (Four in a pass, at two blocks an SM for their registers: 66 us instead of 54 for 32 rows
// over 16 x 4096 slots, 32/8 heads, d = 128; 31 instead of 33 at d = 64.)
int row_columns(int64_t rows) { return rows <= 8 ? 1 : 2; }

// The tensor-core kernel (zl_kv4_chunk.cu) instead: for more than two passes' rows over slots enough to pay for its
// start.  Measured (us; here / there): 32, 48, 64, 128 rows over 16 x 4096 slots of 8 key heads, d = 128: 52 / 56, 71 /
// 58, 88 / 59, 165 / 67; d = 64: 34 / 46, 44 / 46, 75 / 48.  Few slots: 64 rows over 4 x 1000 of 4 heads 10 / 20, 4 x
// 4000 17 / 22, 8 x 1000 of 8 heads 16 / 21, 8 x 2000 31 / 27; 128 rows over 4 x 2000 of 4 heads 17 / 26, 4 x 4000 29 /
// 28.  So by the product, of the slots that the table has room for, as lengths lie on the device.  Not with weights:
// its scores leave a row a thread, which costs what it gains (16 x 2000 slots of 4 heads, 64 and 128 rows: 44 / 48, 76
// / 71 at d = 128, 36 / 42, 61 / 62 at d = 64).
constexpr int64_t kChunkFrom = 33;
constexpr int64_t kChunkWork = int64_t{3} << 21;  // rows x slots x key heads
bool by_chunks(const zl_kv4_cache& c, int64_t rows, bool weights) {
  return !weights && rows >= kChunkFrom && rows * c.n_seqs * c.n_kv_heads >= kChunkWork / std::max(1, c.max_pages * c.page);
}

struct Layout {
  int64_t ml, cuts, scores, total;
  int32_t score_rows;
};
Layout layout(const zl_kv4_cache& c, int32_t group, int32_t max_new, bool weights) {
  const int64_t rows = (int64_t)group * max_new, tile = 8 * row_columns(rows);
  // room for either kernel's parts, so that a call of fewer rows or without weights fits where this one does
  const int64_t part_rows =
      2 * (rows < kChunkFrom ? kMaxBlocks * tile : std::max<int64_t>(kMaxBlocks * tile, kChunkMaxBlocks * kChunkRows));
  Layout l;
  l.ml = part_rows * c.head_dim * 4;
  l.cuts = l.ml + part_rows * 8;
  l.scores = l.cuts + round16(kMaxBlocks * (int64_t)sizeof(Cut));
  l.score_rows = (int32_t)rows;
  l.total = l.scores;
  if (weights) l.total += (int64_t)c.n_seqs * c.n_kv_heads * c.max_pages * c.page * l.score_rows * 4;
  return l;
}

zl_status check_heads(const zl_kv4_cache* c, int32_t n_q_heads, int32_t max_new) {
  if (n_q_heads < 1 || n_q_heads % c->n_kv_heads || max_new < 1) return ZL_ERR_INVALID_ARG;
  const int64_t group = n_q_heads / c->n_kv_heads;
  if (group > 128 || group * max_new > 8192) return ZL_ERR_UNSUPPORTED;
  return ZL_OK;
}

// The join behind either kernel: items may be fewer than its blocks, and described one by one.
template <int D, int kRows, typename Launch>
cudaError_t launch_joined(AttnParams& p, int blocks, cudaStream_t stream, Launch&& launch) {
  p.max_tiles = (p.max_new * p.group + kRows - 1) / kRows;
  const int64_t items = (int64_t)p.c.n_seqs * p.c.heads * p.max_tiles;
  p.by_item = items <= blocks;
  const cudaError_t e = launch();
  if (e != cudaSuccess) return e;
  const unsigned cuts = p.by_item ? (unsigned)items : (unsigned)blocks;
  if (items * 8 <= blocks) return launch_overlapped(zl_kv4_join_kernel<D, kRows, true>, dim3(cuts, kRows), 256, 0, stream, p);
  return launch_overlapped(zl_kv4_join_kernel<D, kRows, false>, dim3(cuts, kRows / 8), 256, 0, stream, p);
}

// Blocks of an item's cluster (2^n up to 8, as far as all are resident), or 0: the dealt-out form.  Clusters save its
// second launch and its search for a block's run, but let a long item wait for its own blocks alone: for slots (that
// the table has room for) of which a warp gets 8 units at most, or 5 where dealing out would have twice as many blocks.
// Measured (us, dealt out / clusters; d = 128, groups of 4, single tokens): 8 items of 300, 2000, 4000, 8000 slots 10.0
// / 5.9, 10.0 / 7.1, 10.7 / 8.7, 11.4 / 12.3; 64 items 11.2 / 7.0, 14.5 / 10.0, 15.5 / 13.7, 24.1 / 22.6; 256 items of
// 300, 1000, 8000 slots 12.9 / 8.3, 16.3 / 13.1, 59.6 / 62.2; one item of 4000, 8000 slots 9.6 / 8.5, 9.4 / 12.0.
// Single row tiles go a block each past the resident ones, too: 1024 items of 300, 1000 slots 21.9 / 18.0, 40.7 / 37.1,
// of 1 to 1024 slots 19.0 / 17.9 (row tiles of a maximum that most sequences may not reach would be blocks without
// work).
int cluster_of(int64_t items, int64_t slots, int tiles, int blocks) {
  int c = kMaxCluster;
  while (c > 1 && items * c > blocks) c /= 2;
  const int64_t units = items * 2 * kMaxCluster <= blocks ? 5 : 8;  // of a warp
  return (items <= blocks || (tiles == 1 && items <= INT32_MAX)) && slots <= c * units * kWarps * kUnit ? c : 0;
}

template <int D, int NT, bool kScores>
cudaError_t launch_clusters(const AttnParams& p, int cluster, cudaStream_t stream) {
  using S = Shape<D, NT>;
  const auto kernel = zl_kv4_attn_kernel<D, NT, kScores, true>;
  static PerDeviceOnce once;
  const cudaError_t e = once.run(
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.c.n_seqs * p.c.heads * p.max_tiles * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int D, int NT, bool kScores>
cudaError_t launch_attn(AttnParams& p, int sms, cudaStream_t stream) {
  using S = Shape<D, NT>;
  const auto kernel = zl_kv4_attn_kernel<D, NT, kScores, false>;
  static PerDeviceInt resident;
  int per_sm = 0;
  cudaError_t e = resident.get(&per_sm, [&](int, int* v) {
    cudaError_t r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (r == cudaSuccess) r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kernel, kThreads, S::kSmem);
    if (*v < 1) *v = 1;
    return r;
  });
  if (e != cudaSuccess) return e;
  const int blocks = sms * per_sm < kMaxBlocks ? sms * per_sm : kMaxBlocks;
  p.max_tiles = (p.max_new * p.group + S::kRows - 1) / S::kRows;
  const int64_t items = (int64_t)p.c.n_seqs * p.c.heads * p.max_tiles, slots = (int64_t)p.c.max_pages << p.c.page_shift;
  if (const int cluster = cluster_of(items, slots, p.max_tiles, blocks)) {
    // all of an item's rows in one cluster: no launch for the weights either (us, with it / without: 8 items of 1000
    // slots 8.4 / 7.7, 128 of 1000 13.3 / 12.0, 512 of 300 13.2 / 11.3)
    p.own_weights = kScores && p.max_tiles == 1;
    return launch_clusters<D, NT, kScores>(p, cluster, stream);
  }
  return launch_joined<D, S::kRows>(p, blocks, stream,
                                    [&] { return launch_overlapped(kernel, blocks, kThreads, S::kSmem, stream, p); });
}
template <int D, bool kScores>
cudaError_t launch_attn(AttnParams& p, int64_t rows, bool chunks, int sms, cudaStream_t stream) {
  if (kScores || !chunks)
    return row_columns(rows) == 1 ? launch_attn<D, 1, kScores>(p, sms, stream) : launch_attn<D, 2, kScores>(p, sms, stream);
  const int blocks = sms < kChunkMaxBlocks ? sms : kChunkMaxBlocks;
  return launch_joined<D, kChunkRows>(p, blocks, stream, [&] { return launch_kv4_chunk(D, p, blocks, stream); });
}

}  // namespace
}  // namespace zl

using namespace zl;

extern "C" zl_status zl_kv4_attn_workspace(const zl_kv4_cache* cache, int32_t n_q_heads, int32_t max_new, int32_t weights,
                                           int64_t* bytes) {
  Kv4 c;
  zl_status s = kv4_check(cache, &c);
  if (s != ZL_OK) return s;
  if (!bytes || (weights != 0 && weights != 1)) return ZL_ERR_INVALID_ARG;
  if ((s = check_heads(cache, n_q_heads, max_new)) != ZL_OK) return s;
  // every factor is within its own limit, their product need not be a number of bytes
  if (weights && (double)cache->n_seqs * cache->max_pages * cache->page * n_q_heads * max_new > 0x1p60) return ZL_ERR_UNSUPPORTED;
  *bytes = layout(*cache, n_q_heads / cache->n_kv_heads, max_new, weights != 0).total;
  return ZL_OK;
}

extern "C" zl_status zl_kv4_attn_fwd(const zl_kv4_cache* cache, const void* q, int64_t q_stride, int64_t n_tokens,
                                     int32_t n_q_heads, const int32_t* starts, int32_t max_new, void* o, float* lse,
                                     const float* weights, float* weights_out, float decay, void* workspace, float scale,
                                     void* stream) {
  NvtxRange range("zl_kv4_attn_fwd");
  AttnParams p{};
  zl_status s = kv4_check(cache, &p.c);
  if (s != ZL_OK) return s;
  if ((s = check_heads(cache, n_q_heads, max_new)) != ZL_OK) return s;
  if (n_tokens < 0 || n_tokens > INT32_MAX || !(scale > 0.f) || !std::isnormal(scale) || !std::isfinite(decay))
    return ZL_ERR_INVALID_ARG;
  if ((!starts && n_tokens != cache->n_seqs) || (weights && !weights_out)) return ZL_ERR_INVALID_ARG;
  if (cache->n_seqs == 0) return ZL_OK;
  if (n_tokens > 0) {  // without tokens the weights still carry over
    if ((s = kv4_check_rows(q, q_stride, (int64_t)n_q_heads * cache->head_dim)) != ZL_OK) return s;
    if (!o || !lse) return ZL_ERR_INVALID_ARG;
    if (!kv4_aligned(o, 16) || !kv4_aligned(lse, 4)) return ZL_ERR_ALIGN;
  } else if (!weights_out) {
    return ZL_OK;
  }
  if (!workspace) return ZL_ERR_INVALID_ARG;
  if (!kv4_aligned(workspace, 16) || !kv4_aligned(starts, 4) || !kv4_aligned(weights, 4) || !kv4_aligned(weights_out, 4))
    return ZL_ERR_ALIGN;
  if (weights_out && (cache->n_seqs > 65535 || cache->n_kv_heads > 65535)) return ZL_ERR_UNSUPPORTED;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  const int32_t group = n_q_heads / cache->n_kv_heads;
  const Layout l = layout(*cache, group, max_new, weights_out != nullptr);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.q_stride = q_stride;
  p.n_tokens = n_tokens;
  p.starts = starts;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  p.scores = reinterpret_cast<float*>(ws + l.scores);
  p.w_in = weights;
  p.w_out = weights_out;
  p.decay = decay;
  p.scale_log2 = scale * kLog2e;
  p.group = group;
  p.q_heads = n_q_heads;
  p.max_new = max_new;
  p.score_rows = l.score_rows;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t rows = (int64_t)group * max_new;
  cudaError_t e = cudaSuccess;
  if (n_tokens > 0) {
    const bool chunks = by_chunks(*cache, rows, weights_out != nullptr);
    if (cache->head_dim == 128)
      e = weights_out ? launch_attn<128, true>(p, rows, chunks, sms, st) : launch_attn<128, false>(p, rows, chunks, sms, st);
    else
      e = weights_out ? launch_attn<64, true>(p, rows, chunks, sms, st) : launch_attn<64, false>(p, rows, chunks, sms, st);
  }
  if (e == cudaSuccess && weights_out && cache->max_pages > 0 && !p.own_weights) {
    const int64_t slots = (int64_t)cache->max_pages * cache->page;
    const bool few = l.score_rows <= 8;
    const int block_slots = kWeightThreads * (few ? 4 : 1);
    const dim3 grid((unsigned)((slots + block_slots - 1) / block_slots), cache->n_kv_heads, cache->n_seqs);
    e = launch_overlapped(few ? zl_kv4_weights_kernel<4, 4> : zl_kv4_weights_kernel<1, 16>, grid, kWeightThreads,
                          (size_t)l.score_rows * 4, st, p);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
