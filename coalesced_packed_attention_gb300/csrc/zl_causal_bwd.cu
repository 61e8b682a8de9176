// Backward of the causal attention over packed sequences with grouped heads (sm_103a).
//
// With P = exp(scale q k^T - LSE) over the visible keys and D_i = rowsum(dO_i * O_i):
//   dV_j = sum_i P_ij dO_i,  dS_ij = P_ij (dO_i . V_j - D_i),
//   dK_j = scale sum_i dS_ij Q_i,  dQ_i = scale sum_j dS_ij K_j,
// the sums over i running over every query head of the key head's group.
//
// Query rows are packed as in the forward (row r = token r / group, head r % group), so the group's sum is the
// product's own sum over rows: a tile is 128 keys of one key head and keeps K, V in shared memory and dK, dV in
// TMEM while it walks the query blocks from the first that sees one of its keys to the sequence's last.  Where the
// tiles of a small problem do not fill the SMs evenly the planner splits such a walk; the parts' dK, dV go to the
// workspace in fp32 and the last kernel adds them.  Every dK, dV element is summed in a fixed order.  Per block:
//   S^T  = K Q_i^T      (SMEM x SMEM -> TMEM R0)   lanes = keys, columns = query rows
//   dP^T = V dO_i^T     (SMEM x SMEM -> TMEM R1)
//   softmax warpgroups (thread = key; each takes 64 columns): P^T (bf16) to TMEM over S^T, dS^T (bf16) to
//   shared memory; a key sees the columns from `first` on, so the causal mask is one comparison a column and
//   only blocks on the diagonal carry it
//   dV  += P^T dO_i     (TMEM x SMEM)
//   dQ_i = dS K         (SMEM x SMEM -> TMEM R1)
//   dK  += dS^T Q_i     (SMEM x SMEM; d = 64: TMEM x SMEM)
//   the dQ warpgroup reads dQ_i, stages it 16 KB at a time and hands each chunk to the bulk-copy engine as one
//   reduce-add into the fp32 accumulator, which a last kernel scales, rounds and writes out.
// The key tiles of one head reach a query block in an order that may differ from run to run, so dQ may differ
// in the last bits of its fp32 sum before it is rounded; dK, dV never do.
//
// Query rows past the sequence (other tokens of the packed tensors) and past tokens x group (never loaded) are
// zeroed in shared memory: their P is 0, but the products over rows would still multiply what lies there, and
// 0 x NaN is NaN.  So are key rows past the sequence.
// Rounding: P and dS are bf16 operands of their products (at most 2^-8 of the value each, independent from pair to
// pair); D is formed from the O that the forward stored, rounded to bf16; S, dP, D and every sum are fp32; dQ, dK, dV
// are rounded once.  Against 64 bits the gradients are 0.0025 off in norm, 0.0017 of that the last rounding alone.
//
// What bounds it at d = 128: shared memory.  A block moves 288 KB of operands, 64 KB of Q and dO, 32 KB of dS and 128 KB of
// staged dQ through it, 4096 cycles at 128 bytes a cycle, and a block was measured to take 4275 (2560 of them
// products); 26 487 tokens, 16/2 heads: 1470 to 1500 us, 1.28 PFLOP/s.  At d = 64 no one stage (timing-only builds of 8192 +
// 4096 tokens, 16/2 heads, when they took 474 us, 432 since: 471 without the loads of Q and dO, 462 with next to no dQ drain, 497 without exponentials, 443
// without the reads of LSE and D): products with N = 64 take 62 cycles where 32 would do, and the warps'
// loads and stores of shared memory wait behind their operands.
// Roles and budget: warps 0-7 softmax (two warpgroups), 8-11 dQ drain, 12 TMA, 13 MMA, 14-15 idle; launched with
// 128 registers a thread, traded with setmaxnreg to 136 / 152 / 88, per sub-partition 2 x 136 + 152 + 88 = 4 x 128,
// exactly the launch allocation.  TMEM (512 columns): R0 [0,128), R1 [128,256), dV [256,256+d), dK [384,384+d), and at
// d = 64 dS^T [448,512).
// (d = 64 has room for dQ columns of its own and a second stage of dS^T and dO, so that dP^T of the next block need
// not wait for the drain; built and measured, it was slower: 133.5 against 129.9 us for the step of 4109 tokens, 24/8
// heads.  Four softmax warpgroups of 32 rows each: 130 against 120.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zl_causal.h"
#include "zl_internal.h"
#include "zl_overlap.cuh"
#include "zl_ptx.cuh"

namespace zl {

namespace {

template <int D>
struct CausalBwdLayout {
  static constexpr int kBox = 128 * 128;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kK = 0;
  static constexpr int kV = kK + kTile;
  // d = 128 fills the shared memory with two stages of Q and one of dO; at d = 64 there is room to load further ahead
  // (with two and one the products waited for Q and dO 500 of a block's 3500 cycles; with three or four of dO
  // nothing waits less, and 8192 + 4096 tokens, 16/2 heads, took 460 and 465 us against 451)
  static constexpr int kQStages = D == 64 ? 4 : 2;
  static constexpr int kDOStages = D == 64 ? 2 : 1;
  static constexpr int kQ = kV + kTile;
  static constexpr int kDO = kQ + kQStages * kTile;    // a stage is free once dV has read it
  static constexpr int kDS = kDO + kDOStages * kTile;  // [128 keys][128 rows] bf16, two 128-byte-swizzled boxes
  static constexpr int kStageBytes = 128 * 32 * 4;    // one 32-column chunk of a block's dQ, fp32
  static constexpr int kStage = kDS + 2 * kBox;  // 2 staging buffers of the dQ drain
  static constexpr int kLD = kStage + 2 * kStageBytes;  // [2 block parities] -LSE*log2(e) and -D of a block's rows
  static constexpr int kBar = kLD + 2 * 2 * 128 * 4;
  static constexpr int kNumBars = 17 + 2 * kQStages + 2 * kDOStages;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 32;
  // d = 64 leaves TMEM columns for a second copy of dS^T, which dK then takes as its operand: 32 KB less a block through
  // the shared memory (training step's gradient of 4109 tokens, 24/8 heads: 78.6 against 81.3 us).  K and V kept
  // there too, as operands of S^T and dP^T, made it 84: products with N = 128 are slower from TMEM.
  static constexpr bool kDSinTmem = D == 64;
  static constexpr uint32_t kDSCol = 448;
};

constexpr float kLog2eC = 1.44269504088896340736f;
constexpr float kInfC = __builtin_huge_valf();

__device__ __forceinline__ bool cbwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit,
                                       int32_t* status) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit) {
      *abort_flag = 1;
      atomicCAS(status, 0, ZL_ERR_TIMEOUT);
      return false;
    }
  }
}

// Bulk reduce-add of fp32 from shared into global memory, tracked by this thread's bulk groups.
__device__ __forceinline__ void bulk_add_f32(float* gdst, uint32_t ssrc, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;" ::"l"(gdst), "r"(ssrc),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit_group() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// until at most one of this thread's bulk groups still has to read its source
__device__ __forceinline__ void bulk_read_all_but_1() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_all_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

constexpr uint32_t kLaunchRegs = 128;
constexpr uint32_t kSoftmaxRegs = 136, kDrainRegs = 152, kMiscRegs = 88;
static_assert(2 * kSoftmaxRegs + kDrainRegs + kMiscRegs == 4 * kLaunchRegs,
              "register split must equal the launch allocation");
template <uint32_t N>
__device__ __forceinline__ void set_regs() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "setmaxnreg takes a multiple of 8 in [24, 256]");
  if constexpr (N > kLaunchRegs)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  else if constexpr (N < kLaunchRegs)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void sts_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void tma_rows(void* dst, const void* map, uint64_t* bar, int c0, int head, int tok) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(0), "r"(head), "r"(tok), "r"(smem_u32(bar))
      : "memory");
}

// The query blocks that a key tile walks, [first, first + n), downwards from one that differs from tile to tile and
// round: tiles of one head that run side by side are then on neighbouring blocks, never the same one (they would
// contend on its dQ rows), and what they read and add to together is a few MB.  (Upwards from each tile's diagonal,
// eight heads to a key head, neighbours are 8 blocks apart, and 8192 tokens of four heads are touched every 20 us,
// past what L2 holds: 2390 us a training step of 26 487 tokens, 16/2 heads, against 2237.)
struct BwdSpan {
  int first, n, nqb, start;
  __device__ __forceinline__ int block(int step) const {
    const int b = start - step;
    return first + (b < 0 ? b + n : b);
  }
};
__device__ __forceinline__ BwdSpan walk_of(const CausalBwdTile& t, int tb) {
  BwdSpan s;
  s.nqb = (t.q_len + tb - 1) / tb;
  s.first = t.first;
  s.n = t.n;
  s.start = s.n > 0 ? s.n - 1 - t.block % s.n : 0;
  return s;
}

template <int D>
__global__ void __launch_bounds__(512, 1)
    zl_causal_bwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                         const CausalBwdParams p) {
  using L = CausalBwdLayout<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* kv_full = bar + 0;
  uint64_t* kv_empty = bar + 1;
  uint64_t* s_full = bar + 2;       // S^T of the block in TMEM R0
  uint64_t* ds_ready = bar + 3;     // dS^T in shared memory, dP^T read out of R1 (256 arrivals)
  uint64_t* dq_full = bar + 4;
  uint64_t* dq_empty = bar + 5;
  uint64_t* kv_done = bar + 6;
  uint64_t* drain = bar + 7;
  uint64_t* ld_full = bar + 8;      // LSE / D of a query block staged in shared memory
  uint64_t* p_ready = bar + 9;      // P^T in TMEM R0 (256 arrivals): the dV product may start
  uint64_t* dp_full = bar + 10;     // dP^T of the block in TMEM R1
  uint64_t* stage_full = bar + 11;  // [2] a dQ chunk written to staging buffer b (128 arrivals)
  uint64_t* stage_free = bar + 13;  // [2] the reduce-add of buffer b has read it
  uint64_t* q_full = bar + 15;      // [kQStages]
  uint64_t* q_empty = q_full + L::kQStages;
  uint64_t* do_full = q_empty + L::kQStages;  // [kDOStages]
  uint64_t* do_empty = do_full + L::kDOStages;  // dV (the last reader of dO) complete
  // stage and phase of the it-th query block's Q and dO
  auto q_stage = [](uint32_t it) { return it % L::kQStages; };
  auto q_phase = [](uint32_t it) { return (it / L::kQStages) & 1; };
  auto do_stage = [](uint32_t it) { return it % L::kDOStages; };
  auto do_phase = [](uint32_t it) { return (it / L::kDOStages) & 1; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);
  float* sLD = reinterpret_cast<float*>(smem + L::kLD);  // block parity b: LSE at 256 b, D at 256 b + 128

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  let_next_start();
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need a 1024-byte aligned base
    wait_for_previous();
    if (threadIdx.x == 0) atomicCAS(p.status, 0, ZL_ERR_UNSUPPORTED);
    return;
  }
  const int tb = tokens_per_block(p.group), box_rows = tb * p.group;
  // rows past the box are never loaded: zero once what lies there
  for (int b = 0; b < (L::kQStages + L::kDOStages) * (D / 64); ++b) {
    uint8_t* box = smem + L::kQ + b * L::kBox;  // the stages of Q and dO lie one behind the other
    for (int i = box_rows * 8 + threadIdx.x; i < 128 * 8; i += 512)
      reinterpret_cast<uint4*>(box)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(stage_full + i, 128);
      mbar_init(stage_free + i, 1);
    }
    for (int i = 0; i < L::kQStages; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
    }
    for (int i = 0; i < L::kDOStages; ++i) {
      mbar_init(do_full + i, 1);
      mbar_init(do_empty + i, 1);
    }
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, 256);
    mbar_init(ds_ready, 256);
    mbar_init(dq_full, 1);
    mbar_init(dq_empty, 128);
    mbar_init(kv_done, 1);
    mbar_init(drain, 1);
    mbar_init(ld_full, 256);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // the plan's tables are written once, before any launch: they need not wait for the kernel before this one
  const int t_begin = p.tile_ptr[blockIdx.x], t_end = p.tile_ptr[blockIdx.x + 1];
  uint32_t into_l1;
  asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(into_l1) : "l"(p.tiles + t_begin));
  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_do);
  }
  if (warp == 13) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  wait_for_previous();
  uint8_t* sK = smem + L::kK;
  uint8_t* sV = smem + L::kV;
  uint8_t* sQ = smem + L::kQ;
  uint8_t* sDO = smem + L::kDO;
  uint8_t* sDS = smem + L::kDS;

  if (warp >= 12) {
    set_regs<kMiscRegs>();
    if (warp == 12) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        const uint32_t row_bytes = (uint32_t)(D / 64) * (uint32_t)box_rows * 128u;
        uint32_t kt = 0, qit = 0, dit = 0;
        bool ok = true;
        for (int t = t_begin; t < t_end && ok; ++t) {
          const CausalBwdTile tl = p.tiles[t];
          const BwdSpan sp = walk_of(tl, tb);
          if (sp.n == 0) continue;
          if (!cbwait(kv_empty, (kt & 1) ^ 1, abort_flag, p.wait_limit, p.status)) break;
          ++kt;
          const int kvrow = tl.kv_row + tl.block * 128;
          mbar_arrive_expect_tx(kv_full, 2 * L::kTile);
          if (p.withhold_load && kt == 1) {
            // test hook: the announced bytes never arrive; a bounded wait runs out
          } else {
            for (int c = 0; c < D / 64; ++c) {
              tma_load_3d(sK + c * L::kBox, &tm_k, kv_full, 64 * c, tl.head, kvrow);
              tma_load_3d(sV + c * L::kBox, &tm_v, kv_full, 64 * c, tl.head, kvrow);
            }
          }
          for (int is = 0; is < sp.n; ++is) {
            const int tok = tl.q_row + sp.block(is) * tb;
            const uint32_t st = q_stage(qit);
            if (!cbwait(q_empty + st, q_phase(qit) ^ 1, abort_flag, p.wait_limit, p.status)) { ok = false; break; }
            mbar_arrive_expect_tx(q_full + st, row_bytes);
            for (int c = 0; c < D / 64; ++c)
              tma_rows(sQ + st * L::kTile + c * L::kBox, &tm_q, q_full + st, 64 * c, tl.head, tok);
            ++qit;
            const uint32_t ds = do_stage(dit);
            if (!cbwait(do_empty + ds, do_phase(dit) ^ 1, abort_flag, p.wait_limit, p.status)) { ok = false; break; }
            mbar_arrive_expect_tx(do_full + ds, row_bytes);
            for (int c = 0; c < D / 64; ++c)
              tma_rows(sDO + ds * L::kTile + c * L::kBox, &tm_do, do_full + ds, 64 * c, tl.head, tok);
            ++dit;
          }
        }
        if (*abort_flag) {
          // the copies in flight land before the block's shared memory goes back (a bounded wait each)
          auto settle = [](uint64_t* b, uint32_t parity) {
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(b), parity) && clock64() - t0 < 2000000) {
            }
          };
          if (kt) settle(kv_full, (kt - 1) & 1);
          for (uint32_t b = 1; b <= (uint32_t)L::kDOStages; ++b)
            if (dit >= b) settle(do_full + do_stage(dit - b), do_phase(dit - b));
          for (uint32_t b = 1; b <= (uint32_t)L::kQStages; ++b)
            if (qit >= b) settle(q_full + q_stage(qit - b), q_phase(qit - b));
        }
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------ MMA issuer (warp-uniform; one elected lane)
      constexpr uint32_t kIdSq = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdKV = idesc_bf16(128, D, false, true);
      constexpr uint32_t kIdDQ = idesc_bf16(128, D, true, true);
      const uint32_t aK = smem_u32(sK), aV = smem_u32(sV), aQ = smem_u32(sQ), aDO = smem_u32(sDO), aDS = smem_u32(sDS);
      const uint32_t tR0 = tmem, tR1 = tmem + 128, tdV = tmem + 256, tdK = tmem + 384;
      auto wait_w = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, cbwait(b, parity, abort_flag, p.wait_limit, p.status));
      };
      // low words of the operand descriptors (K-major: LBO 16 B; MN-major: LBO one 16 KB box)
      const uint32_t kK = sdesc_lo(aK, 16), kV = sdesc_lo(aV, 16), kQ = sdesc_lo(aQ, 16), kDO = sdesc_lo(aDO, 16);
      const uint32_t kDS = sdesc_lo(aDS, 16);
      const uint32_t mK = sdesc_lo(aK, L::kBox), mQ = sdesc_lo(aQ, L::kBox), mDO = sdesc_lo(aDO, L::kBox);
      const uint32_t mDS = sdesc_lo(aDS, L::kBox);
      constexpr int kNextBox = L::kBox / 16 - 4 * 2;  // K steps 0-3 lie in the first box, 4-7 in the second
      uint32_t kt = 0, qit = 0, nblocks = 0;
      bool ok = true;
      for (int t = t_begin; t < t_end && ok; ++t) {
        const CausalBwdTile tl = p.tiles[t];
        const BwdSpan sp = walk_of(tl, tb);
        if (sp.n == 0) continue;
        if (!wait_w(kv_full, kt & 1)) break;
        ++kt;
        const int kvrows = tl.kv_len - tl.block * 128;
        if (kvrows < 128) {
          zero_tile_rows<D>(aK, kvrows, lane);
          zero_tile_rows<D>(aV, kvrows, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        // rows of the sequence's last query block that belong to it
        const int last_rows = (tl.q_len - (sp.nqb - 1) * tb) * p.group;
        auto fix_rows = [&](int is, uint32_t tile) {
          if (last_rows < box_rows && sp.block(is) == sp.nqb - 1) {
            zero_tile_rows<D>(tile, last_rows, lane);
            fence_proxy_async_smem();
            __syncwarp();
          }
        };
        tc_fence_after();
        auto issue_s = [&](uint32_t st) {  // S^T = K Q^T of the query block in stage st
          const uint32_t dq = kQ + ((st * L::kTile) >> 4);
          if constexpr (D == 128) mma_ss8_w<2, kNextBox, 2, kNextBox>(tR0, kK, dq, kIdSq, 0u, s_full);
          else mma_ss4_w<2, 0, 2, 0>(tR0, kK, dq, kIdSq, 0u, s_full);
        };
        // Q, dO of the walk's block `is`, the it-th of all, have landed
        auto q_here = [&](int is, uint32_t it) -> bool {
          if (!wait_w(q_full + q_stage(it), q_phase(it))) return false;
          fix_rows(is, aQ + q_stage(it) * L::kTile);
          return true;
        };
        auto do_here = [&](int is, uint32_t it) -> bool {
          if (!wait_w(do_full + do_stage(it), do_phase(it))) return false;
          fix_rows(is, aDO + do_stage(it) * L::kTile);
          return true;
        };
        // d = 64, whose loads run ahead, waits for them before it waits for the softmax, so that a product follows that at
        // once (8192 + 4096 tokens, 16/2 heads: 432 against 440 us; at d = 128 it would be 800 against 762)
        constexpr bool kAhead = L::kDOStages > 1;
        if (!q_here(0, qit)) break;
        tc_fence_after();
        issue_s(q_stage(qit));
        if (kAhead && !do_here(0, qit)) break;
        for (int is = 0; is < sp.n; ++is) {
          const uint32_t st = q_stage(qit), ds = do_stage(qit);
          const bool next = is + 1 < sp.n;
          if (!kAhead && !do_here(is, qit)) { ok = false; break; }
          if (nblocks > 0 && !wait_w(dq_empty, (nblocks - 1) & 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ddo = kDO + ((ds * L::kTile) >> 4);  // dP^T = V dO^T
          if constexpr (D == 128) mma_ss8_w<2, kNextBox, 2, kNextBox>(tR1, kV, ddo, kIdSq, 0u, dp_full);
          else mma_ss4_w<2, 0, 2, 0>(tR1, kV, ddo, kIdSq, 0u, dp_full);
          if (kAhead && next && !q_here(is + 1, qit + 1)) { ok = false; break; }
          if (!wait_w(p_ready, nblocks & 1)) { ok = false; break; }
          tc_fence_after();
          // dV += P^T dO; P^T of rows 0-63 is packed by warpgroup 0 into R0's columns [0, 32), of rows 64-127 by
          // warpgroup 1 into [64, 96), each over S^T columns it has already read
          mma_ts8_w<8, 32, 128, 0>(tdV, tR0, mDO + ((ds * L::kTile) >> 4), kIdKV, is > 0 ? 1u : 0u, do_empty + ds);
          if (next) {
            // S^T of the next block as soon as dV has read P^T out of R0 (products run in issue order)
            if (!kAhead && !q_here(is + 1, qit + 1)) { ok = false; break; }
            tc_fence_after();
            issue_s(q_stage(qit + 1));
          }
          if (kAhead && next && !do_here(is + 1, qit + 1)) { ok = false; break; }
          if (!wait_w(ds_ready, nblocks & 1)) { ok = false; break; }
          tc_fence_after();
          // dQ = dS K (both operands MN-major), first: the drain starts on it
          mma_ss8_w<128, 0, 128, 0>(tR1, mDS, mK, kIdDQ, 0u, dq_full);
          const uint32_t dq = mQ + ((st * L::kTile) >> 4), more = is > 0 ? 1u : 0u;  // dK += dS^T Q
          if constexpr (L::kDSinTmem) mma_ts8_w<8, 0, 128, 0>(tdK, tmem + L::kDSCol, dq, kIdKV, more, q_empty + st);
          else mma_ss8_w<2, kNextBox, 128, 0>(tdK, kDS, dq, kIdKV, more, q_empty + st);
          ++qit;
          ++nblocks;
        }
        if (!ok) break;
        mma_commit_w(kv_done);
        mma_commit_w(kv_empty);
      }
      // every product has ended before the block's memory goes back, after a wait that gave up too (that wait returns at
      // once; a bounded one of its own then)
      mma_commit_w(drain);
      if (!wait_w(drain, 0)) mbar_wait(drain, 0);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ dQ drain warpgroup (thread = query row)
    set_regs<kDrainRegs>();
    constexpr int kChunks = D / 32;
    const int t_row = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t aStage = smem_u32(smem + L::kStage);
    uint32_t nblocks = 0, sit = 0;  // sit: chunks staged so far
    bool ok = true;
    for (int t = t_begin; t < t_end && ok; ++t) {
      const CausalBwdTile tl = p.tiles[t];
      const BwdSpan sp = walk_of(tl, tb);
      float* acc_hd = p.acc + (int64_t)tl.acc_block * (128 * D);
      for (int is = 0; is < sp.n; ++is) {
        if (!__all_sync(0xffffffffu, cbwait(dq_full, nblocks & 1, abort_flag, p.wait_limit, p.status))) { ok = false; break; }
        tc_fence_after();
        uint32_t u[kChunks][32];  // all of the row: R1 is released before any reduction is issued
#pragma unroll
        for (int c = 0; c < kChunks; ++c) tmem_ld32(tmem + lane_base + 128 + 32 * c, u[c]);
        tmem_ld_wait();
        tc_fence_before();
        mbar_arrive(dq_empty);  // the next block's dP^T may overwrite R1
        // chunk c (columns 32c..32c+31) of a block is 16 KB contiguous in the accumulator, [8 column
        // groups][128 rows][4]; two buffers, so one chunk is staged while the previous one is read
        float* blk = acc_hd + (int64_t)sp.block(is) * (128 * D);
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const uint32_t b = sit & 1, use = sit >> 1;
          if (!__all_sync(0xffffffffu, cbwait(stage_free + b, (use & 1) ^ 1, abort_flag, p.wait_limit, p.status))) {
            ok = false;
            break;
          }
          const uint32_t sb = aStage + b * L::kStageBytes;
#pragma unroll
          for (int g = 0; g < 8; ++g)
            sts_v4(sb + (g * 128 + t_row) * 16, u[c][4 * g], u[c][4 * g + 1], u[c][4 * g + 2], u[c][4 * g + 3]);
          fence_proxy_async_smem();
          mbar_arrive(stage_full + b);
          if (warp == 8 && lane == 0 && cbwait(stage_full + b, use & 1, abort_flag, p.wait_limit, p.status)) {
            bulk_add_f32(blk + c * (32 * 128), sb, L::kStageBytes);
            bulk_commit_group();
            bulk_read_all_but_1();  // the other buffer's reduce-add has read it
            if (sit > 0) mbar_arrive(stage_free + (b ^ 1));
          }
          ++sit;
        }
        if (!ok) break;
        ++nblocks;
      }
    }
    if (warp == 8 && lane == 0) bulk_all_done();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    // Two warpgroups share the TMEM lanes (lane = key) and split the columns: warpgroup wg takes query rows
    // [64wg, 64wg+64) of S^T and dP^T and channels [wg d/2, (wg+1) d/2) of dK and dV.
    set_regs<kSoftmaxRegs>();
    constexpr int kHalfD = D / 2;
    const int wg = warp >> 2;
    const int t_key = threadIdx.x & 127;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const int qc0 = 64 * wg;
    const int dc0 = kHalfD * wg;
    const float sl2 = p.scale_log2;
    const uint32_t aDSrow = smem_u32(sDS) + wg * L::kBox + t_key * 128;
    // warpgroup 0 stages LSE and D: thread t_key holds packed row t_key
    const int rt = t_key / p.group, rh = t_key - rt * p.group;
    uint32_t nblocks = 0, ntiles = 0;
    for (int t = t_begin; t < t_end; ++t) {
      const CausalBwdTile tl = p.tiles[t];
      const BwdSpan sp = walk_of(tl, tb);
      const int key = tl.block * 128 + t_key;
      const bool key_ok = key < tl.kv_len;
      const int64_t ld_base = (int64_t)tl.q_row * p.n_q_heads + (int64_t)tl.head * p.group + rh;
      // LSE and D of the next block's row, on their way while this block is computed: nothing may look at them before
      // they are staged
      float lse_v = -kInfC, d_v = 0.f;
      auto fetch = [&](int blk) {
        const int tok = blk * tb + rt;
        lse_v = -kInfC;
        if (rt < tb && tok < tl.q_len) {
          const int64_t i = ld_base + (int64_t)tok * p.n_q_heads;
          lse_v = p.lse[i];
          d_v = p.row_d[i];
        }
      };
      bool ok = true;
      if (wg == 0 && sp.n > 0) fetch(sp.block(0));
      for (int is = 0; is < sp.n; ++is) {
        if (wg == 0) {
          // rows past the sequence and rows that see no key (LSE = -inf) get exp2(-inf) = 0 everywhere
          const bool none = lse_v == -kInfC;
          sLD[256 * (nblocks & 1) + t_key] = none ? -kInfC : -lse_v * kLog2eC;
          sLD[256 * (nblocks & 1) + 128 + t_key] = none ? 0.f : -d_v;
        }
        mbar_arrive(ld_full);  // bounded stand-in for a barrier of both warpgroups
        if (!__all_sync(0xffffffffu, cbwait(ld_full, nblocks & 1, abort_flag, p.wait_limit, p.status))) { ok = false; break; }
        if (wg == 0 && is + 1 < sp.n) fetch(sp.block(is + 1));
        const float* sLSE = sLD + 256 * (nblocks & 1);
        const float* sD = sLSE + 128;
        // first column (query row of the block) that sees this key; 128: none
        // (clamped before the product: over 2^31 / group keys behind the block it would not fit)
        const int first = key_ok ? max(0, key - (tl.kv_len - tl.q_len) - sp.block(is) * tb) * p.group : 128;
        if (!__all_sync(0xffffffffu, cbwait(s_full, nblocks & 1, abort_flag, p.wait_limit, p.status))) { ok = false; break; }
        tc_fence_after();
        float pr[64];
        {
          uint32_t u0[32], u1[32];
          tmem_ld32(tmem + lane_base + qc0, u0);
          tmem_ld32(tmem + lane_base + qc0 + 32, u1);
          tmem_ld_wait();
          const float2 sl2v = make_float2(sl2, sl2);
          const float2* nl2 = reinterpret_cast<const float2*>(sLSE + qc0);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x0 = fma2(make_float2(__uint_as_float(u0[2 * e]), __uint_as_float(u0[2 * e + 1])), sl2v, nl2[e]);
            const float2 x1 =
                fma2(make_float2(__uint_as_float(u1[2 * e]), __uint_as_float(u1[2 * e + 1])), sl2v, nl2[16 + e]);
            pr[2 * e] = ex2(x0.x);
            pr[2 * e + 1] = ex2(x0.y);
            pr[32 + 2 * e] = ex2(x1.x);
            pr[32 + 2 * e + 1] = ex2(x1.y);
          }
          if (first > qc0) {
#pragma unroll
            for (int e = 0; e < 64; ++e)
              if (qc0 + e < first) pr[e] = 0.f;
          }
        }
        {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) pk[e] = pack_bf16(pr[2 * e], pr[2 * e + 1]);
          tmem_st32(tmem + lane_base + qc0, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_ready);

        // dP^T of this block is issued after the previous block's dQ and dK products, which read the dS^T buffer:
        // once dP^T is complete the buffer may be rewritten
        if (!__all_sync(0xffffffffu, cbwait(dp_full, nblocks & 1, abort_flag, p.wait_limit, p.status))) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t u[32];
          tmem_ld32(tmem + lane_base + 128 + qc0 + 32 * c, u);
          tmem_ld_wait();
          uint32_t pk[16];
          const float2* nd2 = reinterpret_cast<const float2*>(sD + qc0 + 32 * c);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 ds = mul2(add2(make_float2(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1])), nd2[e]),
                                   make_float2(pr[32 * c + 2 * e], pr[32 * c + 2 * e + 1]));
            pk[e] = pack_bf16(ds.x, ds.y);
          }
          if constexpr (L::kDSinTmem) tmem_st16(tmem + lane_base + L::kDSCol + 32 * wg + 16 * c, pk);
          // dS^T row t_key -> box wg of shared memory, 128-byte swizzle
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            const int chunk = 4 * c + g;
            sts_v4(aDSrow + ((chunk ^ (t_key & 7)) << 4), pk[4 * g], pk[4 * g + 1], pk[4 * g + 2], pk[4 * g + 3]);
          }
        }
        fence_proxy_async_smem();
        if constexpr (L::kDSinTmem) tmem_st_wait();
        tc_fence_before();  // the dP^T loads are complete: dQ may overwrite R1
        mbar_arrive(ds_ready);
        ++nblocks;
      }
      if (!ok) break;
      // ---- dK, dV of this tile's keys (this warpgroup's channels)
      if (sp.n > 0) {
        if (!__all_sync(0xffffffffu, cbwait(kv_done, ntiles & 1, abort_flag, p.wait_limit, p.status))) break;
        ++ntiles;
        tc_fence_after();
      }
      // Final values leave as bf16 through this warp's own 4 KB of the dS^T buffer (free: kv_done), so that a store
      // writes whole rows' pieces; a part's fp32 values go to the workspace as [column group][128 keys][4], 512 bytes a
      // store.  (A thread's own row, 16 bytes a store, kept the load/store unit busy for 2 to 4 us a tile.)
      constexpr int kPieces = kHalfD / 8, kPerStep = 32 / kPieces;
      const uint32_t buf = smem_u32(sDS) + wg * L::kBox + (warp & 3) * 4096;
      // the lane, read again: addresses formed from the one above would be held through the loop over blocks
      int ln;
      asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln));
#pragma unroll 1
      for (int m = 0; m < 2; ++m) {  // dV, dK
        const float scale = m ? p.scale : 1.f;
#pragma unroll
        for (int c = 0; c < kHalfD / 32; ++c) {
          uint32_t u[32];
          if (sp.n > 0) {
            tmem_ld32(tmem + lane_base + 256 + 128 * m + dc0 + 32 * c, u);
            tmem_ld_wait();
          } else {  // no query: the keys' gradients are empty sums
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = 0u;
          }
          if (tl.part >= 0) {  // summed, scaled and rounded by the last launch
            uint4* dst = reinterpret_cast<uint4*>(p.part) + ((int64_t)tl.part * 2 + m) * (32 * D) + (dc0 / 4 + 8 * c) * 128 + t_key;
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i * 128] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
          } else {
            auto f = [&](int e) { return __uint_as_float(u[e]) * scale; };
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sts_v4(buf + ln * 128 + (((4 * c + i) ^ (ln & 7)) << 4), pack_bf16(f(8 * i), f(8 * i + 1)),
                     pack_bf16(f(8 * i + 2), f(8 * i + 3)), pack_bf16(f(8 * i + 4), f(8 * i + 5)),
                     pack_bf16(f(8 * i + 6), f(8 * i + 7)));
          }
        }
        if (tl.part < 0) {
          __syncwarp();
          __nv_bfloat16* base = (m ? p.dk : p.dv) + (int64_t)tl.head * D + dc0 + (ln % kPieces) * 8;
          const int64_t stride = m ? p.dk_stride : p.dv_stride;
#pragma unroll
          for (int i = 0; i < 32 / kPerStep; ++i) {
            const int x = i * kPerStep + ln / kPieces, k = tl.block * 128 + (warp & 3) * 32 + x;
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(buf + x * 128 + (((ln % kPieces) ^ (x & 7)) << 4))
                         : "memory");
            if (k < tl.kv_len) *reinterpret_cast<uint4*>(base + ((int64_t)tl.kv_row + k) * stride) = v;
          }
          __syncwarp();
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// D = rowsum(dO * O): d / 8 lanes per row of the [tokens, heads, d] tensors, four rows' loads in flight; each
// block first zeroes its share of the dQ accumulator.  HBM-bound: 4 d bytes read and 4 + 4 d written a row.
template <int D>
__global__ void __launch_bounds__(256) zl_causal_pre_kernel(const __nv_bfloat16* o, const __nv_bfloat16* d_o, float* row_d,
                                                            int64_t rows, float* acc, int64_t acc4) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kUnroll = 4;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, piece = lane % kLanes;
  const int64_t nthreads = (int64_t)gridDim.x * blockDim.x;
  let_next_start();
  wait_for_previous();
  float4* z4 = reinterpret_cast<float4*>(acc);
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < acc4; i += nthreads)
    z4[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t nwarps = nthreads / 32;
  for (int64_t base = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * (kRows * kUnroll); base < rows;
       base += nwarps * (kRows * kUnroll)) {
    uint4 a[kUnroll], b[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t row = base + u * kRows + sub;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if (row < rows) {
        a[u] = reinterpret_cast<const uint4*>(o + row * D)[piece];
        b[u] = reinterpret_cast<const uint4*>(d_o + row * D)[piece];
      }
    }
    auto dot2 = [](uint32_t x, uint32_t y, float s) {
      s = fmaf(__uint_as_float(x << 16), __uint_as_float(y << 16), s);
      return fmaf(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u), s);
    };
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float s = dot2(a[u].w, b[u].w, dot2(a[u].z, b[u].z, dot2(a[u].y, b[u].y, dot2(a[u].x, b[u].x, 0.f))));
#pragma unroll
      for (int k = kLanes / 2; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
      const int64_t row = base + u * kRows + sub;
      if (piece == 0 && row < rows) row_d[row] = s;
    }
  }
}

// dQ: one block per 128-row accumulator block and 64-channel half, read in storage order, turned over in shared
// memory, scaled, rounded to bf16 and written to the rows of its tokens.  After those, one block per split key tile
// and tensor: its parts are added in order, scaled (dK), rounded and written.
template <int D>
__global__ void __launch_bounds__(256) zl_causal_finish_kernel(const CausalFinishParams p) {
  constexpr int kHalves = D / 64;
  __shared__ float4 tile[128][17];
  const int group = p.n_q_heads / p.n_kv_heads, tb = tokens_per_block(group);
  const int64_t n_slabs = p.acc_blocks * kHalves;
  let_next_start();
  wait_for_previous();
  for (int64_t sl = blockIdx.x; sl < n_slabs; sl += gridDim.x) {
    const int64_t blk = sl / kHalves;
    const int half = (int)(sl % kHalves);
    int lo = 0, hi = p.n_seqs - 1;  // last sequence whose first block is <= blk (empty ones share their start)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.seqs[mid].acc_block <= blk) lo = mid; else hi = mid - 1;
    }
    const CausalSeq sq = p.seqs[lo];
    const int nqb = (sq.q_len + tb - 1) / tb;
    const int64_t in_seq = blk - sq.acc_block;
    const int head = (int)(in_seq / nqb), qb = (int)(in_seq % nqb);
    const float4* src = reinterpret_cast<const float4*>(p.acc) + sl * (128 * 16);
    float4 x[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) x[u] = src[u * 256 + threadIdx.x];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int k = u * 256 + threadIdx.x;  // piece (column group k / 128, row k % 128)
      tile[k & 127][k >> 7] = x[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = u * 256 + threadIdx.x;  // row k / 8, 8 channels from 8 (k % 8) on
      const int r = k >> 3, c = k & 7;
      const int rt = r / group, tok = qb * tb + rt;
      if (rt < tb && tok < sq.q_len) {
        const float4 v = tile[r][2 * c], w = tile[r][2 * c + 1];
        *reinterpret_cast<uint4*>(p.dq + (sq.q_offset + tok) * p.dq_stride +
                                  ((int64_t)head * group + (r - rt * group)) * D + half * 64 + 8 * c) =
            make_uint4(pack_bf16(v.x * p.scale, v.y * p.scale), pack_bf16(v.z * p.scale, v.w * p.scale),
                       pack_bf16(w.x * p.scale, w.y * p.scale), pack_bf16(w.z * p.scale, w.w * p.scale));
      }
    }
    __syncthreads();
  }
  // the first item behind the slabs that is this block's: 32 channels of a split key tile's dV or dK, a thread for
  // half of them of one key
  constexpr int kItems = D / 32;
  int64_t it = blockIdx.x;
  if (it < n_slabs) it += (n_slabs - it + gridDim.x - 1) / gridDim.x * gridDim.x;
  for (it -= n_slabs; it < 2 * kItems * (int64_t)p.n_merges; it += gridDim.x) {
    const CausalBwdMerge m = p.merges[it / (2 * kItems)];
    const int of_k = (int)(it / kItems & 1), r = threadIdx.x & 127, g = (int)(it % kItems) * 8 + (threadIdx.x >> 7) * 4;
    const int key = m.block * 128 + r;
    if (key >= m.kv_len) continue;
    const float4* src = reinterpret_cast<const float4*>(p.part) + ((int64_t)m.slot * 2 + of_k) * (32 * D) + g * 128 + r;
    float4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int q = 0; q < m.parts; ++q) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 a = src[(int64_t)q * (2 * 32 * D) + i * 128];
        v[i].x += a.x; v[i].y += a.y; v[i].z += a.z; v[i].w += a.w;
      }
    }
    const float scale = of_k ? p.scale : 1.f;
    uint4* out = reinterpret_cast<uint4*>((of_k ? p.dk : p.dv) + ((int64_t)m.kv_row + key) * (of_k ? p.dk_stride : p.dv_stride) +
                                          (int64_t)m.head * D + 4 * g);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      out[i] = make_uint4(pack_bf16(v[2 * i].x * scale, v[2 * i].y * scale), pack_bf16(v[2 * i].z * scale, v[2 * i].w * scale),
                          pack_bf16(v[2 * i + 1].x * scale, v[2 * i + 1].y * scale),
                          pack_bf16(v[2 * i + 1].z * scale, v[2 * i + 1].w * scale));
  }
}

// Blocks of a grid-stride kernel of 256 threads: as many as can be resident at once, or fewer.
template <typename K>
int resident_grid(PerDeviceInt& resident, K kernel, int64_t blocks, int num_sms) {
  int per_sm = 0;
  resident.get(&per_sm, [&](int, int* v) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, kernel, 256, 0); });
  const int64_t cap = (int64_t)num_sms * (per_sm < 1 ? 1 : per_sm);
  return (int)(blocks < 1 ? 1 : blocks < cap ? blocks : cap);
}

}  // namespace

cudaError_t launch_causal_bwd_pre(int head_dim, const __nv_bfloat16* o, const __nv_bfloat16* d_o, float* row_d,
                                  int64_t rows, float* acc, int64_t acc_floats, int num_sms, cudaStream_t stream) {
  auto k = head_dim == 128 ? zl_causal_pre_kernel<128> : zl_causal_pre_kernel<64>;
  const int64_t by_rows = (rows + 8 * 4 * (256 / head_dim) - 1) / (8 * 4 * (256 / head_dim));
  const int64_t by_acc = (acc_floats / 4 + 255) / 256;
  static PerDeviceInt resident[2];
  return launch_overlapped(k, resident_grid(resident[head_dim == 128], k, by_rows > by_acc ? by_rows : by_acc, num_sms), 256, 0,
                           stream, o, d_o, row_d, rows, acc, acc_floats / 4);
}

cudaError_t launch_causal_bwd(int head_dim, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CausalBwdParams& p, int grid, bool early, cudaStream_t stream) {
  const int smem = head_dim == 128 ? CausalBwdLayout<128>::kBytes : CausalBwdLayout<64>::kBytes;
  const int smem_launch = smem > 120 * 1024 ? smem : 120 * 1024;  // one CTA per SM (TMEM 512 columns)
  auto k = head_dim == 128 ? zl_causal_bwd_kernel<128> : zl_causal_bwd_kernel<64>;
  static PerDeviceOnce configured[2];
  cudaError_t e = configured[head_dim == 128].run([&] {
    cudaError_t r = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_launch);
    if (r != cudaSuccess) return r;
    // the register split adds up to exactly the launch allocation: a kernel built with another per-thread count
    // would leave an increase waiting for registers forever
    cudaFuncAttributes fa;
    r = cudaFuncGetAttributes(&fa, k);
    if (r != cudaSuccess) return r;
    return fa.numRegs == (int)kLaunchRegs ? cudaSuccess : cudaErrorInvalidKernelImage;
  });
  if (e != cudaSuccess) return e;
  return launch_overlapped_if(early, k, grid, 512, smem_launch, stream, tq, tk, tv, tdo, p);
}

cudaError_t launch_causal_finish(int head_dim, const CausalFinishParams& p, int num_sms, cudaStream_t stream) {
  const int64_t items = p.acc_blocks * (head_dim / 64) + 2 * (head_dim / 32) * (int64_t)p.n_merges;
  if (items == 0) return cudaSuccess;
  auto k = head_dim == 128 ? zl_causal_finish_kernel<128> : zl_causal_finish_kernel<64>;
  static PerDeviceInt resident[2];
  return launch_overlapped(k, resident_grid(resident[head_dim == 128], k, items, num_sms), 256, 0, stream, p);
}

}  // namespace zl
