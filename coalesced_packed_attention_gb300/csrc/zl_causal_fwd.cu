// Forward of the causal attention over packed sequences with grouped heads (sm_103a).
//
// Query i of a sequence with n queries and m keys sees the keys j <= m - n + i (the last query sees
// all of them).  For every query head h, with the key head h / group:
//   S = scale q k^T over the visible keys,  O = softmax(S) V,  LSE = ln sum exp S;
// a query that sees no key gets O = 0 and LSE = -inf.
//
// Rows: the query heads that share a key head are packed into one block, row r = (token r / group, head
// r % group), so a block of 128 rows needs each of its key head's K and V tiles once however many query
// heads read them, and a single new token of a sequence still fills `group` rows.  TMA gathers such a block
// directly from [tokens, heads, d]: its box is 64 channels x group heads x 1 key head x 128 / group tokens.
//
// Tile: two neighbouring query blocks (sub-tiles) over a range of 128-key blocks; they share the K/V tiles, and
// the later sub-tile sees as many blocks as the earlier one or more.  Two softmax warpgroups, one per sub-tile,
// work in turn against the tensor core (PV0_{j-1} S0_j PV1_{j-1} S1_j ...), S and P in TMEM, O accumulated in
// TMEM.  S_w,j is issued after PV_w,{j-1}, so the commit that signals S_w,j also says that O_w is stable: the
// warpgroup may rescale its O row at once.  Only blocks on the diagonal and the sequence's last, partial block
// are masked; blocks that no row of a sub-tile sees are not computed.
// The tiles of every thread block are laid down by the planner (longest first, greedily balanced), so launches
// share no counter: two of them may run at once from one plan, and a captured graph replays without a reset.
// Few rows over many keys (single tokens, short chunks) leave SMs idle: the planner then splits the key range of a
// tile, the parts write fp32 O (normalised by their own sum) and LSE to the workspace, and the merge kernel
// below weighs them by exp(LSE_c - LSE).
//
// Tiles follow one another without a pause: the last PV of a tile is issued between the first scores of the next, a
// third warpgroup takes O out of TMEM (the next tile's first PV waits for that alone), scales and stores it.
// Rounding: S, the running maximum and sum, O and LSE are fp32.  P is rounded to bf16 because it is an operand of
// the PV product (at most 2^-8 of a weight, independent from key to key); its sum is taken before the rounding.
// Against 64 bits O is 0.0020 off in norm, 0.0016 of that the last rounding alone.
//
// What bounds it: the chain of one sub-tile, S (512 cycles at d = 128), softmax (1300), PV (512) and the hand-overs between
// them, 2970 cycles a step of two sub-tiles with 2048 of products; a softmax step is 64 pairs at 13 cycles (two
// exponentials, scale, sum and rounding share the issue ports: 10.6 cycles a pair with two warps, measured apart) and the
// row maximum.  One prompt of 16 384 tokens, 32/4 heads: 1.43 to 1.46 ms, 1.5 PFLOP/s, at the board's power limit.
// Scores computed ahead of PV, which d = 64 has the TMEM columns for, were slower (8192 tokens, 20/4 heads: 225 us against
// 195): both warpgroups then form exponentials at the same time instead of in turn.  So do the weights handed to PV in two
// parts (packed batch 261 us against 249).
// Single tokens over long caches are HBM-bound: 64 sequences, 1.5 GB of keys and values, 237 to 240 us, 6.5 TB/s.
// Roles (512 threads, one CTA per SM): warps 0-3 and 4-7 the two softmax warpgroups (thread = TMEM lane = row),
// 8-11 output, 12 TMA, 13 MMA, 14 and 15 idle.  TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d),
// O1 [384,384+d).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zl_causal.h"
#include "zl_internal.h"
#include "zl_overlap.cuh"
#include "zl_ptx.cuh"

namespace zl {

namespace {

template <int D>
struct CausalFwdLayout {
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kBox = 128 * 128;     // one box of up to 128 rows x 128 bytes
  static constexpr int kTile = 128 * D * 2;  // one bf16 [128, D] tile
  static constexpr int kQ = 0;               // Q0, Q1
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kOutWarp = 32 * D * 2;  // 32 rows of O for each output warp
  static constexpr int kOut = kV + kStages * kTile;
  static constexpr int kStat = kOut + 4 * kOutWarp;  // [sub-tile][row] {1 / l, LSE}
  static constexpr int kBar = kStat + 2 * 128 * 8;
  static constexpr int kNumBars = 15 + 2 + 4 * kStages;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16;
};

constexpr float kGrow = 8.0f;  // O is rescaled only when the row maximum grows by more than 2^8
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kNegInf = -__builtin_huge_valf();

// Bounded wait of one barrier; on expiry the status word says so and every role leaves its loop.
__device__ __forceinline__ bool cwait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, long long limit,
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

// Brings the next tile's record into L1 while this one is computed.
__device__ __forceinline__ void touch(const CausalTile* t) {
  uint32_t x;
  asm volatile("ld.global.ca.u32 %0, [%1];" : "=r"(x) : "l"(t));
}

// What a tile's two sub-tiles cover.
struct FwdSpan {
  int tok[2];   // first token of the sub-tile within its sequence
  int toks[2];  // its tokens (0: none)
  int n[2];     // key blocks that some row of it sees, from the tile's first block on
  int nmax;
};
__device__ __forceinline__ FwdSpan span_of(const CausalTile& t, int tb) {
  FwdSpan s;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    s.tok[w] = (t.block + w) * tb;
    s.toks[w] = max(0, min(tb, t.q_len - s.tok[w]));
    const int seen = max(0, t.kv_len - t.q_len + s.tok[w] + s.toks[w]);  // keys the last of its tokens sees
    s.n[w] = s.toks[w] > 0 ? max(0, min((seen + 127) >> 7, t.kv_hi) - t.kv_lo) : 0;
  }
  s.nmax = max(s.n[0], s.n[1]);
  return s;
}

__device__ __forceinline__ void tma_load_4d(void* dst, const void* map, uint64_t* bar, int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
      : "memory");
}

// Launched with 128 registers a thread (four warps to a sub-partition); the softmax warpgroups, which hold a row's
// 128 scores, take 176, the output warpgroup keeps 88 and the warps that issue 72: per sub-partition 2 x 176 + 88 +
// 72 = 4 x 128, the launch allocation.
constexpr int kFwdThreads = 512;
constexpr uint32_t kFwdLaunchRegs = 128, kFwdSoftmaxRegs = 176, kFwdOutRegs = 88, kFwdIssueRegs = 72;
static_assert(2 * kFwdSoftmaxRegs + kFwdOutRegs + kFwdIssueRegs == 4 * kFwdLaunchRegs,
              "register split must equal the launch allocation");

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    zl_causal_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const CausalFwdParams p) {
  using L = CausalFwdLayout<D>;
  constexpr int S = L::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem + L::kQ;
  uint8_t* sK = smem + L::kK;
  uint8_t* sV = smem + L::kV;
  float2* sStat = reinterpret_cast<float2*>(smem + L::kStat);
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bar;           // [2] one per sub-tile, as all pairs below
  uint64_t* q_empty = bar + 2;      // the sub-tile's last scores are done with Q
  uint64_t* s_full = bar + 4;
  uint64_t* p_full = bar + 6;
  uint64_t* o_full = bar + 8;       // last PV of a tile done
  uint64_t* o_free = bar + 10;      // O has been read out of TMEM
  uint64_t* stat_full = bar + 12;
  uint64_t* stat_empty = bar + 14;
  uint64_t* drain = bar + 16;
  uint64_t* k_full = bar + 17;      // [S]
  uint64_t* k_empty = k_full + S;
  uint64_t* v_full = k_empty + S;
  uint64_t* v_empty = v_full + S;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  let_next_start();
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled layouts need a 1024-byte aligned base
    wait_for_previous();
    if (threadIdx.x == 0) atomicCAS(p.status, 0, ZL_ERR_UNSUPPORTED);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(q_empty + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_full + i, 1);
      mbar_init(o_free + i, 128);
      mbar_init(stat_full + i, 128);
      mbar_init(stat_empty + i, 128);
    }
    for (int s = 0; s < S; ++s) {
      mbar_init(k_full + s, 1);
      mbar_init(k_empty + s, 1);
      mbar_init(v_full + s, 1);
      mbar_init(v_empty + s, 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // the plan's tables are written once, before any launch: they need not wait for the kernel before this one
  const int t_begin = p.tile_ptr[blockIdx.x], t_end = p.tile_ptr[blockIdx.x + 1];
  touch(p.tiles + t_begin);
  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
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
  const long long lim = p.wait_limit;
  const int tb = tokens_per_block(p.group);

  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFwdIssueRegs));
    if (warp == 12) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        const uint32_t q_bytes = (uint32_t)(D / 64) * (uint32_t)(tb * p.group) * 128u;
        uint32_t k_it = 0, v_it = 0, q_it[2] = {0, 0};
        bool ok = true;
        for (int t = t_begin; t < t_end && ok; ++t) {
          const CausalTile tl = p.tiles[t];
          const FwdSpan sp = span_of(tl, tb);
          const int kv0 = tl.kv_row + tl.kv_lo * 128;
          for (int j = 0; j < sp.nmax && ok; ++j) {
            const uint32_t s = k_it % S, ph = (k_it / S) & 1;
            if (!cwait(k_empty + s, ph ^ 1, abort_flag, lim, p.status)) { ok = false; break; }
            mbar_arrive_expect_tx(k_full + s, L::kTile);
            if (p.withhold_load && k_it == 0) {
              // test hook: the announced bytes never arrive; a bounded wait runs out
            } else {
              for (int c = 0; c < D / 64; ++c)
                tma_load_3d(sK + s * L::kTile + c * L::kBox, &tm_k, k_full + s, 64 * c, tl.head, kv0 + j * 128);
            }
            ++k_it;
            // the queries behind the first keys: their place is free once the previous tile's last scores are done
            for (int w = 0; w < 2 && j == 0; ++w) {
              if (sp.n[w] == 0) continue;
              if (!cwait(q_empty + w, (q_it[w] & 1) ^ 1, abort_flag, lim, p.status)) { ok = false; break; }
              mbar_arrive_expect_tx(q_full + w, q_bytes);
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(sQ + w * L::kTile + c * L::kBox, &tm_q, q_full + w, 64 * c, 0, tl.head, tl.q_row + sp.tok[w]);
              ++q_it[w];
            }
            if (!ok) break;
            if (!cwait(v_empty + s, ph ^ 1, abort_flag, lim, p.status)) { ok = false; break; }
            mbar_arrive_expect_tx(v_full + s, L::kTile);
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sV + s * L::kTile + c * L::kBox, &tm_v, v_full + s, 64 * c, tl.head, kv0 + j * 128);
            ++v_it;
          }
        }
        if (*abort_flag) {
          // the copies in flight land before the block's shared memory goes back (a bounded wait each)
          auto settle = [](uint64_t* b, uint32_t parity) {
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(b), parity) && clock64() - t0 < 2000000) {
            }
          };
          for (int w = 0; w < 2; ++w)
            if (q_it[w]) settle(q_full + w, (q_it[w] - 1) & 1);
          for (uint32_t b = 1; b <= (uint32_t)S; ++b) {
            if (k_it >= b) settle(k_full + (k_it - b) % S, ((k_it - b) / S) & 1);
            if (v_it >= b) settle(v_full + (v_it - b) % S, ((v_it - b) / S) & 1);
          }
        }
      }
    } else if (warp == 13) {
      // ------------------------------------------------------------ MMA issuer
      // The whole warp runs the loop (control flow, waits and descriptors are warp-uniform); one elected lane
      // executes each product and commit.  A block's PV is issued behind the next block's waits, between that
      // block's scores; "next" may be the next tile's first.
      constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
      const uint32_t aV = smem_u32(sV);
      // low words of the operand descriptors (all share the high word)
      const uint32_t dQ0 = sdesc_lo(smem_u32(sQ), 16), dK0 = sdesc_lo(smem_u32(sK), 16), dV0 = sdesc_lo(aV, L::kBox);
      constexpr int kNextBox = L::kBox / 16 - 4 * 2;  // K steps 0-3 lie in the first box, 4-7 in the second
      uint32_t kv_it = 0, q_it[2] = {0, 0}, p_it[2] = {0, 0}, o_it[2] = {0, 0};
      bool ok = true;
      auto wait_w = [&](uint64_t* b, uint32_t parity) {
        return __all_sync(0xffffffffu, cwait(b, parity, abort_flag, lim, p.status));
      };
      // Q of the next tile is waited for ahead of the weights of this tile's last block at d = 64, behind them at d = 128
      // (8192 + 4096 tokens, 16/2 heads, ahead against behind: 176 and 181 us at d = 64, 239 and 228 at d = 128)
      constexpr bool kQAhead = D == 64;
      // the block whose PV is still to be issued
      bool pend = false, pend_w[2] = {false, false}, first = false, last[2] = {false, false};
      int vrows = 128;
      auto issue_v = [&]() -> bool {  // its values have landed
        const uint32_t ps = (kv_it - 1) % S;
        if (!wait_w(v_full + ps, ((kv_it - 1) / S) & 1)) return false;
        // value rows past the sequence's keys are other tokens: their weights are zero, but 0 x NaN is not
        if (vrows < 128) {
          zero_tile_rows<D>(aV + ps * L::kTile, vrows, lane);
          fence_proxy_async_smem();
          __syncwarp();
        }
        return true;
      };
      auto issue_pv = [&](int w) -> bool {
        const uint32_t ps = (kv_it - 1) % S;
        if (first) {  // O of the previous tile has left TMEM
          if (!wait_w(o_free + w, (o_it[w] & 1) ^ 1)) return false;
          ++o_it[w];
        }
        if (!wait_w(p_full + w, p_it[w] & 1)) return false;
        ++p_it[w];
        tc_fence_after();
        mma_ts8_w<8, 0, 128, 0>(tmem + 256 + 128 * w, tmem + 128 * w, dV0 + ((ps * L::kTile) >> 4), kIdPV, first ? 0u : 1u);
        if (last[w]) mma_commit_w(o_full + w);
        return true;
      };
      for (int t = t_begin; t < t_end && ok; ++t) {
        const CausalTile tl = p.tiles[t];
        const FwdSpan sp = span_of(tl, tb);
        for (int j = 0; j < sp.nmax; ++j) {
          const uint32_t s = kv_it % S, ph = (kv_it / S) & 1;
          if (!wait_w(k_full + s, ph) || (pend && !issue_v())) { ok = false; break; }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            auto q_here = [&]() -> bool {
              if (j > 0 || sp.n[w] == 0) return true;
              return wait_w(q_full + w, q_it[w]++ & 1);
            };
            if (kQAhead && !q_here()) { ok = false; break; }
            if (pend && pend_w[w] && !issue_pv(w)) { ok = false; break; }
            if (j < sp.n[w]) {
              if (!kQAhead && !q_here()) { ok = false; break; }
              tc_fence_after();
              const uint32_t dq = dQ0 + ((w * L::kTile) >> 4), dk = dK0 + ((s * L::kTile) >> 4);
              if constexpr (D == 128) mma_ss8_w<2, kNextBox, 2, kNextBox>(tmem + 128 * w, dq, dk, kIdS, 0u);
              else mma_ss4_w<2, 0, 2, 0>(tmem + 128 * w, dq, dk, kIdS, 0u);
              mma_commit_w(s_full + w);
              if (j == sp.n[w] - 1) mma_commit_w(q_empty + w);
            }
          }
          if (!ok) break;
          if (pend) mma_commit_w(v_empty + (kv_it - 1) % S);
          mma_commit_w(k_empty + s);
          pend = true;
          first = j == 0;
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            pend_w[w] = j < sp.n[w];
            last[w] = j == sp.n[w] - 1;
          }
          vrows = tl.kv_len - (tl.kv_lo + j) * 128;
          ++kv_it;
        }
      }
      if (ok && pend && issue_v()) {
        for (int w = 0; w < 2; ++w)
          if (pend_w[w] && !issue_pv(w)) break;
      }
      // every product has ended before the block's memory goes back, after a wait that gave up too (that wait returns at
      // once; a bounded one of its own then)
      mma_commit_w(drain);
      if (!wait_w(drain, 0)) mbar_wait(drain, 0);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ output warpgroup (thread = row of a sub-tile)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFwdOutRegs));
    const int r = threadIdx.x & 127, rt = r / p.group, rh = r - rt * p.group;  // its token and head
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t buf = smem_u32(smem + L::kOut) + (warp & 3) * L::kOutWarp;
    constexpr int kPieces = D / 8, kPerStep = 32 / kPieces;  // 16-byte pieces of a row, rows of a store
    // piece c of row x lies at c ^ (x mod 8) (within 128 bytes), free of bank conflicts for a row's writer and for a
    // store's readers
    auto at = [&](int x, int c) { return buf + x * (D * 2) + (c >> 3) * 128 + (((c & 7) ^ (x & 7)) << 4); };
    uint32_t it[2] = {0, 0};
    bool ok = true;
    for (int t = t_begin; t < t_end && ok; ++t) {
      const CausalTile tl = p.tiles[t];
      const FwdSpan sp = span_of(tl, tb);
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (sp.toks[w] == 0) continue;
        const bool row_ok = rt < sp.toks[w];
        float2 st = make_float2(0.f, kNegInf);  // no key: O = 0, LSE = -inf
        if (sp.n[w] > 0) {
          // this wait alone lasts a whole tile, up to 2^24 steps of 3200 cycles: 64 times the limit (a role that is stuck
          // gives up at its own limit, and that ends this wait as well)
          if (!__all_sync(0xffffffffu, cwait(stat_full + w, it[w] & 1, abort_flag, lim << 6, p.status) &&
                                           cwait(o_full + w, it[w] & 1, abort_flag, lim, p.status))) { ok = false; break; }
          ++it[w];
          st = sStat[128 * w + r];
          mbar_arrive(stat_empty + w);
          tc_fence_after();
        }
        const int64_t row = ((int64_t)tl.q_row + sp.tok[w] + rt) * p.n_q_heads + (int64_t)tl.head * p.group + rh;
        const int64_t prow = (int64_t)tl.part * 256 + 128 * w + r;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          if (sp.n[w] > 0) {
            tmem_ld32(tmem + lane_base + 256 + 128 * w + 32 * c, u);
            tmem_ld_wait();
          }
          // a row without a key beside rows with some: its weights were all zero, and 0 x Inf or NaN of a value that
          // it does not see must not show
          if (st.x == 0.f) {
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = __uint_as_float(u[8 * i + e]) * st.x;
            if (tl.part < 0) {
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane, 4 * c + i)), "r"(pack_bf16(f[0], f[1])),
                           "r"(pack_bf16(f[2], f[3])), "r"(pack_bf16(f[4], f[5])), "r"(pack_bf16(f[6], f[7]))
                           : "memory");
            } else if (row_ok) {  // [column group][128 rows][4]: a store writes 512 bytes in a row
              float4* dst = reinterpret_cast<float4*>(p.part_o) + ((int64_t)tl.part * 2 + w) * (32 * D) + (8 * c + 2 * i) * 128 + r;
              dst[0] = make_float4(f[0], f[1], f[2], f[3]);
              dst[128] = make_float4(f[4], f[5], f[6], f[7]);
            }
          }
        }
        if (sp.n[w] > 0) {
          tc_fence_before();
          mbar_arrive(o_free + w);  // the next tile's first PV may overwrite O
        }
        if (row_ok) {
          if (tl.part < 0) p.lse[row] = st.y;
          else p.part_lse[prow] = st.y;
        }
        if (tl.part < 0) {
          // a store writes whole rows (two at d = 128): a piece of 32 rows a store kept the load/store unit busy for
          // 2900 cycles a tile
          __syncwarp();
          const int rel = row_ok ? rt * p.n_q_heads + rh : -1;
          __nv_bfloat16* base = p.o + (row - (rt * p.n_q_heads + rh)) * D + (lane % kPieces) * 8;
#pragma unroll 4
          for (int i = 0; i < 32 / kPerStep; ++i) {
            const int x = i * kPerStep + lane / kPieces;
            const int to = __shfl_sync(0xffffffffu, rel, x);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(at(x, lane % kPieces))
                         : "memory");
            if (to >= 0) *reinterpret_cast<uint4*>(base + (int64_t)to * D) = v;
          }
          __syncwarp();  // the buffer is written again
        }
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFwdSoftmaxRegs));
    const int w = warp >> 2;          // sub-tile of this warpgroup
    const int r = threadIdx.x & 127;  // row of the sub-tile == TMEM lane
    const int rt = r / p.group;       // its token
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_base + 128 * w;
    const uint32_t tO = tmem + lane_base + 256 + 128 * w;
    const float sl2 = p.scale_log2;
    uint32_t sc = 0, tiles_done = 0;
    for (int t = t_begin; t < t_end; ++t) {
      const CausalTile tl = p.tiles[t];
      if (t + 1 < t_end && lane == 0) touch(p.tiles + t + 1);
      const FwdSpan sp = span_of(tl, tb);
      const int toks = w ? sp.toks[1] : sp.toks[0], n = w ? sp.n[1] : sp.n[0];
      if (n == 0) continue;
      // keys this row sees, from the tile's first block on; rows that are not stored need no mask
      const int seen = rt < toks ? max(0, tl.kv_len - tl.q_len + (w ? sp.tok[1] : sp.tok[0]) + rt + 1) - tl.kv_lo * 128 : 0x7fffffff;

      float m_used = kNegInf, l = 0.f;
      bool ok = true;
      for (int j = 0; j < n; ++j) {
        if (!__all_sync(0xffffffffu, cwait(s_full + w, sc & 1, abort_flag, lim, p.status))) { ok = false; break; }
        ++sc;
        tc_fence_after();
        float s[128];
        {
          uint32_t u[4][32];  // all four loads in flight, one wait
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, u[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) s[32 * c + e] = __uint_as_float(u[c][e]);
        }
        const int valid = seen - j * 128;
        if (valid < 128) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= valid) s[c] = kNegInf;
        }
        // row maximum as 8 independent chains of three-input maxima; chain e takes s[e + 8k]
        float mx8[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float m = max3(s[e], s[e + 8], s[e + 16]);
#pragma unroll
          for (int k = 3; k < 15; k += 2) m = max3(m, s[e + 8 * k], s[e + 8 * k + 8]);
          mx8[e] = fmaxf(m, s[e + 120]);
        }
        const float mx = fmaxf(max3(mx8[0], mx8[1], mx8[2]), max3(max3(mx8[3], mx8[4], mx8[5]), mx8[6], mx8[7]));
        const float m_blk = mx * sl2;
        const bool need = m_blk > m_used + kGrow;
        const bool rescale = j > 0 && __any_sync(0xffffffffu, need);
        const float f = need ? ex2(m_used - m_blk) : 1.f;  // exp2(-inf) = 0 on the first block
        if (need) { l *= f; m_used = m_blk; }
        // a row that has seen no key yet keeps m = -inf: its exponents are taken against 0, all exp2(-inf)
        const float nmv = m_used == kNegInf ? 0.f : -m_used;
        float2 sum4[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        const float2 sl2v = make_float2(sl2, sl2), nm = make_float2(nmv, nmv);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 x = fma2(make_float2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), sl2v, nm);
            const float2 pp = make_float2(ex2(x.x), ex2(x.y));
            sum4[e & 3] = add2(sum4[e & 3], pp);
            pk[e] = pack_bf16(pp.x, pp.y);
          }
          tmem_st16(tS + 16 * c, pk);
        }
        l += ((sum4[0].x + sum4[0].y) + (sum4[1].x + sum4[1].y)) + ((sum4[2].x + sum4[2].y) + (sum4[3].x + sum4[3].y));
        if (rescale) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(tO + 32 * c, u);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(__uint_as_float(u[e]) * f);
            tmem_st32(tO + 32 * c, u);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(p_full + w);
      }
      if (!ok) break;
      // ---- 1 / l and LSE for the output warpgroup.  l > 0 wherever the row saw a key (its largest weight is >=
      // 2^-8); a NaN sum stays NaN.
      if (!__all_sync(0xffffffffu, cwait(stat_empty + w, (tiles_done & 1) ^ 1, abort_flag, lim, p.status))) break;
      ++tiles_done;
      sStat[128 * w + r] = make_float2(l == 0.f ? 0.f : __frcp_rn(l), l == 0.f ? kNegInf : (m_used + lg2(l)) * kLn2);
      mbar_arrive(stat_full + w);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Combine of a tile's parts: LSE = M + ln sum_c exp(LSE_c - M), O = sum_c exp(LSE_c - LSE) O_c.  A block takes 32
// channels of a sub-tile of one split tile, a thread for each row: the parts' rows lie side by side, so that a
// load reads 512 bytes in a row.  The next part's values are on their way while one is added.  Where no split tile has
// over 32 rows (single tokens: many parts, few rows) the four warps take every fourth part of the same rows and the
// sums are joined in shared memory.  Every order is fixed.
template <int D, bool kFew>
__global__ void __launch_bounds__(128) zl_causal_merge_kernel(const CausalMergeParams p) {
  constexpr int kWays = kFew ? 4 : 1;
  let_next_start();
  wait_for_previous();
  const CausalMerge G = p.groups[blockIdx.x];
  const int r = kFew ? threadIdx.x & 31 : threadIdx.x, way = kFew ? threadIdx.x >> 5 : 0, w = blockIdx.z, c0 = blockIdx.y * 32;
  const int tb = tokens_per_block(p.group), rt = r / p.group, tok = (G.block + w) * tb + rt;
  const bool there = rt < tb && tok < G.q_len;
  float acc[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  float base = 0.f, tot = 0.f;
  if (there) {
    const float* pl = p.part_lse + (int64_t)G.slot * 256 + 128 * w + r;
    const float4* po = reinterpret_cast<const float4*>(p.part_o) + ((int64_t)G.slot * 2 + w) * (32 * D) + (c0 / 4) * 128 + r;
    float4 x[8];
    if (way < G.parts) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = po[(int64_t)way * (2 * 32 * D) + i * 128];
    }
    float m = kNegInf;
#pragma unroll 8
    for (int c = 0; c < G.parts; ++c) m = fmaxf(m, pl[(int64_t)c * 256]);
    base = m == kNegInf ? 0.f : m;
#pragma unroll 8
    for (int c = 0; c < G.parts; ++c) tot += expf(pl[(int64_t)c * 256] - base);
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    for (int c = way; c < G.parts; c += kWays) {
      const float wc = expf(pl[(int64_t)c * 256] - base) * inv;
      float4 y[8];
      if (c + kWays < G.parts) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = po[(int64_t)(c + kWays) * (2 * 32 * D) + i * 128];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[4 * i] = fmaf(wc, x[i].x, acc[4 * i]);
        acc[4 * i + 1] = fmaf(wc, x[i].y, acc[4 * i + 1]);
        acc[4 * i + 2] = fmaf(wc, x[i].z, acc[4 * i + 2]);
        acc[4 * i + 3] = fmaf(wc, x[i].w, acc[4 * i + 3]);
        x[i] = y[i];
      }
    }
  }
  if constexpr (kFew) {
    __shared__ float sums[kWays - 1][32][33];
    if (way > 0) {
#pragma unroll
      for (int e = 0; e < 32; ++e) sums[way - 1][e][r] = acc[e];
    }
    __syncthreads();
    if (way > 0) return;
#pragma unroll
    for (int v = 0; v < kWays - 1; ++v)
#pragma unroll
      for (int e = 0; e < 32; ++e) acc[e] += sums[v][e][r];
  }
  if (!there) return;
  const int64_t row = ((int64_t)G.q_row + tok) * p.n_q_heads + (int64_t)G.head * p.group + (r - rt * p.group);
  uint4* dst = reinterpret_cast<uint4*>(p.o + row * D + c0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    dst[i] = make_uint4(pack_bf16(acc[8 * i], acc[8 * i + 1]), pack_bf16(acc[8 * i + 2], acc[8 * i + 3]),
                        pack_bf16(acc[8 * i + 4], acc[8 * i + 5]), pack_bf16(acc[8 * i + 6], acc[8 * i + 7]));
  if (blockIdx.y == 0) p.lse[row] = tot == 0.f ? kNegInf : base + logf(tot);
}

template <int D>
cudaError_t launch_causal_fwd_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CausalFwdParams& p, int grid, bool early, cudaStream_t stream) {
  using L = CausalFwdLayout<D>;
  const int smem = L::kBytes > 120 * 1024 ? L::kBytes : 120 * 1024;  // one CTA per SM (TMEM 512 columns)
  static PerDeviceOnce configured;
  cudaError_t e = configured.run([&] {
    cudaError_t r = cudaFuncSetAttribute(zl_causal_fwd_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (r != cudaSuccess) return r;
    // a kernel built with another register count would leave an increase waiting for registers forever
    cudaFuncAttributes fa;
    r = cudaFuncGetAttributes(&fa, zl_causal_fwd_kernel<D>);
    if (r != cudaSuccess) return r;
    return fa.numRegs == (int)kFwdLaunchRegs ? cudaSuccess : cudaErrorInvalidKernelImage;
  });
  if (e != cudaSuccess) return e;
  return launch_overlapped_if(early, zl_causal_fwd_kernel<D>, grid, kFwdThreads, smem, stream, tq, tk, tv, p);
}

}  // namespace

cudaError_t launch_causal_fwd(int head_dim, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CausalFwdParams& p, int grid, bool early, cudaStream_t stream) {
  return head_dim == 128 ? launch_causal_fwd_impl<128>(tq, tk, tv, p, grid, early, stream)
                         : launch_causal_fwd_impl<64>(tq, tk, tv, p, grid, early, stream);
}

cudaError_t launch_causal_merge(int head_dim, const CausalMergeParams& p, cudaStream_t stream) {
  if (p.n_groups == 0) return cudaSuccess;
  const dim3 grid(p.n_groups, head_dim / 32, p.rows > kCausalRows ? 2 : 1);
  const bool few = p.rows <= 32;
  auto k = head_dim == 128 ? (few ? zl_causal_merge_kernel<128, true> : zl_causal_merge_kernel<128, false>)
                           : (few ? zl_causal_merge_kernel<64, true> : zl_causal_merge_kernel<64, false>);
  return launch_overlapped(k, grid, 128, 0, stream, p);
}

}  // namespace zl
