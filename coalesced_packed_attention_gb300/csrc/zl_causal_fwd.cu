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
// Rounding: S, the running maximum and sum, O and LSE are fp32.  P is rounded to bf16 because it is an operand of
// the PV product (relative 2^-9 a weight, independent from key to key); its sum is taken before the rounding.
// Roles (384 threads, one CTA per SM): warps 0-3 and 4-7 the two softmax warpgroups (thread = TMEM lane = row),
// warp 8 TMA, warp 9 MMA, 10 and 11 idle.  TMEM (512 columns): S0 [0,128), S1 [128,256), O0 [256,256+d), O1 [384,384+d).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "zl_causal.h"
#include "zl_internal.h"
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
  static constexpr int kOut = kV + kStages * kTile;  // 4 KB for each softmax warp: 32 rows x 64 channels of O
  static constexpr int kBar = kOut + 8 * 4096;
  static constexpr int kNumBars = 2 + 1 + 4 * kStages + 2 + 2 + 2 + 1;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 32;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base to 1024 B
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

// Launched with 168 registers a thread (three warps to a sub-partition); the softmax warpgroups, which hold a
// row's 128 scores, take 216 and leave 72 to the warps that issue: per sub-partition 2 x 216 + 72 = 3 x 168, the launch
// allocation.
constexpr int kFwdThreads = 384;
constexpr uint32_t kFwdLaunchRegs = 168, kFwdSoftmaxRegs = 216, kFwdIssueRegs = 72;
static_assert(2 * kFwdSoftmaxRegs + kFwdIssueRegs == 3 * kFwdLaunchRegs, "register split must equal the launch allocation");

template <int D>
__global__ void __launch_bounds__(kFwdThreads, 1)
    zl_causal_fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, const CausalFwdParams p) {
  using L = CausalFwdLayout<D>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem + L::kQ;
  uint8_t* sK = smem + L::kK;
  uint8_t* sV = smem + L::kV;
  uint64_t* bar = reinterpret_cast<uint64_t*>(smem + L::kBar);
  uint64_t* q_full = bar;  // [2] one per sub-tile
  uint64_t* q_empty = bar + 2;
  uint64_t* k_full = bar + 3;  // [S]
  uint64_t* k_empty = k_full + S;
  uint64_t* v_full = k_empty + S;
  uint64_t* v_empty = v_full + S;
  uint64_t* s_full = v_empty + S;  // [2] per sub-tile
  uint64_t* p_full = s_full + 2;   // [2]
  uint64_t* o_bar = p_full + 2;    // [2] last PV of a tile done
  uint64_t* drain = o_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc + 8);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + i, 1);
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 128);
      mbar_init(o_bar + i, 1);
    }
    mbar_init(q_empty, 1);
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
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const long long lim = p.wait_limit;
  const int tb = tokens_per_block(p.group);
  const int t_begin = p.tile_ptr[blockIdx.x], t_end = p.tile_ptr[blockIdx.x + 1];

  if (warp >= 8) {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFwdIssueRegs));
   if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(D / 64) * (uint32_t)(tb * p.group) * 128u;
      uint32_t kv_it = 0, q_it = 0, q_loads[2] = {0, 0}, k_loads = 0, v_loads = 0;
      bool ok = true;
      for (int t = t_begin; t < t_end && ok; ++t) {
        const CausalTile tl = p.tiles[t];
        const FwdSpan sp = span_of(tl, tb);
        if (sp.nmax == 0) continue;
        if (!cwait(q_empty, (q_it & 1) ^ 1, abort_flag, lim, p.status)) break;
        ++q_it;
        for (int w = 0; w < 2; ++w) {
          if (sp.n[w] == 0) continue;
          mbar_arrive_expect_tx(q_full + w, q_bytes);
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sQ + w * L::kTile + c * L::kBox, &tm_q, q_full + w, 64 * c, 0, tl.head,
                        tl.q_row + sp.tok[w]);
          ++q_loads[w];
        }
        const int kv0 = tl.kv_row + tl.kv_lo * 128;
        for (int j = 0; j < sp.nmax; ++j) {
          const uint32_t s = kv_it % S, ph = (kv_it / S) & 1;
          if (!cwait(k_empty + s, ph ^ 1, abort_flag, lim, p.status)) { ok = false; break; }
          mbar_arrive_expect_tx(k_full + s, L::kTile);
          if (p.withhold_load && kv_it == 0) {
            // test hook: the announced bytes never arrive; a bounded wait runs out
          } else {
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(sK + s * L::kTile + c * L::kBox, &tm_k, k_full + s, 64 * c, tl.head, kv0 + j * 128);
          }
          ++k_loads;
          if (!cwait(v_empty + s, ph ^ 1, abort_flag, lim, p.status)) { ok = false; break; }
          mbar_arrive_expect_tx(v_full + s, L::kTile);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sV + s * L::kTile + c * L::kBox, &tm_v, v_full + s, 64 * c, tl.head, kv0 + j * 128);
          ++v_loads;
          ++kv_it;
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
          if (q_loads[w]) settle(q_full + w, (q_loads[w] - 1) & 1);
        for (uint32_t b = 1; b <= (uint32_t)S; ++b) {
          if (k_loads >= b) settle(k_full + (k_loads - b) % S, ((k_loads - b) / S) & 1);
          if (v_loads >= b) settle(v_full + (v_loads - b) % S, ((v_loads - b) / S) & 1);
        }
      }
    }
   } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    // The whole warp runs the loop (control flow, waits and descriptors are warp-uniform); one elected lane
    // executes each product and commit.
    constexpr uint32_t kIdS = idesc_bf16(128, 128, false, false);
    constexpr uint32_t kIdPV = idesc_bf16(128, D, false, true);
    const uint32_t aV = smem_u32(sV);
    const uint64_t dQ0 = sdesc_sw128(smem_u32(sQ), 16, 1024), dK0 = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV0 = sdesc_sw128(aV, L::kBox, 1024);
    uint32_t kv_it = 0, qcount[2] = {0, 0}, pcount[2] = {0, 0};
    bool ok = true;
    auto wait_w = [&](uint64_t* b, uint32_t parity) {
      return __all_sync(0xffffffffu, cwait(b, parity, abort_flag, lim, p.status));
    };
    auto issue_s = [&](int w, uint32_t stage) {
      const uint64_t dq = sdesc_add(dQ0, w * L::kTile), dk = sdesc_add(dK0, stage * L::kTile);
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t koff = (kk >> 2) * L::kBox + (kk & 3) * 32;
        mma_ss_w(tmem + 128 * w, sdesc_add(dq, koff), sdesc_add(dk, koff), kIdS, kk > 0 ? 1u : 0u);
      }
      mma_commit_w(s_full + w);
    };
    auto issue_pv = [&](int w, uint32_t stage, bool first) -> bool {
      if (!wait_w(p_full + w, pcount[w] & 1)) return false;
      ++pcount[w];
      tc_fence_after();
      const uint64_t dv = sdesc_add(dV0, stage * L::kTile);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_w(tmem + 256 + 128 * w, tmem + 128 * w + kk * 8, sdesc_add(dv, kk * 2048), kIdPV,
                 (first && kk == 0) ? 0u : 1u);
      return true;
    };
    for (int t = t_begin; t < t_end && ok; ++t) {
      const CausalTile tl = p.tiles[t];
      const FwdSpan sp = span_of(tl, tb);
      if (sp.nmax == 0) continue;
      uint32_t ps = 0, pph = 0;
      for (int j = 0; j <= sp.nmax; ++j) {
        const uint32_t s = kv_it % S, ph = (kv_it / S) & 1;
        const bool more = j < sp.nmax;
        if (more && !wait_w(k_full + s, ph)) { ok = false; break; }
        if (j > 0) {
          if (!wait_w(v_full + ps, pph)) { ok = false; break; }
          // value rows past the sequence's keys are other tokens: their weights are zero, but 0 x NaN is not
          const int vrows = tl.kv_len - (tl.kv_lo + j - 1) * 128;
          if (vrows < 128) {
            zero_tile_rows<D>(aV + ps * L::kTile, vrows, lane);
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (j == 0 && sp.n[w] > 0) {
            if (!wait_w(q_full + w, qcount[w] & 1)) { ok = false; break; }
            ++qcount[w];
          }
          tc_fence_after();
          if (j > 0 && j <= sp.n[w]) {
            if (!issue_pv(w, ps, j == 1)) { ok = false; break; }
            if (j == sp.n[w]) mma_commit_w(o_bar + w);
          }
          if (j < sp.n[w]) issue_s(w, s);
        }
        if (!ok) break;
        if (j > 0) mma_commit_w(v_empty + ps);
        if (more) mma_commit_w(k_empty + s);
        if (j == sp.nmax - 1) mma_commit_w(q_empty);
        ps = s;
        pph = ph;
        if (more) ++kv_it;
      }
    }
    mma_commit_w(drain);
    wait_w(drain, 0);
   }
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kFwdSoftmaxRegs));
    const int w = warp >> 2;          // sub-tile of this warpgroup
    const int r = threadIdx.x & 127;  // row of the sub-tile == TMEM lane
    const int rt = r / p.group, rh = r - rt * p.group;  // its token and head
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
      if (toks == 0) continue;
      const int tok = (w ? sp.tok[1] : sp.tok[0]) + rt;
      const bool row_ok = rt < toks;
      // keys this row sees, from the tile's first block on; rows that are not stored need no mask
      const int seen =
          row_ok ? max(0, tl.kv_len - tl.q_len + tok + 1) - tl.kv_lo * 128 : 0x7fffffff;

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
      if (n > 0) {
        if (!__all_sync(0xffffffffu, cwait(o_bar + w, tiles_done & 1, abort_flag, lim, p.status))) break;
        ++tiles_done;
        tc_fence_after();
      }
      // ---- epilogue: O / l and LSE.  l > 0 wherever the row saw a key (its largest weight is >= 2^-8); a NaN
      // sum stays NaN.
      const float inv_l = l == 0.f ? 0.f : __frcp_rn(l);
      const float lse_v = l == 0.f ? kNegInf : (m_used + lg2(l)) * kLn2;
      const int64_t row = ((int64_t)tl.q_row + tok) * p.n_q_heads + (int64_t)tl.head * p.group + rh;
      const int64_t prow = (int64_t)tl.part * 256 + 128 * w + r;
      auto load_o = [&](int c, uint32_t (&u)[32]) {  // 32 channels of O / l
        if (n > 0) {
          tmem_ld32(tO + 32 * c, u);
          tmem_ld_wait();
        }
        // a row without a key beside rows with some: its weights were all zero, and 0 x Inf or NaN of a value
        // that it does not see must not show
#pragma unroll
        for (int e = 0; e < 32; ++e) u[e] = n > 0 && l != 0.f ? __float_as_uint(__uint_as_float(u[e]) * inv_l) : 0u;
      };
      if (tl.part < 0) {
        // 64 channels of the warp's 32 rows through shared memory (16-byte pieces, swizzled by row), so that a store
        // writes four rows' whole 128 bytes: a store per row and thread kept the load/store unit busy for 2900 cycles
        // a tile
        // (the lane is read again here: addresses formed from the one above would be kept in registers through
        // the loop over key blocks, which has none to spare)
        int ln;
        asm volatile("mov.u32 %0, %%laneid;" : "=r"(ln));
        const uint32_t buf = smem_u32(smem + L::kOut) + warp * 4096;
        const int rel = row_ok ? rt * p.n_q_heads + rh : -1;
        __nv_bfloat16* base = p.o + (((int64_t)tl.q_row + tok - rt) * p.n_q_heads + (int64_t)tl.head * p.group) * D + (ln & 7) * 8;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          if (half > 0) __syncwarp();  // the first half has been read
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t u[32];
            load_o(2 * half + c, u);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) v[e] = pack_bf16(__uint_as_float(u[8 * i + 2 * e]), __uint_as_float(u[8 * i + 2 * e + 1]));
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(buf + ln * 128 + (((4 * c + i) ^ (ln & 7)) << 4)),
                           "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                           : "memory");
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int lr = 4 * i + (ln >> 3);  // lane's row of the warp
            const int to = __shfl_sync(0xffffffffu, rel, lr);
            uint4 v;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(buf + lr * 128 + (((ln & 7) ^ (lr & 7)) << 4))
                         : "memory");
            if (to >= 0) *reinterpret_cast<uint4*>(base + (int64_t)to * D + 64 * half) = v;
          }
        }
        __syncwarp();  // the next tile's rows overwrite the buffer
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t u[32];
          load_o(c, u);
          if (row_ok) {
            uint4* dst = reinterpret_cast<uint4*>(p.part_o + prow * D + 32 * c);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = make_uint4(u[4 * i], u[4 * i + 1], u[4 * i + 2], u[4 * i + 3]);
          }
        }
      }
      if (row_ok) {
        if (tl.part < 0) p.lse[row] = lse_v;
        else p.part_lse[prow] = lse_v;
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Combine of a tile's parts: LSE = M + ln sum_c exp(LSE_c - M), O = sum_c exp(LSE_c - LSE) O_c.  One block per
// split tile, one warp per row, d / 32 channels per lane; parts are added in key order.
template <int D>
__global__ void __launch_bounds__(128) zl_causal_merge_kernel(const CausalMergeParams p) {
  constexpr int E = D / 32;
  const CausalMerge G = p.groups[blockIdx.x];
  const CausalSeq sq = p.seqs[G.seq];
  const int lane = threadIdx.x & 31, tb = tokens_per_block(p.group);
  for (int r = threadIdx.x >> 5; r < 256; r += 4) {
    const int rr = r & 127, rt = rr / p.group;
    const int tok = (G.block + (r >> 7)) * tb + rt;
    if (rt >= tb || tok >= sq.q_len) continue;  // warp-uniform
    const float* pl = p.part_lse + (int64_t)G.slot * 256 + r;
    float m = kNegInf;
    for (int c = lane; c < G.parts; c += 32) m = fmaxf(m, pl[(int64_t)c * 256]);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
    const float base = m == kNegInf ? 0.f : m;
    float tot = 0.f;
    for (int c = lane; c < G.parts; c += 32) tot += expf(pl[(int64_t)c * 256] - base);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, s);
    const float inv = tot == 0.f ? 0.f : 1.f / tot;
    float acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    const float* po = p.part_o + ((int64_t)G.slot * 256 + r) * D + lane * E;
#pragma unroll 4
    for (int c = 0; c < G.parts; ++c) {
      const float wc = expf(pl[(int64_t)c * 256] - base) * inv;
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(wc, po[(int64_t)c * 256 * D + e], acc[e]);
    }
    const int64_t row = (sq.q_offset + tok) * p.n_q_heads + (int64_t)G.head * p.group + (rr - rt * p.group);
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.o + row * D + lane * E);
#pragma unroll
    for (int e = 0; e < E; e += 2) dst[e / 2] = pack_bf16(acc[e], acc[e + 1]);
    if (lane == 0) p.lse[row] = tot == 0.f ? kNegInf : base + logf(tot);
  }
}

template <int D>
cudaError_t launch_causal_fwd_impl(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const CausalFwdParams& p, int grid, cudaStream_t stream) {
  using L = CausalFwdLayout<D>;
  const int smem = L::kAlloc > 120 * 1024 ? L::kAlloc : 120 * 1024;  // one CTA per SM (TMEM 512 columns)
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
  zl_causal_fwd_kernel<D><<<grid, kFwdThreads, smem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_causal_fwd(int head_dim, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CausalFwdParams& p, int grid, cudaStream_t stream) {
  return head_dim == 128 ? launch_causal_fwd_impl<128>(tq, tk, tv, p, grid, stream)
                         : launch_causal_fwd_impl<64>(tq, tk, tv, p, grid, stream);
}

cudaError_t launch_causal_merge(int head_dim, const CausalMergeParams& p, int, cudaStream_t stream) {
  if (p.n_groups == 0) return cudaSuccess;
  if (head_dim == 128) zl_causal_merge_kernel<128><<<p.n_groups, 128, 0, stream>>>(p);
  else zl_causal_merge_kernel<64><<<p.n_groups, 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace zl
