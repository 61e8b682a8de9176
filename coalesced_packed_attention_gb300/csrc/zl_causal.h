// Internal tables and launch interfaces of the causal attention (host planner and kernels).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <vector>

#include "../../include/zl.h"

namespace zl {

// A small number kept per device by host code that runs at every launch (a device's SM count, a kernel's
// resident blocks): set once, read without a lock; two threads that set it at once set the same value.
class PerDeviceInt {
 public:
  template <typename F>
  cudaError_t get(int* value, F&& query) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool kept = dev >= 0 && dev < kDevices;
    int v = kept ? v_[dev].load(std::memory_order_relaxed) : 0;
    if (v == 0) {
      e = query(dev, &v);
      if (e != cudaSuccess) return e;
      if (kept) v_[dev].store(v, std::memory_order_relaxed);
    }
    *value = v;
    return cudaSuccess;
  }

 private:
  static constexpr int kDevices = 64;
  std::atomic<int> v_[kDevices] = {};
};

// Query rows are packed by key head: the `group` query heads that share a key head are neighbours, so a
// block of up to 128 rows is (tokens x group) with row r = token r / group, head r % group.  A block holds
// tokens_per_block(group) whole tokens; its rows past tokens x group are never stored.
constexpr int kCausalRows = 128;
__host__ __device__ inline int tokens_per_block(int group) { return kCausalRows / group; }

struct CausalSeq {
  int64_t q_offset, kv_offset;
  int32_t q_len, kv_len;
  int64_t acc_block;  // first 128-row block of the sequence in the dQ accumulator: [kv head][query block]
};

// Tiles carry what the kernels need of their sequence, so that a tile is one load away, not two in a row.
// One forward tile: up to two query blocks of one (sequence, key head) over a range of key blocks.
struct alignas(16) CausalTile {
  int32_t q_row, q_len, kv_row, kv_len;  // the sequence: first rows and lengths
  int32_t head, block;                   // key head; first query block (block, block + 1)
  int32_t kv_lo, kv_hi;                  // key blocks [kv_lo, kv_hi) of 128, as far as the rows see them
  int32_t part;                          // -1: final output; else the tile's slot of partial results
  int32_t seq, pad[2];
};
// One backward tile: 128 keys of one (sequence, key head) over query blocks [first, first + n), all that see one of
// the keys or a part of them.
struct alignas(16) CausalBwdTile {
  int32_t q_row, q_len, kv_row, kv_len;
  int32_t head, block;
  int32_t acc_block;  // the head's first block in the dQ accumulator
  int32_t first, n;
  int32_t part;       // -1: final output; else the tile's slot of partial dK, dV
  int32_t seq, pad;
};
// Rows whose key range was split: the combine of `parts` slots from `slot` on.
struct alignas(16) CausalMerge {
  int32_t q_row, q_len, head, block, slot, parts, pad[2];
};
// Key tiles whose query range was split: the sum of `parts` slots of dK, dV from `slot` on.
struct CausalBwdMerge {
  int32_t kv_row, kv_len, head, block, slot, parts, pad[2];
};

struct CausalFwdParams {
  const CausalTile* tiles;
  const int32_t* tile_ptr;  // tiles of thread block b: [tile_ptr[b], tile_ptr[b + 1])
  int32_t* status;
  long long wait_limit;
  int32_t withhold_load;
  int32_t n_q_heads, group;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;    // [slot][sub-tile][d / 4][128][4]
  float* part_lse;  // [slot][256]
  float scale_log2;
};

struct CausalMergeParams {
  const CausalMerge* groups;
  int32_t n_groups, rows, n_q_heads, group;  // rows: the most that a split tile has, of its 256
  const float* part_o;
  const float* part_lse;
  __nv_bfloat16* o;
  float* lse;
};

struct CausalBwdParams {
  const CausalBwdTile* tiles;
  const int32_t* tile_ptr;
  int32_t* status;
  long long wait_limit;
  int32_t withhold_load;
  int32_t n_q_heads, n_kv_heads, group;
  const float* lse;
  const float* row_d;  // D, [q tokens][q heads]
  float* acc;          // fp32 dQ accumulator, [block][d / 4][128][4]
  float* part;         // [slot][dV, dK][d / 4][128][4], fp32, dK not yet scaled
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int64_t dk_stride, dv_stride;
  float scale, scale_log2;
};

// The last launch of the backward: dQ from its accumulator, and the sums of split key tiles.
struct CausalFinishParams {
  const CausalSeq* seqs;
  const CausalBwdMerge* merges;
  int32_t n_seqs, n_merges, n_q_heads, n_kv_heads;
  int64_t acc_blocks;
  const float* acc;
  const float* part;
  __nv_bfloat16* dq;
  __nv_bfloat16* dk;
  __nv_bfloat16* dv;
  int64_t dq_stride, dk_stride, dv_stride;
  float scale;
};

cudaError_t launch_causal_fwd(int head_dim, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CausalFwdParams& p, int grid, bool early, cudaStream_t stream);
cudaError_t launch_causal_merge(int head_dim, const CausalMergeParams& p, cudaStream_t stream);
// D = rowsum(dO * O) over every row of the query tensor, and zeroing of the dQ accumulator.
cudaError_t launch_causal_bwd_pre(int head_dim, const __nv_bfloat16* o, const __nv_bfloat16* d_o, float* row_d,
                                  int64_t rows, float* acc, int64_t acc_floats, int num_sms, cudaStream_t stream);
cudaError_t launch_causal_bwd(int head_dim, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CausalBwdParams& p, int grid, bool early, cudaStream_t stream);
cudaError_t launch_causal_finish(int head_dim, const CausalFinishParams& p, int num_sms, cudaStream_t stream);

// A plan's tables in device memory.  They belong to the plan and to every graph that captured a launch from it, so that a
// graph may be replayed after its plan is gone.
struct CausalTables {
  void* ptr = nullptr;
  int device = -1;
  std::atomic<int32_t> owners{1};
  CausalTables* next = nullptr;  // in the list of those without owners
};
// Where the stream is being captured, makes its graph an owner of the plan's tables.
zl_status hold_tables(const zl_causal_plan* p, cudaStream_t stream);

}  // namespace zl

struct zl_causal_plan {
  int32_t n_q_heads = 0, n_kv_heads = 0, head_dim = 0, group = 0;
  int64_t q_tokens = 0, kv_tokens = 0;
  int device = -1, num_sms = 0;
  bool host_only = false, test_withhold = false;
  bool shared_keys = false;   // two sequences read the same key rows: no backward
  bool forward_only = false;  // ZL_PLAN_FORWARD_ONLY

  std::vector<zl::CausalSeq> seqs;
  std::vector<zl::CausalTile> fwd_tiles;
  std::vector<int32_t> fwd_ptr;
  std::vector<zl::CausalBwdTile> bwd_tiles;
  std::vector<int32_t> bwd_ptr;
  std::vector<zl::CausalMerge> merges;
  std::vector<zl::CausalBwdMerge> bwd_merges;
  int32_t slots = 0, bwd_slots = 0;
  bool fwd_short = false, bwd_short = false;  // the schedule is under some 100 us: worth setting up early
  int32_t merge_rows = 0;  // rows of a split forward tile that may hold a query (the largest)
  int64_t acc_blocks = 0;
  int64_t fwd_bytes = 0, bwd_bytes = 0;

  zl::CausalTables* tables = nullptr;
  zl::CausalSeq* d_seqs = nullptr;
  zl::CausalTile* d_fwd_tiles = nullptr;
  int32_t* d_fwd_ptr = nullptr;
  zl::CausalBwdTile* d_bwd_tiles = nullptr;
  int32_t* d_bwd_ptr = nullptr;
  zl::CausalMerge* d_merges = nullptr;
  zl::CausalBwdMerge* d_bwd_merges = nullptr;
  int32_t* d_status = nullptr;
};
