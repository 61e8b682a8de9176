// What the attention kernels over the 4-bit cache share: parameters, the schedule, the parts of cut items.
#pragma once
#include "zl_kv4.cuh"
#include "zl_ptx.cuh"

namespace zl {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLow = -1e30f;     // the reference of rows that have seen nothing
constexpr float kRescale = 8.f;    // the maximum may lag by 2^8 before the sums are rescaled
// P = 2^(score - reference) is rounded to fp16, whose smallest number is 2^-24: at a reference of the maximum itself,
// weights below 2^-25 of it would be lost in O but not in the sum (O too small by up to slots x 2^-25, 3 % at 2^20
// slots).  With the reference 2^7 below it P is up to 2^7, with the lag 2^15, of fp16's 2^16, and what is lost lies
// below 2^-32.  Scores of 2^20 and more keep the room for their own rounding instead.
constexpr float kBelow = 7.f, kFar = 0x1p20f;
__device__ __forceinline__ float reference_of(float top) { return fabsf(top) < kFar ? top - kBelow : top; }
__device__ __forceinline__ float lag_of(float ref) { return fabsf(ref) < kFar ? kBelow + kRescale : kRescale; }

// An item cut between blocks: its first block describes it for the join.
struct alignas(16) Cut {
  int32_t parts;   // 0: the item was not cut, or none that begins in this block
  int32_t which;   // part of its first block, 2 block + (0 the block's first segment, 1 another); the next blocks' are their first
  int32_t token0;  // row of the item's sequence in q and o
  int32_t head0;   // first query head
  int32_t row0, rows;
  int32_t pad[2];
};

struct AttnParams {
  Kv4 c;
  const __nv_bfloat16* q;
  int64_t q_stride, n_tokens;
  const int32_t* starts;
  __nv_bfloat16* o;
  float* lse;
  float* part_o;   // [2 blocks][rows][d]
  float2* part_ml; // [2 blocks][rows]: maximum (base 2) and sum
  Cut* cuts;       // by item where there are no more items than blocks, else by the block in which the item begins
  int32_t max_tiles, by_item;  // row tiles of max_new tokens; how cuts is laid out
  float* scores;   // [sequence][key head][score_rows][slot], base 2
  const float* w_in;
  float* w_out;
  float decay;
  float scale_log2;
  int32_t group, q_heads, max_new, score_rows;
  int32_t own_weights;  // the attention kernel adds them up itself
};

// log of a sum l of 2^(score - m); -inf for an empty one, NaN stays.
__device__ __forceinline__ float natural_lse(float m, float l) { return l == 0.f ? -INFINITY : m * kLn2 + logf(l); }

// The items' costs in a row, dealt out evenly: an item costs its units and kItemCost more (its queries, its end), which
// stand before the first unit.  A cut inside them belongs to the first unit.

// A block's run of units, item by item; the producers of the warps and their consumers each walk it by themselves.
template <int kRows, int kUnit, int kItemCost>
struct Walk {
  static constexpr int kCost = kItemCost;
  int64_t left;        // cost of the block's run from this segment on
  int32_t seq, head, tile;  // an item: a key head's row tile
  int32_t n, m, first;      // the sequence's new tokens, slots and first token
  int32_t row_tiles, chunks;
  int32_t a, e;        // this segment: units [a, e) of the item's `chunks`

  __device__ void load(const AttnParams& p) {
    n = kv4_new(p.c, p.starts, p.n_tokens, p.max_new, seq, &first);
    m = kv4_len(p.c, seq);
    row_tiles = (n * p.group + kRows - 1) / kRows;
    chunks = m > 0 ? (m + kUnit - 1) / kUnit : 1;
  }
  __device__ int64_t cost(const AttnParams& p) const { return (int64_t)p.c.heads * row_tiles * (chunks + kItemCost); }
  // at cost `off` of the item: the segment from there on, without units where `left` ends before the first one
  __device__ void enter(int off) {
    const int end = (int)(left < chunks + kItemCost - off ? off + left : chunks + kItemCost);
    a = off > kItemCost ? off - kItemCost : 0;
    e = end > kItemCost ? end - kItemCost : 0;
    left -= end - off;
  }
  __device__ bool done() const { return a >= e; }  // a segment without units is the last
  __device__ void next(const AttnParams& p) {
    a = e = 0;
    if (left <= 0) return;
    if (++tile == row_tiles) {
      tile = 0;
      if (++head == p.c.heads) {
        head = 0;
        do {
          if (++seq >= p.c.n_seqs) {
            left = 0;
            return;
          }
          load(p);
        } while (row_tiles == 0);
      }
    }
    enter(0);
  }
};


// The block's run: false where it has none.  Every thread calls it; warp_sums has a number a warp, *seq_before and *seq
// are shared.  *each: cost of a full run.
template <int kThreads, int kLeast, typename W>
__device__ bool first_segment_of(const AttnParams& p, int64_t* warp_sums, int64_t* seq_before, int* seq, W& w,
                                 int64_t* each_out) {
  if (threadIdx.x == 0) *seq = -1;
  const int n = p.c.n_seqs, per = (n + kThreads - 1) / kThreads;
  const int b0 = min(n, (int)threadIdx.x * per), b1 = min(n, b0 + per);
  int64_t mine = 0, total;
  for (int b = b0; b < b1; ++b) {
    w.seq = b;
    w.load(p);
    mine += w.cost(p);
  }
  int64_t before = kv4_scan<kThreads>(mine, &total, warp_sums);
  const int64_t each = max((total + gridDim.x - 1) / gridDim.x, (int64_t)kLeast);
  const int64_t at = each * blockIdx.x, end = min(total, at + each);
  if (at < end && at >= before && at < before + mine) {
    int b = b0;
    for (;; ++b) {
      w.seq = b;
      w.load(p);
      if (at < before + w.cost(p)) break;
      before += w.cost(p);
    }
    *seq = b;
    *seq_before = before;
  }
  __syncthreads();
  if (threadIdx.x == 0 && !p.by_item) p.cuts[blockIdx.x].parts = 0;  // an item cut at the run's end sets it later
  if (*seq < 0) return false;
  w.seq = *seq;
  w.load(p);
  w.left = end - at;
  const int64_t off = at - *seq_before, of_item = w.chunks + W::kCost;
  const int item = (int)(off / of_item);
  w.head = item / w.row_tiles;
  w.tile = item - w.head * w.row_tiles;
  w.enter((int)(off - item * of_item));
  *each_out = each;
  return true;
}

// Describes a segment's item for the join, where it begins in this segment.
template <typename W>
__device__ __forceinline__ void describe(const AttnParams& p, const W& w, int part, int row0, int rows, int64_t each) {
  const bool whole = w.a == 0 && w.e == w.chunks;
  if (w.a != 0 || (!p.by_item && whole)) return;
  const int rest = w.chunks - w.e;  // full runs follow until the item's end
  Cut c = {whole ? 0 : 1 + (int)((rest + each - 1) / each), part, w.first, w.head * p.group, row0, rows, {0, 0}};
  p.cuts[p.by_item ? ((int64_t)w.seq * p.c.heads + w.head) * p.max_tiles + w.tile : blockIdx.x] = c;
}

// Many rows a key head: tensor-core kernel (zl_kv4_chunk.cu); its blocks and rows of a tile.
constexpr int kChunkRows = 128;
constexpr int kChunkMaxBlocks = 160;
cudaError_t launch_kv4_chunk(int head_dim, const AttnParams& p, int blocks, cudaStream_t stream);

}  // namespace zl
