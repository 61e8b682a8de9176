// Eviction from the 4-bit cache by accumulated attention weight.
//
// Every (sequence, key head) keeps `keep` of its n slots: those with a position above newest - recent first, then
// the largest weights, ties to the lower slot.  Finding the border is a radix selection over the weights' bits, eight at a
// time, by one block; survivors behind slot keep and the slots given up before it are then counted in slot order and
// listed, and a second launch moves the rows, 1.125 d bytes each, over all SMs.  Nothing is sorted and unmoved rows are not
// touched: a step's eviction moves one row a head.
// Bound by latency at serving sizes (a few passes over 4 n bytes by one block) and by the weights' and positions' bytes past them.
#include <cuda_runtime.h>

#include "zl_internal.h"
#include "zl_kv4.cuh"
#include "zl_overlap.cuh"

namespace zl {
namespace {

constexpr int kPickThreads = 1024;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoves = 64;  // rows a block of the second launch moves

struct EvictParams {
  Kv4 c;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int32_t* counts;  // [sequence][key head]: moves
  int32_t* moves;   // [sequence][key head][2][capacity]: slots given up, survivors
  int32_t keep, recent, capacity;
};

// Larger weights have larger numbers; NaN has the smallest, -0 is 0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum of a number over the block; every thread gets it.
__device__ __forceinline__ int block_sum(int x, int* warp_sums) {
  x = __reduce_add_sync(0xffffffffu, x);
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = x;
  __syncthreads();
  int all = 0;
#pragma unroll
  for (int i = 0; i < kPickWarps; ++i) all += warp_sums[i];
  __syncthreads();
  return all;
}

__global__ void __launch_bounds__(kPickThreads) zl_kv4_pick_kernel(const EvictParams p) {
  __shared__ int hist[kPickWarps][256];
  __shared__ int warp_sums[kPickWarps];
  __shared__ int s_digit, s_above;
  let_next_start();
  wait_for_previous();
  const int b = blockIdx.x / p.c.heads, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t base = (int64_t)blockIdx.x * ((int64_t)p.c.max_pages << p.c.page_shift);
  const float* w = p.weights + base;
  const int32_t* pos = p.positions + base;
  float* w_out = p.weights_out + base;
  int32_t* pos_out = p.positions_out + base;
  const bool copy_w = p.weights_out != p.weights, copy_pos = p.positions_out != p.positions;
  const int n = kv4_len(p.c, b), keep = p.keep;
  if (n <= keep) {
    for (int s = threadIdx.x; s < n; s += kPickThreads) {
      if (copy_w) w_out[s] = w[s];
      if (copy_pos) pos_out[s] = pos[s];
    }
    if (threadIdx.x == 0) p.counts[blockIdx.x] = 0;
    return;
  }
  // the newest position, and how many slots lie within `recent` of it
  int newest = INT32_MIN;
  for (int s = threadIdx.x; s < n; s += kPickThreads) newest = max(newest, pos[s]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_sums[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, warp_sums[lane]);
  __syncthreads();
  const int64_t border = (int64_t)newest - p.recent;
  int mine = 0;
  for (int s = threadIdx.x; s < n; s += kPickThreads) mine += pos[s] > border;
  const int safe = block_sum(mine, warp_sums);
  // the slots among which the weights decide: the recent ones where they alone are too many, else the others
  const bool among_recent = safe > keep;
  int need = among_recent ? keep : keep - safe;
  // radix selection: after each round the border's leading digits, and how many of those that share them still count
  uint32_t prefix = 0, mask = 0;
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = lane; i < 256; i += 32) hist[warp][i] = 0;
    __syncwarp();
    for (int s = threadIdx.x; s < n; s += kPickThreads) {
      if ((pos[s] > border) != among_recent) continue;
      const uint32_t r = rank_of(w[s]);
      if ((r & mask) == prefix) atomicAdd(&hist[warp][(r >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 256) {
      int sum = 0;
#pragma unroll
      for (int i = 0; i < kPickWarps; ++i) sum += hist[i][threadIdx.x];
      hist[0][threadIdx.x] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      // counts of digits from the top: the digit at which they reach `need`
      int above = 0;
      for (int d0 = 224; d0 >= 0; d0 -= 32) {
        const int x = hist[0][d0 + 31 - lane];  // lane 0 has the largest digit
        int run = x;
#pragma unroll
        for (int i = 1; i < 32; i <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, run, i);
          if (lane >= i) run += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, above + run >= need);
        if (hit) {
          const int first = __ffs(hit) - 1;
          const int up = __shfl_sync(0xffffffffu, above + run - x, first);
          if (lane == 0) {
            s_digit = d0 + 31 - first;
            s_above = up;
          }
          break;
        }
        above += __shfl_sync(0xffffffffu, run, 31);
      }
    }
    __syncthreads();
    need -= s_above;
    prefix |= (uint32_t)s_digit << shift;
    mask |= 255u << shift;
    __syncthreads();
  }
  // `need` of the slots at the border stay, the lowest ones.  Warps take contiguous runs of slots.
  const int run = ((n + kPickWarps - 1) / kPickWarps + 31) / 32 * 32;
  const int s0 = min(n, warp * run), s1 = min(n, s0 + run);
  // 0: given up, 1: stays, 2: at the border
  auto state = [&](int s) {
    const bool recent = pos[s] > border;
    if (recent != among_recent) return recent ? 1 : 0;
    const uint32_t r = rank_of(w[s]);
    return r > prefix ? 1 : r == prefix ? 2 : 0;
  };
  int ties = 0;
  for (int s = s0; s < s1; s += 32) ties += __popc(__ballot_sync(0xffffffffu, s + lane < s1 && state(s + lane) == 2));
  if (lane == 0) warp_sums[warp] = ties;
  __syncthreads();
  int ties_before = 0;
  for (int i = 0; i < warp; ++i) ties_before += warp_sums[i];
  __syncthreads();
  auto stays = [&](int s, int& tie) {  // of a warp's 32 slots from s on; tie: ties before them
    const int st = s + lane < s1 ? state(s + lane) : 0;
    const unsigned at_border = __ballot_sync(0xffffffffu, st == 2);
    const bool kept = st == 1 || (st == 2 && tie + __popc(at_border & ((1u << lane) - 1)) < need);
    tie += __popc(at_border);
    return kept;
  };
  int holes = 0, movers = 0, tie = ties_before;
  for (int s = s0; s < s1; s += 32) {
    const bool kept = stays(s, tie), in = s + lane < s1;
    holes += __popc(__ballot_sync(0xffffffffu, in && !kept && s + lane < keep));
    movers += __popc(__ballot_sync(0xffffffffu, kept && s + lane >= keep));
  }
  if (lane == 0) {
    hist[0][warp] = holes;
    hist[1][warp] = movers;
  }
  __syncthreads();
  int hole_at = 0, mover_at = 0, total = 0;
  for (int i = 0; i < kPickWarps; ++i) {
    if (i < warp) {
      hole_at += hist[0][i];
      mover_at += hist[1][i];
    }
    total += hist[0][i];
  }
  int32_t* list = p.moves + (int64_t)blockIdx.x * 2 * p.capacity;
  tie = ties_before;
  for (int s = s0; s < s1; s += 32) {
    const bool kept = stays(s, tie), in = s + lane < s1;
    const int slot = s + lane;
    const bool hole = in && !kept && slot < keep, mover = kept && slot >= keep;
    const unsigned h = __ballot_sync(0xffffffffu, hole), m = __ballot_sync(0xffffffffu, mover);
    // within the lists whatever happens to the inputs meanwhile
    const int hole_i = hole_at + __popc(h & ((1u << lane) - 1)), mover_i = mover_at + __popc(m & ((1u << lane) - 1));
    if (hole && hole_i < p.capacity) list[hole_i] = slot;
    if (mover && mover_i < p.capacity) list[p.capacity + mover_i] = slot;
    hole_at += __popc(h);
    mover_at += __popc(m);
    if (kept && slot < keep) {
      if (copy_w) w_out[slot] = w[slot];
      if (copy_pos) pos_out[slot] = pos[slot];
    }
  }
  if (threadIdx.x == 0) p.counts[blockIdx.x] = min(total, p.capacity);
}

// 16 lanes a move: codes of keys and values in 16-byte pieces, scales, weight and position.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) zl_kv4_move_kernel(const EvictParams p) {
  let_next_start();
  wait_for_previous();
  const int item = blockIdx.y + blockIdx.z * 65535;
  if (item >= p.c.n_seqs * p.c.heads) return;
  const int b = item / p.c.heads, h = item - b * p.c.heads;
  const int count = p.counts[item];
  const int32_t* list = p.moves + (int64_t)item * 2 * p.capacity;
  const int64_t base = (int64_t)item * ((int64_t)p.c.max_pages << p.c.page_shift);
  const int end = min(count, ((int)blockIdx.x + 1) * kMoves);
  for (int i = blockIdx.x * kMoves + threadIdx.x / 16; i < end; i += kMoveThreads / 16) {
    const int l = threadIdx.x & 15, to = list[i], from = list[p.capacity + i];
    if (l == 14) p.weights_out[base + to] = p.weights[base + from];
    if (l == 15) p.positions_out[base + to] = p.positions[base + from];
    uint8_t* dst = kv4_tile<D>(p.c, b, h, to);
    const uint8_t* src = kv4_tile<D>(p.c, b, h, from);
    if (!dst || !src) {
      if (l == 0) kv4_report(p.c, ZL_KV4_BAD_PAGE);
      continue;
    }
    constexpr int kPieces = D / 32;  // 16-byte pieces of a row's codes
    const int r0 = to & 15, r1 = from & 15;
    if (l < 2 * kPieces) {
      const int at = (l / kPieces) * 8 * D + (l % kPieces) * 16;
      *reinterpret_cast<uint4*>(dst + at + r0 * (D / 2)) = *reinterpret_cast<const uint4*>(src + at + r1 * (D / 2));
    } else if (l >= 8 && l < 8 + 2 * (D / 64)) {
      const int at = 16 * D + ((l - 8) / (D / 64)) * D + ((l - 8) % (D / 64)) * 4;
      *reinterpret_cast<uint32_t*>(dst + at + r0 * (D / 16)) = *reinterpret_cast<const uint32_t*>(src + at + r1 * (D / 16));
    }
  }
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }

}  // namespace
}  // namespace zl

using namespace zl;

extern "C" zl_status zl_kv4_evict_workspace(const zl_kv4_cache* cache, int64_t* bytes) {
  Kv4 c;
  const zl_status s = kv4_check(cache, &c);
  if (s != ZL_OK) return s;
  if (!bytes) return ZL_ERR_INVALID_ARG;
  const int64_t items = (int64_t)cache->n_seqs * cache->n_kv_heads;
  // moves are no more than half the slots: the slots given up in front are below keep, the survivors past it
  *bytes = round16(items * 4) + items * 2 * ((int64_t)cache->max_pages * cache->page / 2) * 4;
  return ZL_OK;
}

extern "C" zl_status zl_kv4_evict(const zl_kv4_cache* cache, const float* weights, const int32_t* positions, int32_t keep,
                                  int32_t recent, float* weights_out, int32_t* positions_out, void* workspace, void* stream) {
  NvtxRange range("zl_kv4_evict");
  EvictParams p{};
  zl_status s = kv4_check(cache, &p.c);
  if (s != ZL_OK) return s;
  if (keep < 1 || recent < 0) return ZL_ERR_INVALID_ARG;
  if (cache->n_seqs == 0 || cache->max_pages == 0) return ZL_OK;
  if (!weights || !positions || !weights_out || !positions_out || !workspace) return ZL_ERR_INVALID_ARG;
  if (!kv4_aligned(weights, 4) || !kv4_aligned(positions, 4) || !kv4_aligned(weights_out, 4) || !kv4_aligned(positions_out, 4) ||
      !kv4_aligned(workspace, 16))
    return ZL_ERR_ALIGN;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  const int64_t items = (int64_t)cache->n_seqs * cache->n_kv_heads, slots = (int64_t)cache->max_pages * cache->page;
  if (items > INT32_MAX) return ZL_ERR_UNSUPPORTED;
  p.weights = weights;
  p.positions = positions;
  p.weights_out = weights_out;
  p.positions_out = positions_out;
  p.counts = static_cast<int32_t*>(workspace);
  p.moves = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + round16(items * 4));
  p.keep = keep;
  p.recent = recent;
  p.capacity = (int32_t)(slots / 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_overlapped(zl_kv4_pick_kernel, (unsigned)items, kPickThreads, 0, st, p);
  const int64_t most = slots - keep < keep ? slots - keep : keep;  // moves of an item at most
  if (e == cudaSuccess && most > 0) {
    const dim3 grid((unsigned)((most + kMoves - 1) / kMoves), (unsigned)(items < 65535 ? items : 65535), (unsigned)((items + 65534) / 65535));
    e = launch_overlapped(cache->head_dim == 128 ? zl_kv4_move_kernel<128> : zl_kv4_move_kernel<64>, grid, kMoveThreads, 0, st, p);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
