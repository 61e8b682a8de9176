// Eviction from the 4-bit cache by accumulated attention weight.
//
// Every (sequence, key head) keeps `keep` of its n slots: those with a position above newest - recent first, then
// the largest weights, ties to the lower slot.  Finding the border is a radix selection over the weights' bits, eight at a
// time; survivors behind slot keep and the slots given up before it are then numbered in slot order, and the i-th survivor
// moves into the i-th slot given up.  Nothing is sorted and unmoved rows are not touched: a step's eviction moves one row a head.
// Numbering needs one prefix sum: with k(s) slots kept before slot s, a slot given up has number s - k(s), a survivor k(s) - k(keep).
// A cluster of up to 8 blocks takes a head, each a run of its slots, which it loads once and holds in shared memory; they
// exchange histograms and counts through each other's shared memory.  A head's blocks also make its moves where they are few;
// many are made by a second launch over all SMs.
// Bound by latency at serving sizes (seven exchanges and three trips to memory), by the weights' and positions' bytes past them.
#include <cuda_runtime.h>

#include "zl_internal.h"
#include "zl_kv4.cuh"
#include "zl_overlap.cuh"
#include "zl_ptx.cuh"

namespace zl {
namespace {

constexpr int kEvictThreads = 512;  // at least the bins of the first histogram
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kHeldSlots = 24576;  // that a block's shared memory has room for (8 bytes each)
constexpr int kCluster = 8;
constexpr int kMoveThreads = 256;
constexpr int kMoves = 128;        // moves that a block of the second launch makes
constexpr int kMovesApart = 256;   // moves a head from which on a second launch makes them

struct EvictParams {
  Kv4 c;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int32_t* counts;  // [sequence][key head]: moves, where a launch of their own makes them (else null)
  int2* moves;      // [sequence][key head][2][capacity]: slots given up, survivors: slot and tile
  int32_t keep, recent, capacity;
};

// Larger weights have larger numbers; NaN has the smallest, -0 is 0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; what each wrote before it, to shared or global memory, the others see after it.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An int of the same variable in another block of the cluster.
__device__ __forceinline__ int peer(const int* mine, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// Exclusive prefix of a number per warp over the block's warps (lane 0's counts); warp_sums is free again after the next sync.
__device__ __forceinline__ int before_warp(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) warp_sums[warp] = x;
  __syncthreads();
  const int x_of = lane < kEvictWarps ? warp_sums[lane] : 0;
  int run = x_of;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, run, i);
    if (lane >= i) run += y;
  }
  *total = __shfl_sync(0xffffffffu, run, 31);
  return __shfl_sync(0xffffffffu, run, warp) - __shfl_sync(0xffffffffu, x_of, warp);
}

// Moves i, i + step, .. of a head, kAtOnce of them, below `end`: 16 lanes a move, codes of keys and values in 16-byte pieces,
// scales, weight and position.  A lane's piece is found by a pointer rather than by branches, so that all loads are under way
// together (a register that two branches load into is waited for between them: 14 us instead of 5 for 1790 rows of each of 4 heads).
template <int D, int kAtOnce>
__device__ __forceinline__ void move_rows(const EvictParams& p, int item, int i, int step, int end) {
  const int l = threadIdx.x & 15;
  const int64_t base = (int64_t)item * ((int64_t)p.c.max_pages << p.c.page_shift);
  const int2* holes = p.moves + (int64_t)item * 2 * p.capacity;
  constexpr int kPieces = D / 32;  // of a row's codes
  const bool code = l < 2 * kPieces, scale = l >= 8 && l < 8 + 2 * (D / 64), number = l >= 14;
  // where a lane's piece of row 0 lies in a tile, and of the next row
  const int at = code ? (l / kPieces) * 8 * D + (l % kPieces) * 16 : 16 * D + ((l - 8) / (D / 64)) * D + ((l - 8) % (D / 64)) * 4;
  const int pitch = code ? D / 2 : D / 16;
  const uint8_t* in = reinterpret_cast<const uint8_t*>(l == 14 ? static_cast<const void*>(p.weights + base) : p.positions + base);
  uint8_t* out = reinterpret_cast<uint8_t*>(l == 14 ? static_cast<void*>(p.weights_out + base) : p.positions_out + base);
  int2 to[kAtOnce], from[kAtOnce];
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    const int j = min(i + y * step, end - 1);
    to[y] = holes[j];
    from[y] = holes[p.capacity + j];
  }
  uint4 v[kAtOnce];
  uint32_t u[kAtOnce];
  bool does[kAtOnce];
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    const bool bad = (uint32_t)to[y].y == kKv4None || (uint32_t)from[y].y == kKv4None;
    does[y] = i + y * step < end && (number || ((code || scale) && !bad));
    if (bad && l == 0 && i + y * step < end) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    const uint8_t* src = number ? in + (int64_t)from[y].x * 4 : p.c.data + (uint64_t)(uint32_t)from[y].y * (18 * D) + at + (from[y].x & 15) * pitch;
    if (does[y] && code) v[y] = *reinterpret_cast<const uint4*>(src);
    if (does[y] && !code) u[y] = *reinterpret_cast<const uint32_t*>(src);
  }
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    uint8_t* dst = number ? out + (int64_t)to[y].x * 4 : p.c.data + (uint64_t)(uint32_t)to[y].y * (18 * D) + at + (to[y].x & 15) * pitch;
    if (does[y] && code) *reinterpret_cast<uint4*>(dst) = v[y];
    if (does[y] && !code) *reinterpret_cast<uint32_t*>(dst) = u[y];
  }
}

// kHeld: the block's run of slots is kept in shared memory; else (runs past kHeldSlots) it is read again in each pass.
template <int D, bool kHeld>
__global__ void __launch_bounds__(kEvictThreads) zl_kv4_evict_kernel(const EvictParams p) {
  extern __shared__ int held[];  // [2][run]: ranks, positions
  __shared__ int hist[2][512];   // of two rounds in turn; the first round's: others, then the recent ones
  __shared__ int local[4][512];  // of a quarter of the warps
  __shared__ int sum[512];
  __shared__ int warp_sums[kEvictWarps];
  __shared__ int pub[4];  // read by the cluster: newest position, kept below `keep`, kept
  __shared__ int s_digit, s_above;
  const uint32_t cr = cluster_rank(), cn = cluster_size();
  const int item = blockIdx.x / cn, b = item / p.c.heads, h = item - b * p.c.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next_start();
  wait_for_previous();
  const int64_t base = (int64_t)item * ((int64_t)p.c.max_pages << p.c.page_shift);
  const float* w = p.weights + base;
  const int32_t* pos = p.positions + base;
  float* w_out = p.weights_out + base;
  int32_t* pos_out = p.positions_out + base;
  const bool copy_w = p.weights_out != p.weights, copy_pos = p.positions_out != p.positions;
  const int n = kv4_len(p.c, b), keep = p.keep;
  // this block's run of slots
  const int run = ((n + (int)cn - 1) / (int)cn + 31) / 32 * 32;
  const int lo = min(n, (int)cr * run), count = min(n, lo + run) - lo;
  if (n <= keep) {
    for (int i = tid; i < count; i += kEvictThreads) {
      if (copy_w) w_out[lo + i] = w[lo + i];
      if (copy_pos) pos_out[lo + i] = pos[lo + i];
    }
    if (p.counts && cr == 0 && tid == 0) p.counts[item] = 0;
    return;
  }
  uint32_t* held_rank = reinterpret_cast<uint32_t*>(held);
  int* held_pos = held + run;
  auto rank_at = [&](int i) { return kHeld ? held_rank[i] : rank_of(w[lo + i]); };
  auto pos_at = [&](int i) { return kHeld ? held_pos[i] : pos[lo + i]; };
  int newest = INT32_MIN;
#pragma unroll 4
  for (int i = tid; i < count; i += kEvictThreads) {
    const int at = pos[lo + i];
    if constexpr (kHeld) {
      held_rank[i] = rank_of(w[lo + i]);
      held_pos[i] = at;
    }
    newest = max(newest, at);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_sums[warp] = newest;
  for (int i = tid; i < 4 * 512; i += kEvictThreads) (&local[0][0])[i] = 0;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, warp_sums[lane % kEvictWarps]);
  if (cn > 1) {
    if (tid == 0) pub[0] = newest;
    cluster_sync();
    newest = __reduce_max_sync(0xffffffffu, peer(&pub[0], lane < cn ? lane : 0));
  }
  const int64_t border = (int64_t)newest - p.recent;

  // radix selection: after each round the border's leading digits, and how many of those that share them still count
  bool among_recent = false;  // the slots among which the weights decide: the recent ones where they alone are too many
  int need = 0, ties = 0;     // at the end: how many slots of the border's rank stay; how many lie in this block's run
  int ties_before = 0, ties_all = 0;
  uint32_t prefix = 0, mask = 0;
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round, bins = round == 0 ? 512 : 256;
    int* mine = local[warp & 3];
#pragma unroll 4
    for (int i = tid; i < count; i += kEvictThreads) {
      const bool recent = pos_at(i) > border;
      const uint32_t r = rank_at(i);
      if (round == 0) atomicAdd(&mine[(r >> 24) + (recent ? 256 : 0)], 1);
      else if (recent == among_recent && (r & mask) == prefix) atomicAdd(&mine[(r >> shift) & 255], 1);
    }
    __syncthreads();
    int* mine_all = hist[round & 1];
    if (tid < bins) {
      mine_all[tid] = local[0][tid] + local[1][tid] + local[2][tid] + local[3][tid];
#pragma unroll
      for (int i = 0; i < 4; ++i) local[i][tid] = 0;
    }
    if (cn > 1) cluster_sync();
    else __syncthreads();
    if (tid < bins) {
      int all = 0;
      if (cn > 1) for (uint32_t i = 0; i < cn; ++i) all += peer(&mine_all[tid], i);
      else all = mine_all[tid];
      sum[tid] = all;
    }
    __syncthreads();
    if (round == 0) {
      int safe = 0;
#pragma unroll
      for (int i = 0; i < 256; i += 32) safe += sum[256 + i + lane];
      safe = __reduce_add_sync(0xffffffffu, safe);
      among_recent = safe > keep;
      need = among_recent ? keep : keep - safe;
    }
    if (warp == 0) {
      // counts of digits from the top, eight a lane: the digit at which they reach `need`
      const int* bin = sum + (round == 0 && among_recent ? 256 : 0) + 248 - 8 * lane;
      int x[8], mine_sum = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine_sum += x[i] = bin[7 - i];
      int up = mine_sum;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, up, i);
        if (lane >= i) up += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, up >= need);
      if (lane == (hit ? __ffs(hit) - 1 : 31)) {
        int above = up - mine_sum, i = 0;
        while (i < 7 && above + x[i] < need) above += x[i++];
        s_digit = 255 - 8 * lane - i;
        s_above = above;
      }
    }
    __syncthreads();
    need -= s_above;
    prefix |= (uint32_t)s_digit << shift;
    mask |= 255u << shift;
    ties_all = sum[s_digit + (round == 0 && among_recent ? 256 : 0)];
    if (round == 3 || ties_all == need) {  // all that share the digits so far stay, or the digits are the border's rank itself
      const int* at = &mine_all[s_digit + (round == 0 && among_recent ? 256 : 0)];
      const int of = lane < cn ? (cn > 1 ? peer(at, lane) : *at) : 0;
      ties_before = __reduce_add_sync(0xffffffffu, lane < cr ? of : 0);
      ties = __shfl_sync(0xffffffffu, of, cr);
      break;
    }
  }
  // `need` of the slots at the border stay, the lowest ones.  Warps take contiguous parts of the run.
  const int part = ((count + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int i0 = min(count, warp * part), i1 = min(count, i0 + part);
  auto state = [&](int i) {  // 0: given up, 1: stays, 2: at the border
    if (i >= i1) return 0;
    const bool recent = pos_at(i) > border;
    if (recent != among_recent) return recent ? 1 : 0;
    const uint32_t r = rank_at(i) & mask;
    return r > prefix ? 1 : r == prefix ? 2 : 0;
  };
  int tie0 = ties_before;  // ties before this warp's part
  if (ties > 0 && need < ties_all) {
    int mine = 0, all;
    for (int i = i0; i < i1; i += 32) mine += __popc(__ballot_sync(0xffffffffu, state(i + lane) == 2));
    __syncthreads();
    tie0 += before_warp(mine, warp_sums, &all);
  }
  auto stays = [&](int i, int& tie) {  // of a warp's 32 slots from i on; tie: ties before them
    const int st = state(i + lane);
    const unsigned at_border = __ballot_sync(0xffffffffu, st == 2);
    const bool kept = st == 1 || (st == 2 && (need == ties_all || tie + __popc(at_border & ((1u << lane) - 1)) < need));
    tie += __popc(at_border);
    return kept;
  };
  int kept_front = 0, kept = 0, tie = tie0;
  for (int i = i0; i < i1; i += 32) {
    const unsigned k = __ballot_sync(0xffffffffu, stays(i, tie));
    kept += __popc(k);
    const int front = keep - (lo + i);  // of these 32 slots that many lie below `keep`
    if (front > 0) kept_front += __popc(front >= 32 ? k : k & ((1u << front) - 1));
  }
  __syncthreads();
  int front_all, kept_all;
  before_warp(kept_front, warp_sums, &front_all);
  __syncthreads();
  int k = before_warp(kept, warp_sums, &kept_all);  // slots kept before this warp's part
  if (cn > 1) {
    if (tid == 0) {
      pub[1] = front_all;
      pub[2] = kept_all;
    }
    cluster_sync();
    const int f = lane < cn ? peer(&pub[1], lane) : 0, a = lane < cr ? peer(&pub[2], lane) : 0;
    front_all = __reduce_add_sync(0xffffffffu, f);
    k += __reduce_add_sync(0xffffffffu, a);
  }
  int2* holes = p.moves + (int64_t)item * 2 * p.capacity;
  int2* movers = holes + p.capacity;
  tie = tie0;
  for (int i = i0; i < i1; i += 32) {
    const bool kept_here = stays(i, tie);
    const unsigned all = __ballot_sync(0xffffffffu, kept_here);
    const int slot = lo + i + lane, before = k + __popc(all & ((1u << lane) - 1));
    k += __popc(all);
    if (i + lane < i1) {
      // within the lists whatever happens to the inputs meanwhile
      if (!kept_here && slot < keep && slot - before < p.capacity) holes[slot - before] = make_int2(slot, kv4_place(p.c, b, h, slot));
      if (kept_here && slot >= keep && before - front_all < p.capacity) movers[before - front_all] = make_int2(slot, kv4_place(p.c, b, h, slot));
      if (kept_here && slot < keep) {
        if (copy_w) w_out[slot] = w[slot];
        if (copy_pos) pos_out[slot] = pos[slot];
      }
    }
  }
  const int moves = min(keep - front_all, p.capacity);
  if (p.counts) {
    if (cn > 1) cluster_sync();  // no block may end while another reads its shared memory
    if (cr == 0 && tid == 0) p.counts[item] = moves;
    return;
  }
  if (cn > 1) cluster_sync();
  else __syncthreads();
  constexpr int kGroups = kEvictThreads / 16;
  for (int i = (int)cr * kGroups; i < moves; i += (int)cn * kGroups) move_rows<D, 1>(p, item, i + tid / 16, kGroups, min(moves, i + kGroups));
}

// kMoves of a head a block.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) zl_kv4_move_kernel(const EvictParams p) {
  let_next_start();
  wait_for_previous();
  const int item = blockIdx.y + blockIdx.z * 65535;
  if (item >= p.c.n_seqs * p.c.heads) return;
  const int first = blockIdx.x * kMoves, moves = p.counts[item];
  if (first < moves) move_rows<D, kMoves * 16 / kMoveThreads>(p, item, first + threadIdx.x / 16, kMoveThreads / 16, min(moves, first + kMoves));
}

template <int D, bool kHeld>
cudaError_t launch_evict(const EvictParams& p, int cluster, int64_t items, int64_t run, cudaStream_t stream) {
  const auto kernel = zl_kv4_evict_kernel<D, kHeld>;
  static PerDeviceOnce once;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kHeld ? kHeldSlots * 8 : 0); });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * cluster));
  cfg.blockDim = dim3(kEvictThreads);
  cfg.dynamicSmemBytes = kHeld ? (size_t)run * 8 : 0;
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
  *bytes = round16(items * 4) + items * 2 * ((int64_t)cache->max_pages * cache->page / 2) * 8;
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
  if (items * kCluster > INT32_MAX) return ZL_ERR_UNSUPPORTED;
  p.weights = weights;
  p.positions = positions;
  p.weights_out = weights_out;
  p.positions_out = positions_out;
  p.moves = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + round16(items * 4));
  const int64_t most = slots - keep < keep ? slots - keep : keep;  // moves of a head at most
  const bool apart = most > kMovesApart;
  p.counts = apart ? static_cast<int32_t*>(workspace) : nullptr;
  p.keep = keep;
  p.recent = recent;
  p.capacity = (int32_t)(slots / 2);
  // blocks of a head: enough that a thread has four slots at most, as far as the SMs have room for two blocks each; more
  // where its slots would not fit their shared memory
  int cluster = 1;
  while (cluster < kCluster && ((slots > (int64_t)cluster * 4 * kEvictThreads && items * cluster * 2 <= 2 * sms) ||
                                slots > (int64_t)cluster * (kHeldSlots - 32)))
    cluster *= 2;
  const int64_t run = ((slots + cluster - 1) / cluster + 31) / 32 * 32;
  const bool held = run <= kHeldSlots;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->head_dim == 128) e = held ? launch_evict<128, true>(p, cluster, items, run, st) : launch_evict<128, false>(p, cluster, items, run, st);
  else e = held ? launch_evict<64, true>(p, cluster, items, run, st) : launch_evict<64, false>(p, cluster, items, run, st);
  if (e == cudaSuccess && apart) {
    const dim3 grid((unsigned)((most + kMoves - 1) / kMoves), (unsigned)(items < 65535 ? items : 65535), (unsigned)((items + 65534) / 65535));
    e = launch_overlapped(cache->head_dim == 128 ? zl_kv4_move_kernel<128> : zl_kv4_move_kernel<64>, grid, kMoveThreads, 0, st, p);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
