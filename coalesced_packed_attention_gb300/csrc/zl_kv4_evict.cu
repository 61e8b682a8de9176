// Eviction from the 4-bit cache by accumulated attention weight.
//
// Every (sequence, key head) keeps `keep` of its n slots: those with a position above newest - recent first, then the
// largest weights, ties to the lower slot.  Finding the border is a radix selection over the weights' bits, eight at a
// time; survivors behind slot keep and the slots given up before it are then numbered in slot order, and the i-th
// survivor moves into the i-th slot given up.  Nothing is sorted and unmoved rows are not touched: a step's eviction
// moves one row a head.  Numbering needs one prefix sum: with k(s) slots kept before slot s, a slot given up has number
// s - k(s), a survivor k(s) - k(keep).  A cluster of up to 8 blocks takes a head, each a run of its slots, which it
// loads once and holds in shared memory; they exchange histograms and counts through each other's shared memory.  A
// head's blocks also make its moves where they are few; many are made by a second launch over all SMs.
// Bound by latency at serving sizes (seven exchanges and three trips to memory), by the weights' and positions' bytes
// past them.  Measured: one of 1025 slots of each of 64 heads 7.5 us; 16 384 slots of 4 heads to 2048 15 us and 4.5 for
// the moves; 32 x 8 heads of 100 to 8192 slots to 2048, d = 64, 22 us and 21.
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
constexpr int kFew = 4;            // slots given up that are looked for one by one
constexpr int kMoveThreads = 256;
constexpr int kMoves = 64;         // moves that a block of the second launch makes
constexpr uint32_t kGone = 0x80000000u;  // of a listed slot: its row is not there
constexpr int kMovesApart = 256;   // moves a head from which on a second launch makes them

struct EvictParams {
  Kv4 c;
  const float* weights;
  const int32_t* positions;
  float* weights_out;
  int32_t* positions_out;
  int32_t* counts;  // [sequence][key head]: moves, where a launch of their own makes them (else null)
  // [sequence][key head][4][capacity]: slots given up, their rows; survivors' slots, their rows (16 tile + row); see kGone
  uint32_t* moves;
  int32_t keep, recent, capacity;
};

// Larger weights have larger numbers; NaN has the smallest, -0 is 0.
__device__ __forceinline__ uint32_t rank_of(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  const uint32_t r = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return w == w ? r : 0;
}

// An int of the same variable in another block of the cluster.
__device__ __forceinline__ int peer(const int* mine, uint32_t rank) {
  uint32_t a;
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(mine)), "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// 16 lanes a move: codes of keys and values in 16-byte pieces, scales, weight and position.  A lane's piece of a slot
// or of a row is found by a pointer rather than by branches, so that all loads are under way together (a register that
// two branches load into is waited for between them: 14 us instead of 5 for 1790 rows of each of 4 heads).
template <int D>
struct Piece {
  static constexpr int kPieces = D / 32;  // of a row's codes
  bool code, number, idle;
  int at, pitch;
  const uint8_t* in;
  uint8_t* out;
  __device__ Piece(const EvictParams& p, int64_t base) {
    const int l = threadIdx.x & 15;
    code = l < 2 * kPieces;
    number = l >= 14;
    idle = !code && !number && (l < 8 || l >= 8 + 2 * (D / 64));
    at = code ? (l / kPieces) * 8 * D + (l % kPieces) * 16 : 16 * D + ((l - 8) / (D / 64)) * D + ((l - 8) % (D / 64)) * 4;
    pitch = number ? 4 : code ? D / 2 : D / 16;
    in = l == 14   ? reinterpret_cast<const uint8_t*>(p.weights + base)
         : l == 15 ? reinterpret_cast<const uint8_t*>(p.positions + base)
                   : p.c.data;
    out = l == 14   ? reinterpret_cast<uint8_t*>(p.weights_out + base)
          : l == 15 ? reinterpret_cast<uint8_t*>(p.positions_out + base)
                    : p.c.data;
  }
  // bytes to the piece of slot or row x
  __device__ int64_t offset(uint32_t x) const {
    return number ? (int64_t)(x & ~kGone) * 4 : (int64_t)(x >> 4) * (18 * D) + at + (x & 15) * pitch;
  }
};
// Moves i, i + step, .. of a head, kAtOnce of them, whose numbers of slots or rows (a lane's own kind) are known.
template <int D, int kAtOnce>
__device__ __forceinline__ void move_pieces(const EvictParams& p, const Piece<D>& piece, const uint32_t (&to)[kAtOnce],
                                            const uint32_t (&from)[kAtOnce], int i, int step, int end) {
  uint4 v[kAtOnce];
  uint32_t u[kAtOnce];
  bool does[kAtOnce];
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    const bool in = i + y * step < end;
    // a row that is not there takes its weight and position out of the move, too: the slot given up keeps its own
    const bool bad = piece.number ? (int32_t)(to[y] | from[y]) < 0 : to[y] == kKv4None || from[y] == kKv4None;
    does[y] = in && !piece.idle && (piece.number || !bad);
    if (in && bad && (threadIdx.x & 15) == 0) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    const uint8_t* src = piece.in + piece.offset(piece.number && bad ? to[y] : from[y]);
    if (does[y] && piece.code) v[y] = *reinterpret_cast<const uint4*>(src);
    if (does[y] && !piece.code) u[y] = *reinterpret_cast<const uint32_t*>(src);
  }
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    uint8_t* dst = piece.out + piece.offset(to[y]);
    if (does[y] && piece.code) *reinterpret_cast<uint4*>(dst) = v[y];
    if (does[y] && !piece.code) *reinterpret_cast<uint32_t*>(dst) = u[y];
  }
}

// The same for one move whose slots are known: from slot `from` to slot `to`.
template <int D>
__device__ __forceinline__ void move_row(const EvictParams& p, int b, int h, int64_t base, int to, int from) {
  const int l = threadIdx.x & 15;
  uint8_t* dst = kv4_tile<D>(p.c, b, h, to);
  const uint8_t* src = kv4_tile<D>(p.c, b, h, from);
  const bool bad = !dst || !src;
  if (l == 14) p.weights_out[base + to] = p.weights[base + (bad ? to : from)];
  if (l == 15) p.positions_out[base + to] = p.positions[base + (bad ? to : from)];
  if (bad) {
    if (l == 0) kv4_report(p.c, ZL_KV4_BAD_PAGE);
    return;
  }
  constexpr int kPieces = D / 32;
  const int r0 = to & 15, r1 = from & 15;
  if (l < 2 * kPieces) {
    const int at = (l / kPieces) * 8 * D + (l % kPieces) * 16;
    *reinterpret_cast<uint4*>(dst + at + r0 * (D / 2)) = *reinterpret_cast<const uint4*>(src + at + r1 * (D / 2));
  } else if (l >= 8 && l < 8 + 2 * (D / 64)) {
    const int at = 16 * D + ((l - 8) / (D / 64)) * D + ((l - 8) % (D / 64)) * 4;
    *reinterpret_cast<uint32_t*>(dst + at + r0 * (D / 16)) = *reinterpret_cast<const uint32_t*>(src + at + r1 * (D / 16));
  }
}

// kHeld: the block's run of slots is kept in shared memory; else (runs past kHeldSlots) it is read again in each pass.
template <int D, bool kHeld>
__global__ void __launch_bounds__(kEvictThreads) zl_kv4_evict_kernel(const EvictParams p) {
  extern __shared__ int held[];            // [2][run]: weights, positions
  __shared__ int local[4][512];            // a round's histogram, of a quarter of the warps; the first's: others, then recent ones
  __shared__ int hist[2][512];             // of the block, of two rounds in turn
  __shared__ int warp_sums[2][kEvictWarps];
  __shared__ uint64_t warp_least[kEvictWarps];
  __shared__ uint32_t kept_bits[kHeld ? kHeldSlots / 32 : 1];  // of 32 slots each: which stay
  __shared__ int pub[4];                   // read by the cluster: newest position, kept below `keep`, kept
  __shared__ int s_digit, s_above, s_count;
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
  float* held_w = reinterpret_cast<float*>(held);
  int* held_pos = held + run;
  auto w_at = [&](int i) { return kHeld ? held_w[i] : w[lo + i]; };
  auto pos_at = [&](int i) { return kHeld ? held_pos[i] : pos[lo + i]; };
  int newest = INT32_MIN;
#pragma unroll 8
  for (int i = tid; i < count; i += kEvictThreads) {
    const int at = pos[lo + i];
    if constexpr (kHeld) {
      held_w[i] = w[lo + i];
      held_pos[i] = at;
    }
    newest = max(newest, at);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_sums[0][warp] = newest;
  if (tid == 0) s_digit = s_above = s_count = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) local[i][tid] = 0;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, warp_sums[0][lane % kEvictWarps]);
  if (cn > 1) {
    if (tid == 0) pub[0] = newest;
    cluster_sync();
    newest = __reduce_max_sync(0xffffffffu, peer(&pub[0], lane < cn ? lane : 0));
  }
  // position above newest - p.recent: the difference fits 32 bits without a sign
  auto is_recent = [&](int at) { return (uint32_t)newest - (uint32_t)at < (uint32_t)p.recent; };

  // A step gives up a slot or a few: the least in claim, one after another, and no selection by digits.
  if (cn == 1 && kHeld && n - keep <= kFew) {
    int gone[kFew];
#pragma unroll
    for (int y = 0; y < kFew; ++y) {
      gone[y] = INT32_MAX;
      if (y >= n - keep) continue;
      // 33 bits of claim, then 31 of the slot: the highest of equals goes first
      uint64_t least = ~0ull;
      for (int i = tid; i < n; i += kEvictThreads) {
        bool out = false;
#pragma unroll
        for (int z = 0; z < y; ++z) out |= gone[z] == i;
        const uint64_t claim = ((uint64_t)(is_recent(held_pos[i]) ? 1 : 0) << 63) | ((uint64_t)rank_of(held_w[i]) << 31) |
                               (uint32_t)(INT32_MAX - i);
        if (!out && claim < least) least = claim;
      }
#pragma unroll
      for (int i = 16; i > 0; i >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, least, i);
        least = other < least ? other : least;
      }
      if (lane == 0) warp_least[warp] = least;
      __syncthreads();
      least = warp_least[lane % kEvictWarps];
#pragma unroll
      for (int i = kEvictWarps / 2; i > 0; i >>= 1) {
        const uint64_t other = __shfl_xor_sync(0xffffffffu, least, i);
        least = other < least ? other : least;
      }
      gone[y] = INT32_MAX - (int)(least & INT32_MAX);
      __syncthreads();  // the warps' least ones have been read
    }
    if (copy_w || copy_pos)
      for (int i = tid; i < keep; i += kEvictThreads) {
        bool out = false;
#pragma unroll
        for (int y = 0; y < kFew; ++y) out |= gone[y] == i;
        if (out) continue;
        if (copy_w) w_out[i] = held_w[i];
        if (copy_pos) pos_out[i] = held_pos[i];
      }
    // the i-th survivor in the last slots and the i-th slot given up before them, by counting; 16 lanes a move
    int to = INT32_MAX, from = INT32_MAX, moves = 0;
    const int i = tid / 16;
#pragma unroll
    for (int y = 0; y < kFew; ++y) {
      int before = 0;
#pragma unroll
      for (int z = 0; z < kFew; ++z) before += gone[z] < gone[y];
      if (gone[y] < keep) {
        ++moves;
        if (before == i) to = gone[y];
      }
    }
    int number = 0;
    for (int slot = keep; slot < n; ++slot) {
      bool out = false;
#pragma unroll
      for (int y = 0; y < kFew; ++y) out |= gone[y] == slot;
      if (!out && number++ == i) from = slot;
    }
    if (p.counts) {  // for the launch that follows
      if (tid == 0) p.counts[item] = 0;
    }
    if (i < moves && from < n) move_row<D>(p, b, h, base, to, from);
    return;
  }

  // radix selection: after each round the border's leading digits, and how many of those that share them still count
  bool among_recent = false;  // the slots among which the weights decide: the recent ones where they alone are too many
  int need = 0;               // how many slots of the border's digits stay ..
  int ties_all = 0, ties = 0, ties_before = 0;  // .. of how many there are: in all, in this block's run, before it
  uint32_t prefix = 0, mask = 0;
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    int* mine = local[warp & 3];
#pragma unroll 4
    for (int i = tid; i < count; i += kEvictThreads) {
      const bool recent = is_recent(pos_at(i));
      const uint32_t r = rank_of(w_at(i));
      // the largest digit first: threads below number them so
      if (round == 0) atomicAdd(&mine[(255 - (r >> 24)) + (recent ? 256 : 0)], 1);
      else if (recent == among_recent && (r & mask) == prefix) atomicAdd(&mine[255 - ((r >> shift) & 255)], 1);
    }
    __syncthreads();
    int* of_block = hist[round & 1];
    int x = local[0][tid] + local[1][tid] + local[2][tid] + local[3][tid];
    of_block[tid] = x;
    if (cn > 1) {
      cluster_sync();
      int of_peer[kCluster];
#pragma unroll
      for (uint32_t i = 0; i < kCluster; ++i) of_peer[i] = peer(&of_block[tid], min(i, cn - 1));
      x = 0;
#pragma unroll
      for (uint32_t i = 0; i < kCluster; ++i) x += i < cn ? of_peer[i] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) local[i][tid] = 0;
    // counts of digits from the top, of 256 threads each: where they reach `need`
    int up = x;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, up, i);
      if (lane >= i) up += y;
    }
    if (lane == 31) warp_sums[round & 1][warp] = up;
    __syncthreads();
    const int sums = lane < kEvictWarps ? warp_sums[round & 1][lane] : 0;
    if (round == 0) {
      const int safe = __reduce_add_sync(0xffffffffu, lane >= 8 ? sums : 0);
      among_recent = safe > keep;
      need = among_recent ? keep : keep - safe;
    }
    const int of = round == 0 && among_recent ? 8 : 0;  // the first warp of the digits that decide
    const int above = up - x + __reduce_add_sync(0xffffffffu, lane >= of && lane < warp ? sums : 0);
    if (warp >= of && warp < of + 8 && ((above < need && above + x >= need) || (need == 0 && tid == 32 * of))) {
      s_digit = tid & 255;
      s_above = above;
      s_count = x;
    }
    __syncthreads();
    need -= s_above;
    ties_all = s_count;
    prefix |= (uint32_t)(255 - s_digit) << shift;
    mask |= 255u << shift;
    if (round == 3 || ties_all == need) {  // all that share the digits so far stay, or the digits are the border's rank itself
      const int* at = &of_block[s_digit + 32 * of];
      const int there = lane < cn ? (cn > 1 ? peer(at, lane) : *at) : 0;
      ties_before = __reduce_add_sync(0xffffffffu, lane < cr ? there : 0);
      ties = __shfl_sync(0xffffffffu, there, cr);
      break;
    }
  }
  // `need` of the slots at the border stay, the lowest ones.  Warps take contiguous parts of the run.
  const int part = ((count + kEvictWarps - 1) / kEvictWarps + 31) / 32 * 32;
  const int i0 = min(count, warp * part), i1 = min(count, i0 + part);
  // of a warp's 32 slots from i on, as bits: those that stay for sure and those at the border
  auto states = [&](int i, uint32_t* border) {
    const bool in = i + lane < i1;
    const int at = in ? i + lane : i0;
    const bool recent = is_recent(pos_at(at)), decides = recent == among_recent;
    const uint32_t r = rank_of(w_at(at)) & mask;
    *border = __ballot_sync(0xffffffffu, in & decides & (r == prefix));
    return __ballot_sync(0xffffffffu, in & (decides ? r > prefix : recent));
  };
  const bool all_ties = need == ties_all;
  int tie0 = ties_before;  // ties before this warp's part
  if (ties > 0 && !all_ties) {
    int mine = 0;
    for (int i = i0; i < i1; i += 32) {
      uint32_t border;
      states(i, &border);
      mine += __popc(border);
    }
    __syncthreads();  // the rounds' sums have been read
    if (lane == 0) warp_sums[0][warp] = mine;
    __syncthreads();
    tie0 += __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[0][lane % kEvictWarps] : 0);
  }
  auto stays = [&](int i, int& tie) {  // those that stay; tie: ties before them
    uint32_t border;
    const uint32_t sure = states(i, &border);
    if (all_ties) return sure | border;
    const bool in = tie + __popc(border & ((1u << lane) - 1)) < need;
    tie += __popc(border);
    return sure | (border & __ballot_sync(0xffffffffu, in));
  };
  int kept_front = 0, kept = 0, tie = tie0;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = stays(i, tie);
    if constexpr (kHeld)
      if (lane == 0) kept_bits[i / 32] = k;
    kept += __popc(k);
    const int front = min(max(keep - (lo + i), 0), 32);  // of these 32 slots that many lie below `keep`
    kept_front += __popc(k & (uint32_t)((1ull << front) - 1));
  }
  __syncthreads();  // sums have been read
  if (lane == 0) {
    warp_sums[0][warp] = kept_front;
    warp_sums[1][warp] = kept;
  }
  __syncthreads();
  const int sum0 = lane < kEvictWarps ? warp_sums[0][lane] : 0, sum1 = lane < kEvictWarps ? warp_sums[1][lane] : 0;
  int front_all = __reduce_add_sync(0xffffffffu, sum0);               // kept below `keep`
  int k = __reduce_add_sync(0xffffffffu, lane < warp ? sum1 : 0);     // kept before this warp's part
  if (cn > 1) {
    const int kept_all = __reduce_add_sync(0xffffffffu, sum1);
    if (tid == 0) {
      pub[1] = front_all;
      pub[2] = kept_all;
    }
    cluster_sync();
    const int f = lane < cn ? peer(&pub[1], lane) : 0, a = lane < cr ? peer(&pub[2], lane) : 0;
    front_all = __reduce_add_sync(0xffffffffu, f);
    k += __reduce_add_sync(0xffffffffu, a);
  }
  uint32_t* list = p.moves + (int64_t)item * 4 * p.capacity;
  tie = tie0;
  // four times 32 slots at a time, their pages' loads under way together
  constexpr int kAtOnce = 4;
  for (int i = i0; i < i1; i += 32 * kAtOnce) {
    int at[kAtOnce];
    uint32_t place[kAtOnce];
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      at[y] = -1;
      if (i + 32 * y >= i1) continue;  // the whole warp
      const uint32_t all = kHeld ? kept_bits[i / 32 + y] : stays(i + 32 * y, tie);
      const int mine = i + 32 * y + lane, slot = lo + mine, before = k + __popc(all & ((1u << lane) - 1));
      const bool kept_here = (all >> lane) & 1, front = slot < keep;
      k += __popc(all);
      if (mine < i1 && kept_here != front) at[y] = front ? slot - before : 2 * p.capacity + before - front_all;
      if (mine < i1 && kept_here && front) {
        if (copy_w) w_out[slot] = w_at(mine);
        if (copy_pos) pos_out[slot] = pos_at(mine);
      }
    }
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) place[y] = at[y] >= 0 ? kv4_place(p.c, b, h, lo + i + 32 * y + lane) : 0;
#pragma unroll
    for (int y = 0; y < kAtOnce; ++y) {
      // within the lists whatever happens to the inputs meanwhile
      if (at[y] < 0 || (at[y] < 2 * p.capacity ? at[y] : at[y] - 2 * p.capacity) >= p.capacity) continue;
      const int slot = lo + i + 32 * y + lane;
      list[at[y]] = place[y] == kKv4None ? slot | kGone : slot;
      list[at[y] + p.capacity] = place[y] == kKv4None ? kKv4None : place[y] * 16 + (slot & 15);
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
  const Piece<D> piece(p, base);
  const uint32_t* mine = list + (piece.number ? 0 : p.capacity);
  for (int i = (int)cr * kGroups + tid / 16; i < moves; i += (int)cn * kGroups) {
    const uint32_t to[1] = {mine[i]}, from[1] = {mine[i + 2 * p.capacity]};
    move_pieces<D, 1>(p, piece, to, from, i, 0, moves);
  }
}

// kMoves of a head a block, four in each group of 16 lanes; the list is loaded before it is known how far it reaches.
template <int D>
__global__ void __launch_bounds__(kMoveThreads) zl_kv4_move_kernel(const EvictParams p) {
  let_next_start();
  wait_for_previous();
  const int item = blockIdx.y + blockIdx.z * 65535;
  if (item >= p.c.n_seqs * p.c.heads) return;
  constexpr int kGroups = kMoveThreads / 16, kAtOnce = kMoves / kGroups;
  const Piece<D> piece(p, (int64_t)item * ((int64_t)p.c.max_pages << p.c.page_shift));
  const uint32_t* mine = p.moves + (int64_t)item * 4 * p.capacity + (piece.number ? 0 : p.capacity);
  const int i = blockIdx.x * kMoves + threadIdx.x / 16;
  uint32_t to[kAtOnce], from[kAtOnce];
#pragma unroll
  for (int y = 0; y < kAtOnce; ++y) {
    const int at = min(i + y * kGroups, p.capacity - 1);
    to[y] = mine[at];
    from[y] = mine[at + 2 * p.capacity];
  }
  const int moves = p.counts[item];
  if (blockIdx.x * kMoves < moves) move_pieces<D, kAtOnce>(p, piece, to, from, i, kGroups, moves);
}

template <int D, bool kHeld>
cudaError_t launch_evict(const EvictParams& p, int cluster, int64_t items, int64_t run, cudaStream_t stream) {
  const auto kernel = zl_kv4_evict_kernel<D, kHeld>;
  static PerDeviceOnce once;
  constexpr int kMost = kHeld ? kHeldSlots * 8 : 0;
  cudaError_t e = once.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost); });
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
  *bytes = round16(items * 4) + items * 4 * ((int64_t)cache->max_pages * cache->page / 2) * 4;
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
  p.moves = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + round16(items * 4));
  const int64_t most = slots - keep < keep ? slots - keep : keep;  // moves of a head at most
  const bool apart = most > kMovesApart;
  p.counts = apart ? static_cast<int32_t*>(workspace) : nullptr;
  p.keep = keep;
  p.recent = recent;
  p.capacity = (int32_t)(slots / 2);
  // blocks of a head: enough that a thread has four slots at most, as far as the SMs have room for two blocks each;
  // more where its slots would not fit their shared memory
  int cluster = 1;
  while (cluster < kCluster && ((slots > (int64_t)cluster * 4 * kEvictThreads && items * cluster * 2 <= 2 * sms) ||
                                slots > (int64_t)cluster * (kHeldSlots - 32)))
    cluster *= 2;
  const int64_t run = ((slots + cluster - 1) / cluster + 31) / 32 * 32;
  const bool held = run <= kHeldSlots;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->head_dim == 128)
    e = held ? launch_evict<128, true>(p, cluster, items, run, st) : launch_evict<128, false>(p, cluster, items, run, st);
  else
    e = held ? launch_evict<64, true>(p, cluster, items, run, st) : launch_evict<64, false>(p, cluster, items, run, st);
  if (e == cudaSuccess && apart) {
    const dim3 grid((unsigned)((most + kMoves - 1) / kMoves), (unsigned)(items < 65535 ? items : 65535),
                    (unsigned)((items + 65534) / 65535));
    const auto kernel = cache->head_dim == 128 ? zl_kv4_move_kernel<128> : zl_kv4_move_kernel<64>;
    e = launch_overlapped(kernel, grid, kMoveThreads, 0, st, p);
  }
  return e == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
