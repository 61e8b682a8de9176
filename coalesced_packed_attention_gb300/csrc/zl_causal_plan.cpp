// Host planner of the causal attention: validation, tiles, the split of long key ranges, and the static
// schedule (which thread block runs which tiles).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <queue>

#include "zl_causal.h"
#include "zl_internal.h"

using namespace zl;

namespace {

// Costs of the forward schedule in units of one 128-key step of a lone sub-tile (about 1.3 us): a step of two
// sub-tiles, a tile's start and end (Q load, first scores, epilogue), a part's fp32 output, and the merge's launch.
constexpr double kStep1 = 1.0, kStep2 = 1.2, kTileFixed = 1.5, kPartFixed = 1.0, kMergeFixed = 3.0;
// Backward: a query block of a key tile is the unit (about 2 us); a tile's start and end (K, V load, first products, dK,
// dV output), a part's fp32 output and its share of the sum, which the last launch does on its way.
constexpr double kBwdTileFixed = 2.0, kBwdPartFixed = 1.0, kBwdMergeFixed = 1.0;
// Schedules under some 100 us, in those units (see launch_overlapped_if).
constexpr double kShortFwd = 80.0, kShortBwd = 50.0;
// Longest tiles first balances best, but it spreads the blocks over every (sequence, head), and the tiles of one share
// what they read: keys and values forward; queries, dO and the dQ accumulator backward.  Where that does not stay in
// L2 (129 MB) and there are more (sequence, head) pairs than a handful of blocks each can share, the
// pairs are taken one after the other, longest tile first within each.
constexpr double kL2Bytes = 60e6;
constexpr int64_t kFewPairs = 16;

size_t align_up256(size_t n) { return (n + 255) & ~size_t(255); }

struct Load {
  double load;
  int32_t bin;
  bool operator>(const Load& o) const { return load > o.load || (load == o.load && bin > o.bin); }
};

// Greedy list schedule: each tile in turn to the block that is free first.  Returns the makespan; bin_of may be null.
double list_schedule(const std::vector<double>& cost, const std::vector<int32_t>& order, int bins,
                     std::vector<int32_t>* bin_of) {
  std::priority_queue<Load, std::vector<Load>, std::greater<Load>> free_at;
  for (int b = 0; b < bins; ++b) free_at.push({0.0, b});
  double makespan = 0.0;
  for (int32_t i : order) {
    Load l = free_at.top();
    free_at.pop();
    if (bin_of) (*bin_of)[i] = l.bin;
    l.load += cost[i];
    makespan = std::max(makespan, l.load);
    free_at.push(l);
  }
  return makespan;
}

// Lays the tiles out block by block in schedule order; ptr gets bins + 1 entries, bins = min(tiles, sms).
template <typename T>
double schedule(std::vector<T>* tiles, std::vector<double> cost, bool longest_first, int sms, std::vector<int32_t>* ptr) {
  const int n = (int)tiles->size(), bins = std::min(n, sms);
  ptr->assign(bins + 1, 0);
  if (n == 0) return 0.0;
  std::vector<int32_t> order(n), bin_of(n);
  for (int i = 0; i < n; ++i) order[i] = i;
  if (longest_first) std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) { return cost[a] > cost[b]; });
  const double makespan = list_schedule(cost, order, bins, &bin_of);
  for (int i = 0; i < n; ++i) ++(*ptr)[bin_of[i] + 1];
  for (int b = 0; b < bins; ++b) (*ptr)[b + 1] += (*ptr)[b];
  std::vector<int32_t> at(ptr->begin(), ptr->end() - 1);
  std::vector<T> out(n);
  for (int32_t i : order) out[at[bin_of[i]]++] = (*tiles)[i];
  tiles->swap(out);
  return makespan;
}

// Key blocks that the query block sees (its last token's keys), and whether it has tokens at all.
int blocks_seen(const CausalSeq& s, int block, int tb) {
  const int64_t tok = (int64_t)block * tb;
  if (tok >= s.q_len) return 0;
  const int64_t last = std::min<int64_t>(tok + tb, s.q_len);
  const int64_t seen = std::max<int64_t>(0, (int64_t)s.kv_len - s.q_len + last);
  return (int)((seen + 127) / 128);
}

// Pieces of a range of n units when pieces of about `chunk` are wanted (0: none).
int pieces(int n, int chunk) { return chunk > 0 && n > chunk ? (n + chunk - 1) / chunk : 1; }
int piece_at(int n, int k, int c) { return (int)((int64_t)n * c / k); }

// The piece size that gives the shortest schedule: no split, or pieces of about an even share of the work and
// fractions of it, at the price of `merge`.  cost_of(i, n, part) is the cost of n units of item i.
template <typename Item, typename Cost>
int choose_chunk(const std::vector<Item>& items, int sms, double merge, const Cost& cost_of) {
  auto makespan_of = [&](int chunk) {
    std::vector<double> cost;
    for (const Item& u : items) {
      const int k = pieces(u.n, chunk);
      for (int c = 0; c < k; ++c) cost.push_back(cost_of(u, piece_at(u.n, k, c + 1) - piece_at(u.n, k, c), k > 1));
    }
    std::vector<int32_t> order(cost.size());
    for (size_t i = 0; i < order.size(); ++i) order[i] = (int32_t)i;
    std::stable_sort(order.begin(), order.end(), [&](int32_t a, int32_t b) { return cost[a] > cost[b]; });
    return list_schedule(cost, order, std::min<int>((int)cost.size(), sms), nullptr);
  };
  double total = 0.0, longest = 0.0;
  for (const Item& u : items) {
    const double c = cost_of(u, u.n, false);
    total += c;
    longest = std::max(longest, c);
  }
  // many tiles to a block balance by themselves
  if (items.empty() || items.size() > 32u * sms) return 0;
  const double share = total / sms;
  double best = makespan_of(0);
  if (best < 1.04 * share) return 0;
  int chunk = 0;
  for (double f : {1.0, 0.7, 0.5, 0.35, 0.25, 0.15}) {
    const int c = std::max(2, (int)(share * f));
    const double m = makespan_of(c) + merge;
    if (m < 0.97 * best) {
      best = m;
      chunk = c;
    }
  }
  return chunk;
}

struct FwdItem {
  int32_t seq, head, block, n;
  bool two;
};

void build_forward(zl_causal_plan* p, const std::vector<int32_t>& by_len, bool resident) {
  const int tb = tokens_per_block(p->group);
  std::vector<FwdItem> all;
  for (int32_t i : by_len) {
    const CausalSeq& s = p->seqs[i];
    const int nqb = (int)(((int64_t)s.q_len + tb - 1) / tb);
    for (int32_t h = 0; h < p->n_kv_heads; ++h)
      for (int b = (nqb - 1) / 2 * 2; nqb > 0 && b >= 0; b -= 2)
        all.push_back({i, h, b, std::max(blocks_seen(s, b, tb), blocks_seen(s, b + 1, tb)), b + 1 < nqb});
  }
  auto cost_of = [](const FwdItem& u, int n, bool part) {
    return kTileFixed + n * (u.two ? kStep2 : kStep1) + (part ? kPartFixed : 0.0);
  };
  const int chunk = choose_chunk(all, p->num_sms, kMergeFixed, cost_of);
  std::vector<double> cost;
  for (const FwdItem& u : all) {
    const int k = pieces(u.n, chunk);
    const CausalSeq& s = p->seqs[u.seq];
    if (k > 1) {
      p->merges.push_back({u.seq, u.head, u.block, p->slots, k, {0, 0, 0}});
      const int toks = std::min(tb, s.q_len - (u.block + u.two) * tb);  // of the tile's last query block
      p->merge_rows = std::max(p->merge_rows, (u.two ? kCausalRows : 0) + toks * p->group);
    }
    for (int c = 0; c < k; ++c) {
      const int lo = piece_at(u.n, k, c), hi = piece_at(u.n, k, c + 1);
      p->fwd_tiles.push_back({(int32_t)s.q_offset, s.q_len, (int32_t)s.kv_offset, s.kv_len, u.head, u.block, lo, hi,
                              k > 1 ? p->slots++ : -1, u.seq, {0, 0}});
      cost.push_back(cost_of(u, hi - lo, k > 1));
    }
  }
  p->fwd_short = schedule(&p->fwd_tiles, cost, resident, p->num_sms, &p->fwd_ptr) < kShortFwd;
}

struct BwdItem {
  int32_t seq, head, block, first, n, nqb;
};

void build_backward(zl_causal_plan* p, const std::vector<int32_t>& by_len, bool resident) {
  const int tb = tokens_per_block(p->group);
  std::vector<BwdItem> all;
  for (int32_t i : by_len) {
    const CausalSeq& s = p->seqs[i];
    const int nqb = (int)(((int64_t)s.q_len + tb - 1) / tb);
    const int nkb = (int)(((int64_t)s.kv_len + 127) / 128);
    for (int32_t h = 0; h < p->n_kv_heads; ++h)
      for (int b = 0; b < nkb; ++b) {
        // the first token that sees the tile's first key
        const int64_t t0 = std::max<int64_t>(0, (int64_t)b * 128 - ((int64_t)s.kv_len - s.q_len));
        const int first = (int)std::min<int64_t>(nqb, t0 / tb);
        all.push_back({i, h, b, first, nqb - first, nqb});
      }
  }
  auto cost_of = [](const BwdItem&, int n, bool part) { return kBwdTileFixed + n + (part ? kBwdPartFixed : 0.0); };
  const int chunk = choose_chunk(all, p->num_sms, kBwdMergeFixed, cost_of);
  std::vector<double> cost;
  for (const BwdItem& u : all) {
    const int k = pieces(u.n, chunk);
    const CausalSeq& s = p->seqs[u.seq];
    if (k > 1) p->bwd_merges.push_back({(int32_t)s.kv_offset, s.kv_len, u.head, u.block, p->bwd_slots, k, {0, 0}});
    for (int c = 0; c < k; ++c) {
      const int lo = piece_at(u.n, k, c), hi = piece_at(u.n, k, c + 1);
      p->bwd_tiles.push_back({(int32_t)s.q_offset, s.q_len, (int32_t)s.kv_offset, s.kv_len, u.head, u.block,
                              (int32_t)(s.acc_block + (int64_t)u.head * u.nqb), u.first + lo, hi - lo,
                              k > 1 ? p->bwd_slots++ : -1, u.seq, 0});
      cost.push_back(cost_of(u, hi - lo, k > 1));
    }
  }
  p->bwd_short = schedule(&p->bwd_tiles, cost, resident, p->num_sms, &p->bwd_ptr) < kShortBwd;
}

template <typename T>
void put(std::vector<char>* blob, size_t at, const std::vector<T>& v) {
  if (!v.empty()) std::memcpy(blob->data() + at, v.data(), v.size() * sizeof(T));
}

zl_status upload_causal(zl_causal_plan* p) {
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up256(bytes);
    return here;
  };
  const size_t o_status = take(sizeof(int32_t));
  const size_t o_seqs = take(sizeof(CausalSeq) * p->seqs.size());
  const size_t o_ft = take(sizeof(CausalTile) * p->fwd_tiles.size());
  const size_t o_fp = take(sizeof(int32_t) * p->fwd_ptr.size());
  const size_t o_bt = take(sizeof(CausalBwdTile) * p->bwd_tiles.size());
  const size_t o_bp = take(sizeof(int32_t) * p->bwd_ptr.size());
  const size_t o_m = take(sizeof(CausalMerge) * p->merges.size());
  const size_t o_bm = take(sizeof(CausalBwdMerge) * p->bwd_merges.size());
  std::vector<char> blob(at, 0);
  put(&blob, o_seqs, p->seqs);
  put(&blob, o_ft, p->fwd_tiles);
  put(&blob, o_fp, p->fwd_ptr);
  put(&blob, o_bt, p->bwd_tiles);
  put(&blob, o_bp, p->bwd_ptr);
  put(&blob, o_m, p->merges);
  put(&blob, o_bm, p->bwd_merges);
  if (cudaMalloc(&p->dev_blob, at) != cudaSuccess) {
    p->dev_blob = nullptr;
    cudaGetLastError();
    return ZL_ERR_NO_MEMORY;
  }
  // the copy from pageable memory may still be on its way when the call returns; launches on other streams
  // do not wait for it, so it is awaited here
  if (cudaMemcpy(p->dev_blob, blob.data(), at, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaStreamSynchronize(nullptr) != cudaSuccess)
    return ZL_ERR_CUDA;
  char* base = static_cast<char*>(p->dev_blob);
  p->d_status = reinterpret_cast<int32_t*>(base + o_status);
  p->d_seqs = reinterpret_cast<CausalSeq*>(base + o_seqs);
  p->d_fwd_tiles = reinterpret_cast<CausalTile*>(base + o_ft);
  p->d_fwd_ptr = reinterpret_cast<int32_t*>(base + o_fp);
  p->d_bwd_tiles = reinterpret_cast<CausalBwdTile*>(base + o_bt);
  p->d_bwd_ptr = reinterpret_cast<int32_t*>(base + o_bp);
  p->d_merges = reinterpret_cast<CausalMerge*>(base + o_m);
  p->d_bwd_merges = reinterpret_cast<CausalBwdMerge*>(base + o_bm);
  return ZL_OK;
}

// True when two of the non-empty [offset, offset + len) share a row.
bool overlap(std::vector<std::pair<int64_t, int64_t>> r) {
  std::sort(r.begin(), r.end());
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].first < r[i - 1].first + r[i - 1].second) return true;
  return false;
}

zl_status build(const zl_causal_seq* seqs, int32_t n_seqs, uint32_t flags, zl_causal_plan* p) {
  const int64_t kMostRows = (int64_t)INT32_MAX - 512;  // TMA coordinates are 32-bit, a box may start near the end
  std::vector<std::pair<int64_t, int64_t>> q_rows, kv_rows;
  int64_t q_tiles = 0, kv_tiles = 0, kv_sum = 0;
  const int tb = tokens_per_block(p->group);
  for (int32_t i = 0; i < n_seqs; ++i) {
    const zl_causal_seq& s = seqs[i];
    if (s.q_len < 0 || s.kv_len < 0 || s.q_offset < 0 || s.kv_offset < 0 || s.q_offset > p->q_tokens ||
        s.q_len > p->q_tokens - s.q_offset || s.kv_offset > p->kv_tokens || s.kv_len > p->kv_tokens - s.kv_offset)
      return ZL_ERR_INVALID_ARG;
    if (s.q_len) q_rows.push_back({s.q_offset, s.q_len});
    if (s.kv_len) kv_rows.push_back({s.kv_offset, s.kv_len});
    const int64_t nqb = ((int64_t)s.q_len + tb - 1) / tb;
    p->seqs.push_back({s.q_offset, s.kv_offset, s.q_len, s.kv_len, p->acc_blocks});
    p->acc_blocks += nqb * p->n_kv_heads;
    q_tiles += (nqb + 1) / 2 * p->n_kv_heads;
    kv_tiles += ((int64_t)s.kv_len + 127) / 128 * p->n_kv_heads;
    kv_sum += s.kv_len;
  }
  if (p->q_tokens > kMostRows || p->kv_tokens > kMostRows || q_tiles > (1 << 28) || kv_tiles > (1 << 28) ||
      p->acc_blocks > INT32_MAX)
    return ZL_ERR_UNSUPPORTED;
  if (overlap(q_rows)) return ZL_ERR_INVALID_ARG;  // two sequences would write the same output rows
  p->shared_keys = overlap(kv_rows);
  std::vector<int32_t> by_len(n_seqs);
  for (int32_t i = 0; i < n_seqs; ++i) by_len[i] = i;
  std::stable_sort(by_len.begin(), by_len.end(), [&](int32_t a, int32_t b) { return seqs[a].kv_len > seqs[b].kv_len; });
  const bool few = (int64_t)n_seqs * p->n_kv_heads <= kFewPairs;
  build_forward(p, by_len, few || 4.0 * kv_sum * p->n_kv_heads * p->head_dim <= kL2Bytes);
  // of one row: q and dO in bf16, its accumulator in fp32
  build_backward(p, by_len, few || p->acc_blocks * 128 * 8.0 * p->head_dim <= kL2Bytes);
  const int64_t D = p->head_dim;
  p->fwd_bytes = (int64_t)p->slots * 256 * (D + 1) * 4;
  p->bwd_bytes = (int64_t)align_up256((size_t)(p->q_tokens * p->n_q_heads * 4)) + p->acc_blocks * 128 * D * 4 +
                 (int64_t)p->bwd_slots * 2 * 128 * D * 4;
  return p->host_only ? ZL_OK : upload_causal(p);
}

}  // namespace

extern "C" zl_status zl_plan_causal(const zl_causal_seq* seqs, int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                    int32_t head_dim, int64_t q_tokens, int64_t kv_tokens, uint32_t flags,
                                    zl_causal_plan** out) {
  NvtxRange range("zl_plan_causal");
  if (!out) return ZL_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_seqs < 0 || (n_seqs > 0 && !seqs) || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || q_tokens < 0 ||
      kv_tokens < 0 || (flags & ~(ZL_PLAN_HOST_ONLY | ZL_PLAN_TEST_WITHHOLD_LOAD)))
    return ZL_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128) || n_q_heads / n_kv_heads > kCausalRows || n_q_heads > 65536)
    return ZL_ERR_UNSUPPORTED;
  zl_causal_plan* p = new (std::nothrow) zl_causal_plan;
  if (!p) return ZL_ERR_NO_MEMORY;
  p->n_q_heads = n_q_heads;
  p->n_kv_heads = n_kv_heads;
  p->head_dim = head_dim;
  p->group = n_q_heads / n_kv_heads;
  p->q_tokens = q_tokens;
  p->kv_tokens = kv_tokens;
  p->host_only = flags & ZL_PLAN_HOST_ONLY;
  p->test_withhold = flags & ZL_PLAN_TEST_WITHHOLD_LOAD;
  p->num_sms = 152;
  zl_status s = ZL_OK;
  if (!p->host_only) {
    int major = 0, minor = 0;
    if (cudaGetDevice(&p->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, p->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, p->device) != cudaSuccess)
      s = ZL_ERR_CUDA;
    else if (major != 10 || minor != 3)
      s = ZL_ERR_UNSUPPORTED;
  }
  if (s == ZL_OK) {
    try {
      s = build(seqs, n_seqs, flags, p);
    } catch (const std::bad_alloc&) {
      s = ZL_ERR_NO_MEMORY;
    } catch (...) {  // nothing may leave a C entry point
      s = ZL_ERR_INVALID_ARG;
    }
  }
  if (s != ZL_OK) {
    zl_causal_plan_destroy(p);
    return s;
  }
  *out = p;
  return ZL_OK;
}

extern "C" void zl_causal_plan_destroy(zl_causal_plan* p) {
  if (!p) return;
  if (p->dev_blob) {
    int dev = -1;
    const bool other = cudaGetDevice(&dev) == cudaSuccess && dev != p->device;
    if (other) cudaSetDevice(p->device);
    cudaFree(p->dev_blob);
    if (other) cudaSetDevice(dev);
  }
  delete p;
}

extern "C" zl_status zl_causal_plan_workspace(const zl_causal_plan* p, int64_t* fwd_bytes, int64_t* bwd_bytes) {
  if (!p) return ZL_ERR_INVALID_ARG;
  if (fwd_bytes) *fwd_bytes = p->fwd_bytes;
  if (bwd_bytes) *bwd_bytes = p->bwd_bytes;
  return ZL_OK;
}

extern "C" zl_status zl_causal_plan_tiles(const zl_causal_plan* p, int32_t which, int32_t* out, int64_t cap, int64_t* n) {
  if (!p || !n || cap < 0 || (cap > 0 && !out) || which < 0 || which > 1) return ZL_ERR_INVALID_ARG;
  const std::vector<int32_t>& ptr = which == 0 ? p->fwd_ptr : p->bwd_ptr;
  *n = which == 0 ? (int64_t)p->fwd_tiles.size() : (int64_t)p->bwd_tiles.size();
  for (size_t b = 0; b + 1 < ptr.size(); ++b)
    for (int32_t i = ptr[b]; i < ptr[b + 1] && i < cap; ++i) {
      int32_t* o = out + 7 * (int64_t)i;
      if (which == 0) {
        const CausalTile& t = p->fwd_tiles[i];
        const int32_t v[7] = {t.seq, t.head, t.block, t.kv_lo, t.kv_hi, t.part, (int32_t)b};
        std::memcpy(o, v, sizeof(v));
      } else {
        const CausalBwdTile& t = p->bwd_tiles[i];
        const int32_t v[7] = {t.seq, t.head, t.block, t.first, t.first + t.n, t.part, (int32_t)b};
        std::memcpy(o, v, sizeof(v));
      }
    }
  return ZL_OK;
}
