// Host planner of the causal attention: validation, tiles, the split of long key ranges, and the static
// schedule (which thread block runs which tiles).
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <mutex>
#include <new>
#include <utility>

#include "zl_causal.h"
#include "zl_internal.h"

using namespace zl;

namespace {

// What a schedule is weighed by, in microseconds as measured on one GB300 (kernels of a few tiles a thread block):
// a step (forward: 128 keys of one or of two sub-tiles; backward: a query block of a key tile), a tile's start and
// end, a part's fp32 output, and for the sum of the parts a launch (forward; the backward's last launch is there
// anyway) and their bytes, written and read again at some 2.4 TB/s in all.
struct Rates {
  double step1, step2, fixed, part, merge, part_bytes;
};
Rates fwd_rates(int d) { return d == 128 ? Rates{1.4, 1.5, 2.0, 0.7, 3.5, 256.0 * 128 * 4} : Rates{1.15, 1.35, 1.8, 0.5, 3.5, 256.0 * 64 * 4}; }
Rates bwd_rates(int d) { return d == 128 ? Rates{2.15, 2.15, 4.5, 1.0, 0.5, 256.0 * 128 * 4} : Rates{1.75, 1.75, 4.0, 0.7, 0.5, 256.0 * 64 * 4}; }
constexpr double kPartBytesPerUs = 2.4e6;  // of the parts, written and then read
// A launch shorter than this is set up early (see launch_overlapped_if).
constexpr double kShortUs = 100.0;
// Longest tiles first balances best, but it spreads the blocks over every (sequence, head), and the tiles of one share
// what they read: keys and values forward; queries, dO and the dQ accumulator backward.  Where that does not stay in
// L2 (129 MB) and there are more (sequence, head) pairs than a handful of blocks each can share, the
// pairs are taken one after the other, longest tile first within each.  Longest first against pair by pair, us: forward, MB
// of keys and values: 34 MB 116 / 123, 67 MB 381 / 392, 134 MB 1470 / 1468, 268 MB 2959 / 2925; gradient, MB of queries,
// dO and accumulator: 31 MB 69 / 68, 268 MB 751 / 762, 537 MB 1218 / 1294, 1074 MB 4746 / 4517, 2147 MB 12 974 / 8822;
// gradient of one sequence, pairs: 4 of 16 384 tokens 4306 / 4425, 8 of 32 768 4230 / 4155, 16 9120 / 8343.  (Between
// 60 and 500 MB either order is within 6 % of the other.)
constexpr double kL2Bytes = 60e6;
constexpr int64_t kFewPairs = 16;
// Up to this much of queries, dO and accumulator the backward's walks may be cut at an even load: 79 MB, 132 us
// against 139 in equal pieces; 92 MB, 160 against 156 whole; 325 MB, 2450 against 2262.
constexpr double kCutBytes = 85e6;

size_t align_up256(size_t n) { return (n + 255) & ~size_t(255); }

// Pieces of the items (query blocks forward, key tiles backward) in the order and on the thread blocks that run
// them: units [lo, hi) of an item's n.
struct Piece {
  int32_t item, lo, hi, bin;
  bool cut;  // one of several of its item
};

// Thread blocks by load, the least loaded (then the lowest) first: a binary heap of which only the top ever grows.
struct LeastLoaded {
  std::vector<std::pair<double, int32_t>> heap;
  explicit LeastLoaded(int n) {
    for (int b = 0; b < n; ++b) heap.push_back({0.0, b});
  }
  // Adds to the top block's load; returns the block and its load.
  std::pair<double, int32_t> add(double cost) {
    std::pair<double, int32_t> top = heap[0];
    top.first += cost;
    size_t i = 0;
    for (;;) {
      size_t c = 2 * i + 1;
      if (c >= heap.size()) break;
      if (c + 1 < heap.size() && heap[c + 1] < heap[c]) ++c;
      if (!(heap[c] < top)) break;
      heap[i] = heap[c];
      i = c;
    }
    heap[i] = top;
    return top;
  }
};

// Costs of a schedule in microseconds: a piece of n units of item i takes fixed + n * step(i), and `part` more if its
// item is cut; rows(i) of the 256 rows of a part are there.
template <typename Item, typename Step, typename Rows>
struct Costs {
  const std::vector<Item>& items;
  Rates r;
  Step step;
  Rows rows;
  double of(int32_t i, int n, bool cut) const { return r.fixed + n * step(items[i]) + (cut ? r.part : 0.0); }
  // what the parts cost beside the schedule
  double merge(const std::vector<Piece>& pieces) const {
    double bytes = 0.0;
    for (const Piece& p : pieces)
      if (p.cut) bytes += r.part_bytes * rows(items[p.item]) / 256.0;
    return bytes > 0.0 ? r.merge + bytes / kPartBytesPerUs : 0.0;
  }
};

// The given pieces, each in turn to the thread block that is free first (longest first, or in the order given).
// Returns the makespan; sets the pieces' blocks and orders them as scheduled.
template <typename C>
double list_schedule(const C& c, bool longest_first, int sms, std::vector<Piece>* pieces) {
  const size_t n = pieces->size();
  std::vector<std::pair<double, int32_t>> order(n);  // {-cost, index}: longest first, ties in the order given
  for (size_t i = 0; i < n; ++i)
    order[i] = {-c.of((*pieces)[i].item, (*pieces)[i].hi - (*pieces)[i].lo, (*pieces)[i].cut), (int32_t)i};
  if (longest_first && !std::is_sorted(order.begin(), order.end())) std::sort(order.begin(), order.end());
  LeastLoaded blocks(std::max(1, std::min<int>(sms, (int)n)));
  double makespan = 0.0;
  std::vector<Piece> out(n);
  for (size_t i = 0; i < n; ++i) {
    const std::pair<double, int32_t> load = blocks.add(-order[i].first);
    out[i] = (*pieces)[order[i].second];
    out[i].bin = load.second;
    makespan = std::max(makespan, load.first);
  }
  pieces->swap(out);
  return makespan;
}

// Every item in equal pieces of at most `chunk` units (0: whole).
template <typename C>
std::vector<Piece> equal_pieces(const C& c, int chunk) {
  std::vector<Piece> out;
  for (int32_t i = 0; i < (int32_t)c.items.size(); ++i) {
    const int n = c.items[i].n, k = chunk > 0 && n > chunk ? (n + chunk - 1) / chunk : 1;
    for (int j = 0; j < k; ++j) out.push_back({i, (int)((int64_t)n * j / k), (int)((int64_t)n * (j + 1) / k), 0, k > 1});
  }
  return out;
}

// Thread blocks filled one after the other up to a load of `top`, items cut where one is full: an even share of the
// work each for at most one cut a block.  Pieces have at least kLeastPiece units.  False when the bins do not
// suffice.
constexpr int kLeastPiece = 2;
template <typename C>
bool cut_schedule(const C& c, double top, int bins, std::vector<Piece>* out) {
  out->clear();
  int bin = 0;
  double room = top;
  for (int32_t i = 0; i < (int32_t)c.items.size(); ++i) {
    const int n = c.items[i].n;
    const double step = c.step(c.items[i]);
    for (int lo = 0;;) {
      const int rest = n - lo;
      if (c.of(i, rest, lo > 0) <= room) {  // the rest of the item, or all of it
        out->push_back({i, lo, n, bin, lo > 0});
        room -= c.of(i, rest, lo > 0);
        break;
      }
      int fit = (int)std::max(0.0, (room - c.r.fixed - c.r.part) / step);
      if (rest - fit < kLeastPiece) fit = rest - kLeastPiece;
      if (fit >= kLeastPiece) {
        out->push_back({i, lo, lo + fit, bin, true});
        lo += fit;
      } else if (room == top) {
        return false;  // not even an empty block takes a piece
      }
      room = top;
      if (++bin == bins) return false;
    }
  }
  return true;
}

// The pieces and their thread blocks: whole items where they balance; where too few of them do not fill the SMs
// evenly, the best of equal pieces and of cutting at an even load, if it wins more than its parts cost.  `apart`: cuts
// at an even load may be made (they spread the pieces of neighbouring items over time, and with it what those share).
template <typename C>
std::vector<Piece> make_schedule(const C& c, bool longest_first, bool apart, int sms, double* makespan) {
  std::vector<Piece> best = equal_pieces(c, 0);
  *makespan = list_schedule(c, longest_first, sms, &best);
  double total = 0.0, units = 0.0;
  for (size_t i = 0; i < c.items.size(); ++i) {
    total += c.of((int32_t)i, c.items[i].n, false);
    units += c.items[i].n;
  }
  // many items to a thread block balance by themselves
  if (c.items.empty() || c.items.size() > 32u * sms || *makespan < 1.05 * total / sms) return best;
  double price = 0.95 * *makespan;  // the model is good to some 5 %
  auto take = [&](std::vector<Piece>* trial, double span) {
    const double with_merge = span + c.merge(*trial);
    if (with_merge >= price) return;
    price = with_merge;
    *makespan = span;
    best.swap(*trial);
  };
  std::vector<Piece> trial;
  int last = 0;
  for (double f : {1.5, 1.25, 1.0, 0.8, 0.6, 0.45, 0.3, 0.2}) {
    const int chunk = std::max(kLeastPiece, (int)(units / sms * f));
    if (chunk == last) continue;
    last = chunk;
    trial = equal_pieces(c, chunk);
    const double span = list_schedule(c, longest_first, sms, &trial);
    take(&trial, span);
  }
  if (!apart) return best;
  double lo = total / sms, hi = 2.0 * lo + c.r.fixed + c.r.part;
  std::vector<Piece> found;
  for (int k = 0; k < 10 && hi - lo > 0.02 * lo; ++k) {
    const double mid = k == 0 ? hi : 0.5 * (lo + hi);
    if (cut_schedule(c, mid, sms, &trial)) {
      found.swap(trial);
      hi = mid;
    } else if (k == 0) {
      break;
    } else {
      lo = mid;
    }
  }
  if (!found.empty()) take(&found, hi);
  return best;
}

// The pieces by thread block, in the order of the schedule; ptr gets one entry more than there are blocks.
std::vector<Piece> by_block(const std::vector<Piece>& pieces, std::vector<int32_t>* ptr) {
  int32_t bins = 0;
  for (const Piece& p : pieces) bins = std::max(bins, p.bin + 1);
  ptr->assign(bins + 1, 0);
  for (const Piece& p : pieces) ++(*ptr)[p.bin + 1];
  for (int b = 0; b < bins; ++b) (*ptr)[b + 1] += (*ptr)[b];
  std::vector<int32_t> at(ptr->begin(), ptr->end() - 1);
  std::vector<Piece> out(pieces.size());
  for (const Piece& p : pieces) out[at[p.bin]++] = p;
  return out;
}

// Key blocks that the query block sees (its last token's keys), and whether it has tokens at all.
int blocks_seen(const CausalSeq& s, int block, int tb) {
  const int64_t tok = (int64_t)block * tb;
  if (tok >= s.q_len) return 0;
  const int64_t last = std::min<int64_t>(tok + tb, s.q_len);
  const int64_t seen = std::max<int64_t>(0, (int64_t)s.kv_len - s.q_len + last);
  return (int)((seen + 127) / 128);
}

// Gives the parts of a cut item, marked by their first unit in `part`, the item's slots in that order; `item_of` is
// where a tile holds its item's number, cleared here.
template <typename T, typename F>
void number_parts(std::vector<T>* tiles, const std::vector<int32_t>& first_slot, const F& item_of) {
  std::vector<int32_t> cut;
  for (int32_t i = 0; i < (int32_t)tiles->size(); ++i)
    if ((*tiles)[i].part >= 0) cut.push_back(i);
  std::sort(cut.begin(), cut.end(), [&](int32_t a, int32_t b) {
    T &x = (*tiles)[a], &y = (*tiles)[b];
    return item_of(x) != item_of(y) ? item_of(x) < item_of(y) : x.part < y.part;
  });
  for (size_t k = 0, nth = 0; k < cut.size(); ++k) {
    T& x = (*tiles)[cut[k]];
    nth = k > 0 && item_of((*tiles)[cut[k - 1]]) == item_of(x) ? nth + 1 : 0;
    x.part = first_slot[item_of(x)] + (int32_t)nth;
  }
  for (T& x : *tiles) item_of(x) = 0;
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
  const Rates r = fwd_rates(p->head_dim);
  auto step = [&](const FwdItem& u) { return u.two ? r.step2 : r.step1; };
  auto rows = [&](const FwdItem& u) {
    return (u.two ? kCausalRows : 0) + std::min(tb, p->seqs[u.seq].q_len - (u.block + u.two) * tb) * p->group;
  };
  const Costs<FwdItem, decltype(step), decltype(rows)> costs{all, r, step, rows};
  double makespan = 0.0;
  const std::vector<Piece> pieces = make_schedule(costs, resident, true, p->num_sms, &makespan);
  p->fwd_short = makespan < kShortUs;
  // an item's parts take neighbouring slots, in the order of their keys
  std::vector<int32_t> first_slot(all.size(), -1), parts(all.size(), 0);
  for (const Piece& x : pieces)
    if (x.cut) ++parts[x.item];
  for (size_t i = 0; i < all.size(); ++i) {
    if (parts[i] == 0) continue;
    const FwdItem& u = all[i];
    first_slot[i] = p->slots;
    const CausalSeq& s = p->seqs[u.seq];
    p->merges.push_back({(int32_t)s.q_offset, s.q_len, u.head, u.block, p->slots, parts[i], {0, 0}});
    p->slots += parts[i];
    p->merge_rows = std::max(p->merge_rows, rows(u));
  }
  for (const Piece& x : by_block(pieces, &p->fwd_ptr)) {
    const FwdItem& u = all[x.item];
    const CausalSeq& s = p->seqs[u.seq];
    p->fwd_tiles.push_back({(int32_t)s.q_offset, s.q_len, (int32_t)s.kv_offset, s.kv_len, u.head, u.block, x.lo, x.hi,
                            x.cut ? x.lo : -1, u.seq, {x.item, 0}});
  }
  number_parts(&p->fwd_tiles, first_slot, [](CausalTile& t) -> int32_t& { return t.pad[0]; });
}

struct BwdItem {
  int32_t seq, head, block, first, n, nqb;
};

void build_backward(zl_causal_plan* p, const std::vector<int32_t>& by_len, bool resident, bool in_l2) {
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
  const Rates r = bwd_rates(p->head_dim);
  auto step = [&](const BwdItem&) { return r.step1; };
  auto rows = [](const BwdItem&) { return 256; };  // dK and dV of 128 keys
  const Costs<BwdItem, decltype(step), decltype(rows)> costs{all, r, step, rows};
  double makespan = 0.0;
  const std::vector<Piece> pieces = make_schedule(costs, resident, in_l2, p->num_sms, &makespan);
  p->bwd_short = makespan < kShortUs;
  std::vector<int32_t> first_slot(all.size(), -1), parts(all.size(), 0);
  for (const Piece& x : pieces)
    if (x.cut) ++parts[x.item];
  for (size_t i = 0; i < all.size(); ++i) {
    if (parts[i] == 0) continue;
    const BwdItem& u = all[i];
    const CausalSeq& s = p->seqs[u.seq];
    first_slot[i] = p->bwd_slots;
    p->bwd_merges.push_back({(int32_t)s.kv_offset, s.kv_len, u.head, u.block, p->bwd_slots, parts[i], {0, 0}});
    p->bwd_slots += parts[i];
  }
  for (const Piece& x : by_block(pieces, &p->bwd_ptr)) {
    const BwdItem& u = all[x.item];
    const CausalSeq& s = p->seqs[u.seq];
    p->bwd_tiles.push_back({(int32_t)s.q_offset, s.q_len, (int32_t)s.kv_offset, s.kv_len, u.head, u.block,
                            (int32_t)(s.acc_block + (int64_t)u.head * u.nqb), u.first + x.lo, x.hi - x.lo,
                            x.cut ? x.lo : -1, u.seq, x.item});
  }
  number_parts(&p->bwd_tiles, first_slot, [](CausalBwdTile& t) -> int32_t& { return t.pad; });
}

template <typename T>
void put(std::vector<char>* blob, size_t at, const std::vector<T>& v) {
  if (!v.empty()) std::memcpy(blob->data() + at, v.data(), v.size() * sizeof(T));
}

// Tables that no plan and no graph owns any more.  The last owner may be a graph, whose end is told on a thread that must
// not call CUDA, so they are freed by the next plan that is made or destroyed.
std::mutex dead_lock;
CausalTables* dead = nullptr;

void disown(void* tables) {
  CausalTables* t = static_cast<CausalTables*>(tables);
  if (t->owners.fetch_sub(1, std::memory_order_acq_rel) != 1) return;
  std::lock_guard<std::mutex> lock(dead_lock);
  t->next = dead;
  dead = t;
}

void free_dead() {
  CausalTables* list;
  {
    std::lock_guard<std::mutex> lock(dead_lock);
    list = dead;
    dead = nullptr;
  }
  if (!list) return;
  // a plan may go while this thread captures a stream, which a plain cudaFree would spoil
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  const bool relaxed = cudaThreadExchangeStreamCaptureMode(&mode) == cudaSuccess;
  int dev = -1;
  const bool known = cudaGetDevice(&dev) == cudaSuccess;
  while (list) {
    CausalTables* t = list;
    list = t->next;
    if (known && t->device != dev) cudaSetDevice(t->device);
    if (t->ptr) cudaFree(t->ptr);
    if (known && t->device != dev) cudaSetDevice(dev);
    delete t;
  }
  if (relaxed) cudaThreadExchangeStreamCaptureMode(&mode);
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
  p->tables = new CausalTables;
  p->tables->device = p->device;
  if (cudaMalloc(&p->tables->ptr, at) != cudaSuccess) {
    p->tables->ptr = nullptr;
    cudaGetLastError();
    return ZL_ERR_NO_MEMORY;
  }
  // the copy from pageable memory may still be on its way when the call returns; launches on other streams
  // do not wait for it, so it is awaited here
  if (cudaMemcpy(p->tables->ptr, blob.data(), at, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaStreamSynchronize(nullptr) != cudaSuccess)
    return ZL_ERR_CUDA;
  char* base = static_cast<char*>(p->tables->ptr);
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
  const double shared = p->acc_blocks * 128 * 8.0 * p->head_dim;
  if (!p->forward_only) build_backward(p, by_len, few || shared <= kL2Bytes, shared <= kCutBytes);
  const int64_t D = p->head_dim;
  p->fwd_bytes = (int64_t)p->slots * 256 * (D + 1) * 4;
  if (!p->forward_only)
    p->bwd_bytes = (int64_t)align_up256((size_t)(p->q_tokens * p->n_q_heads * 4)) + p->acc_blocks * 128 * D * 4 +
                 (int64_t)p->bwd_slots * 2 * 128 * D * 4;
  return p->host_only ? ZL_OK : upload_causal(p);
}

}  // namespace

zl_status zl::hold_tables(const zl_causal_plan* p, cudaStream_t stream) {
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  cudaGraph_t graph = nullptr;
  if (cudaStreamGetCaptureInfo(stream, &status, nullptr, &graph) != cudaSuccess) return ZL_ERR_CUDA;
  if (status != cudaStreamCaptureStatusActive) return ZL_OK;
  cudaUserObject_t object;
  p->tables->owners.fetch_add(1, std::memory_order_relaxed);
  if (cudaUserObjectCreate(&object, p->tables, disown, 1, cudaUserObjectNoDestructorSync) != cudaSuccess) {
    disown(p->tables);
    return ZL_ERR_CUDA;
  }
  if (cudaGraphRetainUserObject(graph, object, 1, cudaGraphUserObjectMove) != cudaSuccess) {
    cudaUserObjectRelease(object, 1);
    return ZL_ERR_CUDA;
  }
  return ZL_OK;
}

extern "C" zl_status zl_plan_causal(const zl_causal_seq* seqs, int32_t n_seqs, int32_t n_q_heads, int32_t n_kv_heads,
                                    int32_t head_dim, int64_t q_tokens, int64_t kv_tokens, uint32_t flags,
                                    zl_causal_plan** out) {
  NvtxRange range("zl_plan_causal");
  if (!out) return ZL_ERR_INVALID_ARG;
  *out = nullptr;
  if (n_seqs < 0 || (n_seqs > 0 && !seqs) || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || q_tokens < 0 ||
      kv_tokens < 0 || (flags & ~(ZL_PLAN_HOST_ONLY | ZL_PLAN_TEST_WITHHOLD_LOAD | ZL_PLAN_FORWARD_ONLY)))
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
  p->forward_only = flags & ZL_PLAN_FORWARD_ONLY;
  p->num_sms = 152;
  free_dead();
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
  if (p->tables) disown(p->tables);
  free_dead();
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
