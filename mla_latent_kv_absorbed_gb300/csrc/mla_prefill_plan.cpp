// Host plan of the expanded attention: which query rows and keys one work item
// of the kernel takes, and in what order items are launched.
//
//   * an item is up to 256 query rows of one request (two tiles of 128) and
//     the keys they see, for every head, or 512 for a pair of CTAs: whichever
//     of the two schedules ends first; causal items end at the last key of
//     their last row, so no tile without a visible key is visited;
//   * items are launched heaviest first (blocks start in launch order as SMs
//     fall free, so the short ones fill the end), for a group of heads at a
//     time: the group's keys and values stay in L2 while all its rows pass.
//     The shortest items of all groups are kept for the very end, where that
//     evens out the SMs (12 ragged requests x 32 heads: SMs ended between 105
//     and 135 us without);
//   * where whole items would leave SMs idle (few rows over long keys), an
//     item's keys are cut into pieces of whole tiles whose partial outputs a
//     second kernel joins.  Tried are the cuts that fill the SMs once, twice,
//     ... with pieces of about equal cost; taken is the one whose greedy
//     schedule ends first, if it ends before the uncut one.
// The plan is deterministic: equal inputs give identical words.
#include <algorithm>
#include <cstdint>
#include <functional>
#include <queue>
#include <vector>

#include "mla_prompt.h"

namespace mla {
namespace {

struct Tile {
  int b, q0, nq, k0, nk, off;
};
struct Piece {
  int tile, t0, n;           // key tiles [t0, t0 + n) of the tile
  long long cost;
};

// Costs in twentieths of a key tile against two row tiles of one CTA (a unit is
// about 180 cycles): a partial output written and read again, the joining
// kernel's launch.  They were fitted to causal and ragged batches while two
// threads shared a row of scores; beside each stands what the kernel takes with
// four.  Both sides of the choice between the forms are measured in
// mla_prefill.cu: at each size there the plan takes the faster one.
constexpr long long kPieceCost = 8;
constexpr long long kJoinCost = 24;
constexpr long long kL2Bytes = 64ll << 20;
constexpr int kMostTiles = 1 << 17;   // of an item: a quarter of a second, well under the limit of a wait for its last
constexpr int kMostSms = 4096;        // planned for: more than any device has

inline int key_tiles(int nk) { return (nk + kPfKeys - 1) / kPfKeys; }
// A key tile: 3540 cycles against two row tiles (about 4000 without a causal
// limit); one has no other to fill its softmax's time (2740).  A pair's two tiles
// of 256 rows take 3070, on two SMs.
inline long long tile_cost(int nq, int rows) {
  if (rows == kPfRows) return nq > rows / 2 ? 20 : 17;
  return nq > rows / 2 ? 17 : 16;
}
// An item's first loads and scores and its epilogue, as far as nothing fills
// them: 7800 cycles, a pair's 11400.
inline long long item_cost(int rows) { return rows == kPfRows ? 40 : 54; }

// Parts of a tile whose keys are cut into pieces of at most `cap` (0: as few as can be), none under four key tiles.
int parts_of(const Tile& t, int rows, long long cap) {
  const int nt = key_tiles(t.nk);
  if (nt <= 1) return 1;
  const long long most = cap <= 0 ? kMostTiles : std::min<long long>(kMostTiles, std::max<long long>(4, cap / tile_cost(t.nq, rows)));
  return static_cast<int>((nt + most - 1) / most);
}

long long count_pieces(const std::vector<Tile>& tiles, int rows, long long cap) {
  long long n = 0;
  for (const Tile& t : tiles) n += parts_of(t, rows, cap);
  return n;
}

void cut(const std::vector<Tile>& tiles, int rows, long long cap, std::vector<Piece>& pieces) {
  pieces.clear();
  for (size_t i = 0; i < tiles.size(); ++i) {
    const int nt = key_tiles(tiles[i].nk);
    const long long c = tile_cost(tiles[i].nq, rows);
    const int parts = parts_of(tiles[i], rows, cap);
    for (int k = 0; k < parts; ++k) {
      const int a = static_cast<int>(static_cast<long long>(nt) * k / parts);
      const int e = static_cast<int>(static_cast<long long>(nt) * (k + 1) / parts);
      pieces.push_back({static_cast<int>(i), a, e - a, c * (e - a) + item_cost(rows) + (parts > 1 ? kPieceCost : 0)});
    }
  }
  std::stable_sort(pieces.begin(), pieces.end(), [](const Piece& x, const Piece& y) { return x.cost > y.cost; });
}

// Heads whose items are launched together: their keys and values should stay
// in L2 while the rows pass; the groups are of about equal size, so that the
// last one has enough items to even out the SMs.
int group_of(int heads, long long kv_tokens, size_t pieces, int sms) {
  const long long per_head = std::max<long long>(1, kv_tokens * 2 * kNope * 2);
  long long group = std::max<long long>(kL2Bytes / per_head, pieces ? (2ll * sms + pieces - 1) / pieces : 1);
  group = std::min<long long>(heads, std::max<long long>(1, group));
  const long long groups = (heads + group - 1) / group;
  return static_cast<int>((heads + groups - 1) / groups);
}

// End of the greedy schedule of the pieces in launch order on `sms`, the last `tail` of them behind all heads' others.
long long makespan(const std::vector<Piece>& pieces, int heads, int group, int sms, size_t tail = 0) {
  std::priority_queue<long long, std::vector<long long>, std::greater<long long>> free_at;
  for (int i = 0; i < sms; ++i) free_at.push(0);
  long long end = 0;
  auto take = [&](long long cost) {
    const long long t = free_at.top() + cost;
    free_at.pop();
    free_at.push(t);
    end = std::max(end, t);
  };
  for (int h0 = 0; h0 < heads; h0 += group)
    for (size_t i = 0; i + tail < pieces.size(); ++i)
      for (int h = h0; h < std::min(heads, h0 + group); ++h) take(pieces[i].cost);
  for (size_t i = pieces.size() - tail; i < pieces.size(); ++i)
    for (int h = 0; h < heads; ++h) take(pieces[i].cost);
  return end;
}

// How many of the pieces to keep for the end: up to a quarter of the work (they find less of their keys in L2).
size_t tail_of(const std::vector<Piece>& pieces, int heads, int group, int sms) {
  if (group >= heads || pieces.size() < 2 || static_cast<long long>(pieces.size()) * heads > (1 << 16)) return 0;
  long long total = 0;
  for (const Piece& p : pieces) total += p.cost;
  long long end = makespan(pieces, heads, group, sms), sum = 0;
  size_t best = 0, n = 0;
  for (int part = 1; part <= 4; ++part) {               // a sixteenth of the work, an eighth, ...
    while (n + 1 < pieces.size() && 16 * (sum + pieces[pieces.size() - 1 - n].cost) <= total * part)
      sum += pieces[pieces.size() - 1 - n++].cost;
    const long long e = makespan(pieces, heads, group, sms, n);
    if (e < end) {
      end = e;
      best = n;
    }
  }
  return best;
}

// The tiles of `rows` query rows and their pieces in launch order; returns the
// end of the greedy schedule.
long long plan_rows(const int32_t* qp, const int32_t* kp, int B, int H, int causal, int rows, int workers,
                    std::vector<Tile>& tiles, std::vector<Piece>& best) {
  tiles.clear();
  for (int b = 0; b < B; ++b) {
    const int lq = qp[b + 1] - qp[b], lk = kp[b + 1] - kp[b];
    for (int r = 0; r < lq; r += rows) {
      const int nq = std::min(rows, lq - r);
      // row r + i sees keys j <= r + i + lk - lq
      const long long off = causal ? static_cast<long long>(r) + lk - lq : kPfNoLimit;
      const long long seen = std::min<long long>(lk, std::max<long long>(0, off + nq));
      tiles.push_back({b, qp[b] + r, nq, kp[b], static_cast<int>(seen), static_cast<int>(off)});
    }
  }
  cut(tiles, rows, 0, best);
  long long total = 0, most = 0;
  for (const Piece& p : best) {
    total += p.cost * H;
    most = std::max(most, p.cost);
  }
  const long long mean = (total + workers - 1) / workers;
  const long long whole = static_cast<long long>(tiles.size()) * H;
  if (tiles.empty()) return 0;
  if (whole > (1 << 16)) return mean + most;                  // too many to simulate (a long one among them stays whole)
  long long end = makespan(best, H, group_of(H, kp[B], best.size(), workers), workers);
  // the schedule of many items, none of them long, cannot be improved by cutting
  if (whole >= 8ll * workers && most <= mean / 2) return end;
  std::vector<Piece> trial;
  long long waves = whole / workers + 1;
  for (int tried = 0; tried < 5; ++tried, ++waves) {
    const long long pieces = waves * workers / H;             // that fill the SMs `waves` times
    if (pieces <= static_cast<long long>(tiles.size()) || pieces > 65535) continue;
    long long lo = 1, hi = most;                              // the smallest cap with no more pieces than that
    while (lo < hi) {
      const long long mid = (lo + hi) / 2;
      if (count_pieces(tiles, rows, mid) <= pieces) hi = mid;
      else lo = mid + 1;
    }
    cut(tiles, rows, lo, trial);
    if (trial.size() == tiles.size()) continue;
    const long long e = makespan(trial, H, group_of(H, kp[B], trial.size(), workers), workers) + kJoinCost;
    if (e < end) {
      end = e;
      best.swap(trial);
    }
  }
  return end;
}

}  // namespace

int build_prefill_plan(const int32_t* qp, const int32_t* kp, int B, int H, int causal, int num_sms,
                       std::vector<int32_t>& words) {
  std::vector<Tile> tiles;
  std::vector<Piece> best;
  const int sms = std::min(num_sms, kMostSms);
  int rows = kPfRows, workers = sms;
  const long long end = plan_rows(qp, kp, B, H, causal, rows, workers, tiles, best);
  if (sms >= 2) {
    std::vector<Tile> pair_tiles;
    std::vector<Piece> pair_best;
    if (plan_rows(qp, kp, B, H, causal, 2 * kPfRows, sms / 2, pair_tiles, pair_best) < end) {
      tiles.swap(pair_tiles);
      best.swap(pair_best);
      rows = 2 * kPfRows;
      workers = sms / 2;
    }
  }
  // partial slots, in tile order, and the merge entries
  std::vector<int> parts(tiles.size(), 0), first(tiles.size(), 0), next(tiles.size(), 0);
  for (const Piece& p : best) ++parts[p.tile];
  int partials = 0, merges = 0;
  for (size_t i = 0; i < tiles.size(); ++i)
    if (parts[i] > 1) {
      first[i] = partials;
      partials += parts[i];
      ++merges;
    }
  const long long n_words = kPfHeaderWords + static_cast<long long>(kPfItemWords) * best.size() +
                            static_cast<long long>(kPfMergeWords) * merges;
  const long long blocks = static_cast<long long>(best.size()) * H;
  if (n_words > 0x7FFFFFFFll || blocks > kPfMaxBlocks || merges > 65535) return MLA_ERR_UNSUPPORTED;
  const int group = group_of(H, kp[B], best.size(), workers);
  words.assign(static_cast<size_t>(n_words), 0);
  words[kPMagic] = kPfMagic;
  words[kPVersion] = kPfVersion;
  words[kPBatch] = B;
  words[kPHeads] = H;
  words[kPCausal] = causal ? 1 : 0;
  words[kPQTokens] = qp[B];
  words[kPKvTokens] = kp[B];
  words[kPItems] = static_cast<int32_t>(best.size());
  words[kPPartials] = partials;
  words[kPMerges] = merges;
  words[kPHeadGroup] = group;
  words[kPTotalWords] = static_cast<int32_t>(n_words);
  words[kPNumSms] = num_sms;
  words[kPTail] = static_cast<int32_t>(tail_of(best, H, group, workers));
  words[kPRows] = rows;
  words[kPSolo] = std::all_of(tiles.begin(), tiles.end(), [](const Tile& t) { return t.nq <= kPfRows / 2; }) ? 1 : 0;
  int32_t* w = words.data() + kPfHeaderWords;
  for (const Piece& p : best) {
    const Tile& t = tiles[p.tile];
    const int k = p.t0 * kPfKeys;
    const int nk = std::min(t.nk - k, p.n * kPfKeys);
    w[0] = t.b;
    w[1] = t.q0;
    w[2] = t.nq;
    w[3] = t.k0 + k;
    w[4] = nk;
    w[5] = causal ? t.off - k : kPfNoLimit;
    w[6] = parts[p.tile] > 1 ? first[p.tile] + next[p.tile]++ : -1;
    w += kPfItemWords;
  }
  for (size_t i = 0; i < tiles.size(); ++i)
    if (parts[i] > 1) {
      w[0] = tiles[i].q0;
      w[1] = tiles[i].nq;
      w[2] = first[i];
      w[3] = first[i] + parts[i];
      w += kPfMergeWords;
    }
  return MLA_OK;
}

}  // namespace mla
