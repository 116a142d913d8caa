// How a qsa_tree_attention call is cut over the GPU: host arithmetic alone (the file compiles without CUDA).
#pragma once
#include <algorithm>
#include <cmath>

namespace qsa {

// Rows of a block, cells of a tile, heads a group, groups, and drafted tokens a sequence at most.
constexpr int kPlanRows = 256, kPlanCells = 128, kPlanHeads = 12, kPlanGroups = 2, kPlanDrafted = 256;

// Blocks of a call at most (their places in the grid: each sequence rounds up by itself).
#ifdef __CUDACC__
__host__ __device__
#endif
inline int tree_blocks_most(int n_seq, int n_tok) { return (int)((long long)n_tok * kPlanHeads / kPlanRows) + n_seq; }

// How a call is cut: blocks (grid indices; a ragged batch leaves about half a block a sequence unused), and for each
// block and group either one cluster of `pairs` pairs that merge in it, or `runs` clusters of one pair whose parts
// tree_join_kernel joins.  A launch takes about waves x (a fixed part + the tiles of a pair), in units of one tile's
// time (1.7 us; fixed: 8 us for one pair, 10 to 12 with a merge in the cluster), and the join its own time by the
// blocks and their parts.  A wave is as many clusters of that size as the GPU holds at once (a cluster stays inside a
// GPC).  How many tokens and cells a sequence has is on the device, so waves is the mean of what equal and spread
// sequences give, each with equal and with spread lengths: the blocks of equal sequences rounded up, or half a block
// of rounding a sequence; whole waves, or 0.9 of a wave for every filling of the GPU.  Measured on a GB300 (us a call):
//                                         pairs 1   2   3   5   6   8     runs 2   4   6   9  12  19  38
//    1 tree  of 61 after  1,984 cells          38  29  25  20  18  16       29  23  22  20  21  32  43
//    1 tree  of 16 after  8,192               158  99  78  61  56  53       98  68  58  52  48  45  44
//    1 tree  of 16 after 30,000               494 272 200 141 126 107      272 162 125 100  88  77  69
//    2 trees of 61 after 30,000               542 320 239 173 249 209      323 204 167 199 175 190 238
//    4 trees of 44 after 30,000               607 364 433 323 387 387      373 373 302 310 318 345 415
//    8 trees of 16 after 30,000               637 368 271 317 285 315      373 236 284 232 253 255 311
//   12 trees of 61 after  8,192               285 309 378 386 474 471      339 370 399 431 461 546 784
//   32 trees of 4-64 after 64-1,984            68 121 150 201 303 314      156 205 247 296 341 438 653
//   24 trees of 1-32 after 200-16,000         353 245 259 295 368 360      258 277 297 323 350 415 579
//    4 trees of 33-48 after 30,000, all cells 448 223 153 189 239 190      238 237 173 181 189 185 258
// (the last takes 157 in the seven runs that the estimate picks, which counts a part-filled wave as less than a whole one)
//
// Several pairs to a block write unmerged parts, 264 KB a pair.  What a call may write is bounded by its arguments
// alone, in a way that grows with each of them (parts_most), so that a workspace for a server's largest batch serves
// every smaller one: the plans above stay inside it but for a few that gain under 5%.
struct DensePlan {
  int blocks, pairs, runs;
};
constexpr double kJoinBlock = 0.2, kJoinPart = 0.02;  // tree_join_kernel's time a block and group, and a part of it
constexpr int kPlanSizesN = 7, kPlanSizes[kPlanSizesN] = {1, 2, 3, 4, 5, 6, 8};  // pairs of a cluster
constexpr int kMaxRuns = 38;  // clusters of one pair that a block and group may share: half of a GB300's

// Clusters of each of those sizes that the GPU holds at once; 0: it takes none.
struct PlanHeld {
  int n[kPlanSizesN];
};

inline int plan_tiles(long long cells) { return (int)((cells + kPlanCells - 1) / kPlanCells); }

// Pairs that may write parts in a call.
constexpr int kFewPairs = 480, kMostPairs = 1600;
inline long long parts_most(int n_seq, int n_tok, int max_n_kv) {
  const long long blocks = tree_blocks_most(n_seq, n_tok);
  const int tiles = plan_tiles(max_n_kv);
  if (tiles < 2) return 0;
  return std::min(blocks * kPlanGroups * std::min(kMaxRuns, tiles + 1),
                  std::min<long long>(kMostPairs, std::max<long long>(kFewPairs, 4 * blocks)));
}

inline DensePlan dense_plan(const PlanHeld& held, int n_seq, int n_tok, int max_n_kv, int identity_max, bool with_selected) {
  DensePlan d{tree_blocks_most(n_seq, n_tok), 1, 1};
  const long long rows = (long long)n_tok * kPlanHeads;
  const long long even = n_seq * ((rows + (long long)n_seq * kPlanRows - 1) / ((long long)n_seq * kPlanRows));
  const long long spread =
      n_seq == 1 ? even : std::max<long long>(n_seq, (rows + kPlanRows / 2 * (long long)n_seq + kPlanRows - 1) / kPlanRows);
  const long long longest = with_selected ? max_n_kv : std::min<long long>(max_n_kv, (long long)identity_max + kPlanDrafted);
  const int tiles = plan_tiles(longest);
  const long long most = parts_most(n_seq, n_tok, max_n_kv);
  auto fits = [&](int split) { return split == 1 || (long long)d.blocks * kPlanGroups * split <= most; };
  auto waves = [&](double a_cluster, int fit) {  // of `a_cluster` clusters a block and group
    const double we = (double)(even * kPlanGroups) * a_cluster / fit, ws = (double)(spread * kPlanGroups) * a_cluster / fit;
    if (n_seq == 1) return std::ceil(we);
    return 0.25 * (std::ceil(we) + std::max(1.0, 0.9 * we) + std::ceil(ws) + std::max(1.0, 0.9 * ws));
  };
  double best_t = 0.0;
  for (int i = 0; i < kPlanSizesN; ++i) {
    const int S = kPlanSizes[i];
    if (!fits(S)) break;
    if (held.n[i] <= 0) continue;
    const double t = waves(1.0, held.n[i]) * ((S == 1 ? 5.0 : 6.0 + 0.1 * S) + (tiles + S - 1) / S);
    if (i == 0 || t < best_t) {
      d.pairs = S;
      best_t = t;
    }
  }
  const double clusters = 0.5 * (double)((even + spread) * kPlanGroups);
  for (int runs = 2; runs <= std::min(kMaxRuns, tiles) && runs * clusters <= 4 * held.n[0] && fits(runs); ++runs) {
    const double t = waves(runs, held.n[0]) * (5.0 + (tiles + runs - 1) / runs) + 2.5 + (kJoinBlock + kJoinPart * runs) * clusters;
    if (t < best_t) {
      d.pairs = 1;
      d.runs = runs;
      best_t = t;
    }
  }
  return d;
}

}  // namespace qsa
