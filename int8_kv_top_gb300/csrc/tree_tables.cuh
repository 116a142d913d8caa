// The tables of a drafted-token call and of a shared call (qsa_prefix_attention): which entries keep the contract, whose a
// token is, which cells it sees, and where its rows lie in the launches' grids and workspaces.  Integers alone: with
// CUDA's few names given the file compiles without it.
#pragma once
#include "tree_plan.cuh"

namespace qsa {

struct TreeBatch {
  const int4* seqs;  // per sequence {first pool cell, n_cells, pos0, first token row}
  long long n_pool;
  int n_seq, n_tok;
  const uint32_t* tree;  // [n_tok][tree_words]; of a shared call null as well: causal
  int tree_words, max_n_kv, identity_max;
  // shared calls (qsa_prefix_attention) alone; max_n_kv then counts the prefix's cells too
  const int4* prefixes = nullptr;  // per prefix {first pool cell, cells, first sequence, -}
  int n_prefix = 0, max_prefix = 0;
  int4* tok = nullptr;             // per token {sequence or -1, n_kv, prefix cells, prefix}: made by the call's first launch
};

// What a kernel that serves both kinds of calls works on: a tree call's sequences; the prefixes of a shared call, each
// a sequence of committed cells whose tokens are those of all its sequences; the own cells of a shared call's sequences.
enum CellsOf { kTreeCells, kPrefixCells, kOwnCells };

// Sequence s's token count, or -1 when its entry breaks the contract; a padding sequence (no cells) has none.
__device__ __forceinline__ int tree_seq_tokens(const TreeBatch& b, int s, int4* e_out) {
  const int4 e = __ldg(&b.seqs[s]);
  const int next = s + 1 < b.n_seq ? __ldg(&b.seqs[s + 1].w) : b.n_tok;
  *e_out = e;
  const bool rows_ok = (s == 0 ? e.w == 0 : e.w >= 0) && next >= e.w && next <= b.n_tok;
  if (rows_ok && e.y == 0) return 0;
  const long long T = (long long)next - e.w, end = (long long)e.z + T;
  const bool ok = rows_ok && e.x >= 0 && e.y >= 1 && e.z >= 0 && end <= e.y && (long long)e.x + e.y <= b.n_pool &&
                  end <= b.max_n_kv && T <= 32 * b.tree_words;
  return ok ? (int)T : -1;
}

// Word w of token row's mask, with the bits past the sequence's T drafted tokens cleared.
__device__ __forceinline__ uint32_t tree_mask_word(const TreeBatch& b, int row, int w, int T) {
  const int left = T - 32 * w;
  if (w >= b.tree_words || left <= 0) return 0u;
  const uint32_t m = __ldg(b.tree + (size_t)row * b.tree_words + w);
  return left >= 32 ? m : m & ((1u << left) - 1u);
}

// ---------------------------------------------------------------- shared calls
// Prefix p: its tokens (rows of all its sequences), or -1 when its entry breaks the contract; *e_out = {first pool cell,
// cells, first sequence, first token row}.
__device__ __forceinline__ int prefix_tokens(const TreeBatch& b, int p, int4* e_out) {
  int4 e = __ldg(&b.prefixes[p]);
  const int next = p + 1 < b.n_prefix ? __ldg(&b.prefixes[p + 1].z) : b.n_seq;
  const bool seqs_ok = (p == 0 ? e.z == 0 : e.z >= 0) && next >= e.z && next <= b.n_seq;
  const int row0 = seqs_ok && e.z < b.n_seq ? __ldg(&b.seqs[e.z].w) : b.n_tok;
  const int row1 = seqs_ok && next < b.n_seq ? __ldg(&b.seqs[next].w) : b.n_tok;
  e.w = row0;
  *e_out = e;
  const bool ok = seqs_ok && row0 >= 0 && row1 >= row0 && row1 <= b.n_tok && e.x >= 0 && e.y >= 0 && e.y <= b.max_prefix &&
                  (long long)e.x + e.y <= b.n_pool;
  return ok ? row1 - row0 : -1;
}

// The last of n whose key is not above `at` (the first where all are).
template <class Key>
__device__ __forceinline__ int last_at(int n, int at, Key key) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (key(mid) <= at) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// The prefix of sequence s (the last whose first sequence is not behind s); -1 without prefixes.
__device__ __forceinline__ int prefix_of(const TreeBatch& b, int s) {
  return b.n_prefix == 0 ? -1 : last_at(b.n_prefix, s, [&](int i) { return __ldg(&b.prefixes[i].z); });
}

// A shared call's sequence, behind prefix p (-1: none): its entry, tokens as in tree_seq_tokens, and the prefix's tokens
// and {first pool cell, cells, first sequence, first token row}.
struct SharedSeq {
  int4 e, pe;
  int T, pT;
};
__device__ __forceinline__ SharedSeq shared_seq(const TreeBatch& b, int s, int p) {
  SharedSeq x;
  x.e = __ldg(&b.seqs[s]);
  const int next = s + 1 < b.n_seq ? __ldg(&b.seqs[s + 1].w) : b.n_tok;
  x.pe = make_int4(0, 0, 0, 0);
  x.pT = p < 0 ? 0 : prefix_tokens(b, p, &x.pe);
  const bool rows_ok = (s == 0 ? x.e.w == 0 : x.e.w >= 0) && next >= x.e.w && next <= b.n_tok;
  const long long T = (long long)next - x.e.w, end = (long long)x.e.z + T;
  const bool ok = x.pT >= 0 && rows_ok && x.e.x >= 0 && x.e.y >= 1 && x.e.z >= 0 && end <= x.e.y &&
                  (long long)x.e.x + x.e.y <= b.n_pool && x.pe.y + end <= b.max_n_kv && T <= 32 * (b.tree ? b.tree_words : kTreeWords);
  x.T = rows_ok && x.e.y == 0 ? 0 : ok ? (int)T : -1;
  return x;
}
__device__ __forceinline__ int shared_seq_tokens(const TreeBatch& b, int s, int4* e_out) {
  const SharedSeq x = shared_seq(b, s, prefix_of(b, s));
  *e_out = x.e;
  return x.T;
}

// Word w of the mask of token i (row `row`) of a shared call's sequence of T tokens.
__device__ __forceinline__ uint32_t shared_mask_word(const TreeBatch& b, int row, int i, int w, int T) {
  if (b.tree != nullptr) return tree_mask_word(b, row, w, T);
  const int n = i + 1 - 32 * w;  // causal
  return n >= 32 ? 0xffffffffu : n > 0 ? (1u << n) - 1u : 0u;
}

// Columns of a shared call's rows of scores and selected cells: the prefix's cells, a gap up to a whole tile, which holds anything
// (its cells, counted on from either side, may be outside the pool) and is never read as a score, the own cells.
__device__ __forceinline__ int own_column(int prefix_cells) { return (prefix_cells + 127) & ~127; }

// What the later launches need of a token besides its record (TreeBatch::tok): its sequence's {first pool cell, committed own
// cells, tokens, first token row}.
struct TokMore {
  int4 seq;
};

// Token t's record (TreeBatch::tok), of sequence s behind prefix p; `more` is written where it is a valid sequence's.  Where
// rows or first sequences run backwards, a sequence's rows may lie outside its prefix's, where the prefix's parts have none for it.
__device__ __forceinline__ int4 shared_record(const TreeBatch& b, int t, int s, int p, TokMore* more) {
  const SharedSeq v = shared_seq(b, s, p);
  if (v.T <= 0 || t < v.e.w || t >= v.e.w + v.T || (p >= 0 && (t < v.pe.w || t >= v.pe.w + v.pT))) return make_int4(-1, 0, 0, -1);
  int seen = v.pe.y + v.e.z;
  for (int i = 0; 32 * i < v.T; ++i) seen += __popc(shared_mask_word(b, t, t - v.e.w, i, v.T));
  *more = TokMore{make_int4(v.e.x, v.e.z, v.T, v.e.w)};
  return make_int4(s, seen, v.pe.y, p);
}

// Token row's record, as a launch over the cells of prefix or sequence i (kOwnCells) takes it: none where the token is
// another's.  First rows that run backwards give a row to several sequences, of which its record names one, and the others'
// cells and columns are not those that its rows of scores and selected cells are made for.
__device__ __forceinline__ int4 record_in(const TreeBatch& b, CellsOf of, int i, int row) {
  const int4 ti = __ldcg(&b.tok[row]);
  return (of == kPrefixCells ? ti.w : ti.x) == i ? ti : make_int4(-1, 0, 0, -1);
}

// The column of a row of scores at which the cells of a prefix, or a sequence's own ones behind prefix_cells, begin.
__device__ __forceinline__ int score_column(CellsOf of, int prefix_cells) { return of == kPrefixCells ? 0 : own_column(prefix_cells); }

// ---------------------------------------------------------------- blocks of an attention launch
constexpr int kTileCells = 128;    // cells of a tile
constexpr int kTreeBlock = 256;    // (token, head) rows of a block: a CTA pair's UMMA M
constexpr int kTokChunk = 32;      // tokens of a score CTA: UMMA N is at most twice that

// Rows of a block that exist are shared out evenly: its CTA `half` of each pair has rows [x, x + n) of the tree, so
// that the loads of Q and the stores of O, 1 KB a row, are halved where a block is not full.
__device__ __forceinline__ int cta_rows(int T, int blk_row0, int half, int* x) {
  const int n = min(kTreeBlock, T * kHPG - blk_row0), first = (n + 1) / 2;
  *x = blk_row0 + half * first;
  return half ? n - first : first;
}

// The clusters of a shared call's only prefix, of T tokens and `cells` cells, as plan_prefixes (prefix.cu) shares them out:
// {first, runs a block and group, first token row, tokens}.
__device__ __forceinline__ int4 only_prefix_plan(int row0, int T, int cells, int clusters) {
  const int tiles = (cells + kTileCells - 1) / kTileCells, blocks = (T * kHPG + kTreeBlock - 1) / kTreeBlock * kGroups;
  if (T <= 0 || tiles == 0) return make_int4(0, 0, row0, max(T, 0));
  const int most = max(1, min(min(clusters / blocks, kMaxRuns), tiles)), L = (tiles + most - 1) / most;
  return make_int4(0, (tiles + L - 1) / L, row0, T);
}

// Runs of a block and group of a shared call over n_tiles tiles: as many of run_tiles as it takes, `runs` at most.
__device__ __forceinline__ int shared_runs(int n_tiles, int runs, int run_tiles) {
  return max(1, min(runs, (n_tiles + run_tiles - 1) / run_tiles));
}

// Index of a sequence's first block in the grid: block k of sequence s has index first_block(s) + k.
// The sequences' ranges never meet, since floor((a + b) / 256) + 1 >= floor(a / 256) + ceil(b / 256), so
// a block finds its sequence by a search over the table, without a prefix sum; some indices stay unused.
__device__ __forceinline__ long long first_block(long long first_row, int s) { return first_row * kHPG / kTreeBlock + s; }

// First token chunk of a sequence: as first_block, for chunks of 32 tokens.
__device__ __forceinline__ long long first_chunk(long long first_row, int s) { return first_row / kTokChunk + s; }

// Where row R of T tokens' (12 a token) lies among the parts: CTA of run 0, and row of that CTA.  first: their first pair.
__device__ __forceinline__ void part_row(long long first, int T, int g, int runs, int R, size_t* cta, int* row) {
  const int k = R / kTreeBlock, r = R % kTreeBlock;
  const int n = min(kTreeBlock, T * kHPG - k * kTreeBlock), half_rows = (n + 1) / 2;
  const int half = r >= half_rows;
  *cta = ((size_t)first + (size_t)(k * kGroups + g) * runs) * 2 + half;
  *row = half ? r - half_rows : r;
}

}  // namespace qsa
