// qsa_tree_attention on the tcgen05 tensor cores, straight from the int8 cache: attention of drafted token
// trees over every cell that they see (identity tokens, n_kv <= identity_max) or over their selected cells
// (bitmaps of tree_select.cu).
//
//   out[t,h,:] = sum_c softmax_c(sm_scale q[t,h,:] . k^[c]) v^[c],  c over the token's cells;
//   k^ = fp16(kq * ksc), v^ = fp16(vq * vsc).
//
// All of a tree's tokens read the same committed cells and the 12 heads of a group share their K/V, so the
// (token, head) rows of a sequence and group, packed 12 a token, are cut into blocks of 256 rows (21 1/3
// tokens), the M of one MMA over a pair of CTAs (128 rows each).  Selected tokens attend through the same
// dense tiles, their other cells masked: gathering 2,048 cells a token costs an SM about 25 us, a masked
// 128-cell tile for 21 tokens 1.7 us of a pair.  A cluster of 2 S CTAs takes one block and group, each pair a run of its
// 128-cell tiles (how many: tree_plan.cuh), and the pairs merge by log-sum-exp in a fixed order, so that a call of few rows still
// spreads over the GPU and results do not depend on timing.  The statistics are exchanged through
// distributed shared memory, the rows through a workspace that stays in L2: 128 KB a CTA by remote shared
// memory took 6.5 us, stores or coalesced loads alike.
//
// The cache is read as int8 once per block and dequantised by producer warps into 128B-swizzled operand
// tiles; no fp16 mirror is written (a drafting step reads the cache a few times, and the mirror would cost
// three times the cache's own bytes).  In a pair each CTA holds half of a K^ tile (64 cells) and half of
// a V^ tile (128 dims), so per 128 cells an SM converts 32 KB of codes, moves about 210 KB through shared
// memory (1,650 cycles) and its half of the MMAs takes about 2,050 cycles; measured 3,300 cycles a tile.  One CTA
// per block instead converts and stores twice as much and is bound by shared memory (3,100 cycles; measured
// 5,400 a tile of 128 rows).
//
// 4 trees of 33-48 tokens after 30,000 cells, all of them attended to: 156 us, 0.40 of the measured bf16 rate over
// the call, in seven runs a block; over the CTAs' own time the tensor pipe is 54% active.  0.45 instructions are
// issued a cycle and scheduler; the MMAs take about 95 cycles an instruction (of 64 and 128 cycles of arithmetic), and a
// tile's softmax about 2,400.  The roles run at once, so the
// loop bodies share the instruction cache: with separate K and V producer bodies a quarter of all stalls were
// instruction fetches, and the call took 196 us.  A single S buffer with P kept apart (so that QK never waits on
// a PV): 208 us.  Persistent pairs over an even share of all tiles, merged by a second launch, were measured only
// with the separate bodies: 217 against 221 us then, and slower by 5 to 60 us for short caches, whose calls a second
// launch and the write-out weigh down.
//
// A cluster holds eight pairs at most, and with few sequences over long caches that leaves most of the GPU idle; then
// pairs of their own (up to half of the GPU's a block and group) take the tiles and a second launch joins their parts.
// One tree of 16 tokens after 8,192 cells (selection included) 53 us with a cluster of eight pairs and 44 with pairs of
// their own, after 30,000 107 and 69.
//
//   warps 0-3    K producers: stage = 128 dims of this CTA's 64 cells (16 KB), ring of four (two tiles)
//   warps 4-7    V producers: stage = 64 cells x this CTA's 128 dims (16 KB), ring of four (two tiles)
//   warps 8-15   load Q; two softmax warpgroups, one row per thread in each, half of the columns each:
//                mask, online softmax in base-2 units (running maximum and sum in fp32), P as fp16 into
//                TMEM over S, lazy O rescale (only when the maximum grows by more than 2^8)
//   warp 16      TMEM; rank 1 of the pair: forwards its CTA's completed operand stages to rank 0's barriers
//                rank 0: MMA issue in the order QK(0), QK(1), PV(0), QK(2), PV(1), ...
//                  S = Q K^T  (A = Q K-major, B = K^ K-major)      M=256 N=128, 16 K-steps
//                  O += P V^  (A = P from TMEM, B = V^ MN-major)   M=256 N=256, 8 K-steps
//
// Roundings below fp32: k^ and v^ (the values the library's prefill attends to), P (11 bits for cells down to 21
// binades below the row's running maximum, then fewer, none below 32: kPShift), and the output; statistics and
// sums are fp32.  Each is 2.1e-4 rms of the output on random data, 4.2e-4 together.  k^ or v^ in two fp16 parts each would
// double its half of the MMAs and of the operand tiles.  The MMAs' own sums are fp32 with about one bit more: a product
// more than some 25 binades below the output that has been added up so far is cut off whatever P holds (131,072 cells
// 17 nats below one of the same V: up to 0.3% of the output).
//
// TMEM columns (each CTA): O [0, 256), S/P buffers [256 + 128 b, 384 + 128 b), b = 0, 1.
// Every mbarrier wait is bounded; after a timeout a CTA still meets the cluster's barriers.
#include <atomic>

#include "tree_common.cuh"

namespace qsa {
namespace {

constexpr int kRows = kTreeBlock / 2;       // (token, head) rows of a CTA, 256 of a block (UMMA M)
constexpr int kParts = 2;                   // ring stages per tile and operand
constexpr int kMaxTok = (2 * kRows + kHPG - 2) / kHPG + 1;  // tokens a block's rows may touch
constexpr int kThreads = 17 * 32;
constexpr int kMaxS = kPlanSizes[kPlanSizesN - 1];  // pairs of a cluster at most
constexpr int kNS = 2;
constexpr int kOffK = 0, kOffV = kTileStages * kTileStageBytes, kOffQ = 2 * kTileStages * kTileStageBytes;
constexpr int kOffML = kOffQ + kRows * kD * 2;          // float2 (m, l) [kMaxS][kRows], pushed by every pair
constexpr int kSmem = kOffML + kMaxS * kRows * 8 + 1024;  // + alignment slack
constexpr int kOStride = kD + 4;            // floats per staged output row: 16 bytes of padding spread the banks
static_assert(kRows * kOStride * 4 <= kOffML, "the staged rows fit over the operand tiles");
static_assert(kSmem <= 227 * 1024, "shared memory");
static_assert(kMaxTok <= 32, "a lane per token of the block");
static_assert(kPlanRows == kTreeBlock && kPlanCells == kTileCells && kPlanHeads == kHPG && kPlanGroups == kGroups &&
                  kPlanDrafted == 32 * kTreeWords && 2 * kMaxS <= 16,
              "the plan's sizes are this kernel's");
constexpr uint32_t kColO = 0, kColS = 256;
constexpr float kRescaleThreshold = 8.0f;   // log2 units
// P is held as 2^(s - m + 7): at most 2^15 with the lazy maximum, so that fp16 keeps its 11 bits down to 21 binades
// below the running maximum and something down to 32.  The sum takes the same factor, which cancels in O / l.
constexpr float kPShift = 7.0f;
static_assert(kRescaleThreshold + kPShift < 16.0f, "P stays below fp16's largest value");
constexpr uint16_t kBoth = 0x3;

struct DenseTreeArgs {
  TreeBatch b;
  const __half* q;
  const int8_t* kq;
  const int8_t* vq;
  const __half* ksc;
  const __half* vsc;
  const uint32_t* bits;  // selected cells [2][n_tok][bits_pitch words], or null: selected tokens are not ours
  int bits_pitch;
  float scale_log2;
  const __half* gate;
  __half* out;
  const int4* plan;      // the blocks, longest first (tree_plan_blocks), or null: in the table's order
  float* part;           // unmerged O, [CTA of the grid][kD / 4][kRows][4]; null for one pair per block
  float2* part_ml;       // and its (m, l), [CTA of the grid][kRows], where the parts are joined by a launch of their own
  int runs;              // clusters that share a block: 1, or (with one pair a cluster) more and tree_join_kernel
  int run_tiles;         // shared calls: tiles of a run at most, so that a shorter prefix takes fewer of them
  bool behind_dense;     // own cells launched behind the prefixes'
  int clusters;          // of the prefixes' launch; without a plan there is one prefix, and there are no records
  int* status;
};

struct __align__(8) TreeBars {
  // k_full, v_full, q_full: arrived on by the warps of their own CTA, and on rank 0 once more when rank 1's
  // phase is complete.  p_full: on rank 0 only, by the warps of both.  The others receive the pair MMAs' commits
  // in both CTAs
  uint64_t k_full[kTileStages], k_empty[kTileStages], v_full[kTileStages], v_empty[kTileStages];
  uint64_t s_full[kNS], p_full[kNS], pv_done[kNS];
  uint64_t q_full, tmem_ready, drain;
};

// Block `blk` of the grid, by a warp: whether there is one, its sequence's {first pool cell, -, committed cells, first
// token row}, tokens, drafted cells and the block's first row; for lane = token of the block its mask words, whether it is
// computed here and whether it is a selected one.
struct BlockAt {
  int4 e;
  int T, drafted, row0;
  int g, run, runs;  // of a prefix: the group, and which of the runs that share the block this is
  uint32_t m[kTreeWords];
  bool ours, sel;
};
template <CellsOf kOf>
__device__ __forceinline__ BlockAt tree_block_at(const TreeBatch& b, const int4* plan, bool with_selected, int blk, int lane,
                                                 int clusters = 0) {
  BlockAt x;
  bool here;
  int sq = 0;
  if (kOf == kTreeCells && plan != nullptr) {
    const int4 head = __ldg(&plan[0]), at = __ldg(&plan[1 + 2 * blk]);
    x.row0 = __ldg(&plan[2 + 2 * blk].x);
    here = blk < head.x;
    x.e = make_int4(at.x, 0, at.y, at.w);
    x.T = at.z;
  } else {
    if constexpr (kOf == kPrefixCells) {
      // `blk` is the cluster's index and `plan` the prefixes' clusters
      int4 at, pe;
      int all;
      if (plan != nullptr) {
        sq = warp_find_seq(b.n_prefix, blk, [&](int p) { return (long long)__ldg(&plan[p]).x; });
        at = __ldg(&plan[sq]);
        pe = __ldg(&b.prefixes[sq]);
        all = __ldg(&plan[b.n_prefix].x);
      } else {
        const int T = prefix_tokens(b, 0, &pe);
        at = only_prefix_plan(pe.w, T, pe.y, clusters);
        all = (at.w * kHPG + kTreeBlock - 1) / kTreeBlock * kGroups * at.y;
      }
      const int i = blk - at.x, runs = max(at.y, 1);
      x.T = blk < all && at.y > 0 ? at.w : 0;
      x.e = make_int4(pe.x, 0, pe.y, at.z);
      x.g = i / runs % kGroups;
      x.run = i % runs;
      x.runs = runs;
      blk = i / runs / kGroups;  // of the prefix
    } else {
      sq = warp_find_seq(b.n_seq, blk, [&](int s) { return first_block(__ldg(&b.seqs[s].w), s); });
      x.T = kOf == kTreeCells ? tree_seq_tokens(b, sq, &x.e) : shared_seq_tokens(b, sq, &x.e);
    }
    const long long k = kOf == kPrefixCells ? blk : blk - first_block(x.e.w, sq);
    here = x.T > 0 && k >= 0 && k * kTreeBlock < (long long)x.T * kHPG;
    x.row0 = here ? (int)k * kTreeBlock : 0;
  }
  x.drafted = kOf == kPrefixCells ? 0 : x.T;
  const int tok = x.row0 / kHPG + lane;
  const bool live = here && lane < kMaxTok && tok < x.T && tok * kHPG < x.row0 + 2 * kRows;
  int n_kv = x.e.z;
#pragma unroll
  for (int w = 0; w < kTreeWords; ++w) {
    x.m[w] = 0u;
    if (kOf != kPrefixCells && live)
      x.m[w] = kOf == kTreeCells ? tree_mask_word(b, x.e.w + tok, w, x.T) : shared_mask_word(b, x.e.w + tok, tok, w, x.T);
    n_kv += __popc(x.m[w]);
  }
  if (kOf == kPrefixCells && plan == nullptr) {  // no records: rows that are nobody's are computed and not read
    x.ours = live;
    x.sel = false;
    return x;
  }
  if constexpr (kOf != kTreeCells) {
    const int4 t = live ? record_in(b, kOf, sq, x.e.w + tok) : make_int4(-1, 0, 0, 0);
    x.ours = t.x >= 0;
    x.sel = x.ours && t.y > b.identity_max;
    return x;
  }
  x.sel = live && n_kv > b.identity_max;
  x.ours = live && (!x.sel || with_selected);
  return x;
}

__global__ void __launch_bounds__(kPlanThreads) tree_plan_kernel(const TreeBatch b, int4* __restrict__ plan) {
  pdl_begin();
  tree_plan_blocks(b, false, plan, tree_blocks_most(b.n_seq, b.n_tok));
}

template <CellsOf kOf>
__global__ void __launch_bounds__(kThreads, 1) tree_dense_kernel(const __grid_constant__ DenseTreeArgs a, int S) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ TreeBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_blk[10];  // active, first pool cell, pos0, T, first token row, first row, drafted cells; of a prefix: group, run, runs
  __shared__ uint32_t s_mask[kMaxTok][kTreeWords];
  __shared__ uint32_t s_union[kTreeWords];       // drafted cells that some token of ours sees
  __shared__ int s_ours, s_sel;                  // bit i: token i of the block is computed here; is a selected one
  __shared__ float s_xm[2][kRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const int half = rank & 1, pair = rank >> 1;  // rows 128 half .. of the block
  const int pairs = S * a.runs;  // of the block; run `run` of its tiles
  const int blk = kOf == kPrefixCells ? blockIdx.x >> 1 : (blockIdx.x >> 1) / pairs / kGroups;
  if (tid == 0) s_abort = 0;
  if (tid < 32) {
    // a lane a barrier, in the order of the members
    static_assert(sizeof(TreeBars) == (4 * kTileStages + 3 * kNS + 3) * 8 && sizeof(TreeBars) <= 32 * 8, "a lane a barrier");
    const int i = lane - 4 * kTileStages;
    const uint32_t fwd = half ? 0u : 1u;  // rank 1's phase, forwarded
    const uint32_t count = i < 0 ? ((lane / kTileStages) & 1 ? 1u : 4u + fwd)  // k_full, k_empty, v_full, v_empty
                                 : i >= kNS && i < 2 * kNS ? 16u               // p_full
                                 : i == 3 * kNS ? 8u + fwd                     // q_full
                                                : 1u;                          // s_full, pv_done, tmem_ready, drain
    if (lane < (int)(sizeof(TreeBars) / 8)) mbar_init(reinterpret_cast<uint64_t*>(&bars) + lane, count);
    fence_mbar_init();
  }
  cluster_arrive_all();  // #0, waited for before the first remote access: every CTA's barriers are set up
  // Own cells need nothing of the prefixes' launch before them, which triggered this one when all launches before it were
  // complete: one CTA waits for it at its end, so that this launch ends no earlier (ptx.cuh, pdl_trigger: launches D and O).
  const bool late = kOf == kOwnCells && a.behind_dense;
  if (!late) pdl_begin();
  if constexpr (kOf != kTreeCells) pdl_trigger();  // the next launch's CTAs may start, or wait, beside these
  if (kOf == kTreeCells && blockIdx.x == 0) {  // one CTA looks over the whole table and flags bad entries
    for (int s = tid; s < a.b.n_seq; s += kThreads) {
      int4 e;
      if (tree_seq_tokens(a.b, s, &e) < 0) set_dev_status(a.status, QSA_DEV_BAD_ID);
    }
  }
  if (warp == 0) {
    const BlockAt x = tree_block_at<kOf>(a.b, a.plan, a.bits != nullptr, blk, lane, a.clusters);
    const unsigned all_ours = __ballot_sync(0xffffffffu, x.ours), all_sel = __ballot_sync(0xffffffffu, x.sel);
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) {
      const uint32_t u = __reduce_or_sync(0xffffffffu, x.ours ? x.m[w] : 0u);
      if (lane < kMaxTok) s_mask[lane][w] = x.m[w];
      if (lane == 0) s_union[w] = u;
    }
    if (lane == 0) {
      s_ours = (int)all_ours;
      s_sel = (int)all_sel;
      s_blk[0] = all_ours != 0u;
      s_blk[1] = x.e.x;
      s_blk[2] = x.e.z;
      s_blk[3] = x.T;
      s_blk[4] = x.e.w;
      s_blk[5] = x.row0;
      s_blk[6] = x.drafted;
      if constexpr (kOf == kPrefixCells) {
        s_blk[7] = x.g;
        s_blk[8] = x.run;
        s_blk[9] = x.runs;
      }
    }
  }
  __syncthreads();
  if (!s_blk[0]) {  // the same in every CTA of the cluster: an unused index, or no token of ours
    cluster_wait_all();
    if (late && blockIdx.x == 0) pdl_begin();
    return;
  }
  const long long cell0 = s_blk[1];
  const int pos0 = s_blk[2], T = s_blk[3], first = s_blk[4], blk_row0 = s_blk[5];
  int row0;  // this CTA's first row
  const int n_rows = cta_rows(T, blk_row0, half, &row0);
  const int drafted = kOf == kTreeCells ? T : s_blk[6];  // cells behind the committed ones
  const int n_scan = pos0 + drafted;
  const int n_tiles = (n_scan + kTileCells - 1) / kTileCells;
  const int g = kOf == kPrefixCells ? s_blk[7] : (blockIdx.x >> 1) / pairs % kGroups;
  const int run = kOf == kPrefixCells ? s_blk[8] : (blockIdx.x >> 1) % pairs;
  const int my_runs = kOf == kPrefixCells ? s_blk[9] : kOf == kOwnCells ? shared_runs(n_tiles, a.runs, a.run_tiles) : pairs;
  if (kOf == kOwnCells && run >= my_runs) {  // uniform over the cluster
    cluster_wait_all();
    return;  // not the first CTA: run 0 there is
  }
  const int j_begin = n_tiles * run / my_runs, J = n_tiles * (run + 1) / my_runs - j_begin;  // the same in both CTAs of a pair
  auto pair_addr = [&](const void* p) { return mapa_shared(smem_u32(p), (uint32_t)rank & ~1u); };  // in rank 0
  const bool merges = kOf == kTreeCells && a.runs == 1;  // in this launch; else the parts are joined by another
  float m_run = -INFINITY, l_run = 0.f;  // softmax threads: the row's running maximum (log2 units), this half's sum
  bool ok = true;

  if (warp < 8) {
    const TileRun t{cell0, pos0, drafted, j_begin, J, g, s_union, &s_abort, a.status, half};
    const bool is_v = warp >= 4;
    produce_tiles<kPair>(t, is_v ? a.vq : a.kq, is_v ? a.vsc : a.ksc, smem_u32(smem + (is_v ? kOffV : kOffK)),
                         is_v ? bars.v_full : bars.k_full, is_v ? bars.v_empty : bars.k_empty, warp & 3, lane, 0, is_v);
    cluster_wait_all();  // #0
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issue
    if (J > 0) {
      tmem_alloc_pair(&s_tmem, 512);
      tmem_relinquish_pair();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.tmem_ready);
    }
    cluster_wait_all();  // #0
    if (lane == 0 && J > 0 && half == 0) {
      tc_fence_after();
      const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
      const uint32_t idesc_qk = idesc_f16_f32(2 * kRows, kTileCells, 0, 0);
      const uint32_t idesc_pv = idesc_f16_f32(2 * kRows, kD, 0, 1);
      const uint32_t k0 = smem_u32(smem + kOffK), v0 = smem_u32(smem + kOffV);
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + kOffQ), 16, 1024);
      auto issue_qk = [&](int j) -> bool {
        const int b = j % kNS;
        if (j >= kNS && !mbar_wait_poll(&bars.pv_done[b], ((j / kNS) - 1) & 1, a.status, &s_abort)) return false;
        for (int d = 0; d < kParts; ++d) {
          const int s = j * kParts + d, slot = s % kTileStages;
          if (!mbar_wait_poll(&bars.k_full[slot], (s / kTileStages) & 1, a.status, &s_abort)) return false;
          tc_fence_after();
          const uint64_t kdesc = sdesc_sw128(k0 + slot * kTileStageBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma2_ss(tmem + kColS + b * kTileCells,
                     qdesc + (uint64_t)(((2 * d + (kk >> 2)) * (kRows * 128) + (kk & 3) * 32) >> 4),
                     kdesc + (uint64_t)(((kk >> 2) * (kTileStageBytes / 2) + (kk & 3) * 32) >> 4), idesc_qk,
                     (d > 0 || kk > 0) ? 1u : 0u);
          umma2_commit(&bars.k_empty[slot], kBoth << (rank & ~1));
        }
        umma2_commit(&bars.s_full[b], kBoth << (rank & ~1));
        return true;
      };
      auto issue_pv = [&](int j) -> bool {
        const int b = j % kNS;
        if (!mbar_wait_poll(&bars.p_full[b], (j / kNS) & 1, a.status, &s_abort)) return false;
        for (int c = 0; c < kParts; ++c) {
          const int s = j * kParts + c, slot = s % kTileStages;
          if (!mbar_wait_poll(&bars.v_full[slot], (s / kTileStages) & 1, a.status, &s_abort)) return false;
          tc_fence_after();
          const uint64_t vdesc = sdesc_sw128(v0 + slot * kTileStageBytes, kTileStageBytes / 2, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma2_ts(tmem + kColO, tmem + kColS + b * kTileCells + (4 * c + kk) * 8, vdesc + (uint64_t)((kk * 2048) >> 4),
                     idesc_pv, (j > 0 || c > 0 || kk > 0) ? 1u : 0u);
          umma2_commit(&bars.v_empty[slot], kBoth << (rank & ~1));
        }
        umma2_commit(&bars.pv_done[b], kBoth << (rank & ~1));
        return true;
      };
      bool go = mbar_wait_poll(&bars.q_full, 0, a.status, &s_abort) && issue_qk(0);
      for (int j = 0; go && j < J; ++j) {
        if (j + 1 < J) go = issue_qk(j + 1);
        go = go && issue_pv(j);
      }
      umma2_commit(&bars.drain, (uint16_t)(1u << rank));  // everything issued completes before TMEM is released
      mbar_wait(&bars.drain, 0, a.status);
    } else if (lane == 0 && J > 0) {
      // rank 1: its operands to rank 0, in the order in which the MMAs take them.  Its warps stored them with
      // ordinary stores; this thread acquires their local phases and releases them at cluster scope, with one fence
      // a tile (about 0.7 us, and little of it shows: 4 dense trees 155 -> 156 us, 32 trees 66 -> 68; a releasing
      // arrive a stage 213 and 83, and by the storing warps themselves, whose loads are in flight, 207 and 84).
      auto stored = [&](uint64_t* full, int j) -> bool {  // tile j's stages
        bool go = true;
        for (int s = j * kParts; go && s < (j + 1) * kParts; ++s)
          go = mbar_wait_poll<false>(&full[s % kTileStages], (s / kTileStages) & 1, a.status, &s_abort);
        return go;
      };
      auto forward = [&](uint64_t* full, int j) {
        for (int s = j * kParts; s < (j + 1) * kParts; ++s) mbar_arrive_cluster(pair_addr(&full[s % kTileStages]));
      };
      bool go = mbar_wait_poll<false>(&bars.q_full, 0, a.status, &s_abort) && stored(bars.k_full, 0);
      for (int j = -1; go && j < J; ++j) {  // K of tile j + 1, V of tile j
        if (j >= 0) go = (j + 1 == J || stored(bars.k_full, j + 1)) && stored(bars.v_full, j);
        if (!go) break;
        fence_cluster();
        if (j < 0) mbar_arrive_cluster(pair_addr(&bars.q_full));
        if (j + 1 < J) forward(bars.k_full, j + 1);
        if (j >= 0) forward(bars.v_full, j);
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ Q, then softmax rows
    const int st = tid - 256, wg = warp >= 12 ? 1 : 0, quarter = warp & 3;
    {
      // 16-byte chunk c of rows st / 32 + 8 i.  Rows past the last are not loaded: whatever their place holds gives
      // rows of S that are masked as a whole and rows of O that nothing reads.
      const int c = st & 31, r0 = st >> 5;
      int h = (row0 + r0) % kHPG;
      const __half* src = a.q + ((size_t)(first + (row0 + r0) / kHPG) * kHeads + g * kHPG + h) * kD + c * 8;
      uint32_t dst = smem_u32(smem + kOffQ) + (c >> 3) * (kRows * 128) + r0 * 128 + (((c & 7) ^ (r0 & 7)) << 4);
#pragma unroll 4
      for (int left = n_rows - r0; left > 0; left -= 8) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
        dst += 8 * 128;
        h += 8;
        src += 8 * kD;
        if (h >= kHPG) {  // on to the next token's rows of this group
          h -= kHPG;
          src += (kHeads - kHPG) * kD;
        }
      }
      if (a.gate && merges && pairs == 1) {  // 512 bytes a row: into L2 while the tiles run
        for (int i = st; i < n_rows * 4; i += 256) {
          const int R = row0 + (i >> 2);
          const __half* at = a.gate + ((size_t)(first + R / kHPG) * kHeads + g * kHPG + R % kHPG) * kD + (i & 3) * 64;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(at));
        }
      }
      cp_async_wait_all();
      fence_proxy_async_smem();
      __syncwarp();
      cluster_wait_all();  // #0
      if (lane == 0) mbar_arrive(&bars.q_full);
    }
    uint32_t tmem = 0u;
    if (J > 0) {
      ok = tile_wait_warp(&bars.tmem_ready, 0, a.status, &s_abort);
      tc_fence_after();
      tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
    }
    const uint32_t p_full0 = pair_addr(&bars.p_full[0]);
    const int r = quarter * 32 + lane;  // TMEM lane == this CTA's row
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int R = row0 + r;
    const int ti = R / kHPG - blk_row0 / kHPG;  // token of the block
    const bool active = r < n_rows && ((s_ours >> min(ti, 31)) & 1), chosen = active && ((s_sel >> min(ti, 31)) & 1);
    const uint2* sel_bits = reinterpret_cast<const uint2*>(
        chosen ? a.bits + (size_t)(g * a.b.n_tok + first + R / kHPG) * a.bits_pitch : nullptr);
    if (kOf == kOwnCells && chosen) sel_bits += own_column(__ldcg(&a.b.tok[first + R / kHPG].z)) / 64;
    uint2 m_next = make_uint2(0u, 0u);  // a selected row's bits, loaded a tile ahead
    auto sel_at = [&](int j) { return kOf == kOwnCells ? __ldcg(sel_bits + 2 * j + wg) : __ldg(sel_bits + 2 * j + wg); };
    if (chosen && J > 0) m_next = sel_at(j_begin);
    // 32 visibility bits from drafted cell x on: cells before the drafted ones are seen, those past the mask not
    auto bits32 = [&](int x) -> uint32_t {
      const int w = x >> 5;  // floor (called for active rows: ti is a token of the block)
      const uint32_t lo = w < 0 ? 0xffffffffu : w < kTreeWords ? s_mask[ti][w] : 0u;
      const uint32_t hi = w + 1 < 0 ? 0xffffffffu : w + 1 < kTreeWords ? s_mask[ti][w + 1] : 0u;
      return __funnelshift_r(lo, hi, x & 31);
    };
    // a CTA without a row of ours only keeps the pair's barriers going: its rows of S, P and O are not read
    const bool any_row = named_bar_any(1, 256, active);
    for (int j = 0; !any_row && j < J; ++j) {
      if (!tile_wait_warp(&bars.s_full[j % kNS], (j / kNS) & 1, a.status, &s_abort)) break;
      if (lane == 0) {
        if (half) mbar_arrive_cluster(p_full0 + 8u * (uint32_t)(j % kNS));
        else mbar_arrive(&bars.p_full[j % kNS]);
      }
    }
    for (int j = 0; any_row && j < J; ++j) {
      const int b = j % kNS;
      const bool w_ok = tile_wait_warp(&bars.s_full[b], (j / kNS) & 1, a.status, &s_abort);
      tc_fence_after();
      float s[64];
      {
        uint32_t sa[32], sb[32];
        tmem_ld32(lane_base + kColS + b * kTileCells + wg * 64, sa);
        tmem_ld32(lane_base + kColS + b * kTileCells + wg * 64 + 32, sb);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = __uint_as_float(sa[i]);
          s[32 + i] = __uint_as_float(sb[i]);
        }
      }
      const int x0 = (j_begin + j) * kTileCells + wg * 64 - pos0;  // drafted index of this half's first cell
      const uint2 m_sel = m_next;
      if (chosen && j + 1 < J) m_next = sel_at(j_begin + j + 1);
      if (x0 + 64 > 0 || !active || chosen) {  // an identity row needs no mask over committed cells
        const uint32_t m0 = !active ? 0u : chosen ? m_sel.x : bits32(x0);
        const uint32_t m1 = !active ? 0u : chosen ? m_sel.y : bits32(x0 + 32);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          s[i] = (m0 >> i) & 1u ? s[i] : -INFINITY;
          s[32 + i] = (m1 >> i) & 1u ? s[32 + i] : -INFINITY;
        }
      }
      float mx[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) mx[i] = fmaxf(s[i], s[i + 32]);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) mx[i] = fmaxf(mx[i], mx[i + w]);
      const float m_half = mx[0] * a.scale_log2;  // the scale is positive
      const bool fail = !w_ok || !ok;
      // One barrier reduction per tile (it also orders every S read before the P stores over it); the half-row
      // maxima are exchanged only at the first tile and when some row outgrows its running maximum.
      if (named_bar_any(1, 256, fail || j == 0 || m_half > m_run + kRescaleThreshold)) {
        s_xm[wg][r] = m_half;
        if (named_bar_any(1, 256, fail)) {
          ok = false;
          break;
        }
        const float m_new = fmaxf(m_run, fmaxf(m_half, s_xm[wg ^ 1][r]));
        if (j == 0) {
          m_run = m_new;
        } else {
          const bool need = m_new > m_run + kRescaleThreshold;  // the same in both warpgroups
          if (__any_sync(0xffffffffu, need)) {
            if (tile_wait_warp(&bars.pv_done[(j - 1) % kNS], ((j - 1) / kNS) & 1, a.status, &s_abort)) {
              tc_fence_after();
              const float f = need ? fast_exp2(m_run - m_new) : 1.f;
#pragma unroll 1
              for (int c0 = wg * 128; c0 < wg * 128 + 128; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(lane_base + kColO + c0, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tmem_st16(lane_base + kColO + c0, o);
              }
              tmem_wait_st();
              if (need) {
                l_run *= f;
                m_run = m_new;
              }
            } else {
              ok = false;  // reported at the next barrier reduction
            }
          }
        }
      }
      const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
      const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), nm2 = make_float2(kPShift - m_use, kPShift - m_use);
      float2 lsum = make_float2(0.f, 0.f);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = fma2(make_float2(s[32 * hf + 2 * i], s[32 * hf + 2 * i + 1]), sc2, nm2);
          e.x = fast_exp2(e.x);
          e.y = fast_exp2(e.y);
          lsum = add2(lsum, e);
          p[i] = pack_half2(e.x, e.y);
        }
        tmem_st16(lane_base + kColS + b * kTileCells + wg * 32 + 16 * hf, p);
      }
      l_run += lsum.x + lsum.y;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (half) mbar_arrive_cluster(p_full0 + 8u * (uint32_t)b);
        else mbar_arrive(&bars.p_full[b]);
      }
    }
    if (J > 0 && ok) ok = tile_wait_warp(&bars.pv_done[(J - 1) % kNS], ((J - 1) / kNS) & 1, a.status, &s_abort);
    // (m, l) of the row to the CTAs that hold the same rows; a failed or empty run contributes nothing
    const bool all_ok = !named_bar_any(1, 256, !ok);
    s_xm[wg][r] = l_run;
    named_bar_any(1, 256, false);
    const float l = l_run + s_xm[wg ^ 1][r];
    // NaN among the row's scores: a weight that the join cannot lose (the running maximum passes over NaN)
    if (kOf != kTreeCells && l != l) m_run = INFINITY;
    if (!all_ok) m_run = -INFINITY;
    if (wg == 0) {
      if (!merges) a.part_ml[(size_t)blockIdx.x * kRows + r] = make_float2(m_run, l);
      const uint32_t at = smem_u32(smem + kOffML) + (uint32_t)(pair * kRows + r) * 8u;
      for (int c = 0; c < S; ++c)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(at, 2 * c + half)), "f"(m_run), "f"(l)
                     : "memory");
    }
    // O (unscaled): to the workspace, or over the operand tiles when the block has but one pair (the last PV is
    // complete, so both CTAs' MMAs are done with them)
    if (J > 0 && any_row) {
      tc_fence_after();
      float4* grow = reinterpret_cast<float4*>(a.part) + (size_t)blockIdx.x * (kRows * kD / 4) + r;
#pragma unroll 1
      for (int c0 = wg * 128; c0 < wg * 128 + 128; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(lane_base + kColO + c0, o);
        tmem_wait_ld();
        if (merges && pairs == 1) {
          float4* dst = reinterpret_cast<float4*>(smem + (size_t)r * (kOStride * 4)) + c0 / 4;
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]), __uint_as_float(o[4 * i + 2]),
                                 __uint_as_float(o[4 * i + 3]));
        } else if (m_run != -INFINITY) {  // a warp's rows lie side by side: 512 bytes a store
#pragma unroll
          for (int i = 0; i < 8; ++i)
            grow[(size_t)(c0 / 4 + i) * kRows] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                             __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
        }
      }
    }
  }

  // ---------------------------------------------------------------- merge
  // Run c's CTA owns an S-th of its half's rows and adds every run's part in the runs' order: out = sum_c O_c 2^(m_c - M) / L.
  tc_fence_before();
  __syncwarp();
  cluster_arrive_all();
  const int per = ((n_rows + S - 1) / S + 7) & ~7;  // rows of an owner: loads of 128 bytes at least
  cluster_wait_all();  // #1: the cluster's rows and statistics are visible; no CTA touches another after this
  tc_fence_after();
  if (warp == 16 && J > 0) tmem_dealloc_pair(*reinterpret_cast<volatile uint32_t*>(&s_tmem), 512);
  if (warp < 16 && merges) {  // else tree_join_kernel, or prefix_join_kernel, merges
    const float2* ml = reinterpret_cast<const float2*>(smem + kOffML);
    auto row_at = [&](int r, size_t* at) {  // this CTA's row r: is it one of ours, and where its output starts
      const int R = row0 + r, ti = R / kHPG - blk_row0 / kHPG;
      if (r >= n_rows || !((s_ours >> ti) & 1)) return false;
      *at = ((size_t)(first + R / kHPG) * kHeads + g * kHPG + R % kHPG) * kD;
      return true;
    };
    if (S == 1) {  // a warp a row, 8 dims a lane, from shared memory; four rows' gates are loaded before any is used
      const int d8 = tid & 31;
#pragma unroll 1
      for (int r0 = tid >> 5; r0 < n_rows; r0 += 64) {
        size_t at[4];
        uint4 gw[4];
        bool mine[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          mine[u] = row_at(r0 + 16 * u, &at[u]);
          if (a.gate && mine[u]) gw[u] = __ldg(reinterpret_cast<const uint4*>(a.gate + at[u]) + d8);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (!mine[u]) continue;
          const int r = r0 + 16 * u;
          const float l = ml[r].x == -INFINITY ? 0.f : ml[r].y, inv = l > 0.f ? 1.f / l : 0.f;  // sees nothing: zeros
          float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (l > 0.f) {
            const float4* src = reinterpret_cast<const float4*>(smem + (size_t)r * (kOStride * 4)) + 2 * d8;
            const float4 x = src[0], y = src[1];
            const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = f[i] * inv;
          }
          if (a.gate) apply_gate(v, gw[u]);
          reinterpret_cast<uint4*>(a.out + at[u])[d8] = pack_out(v);
        }
      }
    } else {  // eight rows at a time, by half of the threads each: a lane has 8 dims of a row
      const int d8 = (tid >> 3) & 31;
      for (int x = (tid >> 8) * 8 + (tid & 7); x < per; x += 16) {
        const int r = pair * per + x;
        size_t at;
        if (!row_at(r, &at)) continue;
        // CTA 0 of the cluster with this half's rows, the next pair's two CTAs further: all parts are loaded at once
        // (a part of a run that has none is read and dropped)
        const float4* src = reinterpret_cast<const float4*>(a.part) + (size_t)(blockIdx.x - 2 * pair) * (kRows * kD / 4) +
                            (size_t)(2 * d8) * kRows + r;
        float4 p[kMaxS][2];
#pragma unroll
        for (int c = 0; c < kMaxS; ++c) {
          const float4* from = src + (size_t)min(c, S - 1) * (2 * kRows * kD / 4);
          p[c][0] = __ldcg(from);
          p[c][1] = __ldcg(from + kRows);
        }
        uint4 gw = make_uint4(0u, 0u, 0u, 0u);
        if (a.gate) gw = __ldg(reinterpret_cast<const uint4*>(a.gate + at) + d8);
        float M = -INFINITY, L = 0.f;
        for (int c = 0; c < S; ++c) M = fmaxf(M, ml[c * kRows + r].x);
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kMaxS; ++c) {
          const float2 st = ml[min(c, S - 1) * kRows + r];
          if (c >= S || st.x == -INFINITY) continue;  // past the last run, or nothing of this row there
          const float f = fast_exp2(st.x - M);
          L = fmaf(st.y, f, L);
          const float y[8] = {p[c][0].x, p[c][0].y, p[c][0].z, p[c][0].w, p[c][1].x, p[c][1].y, p[c][1].z, p[c][1].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = fmaf(y[i], f, v[i]);
        }
        const float inv = L > 0.f ? 1.f / L : 0.f;  // a token that sees nothing: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= inv;
        if (a.gate) apply_gate(v, gw);
        reinterpret_cast<uint4*>(a.out + at)[d8] = pack_out(v);
      }
    }
  }
  if (late && blockIdx.x == 0) pdl_begin();
}

// Joins the parts of blocks that several clusters share, in the runs' order within a slice and then slice by
// slice.  A CTA owns four rows of a block and group (so that one block's rows spread over 128 CTAs), a thread
// eight dims of a row and every fourth part, four of them loaded at once: a few round trips to L2.
constexpr int kJoinRows = 4, kJoinSlices = 4, kJoinDepth = 4, kJoinItems = kJoinRows * (kD / 8);
constexpr int kJoinThreads = kJoinItems * kJoinSlices;
__global__ void __launch_bounds__(kJoinThreads, 2) tree_join_kernel(const __grid_constant__ DenseTreeArgs a) {
  __shared__ float2 s_ml[kMaxRuns][kJoinRows];
  __shared__ float s_v[kJoinSlices - 1][9][kJoinItems];
  __shared__ int s_blk[3];
  __shared__ unsigned s_ours;
  pdl_begin();
  constexpr int kChunks = 2 * kRows / kJoinRows;
  const int tid = threadIdx.x;
  const int chunk = blockIdx.x % kChunks, g = blockIdx.x / kChunks % kGroups, blk = blockIdx.x / kChunks / kGroups;
  const int half = chunk / (kChunks / 2), r0 = chunk % (kChunks / 2) * kJoinRows;
  if (tid < 32) {
    const BlockAt x = tree_block_at<kTreeCells>(a.b, a.plan, a.bits != nullptr, blk, tid);
    const unsigned all_ours = __ballot_sync(0xffffffffu, x.ours);
    if (tid == 0) {
      s_ours = all_ours;
      s_blk[0] = x.T;
      s_blk[1] = x.e.w;
      s_blk[2] = x.row0;
    }
  }
  __syncthreads();
  const int T = s_blk[0], first = s_blk[1], blk_row0 = s_blk[2];
  int row0;
  const int n_rows = s_ours ? cta_rows(T, blk_row0, half, &row0) - r0 : 0;
  if (n_rows <= 0) return;  // the same in all threads; without tokens of ours no part was written
  const size_t cta0 = (size_t)(blk * kGroups + g) * a.runs * 2 + half;  // run 0's CTA with these rows
  for (int i = tid; i < a.runs * kJoinRows; i += kJoinThreads)
    s_ml[i / kJoinRows][i % kJoinRows] = __ldcg(&a.part_ml[(cta0 + 2 * (i / kJoinRows)) * kRows + r0 + i % kJoinRows]);
  __syncthreads();
  const int rr = tid % kJoinRows, d8 = tid / kJoinRows % (kD / 8), slice = tid / kJoinItems;
  const int R = row0 + r0 + rr, ti = R / kHPG - blk_row0 / kHPG;
  const bool mine = rr < n_rows && ((s_ours >> min(ti, 31)) & 1);
  const size_t at = ((size_t)(first + R / kHPG) * kHeads + g * kHPG + R % kHPG) * kD;
  uint4 gw = make_uint4(0u, 0u, 0u, 0u);
  if (a.gate && mine && slice == 0) gw = __ldg(reinterpret_cast<const uint4*>(a.gate + at) + d8);
  float M = -INFINITY, L = 0.f;
  for (int c = 0; c < a.runs; ++c) M = fmaxf(M, s_ml[c][rr].x);
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const float4* src = reinterpret_cast<const float4*>(a.part) + cta0 * (kRows * kD / 4) + (size_t)(2 * d8) * kRows + r0 + rr;
  for (int c0 = slice; mine && c0 < a.runs; c0 += kJoinDepth * kJoinSlices) {
    float4 p[kJoinDepth][2];
#pragma unroll
    for (int u = 0; u < kJoinDepth; ++u) {
      const float4* from = src + (size_t)min(c0 + u * kJoinSlices, a.runs - 1) * (2 * kRows * kD / 4);
      p[u][0] = __ldcg(from);
      p[u][1] = __ldcg(from + kRows);
    }
#pragma unroll
    for (int u = 0; u < kJoinDepth; ++u) {
      const int c = c0 + u * kJoinSlices;
      const float2 st = s_ml[min(c, a.runs - 1)][rr];
      if (c >= a.runs || st.x == -INFINITY) continue;  // a run that has nothing of this row wrote nothing
      const float f = fast_exp2(st.x - M);
      L = fmaf(st.y, f, L);
      const float y[8] = {p[u][0].x, p[u][0].y, p[u][0].z, p[u][0].w, p[u][1].x, p[u][1].y, p[u][1].z, p[u][1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(y[i], f, v[i]);
    }
  }
  const int item = tid % kJoinItems;
  if (slice > 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s_v[slice - 1][i][item] = v[i];
    s_v[slice - 1][8][item] = L;
  }
  __syncthreads();
  if (slice == 0 && mine) {
#pragma unroll
    for (int c = 0; c < kJoinSlices - 1; ++c) {
      L += s_v[c][8][item];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += s_v[c][i][item];
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;  // a token that sees nothing: zeros
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    if (a.gate) apply_gate(v, gw);
    reinterpret_cast<uint4*>(a.out + at)[d8] = pack_out(v);
  }
}

cudaLaunchConfig_t tree_config(int S, int clusters, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(clusters * 2 * S);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2 * S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Per device, once: the kernel's attributes, and how many clusters of each size the GPU holds (threads that race here
// find the same).  On a GB300 76, 36, 23, 15, 13, 8 and 7.
cudaError_t tree_setup(PlanHeld* held) {
  static std::atomic<int> ready[64];
  static std::atomic<int> counts[64][kPlanSizesN];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    for (auto* k : {tree_dense_kernel<kTreeCells>, tree_dense_kernel<kPrefixCells>, tree_dense_kernel<kOwnCells>})
      if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(tree_dense_kernel<kTreeCells>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    for (int i = 0; i < kPlanSizesN; ++i) {
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = tree_config(kPlanSizes[i], 1, nullptr, attr);
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, tree_dense_kernel<kTreeCells>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // a size that this GPU does not take
        n = 0;
      }
      counts[dev][i].store(n, std::memory_order_relaxed);
    }
    if (counts[dev][0].load(std::memory_order_relaxed) <= 0) return cudaErrorInvalidConfiguration;
    ready[dev].store(1, std::memory_order_release);
  }
  for (int i = 0; i < kPlanSizesN; ++i) held->n[i] = counts[dev][i].load(std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace

namespace {
// Rows of the unmerged parts, [kD] floats and a float2 (m, l) each, at the start of the workspace.
size_t part_rows(int n_seq, int n_tok, int max_n_kv) { return (size_t)parts_most(n_seq, n_tok, max_n_kv) * 2 * kRows; }
size_t part_bytes(int n_seq, int n_tok, int max_n_kv) {
  return part_rows(n_seq, n_tok, max_n_kv) * (kD * sizeof(float) + sizeof(float2));
}
}  // namespace

size_t tree_dense_workspace_bytes(int n_seq, int n_tok, int max_n_kv) {
  const size_t list = (1 + 2 * (size_t)tree_blocks_most(n_seq, n_tok)) * sizeof(int4);
  return part_bytes(n_seq, n_tok, max_n_kv) + (n_seq >= kPlanSeqs ? (list + 255) / 256 * 256 : 0);
}

int4* tree_dense_plan(const TreeBatch& b, void* ws) {
  if (b.n_seq < kPlanSeqs) return nullptr;
  return reinterpret_cast<int4*>(static_cast<uint8_t*>(ws) + part_bytes(b.n_seq, b.n_tok, b.max_n_kv));
}

cudaError_t launch_tree_dense(const TreeBatch& b, const __half* q, const int8_t* kq, const int8_t* vq, const __half* ksc,
                              const __half* vsc, const uint32_t* bits, int bits_pitch, const __half* gate, __half* out,
                              void* ws, float sm_scale, int* status, cudaStream_t stream) {
  PlanHeld held;
  cudaError_t e = tree_setup(&held);
  if (e != cudaSuccess) return e;
  const DensePlan d = dense_plan(held, b.n_seq, b.n_tok, b.max_n_kv, b.identity_max, bits != nullptr);
  int4* plan = tree_dense_plan(b, ws);
  if (plan && !bits) {  // with selected tokens the selection's first launch has made it
    e = launch_pdl(tree_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, b, plan);
    if (e != cudaSuccess) return e;
  }
  const DenseTreeArgs a{b, q, kq, vq, ksc, vsc, bits, bits_pitch, sm_scale * kLog2e, gate, out, plan,
                        static_cast<float*>(ws),
                        reinterpret_cast<float2*>(static_cast<float*>(ws) + part_rows(b.n_seq, b.n_tok, b.max_n_kv) * kD),
                        d.runs, 0, false, 0, status};
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = tree_config(d.pairs, d.blocks * kGroups * d.runs, stream, attr);
  if ((e = cudaLaunchKernelEx(&cfg, tree_dense_kernel<kTreeCells>, a, d.pairs)) != cudaSuccess || d.runs == 1) return e;
  return launch_pdl(tree_join_kernel, dim3(d.blocks * kGroups * (2 * kRows / kJoinRows)), dim3(kJoinThreads), 0, stream, a);
}

// The parts of a shared call: of its prefixes' cells (`clusters` pairs, shared out by `plan`), or of its sequences' own
// ones (about `cells` a sequence).
size_t tree_parts_workspace_bytes(int n, int n_tok, int max_cells) {
  return (size_t)shared_parts_most(n, n_tok, max_cells) * 2 * kRows * (kD * sizeof(float) + sizeof(float2));
}

namespace {
int own_part_runs(const PlanHeld& held, const TreeBatch& b, int cells) {
  return shared_plan_runs(held.n[0], b.n_seq, b.n_tok, cells, shared_parts_most(b.n_seq, b.n_tok, b.max_n_kv));
}
}  // namespace

// own_ctas: prefix_own_kernel's, each over own_cells cells; 0: the own cells go to launch_own_parts
cudaError_t prefix_clusters(const TreeBatch& b, int own_cells, int own_ctas, int* clusters) {
  PlanHeld held;
  const cudaError_t e = tree_setup(&held);
  if (e != cudaSuccess) return e;
  const Beside o = own_ctas > 0 ? beside_own(own_ctas, own_cells)
                                : beside_own_parts(b.n_seq, b.n_tok, own_cells, own_part_runs(held, b, own_cells));
  *clusters = shared_plan_clusters(held.n[0], b.n_prefix, b.n_tok, b.max_prefix, o, shared_parts_most(b.n_prefix, b.n_tok, b.max_prefix));
  return e;
}

namespace {
template <CellsOf kOf>
cudaError_t launch_parts(const TreeBatch& b, int clusters, int runs, int run_tiles, bool behind_dense, int n, int most_cells,
                         const int4* plan, const __half* q, const int8_t* kq, const int8_t* vq, const __half* ksc, const __half* vsc,
                         const uint32_t* bits, int bits_pitch, void* ws, float sm_scale, TreeParts* parts, int* status,
                         cudaStream_t stream) {
  const size_t rows = (size_t)shared_parts_most(n, b.n_tok, most_cells) * 2 * kRows;
  float* part = static_cast<float*>(ws);
  float2* ml = reinterpret_cast<float2*>(part + rows * kD);
  *parts = TreeParts{reinterpret_cast<const float4*>(part), ml, runs, run_tiles};
  const DenseTreeArgs a{b, q, kq, vq, ksc, vsc, bits, bits_pitch, sm_scale * kLog2e, nullptr, nullptr, plan, part, ml, runs, run_tiles,
                        behind_dense, clusters, status};
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = tree_config(1, clusters, stream, attr);
  return cudaLaunchKernelEx(&cfg, tree_dense_kernel<kOf>, a, 1);
}
}  // namespace

cudaError_t launch_prefix_parts(const TreeBatch& b, int clusters, const int4* plan, const __half* q, const int8_t* kq, const int8_t* vq,
                                const __half* ksc, const __half* vsc, const uint32_t* bits, int bits_pitch, void* ws,
                                float sm_scale, TreeParts* parts, int* status, cudaStream_t stream) {
  return launch_parts<kPrefixCells>(b, clusters, 1, 0, false, b.n_prefix, b.max_prefix, plan, q, kq, vq, ksc, vsc, bits, bits_pitch, ws,
                                    sm_scale, parts, status, stream);
}

cudaError_t launch_own_parts(const TreeBatch& b, int cells, bool behind_dense, const __half* q, const int8_t* kq, const int8_t* vq,
                             const __half* ksc, const __half* vsc, const uint32_t* bits, int bits_pitch, void* ws, float sm_scale,
                             TreeParts* parts, int* status, cudaStream_t stream) {
  PlanHeld held;
  const cudaError_t e = tree_setup(&held);
  if (e != cudaSuccess) return e;
  const int runs = own_part_runs(held, b, cells);
  return launch_parts<kOwnCells>(b, tree_blocks_most(b.n_seq, b.n_tok) * kGroups * runs, runs, (plan_tiles(cells) + runs - 1) / runs,
                                 behind_dense, b.n_seq, b.max_n_kv, nullptr, q, kq, vq, ksc, vsc, bits, bits_pitch, ws, sm_scale, parts,
                                 status, stream);
}

}  // namespace qsa
