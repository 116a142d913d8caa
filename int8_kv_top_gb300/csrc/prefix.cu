// qsa_prefix_attention: attention of a batch whose sequences share prefixes.
//
//   out[t,h,:] = sum_c softmax_c(sm_scale q[t,h,:] . k^[c]) v^[c],  c over the cells of the token's prefix and of its own
//   sequence (all that it sees, or its topk selected ones);  k^ = fp16(kq * ksc), v^ = fp16(vq * vsc).
//
// The softmax over both sets is joined from the parts (O, m, l) of each: M = max m, L = sum l e^(m - M), out = sum O e^(m - M) / L.
// So the prefix's cells are attended to once for all tokens behind it: their (token, head) rows, 12 a token and group, are
// packed into blocks of 256, the M of the tensor-core kernel of tree.cu, which reads the int8 cells once a block and
// writes the parts.  A sequence's own cells serve its own few tokens alone: 12 rows fill no such block, and the cells
// have nothing to share, so prefix_own_kernel streams them past a 16-row mma.sync tile, a few CTAs a token and group.
// It is launched behind the prefixes' kernel, but starts on the SMs that that one leaves and fills the others as they
// fall idle.  Sequences of many tokens (drafted trees) take the tensor-core kernel for their own cells too.
// prefix_join_kernel joins the parts.  Calls of few tokens behind short prefixes are one launch of prefix_own_kernel over
// both sets of cells: its clusters join the parts themselves.
//
// Measured (GB300; replayed graphs over warm caches): 64 tokens behind 30,000 cells, all attended to, own cells 100-600: 64 us, of
// which the tensor-core tiles' operations would take 24 at cuBLAS's rate; 48 tokens behind 16,000 that select 2,048 of
// them each: 80 us; 40 sequences of 1-16 tokens behind three prompts of 900-12,000: 145 us; 8 tokens behind 1,800: 13 us.
//
// Selection (n_kv > identity_max) shares the prefix's codes in the same way: tree_select.cu scores them once for all
// tokens behind the prefix and each sequence's own cells for its tokens, into rows of columns {prefix cells, gap up to a
// tile, own cells}; the exact top-k of select.cu gives bitmaps over these columns.
#include <algorithm>

#include "select_math.cuh"
#include "tree_common.cuh"

namespace qsa {
namespace {

// ---------------------------------------------------------------- 1. records, queries' sums, maxima
// The tables' first rows and first sequences, in shared memory where they are short, and what is looked up in them.
constexpr int kNearSeqs = 1024, kNearPrefixes = 256;
struct Finder {
  const TreeBatch& b;
  const int *row, *seq;  // shared memory, or null
  __device__ __forceinline__ Finder(const TreeBatch& batch, int* room, int tid, int threads) : b(batch) {
    row = b.n_seq <= kNearSeqs ? room : nullptr;
    seq = b.n_prefix <= kNearPrefixes ? room + kNearSeqs : nullptr;
    for (int i = tid; row && i < b.n_seq; i += threads) room[i] = __ldg(&b.seqs[i].w);
    for (int i = tid; seq && i < b.n_prefix; i += threads) room[kNearSeqs + i] = __ldg(&b.prefixes[i].z);
    __syncthreads();
  }
  __device__ __forceinline__ int prefix_at(int s) const {
    if (b.n_prefix == 0) return -1;
    return seq ? last_at(b.n_prefix, s, [&](int i) { return seq[i]; }) : prefix_of(b, s);
  }
  // Token t's record; its `more` is written where the record is that of a valid sequence.
  __device__ __forceinline__ int4 record(int t, TokMore* more) const {
    const int s = row ? last_at(b.n_seq, t, [&](int i) { return row[i]; }) : last_at(b.n_seq, t, [&](int i) { return __ldg(&b.seqs[i].w); });
    return shared_record(b, t, s, prefix_at(s), more);
  }
};

// Flags the entries that break the contract; `of` callers take them in turn.
__device__ __forceinline__ void check_tables(const TreeBatch& b, int first, int of, int* status) {
  for (int s = first; s < b.n_seq; s += of)
    if (shared_seq(b, s, prefix_of(b, s)).T < 0) set_dev_status(status, QSA_DEV_BAD_ID);
  for (int p = first; p < b.n_prefix; p += of) {
    int4 e;
    if (prefix_tokens(b, p, &e) < 0) set_dev_status(status, QSA_DEV_BAD_ID);
  }
}

// The runs of the prefixes' blocks, by a CTA of 256 threads: of L tiles at most each, L the smallest with which all runs
// find a cluster and no block has more than kMaxRuns.  Beyond 256 prefixes, whose blocks are many, one run each.
__device__ __forceinline__ void plan_prefixes(const TreeBatch& b, int4* __restrict__ plan, int clusters, int* room) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int4 e = make_int4(0, 0, 0, 0);
  int T = 0;
  auto look = [&](int p, int* blocks, int* tiles) {
    T = p < b.n_prefix ? max(prefix_tokens(b, p, &e), 0) : 0;
    *tiles = T > 0 ? (e.y + kTileCells - 1) / kTileCells : 0;
    *blocks = *tiles > 0 ? (T * kHPG + kTreeBlock - 1) / kTreeBlock * kGroups : 0;
  };
  auto sum = [&](int v) {  // over the CTA
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if (lane == 0) room[warp] = v;
    __syncthreads();
    v = 0;
    for (int i = 0; i < 8; ++i) v += room[i];
    return v;
  };
  int blocks, tiles, L = 1 << 30;
  look(tid, &blocks, &tiles);
  if (b.n_prefix <= 256) {
    int most = __reduce_max_sync(0xffffffffu, tiles);
    __syncthreads();
    if (lane == 0) room[warp] = most;
    __syncthreads();
    for (int i = 0; i < 8; ++i) most = max(most, room[i]);
    int lo = max(1, (most + kMaxRuns - 1) / kMaxRuns), hi = max(most, lo);
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (sum(blocks * ((tiles + mid - 1) / mid)) <= clusters) hi = mid;
      else lo = mid + 1;
    }
    L = lo;
  }
  int base = 0;
  for (int p0 = 0; p0 < b.n_prefix; p0 += 256) {
    if (p0 > 0) look(p0 + tid, &blocks, &tiles);
    const int runs = blocks > 0 ? (int)(((long long)tiles + L - 1) / L) : 0, n = blocks * runs;
    int x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) room[warp] = x;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < 8; ++i) {
      if (i < warp) before += room[i];
      all += room[i];
    }
    // rows that overlap (a broken table, flagged elsewhere) may ask for more clusters than there are: those prefixes get none
    const int first = base + before + x - n;
    if (p0 + tid < b.n_prefix) plan[p0 + tid] = make_int4(first, first + n <= clusters ? runs : 0, e.w, T);
    base += all;
  }
  if (tid == 0) plan[b.n_prefix] = make_int4(base, 0, 0, 0);
}

// Blocks, in this order: (token, group): Qsum and its error terms; (prefix, chunk of 2,048 cells) and (sequence, every
// own_chunks-th chunk): max |ksc|; the first three only where tokens may select.  Then 256 tokens' records each, and, where
// prefixes are attended to, a last one that shares `clusters` CTA pairs out over them: plan[p] = {first pair, runs a block and
// group, first token row, tokens}, plan[n_prefix] = {pairs in all}.
__global__ void __launch_bounds__(256) prefix_prep_kernel(const TreeBatch b, const TreeSelect w, TokMore* __restrict__ more,
                                                          bool select, int own_chunks, int4* __restrict__ plan, int clusters,
                                                          const __half* __restrict__ q, const __half* __restrict__ ksc, int* status) {
  __shared__ long long s_e[8], s_h[8];
  __shared__ uint32_t s_union[kTreeWords];
  __shared__ float s_max[8][kGroups * kNB];
  __shared__ int s_room[kNearSeqs + kNearPrefixes];
  pdl_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int x = blockIdx.x;
  if (select) {
    if (x < kGroups * b.n_tok) {
      const int t = x >> 1, g = x & 1;
      __half hi, lo;
      long long e, h_abs;
      qsum_split(q, t, g, tid, hi, lo, e, h_abs);
      __half* dst = w.qhl + (size_t)(g * b.n_tok + t) * (2 * kD) + (tid >> 6) * 128 + (tid & 63);
      dst[0] = hi;
      dst[64] = lo;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        e += __shfl_xor_sync(0xffffffffu, e, o);
        h_abs += __shfl_xor_sync(0xffffffffu, h_abs, o);
      }
      if (lane == 0) {
        s_e[warp] = e;
        s_h[warp] = h_abs;
      }
      __syncthreads();
      if (tid < kNB) {
        constexpr float kUnit = 5.9604644775390625e-8f;  // 2^-24, exact scaling
        float* row = w.eh + (size_t)(g * b.n_tok + t) * 8;
        row[tid] = __ll2float_ru(s_e[2 * tid] + s_e[2 * tid + 1]) * kUnit;
        row[kNB + tid] = __ll2float_ru(s_h[2 * tid] + s_h[2 * tid + 1]) * kUnit;
      }
      return;
    }
    x -= kGroups * b.n_tok;
    const int prefix_blocks = b.n_prefix * w.chunks_prefix, own_blocks = b.n_seq * own_chunks;
    if (x < prefix_blocks + own_blocks) {
      const bool own = x >= prefix_blocks;
      const int i = own ? (x - prefix_blocks) / own_chunks : x / w.chunks_prefix;
      const int first = own ? (x - prefix_blocks) % own_chunks : x % w.chunks_prefix;
      int4 e;
      const int T = own ? shared_seq_tokens(b, i, &e) : prefix_tokens(b, i, &e);
      if (T <= 0) return;
      const int pos0 = own ? e.z : e.y, n = own ? pos0 + T : pos0;
      float* out = own ? w.kmax + (size_t)i * w.chunks * (kGroups * kNB) : w.kmax_prefix + (size_t)i * w.chunks_prefix * (kGroups * kNB);
      for (int ch = first; ch * kTreeChunk < n; ch += own ? own_chunks : w.chunks_prefix) {
        const int c0 = ch * kTreeChunk, c1 = min(c0 + kTreeChunk, n);
        __syncthreads();
        if (tid < kTreeWords) s_union[tid] = 0u;
        __syncthreads();
        if (c1 > pos0)
          for (int j = tid; j < T * kTreeWords; j += 256) {
            const uint32_t m = shared_mask_word(b, e.w + (j >> 3), j >> 3, j & 7, T);
            if (m) atomicOr(&s_union[j & 7], m);
          }
        static_assert(kTreeWords == 8, "mask words by j mod 8");
        __syncthreads();
        float mx[kGroups * kNB];
#pragma unroll
        for (int j = 0; j < kGroups * kNB; ++j) mx[j] = 0.f;
        constexpr int kAtOnce = 4;  // cells a thread loads before it uses any
#pragma unroll 1
        for (int c = c0 + tid; c < c1; c += 256 * kAtOnce) {
          uint4 v[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int x = c + 256 * i, dj = x - pos0;
            v[i] = make_uint4(0u, 0u, 0u, 0u);  // none, or a drafted cell that no token sees
            if (x < c1 && (dj < 0 || ((s_union[dj >> 5] >> (dj & 31)) & 1u)))
              v[i] = __ldg(reinterpret_cast<const uint4*>(ksc + ((size_t)e.x + x) * (kGroups * kNB)));
          }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const uint32_t u[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
              mx[2 * j] = fmaxf(mx[2 * j], fabsf(f.x));
              mx[2 * j + 1] = fmaxf(mx[2 * j + 1], fabsf(f.y));
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kGroups * kNB; ++j) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], o));
          if (lane == 0) s_max[warp][j] = mx[j];
        }
        __syncthreads();
        if (tid < kGroups * kNB) {
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, s_max[j][tid]);
          out[(size_t)ch * (kGroups * kNB) + tid] = m;
        }
      }
      return;
    }
    x -= prefix_blocks + own_blocks;
  }
  if (x == (b.n_tok + 255) / 256) {
    plan_prefixes(b, plan, clusters, s_room);
    return;
  }
  const Finder find(b, s_room, tid, 256);
  const int t = x * 256 + tid;
  if (t < b.n_tok) b.tok[t] = find.record(t, &more[t]);
  check_tables(b, t, (b.n_tok + 255) / 256 * 256, status);
}

// ---------------------------------------------------------------- 2. own cells
constexpr int kOwnWarps = 4, kOwnThreads = kOwnWarps * 32;
constexpr int kTile = 16;                      // cells of a warp's step
constexpr int kStages = 3;                     // of its ring
constexpr int kStageBytes = 2 * kTile * kD + 2 * kTile * kNB * 2;  // codes of K and V, scales
constexpr int kQPitch = kD * 2 + 16;           // bytes of a query row: 16 of padding spread the banks
constexpr int kOffRing = 16 * kQPitch;
constexpr int kOwnSmem = kOffRing + kOwnWarps * kStages * kStageBytes;
constexpr int kMaxOwn = 32, kMostOwn = 2048;  // CTAs that share a (token, group), and of a call and group where they do
static_assert(2 * (kOwnSmem + 3 * 1024) <= 228 * 1024, "two CTAs on an SM");
constexpr int kOwnSmemAlone = 116 * 1024;      // one: clusters otherwise put two of their CTAs on an SM while others have none
// A warp's unmerged rows, over the ring once the cells are attended to: 4 floats of padding every 32 dims and a pitch of 16 banks
// more, so that the eight lanes of a store's phase (two rows, four runs of 32 dims) meet different banks.
__device__ __forceinline__ constexpr int o_at(int dim) { return dim + dim / 32 * 4; }
constexpr int kOPitch = kD + kD / 32 * 4 + 16;
static_assert(kOwnWarps * kHPG * kOPitch * 4 <= kOwnWarps * kStages * kStageBytes, "the rows fit over the ring");
constexpr int kMaxMerge = 8;  // CTAs of a cluster that merges
constexpr int kOffMerge = kOffRing + kOwnWarps * kHPG * kOPitch * 4;  // behind them, the parts of a cluster's CTAs: [CTA][item][8 dims]
static_assert(kOffMerge + kHPG * kD * 4 <= kOwnSmem && kOffMerge % 16 == 0 && kHPG * (kD / 8) % kMaxMerge == 0, "fit over it too");
static_assert((kNearSeqs + kNearPrefixes) * 4 <= kOwnWarps * kStages * kStageBytes, "and before them, the tables");
static_assert(kOffRing % 16 == 0 && kStageBytes % 16 == 0, "16-byte copies");
constexpr float kRescaleBy = 8.f, kPUp = 7.f;  // log2 units; as in tree.cu

struct OwnArgs {
  TreeBatch b;
  TokMore* more;
  bool behind_dense;     // launched behind the prefixes' kernel
  bool shared;           // the prefixes' cells are attended to here too: no other kernel does
  bool records;          // made here, and the tables checked (else by prefix_prep_kernel)
  int* status;
  const __half* q;
  const int8_t* kq;
  const int8_t* vq;
  const __half* ksc;
  const __half* vsc;
  const uint32_t* bits;  // selected columns [2][n_tok][bits_pitch words], or null
  int bits_pitch;
  float scale_log2;
  const __half* gate;    // gate and out: where these are all of a token's cells, and one cluster has them
  __half* out;
  float* o;              // else unmerged rows [n_tok][2][S][kHPG][kD], and their (m, l) [n_tok][2][S][kHPG]
  float2* ml;
};

// S CTAs a (token, group), an S-th of its tiles of 16 cells each.  The warps take the tiles in turn, each through a ring of its own:
//   S = Q K^T  (A = 16 rows of Q, 12 of them heads; B = K^, two n8 tiles), 16 k16 steps
//   O += P V^  (A = P as it stands in S's registers, B = V^, 32 n8 tiles), one k16 step
// 64 MMAs a tile, of which an SM starts one in about 8.5 cycles (34 on each of its four tensor cores): the 24,600 cells of 48 tokens
// with 50-900 own cells take 10,100 cycles of its matrix pipe out of 30,600 active ones in a kernel of 23.6 us (alone; 25.8 MB from
// DRAM, issue slots 24-33% in use).  So no unit is full: what bounds it is a warp's tiles in line (loads, the MMAs, the
// softmax between the two products), in the CTA of the longest sequence, which has seven rounds where the shortest has one.
// Lanes take the k dims, and V's n dims, in an order of their own, the same for both operands, so that a lane's codes are 16
// bytes side by side: of a k64 block lane (n, i) has dims 16 i .. 16 i + 15 of cell n, four k16 steps of four; of V lane
// (n, i) has dims 16 n .. 16 n + 15 of a half of cells 2 i, 2 i + 1, 2 i + 8 and 2 i + 9, which sixteen n8 tiles take one by one.  The
// 16-byte chunks of a cell's row are xored by a bit (K: the cell's lowest, times 4; V: its next two, times 2), so that
// the eight lanes of a shared-memory phase meet different banks.
__global__ void __launch_bounds__(kOwnThreads, 2) prefix_own_kernel(const __grid_constant__ OwnArgs a, int S) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 s_ml[kOwnWarps][16];   // (m, l) of the warps' rows
  __shared__ float s_wf[kOwnWarps][kHPG];  // what the warps' rows are multiplied by
  __shared__ float2 s_sum[kHPG];           // (m, l) of the CTA's
  __shared__ float2 s_all[kMaxMerge][kHPG];  // and of the cluster's CTAs
  // Behind the prefixes' kernel nothing here needs what that one writes, and it triggered this launch when all launches
  // before it were complete: no wait (launch O of ptx.cuh, pdl_trigger).  One CTA waits for it at its end, so that this launch
  // ends no earlier.
  if (!a.behind_dense) pdl_begin();
  if (a.out == nullptr) pdl_trigger();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % S, g = blockIdx.x / S % kGroups, t = blockIdx.x / S / kGroups;
  const size_t out_row = ((size_t)t * kHeads + g * kHPG) * kD;
  // ---- the queries' rows; 12 .. 15 are zeros
#pragma unroll 1
  for (int i = tid; i < 16 * 32; i += kOwnThreads) {
    const int r = i >> 5, c = i & 31;
    uint8_t* to = smem + r * kQPitch + c * 16;
    if (r < kHPG)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to)),
                   "l"(reinterpret_cast<uint64_t>(a.q + out_row + (size_t)r * kD + c * 8))
                   : "memory");
    else
      *reinterpret_cast<uint4*>(to) = make_uint4(0u, 0u, 0u, 0u);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  int4 ti, e;
  if (a.records) {
    const Finder find(a.b, reinterpret_cast<int*>(smem + kOffRing), tid, kOwnThreads);
    TokMore more;
    ti = find.record(t, &more);
    e = more.seq;
    if (g == 0 && rank == 0 && tid == 0) {
      a.b.tok[t] = ti;
      a.more[t] = more;
    }
    __syncthreads();  // the ring is free
  } else {
    ti = __ldcg(&a.b.tok[t]);
    e = __ldcg(&a.more[t].seq);
  }
  auto last = [&] {  // off the path
    if (a.records) check_tables(a.b, blockIdx.x * kOwnThreads + tid, gridDim.x * kOwnThreads, a.status);
    if (a.behind_dense && blockIdx.x == 0) pdl_begin();
  };
  if (ti.x < 0) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    last();
    return;
  }
  const int T = e.z, i_tok = t - e.w, pos0 = e.y;
  const bool chosen = a.bits != nullptr && ti.y > a.b.identity_max;
  const int n_own = pos0 + (a.b.tree ? T : i_tok + 1), n_px = a.shared ? ti.z : 0;
  const int px_tiles = (n_px + kTile - 1) / kTile, n_tiles = px_tiles + (n_own + kTile - 1) / kTile;  // the prefix's come first
  const int begin = (int)((long long)n_tiles * rank / S), end = (int)((long long)n_tiles * (rank + 1) / S);
  const int mine = max(0, (end - begin - warp + kOwnWarps - 1) / kOwnWarps);  // tiles begin + warp + 4 j
  const uint8_t* my_ring = smem + kOffRing + warp * (kStages * kStageBytes);
  const uint32_t ring = smem_u32(my_ring);
  const size_t own0 = (size_t)e.x, px0 = px_tiles > 0 ? (size_t)__ldg(&a.b.prefixes[ti.w].x) : 0;
  auto load = [&](int j) {
    if (j < mine) {
      const int tile = begin + warp + kOwnWarps * j;
      const bool own = tile >= px_tiles;
      const int c0 = (own ? tile - px_tiles : tile) * kTile, n = own ? n_own : n_px;
      const size_t cell0 = own ? own0 : px0;
      const uint32_t st = ring + (j % kStages) * kStageBytes;
      const int chunk = lane & 15;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = 2 * i + (lane >> 4);
        const size_t row = ((cell0 + min(c0 + c, n - 1)) * kGroups + g) * kD + chunk * 16;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(st + c * kD + ((chunk ^ ((c & 1) << 2)) << 4)),
                     "l"(reinterpret_cast<uint64_t>(a.kq + row))
                     : "memory");
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(st + kTile * kD + c * kD + ((chunk ^ (((c >> 1) & 3) << 1)) << 4)),
                     "l"(reinterpret_cast<uint64_t>(a.vq + row))
                     : "memory");
      }
      const __half* sc = (lane < 16 ? a.ksc : a.vsc) + ((cell0 + min(c0 + (lane & 15), n - 1)) * kGroups + g) * kNB;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(st + 2 * kTile * kD + lane * 8), "l"(reinterpret_cast<uint64_t>(sc))
                   : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const uint32_t* bit_row = chosen ? a.bits + (size_t)(g * a.b.n_tok + t) * a.bits_pitch : nullptr;
  // the 16 cells of a tile that are attended to, as bits
  auto seen16 = [&](int tile) -> uint32_t {
    const bool own = tile >= px_tiles;
    const int c0 = (own ? tile - px_tiles : tile) * kTile;
    if (chosen) {
      const int column = c0 + (own ? own_column(ti.z) : 0);
      return (__ldcg(bit_row + (column >> 5)) >> (column & 31)) & 0xffffu;
    }
    if (!own) return 0xffffu >> max(c0 + kTile - n_px, 0);
    if (c0 + kTile <= pos0) return 0xffffu;
    const int c = c0 + (lane & 15), dj = c - pos0;
    const bool s = dj < 0 || (dj < T && ((shared_mask_word(a.b, t, i_tok, min(dj >> 5, kTreeWords - 1), T) >> (dj & 31)) & 1u));
    return __ballot_sync(0xffffffffu, s) & 0xffffu;
  };
  float o[32][4];
#pragma unroll
  for (int i = 0; i < 32; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;  // rows lane / 4 and 8 above: running maximum (log2 units), lane's sum
  load(0);
  load(1);
  asm volatile("cp.async.wait_group 2;" ::: "memory");
  __syncthreads();  // the queries are in shared memory
  const int r = lane >> 2, i4 = lane & 3;
  const uint8_t *q_lo = smem + r * kQPitch + i4 * 32, *q_hi = q_lo + 8 * kQPitch;
  auto at128 = [](const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); };
  for (int j = 0; j < mine; ++j) {
    load(j + 2);
    const uint32_t seen = seen16(begin + warp + kOwnWarps * j);
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    __syncwarp();
    const uint8_t* st = my_ring + (j % kStages) * kStageBytes;
    const uint16_t *k_sc = reinterpret_cast<const uint16_t*>(st + 2 * kTile * kD), *v_sc = k_sc + kTile * kNB;
    if (seen) {
      float s[2][4] = {}, s_odd[2][4] = {};  // two sums each: chains of eight MMAs
#pragma unroll
      for (int b = 0; b < kNB; ++b) {
        const uint4 qa = at128(q_lo + b * 128), qb = at128(q_lo + b * 128 + 16);
        const uint4 qc = at128(q_hi + b * 128), qd = at128(q_hi + b * 128 + 16);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int c = 8 * i + r;
          const uint4 k = at128(st + c * kD + (((4 * b + i4) ^ ((c & 1) << 2)) << 4));
          const __half2 sc = __half2half2(__ushort_as_half(k_sc[c * kNB + b]));
          float(&sum)[4] = b & 1 ? s_odd[i] : s[i];
          uint32_t x[4], y[4];
          dequant8(k.x, k.y, sc, x);
          dequant8(k.z, k.w, sc, y);
          mma16816(sum, qa.x, qc.x, qa.y, qc.y, x[0], x[1]);
          mma16816(sum, qa.z, qc.z, qa.w, qc.w, x[2], x[3]);
          mma16816(sum, qb.x, qd.x, qb.y, qd.y, y[0], y[1]);
          mma16816(sum, qb.z, qd.z, qb.w, qd.w, y[2], y[3]);
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          s[i][k] = (seen >> (8 * i + 2 * i4 + (k & 1))) & 1u ? s[i][k] + s_odd[i][k] : -INFINITY;
      float x0 = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1]));
      float x1 = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]));
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, d));
        x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, d));
      }
      x0 *= a.scale_log2;  // the scale is positive
      x1 *= a.scale_log2;
      if (__any_sync(0xffffffffu, x0 > m0 + kRescaleBy || x1 > m1 + kRescaleBy)) {
        const float n0 = x0 > m0 + kRescaleBy ? x0 : m0, n1 = x1 > m1 + kRescaleBy ? x1 : m1;
        const float f0 = m0 == -INFINITY ? 0.f : fast_exp2(m0 - n0), f1 = m1 == -INFINITY ? 0.f : fast_exp2(m1 - n1);
        m0 = n0;
        m1 = n1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          o[i][0] *= f0;
          o[i][1] *= f0;
          o[i][2] *= f1;
          o[i][3] *= f1;
        }
      }
      // a row that has seen nothing yet: its scores are all -inf, and so is its maximum
      const float d0 = kPUp - (m0 == -INFINITY ? 0.f : m0), d1 = kPUp - (m1 == -INFINITY ? 0.f : m1);
      uint32_t p[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float e0 = fast_exp2(fmaf(s[i][0], a.scale_log2, d0)), e1 = fast_exp2(fmaf(s[i][1], a.scale_log2, d0));
        const float e2 = fast_exp2(fmaf(s[i][2], a.scale_log2, d1)), e3 = fast_exp2(fmaf(s[i][3], a.scale_log2, d1));
        l0 += e0 + e1;
        l1 += e2 + e3;
        p[2 * i] = pack_half2(e0, e1);
        p[2 * i + 1] = pack_half2(e2, e3);
      }
      const uint8_t* vs = st + kTile * kD;
      const int ca = 2 * i4;  // this lane's cells: ca, ca + 1, ca + 8, ca + 9
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // cells that are not attended to count with a scale of 0, whatever they hold
        auto scale = [&](int c) {
          const uint16_t x = v_sc[c * kNB + 2 * hf + (r >> 2)];
          return __ushort_as_half((seen >> c) & 1u ? x : (uint16_t)0);
        };
        const __half2 sa = __halves2half2(scale(ca), scale(ca + 1)), sb = __halves2half2(scale(ca + 8), scale(ca + 9));
        auto codes = [&](int c) { return at128(vs + c * kD + (((8 * hf + r) ^ (((c >> 1) & 3) << 1)) << 4)); };
        const uint4 v0 = codes(ca), v1 = codes(ca + 1), v2 = codes(ca + 8), v3 = codes(ca + 9);
        const uint32_t w0[4] = {v0.x, v0.y, v0.z, v0.w}, w1[4] = {v1.x, v1.y, v1.z, v1.w};
        const uint32_t w2[4] = {v2.x, v2.y, v2.z, v2.w}, w3[4] = {v3.x, v3.y, v3.z, v3.w};
        const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152, as in dequant8
        auto pair = [&](uint32_t x, uint32_t sel, const __half2& sc) {  // two cells' codes of one dim, times their scales
          uint32_t h = __byte_perm(x, 0x64646464u, sel);
          __half2 v = __hmul2(__hsub2(*reinterpret_cast<__half2*>(&h), bias), sc);
          return *reinterpret_cast<uint32_t*>(&v);
        };
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t ab = __byte_perm(w0[w], w1[w], y ? 0x7362 : 0x5140) ^ 0x80808080u;
            const uint32_t cd = __byte_perm(w2[w], w3[w], y ? 0x7362 : 0x5140) ^ 0x80808080u;
            const int n = 16 * hf + 4 * w + 2 * y;
            mma16816(o[n], p[0], p[1], p[2], p[3], pair(ab, 0x4140, sa), pair(cd, 0x4140, sb));
            mma16816(o[n + 1], p[0], p[1], p[2], p[3], pair(ab, 0x4342, sa), pair(cd, 0x4342, sb));
          }
        }
      }
    }
    __syncwarp();  // the stage is free
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, d);
    l1 += __shfl_xor_sync(0xffffffffu, l1, d);
  }
  if (i4 == 0) {  // NaN among a row's scores: a maximum that keeps its weight from being lost (fmaxf passes over NaN)
    s_ml[warp][r] = make_float2(l0 != l0 ? INFINITY : m0, l0);
    s_ml[warp][r + 8] = make_float2(l1 != l1 ? INFINITY : m1, l1);
  }
  __syncthreads();  // every warp is done with its ring
  const bool merges = a.out != nullptr && S > 1;
  if (merges) cluster_arrive_all();
  if (tid < kHPG) {  // the warps' weights, and (m, l) of the CTA
    float2 x[kOwnWarps];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      x[w] = s_ml[w][tid];
      m = fmaxf(m, x[w].x);
    }
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float f = x[w].x == -INFINITY ? 0.f : fast_exp2(x[w].x - m);
      s_wf[w][tid] = f;
      l = fmaf(x[w].y, f, l);
    }
    s_sum[tid] = make_float2(m, l);
    if (a.out == nullptr) a.ml[(size_t)blockIdx.x * kHPG + tid] = make_float2(m, l);
  }
  // O: lane (r, i) has dims 128 hf + 32 i + {0, 16} + n of rows r and r + 8
  float* rows = reinterpret_cast<float*>(smem + kOffRing) + warp * (kHPG * kOPitch);
#pragma unroll
  for (int hf = 0; hf < 2; ++hf)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = r + (k >> 1) * 8, dim = 128 * hf + 32 * i4 + 16 * (k & 1);
      if (row < kHPG) {
#pragma unroll
        for (int n = 0; n < 16; n += 4)
          *reinterpret_cast<float4*>(rows + row * kOPitch + o_at(dim) + n) =
              make_float4(o[16 * hf + n][k], o[16 * hf + n + 1][k], o[16 * hf + n + 2][k], o[16 * hf + n + 3][k]);
      }
    }
  // a CTA is (token, group, rank), as its rows are in `o`
  static_assert(kGroups == 2, "blocks in the order of the rows");
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(smem + kOffRing);
  // A cluster's CTA owns an S-th of the items (8 dims of a row): each CTA's part of them is pushed to it.
  const int per = kHPG * (kD / 8) / S;
  if (merges) {
    cluster_wait_all();  // every CTA's ring is free
    if (tid < kHPG * S)
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(&s_all[rank][tid % kHPG]), tid / kHPG)),
                   "f"(s_sum[tid % kHPG].x), "f"(s_sum[tid % kHPG].y)
                   : "memory");
  }
#pragma unroll 1
  for (int i = tid; i < kHPG * (kD / 8); i += kOwnThreads) {
    const int h = i / (kD / 8), d = i % (kD / 8) * 8;
    if (a.out == nullptr && s_sum[h].x == -INFINITY) continue;  // nothing of this row here
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float f = s_wf[w][h];
      const float4* z = reinterpret_cast<const float4*>(all + (w * kHPG + h) * kOPitch + o_at(d));
      const float4 x = z[0], y = z[1];
      const float u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(u[k], f, v[k]);  // a row that has seen nothing holds zeros
    }
    if (a.out == nullptr) {
      float4* to = reinterpret_cast<float4*>(a.o + ((size_t)blockIdx.x * kHPG + h) * kD + d);
      to[0] = make_float4(v[0], v[1], v[2], v[3]);
      to[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else if (merges) {
      const uint32_t to = mapa_shared(smem_u32(smem + kOffMerge) + (uint32_t)(rank * per + i % per) * 32u, i / per);
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(to + 16u), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                   : "memory");
    } else {
      const float l = s_sum[h].y, inv = l > 0.f ? 1.f / l : 0.f;  // a token that sees nothing: zeros
      const size_t at = out_row + (size_t)h * kD + d;
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
      if (a.gate) apply_gate(v, __ldg(reinterpret_cast<const uint4*>(a.gate + at)));
      *reinterpret_cast<uint4*>(a.out + at) = pack_out(v);
    }
  }
  if (merges) {
    cluster_arrive_all();
    cluster_wait_all();  // the parts are here; no CTA touches another's memory after this
#pragma unroll 1
    for (int j = tid; j < per; j += kOwnThreads) {
      const int i = rank * per + j, h = i / (kD / 8);
      const size_t at = out_row + (size_t)h * kD + i % (kD / 8) * 8;
      uint4 gw = make_uint4(0u, 0u, 0u, 0u);
      if (a.gate) gw = __ldg(reinterpret_cast<const uint4*>(a.gate + at));
      float M = -INFINITY, L = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < S; ++c) M = fmaxf(M, s_all[c][h].x);
#pragma unroll 2
      for (int c = 0; c < S; ++c) {
        const float f = s_all[c][h].x == -INFINITY ? 0.f : fast_exp2(s_all[c][h].x - M);
        const float4* z = reinterpret_cast<const float4*>(smem + kOffMerge + (size_t)(c * per + j) * 32);
        const float4 x = z[0], y = z[1];
        const float u[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        if (f == 0.f) continue;  // a part that has nothing of the row
        L = fmaf(s_all[c][h].y, f, L);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = fmaf(u[k], f, v[k]);
      }
      const float inv = L > 0.f ? 1.f / L : 0.f;  // a token that sees nothing: zeros
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] *= inv;
      if (a.gate) apply_gate(v, gw);
      *reinterpret_cast<uint4*>(a.out + at) = pack_out(v);
    }
  }
  last();
}

// ---------------------------------------------------------------- 3. the join
// A CTA a (token, group) and slice of the dims.  The parts' slices are fetched to shared memory at once (a part's rows
// of a token lie side by side, 192 bytes a float4 of dims), while a warp a row, or three, makes the weights e^(m - M).
// Few tokens take eight slices, whose small CTAs wait on the SMs beside those of the launch before; of many tokens two, so that
// less is looked up again.  The whole call behind 6,000 cells, us with 8 / 4 / 2 / 1 slices: 16 tokens 27/29/28/32, 64 31/32/34/35, 100 42/40/41/41,
// 250 114/108/106/105; 40 sequences of 8 tokens 88/82/78/79.  kFit parts are fetched at a time.
template <int kSlices>
struct JoinShape {
  static constexpr int kQuads = kD / kSlices / 4, kFit = 2 * kSlices;
  static constexpr int kThreads = std::max(128, kHPG * kQuads / 2);
};
struct PartSet {  // parts of a token's rows, as the tensor-core kernel or prefix_own_kernel leaves them
  TreeParts p;
  bool rows;      // of prefix_own_kernel: [n_tok][2][runs][kHPG]
};
struct JoinArgs {
  TreeBatch b;
  const TokMore* more;
  PartSet prefix, own;  // runs 0: none
  const int4* plan;     // of the prefixes' parts; null: one prefix, and the launch before makes the records
  int clusters;
  const __half* gate;
  __half* out;
};
constexpr int kMostParts = kMaxRuns + kMaxRuns;
constexpr int kJoinMany = 88;  // tokens
template <int kSlices>
__global__ void __launch_bounds__(JoinShape<kSlices>::kThreads) prefix_join_kernel(const __grid_constant__ JoinArgs a) {
  constexpr int kQuads = JoinShape<kSlices>::kQuads, kFit = JoinShape<kSlices>::kFit, kJoinThreads = JoinShape<kSlices>::kThreads;
  static_assert(kJoinThreads % 32 == 0 && kHPG % (kJoinThreads / 32) == 0, "whole rows a warp");
  __shared__ __align__(16) float4 s_part[kFit * kQuads * kHPG];  // [part][quad][row]
  __shared__ float s_w[kMostParts][kHPG];                        // weights of the parts
  __shared__ size_t s_from[2][kHPG], s_ml[2][kHPG];              // a row of part 0 (prefix, own): its O, in float4, and its (m, l)
  __shared__ float s_inv[kHPG];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int slice = blockIdx.x % kSlices, g = blockIdx.x / kSlices % kGroups, t = blockIdx.x / kSlices / kGroups;
  // With a plan, the launch before triggered this one when the one that makes the records was complete (ptx.cuh, pdl_trigger).
  const bool early = a.plan != nullptr;
  if (!early) pdl_begin();
  const int4 ti = __ldcg(&a.b.tok[t]), e = __ldcg(&a.more[t].seq);
  int4 pl = make_int4(0, 0, 0, 0);
  if (a.prefix.p.runs > 0 && ti.x >= 0 && ti.z > 0) {
    if (early) {
      pl = __ldcg(&a.plan[ti.w]);
    } else {
      int4 pe;
      const int T = prefix_tokens(a.b, 0, &pe);
      pl = only_prefix_plan(pe.w, T, pe.y, a.clusters);
    }
  }
  const int px_runs = pl.y;
  const int own_runs = a.own.rows ? a.own.p.runs : a.own.p.runs ? shared_runs((e.y + e.z + kTileCells - 1) / kTileCells, a.own.p.runs, a.own.p.run_tiles) : 0;
  const int n = px_runs + own_runs;
  if (ti.x >= 0 && tid < 2 * kHPG) {
    const bool own = tid >= kHPG;
    const int h = own ? tid - kHPG : tid;
    if (own && a.own.rows) {
      s_ml[1][h] = ((size_t)t * kGroups + g) * a.own.p.runs * kHPG + h;
      s_from[1][h] = s_ml[1][h] * (kD / 4);
    } else if (own ? a.own.p.runs > 0 : px_runs > 0) {
      size_t cta;
      int row;
      if (own) part_row(first_block(e.w, ti.x) * kGroups * a.own.p.runs, e.z, g, a.own.p.runs, (t - e.w) * kHPG + h, &cta, &row);
      else part_row(pl.x, pl.w, g, px_runs, (t - pl.z) * kHPG + h, &cta, &row);
      s_ml[own][h] = cta * (kTreeBlock / 2) + row;
      s_from[own][h] = cta * (kTreeBlock / 2 * kD / 4) + row;
    }
  }
  // this thread's eight dims of a row
  const int h = tid % kHPG, d8 = tid / kHPG;
  const bool mine = ti.x >= 0 && d8 < kQuads / 2;
  const size_t at = ((size_t)t * kHeads + g * kHPG + h) * kD + slice * (kD / kSlices) + d8 * 8;
  uint4 gw = make_uint4(0u, 0u, 0u, 0u);
  if (mine && a.gate) gw = __ldg(reinterpret_cast<const uint4*>(a.gate + at));
  __syncthreads();
  if (early) pdl_begin();
  if (ti.x < 0) return;
  // float4 between the dims of a row, float4 between parts, and (m, l) between parts
  constexpr int kDimStep = kTreeBlock / 2, kMlStep = kTreeBlock;
  constexpr size_t kRunStep = (size_t)kTreeBlock * kD / 4;
  const int own_dim = a.own.rows ? 1 : kDimStep, own_ml = a.own.rows ? kHPG : kMlStep;
  const size_t own_run = a.own.rows ? (size_t)kHPG * kD / 4 : kRunStep;
  auto fetch = [&](int u0, int count) {  // parts u0 .. u0 + count - 1
    const uint32_t to = smem_u32(s_part);
    int r = h, x = d8;  // row, and part x quad
#pragma unroll 2
    for (int i = tid; i < count * kQuads * kHPG; i += kJoinThreads) {
      const int u = u0 + x / kQuads, d = slice * kQuads + x % kQuads;
      const float4* from = u < px_runs ? a.prefix.p.o + s_from[0][r] + u * kRunStep + d * kDimStep
                                       : a.own.p.o + s_from[1][r] + (u - px_runs) * own_run + d * own_dim;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(reinterpret_cast<uint64_t>(from)) : "memory");
      r += kJoinThreads % kHPG;
      x += kJoinThreads / kHPG;
      if (r >= kHPG) {
        r -= kHPG;
        ++x;
      }
    }
  };
  // weights, a warp three rows, a lane a part (and the 32nd, 64th behind it)
  constexpr int kRowsPerWarp = kHPG / (kJoinThreads / 32), kPerLane = (kMostParts + 31) / 32;
  float2 st[kRowsPerWarp][kPerLane];
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k)
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const int r = warp + k * (kJoinThreads / 32), u = lane + 32 * j;
      st[k][j] = make_float2(-INFINITY, 0.f);
      if (u < n)
        st[k][j] = __ldcg(u < px_runs ? a.prefix.p.ml + s_ml[0][r] + u * kMlStep : a.own.p.ml + s_ml[1][r] + (u - px_runs) * own_ml);
    }
  fetch(0, min(n, kFit));  // behind the loads of (m, l), which are waited for first
#pragma unroll
  for (int k = 0; k < kRowsPerWarp; ++k) {
    const int r = warp + k * (kJoinThreads / 32);
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) M = fmaxf(M, st[k][j].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int j = 0; j < kPerLane; ++j) {
      const float f = st[k][j].x == -INFINITY ? 0.f : fast_exp2(st[k][j].x - M);  // nothing of this row there: weight 0
      if (f != 0.f) L = fmaf(st[k][j].y, f, L);
      if (lane + 32 * j < n) s_w[lane + 32 * j][r] = f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_inv[r] = L > 0.f ? 1.f / L : 0.f;  // a token that sees nothing: zeros
  }
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int u0 = 0; u0 < n; u0 += kFit) {
    const int count = min(n - u0, kFit);
    if (u0 > 0) {
      __syncthreads();  // the round before is read
      fetch(u0, count);
    }
    cp_async_wait_all();
    __syncthreads();
    if (!mine) continue;
#pragma unroll 2
    for (int u = 0; u < count; ++u) {
      const float f = s_w[u0 + u][h];
      if (f == 0.f) continue;  // a part that has nothing of the row wrote nothing
      const float4 p = s_part[(u * kQuads + 2 * d8) * kHPG + h], q = s_part[(u * kQuads + 2 * d8 + 1) * kHPG + h];
      const float z[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = fmaf(z[k], f, v[k]);
    }
  }
  if (!mine) return;
  const float inv = s_inv[h];
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] *= inv;
  if (a.gate) apply_gate(v, gw);
  *reinterpret_cast<uint4*>(a.out + at) = pack_out(v);
}

// ---------------------------------------------------------------- the call
// Up to how many own cells (about) of a token or two a sequence the top-k kernel scores them itself.
constexpr int kOwnInTopk = 2048;
// From how many tokens a sequence (on average) their own cells go to the tensor-core kernel: five, or four with many own cells.  40
// sequences behind 6,000 cells with 50, 300, 1,000, 2,000 own cells, all attended to, us on prefix_own_kernel / the tensor cores: 3 tokens
// each 38/47, 47/53, 66/68, 98/95; 4 tokens 47/49, 49/58, 82/63, 119/94; 5 tokens 53/58, 61/62, 97/83, 140/97; 6 tokens 60/63, 75/64, 112/80, 165/103.
constexpr int kOwnTokens = 4, kManyOwnCells = 512;
// Up to how many tokens times prefix cells prefix_own_kernel takes the prefixes' cells too: it reads and multiplies them
// again for every token, but the tensor-core kernel takes 11 us for the first tile and a join of 5.  Own cells 50-150; us with
// prefix_own_kernel alone / with both: 1 token behind 250 cells 10/16, behind 2,000 15/19, 16,000 24/28; 8 tokens behind 250 11/17, 2,000
// 16/21, 4,000 24/33, 8,000 43/26; 16 tokens behind 2,000 19/24, 4,000 39/32; 64 tokens behind 500 20/20, 1,000 35/28.
constexpr long long kFewCells = 1ll << 15;

inline int own_rows(int n_tok) { return std::max(n_tok, std::min(kMaxOwn * n_tok, kMostOwn)); }  // tokens x CTAs that share one

struct Layout {
  size_t tok, more, plan, prefix, own, select, kmax, bytes;
};
Layout layout(int n_prefix, int n_seq, int n_tok, int max_prefix, int max_n_kv, int identity_max) {
  Layout l{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return at;
  };
  l.tok = take((size_t)n_tok * sizeof(int4));
  l.more = take((size_t)n_tok * sizeof(TokMore));
  l.plan = take(((size_t)n_prefix + 1) * sizeof(int4));
  l.prefix = take(n_prefix > 0 && max_prefix > 0 ? tree_parts_workspace_bytes(n_prefix, n_tok, max_prefix) : 0);
  // rows of prefix_own_kernel, or parts of the tensor-core kernel (which a call of fewer sequences may take)
  l.own = take(std::max((size_t)own_rows(n_tok) * kHeads * (kD * sizeof(float) + sizeof(float2)),
                        n_tok >= kOwnTokens ? tree_parts_workspace_bytes(n_seq, n_tok, max_n_kv) : (size_t)0));
  if (max_n_kv > identity_max) {
    const int cells = std::min(max_n_kv, select_max_cells() - 127);
    l.select = take(tree_select_layout(n_seq, n_tok, cells + 127, nullptr, nullptr));
    l.kmax = take((size_t)n_prefix * ((max_prefix + kTreeChunk - 1) / kTreeChunk) * kGroups * kNB * sizeof(float));
  }
  l.bytes = o;
  return l;
}

cudaLaunchConfig_t own_config(int ctas, int S, bool cluster, bool alone, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kOwnThreads);
  cfg.dynamicSmemBytes = alone ? kOwnSmemAlone : kOwnSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cfg;
}

// fit[i]: how many clusters of kSplits[i] CTAs, each on an SM of its own, the device holds at once.
constexpr int kNumSplits = 5, kSplits[kNumSplits + 1] = {8, 6, 4, 3, 2, 1};
cudaError_t own_setup(int (&fit)[kNumSplits]) {
  static std::atomic<int> ready[64], known[64][kNumSplits];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(prefix_own_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kOwnSmemAlone)) != cudaSuccess) return e;
    for (int i = 0; i < kNumSplits; ++i) {
      cudaLaunchAttribute attr[2];
      const cudaLaunchConfig_t cfg = own_config(kSplits[i], kSplits[i], true, true, nullptr, attr);
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, prefix_own_kernel, &cfg)) != cudaSuccess) return e;
      known[dev][i].store(n, std::memory_order_relaxed);
    }
    ready[dev].store(1, std::memory_order_release);
  }
  for (int i = 0; i < kNumSplits; ++i) fit[i] = known[dev][i].load(std::memory_order_relaxed);
  return cudaSuccess;
}

// CTAs of prefix_own_kernel that share a (token, group), over about `cells` cells.  Beside the prefixes' kernel: one for every 512
// cells of the longest, and more of them while the GPU has room.  Alone: the largest cluster with an SM for every CTA of which as
// many fit (and whose warps have a tile each), or for every 512 cells, two on an SM.
cudaError_t own_split(const TreeBatch& b, int cells, bool dense, int* split, bool* alone) {
  int fit[kNumSplits], S = 1;
  const cudaError_t e = own_setup(fit);
  if (e != cudaSuccess) return e;
  *alone = false;
  for (int i = 0; !dense && !*alone && i < kNumSplits; ++i)
    if (cells > kOwnWarps * kTile * kSplits[i + 1] && b.n_tok * kGroups <= fit[i]) {
      S = kSplits[i];
      *alone = true;
    }
  while (2 * S <= kMaxOwn && 2 * S * b.n_tok <= kMostOwn &&
         (cells > 512 * S || (dense && cells > 64 * S && b.n_tok * kGroups * S * 2 <= 152))) {
    S *= 2;
    *alone = false;
  }
  *split = S;
  return e;
}

}  // namespace

size_t prefix_attention_workspace_bytes(int n_prefix, int n_seq, int n_tok, int max_prefix, int max_n_kv, int identity_max) {
  return layout(n_prefix, n_seq, n_tok, max_prefix, max_n_kv, identity_max).bytes;
}

cudaError_t launch_prefix_attention(const TreeBatch& batch, const __half* q, const int8_t* kq, const int8_t* vq, const __half* ksc,
                                    const __half* vsc, int32_t* ids, const __half* gate, __half* out, void* ws, Params p,
                                    int* status, cudaStream_t stream) {
  const Layout l = layout(batch.n_prefix, batch.n_seq, batch.n_tok, batch.max_prefix, batch.max_n_kv, batch.identity_max);
  uint8_t* base = static_cast<uint8_t*>(ws);
  TreeBatch b = batch;
  b.tok = reinterpret_cast<int4*>(base + l.tok);
  TokMore* more = reinterpret_cast<TokMore*>(base + l.more);
  const bool select = b.max_n_kv > b.identity_max;
  // own cells of a sequence, for the shapes of launches (any number gives the same results): what the longest prefix leaves
  const int own_cells = std::max(std::min(b.max_n_kv, 128), b.max_n_kv - b.max_prefix);
  const bool shared = b.n_prefix > 0 && b.max_prefix > 0;
  const bool own_dense = b.n_tok >= (long long)(own_cells > kManyOwnCells ? kOwnTokens : kOwnTokens + 1) * b.n_seq;
  const bool few = shared && !own_dense && (long long)b.n_tok * b.max_prefix <= kFewCells, dense = shared && !few;
  TreeSelect w{};
  int own_chunks = 1;
  if (select) {
    tree_select_layout(b.n_seq, b.n_tok, b.max_n_kv + 127, base + l.select, &w);
    w.kmax_prefix = reinterpret_cast<float*>(base + l.kmax);
    w.chunks_prefix = (b.max_prefix + kTreeChunk - 1) / kTreeChunk;
    own_chunks = (own_cells + kTreeChunk - 1) / kTreeChunk;
    // A few own cells of a token or two cost the top-k kernel less than CTAs of the score kernel (48 tokens of 50-900 own cells 7 us
    // against 11; 40 sequences of 1-16 tokens and 0-400 own cells 12 against 4).
    w.own_in_topk = own_cells <= kOwnInTopk && !own_dense;
  }
  int4* plan = reinterpret_cast<int4*>(base + l.plan);
  int clusters = 0;
  int S = 1;
  bool alone = false;
  cudaError_t e = own_dense ? cudaSuccess : own_split(b, few ? b.max_n_kv : own_cells, dense, &S, &alone);
  if (e != cudaSuccess) return e;
  if (dense) {
    e = own_dense ? prefix_clusters(b, own_cells, 0, &clusters) : prefix_clusters(b, (own_cells + S - 1) / S, b.n_tok * kGroups * S, &clusters);
    if (e != cudaSuccess) return e;
  }
  // No selection, few tokens a sequence, and at most one prefix on the tensor-core kernel: the launches find their way
  // without prefix_prep_kernel (3 us).
  const bool records = !select && !own_dense && (b.n_prefix <= 1 || !dense);
  if (records) {
    plan = nullptr;
  } else {
    const int prep = (select ? kGroups * b.n_tok + b.n_prefix * w.chunks_prefix + b.n_seq * own_chunks : 0) + (b.n_tok + 255) / 256 + dense;
    e = launch_pdl(prefix_prep_kernel, dim3(prep), dim3(256), 0, stream, b, w, more, select, own_chunks, plan, clusters, q, ksc, status);
    if (e != cudaSuccess) return e;
  }
  if (select && (e = launch_shared_select(b, w, own_cells, q, kq, ksc, ids, p, status, stream)) != cudaSuccess) return e;
  const uint32_t* bits = select ? w.bits : nullptr;
  const int pitch = w.pitch / 32;
  JoinArgs j{b, more, {}, {}, plan, clusters, gate, out};
  if (dense && (e = launch_prefix_parts(b, clusters, plan, q, kq, vq, ksc, vsc, bits, pitch, base + l.prefix, p.sm_scale, &j.prefix.p,
                                        status, stream)) != cudaSuccess)
    return e;
  if (own_dense) {
    e = launch_own_parts(b, own_cells, dense, q, kq, vq, ksc, vsc, bits, pitch, base + l.own, p.sm_scale, &j.own.p, status, stream);
    if (e != cudaSuccess) return e;
  } else {
    const bool last = !dense && kHPG * (kD / 8) % S == 0 && S <= kMaxMerge;  // its clusters merge
    float* o = reinterpret_cast<float*>(base + l.own);
    float2* ml = reinterpret_cast<float2*>(o + (size_t)b.n_tok * kHeads * S * kD);
    const OwnArgs a{b, more, dense, few, records, status, q, kq, vq, ksc, vsc, bits, pitch, p.sm_scale * kLog2e, gate, last ? out : nullptr, o, ml};
    cudaLaunchAttribute attr[2];
    const cudaLaunchConfig_t cfg = own_config(b.n_tok * kGroups * S, S, last && S > 1, alone, stream, attr);
    e = cudaLaunchKernelEx(&cfg, prefix_own_kernel, a, S);
    if (e != cudaSuccess || last) return e;
    j.own = PartSet{{reinterpret_cast<const float4*>(o), ml, S, 0}, true};
  }
  auto join = [&](auto kernel, int slices, int threads) {
    return launch_pdl(kernel, dim3((unsigned)(b.n_tok * kGroups * slices)), dim3(threads), 0, stream, j);
  };
  if (b.n_tok >= kJoinMany) return join(prefix_join_kernel<2>, 2, JoinShape<2>::kThreads);
  return join(prefix_join_kernel<8>, 8, JoinShape<8>::kThreads);
}

}  // namespace qsa
