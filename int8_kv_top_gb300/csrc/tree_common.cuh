// Drafted-token trees: the batch of a qsa_tree_attention call as its kernels see it, and which cells a
// drafted token sees.
#pragma once
#include "common.cuh"
#include "tree_plan.cuh"
#include "tree_tables.cuh"

namespace qsa {

// The two halves of a cluster barrier, executed by every thread of the cluster once per phase.
__device__ __forceinline__ void cluster_arrive_all() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait_all() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// The last sequence whose key(s) is not above `at`, by a whole warp (32 probes a step); key is increasing and
// key(0) is at most `at` in a valid table (else some sequence, whose entry the caller checks).
template <class Key>
__device__ __forceinline__ int warp_find_seq(int n_seq, long long at, Key key) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = n_seq;
  while (n > 1) {
    const int step = (n + 31) / 32, s = lo + lane * step;
    const bool le = lane * step < n && key(s) <= at;
    const int c = max(__popc(__ballot_sync(0xffffffffu, le)), 1);
    n = min(step, n - (c - 1) * step);
    lo += (c - 1) * step;
  }
  return lo;
}

// Selection of many tree tokens at once (tree_select.cu, and the top-k of select.cu): workspace pointers and
// strides.  Rows are (group, token row); pitches are in cells.
struct TreeSelect {
  __half* qhl;       // [2][n_tok][512]: per 64-dim block hi (64) | lo (64) of the group's summed queries
  float* eh;         // [2][n_tok][8]: E_b, H_b (the score's error terms)
  float* kmax;       // [n_seq][chunks][8]: max |ksc| per (group, block) over a chunk's visible cells
  __half* scores;    // [2][n_tok][pitch]
  uint32_t* bits;    // [2][n_tok][pitch / 32]: the selected cells
  int pitch, chunks;
  float* kmax_prefix;  // shared calls: [n_prefix][chunks_prefix][8], likewise; kmax then counts the own cells
  int chunks_prefix;
  bool own_in_topk;    // shared calls: the top-k kernel scores the own cells itself
};
constexpr int kTreeChunk = 2048;  // cells of a kmax chunk

// max |ksc| per scale block of group g over the cells of sequence s (n_scan of them), by a whole warp: every lane
// loads a chunk's maxima at once (32 chunks are the 65,536 cells that the score path holds).
__device__ __forceinline__ void warp_kmax(const TreeSelect& w, int s, int g, int n_scan, int lane, float (&km)[kNB]) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (lane * kTreeChunk < n_scan)
    v = __ldg(reinterpret_cast<const float4*>(w.kmax + ((size_t)s * w.chunks + lane) * (kGroups * kNB) + g * kNB));
  km[0] = v.x;
  km[1] = v.y;
  km[2] = v.z;
  km[3] = v.w;
#pragma unroll
  for (int b = 0; b < kNB; ++b)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) km[b] = fmaxf(km[b], __shfl_xor_sync(0xffffffffu, km[b], o));
}

// The same by one thread, raising km (own cells of a shared call's sequence: a few chunks).
__device__ __forceinline__ void raise_kmax(const float* kmax, int i, int chunks, int g, int n_scan, float (&km)[kNB]) {
  for (int c = 0; c * kTreeChunk < n_scan; ++c) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(kmax + ((size_t)i * chunks + c) * (kGroups * kNB) + g * kNB));
    km[0] = fmaxf(km[0], v.x);
    km[1] = fmaxf(km[1], v.y);
    km[2] = fmaxf(km[2], v.z);
    km[3] = fmaxf(km[3], v.w);
  }
}

// Of a shared call's token (its record, and its sequence's own cells), by a whole warp.
__device__ __forceinline__ void shared_kmax(const TreeBatch& b, const TreeSelect& w, const int4& tok, int n_own, int g, int lane,
                                            float (&km)[kNB]) {
  if (tok.w >= 0) {
    TreeSelect v = w;
    v.kmax = w.kmax_prefix;
    v.chunks = w.chunks_prefix;
    warp_kmax(v, tok.w, g, tok.z, lane, km);
  }
  raise_kmax(w.kmax, tok.x, w.chunks, g, n_own, km);
}

// D += A B for 16 x 8 x 16 fp16 tiles with fp32 sums, by a warp.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A power of two that keeps a row's scores inside fp16: |score| <= sm_scale 128 sum_b kmax_b H_b.
__device__ __forceinline__ float tree_row_scale(const float* eh, const float (&kmax)[kNB], float sm_scale) {
  float h = 0.f;
#pragma unroll
  for (int b = 0; b < kNB; ++b) h = fmaf(kmax[b], eh[kNB + b], h);
  h *= sm_scale * 128.f;
  return h > 32768.f ? exp2f(-ceilf(log2f(h * (1.f / 32768.f)))) : 1.f;
}

// ---------------------------------------------------------------- blocks of an attention launch
constexpr int kPlanSeqs = 8;       // sequences from which on a launch takes its blocks from a list, longest first
constexpr int kPlanThreads = 256;

// The list, by one CTA of kPlanThreads: plan[0].x blocks, then for block i plan[1 + 2 i] = {first pool cell,
// committed cells, drafted tokens, first token row} of its sequence and plan[2 + 2 i].x = its first row, in decreasing
// order of tiles (a counting sort), so that the long blocks of a ragged batch start first and the short ones
// fill the gaps (24 trees after 200-16,000 cells: attention 213 -> 159 us when it was added).  Blocks of equal length come in
// any order, which no result depends on.  A table whose rows overlap (its bad entries are flagged elsewhere) may
// name more blocks than the list holds: those past `cap` are dropped.
__device__ __forceinline__ void tree_plan_blocks(const TreeBatch& b, bool with_selected, int4* __restrict__ plan, int cap) {
  constexpr int kBins = 1024, kPer = kBins / kPlanThreads;  // tiles 1 .. 1024 (131,072 cells)
  __shared__ int s_bin[kBins], s_sum[kPlanThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int4 e;
  int T = 0;
  auto blocks_of = [&](int s, int* bin) {
    T = tree_seq_tokens(b, s, &e);
    if (T <= 0 || (!with_selected && e.z > b.identity_max)) return 0;  // all of its tokens select
    *bin = min((e.z + T + kTileCells - 1) / kTileCells, kBins) - 1;
    return (T * kHPG + kTreeBlock - 1) / kTreeBlock;
  };
  for (int i = tid; i < kBins; i += kPlanThreads) s_bin[i] = 0;
  __syncthreads();
  for (int s = tid; s < b.n_seq; s += kPlanThreads) {
    int bin = 0;
    const int n = blocks_of(s, &bin);
    if (n) atomicAdd(&s_bin[bin], n);
  }
  __syncthreads();
  int v[kPer], sum = 0;  // exclusive scan from the last bin down: thread i takes bins kBins - 1 - kPer i ..
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    v[u] = s_bin[kBins - 1 - kPer * tid - u];
    sum += v[u];
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int at = x - sum;
  for (int i = 0; i < warp; ++i) at += s_sum[i];
  if (tid == kPlanThreads - 1) plan[0] = make_int4(at + sum, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    s_bin[kBins - 1 - kPer * tid - u] = at;
    at += v[u];
  }
  __syncthreads();
  for (int s = tid; s < b.n_seq; s += kPlanThreads) {
    int bin = 0;
    const int n = blocks_of(s, &bin);
    for (int k = 0; k < n; ++k) {
      const int pos = atomicAdd(&s_bin[bin], 1);
      if (pos < cap) {
        plan[1 + 2 * pos] = make_int4(e.x, e.z, T, e.w);
        plan[2 + 2 * pos] = make_int4(k * kTreeBlock, 0, 0, 0);
      }
    }
  }
}

// Eight dims of an output row: the gate's sigmoid, and the rounding to fp16.
__device__ __forceinline__ void apply_gate(float (&v)[8], uint4 gw) {
  const uint32_t w[4] = {gw.x, gw.y, gw.z, gw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    v[2 * i] *= gate_sigmoid(f.x);
    v[2 * i + 1] *= gate_sigmoid(f.y);
  }
}
__device__ __forceinline__ uint4 pack_out(const float (&v)[8]) {
  return make_uint4(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]), pack_half2(v[4], v[5]), pack_half2(v[6], v[7]));
}

// ---------------------------------------------------------------- waits
// Bounded waits in few instructions: the roles of a kernel run different loops at the same time, and their
// code has to fit the SM's instruction cache together.  A failed probe suspends the thread for up to
// kSuspendHintNs, so kWaitProbes of them take at most about two seconds.
constexpr int kWaitProbes = 1000000;
__device__ __forceinline__ bool tile_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
#pragma unroll 1
  for (int it = 0; it < kWaitProbes; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort) return false;
  }
  set_dev_status(status, QSA_DEV_WAIT_TIMEOUT);
  *abort = 1;
  return false;
}
__device__ __forceinline__ bool tile_wait_warp(uint64_t* bar, uint32_t parity, int* status, volatile int* abort) {
  return __all_sync(0xffffffffu, tile_wait(bar, parity, status, abort));
}

// ---------------------------------------------------------------- tile producers
constexpr int kTileStages = 4;   // ring depth
constexpr int kTileStageBytes = 16 * 1024;

// What the producers need of a run of tiles.
struct TileRun {
  long long cell0;
  int pos0, T, j_begin, J, g;
  const uint32_t* seen;  // drafted cells that some token of the block sees (bits)
  volatile int* abort;
  int* status;
  int half;              // rank within a CTA pair: which half of the tile's K cells and of V's dims is ours
};

// Four producer warps that turn the tiles' int8 codes into fp16 operand stages of 16 KB, 128B-swizzled:
//   kScoreCodes  stage p: 128 cells x dims 64 p .. (four a tile); the codes themselves, exact integers
//   kPair        K stage p: this CTA's 64 cells x dims 128 p .. (two a tile), code * scale;
//                V stage p (is_v): cells 64 p .. of the tile x this CTA's 128 dims (two a tile).  One body serves
//                both: the kernel's roles share the SM's instruction cache (see tree.cu)
// Four lanes take the 64 codes of a (cell, scale block), a warp eight cells a load, so row r of a stage lies at
// 128 r with its 16-byte chunks xored by r mod 8, which is the lane's cell: every store address is a constant
// past the stage's.  Two stages are in flight in registers while a third is converted (kTeams
// teams of four warps take the stages in turn).  The loads are not
// predicated (cells past the sequence read its last one): a predicated load is merged with its default as
// it arrives, and the thread waits there for its latency.
enum TileMode { kScoreCodes, kPair };
template <TileMode kMode, int kTeams = 1>
__device__ __forceinline__ void produce_tiles(const TileRun& t, const int8_t* __restrict__ codes,
                                              const __half* __restrict__ scales, uint32_t ring, uint64_t* full,
                                              uint64_t* empty, int w4, int lane, int team = 0, bool is_v = false) {
  constexpr bool kScaled = kMode == kPair;
  constexpr int kParts = kScaled ? 2 : 4;   // stages a tile
  constexpr int kStep = kScaled ? 8 : 32;   // cells between a thread's four loads of a stage
  const int sub = lane >> 2, piece = lane & 3;
  const int db = kScaled ? w4 & 1 : 0;      // dim block within the stage
  const int r0 = sub + (kScaled ? (w4 >> 1) * 32 : w4 * 8);
  const int n_scan = t.pos0 + t.T, n_st = t.J * kParts;
  const size_t row0 = (size_t)t.cell0 * kGroups + t.g;
  const int8_t* my_codes = codes + row0 * kD + piece * 16;
  const uint16_t* my_scales = reinterpret_cast<const uint16_t*>(scales) + row0 * kNB;
  const uint32_t dst0 = ring + db * (kTileStageBytes / 2) + r0 * 128 + (((2 * piece) ^ sub) << 4);
  const uint32_t dst1 = ring + db * (kTileStageBytes / 2) + r0 * 128 + (((2 * piece + 1) ^ sub) << 4);
  auto first_cell = [&](int tile, int part) {  // the thread's first cell of a stage
    return tile * kTileCells + r0 + (kScaled ? (is_v ? part : t.half) * 64 : 0);
  };
  auto load = [&](int s, uint4 (&w)[4], uint16_t (&sc)[4]) {
    const int tile = t.j_begin + s / kParts, part = s % kParts, c0 = first_cell(tile, part);
    const int blk = !kScaled ? part : 2 * (is_v ? t.half : part) + db;
    const int past = n_scan - 1 - c0;  // the sequence's last cell, from the thread's first
    const int8_t* cp = my_codes + blk * kBlk + (int64_t)c0 * (kGroups * kD);
    const uint16_t* sp = my_scales + blk + (int64_t)c0 * (kGroups * kNB);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = min(i * kStep, past);
      w[i] = __ldg(reinterpret_cast<const uint4*>(cp + c * (kGroups * kD)));
      if (kScaled) sc[i] = __ldg(sp + c * (kGroups * kNB));
    }
  };
  auto store = [&](int s, const uint4 (&w)[4], uint16_t (&sc)[4]) -> bool {
    const int slot = s % kTileStages, tile = t.j_begin + s / kParts;
    if (s >= kTileStages && !tile_wait_warp(&empty[slot], ((s / kTileStages) & 1) ^ 1, t.status, t.abort)) return false;
    if (kScaled && (tile + 1) * kTileCells > t.pos0) {  // cells past the sequence, and drafted ones unseen here: zeros
      const int c0 = first_cell(tile, s % kParts);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int dj = c0 + i * kStep - t.pos0;
        if (dj >= 0 && (dj >= t.T || !((t.seen[dj >> 5] >> (dj & 31)) & 1u))) sc[i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo[4], hi[4];
      const __half2 s2 = __half2half2(__ushort_as_half(kScaled ? sc[i] : (uint16_t)0x3C00));
      dequant8(w[i].x, w[i].y, s2, lo);
      dequant8(w[i].z, w[i].w, s2, hi);
      const uint32_t at = slot * kTileStageBytes + i * kStep * 128;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + at), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst1 + at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                   : "memory");
    }
    fence_proxy_async_smem();  // this thread's part is visible to the tensor core before the arrive
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[slot]);  // of this CTA: rank 1 of a pair has its phases forwarded to rank 0
    return true;
  };
  if (n_st == 0) return;
  uint4 wa[4], wb[4];
  uint16_t sa[4] = {}, sb[4] = {};
  load(team, wa, sa);
  load(team + kTeams, wb, sb);
  for (int s = team; s < n_st; s += 2 * kTeams) {  // n_st is a multiple of kParts
    if (!store(s, wa, sa)) break;
    if (s + 2 * kTeams < n_st) load(s + 2 * kTeams, wa, sa);
    if ((kParts % (2 * kTeams) && s + kTeams >= n_st) || !store(s + kTeams, wb, sb)) break;
    if (s + 3 * kTeams < n_st) load(s + 3 * kTeams, wb, sb);
  }
}

}  // namespace qsa
