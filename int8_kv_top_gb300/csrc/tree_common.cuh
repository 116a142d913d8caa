// Drafted-token trees: the batch of a qsa_tree_attention call as its kernels see it, and which cells a
// drafted token sees.
#pragma once
#include "common.cuh"

namespace qsa {

struct TreeBatch {
  const int4* seqs;  // per sequence {first pool cell, n_cells, pos0, first token row}
  long long n_pool;
  int n_seq, n_tok;
  const uint32_t* tree;  // [n_tok][tree_words]
  int tree_words, max_n_kv, identity_max;
};

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
};
constexpr int kTreeChunk = 2048;  // cells of a kmax chunk

// A power of two that keeps a row's scores inside fp16: |score| <= sm_scale 128 sum_b kmax_b H_b.
__device__ __forceinline__ float tree_row_scale(const float* eh, const float (&kmax)[kNB], float sm_scale) {
  float h = 0.f;
#pragma unroll
  for (int b = 0; b < kNB; ++b) h = fmaf(kmax[b], eh[kNB + b], h);
  h *= sm_scale * 128.f;
  return h > 32768.f ? exp2f(-ceilf(log2f(h * (1.f / 32768.f)))) : 1.f;
}

// ---------------------------------------------------------------- tile producers
constexpr int kTileCells = 128;  // cells of a tile
constexpr int kTileParts = 4;    // ring stages per tile and operand
constexpr int kTileStages = 4;   // ring depth
constexpr int kTileStageBytes = 16 * 1024;

// What the producers need of a run of tiles.
struct TileRun {
  long long cell0;
  int pos0, T, j_begin, J, g;
  const uint32_t* seen;  // drafted cells that some token of the block sees (bits)
  volatile int* abort;
  int* status;
};

// The K (kV false) or V producers: four warps that turn the tiles' int8 codes into the fp16 operand stages.
// Four lanes take the 64 codes of a (cell, scale block), a warp eight cells a load.  K stage p holds dims
// 64 p .. of the tile's 128 cells, its warps take 8 of every 32 cells; V stage p holds cells 32 p .. of
// the tile, warp w its dims 64 w ...  Row r of a stage lies at 128 r with its 16-byte chunks xored by
// r mod 8, which is the lane's cell, so every store address is a constant past the stage's; two stages are
// in flight in registers while a third is converted.  The loads are not predicated (cells past the sequence
// read its last one): a predicated load is merged with its default as it arrives, and the thread waits
// there for its latency.
//
// kCodes: the codes themselves as fp16 (exact integers) instead of code * scale; the scales are not read.
template <bool kV, bool kCodes>
__device__ __forceinline__ void produce_tiles(const TileRun& t, const int8_t* __restrict__ codes,
                                        const __half* __restrict__ scales, uint32_t ring, uint64_t* full, uint64_t* empty,
                                        int w4, int lane) {
  constexpr int kStep = kV ? 8 : 32;  // cells between a thread's four loads of a stage
  const int sub = lane >> 2, piece = lane & 3, r0 = sub + (kV ? 0 : w4 * 8);
  const int n_scan = t.pos0 + t.T, n_st = t.J * kTileParts;
  const size_t row0 = (size_t)t.cell0 * kGroups + t.g;
  const int8_t* my_codes = codes + row0 * kD + piece * 16 + (kV ? w4 * kBlk : 0);
  const uint16_t* my_scales = reinterpret_cast<const uint16_t*>(scales) + row0 * kNB + (kV ? w4 : 0);
  const uint32_t dst0 = ring + (kV ? w4 * 4096 : 0) + r0 * 128 + (((2 * piece) ^ sub) << 4);
  const uint32_t dst1 = ring + (kV ? w4 * 4096 : 0) + r0 * 128 + (((2 * piece + 1) ^ sub) << 4);
  auto load = [&](int s, uint4 (&w)[4], uint16_t (&sc)[4]) {
    const int part = s & 3, c0 = (t.j_begin + (s >> 2)) * kTileCells + r0 + (kV ? part * 32 : 0);
    const int8_t* cp = my_codes + (kV ? 0 : part * kBlk);
    const uint16_t* sp = my_scales + (kV ? 0 : part);
    if ((t.j_begin + (s >> 2) + 1) * kTileCells <= n_scan) {
      cp += (size_t)c0 * (kGroups * kD);
      sp += (size_t)c0 * (kGroups * kNB);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w[i] = __ldg(reinterpret_cast<const uint4*>(cp + i * kStep * (kGroups * kD)));
        if (!kCodes) sc[i] = __ldg(sp + i * kStep * (kGroups * kNB));
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const size_t cell = min(c0 + i * kStep, n_scan - 1);
        w[i] = __ldg(reinterpret_cast<const uint4*>(cp + cell * (kGroups * kD)));
        if (!kCodes) sc[i] = __ldg(sp + cell * (kGroups * kNB));
      }
    }
  };
  auto store = [&](int s, const uint4 (&w)[4], uint16_t (&sc)[4]) -> bool {
    const int slot = s % kTileStages, tile = t.j_begin + (s >> 2);
    if (s >= kTileStages && !mbar_wait_warp(&empty[slot], ((s / kTileStages) & 1) ^ 1, t.status, t.abort)) return false;
    if (!kCodes && (tile + 1) * kTileCells > t.pos0) {  // cells past the sequence, and drafted ones that nobody here sees: zeros
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int dj = tile * kTileCells + r0 + (kV ? (s & 3) * 32 : 0) + i * kStep - t.pos0;
        if (dj >= 0 && (dj >= t.T || !((t.seen[dj >> 5] >> (dj & 31)) & 1u))) sc[i] = 0;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t lo[4], hi[4];
      const __half2 s2 = __half2half2(__ushort_as_half(kCodes ? (uint16_t)0x3C00 : sc[i]));
      dequant8(w[i].x, w[i].y, s2, lo);
      dequant8(w[i].z, w[i].w, s2, hi);
      const uint32_t at = slot * kTileStageBytes + i * kStep * 128;
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + at), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                   : "memory");
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst1 + at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                   : "memory");
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&full[slot]);
    return true;
  };
  if (n_st == 0) return;
  uint4 wa[4], wb[4];
  uint16_t sa[4] = {}, sb[4] = {};
  load(0, wa, sa);
  load(1, wb, sb);
  for (int s = 0; s < n_st; s += 2) {  // n_st is a multiple of kTileParts
    if (!store(s, wa, sa)) break;
    if (s + 2 < n_st) load(s + 2, wa, sa);
    if (!store(s + 1, wb, sb)) break;
    if (s + 3 < n_st) load(s + 3, wb, sb);
  }
}

}  // namespace qsa
