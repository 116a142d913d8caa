// Selection for drafted token trees: the exact top-k cells of every selected token (n_kv > identity_max) of a
// qsa_tree_attention call, the tokens of a sequence sharing one read of its K codes.
//
// As in select.cu the score of cell c for token t and group g is sm_scale sum_b ksc_b S_b with S_b = the dot
// product of a 64-dim block of the group's summed queries Qsum (hi + lo fp16 split) and the int8 codes, formed
// per scale block on the tensor cores with products exact in fp32; topk_kernel (select.cu) then proves the
// order from the error bound and re-ranks the undecided band with exact integer keys.  Three launches:
//
//  1. tree_prep   Qsum = hi + lo + residual of every selected (token, group) with its error terms, and the
//                 largest |ksc| of every 2,048 cells (bounds; only cells that some token sees count).
//  2. tree_score  the tree's tokens are few and the cells many, so the operands are swapped: M = 128 cells
//                 (A = the codes as fp16, made from int8 by producer warps as in tree.cu), N = the hi rows and
//                 behind them the lo rows of up to 32 tokens, one TMEM accumulator per scale block.  An epilogue
//                 thread owns a cell, so its four K scales are in registers.  Cells that a token does not see
//                 score -inf.  A tile's 16 MMAs take about 100 cycles each, whatever N (A's 4 KB come from shared
//                 memory); hi and lo in one N instead of two MMAs each halves their number.
//  3. topk_kernel<V, true>.
//
// 24 trees of 1-32 tokens after 200-16,000 cells (414 tokens): prep 14, score 47, top-k 54, the attention 145 us, each
// launched alone from a cold L2 (243 us as the call runs).  The score reads 88 MB; by a clock trace a tile takes
// 2,400 cycles, 1,900 of them the issue of its MMAs, the rest between tiles; neither memory nor arithmetic (tensor 7%)
// bounds it.  Two teams of producers and an epilogue that read each token's scale as it stored: 247 us.
#include "select_math.cuh"
#include "tree_common.cuh"

namespace qsa {
namespace {

constexpr int kTokChunk = 32;  // tokens per score CTA: UMMA N is at most twice that

// ---------------------------------------------------------------- 1. prep
// Blocks [0, 2 n_tok): (token row, group), thread = dim.  Blocks behind them: (sequence, chunk of cells); then, where
// a plan is wanted, one that lists the attention's blocks.
__global__ void __launch_bounds__(256) tree_prep_kernel(const TreeBatch b, const TreeSelect w,
                                                        const __half* __restrict__ q, const __half* __restrict__ ksc,
                                                        int4* __restrict__ plan) {
  __shared__ long long s_e[8], s_h[8];
  __shared__ uint32_t s_union[kTreeWords];
  __shared__ float s_max[8][kGroups * kNB];
  pdl_begin();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int x = blockIdx.x;
  if (x < kGroups * b.n_tok) {
    const int t = x >> 1, g = x & 1;
    const int s = warp_find_seq(b.n_seq, t, [&](int i) { return (long long)__ldg(&b.seqs[i].w); });
    int4 e4;
    const int T = tree_seq_tokens(b, s, &e4);
    if (T <= 0 || t < e4.w || t >= e4.w + T) return;  // uniform over the block, as the next
    int seen = e4.z;
    for (int i = 0; i < b.tree_words; ++i) seen += __popc(tree_mask_word(b, t, i, T));
    if (seen <= b.identity_max) return;
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
  if (x == b.n_seq * w.chunks) {
    static_assert(kPlanThreads == 256, "this kernel's block");
    tree_plan_blocks(b, true, plan, tree_blocks_most(b.n_seq, b.n_tok));
    return;
  }
  const int s = x / w.chunks, ch = x % w.chunks;
  int4 e4;
  const int T = tree_seq_tokens(b, s, &e4);
  const int pos0 = e4.z, n_scan = pos0 + T, c0 = ch * kTreeChunk, c1 = min(c0 + kTreeChunk, n_scan);
  if (T <= 0 || n_scan <= b.identity_max || c0 >= c1) return;
  if (tid < kTreeWords) s_union[tid] = 0u;
  __syncthreads();
  if (c1 > pos0)
    for (int i = tid; i < T * kTreeWords; i += 256) {
      const uint32_t m = tree_mask_word(b, e4.w + (i >> 3), i & 7, T);
      if (m) atomicOr(&s_union[i & 7], m);
    }
  static_assert(kTreeWords == 8, "mask words by i mod 8");
  __syncthreads();
  float mx[kGroups * kNB];
#pragma unroll
  for (int i = 0; i < kGroups * kNB; ++i) mx[i] = 0.f;
  for (int c = c0 + tid; c < c1; c += 256) {
    const int dj = c - pos0;
    if (dj >= 0 && !((s_union[dj >> 5] >> (dj & 31)) & 1u)) continue;
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(ksc + ((size_t)e4.x + c) * (kGroups * kNB)));
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
      mx[2 * i] = fmaxf(mx[2 * i], fabsf(f.x));
      mx[2 * i + 1] = fmaxf(mx[2 * i + 1], fabsf(f.y));
    }
  }
#pragma unroll
  for (int i = 0; i < kGroups * kNB; ++i) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], o));
    if (lane == 0) s_max[warp][i] = mx[i];
  }
  __syncthreads();
  if (tid < kGroups * kNB) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, s_max[i][tid]);
    w.kmax[(size_t)x * (kGroups * kNB) + tid] = m;
  }
}

// ---------------------------------------------------------------- 2. score
constexpr int kTeams = 4;            // of producers, four warps each: a stage of every tile each
constexpr int kEpiWarp = 4 * kTeams, kMmaWarp = kEpiWarp + 8;  // epilogue (16 tokens each half of it), then MMA
constexpr int kScoreThreads = (kMmaWarp + 1) * 32;
constexpr int kOffB = kTileStages * kTileStageBytes;  // 4 dim blocks of [hi rows, lo rows][64] SW128
constexpr int kBBlock = 2 * kTokChunk * 128;
constexpr int kScoreSmem = kOffB + kNB * kBBlock + 1024;

struct __align__(8) TreeScoreBars {
  uint64_t full[kTileStages], empty[kTileStages], acc_full[2], acc_empty[2], b_full, tmem_ready, drain;
};

// First token chunk of a sequence: as first_block in tree.cu, for chunks of 32 tokens.
__device__ __forceinline__ long long first_chunk(long long first_row, int s) { return first_row / kTokChunk + s; }

__global__ void __launch_bounds__(kScoreThreads, 1)
    tree_score_kernel(const TreeBatch b, const TreeSelect w, const int8_t* __restrict__ kq,
                      const __half* __restrict__ ksc, int tiles_per_cta, float sm_scale, int* status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ TreeScoreBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ uint32_t s_mask[kTokChunk][kTreeWords];
  __shared__ __align__(16) float s_scale[kTokChunk];  // sm_scale x the row's power of two; 0: not a selected token
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = blockIdx.y;
  pdl_begin();
  const int sq = warp_find_seq(b.n_seq, blockIdx.z, [&](int i) { return first_chunk(__ldg(&b.seqs[i].w), i); });
  int4 e4;
  const int T = tree_seq_tokens(b, sq, &e4);
  const long long kc = (long long)blockIdx.z - first_chunk(e4.w, sq);
  const int pos0 = e4.z, n_scan = pos0 + T;
  const int j_begin = blockIdx.x * tiles_per_cta;
  const int J = min(tiles_per_cta, (n_scan + kTileCells - 1) / kTileCells - j_begin);
  if (T <= 0 || kc < 0 || kc * kTokChunk >= T || J <= 0 || n_scan <= b.identity_max) return;  // uniform
  const int t0 = e4.w + (int)kc * kTokChunk;  // first token row
  const int n_here = min(kTokChunk, T - (int)kc * kTokChunk);
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&bars.full[i], 4);
      mbar_init(&bars.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.acc_full[i], 1);
      mbar_init(&bars.acc_empty[i], 8);
    }
    mbar_init(&bars.b_full, 8);
    mbar_init(&bars.tmem_ready, 1);
    mbar_init(&bars.drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  const int n16 = (n_here + 15) / 16 * 16, N = 2 * n16;  // row n: hi of token n; row n16 + n: lo

  if (warp < kEpiWarp) {
    const TileRun t{e4.x, pos0, T, j_begin, J, g, nullptr, &s_abort, status, 0};
    produce_tiles<kScoreCodes, kTeams>(t, kq, nullptr, smem_u32(smem), bars.full, bars.empty, warp & 3, lane, warp >> 2);
  } else if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars.tmem_ready);
      tc_fence_after();
      const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&s_tmem);
      const uint32_t idesc = idesc_f16_f32(kTileCells, N, 0, 0);
      const uint64_t bdesc = sdesc_sw128(smem_u32(smem + kOffB), 16, 1024);
      bool go = mbar_wait_poll<false>(&bars.b_full, 0, status, &s_abort);
      for (int j = 0; go && j < J; ++j) {
        const int buf = j & 1;
        if (j >= 2 && !mbar_wait_poll<false>(&bars.acc_empty[buf], ((j >> 1) - 1) & 1, status, &s_abort)) break;
        for (int d = 0; go && d < kNB; ++d) {
          const int st = j * kNB + d, slot = st % kTileStages;
          go = mbar_wait_poll<false>(&bars.full[slot], (st / kTileStages) & 1, status, &s_abort);
          if (!go) break;
          tc_fence_after();
          const uint64_t adesc = sdesc_sw128(smem_u32(smem) + slot * kTileStageBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(tmem + buf * 256 + d * (2 * kTokChunk), adesc + (uint64_t)((kk * 32) >> 4),
                    bdesc + (uint64_t)((d * kBBlock + kk * 32) >> 4), idesc, kk > 0 ? 1u : 0u);
          umma_commit(&bars.empty[slot]);
        }
        if (go) umma_commit(&bars.acc_full[buf]);
      }
      umma_commit(&bars.drain);
      mbar_wait(&bars.drain, 0, status);
    }
    __syncwarp();
  } else {
    const int et = tid - 32 * kEpiWarp, quarter = warp & 3, n0 = 16 * ((warp - kEpiWarp) >> 2);  // this warp's cells and tokens
    {
      // 16-byte chunk c of token r's hi | lo row: four rows' loads before any store.  Rows of tokens that do not
      // select were not written by tree_prep: what they hold only reaches their own scores, which are not stored.
      const int c = et & 63, d = c >> 4;
      uint4 v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (et >> 6) + 4 * i;
        v[i] = make_uint4(0u, 0u, 0u, 0u);
        if (r < n_here) v[i] = __ldg(reinterpret_cast<const uint4*>(w.qhl + (size_t)(g * b.n_tok + t0 + r) * (2 * kD)) + c);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = (et >> 6) + 4 * i, row = r + (c & 8 ? n16 : 0);
        if (r < n16) *reinterpret_cast<uint4*>(smem + kOffB + d * kBBlock + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[i];
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.b_full);
    if (warp == kEpiWarp) {  // lane = token: its mask and what its scores are multiplied by
      float km[kNB];
      warp_kmax(w, sq, g, n_scan, lane, km);
      int seen = pos0;
#pragma unroll
      for (int i = 0; i < kTreeWords; ++i) {
        const uint32_t m = lane < n_here ? tree_mask_word(b, t0 + lane, i, T) : 0u;
        s_mask[lane][i] = m;
        seen += __popc(m);
      }
      s_scale[lane] = lane < n_here && seen > b.identity_max
                          ? sm_scale * tree_row_scale(w.eh + (size_t)(g * b.n_tok + t0 + lane) * 8, km, sm_scale)
                          : 0.f;
    }
    const bool t_ok = tile_wait_warp(&bars.tmem_ready, 0, status, &s_abort);
    tc_fence_after();
    named_bar_any(1, 256, false);  // masks and scales are in shared memory
    const uint32_t lane_base = *reinterpret_cast<volatile uint32_t*>(&s_tmem) + ((uint32_t)(quarter * 32) << 16) + n0;
    auto scales_of = [&](int j) {  // this thread's cell: the four K scales of the group
      const size_t c = min((j_begin + j) * kTileCells + quarter * 32 + lane, n_scan - 1);
      return __ldg(reinterpret_cast<const uint2*>(ksc + ((size_t)e4.x + c) * (kGroups * kNB) + g * kNB));
    };
    uint2 sw_next = scales_of(0);
    __half* dst0 = w.scores + (size_t)(g * b.n_tok + t0 + n0) * w.pitch;
    for (int j = 0; t_ok && j < J; ++j) {
      const int buf = j & 1, cell = (j_begin + j) * kTileCells + quarter * 32 + lane, dj = cell - pos0;
      const uint2 sw = sw_next;
      if (j + 1 < J) sw_next = scales_of(j + 1);
      const float2 s01 = __half22float2(*reinterpret_cast<const __half2*>(&sw.x));
      const float2 s23 = __half22float2(*reinterpret_cast<const __half2*>(&sw.y));
      if (!tile_wait_warp(&bars.acc_full[buf], (j >> 1) & 1, status, &s_abort)) break;
      tc_fence_after();
      float acc[16];
      if (n0 < n16) {
#pragma unroll
        for (int d = 0; d < kNB; ++d) {
          uint32_t hi[16], lo[16];
          const uint32_t at = lane_base + buf * 256 + d * (2 * kTokChunk);
          tmem_ld16(at, hi);
          tmem_ld16(at + n16, lo);
          tmem_wait_ld();
          const float sd = d == 0 ? s01.x : d == 1 ? s01.y : d == 2 ? s23.x : s23.y;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(hi[i]) + __uint_as_float(lo[i]);
            acc[i] = d == 0 ? sd * x : fmaf(sd, x, acc[i]);
          }
        }
      }
      tc_fence_before();  // the accumulators are in registers
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.acc_empty[buf]);
      if (n0 >= n16 || cell >= n_scan) continue;
      __half* dst = dst0 + cell;
      const bool drafted = (j_begin + j + 1) * kTileCells > pos0;
      const float4* sc4 = reinterpret_cast<const float4*>(s_scale + n0);
      float sc[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 x = sc4[i];
        sc[4 * i] = x.x;
        sc[4 * i + 1] = x.y;
        sc[4 * i + 2] = x.z;
        sc[4 * i + 3] = x.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[i] *= sc[i];
      if (drafted && dj >= 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (!((s_mask[n0 + i][dj >> 5] >> (dj & 31)) & 1u)) acc[i] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (sc[i] != 0.f) *dst = __float2half_rn(acc[i]);  // the same for the whole warp
        dst += w.pitch;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(&s_tmem), 512);
}

}  // namespace

size_t tree_select_layout(int n_seq, int n_tok, int max_n_kv, void* ws, TreeSelect* out) {
  TreeSelect w{};
  w.pitch = (max_n_kv + 255) / 256 * 256;
  w.chunks = (max_n_kv + kTreeChunk - 1) / kTreeChunk;
  const size_t rows = (size_t)kGroups * n_tok;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return static_cast<uint8_t*>(ws) + at;
  };
  w.qhl = reinterpret_cast<__half*>(take(rows * 2 * kD * sizeof(__half)));
  w.eh = reinterpret_cast<float*>(take(rows * 8 * sizeof(float)));
  w.kmax = reinterpret_cast<float*>(take((size_t)n_seq * w.chunks * kGroups * kNB * sizeof(float)));
  w.scores = reinterpret_cast<__half*>(take(rows * w.pitch * sizeof(__half)));
  w.bits = reinterpret_cast<uint32_t*>(take(rows * (w.pitch / 8)));
  if (out) *out = w;
  return o;
}

cudaError_t launch_tree_select(const TreeBatch& b, const TreeSelect& w, const __half* q, const int8_t* kq,
                               const __half* ksc, int32_t* ids, int4* plan, Params p, int* status, cudaStream_t stream) {
  cudaError_t e = launch_pdl(tree_prep_kernel, dim3(kGroups * b.n_tok + b.n_seq * w.chunks + (plan ? 1 : 0)), dim3(256), 0,
                             stream, b, w, q, ksc, plan);
  if (e != cudaSuccess) return e;
  if ((e = cudaFuncSetAttribute(tree_score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kScoreSmem)) !=
      cudaSuccess)
    return e;
  // tiles per CTA: as few as keep the CTAs near two waves of one per SM (a CTA's set-up, its B rows above all,
  // costs about as much as three tiles); ragged batches leave about half of the grid empty
  const int tiles = (b.max_n_kv + kTileCells - 1) / kTileCells;
  const int zb = b.n_tok / kTokChunk + b.n_seq;
  int per = 2;
  while (per < 8 && (long long)((tiles + per - 1) / per) * kGroups * zb > 304) per *= 2;
  e = launch_pdl(tree_score_kernel, dim3((tiles + per - 1) / per, kGroups, zb), dim3(kScoreThreads), kScoreSmem, stream, b,
                 w, kq, ksc, per, p.sm_scale, status);
  if (e != cudaSuccess) return e;
  return launch_tree_topk(b, w, q, kq, ksc, ids, p, status, stream);
}

}  // namespace qsa
