// qsa_tree_attention, identity tokens (n_kv <= identity_max): attention of drafted token trees over
// every cell that they see, on the tcgen05 tensor cores straight from the int8 cache.
//
//   out[t,h,:] = sum_c softmax_c(sm_scale q[t,h,:] . k^[c]) v^[c],  c over the committed cells and the
//   drafted cells of token t's mask;  k^ = fp16(kq * ksc), v^ = fp16(vq * vsc).
//
// All of a tree's tokens read the same committed cells and the 12 heads of a group share their K/V, so
// the (token, head) rows of a sequence and group, packed 12 a token, are cut into blocks of 128 rows (the
// M of one MMA): a tree of 32 tokens is exactly three blocks.  A cluster of C CTAs takes one block, each
// CTA a run of its 128-cell tiles, and the CTAs merge by log-sum-exp through distributed shared memory in
// a fixed order, so that a call of few rows still spreads over the GPU and results do not depend on timing.
//
// The cache is read as int8 once per block and dequantised by producer warps into the 128B-swizzled
// operand tiles; no fp16 mirror is written (a drafting step reads a cache a few times, and the mirror
// would cost three times the cache's own bytes).  Per 128-cell tile an SM does 2 x 128 x 128 x 256
// multiply-adds (about 2,050 cycles at the tensor pipe's rate), reads 64 KB of codes and writes 128 KB of
// fp16 operands.
//
//   warps 0-3    K producers: stage = 64 dims of the tile's 128 cells (16 KB), ring of four
//   warps 4-7    V producers: stage = 32 cells x 256 dims (16 KB), ring of four
//   warps 8-15   load Q; two softmax warpgroups, one row per thread in each, half of the columns each:
//                mask, online softmax in base-2 units (running maximum and sum in fp32), P as fp16 into
//                TMEM over S, lazy O rescale (only when the maximum grows by more than 2^8)
//   warp 16      TMEM, MMA issue in the order QK(0), QK(1), PV(0), QK(2), PV(1), ...
//                  S = Q K^T  (A = Q K-major, B = K^ K-major)      M=128 N=128, 16 K-steps
//                  O += P V^  (A = P from TMEM, B = V^ MN-major)   M=128 N=256, 8 K-steps
//
// Roundings below fp32: k^ and v^ (the values the library's prefill attends to), P (at most 2^8 after the
// lazy rescale, so fp16 holds it with 11 bits), and the output; statistics and sums are fp32.
//
// TMEM columns: O [0, 256), S/P buffers [256 + 128 b, 384 + 128 b), b = 0, 1.
// Every mbarrier wait is bounded; after a timeout the CTA still meets the cluster's barriers.
#include <algorithm>
#include <atomic>

#include "tree_common.cuh"

namespace qsa {
namespace {

constexpr int kRows = 128;                  // (token, head) rows of a block (UMMA M); 128-cell tiles are N of QK^T
constexpr int kMaxTok = (kRows + kHPG - 2) / kHPG + 1;  // tokens a block's rows may touch
constexpr int kThreads = 17 * 32;
constexpr int kMaxC = 16;
constexpr int kNS = 2;
constexpr int kOffK = 0, kOffV = kTileStages * kTileStageBytes, kOffQ = 2 * kTileStages * kTileStageBytes;
constexpr int kOffML = kOffQ + kRows * kD * 2;          // float2 (m, l) [kMaxC][kRows], pushed by every CTA
constexpr int kSmem = kOffML + kMaxC * kRows * 8 + 1024;  // + alignment slack
constexpr int kOStride = kD + 4;            // floats per merged row: 16 bytes of padding spread the banks
static_assert(kRows * kOStride * 4 <= kOffML, "the merge buffer fits over the operand tiles");
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr uint32_t kColO = 0, kColS = 256;
constexpr float kRescaleThreshold = 8.0f;   // log2 units

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
  int* status;
};

struct __align__(8) TreeBars {
  uint64_t k_full[kTileStages], k_empty[kTileStages], v_full[kTileStages], v_empty[kTileStages];
  uint64_t s_full[kNS], p_full[kNS], pv_done[kNS];
  uint64_t q_full, drain;
};

// Index of a sequence's first block in the grid: block k of sequence s has index first_block(s) + k.
// The sequences' ranges never meet, since floor((a + b) / 128) + 1 >= floor(a / 128) + ceil(b / 128), so
// a block finds its sequence by a search over the table, without a prefix sum; some indices stay unused.
__device__ __forceinline__ long long first_block(long long first_row, int s) { return first_row * kHPG / kRows + s; }

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

__global__ void __launch_bounds__(kThreads, 1) tree_dense_kernel(const __grid_constant__ DenseTreeArgs a, int nC) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ TreeBars bars;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ int s_blk[8];                       // active, first pool cell, pos0, T, first token row, first row
  __shared__ uint32_t s_mask[kMaxTok][kTreeWords];
  __shared__ uint32_t s_union[kTreeWords];       // drafted cells that some token of ours sees
  __shared__ int s_ours, s_sel;                  // bit i: token i of the block is computed here; is a selected one
  __shared__ float s_xm[2][kRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank(), g = blockIdx.y;
  const int blk = blockIdx.x / nC;
  if (tid == 0) {
    s_abort = 0;
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&bars.k_full[i], 4);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 4);
      mbar_init(&bars.v_empty[i], 1);
    }
    for (int i = 0; i < kNS; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], 8);
      mbar_init(&bars.pv_done[i], 1);
    }
    mbar_init(&bars.q_full, 8);
    mbar_init(&bars.drain, 1);
    fence_mbar_init();
  }
  pdl_begin();
  if (blk == 0 && rank == 0 && g == 0) {  // one CTA looks over the whole table and flags bad entries
    for (int s = tid; s < a.b.n_seq; s += kThreads) {
      int4 e;
      if (tree_seq_tokens(a.b, s, &e) < 0) set_dev_status(a.status, QSA_DEV_BAD_ID);
    }
  }
  if (warp == 0) {
    const int sq = warp_find_seq(a.b.n_seq, blk, [&](int s) { return first_block(__ldg(&a.b.seqs[s].w), s); });
    int4 e;
    const int T = tree_seq_tokens(a.b, sq, &e);
    const long long k = blk - first_block(e.w, sq);
    const bool here = T > 0 && k >= 0 && k * kRows < (long long)T * kHPG;
    const int row0 = here ? (int)k * kRows : 0;
    const int tok = row0 / kHPG + lane;  // lane = token of the block
    const bool live = here && lane < kMaxTok && tok < T && tok * kHPG < row0 + kRows;
    int n_kv = e.z;
    uint32_t m[kTreeWords];
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) {
      m[w] = live ? tree_mask_word(a.b, e.w + tok, w, T) : 0u;
      n_kv += __popc(m[w]);
    }
    const bool sel = live && n_kv > a.b.identity_max, ours = live && (!sel || a.bits != nullptr);
    const unsigned all_ours = __ballot_sync(0xffffffffu, ours), all_sel = __ballot_sync(0xffffffffu, sel);
#pragma unroll
    for (int w = 0; w < kTreeWords; ++w) {
      const uint32_t u = __reduce_or_sync(0xffffffffu, ours ? m[w] : 0u);
      if (lane < kMaxTok) s_mask[lane][w] = m[w];
      if (lane == 0) s_union[w] = u;
    }
    if (lane == 0) {
      s_ours = (int)all_ours;
      s_sel = (int)all_sel;
      s_blk[0] = all_ours != 0u;
      s_blk[1] = e.x;
      s_blk[2] = e.z;
      s_blk[3] = T;
      s_blk[4] = e.w;
      s_blk[5] = row0;
    }
  }
  __syncthreads();
  if (!s_blk[0]) return;  // the same in every CTA of the cluster: an unused index, or no token of ours
  const long long cell0 = s_blk[1];
  const int pos0 = s_blk[2], T = s_blk[3], first = s_blk[4], row0 = s_blk[5];
  const int n_scan = pos0 + T;
  const int n_tiles = (n_scan + kTileCells - 1) / kTileCells;
  const int j_begin = n_tiles * rank / nC, J = n_tiles * (rank + 1) / nC - j_begin;
  if (warp == 16) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_arrive();  // #0, waited for before the first remote store: every CTA has started
  const uint32_t tmem = s_tmem;
  float m_run = -INFINITY, l_run = 0.f;  // softmax threads: the row's running maximum (log2 units), this half's sum
  bool ok = true;

  if (warp < 8) {
    const TileRun t{cell0, pos0, T, j_begin, J, g, s_union, &s_abort, a.status};
    if (warp < 4)
      produce_tiles<false, false>(t, a.kq, a.ksc, smem_u32(smem + kOffK), bars.k_full, bars.k_empty, warp, lane);
    else
      produce_tiles<true, false>(t, a.vq, a.vsc, smem_u32(smem + kOffV), bars.v_full, bars.v_empty, warp - 4, lane);
  } else if (warp == 16) {
    // ------------------------------------------------------------ MMA issue
    if (lane == 0 && J > 0) {
      const uint32_t idesc_qk = idesc_f16_f32(kRows, kTileCells, 0, 0);
      const uint32_t idesc_pv = idesc_f16_f32(kRows, kD, 0, 1);
      const uint32_t k0 = smem_u32(smem + kOffK), v0 = smem_u32(smem + kOffV);
      const uint64_t qdesc = sdesc_sw128(smem_u32(smem + kOffQ), 16, 1024);
      auto issue_qk = [&](int j) -> bool {
        const int b = j % kNS;
        if (j >= kNS && !mbar_wait_poll<false>(&bars.pv_done[b], ((j / kNS) - 1) & 1, a.status, &s_abort)) return false;
        for (int d = 0; d < kTileParts; ++d) {
          const int s = j * kTileParts + d, slot = s % kTileStages;
          if (!mbar_wait_poll<false>(&bars.k_full[slot], (s / kTileStages) & 1, a.status, &s_abort)) return false;
          tc_fence_after();
          const uint64_t kdesc = sdesc_sw128(k0 + slot * kTileStageBytes, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_ss(tmem + kColS + b * kTileCells, qdesc + (uint64_t)((d * (kRows * 128) + kk * 32) >> 4),
                    kdesc + (uint64_t)((kk * 32) >> 4), idesc_qk, (d > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars.k_empty[slot]);
        }
        umma_commit(&bars.s_full[b]);
        return true;
      };
      auto issue_pv = [&](int j) -> bool {
        const int b = j % kNS;
        if (!mbar_wait_poll<false>(&bars.p_full[b], (j / kNS) & 1, a.status, &s_abort)) return false;
        for (int c = 0; c < kTileParts; ++c) {
          const int s = j * kTileParts + c, slot = s % kTileStages;
          if (!mbar_wait_poll<false>(&bars.v_full[slot], (s / kTileStages) & 1, a.status, &s_abort)) return false;
          tc_fence_after();
          const uint64_t vdesc = sdesc_sw128(v0 + slot * kTileStageBytes, 4096, 1024);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            umma_ts(tmem + kColO, tmem + kColS + b * kTileCells + (2 * c + kk) * 8, vdesc + (uint64_t)((kk * 2048) >> 4),
                    idesc_pv, (j > 0 || c > 0 || kk > 0) ? 1u : 0u);
          umma_commit(&bars.v_empty[slot]);
        }
        umma_commit(&bars.pv_done[b]);
        return true;
      };
      bool go = mbar_wait_poll<false>(&bars.q_full, 0, a.status, &s_abort) && issue_qk(0);
      for (int j = 0; go && j < J; ++j) {
        if (j + 1 < J) go = issue_qk(j + 1);
        go = go && issue_pv(j);
      }
      umma_commit(&bars.drain);  // everything issued completes before TMEM is released
      mbar_wait(&bars.drain, 0, a.status);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ Q, then softmax rows
    const int st = tid - 256, wg = warp >= 12 ? 1 : 0, quarter = warp & 3;
    {
      const int c = st & 31;  // 16-byte chunk of a row
#pragma unroll 1
      for (int i0 = 0; i0 < kRows / 8; i0 += 8) {
        uint4 w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int R = row0 + (i0 + i) * 8 + (st >> 5);
          w[i] = make_uint4(0u, 0u, 0u, 0u);
          if (R < T * kHPG)
            w[i] = __ldg(reinterpret_cast<const uint4*>(
                             a.q + ((size_t)(first + R / kHPG) * kHeads + g * kHPG + R % kHPG) * kD) + c);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = (i0 + i) * 8 + (st >> 5);
          *reinterpret_cast<uint4*>(smem + kOffQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = w[i];
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_full);
    }
    const int r = quarter * 32 + lane;  // TMEM lane == block row
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const int R = row0 + r;
    const int ti = R / kHPG - row0 / kHPG;  // token of the block
    const bool active = R < T * kHPG && ((s_ours >> ti) & 1), chosen = active && ((s_sel >> ti) & 1);
    const uint2* sel_bits = reinterpret_cast<const uint2*>(
        chosen ? a.bits + (size_t)(g * a.b.n_tok + first + R / kHPG) * a.bits_pitch : nullptr);
    uint2 m_next = make_uint2(0u, 0u);  // a selected row's bits, loaded a tile ahead
    if (chosen && J > 0) m_next = __ldg(sel_bits + 2 * j_begin + wg);
    // 32 visibility bits from drafted cell x on: cells before the drafted ones are seen, those past the mask not
    auto bits32 = [&](int x) -> uint32_t {
      const int w = x >> 5;  // floor
      const uint32_t lo = w < 0 ? 0xffffffffu : w < kTreeWords ? s_mask[ti][w] : 0u;
      const uint32_t hi = w + 1 < 0 ? 0xffffffffu : w + 1 < kTreeWords ? s_mask[ti][w + 1] : 0u;
      return __funnelshift_r(lo, hi, x & 31);
    };
    for (int j = 0; j < J; ++j) {
      const int b = j % kNS;
      const bool w_ok = mbar_wait_warp(&bars.s_full[b], (j / kNS) & 1, a.status, &s_abort);
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
      if (chosen && j + 1 < J) m_next = __ldg(sel_bits + 2 * (j_begin + j + 1) + wg);
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
            if (mbar_wait_warp(&bars.pv_done[(j - 1) % kNS], ((j - 1) / kNS) & 1, a.status, &s_abort)) {
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
      float lsum = 0.f;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t p[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float p0 = fast_exp2(fmaf(s[32 * hf + 2 * i], a.scale_log2, -m_use));
          const float p1 = fast_exp2(fmaf(s[32 * hf + 2 * i + 1], a.scale_log2, -m_use));
          lsum += p0 + p1;
          p[i] = pack_half2(p0, p1);
        }
        tmem_st16(lane_base + kColS + b * kTileCells + wg * 32 + 16 * hf, p);
      }
      l_run += lsum;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full[b]);
    }
    if (J > 0 && ok) ok = mbar_wait_warp(&bars.pv_done[(J - 1) % kNS], ((J - 1) / kNS) & 1, a.status, &s_abort);
    // (m, l) of the row to every CTA of the cluster; a failed or empty CTA contributes nothing
    const bool all_ok = !named_bar_any(1, 256, !ok);
    s_xm[wg][r] = l_run;
    named_bar_any(1, 256, false);
    if (!all_ok) m_run = -INFINITY;
    cluster_wait();  // #0
    if (wg == 0) {
      const float l = l_run + s_xm[1][r];
      const uint32_t at = smem_u32(smem + kOffML) + (uint32_t)(rank * kRows + r) * 8u;
      for (int c = 0; c < nC; ++c)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(at, c)), "f"(m_run), "f"(l) : "memory");
    }
  }

  // ---------------------------------------------------------------- merge
  // CTA c owns the block's rows [c * 128 / nC, (c + 1) * 128 / nC).  Past this barrier every CTA's MMAs are
  // complete, so its operand tiles take the partial rows that the others push: O 2^(m - M) / L.
  if (warp < 8 || warp == 16) cluster_wait();  // #0
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();  // #1
  tc_fence_after();
  const float2* ml = reinterpret_cast<const float2*>(smem + kOffML);
  const int per = kRows / nC;
  if (warp >= 8 && warp < 16) {
    const int wg = warp >= 12 ? 1 : 0, quarter = warp & 3, r = quarter * 32 + lane;
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    float M = -INFINITY, L = 0.f;
    for (int c = 0; c < nC; ++c) M = fmaxf(M, ml[c * kRows + r].x);
    for (int c = 0; c < nC; ++c) {
      const float2 v = ml[c * kRows + r];
      if (v.x != -INFINITY) L = fmaf(v.y, fast_exp2(v.x - M), L);
    }
    const float f = m_run == -INFINITY ? 0.f : fast_exp2(m_run - M) / L;
    const int owner = r / per;
    const uint32_t dst = mapa_shared(smem_u32(smem) + (uint32_t)((rank * per + r % per) * kOStride) * 4u, owner);
    if (J > 0) {  // uniform over the warp, as the TMEM loads need
#pragma unroll 1
      for (int c0 = wg * 128; c0 < wg * 128 + 128; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(lane_base + kColO + c0, o);
        tmem_wait_ld();
        if (m_run != -INFINITY) {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (uint32_t)(c0 + i) * 4u),
                         "f"(__uint_as_float(o[i]) * f), "f"(__uint_as_float(o[i + 1]) * f),
                         "f"(__uint_as_float(o[i + 2]) * f), "f"(__uint_as_float(o[i + 3]) * f)
                         : "memory");
        }
      }
    }
  }
  tc_fence_before();
  __syncwarp();
  cluster_arrive();
  cluster_wait();  // #2: no CTA touches another after this
  if (warp == 16) tmem_dealloc(tmem, 512);
  if (warp < 16) {
    for (int x = tid; x < per * 32; x += 512) {
      const int rr = x >> 5, d8 = x & 31, r = rank * per + rr, R = row0 + r;
      const int ti = R / kHPG - row0 / kHPG;
      if (R >= T * kHPG || !((s_ours >> ti) & 1)) continue;
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int c = 0; c < nC; ++c) {
        if (ml[c * kRows + r].x == -INFINITY) continue;  // nothing pushed for this row
        const float4* src = reinterpret_cast<const float4*>(smem + (size_t)((c * per + rr) * kOStride) * 4) + 2 * d8;
        const float4 u = src[0], v = src[1];
        acc[0] += u.x;
        acc[1] += u.y;
        acc[2] += u.z;
        acc[3] += u.w;
        acc[4] += v.x;
        acc[5] += v.y;
        acc[6] += v.z;
        acc[7] += v.w;
      }
      const size_t at = ((size_t)(first + R / kHPG) * kHeads + g * kHPG + R % kHPG) * kD + d8 * 8;
      if (a.gate) {
        const uint4 gw = __ldg(reinterpret_cast<const uint4*>(a.gate + at));
        const uint32_t w[4] = {gw.x, gw.y, gw.z, gw.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
          acc[2 * i] *= gate_sigmoid(v.x);
          acc[2 * i + 1] *= gate_sigmoid(v.y);
        }
      }
      *reinterpret_cast<uint4*>(a.out + at) = make_uint4(pack_half2(acc[0], acc[1]), pack_half2(acc[2], acc[3]),
                                                         pack_half2(acc[4], acc[5]), pack_half2(acc[6], acc[7]));
    }
  }
}

constexpr int kSizes[5] = {1, 2, 4, 8, 16};

cudaLaunchConfig_t tree_config(int C, int blocks, cudaStream_t stream, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks * C, kGroups);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Per device, set once: the kernel's attributes, and how many clusters of each size the GPU holds at once
// (0: none of that size); threads that race here store the same values.
cudaError_t tree_setup(int (&n_max)[5]) {
  static std::atomic<int> ready[64];
  static std::atomic<int> held[64][5];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (ready[dev].load(std::memory_order_acquire) == 0) {
    if ((e = cudaFuncSetAttribute(tree_dense_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess)
      return e;
    if ((e = cudaFuncSetAttribute(tree_dense_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
      return e;
    for (int i = 0; i < 5; ++i) {
      cudaLaunchAttribute attr[2];
      cudaLaunchConfig_t cfg = tree_config(kSizes[i], 1, nullptr, attr);
      int n = 0;
      if ((e = cudaOccupancyMaxActiveClusters(&n, tree_dense_kernel, &cfg)) != cudaSuccess) return e;
      held[dev][i].store(n, std::memory_order_relaxed);
    }
    ready[dev].store(1, std::memory_order_release);
  }
  for (int i = 0; i < 5; ++i) n_max[i] = held[dev][i].load(std::memory_order_relaxed);
  return n_max[0] > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
}

}  // namespace

cudaError_t launch_tree_dense(const TreeBatch& b, const __half* q, const int8_t* kq, const int8_t* vq, const __half* ksc,
                              const __half* vsc, const uint32_t* bits, int bits_pitch, const __half* gate, __half* out,
                              float sm_scale, int* status, cudaStream_t stream) {
  int n_max[5];
  cudaError_t e = tree_setup(n_max);
  if (e != cudaSuccess) return e;
  const int blocks = (int)((long long)b.n_tok * kHPG / kRows) + b.n_seq;  // indices; a ragged batch leaves about half a
  const long long likely = ((long long)b.n_tok * kHPG + kRows / 2 * (b.n_seq - 1LL) + kRows - 1) / kRows;  // block each unused
  // Cluster size: waves x (a fixed part + the tiles of a CTA), in units of one tile's time.
  const long long longest = bits ? b.max_n_kv : std::min<long long>(b.max_n_kv, (long long)b.identity_max + 32 * b.tree_words);
  const int tiles = (int)((longest + kTileCells - 1) / kTileCells);
  int best = 1;
  double best_t = 0.0;
  for (int i = 0; i < 5; ++i) {
    const int C = kSizes[i];
    if (n_max[i] <= 0 || (C > 1 && C > tiles)) continue;
    const int per = (tiles + C - 1) / C;
    const double waves = (double)((likely * kGroups + n_max[i] - 1) / n_max[i]);
    const double t = waves * (5.5 + 0.8 * i + per);
    if (i == 0 || t < best_t) {
      best = C;
      best_t = t;
    }
  }
  const DenseTreeArgs a{b, q, kq, vq, ksc, vsc, bits, bits_pitch, sm_scale * kLog2e, gate, out, status};
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = tree_config(best, blocks, stream, attr);
  return cudaLaunchKernelEx(&cfg, tree_dense_kernel, a, best);
}

}  // namespace qsa
