// qsa_prefix_attention: attention of a batch whose sequences share prefixes.
//
//   out[t,h,:] = sum_c softmax_c(sm_scale q[t,h,:] . k^[c]) v^[c],  c over the cells of the token's prefix and of its own
//   sequence (all that it sees, or its topk selected ones);  k^ = fp16(kq * ksc), v^ = fp16(vq * vsc).
//
// The softmax over both sets is joined from the parts (O, m, l) of each: M = max m, L = sum l e^(m - M), out = sum O e^(m - M) / L.
// So the prefix's cells are attended to once for all tokens behind it: their (token, head) rows, 12 a token and group, are
// packed into blocks of 256, the M of the tensor-core kernel of tree.cu, which reads the int8 cells once a block and
// writes the parts.  A sequence's own cells serve its own few tokens alone: 12 rows fill no such block, and the cells
// bound the time by their bytes, so prefix_join_kernel streams them past a 16-row mma.sync tile, a CTA a token and
// group, and joins the prefix's parts in the same launch.  Sequences of many tokens (drafted trees) take the
// tensor-core kernel for their own cells too, and the launch joins both.
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
// What the join needs of a token besides its record (TreeBatch::tok): its sequence's {first pool cell, committed own cells,
// tokens, first token row}, and its prefix's {first token row, tokens, -, -}.
struct TokMore {
  int4 seq, prefix;
};

// Blocks, in this order: (token, group): Qsum and its error terms; (prefix, chunk of 2,048 cells) and (sequence, every
// own_chunks-th chunk): max |ksc|; the first three only where tokens may select.  Then 256 tokens' records each.
constexpr int kNearSeqs = 1024, kNearPrefixes = 256;  // tables up to so long are searched in shared memory
__global__ void __launch_bounds__(256) prefix_prep_kernel(const TreeBatch b, const TreeSelect w, TokMore* __restrict__ more,
                                                          bool select, int own_chunks, const __half* __restrict__ q,
                                                          const __half* __restrict__ ksc, int* status) {
  __shared__ long long s_e[8], s_h[8];
  __shared__ uint32_t s_union[kTreeWords];
  __shared__ float s_max[8][kGroups * kNB];
  __shared__ int s_row[kNearSeqs], s_seq[kNearPrefixes];
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
        for (int c = c0 + tid; c < c1; c += 256) {
          const int dj = c - pos0;
          if (dj >= 0 && !((s_union[dj >> 5] >> (dj & 31)) & 1u)) continue;  // a drafted cell that no token sees
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(ksc + ((size_t)e.x + c) * (kGroups * kNB)));
          const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u[j]));
            mx[2 * j] = fmaxf(mx[2 * j], fabsf(f.x));
            mx[2 * j + 1] = fmaxf(mx[2 * j + 1], fabsf(f.y));
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
  const bool near = b.n_seq <= kNearSeqs, near_prefixes = b.n_prefix <= kNearPrefixes;
  for (int i = tid; near && i < b.n_seq; i += 256) s_row[i] = __ldg(&b.seqs[i].w);
  for (int i = tid; near_prefixes && i < b.n_prefix; i += 256) s_seq[i] = __ldg(&b.prefixes[i].z);
  __syncthreads();
  auto last_at = [](int n, int at, auto key) {  // the last of n whose key is not above `at`
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (key(mid) <= at) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  };
  auto prefix_at = [&](int s) {
    if (b.n_prefix == 0) return -1;
    return near_prefixes ? last_at(b.n_prefix, s, [&](int i) { return s_seq[i]; }) : prefix_of(b, s);
  };
  const int n_blocks = (b.n_tok + 255) / 256;
  const int t = x * 256 + tid;
  if (t < b.n_tok) {
    const int s = near ? last_at(b.n_seq, t, [&](int i) { return s_row[i]; }) : last_at(b.n_seq, t, [&](int i) { return __ldg(&b.seqs[i].w); });
    const int p = prefix_at(s);
    const SharedSeq v = shared_seq(b, s, p);
    int4 r = make_int4(-1, 0, 0, -1);
    if (v.T > 0 && t >= v.e.w && t < v.e.w + v.T) {
      int seen = v.pe.y + v.e.z;
      for (int i = 0; 32 * i < v.T; ++i) seen += __popc(shared_mask_word(b, t, t - v.e.w, i, v.T));
      r = make_int4(s, seen, v.pe.y, p);
      more[t] = TokMore{make_int4(v.e.x, v.e.z, v.T, v.e.w), make_int4(v.pe.w, v.pT, 0, 0)};
    }
    b.tok[t] = r;
  }
  for (int s = t; s < b.n_seq; s += n_blocks * 256)
    if (shared_seq(b, s, prefix_at(s)).T < 0) set_dev_status(status, QSA_DEV_BAD_ID);
  for (int p = t; p < b.n_prefix; p += n_blocks * 256) {
    int4 e;
    if (prefix_tokens(b, p, &e) < 0) set_dev_status(status, QSA_DEV_BAD_ID);
  }
}

// ---------------------------------------------------------------- 2. own cells, and the join
constexpr int kJoinWarps = 4, kJoinThreads = kJoinWarps * 32;
constexpr int kTile = 16;                      // cells of a warp's step
constexpr int kStages = 3;                     // of its ring
constexpr int kStageBytes = 2 * kTile * kD + 2 * kTile * kNB * 2;  // codes of K and V, scales
constexpr int kQPitch = kD * 2 + 16;           // bytes of a query row: 16 of padding spread the banks
constexpr int kOffRing = 16 * kQPitch;
constexpr int kJoinSmem = kOffRing + kJoinWarps * kStages * kStageBytes;
constexpr int kMaxJoin = 8;                    // CTAs of a cluster
static_assert(2 * (kJoinSmem + 3 * 1024) <= 228 * 1024, "two CTAs on an SM");
// Over the ring, once the own cells are attended to: the CTA's slice of every CTA's own rows (pushed by them), then the
// warps' unmerged rows and, when those are merged, the slice of the parts.
constexpr int kOPitch = kD + 4;                // floats of a warp's unmerged row
constexpr int kRecvBytes = kHPG * kD * 4;      // [S][kHPG][kD / S]
constexpr int kOffRows = kRecvBytes;           // [kJoinWarps][kHPG][kOPitch]
constexpr int kPartBytes = kJoinWarps * kStages * kStageBytes - kRecvBytes;  // behind the slices of own rows: parts of as many runs as fit
static_assert(kJoinWarps * kHPG * kOPitch * 4 <= kPartBytes && kPartBytes >= 7 * kHPG * kD * 4, "the rows fit over the ring");
static_assert(kOffRing % 16 == 0 && kStageBytes % 16 == 0, "16-byte copies");
static_assert(2 * kMaxRuns * kHPG * 8 <= kOffRing, "the parts' (m, l) lie over the queries");
constexpr float kRescaleBy = 8.f, kPUp = 7.f;  // log2 units; as in tree.cu

struct JoinArgs {
  TreeBatch b;
  const TokMore* more;
  const __half* q;
  const int8_t* kq;
  const int8_t* vq;
  const __half* ksc;
  const __half* vsc;
  const uint32_t* bits;  // selected columns [2][n_tok][bits_pitch words], or null
  int bits_pitch;
  float scale_log2;
  const __half* gate;
  __half* out;
  TreeParts prefix, own;  // parts to join; runs 0: none (own cells are then attended to here)
};

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds16(uint32_t at) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at) : "memory");
  return v;
}
// Where row R of the rows behind `first_row` (12 a token; T tokens; table index i) lies among the parts: CTA of run 0,
// and row of that CTA.
__device__ __forceinline__ void part_row(int first_row, int i, int T, int g, int runs, int R, size_t* cta, int* row) {
  const int k = R / kTreeBlock, r = R % kTreeBlock;
  const int n = min(kTreeBlock, T * kHPG - k * kTreeBlock), first = (n + 1) / 2;
  const int half = r >= first;
  *cta = ((size_t)(first_block(first_row, i) + k) * kGroups + g) * runs * 2 + half;
  *row = half ? r - first : r;
}

// A cluster of S CTAs a (token, group).  The warps take the tiles of 16 own cells in turn, each through a ring of its own:
//   S = Q K^T  (A = 16 rows of Q, 12 of them heads; B = K^, two n8 tiles), 16 k16 steps
//   O += P V^  (A = P as it stands in S's registers, B = V^, 32 n8 tiles), one k16 step
// Lanes take the k dims, and V's n dims, in an order of their own, the same for both operands, so that a lane's codes are 16
// bytes side by side: of a k64 block lane (n, i) has dims 16 i .. 16 i + 15 of cell n, four k16 steps of four; of V lane
// (n, i) has dims 16 n .. 16 n + 15 of a half of cells 2 i, 2 i + 1, 2 i + 8 and 2 i + 9, which sixteen n8 tiles take one by one.  The
// 16-byte chunks of a cell's row are xored by a bit (K: the cell's lowest, times 4; V: its next two, times 2), so that
// the eight lanes of a shared-memory phase meet different banks.
__global__ void __launch_bounds__(kJoinThreads, 2) prefix_join_kernel(const __grid_constant__ JoinArgs a, int S) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 s_ml[kJoinWarps][16];   // (m, l) of the warps' rows
  __shared__ float2 s_sum[kHPG];            // and of the CTA's
  __shared__ float s_wf[kJoinWarps][kHPG];  // what the warps' rows are multiplied by
  __shared__ float2 s_own[kMaxJoin][kHPG];  // (m, l) of the CTAs' own rows; then their weights
  __shared__ float s_inv[kHPG];
  __shared__ size_t s_from[2][kHPG];        // where the rows of run 0's part start (prefix, own), in float4
  cluster_arrive_all();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blockIdx.x % S, g = blockIdx.x / S % kGroups, t = blockIdx.x / S / kGroups;
  // With own cells to attend to, the launch before is the prefixes' one, if there are any: its CTAs trigger this launch once
  // all before it are complete, and the own cells need nothing of it.
  const bool here = a.own.runs == 0;
  if (!here || a.prefix.runs == 0) pdl_begin();
  const int4 ti = a.b.tok[t], e = a.more[t].seq, pe = a.more[t].prefix;
  if (ti.x < 0) {  // the same in all CTAs of the cluster
    pdl_begin();
    cluster_wait_all();
    return;
  }
  const int T = e.z, i_tok = t - e.w, pos0 = e.y;
  const bool chosen = a.bits != nullptr && ti.y > a.b.identity_max;
  const size_t out_row = ((size_t)t * kHeads + g * kHPG) * kD;
  if (here) {
    // ---- the queries' rows; 12 .. 15 are zeros
    for (int i = tid; i < 16 * 32; i += kJoinThreads) {
      const int r = i >> 5, c = i & 31;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (r < kHPG) v = __ldg(reinterpret_cast<const uint4*>(a.q + out_row + (size_t)r * kD) + c);
      *reinterpret_cast<uint4*>(smem + r * kQPitch + c * 16) = v;
    }
    const int n_own = pos0 + (a.b.tree ? T : i_tok + 1);
    const int n_tiles = (n_own + kTile - 1) / kTile;
    const int begin = (int)((long long)n_tiles * rank / S), end = (int)((long long)n_tiles * (rank + 1) / S);
    const int mine = max(0, (end - begin - warp + kJoinWarps - 1) / kJoinWarps);  // tiles begin + warp + 4 j
    const uint32_t ring = smem_u32(smem + kOffRing) + warp * (kStages * kStageBytes);
    const size_t cell0 = (size_t)e.x;
    auto load = [&](int j) {
      if (j < mine) {
        const int c0 = (begin + warp + kJoinWarps * j) * kTile;
        const uint32_t st = ring + (j % kStages) * kStageBytes;
        const int chunk = lane & 15;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = 2 * i + (lane >> 4);
          const size_t row = ((cell0 + min(c0 + c, n_own - 1)) * kGroups + g) * kD + chunk * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(st + c * kD + ((chunk ^ ((c & 1) << 2)) << 4)),
                       "l"(reinterpret_cast<uint64_t>(a.kq + row))
                       : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(st + kTile * kD + c * kD + ((chunk ^ (((c >> 1) & 3) << 1)) << 4)),
                       "l"(reinterpret_cast<uint64_t>(a.vq + row))
                       : "memory");
        }
        const __half* sc = (lane < 16 ? a.ksc : a.vsc) + ((cell0 + min(c0 + (lane & 15), n_own - 1)) * kGroups + g) * kNB;
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(st + 2 * kTile * kD + lane * 8), "l"(reinterpret_cast<uint64_t>(sc))
                     : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const uint32_t* bit_row =
        chosen ? a.bits + (size_t)(g * a.b.n_tok + t) * a.bits_pitch + own_column(ti.z) / 32 : nullptr;
    // the 16 cells from c0 on that are attended to, as bits
    auto seen16 = [&](int c0) -> uint32_t {
      if (chosen) return (__ldg(bit_row + (c0 >> 5)) >> (c0 & 31)) & 0xffffu;
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
    __syncthreads();  // the queries are in shared memory
    const int r = lane >> 2, i4 = lane & 3;
    const uint32_t q_lo = smem_u32(smem) + r * kQPitch + i4 * 32, q_hi = q_lo + 8 * kQPitch;
    for (int j = 0; j < mine; ++j) {
      load(j + 2);
      const uint32_t seen = seen16((begin + warp + kJoinWarps * j) * kTile);
      asm volatile("cp.async.wait_group 2;" ::: "memory");
      __syncwarp();
      const uint32_t st = ring + (j % kStages) * kStageBytes;
      if (seen) {
        float s[2][4] = {};
#pragma unroll
        for (int b = 0; b < kNB; ++b) {
          const uint4 qa = lds128(q_lo + b * 128), qb = lds128(q_lo + b * 128 + 16);
          const uint4 qc = lds128(q_hi + b * 128), qd = lds128(q_hi + b * 128 + 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int c = 8 * i + r;
            const uint4 k = lds128(st + c * kD + (((4 * b + i4) ^ ((c & 1) << 2)) << 4));
            const __half2 sc = __half2half2(__ushort_as_half(lds16(st + 2 * kTile * kD + c * 8 + b * 2)));
            uint32_t x[4], y[4];
            dequant8(k.x, k.y, sc, x);
            dequant8(k.z, k.w, sc, y);
            mma16816(s[i], qa.x, qc.x, qa.y, qc.y, x[0], x[1]);
            mma16816(s[i], qa.z, qc.z, qa.w, qc.w, x[2], x[3]);
            mma16816(s[i], qb.x, qd.x, qb.y, qd.y, y[0], y[1]);
            mma16816(s[i], qb.z, qd.z, qb.w, qd.w, y[2], y[3]);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (!((seen >> (8 * i + 2 * i4 + (k & 1))) & 1u)) s[i][k] = -INFINITY;
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
        const uint32_t vs = st + kTile * kD;
        const int ca = 2 * i4;  // this lane's cells: ca, ca + 1, ca + 8, ca + 9
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          // cells that are not attended to count with a scale of 0, whatever they hold
          auto scale = [&](int c) {
            const uint16_t x = lds16(st + 2 * kTile * kD + kTile * 8 + c * 8 + (2 * hf + (r >> 2)) * 2);
            return __ushort_as_half((seen >> c) & 1u ? x : (uint16_t)0);
          };
          const __half2 sa = __halves2half2(scale(ca), scale(ca + 1)), sb = __halves2half2(scale(ca + 8), scale(ca + 9));
          auto codes = [&](int c) { return lds128(vs + c * kD + (((8 * hf + r) ^ (((c >> 1) & 3) << 1)) << 4)); };
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
    if (i4 == 0) {
      s_ml[warp][r] = make_float2(m0, l0);
      s_ml[warp][r + 8] = make_float2(m1, l1);
    }
    __syncthreads();  // every warp is done with its ring
    // O: lane (r, i) has dims 128 hf + 32 i + {0, 16} + n of rows r and r + 8
    float* rows = reinterpret_cast<float*>(smem + kOffRing + kOffRows) + warp * (kHPG * kOPitch);
#pragma unroll
    for (int hf = 0; hf < 2; ++hf)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = r + (k >> 1) * 8, dim = 128 * hf + 32 * i4 + 16 * (k & 1);
        if (row < kHPG) {
#pragma unroll
          for (int n = 0; n < 16; n += 4)
            *reinterpret_cast<float4*>(rows + row * kOPitch + dim + n) =
                make_float4(o[16 * hf + n][k], o[16 * hf + n + 1][k], o[16 * hf + n + 2][k], o[16 * hf + n + 3][k]);
        }
      }
  }
  // ---- the warps' own rows in one, each CTA's slice of 256 / S dims pushed to it
  cluster_wait_all();    // every CTA of the cluster runs
  cluster_arrive_all();  // this one is past its ring
  const int dims = kD / S;
  if (here) {
    __syncthreads();
    if (tid < kHPG) {
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_ml[w][tid].x);
#pragma unroll 1
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = s_ml[w][tid].x == -INFINITY ? 0.f : fast_exp2(s_ml[w][tid].x - m);
        s_wf[w][tid] = f;
        l = fmaf(s_ml[w][tid].y, f, l);
      }
      s_sum[tid] = make_float2(m, l);
    }
    __syncthreads();
  }
  cluster_wait_all();  // and so are the others
  if (here) {
    if (tid < kHPG) {
      const float m = s_sum[tid].x, l = s_sum[tid].y;
#pragma unroll 1
      for (int c = 0; c < S; ++c)
        asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(&s_own[rank][tid]), c)), "f"(m), "f"(l) : "memory");
    }
    const float* rows = reinterpret_cast<const float*>(smem + kOffRing + kOffRows);
#pragma unroll 1
    for (int i = tid; i < kHPG * (kD / 4); i += kJoinThreads) {
      const int h = i / (kD / 4), d = i % (kD / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) {
        const float f = s_wf[w][h];
        const float4 x = *reinterpret_cast<const float4*>(rows + (w * kHPG + h) * kOPitch + d);
        v.x = fmaf(x.x, f, v.x);  // a row that has seen nothing holds zeros
        v.y = fmaf(x.y, f, v.y);
        v.z = fmaf(x.z, f, v.z);
        v.w = fmaf(x.w, f, v.w);
      }
      const uint32_t at = smem_u32(smem + kOffRing) + (uint32_t)((rank * kHPG + h) * dims + d % dims) * 4u;
      asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(mapa_shared(at, d / dims)), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                   : "memory");
    }
  }
  cluster_arrive_all();
  // ---- the parts of the launches before
  pdl_begin();
  const int px_runs = ti.z > 0 ? a.prefix.runs : 0, runs = px_runs + a.own.runs;
  if (tid < 2 * kHPG) {
    const bool own = tid >= kHPG;
    const int h = own ? tid - kHPG : tid;
    if (own ? a.own.runs > 0 : px_runs > 0) {
      size_t cta;
      int row;
      if (own) part_row(e.w, ti.x, T, g, a.own.runs, i_tok * kHPG + h, &cta, &row);
      else part_row(pe.x, ti.w, pe.y, g, px_runs, (t - pe.x) * kHPG + h, &cta, &row);
      s_from[own][h] = cta * (kTreeBlock / 2 * kD / 4) + row;
    }
  }
  cluster_wait_all();  // the slices have arrived, and every warp here is past the rows (and the queries)
  __syncthreads();
  constexpr int kRowStep = kTreeBlock / 2;               // float4 between the dims of a row
  constexpr size_t kRunStep = 2 * (size_t)kRowStep * kD / 4;  // and between runs
  float2(*s_part)[kHPG] = reinterpret_cast<float2(*)[kHPG]>(smem);  // over the queries: (m, l), then the weight
  const float4* parts = reinterpret_cast<const float4*>(smem + kOffRing + kRecvBytes);
  const int quads = dims / 4, fit = kPartBytes / (kHPG * 16) / quads;  // float4 of a row's slice; runs in a round
  auto fetch = [&](int u0, int n) {  // runs u0 .. u0 + n - 1: [run][quad][row] float4
    const uint32_t to = smem_u32(parts);
#pragma unroll 1
    for (int i = tid; i < n * quads * kHPG; i += kJoinThreads) {
      const int h = i % kHPG, x = i / kHPG, u = u0 + x / quads, d = rank * quads + x % quads;
      const bool own = u >= px_runs;
      const float4* from = (own ? a.own.o : a.prefix.o) + s_from[own][h] + (own ? u - px_runs : u) * kRunStep + (size_t)d * kRowStep;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(reinterpret_cast<uint64_t>(from)) : "memory");
    }
  };
  fetch(0, min(runs, fit));
#pragma unroll 1
  for (int i = tid; i < runs * kHPG; i += kJoinThreads) {
    const int h = i % kHPG, u = i / kHPG;
    const bool own = u >= px_runs;
    const size_t at = s_from[own][h];
    const size_t cta = at / (kTreeBlock / 2 * kD / 4) + 2 * (own ? u - px_runs : u), row = at % (kTreeBlock / 2);
    s_part[u][h] = __ldcg((own ? a.own.ml : a.prefix.ml) + cta * (kTreeBlock / 2) + row);
  }
  __syncthreads();
  // ---- weights e^(m - M) of the parts and of the CTAs' own rows, and 1 / L: a warp a row, a lane a part
#pragma unroll 1
  for (int h = warp; h < kHPG; h += kJoinWarps) {
    const int n = runs + (here ? S : 0);
    float2* mine[3];
    float M = -INFINITY, L = 0.f;
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int u = lane + 32 * k;
      mine[k] = u < runs ? &s_part[u][h] : u < n ? &s_own[u - runs][h] : nullptr;
      if (mine[k]) M = fmaxf(M, mine[k]->x);
    }
    static_assert(2 * kMaxRuns <= 96 && kMaxRuns + kMaxJoin <= 96, "three parts a lane");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (mine[k]) {
        const float f = mine[k]->x == -INFINITY ? 0.f : fast_exp2(mine[k]->x - M);  // nothing of this row there: weight 0
        if (f != 0.f) L = fmaf(mine[k]->y, f, L);
        mine[k]->x = f;
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
    if (lane == 0) s_inv[h] = L > 0.f ? 1.f / L : 0.f;  // a token that sees nothing: zeros
  }
  // ---- the sum, eight dims of a row a thread
  float* recv = reinterpret_cast<float*>(smem + kOffRing);
#pragma unroll 1
  for (int u0 = 0; u0 < runs || u0 == 0; u0 += fit) {
    const int n = min(runs - u0, fit);
    if (u0 > 0) {
      __syncthreads();  // the round before is read
      fetch(u0, n);
    }
    cp_async_wait_all();
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i < kHPG * dims / 8; i += kJoinThreads) {
      const int h = i % kHPG, d8 = i / kHPG;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      auto add = [&](float f, const float4& p, const float4& q) {
        x.x = fmaf(p.x, f, x.x);
        x.y = fmaf(p.y, f, x.y);
        x.z = fmaf(p.z, f, x.z);
        x.w = fmaf(p.w, f, x.w);
        y.x = fmaf(q.x, f, y.x);
        y.y = fmaf(q.y, f, y.y);
        y.z = fmaf(q.z, f, y.z);
        y.w = fmaf(q.w, f, y.w);
      };
      float4* keep = reinterpret_cast<float4*>(recv + h * dims + d8 * 8);  // rank 0's slice; later rounds: the sum so far
      if (u0 > 0) {
        add(1.f, keep[0], keep[1]);
      } else if (here) {
#pragma unroll 1
        for (int c = 0; c < S; ++c) {
          const float4* z = reinterpret_cast<const float4*>(recv + (c * kHPG + h) * dims + d8 * 8);
          add(s_own[c][h].x, z[0], z[1]);
        }
      }
      const float4* z = parts + 2 * d8 * kHPG + h;
#pragma unroll 2
      for (int u = 0; u < n; ++u, z += quads * kHPG) {
        const float f = s_part[u0 + u][h].x;
        if (f != 0.f) add(f, z[0], z[kHPG]);  // a run that has nothing of the row wrote nothing
      }
      if (u0 + fit < runs) {
        keep[0] = x;
        keep[1] = y;
        continue;
      }
      const size_t at = out_row + (size_t)h * kD + rank * dims + d8 * 8;
      const float inv = s_inv[h];
      float v[8] = {x.x * inv, x.y * inv, x.z * inv, x.w * inv, y.x * inv, y.y * inv, y.z * inv, y.w * inv};
      if (a.gate) apply_gate(v, __ldg(reinterpret_cast<const uint4*>(a.gate + at)));
      *reinterpret_cast<uint4*>(a.out + at) = pack_out(v);
    }
  }
}

// ---------------------------------------------------------------- the call
// From how many tokens a sequence (on average) their own cells go to the tensor-core kernel.
constexpr int kOwnTokens = 4;

struct Layout {
  size_t tok, more, prefix, own, select, kmax, bytes;
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
  l.prefix = take(n_prefix > 0 && max_prefix > 0 ? tree_parts_workspace_bytes(n_prefix, n_tok, max_prefix) : 0);
  l.own = take(n_tok >= kOwnTokens ? tree_parts_workspace_bytes(n_seq, n_tok, max_n_kv) : 0);  // a call of fewer sequences may take it
  if (max_n_kv > identity_max) {
    const int cells = std::min(max_n_kv, select_max_cells() - 127);
    l.select = take(tree_select_layout(n_seq, n_tok, cells + 127, nullptr, nullptr));
    l.kmax = take((size_t)n_prefix * ((max_prefix + kTreeChunk - 1) / kTreeChunk) * kGroups * kNB * sizeof(float));
  }
  l.bytes = o;
  return l;
}

cudaError_t join_setup() {
  static std::atomic<int> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_acquire)) {
    if ((e = cudaFuncSetAttribute(prefix_join_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kJoinSmem)) != cudaSuccess) return e;
    ready[dev].store(1, std::memory_order_release);
  }
  return cudaSuccess;
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
  TreeSelect w{};
  int own_chunks = 1;
  if (select) {
    tree_select_layout(b.n_seq, b.n_tok, b.max_n_kv + 127, base + l.select, &w);
    w.kmax_prefix = reinterpret_cast<float*>(base + l.kmax);
    w.chunks_prefix = (b.max_prefix + kTreeChunk - 1) / kTreeChunk;
    own_chunks = (own_cells + kTreeChunk - 1) / kTreeChunk;
  }
  const int prep = (select ? kGroups * b.n_tok + b.n_prefix * w.chunks_prefix + b.n_seq * own_chunks : 0) + (b.n_tok + 255) / 256;
  cudaError_t e = launch_pdl(prefix_prep_kernel, dim3(prep), dim3(256), 0, stream, b, w, more, select, own_chunks, q, ksc, status);
  if (e != cudaSuccess) return e;
  if (select && (e = launch_shared_select(b, w, own_cells, q, kq, ksc, ids, p, status, stream)) != cudaSuccess) return e;
  const uint32_t* bits = select ? w.bits : nullptr;
  JoinArgs a{b, more, q, kq, vq, ksc, vsc, bits, w.pitch / 32, p.sm_scale * kLog2e, gate, out, {}, {}};
  if (b.n_prefix > 0 && b.max_prefix > 0) {
    e = launch_tree_parts(b, false, b.max_prefix, q, kq, vq, ksc, vsc, bits, w.pitch / 32, base + l.prefix, p.sm_scale, &a.prefix,
                          status, stream);
    if (e != cudaSuccess) return e;
  }
  if ((long long)b.n_tok >= (long long)kOwnTokens * b.n_seq) {
    e = launch_tree_parts(b, true, own_cells, q, kq, vq, ksc, vsc, bits, w.pitch / 32, base + l.own, p.sm_scale, &a.own, status, stream);
    if (e != cudaSuccess) return e;
  }
  if ((e = join_setup()) != cudaSuccess) return e;
  // CTAs a (token, group): as many as fit on the GPU at once, two on an SM
  int S = 1;
  while (S < 8 && (long long)b.n_tok * kGroups * S * 2 <= 2 * 152) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(b.n_tok * kGroups * S));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = kJoinSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = S;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, prefix_join_kernel, a, S);
}

}  // namespace qsa
