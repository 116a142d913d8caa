// qsa_tree_verify: which path of a drafted tree the target accepts, and the token that follows it.
//
// Speculative sampling with several candidates: at the accepted token `cur` the target's distribution is w / c
// (w = p[cur], c = 1 at first) and the drafter's d[cur].  Its children are tried in their order; child k with token x is
// accepted iff u_k c d(x) < w(x).  A refused one leaves w <- max(w - c d, 0), c <- sum w, and where no child is left
// the next token is drawn from w / c by the inverse of its running sum.  Tokens then have the target's distribution
// whatever the drafter's is.  Without d the drafted tokens are point masses: accepted iff u_k c < w(x), and a refused
// one leaves w(x) <- 0.
//
// The walk needs two numbers a drafted token, p[parent][x] and d[parent][x], gathered at once.  What costs is the
// row: 8 bytes a vocabulary entry and sequence for the draw and for every refusal that has a sibling behind it.  A
// cluster takes a sequence, each CTA a part of the vocabulary; all CTAs walk alike.
//
// Running sums over 100,000 entries have neighbours 1e-5 apart and less, and fp32 sums would land beside the border.  Sums are
// whole numbers instead: a probability is taken in units of 2^-44 (fp32 holds 2^-24 of itself), so sums and
// differences are exact, in any order, and only w = max(w - c d, 0) after a second refusal rounds (to a unit).
//
// Measured (GB300, rows from DRAM): 64 trees of 4-24 tokens over 131,071 entries 40-53 us over runs for 84-92 MB of rows (13 us at a plain copy's
// rate): the pass that every sequence has ends after 14 us, near the memory's rate; the second and third pass of the 21-27
// sequences with several refusals take 8-18 us each, bound by their 64-bit arithmetic, since the hardware puts up to four CTAs of a
// cluster on one SM while others are idle (a spreading preference of the launch changed nothing).  48 trees without drafts'
// probabilities over 100,003 entries 11.7 us; one chain of 8 over 32,768 entries 6.6 us: start, gathers, a pass and the draw,
// each a round trip to memory.  Tried without a gain: all blocks' loads ahead (spilled), prefetches into L2 (48.6 to 53 us), pairs
// of floats for whole numbers, products of 32-bit halves written out (48.7 to 51).
#include "tree_common.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kMaxTokens = 32 * kTreeWords;  // drafted tokens of a sequence
constexpr int kBlock = 2 * kThreads;         // vocabulary entries of a warp's step (16 a lane), and of the draw (two a thread)
constexpr int kMaxBlocks = 512;              // 262,144 entries
constexpr int kMaxCluster = 8;
constexpr long long kUnit = 1ll << 44;

// Probability x in units of 2^-44, as hi 2^22 + lo with lo in [-2^21, 2^21], by two roundings to whole numbers in
// fp32 (adding 2^23, whose unit is 1).  hi and lo are added to sums that wrap, biased by kHiBias and kLoBias each.  x is
// in [0, 1]: values outside count as the nearer end, NaN as 0 (saturated).
constexpr uint32_t kHiBias = 0x4B000000u, kLoBias = 0x4B400000u;  // the bits of 2^23 and of 1.5 2^23
struct Parts {
  uint32_t hi, lo;
};
__device__ __forceinline__ Parts parts_of(float x) {
  const float t = fmaf(x, 4194304.f, 8388608.f);
  const float r = fmaf(x, 4194304.f, 8388608.f - t);  // exact
  return {__float_as_uint(t), __float_as_uint(fmaf(r, 4194304.f, 12582912.f))};
}
__device__ __forceinline__ long long units(uint32_t hi, uint32_t lo) { return ((long long)(int)hi << 22) + (int)lo; }
__device__ __forceinline__ long long fixed(float x) {
  const Parts f = parts_of(__saturatef(x));
  return units(f.hi - kHiBias, f.lo - kLoBias);
}

struct VerifyArgs {
  const float* p;
  const float* d;      // or null
  int64_t p_stride, d_stride;
  int vocab;
  bool vec_p, vec_d;   // rows start on 16 bytes
  const int32_t* token;
  const int32_t* parent;
  const float* u;
  const float* u_end;
  const int4* seqs;
  int n_seq, n_tok;
  int32_t* path;
  int32_t* n_path;
  int32_t* next;
  int path_cap;
  int* status;
};

// Entries j .. j + 3 of a row; those past the vocabulary are 0.
__device__ __forceinline__ float4 load4(const float* row, int j, int vocab, bool vec) {
  if (vec && j + 4 <= vocab) return __ldg(reinterpret_cast<const float4*>(row + j));
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (j < vocab) v.x = __ldg(row + j);
  if (j + 1 < vocab) v.y = __ldg(row + j + 1);
  if (j + 2 < vocab) v.z = __ldg(row + j + 2);
  if (j + 3 < vocab) v.w = __ldg(row + j + 3);
  return v;
}

// w after `refused` refusals of N entries side by side, from their p and d and the masses c[0 .. refused), each below 4 (2^46 units).
template <int N>
__device__ __forceinline__ void left_over(const float (&p)[N], const float (&d)[N], const long long* mass, int refused, long long (&w)[N]) {
  unsigned long long df[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const float x = __saturatef(p[q]), y = __saturatef(d[q]);
    const Parts f = parts_of(x), m = parts_of(refused > 0 ? fminf(x, y) : 0.f);  // c[0] = 1: max(p - d, 0) = p - min(p, d)
    const Parts g = parts_of(y);
    w[q] = units(f.hi - m.hi, f.lo - m.lo);
    df[q] = (unsigned long long)units(g.hi - kHiBias, g.lo - kLoBias) << 2;
  }
#pragma unroll 1
  for (int r = 1; r < refused; ++r) {
    const unsigned long long c = (unsigned long long)mass[r] << 18;
#pragma unroll
    for (int q = 0; q < N; ++q) w[q] = max(w[q] - (long long)__umul64hi(c, df[q]), 0ll);
  }
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__global__ void __launch_bounds__(kThreads, 4) tree_verify_kernel(const __grid_constant__ VerifyArgs a, int C) {
  __shared__ int s_parent[kMaxTokens], s_token[kMaxTokens], s_path[kMaxTokens], s_out[kMaxTokens];
  __shared__ float s_u[kMaxTokens], s_p[kMaxTokens], s_d[kMaxTokens];
  __shared__ long long s_mass[kMaxTokens + 1];
  __shared__ long long s_block[kMaxBlocks];
  __shared__ long long s_warp[kWarps];
  __shared__ long long s_total[2][kMaxCluster];  // a pass's sums of the cluster's CTAs
  __shared__ int s_n, s_cur, s_refused, s_out_n, s_at, s_more;
  cluster_arrive_all();  // waited for before the first remote store: every CTA of the cluster runs
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int s = blockIdx.x / C, rank = blockIdx.x % C;
  const int4 e = __ldg(&a.seqs[s]);
  const int after = s + 1 < a.n_seq ? __ldg(&a.seqs[s + 1].w) : a.n_tok;
  const bool rows_ok = (s == 0 ? e.w == 0 : e.w >= 0) && after >= e.w && after <= a.n_tok;
  const int T = rows_ok && e.y != 0 ? after - e.w : 0;
  bool bad = !rows_ok || T > kMaxTokens;
  if (!bad && tid < T) {
    const int t = e.w + tid, up = __ldg(a.parent + t), x = __ldg(a.token + t);
    bad = tid == 0 ? up != -1 : up < 0 || up >= tid || x < 0 || x >= a.vocab;
    s_parent[tid] = up;
    s_token[tid] = x;
    s_u[tid] = __ldg(a.u + t);
    if (!bad && tid > 0) {
      s_p[tid] = __ldg(a.p + (e.w + up) * a.p_stride + x);
      s_d[tid] = a.d ? __ldg(a.d + (e.w + up) * a.d_stride + x) : 1.f;
    }
  }
  bad = __syncthreads_or(bad);  // the same in all CTAs of the cluster
  cluster_wait_all();
  if (bad || T == 0) {
    if (rank == 0 && tid == 0) {
      if (bad) set_dev_status(a.status, QSA_DEV_BAD_ID);
      a.n_path[s] = 0;
      a.next[s] = -1;
    }
    return;
  }
  if (tid == 0) {
    s_n = 1;
    s_path[0] = 0;
    s_cur = 0;
    s_refused = 0;
    s_out_n = 0;
    s_at = 1;
    s_mass[0] = kUnit;
  }
  __syncthreads();
  const int blocks = (a.vocab + kBlock - 1) / kBlock;
  const int b0 = blocks * rank / C, b1 = blocks * (rank + 1) / C;
  bool empty = false;  // the rest of the row is empty: the draw is from p itself
  for (int pass = 0;; ++pass) {
    // ---- the walk, by one warp, until a pass over the row is needed: more = a sibling is left to try after it
    if (warp == 0 && !empty) {
      int n = s_n, cur = s_cur, refused = s_refused, out_n = s_out_n, at = s_at;
      int more = 0;
      for (;;) {
        // the next child of cur from token `at` on
        int k = T;
        for (int base = at; base < T && k == T && n < a.path_cap; base += 32) {
          const unsigned m = __ballot_sync(0xffffffffu, base + lane < T && s_parent[base + lane] == cur);
          if (m) k = base + __ffs(m) - 1;
        }
        if (k == T) break;
        if (a.d && refused > 0 && !more && s_mass[refused] < 0) {  // the mass after the last refusal is not known yet
          more = 1;
          at = k;
          break;
        }
        const float pk = s_p[k], dk = s_d[k];
        const int x = s_token[k];
        double w;
        bool out = false;
        if (a.d) {
          if (refused == 0) {
            w = (double)__saturatef(pk);
          } else {
            long long left[1];
            left_over<1>({pk}, {dk}, s_mass, refused, left);
            w = (double)left[0] * (1.0 / kUnit);
          }
        } else {
          for (int i = lane; i < out_n; i += 32) out |= s_out[i] == x;  // refused before
          out = __any_sync(0xffffffffu, out);
          w = out ? 0.0 : (double)__saturatef(pk);
        }
        const double c = refused == 0 ? 1.0 : (double)s_mass[refused] * (1.0 / kUnit);
        __syncwarp();
        if ((double)s_u[k] * (double)__saturatef(dk) * c < w) {
          if (lane == 0) s_path[n] = k;
          ++n;
          cur = k;
          refused = 0;
          out_n = 0;
        } else {
          if (lane == 0) {
            s_mass[refused + 1] = a.d ? -1 : max(s_mass[refused] - (out ? 0ll : fixed(pk)), 0ll);
            if (!a.d && !out) s_out[out_n] = x;
          }
          ++refused;
          if (!a.d && !out) ++out_n;
        }
        at = k + 1;
        __syncwarp();
      }
      if (lane == 0) {
        s_n = n;
        s_cur = cur;
        s_refused = refused;
        s_out_n = out_n;
        s_at = at;
        s_more = more;
      }
    }
    __syncthreads();
    // ---- this CTA's part of the row: what is left of it, block by block
    const int refused = empty ? 0 : s_refused, out_n = empty ? 0 : s_out_n;
    const float* prow = a.p + (size_t)(e.w + s_cur) * a.p_stride;
    const float* drow = a.d && refused > 0 ? a.d + (size_t)(e.w + s_cur) * a.d_stride : nullptr;
    for (int b = b0 + warp; b < b1; b += kWarps) {
      const int j0 = b * kBlock + lane * 4;
      constexpr int kQuads = kBlock / 128;  // loads of four entries a lane
      long long sum = 0;
      if (drow == nullptr) {
        uint32_t hs = -4u * kQuads * kHiBias, ls = -4u * kQuads * kLoBias;
        float4 v[kQuads];
#pragma unroll
        for (int i = 0; i < kQuads; ++i) v[i] = load4(prow, j0 + 128 * i, a.vocab, a.vec_p);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          const float f[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const Parts x = parts_of(__saturatef(f[q]));
            hs += x.hi;
            ls += x.lo;
          }
        }
        sum = units(hs, ls);
        for (int i = lane; i < out_n; i += 32) {
          const int x = s_out[i];
          if (x / kBlock == b) sum -= fixed(__ldg(prow + x));
        }
      } else {
        uint32_t hs = 0u, ls = 0u;  // p - min(p, d): the biases cancel
        static_assert(kQuads == 4, "four of each row");
        if (refused == 1) {
          float4 v[4], z[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = load4(prow, j0 + 128 * i, a.vocab, a.vec_p);
            z[i] = load4(drow, j0 + 128 * i, a.vocab, a.vec_d);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f[4] = {v[i].x, v[i].y, v[i].z, v[i].w}, g[4] = {z[i].x, z[i].y, z[i].z, z[i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float x = __saturatef(f[q]);
              const Parts y = parts_of(x), m = parts_of(fminf(x, __saturatef(g[q])));
              hs += y.hi - m.hi;
              ls += y.lo - m.lo;
            }
          }
        } else {  // a quad ahead: all of them at once, as above, spilled (64 drafts 48.7 us against 46.2)
          float4 x = load4(prow, j0, a.vocab, a.vec_p), y = load4(drow, j0, a.vocab, a.vec_d);
#pragma unroll 1
          for (int i = 1; i <= 4; ++i) {
            float4 nx = x, ny = y;
            if (i < 4) {
              nx = load4(prow, j0 + 128 * i, a.vocab, a.vec_p);
              ny = load4(drow, j0 + 128 * i, a.vocab, a.vec_d);
            }
            long long left[4];
            left_over<4>({x.x, x.y, x.z, x.w}, {y.x, y.y, y.z, y.w}, s_mass, refused, left);
            sum += left[0] + left[1] + left[2] + left[3];
            x = nx;
            y = ny;
          }
        }
        sum += units(hs, ls);
      }
      sum = warp_sum(sum);
      if (lane == 0) s_block[b] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      long long sum = 0;
      for (int b = b0 + lane; b < b1; b += 32) sum += s_block[b];
      sum = warp_sum(sum);
      // every CTA's sum to every CTA; the two buffers alternate, and a CTA is at most one pass ahead of another
      if (lane < C)
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(mapa_shared(smem_u32(&s_total[pass & 1][rank]), (uint32_t)lane)), "l"(sum)
                     : "memory");
    }
    cluster_arrive_all();
    cluster_wait_all();
    long long total = 0, before = 0;
    for (int r = 0; r < C; ++r) {
      const long long x = s_total[pass & 1][r];
      if (r < rank) before += x;
      total += x;
    }
    if (!empty && s_more) {  // the mass that the walk asked for
      __syncthreads();
      if (tid == 0) s_mass[refused] = min(total, 4 * kUnit - 1);
      __syncthreads();
      continue;
    }
    if (total == 0 && !empty && (refused > 0)) {  // nothing is left of the row
      empty = true;
      __syncthreads();
      continue;
    }
    // ---- the draw: the first entry whose running sum is above u total, by the CTA that holds it
    const float u = __ldg(a.u_end + s);
    const unsigned long long u64 = !(u > 0.f) ? 0ull : u >= 1.f ? ~0ull : (unsigned long long)((double)u * 18446744073709551616.0);
    const long long target = (long long)__umul64hi(u64, (unsigned long long)total);  // floor(u total)
    const long long mine = s_total[pass & 1][rank];
    if (total > 0 && target >= before && target < before + mine) {  // the same in all threads
      long long run = before;
      int b = b0;
      for (int base = b0; base < b1; base += 32) {  // 32 blocks at a time: the one in which the sum passes the target
        long long x = base + lane < b1 ? s_block[base + lane] : 0ll;
        const long long v = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        const unsigned m = __ballot_sync(0xffffffffu, run + x > target);
        if (m) {
          const int f = __ffs(m) - 1;
          b = base + f;
          run += __shfl_sync(0xffffffffu, x - v, f);
          break;
        }
        run += __shfl_sync(0xffffffffu, x, 31);
      }
      // the block's entries, two a thread (a warp alone takes microseconds over them: code that runs once is fetched as it runs)
      const int j = b * kBlock + 2 * tid;
      float f[2] = {0.f, 0.f}, g[2] = {0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if (j + q < a.vocab) f[q] = __ldg(prow + j + q);
        if (drow && j + q < a.vocab) g[q] = __ldg(drow + j + q);
      }
      long long w[2];
      left_over<2>(f, g, s_mass, drow ? refused : 0, w);
      for (int o = 0; o < out_n; ++o) {
        const int x = s_out[o] - j;
        if (x == 0) w[0] = 0;
        if (x == 1) w[1] = 0;
      }
      long long up = w[0] + w[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += y;
      }
      if (lane == 31) s_warp[warp] = up;
      __syncthreads();
      for (int i = 0; i < warp; ++i) run += s_warp[i];
      up += run;  // with this thread's entries; before them up - w0 - w1
      if (up > target && up - w[0] - w[1] <= target) a.next[s] = up - w[1] > target ? j : j + 1;
    }
    if (rank == 0) {
      const int n = s_n;
      for (int i = tid; i < n; i += kThreads) a.path[(size_t)s * a.path_cap + i] = s_path[i];
      if (tid == 0) {
        a.n_path[s] = n;
        if (total <= 0) a.next[s] = -1;  // a row without any mass
      }
    }
    break;
  }
}

}  // namespace

int verify_max_vocab() { return kMaxBlocks * kBlock; }

cudaError_t launch_tree_verify(const float* p, int64_t p_stride, const float* d, int64_t d_stride, int vocab, const int32_t* token,
                               const int32_t* parent, const float* u, const float* u_end, const int4* seqs, int n_seq, int n_tok,
                               int32_t* path, int path_cap, int32_t* n_path, int32_t* next, int* status, cudaStream_t stream) {
  auto vec = [](const float* x, int64_t stride) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && stride % 4 == 0; };
  const VerifyArgs a{p,     d,    p_stride, d_stride, vocab,  vec(p, p_stride), vec(d, d_stride), token, parent, u, u_end,
                     seqs,  n_seq, n_tok,   path,     n_path, next,             path_cap,         status};
  // CTAs a sequence: four on every SM of a GB300 where the sequences are few, and a block of entries a warp
  int C = 1;
  while (C < kMaxCluster && (long long)n_seq * C * 2 <= 4 * 152 && C * kWarps * kBlock < vocab) C *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(n_seq * C));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, tree_verify_kernel, a, C);
}

}  // namespace qsa
