// Runs of cells of the int8 pool moved as they are: qsa_cache_copy (forks) and qsa_cache_compact (the runs of a
// server's tables put side by side at the front of the pool, in place).
//
// Both are copies bound by memory: a cell is 1,056 bytes (K and V codes, 512 bytes each, and their scales, 16 bytes
// each), read once and written once.  A warp takes eight cells, all loaded into registers before any is stored: 17 loads of
// 16 bytes a lane in flight.  Measured (GB300): 96 runs of 40-3,000 cells 45 us, 6.2 TB/s of the 278 MB read and written, 0.92 of a
// plain copy's rate; 500 runs compacted, 461 MB, 89 us, 5.2 TB/s (flags and the look-up of runs cost the rest); 3 runs of 500 5 us
// and 8 runs 7-8 us are the latency of one and two launches.
#include <algorithm>

#include "tree_common.cuh"

namespace qsa {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kCopyCells = 8, kMoveCells = 8;  // cells that a warp of a copy and of a compaction holds at once
constexpr int kCopyChunk = kWarps * kCopyCells, kMoveChunk = kWarps * kMoveCells;  // and a CTA

struct Pool {
  int8_t* kq;
  __half* ksc;
  int8_t* vq;
  __half* vsc;
};

// N cells in registers: codes of K and V by all lanes (16 bytes each), scales by the first 2 N lanes (lane 2 u: K of
// cell u, 2 u + 1: V).  Cell u of the warp is `from` of lane u; negative: none.
template <int N>
struct Cells {
  uint4 k[N], v[N], s;
};
template <int N>
__device__ __forceinline__ void load_cells(const Pool& p, int64_t from, int lane, Cells<N>& c) {
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int64_t x = __shfl_sync(0xffffffffu, from, u);
    if (x < 0) continue;  // warp-uniform
    c.k[u] = reinterpret_cast<const uint4*>(p.kq)[x * 32 + lane];
    c.v[u] = reinterpret_cast<const uint4*>(p.vq)[x * 32 + lane];
  }
  const int64_t y = __shfl_sync(0xffffffffu, from, (lane >> 1) & (N - 1));
  if (lane < 2 * N && y >= 0) c.s = reinterpret_cast<const uint4*>(lane & 1 ? p.vsc : p.ksc)[y];
}
template <int N>
__device__ __forceinline__ void store_cells(const Pool& p, int64_t to, int lane, const Cells<N>& c) {
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const int64_t x = __shfl_sync(0xffffffffu, to, u);
    if (x < 0) continue;
    reinterpret_cast<uint4*>(p.kq)[x * 32 + lane] = c.k[u];
    reinterpret_cast<uint4*>(p.vq)[x * 32 + lane] = c.v[u];
  }
  const int64_t y = __shfl_sync(0xffffffffu, to, (lane >> 1) & (N - 1));
  if (lane < 2 * N && y >= 0) reinterpret_cast<uint4*>(lane & 1 ? p.vsc : p.ksc)[y] = c.s;
}

// ---------------------------------------------------------------- copy
// blockIdx.y takes kSliceRuns runs of the table, whose lengths it sums up in shared memory, and the CTAs of a slice
// share its cells evenly, wherever a run begins or ends.
constexpr int kSliceRuns = 1024, kRunsPerThread = kSliceRuns / kThreads;
__global__ void __launch_bounds__(kThreads)
    cache_copy_kernel(const Pool pool, int64_t n_pool, const int4* __restrict__ runs, int n_run, int max_cells, int* status) {
  __shared__ int64_t s_end[kSliceRuns];  // cells up to and with a run
  __shared__ int2 s_at[kSliceRuns];      // source, destination
  __shared__ int64_t s_sum[kWarps];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r0 = blockIdx.y * kSliceRuns, n = min(kSliceRuns, n_run - r0);
  int64_t len[kRunsPerThread], sum = 0;
#pragma unroll
  for (int i = 0; i < kRunsPerThread; ++i) {
    const int r = tid * kRunsPerThread + i;
    int4 e = make_int4(0, 0, 0, 0);
    if (r < n) e = __ldg(&runs[r0 + r]);
    const bool ok = e.x >= 0 && e.y >= 0 && e.z >= 0 && e.z <= max_cells && (int64_t)e.x + e.z <= n_pool &&
                    (int64_t)e.y + e.z <= n_pool;
    if (!ok && blockIdx.x == 0) set_dev_status(status, QSA_DEV_BAD_ID);
    len[i] = ok ? e.z : 0;
    sum += len[i];
    s_at[r] = make_int2(e.x, e.y);
  }
  int64_t x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int64_t at = x - sum;
  for (int i = 0; i < warp; ++i) at += s_sum[i];
#pragma unroll
  for (int i = 0; i < kRunsPerThread; ++i) {
    at += len[i];
    s_end[tid * kRunsPerThread + i] = at;
  }
  __syncthreads();
  const int64_t total = s_end[kSliceRuns - 1];
  for (int64_t c0 = (int64_t)blockIdx.x * kCopyChunk + warp * kCopyCells; c0 < total; c0 += (int64_t)gridDim.x * kCopyChunk) {
    const int64_t c = c0 + (lane & (kCopyCells - 1));
    int64_t from = -1, to = -1;
    if (c < total) {  // the first run that ends behind c
      int lo = 0, hi = kSliceRuns - 1;
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_end[mid] > c) hi = mid;
        else lo = mid + 1;
      }
      const int64_t in = c - (lo ? s_end[lo - 1] : 0);
      from = s_at[lo].x + in;
      to = s_at[lo].y + in;
    }
    Cells<kCopyCells> w;
    load_cells(pool, from, lane, w);
    store_cells(pool, to, lane, w);
  }
}

// ---------------------------------------------------------------- compaction
// Two launches.  The first ranks the runs by their first cell: a run's place is the number of cells of the runs
// before it, by comparing all pairs of runs (500 runs 2 us; no sort, and any order of the table).  The second moves
// the cells, in place and in one pass: cells only move down, so the places [a, b) of a chunk are the source of
// cells of this chunk and of earlier ones alone.  CTAs take chunks in order by a ticket, load theirs, say so by
// a flag, wait for the flags of the (at most two) earlier chunks that read from [a, b), and store.  A chunk's load
// waits for nothing, and earlier chunks are held by CTAs that run already, so every wait ends.
struct CompactWs {
  int4* runs;           // by rank: first cell, first cell to be, cells, 0
  int* place;           // by table entry: the first cell to be
  int* bad;             // by rank CTA: it saw a bad entry
  int* head;            // [0] next ticket, [1] runs, [2] cells in all
  uint32_t* loaded;     // by chunk
  size_t bytes;
};
constexpr int kRankEntries = kWarps;  // entries of a rank CTA, a warp each

CompactWs compact_ws(void* ws, int64_t n_pool, int n) {
  CompactWs w{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += (bytes + 255) / 256 * 256;
    return static_cast<uint8_t*>(ws) + at;
  };
  w.runs = reinterpret_cast<int4*>(take((size_t)n * sizeof(int4)));
  w.place = reinterpret_cast<int*>(take((size_t)n * sizeof(int)));
  w.bad = reinterpret_cast<int*>(take((size_t)((n + kRankEntries - 1) / kRankEntries) * sizeof(int)));
  w.head = reinterpret_cast<int*>(take(4 * sizeof(int)));
  w.loaded = reinterpret_cast<uint32_t*>(take((size_t)((n_pool + kMoveChunk - 1) / kMoveChunk) * sizeof(uint32_t)));
  w.bytes = o;
  return w;
}

struct Tables {
  const int4* prefixes;
  const int4* seqs;
  int n_prefix, n;  // entries of the first, and of both
  __device__ __forceinline__ int4 at(int i) const { return i < n_prefix ? __ldg(&prefixes[i]) : __ldg(&seqs[i - n_prefix]); }
};

__global__ void __launch_bounds__(kThreads) compact_rank_kernel(const Tables t, int64_t n_pool, const CompactWs w) {
  __shared__ int2 s_run[kThreads];
  pdl_begin();
  const int tid = threadIdx.x;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + tid; i < (n_pool + kMoveChunk - 1) / kMoveChunk; i += (int64_t)gridDim.x * kThreads)
    w.loaded[i] = 0u;
  const int i = blockIdx.x * kRankEntries + tid / 32, part = tid & 31;
  const int4 e = i < t.n ? t.at(i) : make_int4(0, 0, 0, 0);
  bool bad = e.x < 0 || e.y < 0 || (int64_t)e.x + e.y > n_pool;
  int64_t before = 0, all = 0;
  int rank = 0, count = 0;
  for (int j0 = 0; j0 < t.n; j0 += kThreads) {
    __syncthreads();
    int2 r = make_int2(0, 0);
    if (j0 + tid < t.n) {
      const int4 f = t.at(j0 + tid);
      r = make_int2(f.x, f.y);
    }
    s_run[tid] = r;
    __syncthreads();
    const int n = min(kThreads, t.n - j0);
    for (int k = part; k < n; k += 32) {
      const int2 f = s_run[k];
      if (f.y <= 0) continue;  // an entry without cells; one with fewer is found by its own threads
      all += f.y;
      ++count;
      if (f.x < e.x || (f.x == e.x && j0 + k < i)) {  // (of the same cell only where one of the two is empty)
        before += f.y;
        ++rank;
      }
      // another run with this one's first cell in it: the tables overlap
      bad |= e.y > 0 && j0 + k != i && f.x <= e.x && (int64_t)f.x + f.y > e.x;
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    all += __shfl_xor_sync(0xffffffffu, all, o);
    rank += __shfl_xor_sync(0xffffffffu, rank, o);
    count += __shfl_xor_sync(0xffffffffu, count, o);
  }
  if (part == 0 && i < t.n) {
    w.place[i] = (int)before;
    // sums of a broken table may be anything: what is stored is then not used
    if (e.y > 0) w.runs[rank] = make_int4(e.x, (int)before, e.y, 0);
    if (i == 0) {
      w.head[0] = 0;
      w.head[1] = count;
      w.head[2] = (int)all;
    }
  }
  const int any = __syncthreads_or(bad);
  if (tid == 0) w.bad[blockIdx.x] = any;
}

constexpr unsigned long long kFlagBudgetNs = 2000000000ull;
__device__ __forceinline__ bool wait_loaded(const uint32_t* flag, int* status) {
  unsigned long long t0 = 0;
  for (unsigned it = 0;; ++it) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v) return true;
    if ((it & 255u) == 255u) {
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kFlagBudgetNs) break;
    }
  }
  set_dev_status(status, QSA_DEV_WAIT_TIMEOUT);
  return false;
}

constexpr int kNearRuns = 1024;  // a table up to so long is looked up in shared memory
// on an SM (measured with a relaxed flag, 500 runs: 84 us; 3 of them, spilled, 105; with four cells a warp 4 CTAs 92, 5 97)
constexpr int kMoveCtas = 2;
__global__ void __launch_bounds__(kThreads, kMoveCtas)
    compact_move_kernel(const Pool pool, const Tables t, const CompactWs w, int rank_ctas, int4* prefixes_out, int4* seqs_out,
                        int* used_out, int* status) {
  __shared__ int4 s_runs[kNearRuns];
  __shared__ int s_next, s_wait[2];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_next = atomicAdd(&w.head[0], 1);
  const int n = __ldg(&w.head[1]), used = __ldg(&w.head[2]);
  bool bad = false;
  for (int i = tid; i < rank_ctas; i += kThreads) bad |= __ldg(&w.bad[i]) != 0;
  bad = __syncthreads_or(bad);
  for (int i = blockIdx.x * kThreads + tid; i < t.n; i += gridDim.x * kThreads) {
    int4 e = i < t.n_prefix ? t.prefixes[i] : t.seqs[i - t.n_prefix];
    if (!bad) e.x = __ldg(&w.place[i]);
    if (i < t.n_prefix) prefixes_out[i] = e;
    else seqs_out[i - t.n_prefix] = e;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (bad) set_dev_status(status, QSA_DEV_BAD_ID);
    if (used_out) *used_out = bad ? -1 : used;
  }
  if (bad) return;  // the pool is left as it is
  const int4* runs = w.runs;
  if (n <= kNearRuns) {
    for (int i = tid; i < n; i += kThreads) s_runs[i] = __ldg(&w.runs[i]);
    runs = s_runs;
    __syncthreads();
  }
  // Where this warp's cells of a chunk come from and go to (lane u: cell u; -1: none).
  auto look_up = [&](int chunk, int64_t& from, int64_t& to) {
    from = to = -1;
    const int64_t c0 = (int64_t)chunk * kMoveChunk + warp * kMoveCells;
    if (c0 >= used) return;
    const int k = warp_find_seq(n, c0, [&](int i) { return (long long)runs[i].y; });
    const int4 e = runs[min(k + lane, n - 1)];  // the run of cell c0, and with a lane each those behind it (no run is empty)
    const bool have = k + lane < n;
#pragma unroll
    for (int u = 0; u < kMoveCells; ++u) {
      const int c = (int)c0 + u;
      const int r = max(__popc(__ballot_sync(0xffffffffu, have && e.y <= c)) - 1, 0);
      const int src = __shfl_sync(0xffffffffu, e.x, r), dst = __shfl_sync(0xffffffffu, e.y, r);
      if (lane == u && c < used) {
        to = c;
        from = src + (c - dst);
      }
    }
  };
  int chunk = s_next;
  int64_t from, to;
  look_up(chunk, from, to);
  while ((int64_t)chunk * kMoveChunk < used) {
    __syncthreads();  // every thread has read s_next
    if (tid == 0) s_next = atomicAdd(&w.head[0], 1);
    const bool moves = __syncthreads_or(from != to);  // else every cell is where it belongs, and none is read
    Cells<kMoveCells> x;
    if (moves) load_cells(pool, from, lane, x);
    // while they arrive: the next chunk's runs, and whom this one waits for
    const int next = s_next;
    int64_t next_from, next_to;
    look_up(next, next_from, next_to);
    if (warp == 0 && moves) {
      // the earlier chunks that read from places [a, b): of the first and the last cell there that is in a run
      const int a = chunk * kMoveChunk, b = min(a + kMoveChunk, used);
      auto src = [&](int i) { return (long long)runs[i].x; };
      const int ka = warp_find_seq(n, a, src), kb = warp_find_seq(n, b - 1, src);
      if (lane == 0) {
        const int4 ea = runs[ka], eb = runs[kb];
        // cell a is in run ka, or the first cell behind it is a run's first: the next one's, or (before all of them) run 0's
        const int xa = a >= ea.x && a - ea.x < ea.z ? ea.y + (a - ea.x) : ea.x > a ? ea.y : ea.y + ea.z;
        const int xb = eb.x > b - 1 ? -1 : eb.y + min(b - 1 - eb.x, eb.z - 1);
        s_wait[0] = xa / kMoveChunk;
        s_wait[1] = xb < 0 ? -1 : xb / kMoveChunk;
      }
    }
    // The flag says that every thread's loads are behind it.  Only a release orders a load before a store of another SM: it
    // waits for this CTA's earlier stores as well (500 runs 89 us; with a relaxed flag behind a use of every loaded word 86, and
    // nothing in the memory model that keeps the loads before it).
    __syncthreads();
    if (tid == 0) asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(w.loaded + chunk), "r"(1u) : "memory");
    if (moves) {
      bool ok = true;
      const int j = s_wait[0] + tid;
      if (j <= s_wait[1] && j < chunk) ok = wait_loaded(w.loaded + j, status);
      if (!__syncthreads_and(ok)) return;
      store_cells(pool, to == from ? -1 : to, lane, x);
    }
    chunk = next;
    from = next_from;
    to = next_to;
  }
}

}  // namespace

cudaError_t launch_cache_copy(int8_t* kq, __half* ksc, int8_t* vq, __half* vsc, int64_t n_pool, const int4* runs, int n_run,
                              int max_cells, int* status, cudaStream_t stream) {
  const int slices = (n_run + kSliceRuns - 1) / kSliceRuns;
  const int64_t most = ((int64_t)std::min(n_run, kSliceRuns) * max_cells + kCopyChunk - 1) / kCopyChunk;
  const int64_t want = std::max<int64_t>(1, 152 * 4 / slices);
  return launch_pdl(cache_copy_kernel, dim3((unsigned)std::min(most, want), slices), dim3(kThreads), 0, stream,
                    Pool{kq, ksc, vq, vsc}, n_pool, runs, n_run, max_cells, status);
}

size_t cache_compact_workspace_bytes(int64_t n_pool, int n) { return compact_ws(nullptr, n_pool, n).bytes; }

cudaError_t launch_cache_compact(int8_t* kq, __half* ksc, int8_t* vq, __half* vsc, int64_t n_pool, const int4* prefixes,
                                 int n_prefix, const int4* seqs, int n_seq, int4* prefixes_out, int4* seqs_out, int* used,
                                 void* ws, int* status, cudaStream_t stream) {
  const Tables t{prefixes, seqs, n_prefix, n_prefix + n_seq};
  const CompactWs w = compact_ws(ws, n_pool, t.n);
  const int ranks = (t.n + kRankEntries - 1) / kRankEntries;
  cudaError_t e = launch_pdl(compact_rank_kernel, dim3(ranks), dim3(kThreads), 0, stream, t, n_pool, w);
  if (e != cudaSuccess) return e;
  const int64_t chunks = (n_pool + kMoveChunk - 1) / kMoveChunk;
  return launch_pdl(compact_move_kernel, dim3((unsigned)std::min<int64_t>(chunks, 152 * kMoveCtas)), dim3(kThreads), 0, stream,
                    Pool{kq, ksc, vq, vsc}, t, w, ranks, prefixes_out, seqs_out, used, status);
}

}  // namespace qsa
