// Cells of the int8 pool by index: qsa_cache_read gives them back as fp16 rows, qsa_cache_commit
// moves each sequence's accepted draft path to the front of its drafted cells.
//
// Both are copies bound by memory.  A cell is 1,056 bytes: codes of K and V for both groups (2 x 512
// bytes) and their scales (2 x 16 bytes).  Reading back 131,072 cells moves 407 MB in 68 us (6.0 TB/s, 0.88 of the
// measured copy); 2,051 cells 2.8 us, a launch; committing one sequence 2.2 us, 512 sequences 5.2 us.
#include "common.cuh"

namespace qsa {
namespace {

// A warp per cell: lane l holds 16 codes of the K row pair and 16 of V (dims 16 (l mod 16) of group
// l / 16), whose scale is entry l / 4 of the cell's eight, and writes 32 bytes of each fp16 row.
__global__ void __launch_bounds__(256) cache_read_kernel(const int8_t* __restrict__ kq, const __half* __restrict__ ksc,
                                                         const int8_t* __restrict__ vq, const __half* __restrict__ vsc,
                                                         int64_t n_pool, const int32_t* __restrict__ cells, int64_t n,
                                                         __half* __restrict__ k16, __half* __restrict__ v16,
                                                         int* status) {
  pdl_begin();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); i < n; i += warps) {
    const int cell = __ldg(cells + i);
    if (cell < 0 || cell >= n_pool) {  // warp-uniform
      if (cell != -1 && lane == 0) set_dev_status(status, QSA_DEV_BAD_ID);
      continue;
    }
    auto row = [&](const int8_t* codes, const __half* scales, __half* dst) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(codes + (size_t)cell * (kGroups * kD)) + lane);
      const __half2 s = __half2half2(scales[(size_t)cell * (kGroups * kNB) + (lane >> 2)]);
      uint32_t a[4], b[4];
      dequant8(w.x, w.y, s, a);
      dequant8(w.z, w.w, s, b);
      uint4* o = reinterpret_cast<uint4*>(dst + (size_t)i * (kGroups * kD) + lane * 16);
      o[0] = make_uint4(a[0], a[1], a[2], a[3]);
      o[1] = make_uint4(b[0], b[1], b[2], b[3]);
    };
    if (k16) row(kq, ksc, k16);
    if (v16) row(vq, vsc, v16);
  }
}

constexpr int kCommitPieces = 66;   // 16-byte pieces of a cell: 32 of K codes, 32 of V codes, two of scales
constexpr int kCommitThreads = 96;
constexpr int kCommitBatch = 8;     // pieces a thread loads before it stores any

// One CTA per sequence, one thread per 16-byte piece of a cell, walking the path in order.  The path
// is strictly ascending (checked first), so entry i names a cell at or behind its place i: a thread
// that loads entries i .. i + 7 before it stores them never reads a cell that an earlier store of its
// own has overwritten, and no two threads touch the same bytes.
__global__ void __launch_bounds__(kCommitThreads)
    cache_commit_kernel(int8_t* kq, __half* ksc, int8_t* vq, __half* vsc, int64_t n_pool, const int4* __restrict__ seqs,
                        const int32_t* __restrict__ path, const int32_t* __restrict__ n_path, int path_cap,
                        int* status) {
  pdl_begin();
  const int s = blockIdx.x, tid = threadIdx.x;
  const int4 e = __ldg(&seqs[s]);
  const int n = __ldg(&n_path[s]);
  if (n == 0 || e.y == 0) return;  // uniform: nothing accepted, or a padding sequence
  const int32_t* p = path + (size_t)s * path_cap;
  bool bad = n < 0 || n > path_cap || e.x < 0 || e.y < 0 || e.z < 0 || (int64_t)e.x + e.y > n_pool;
  if (!bad)
    for (int i = tid; i < n; i += kCommitThreads) {
      const int c = __ldg(p + i);
      bad |= c < 0 || (i > 0 && c <= __ldg(p + i - 1)) || (int64_t)e.z + c >= e.y;
    }
  if (__syncthreads_or(bad)) {
    if (tid == 0) set_dev_status(status, QSA_DEV_BAD_ID);
    return;
  }
  if (tid >= kCommitPieces) return;
  const size_t cell0 = (size_t)e.x + e.z;
  uint4* base;
  int stride, piece;  // 16-byte words of a cell in this thread's array, and its word of the cell
  if (tid < 64) {
    base = reinterpret_cast<uint4*>(tid < 32 ? kq : vq);
    stride = 32;
    piece = tid & 31;
  } else {
    base = reinterpret_cast<uint4*>(tid == 64 ? ksc : vsc);
    stride = 1;
    piece = 0;
  }
  for (int i0 = 0; i0 < n; i0 += kCommitBatch) {
    uint4 w[kCommitBatch];
#pragma unroll
    for (int u = 0; u < kCommitBatch; ++u)
      if (i0 + u < n) w[u] = base[(cell0 + __ldg(p + i0 + u)) * stride + piece];
#pragma unroll
    for (int u = 0; u < kCommitBatch; ++u)
      if (i0 + u < n) base[(cell0 + i0 + u) * stride + piece] = w[u];
  }
}

}  // namespace

cudaError_t launch_cache_read(const int8_t* kq, const __half* ksc, const int8_t* vq, const __half* vsc, int64_t n_pool,
                              const int32_t* cells, int64_t n, __half* k16, __half* v16, int* status,
                              cudaStream_t stream) {
  const int64_t want = (n + 7) / 8;
  const int grid = (int)(want < 152 * 32 ? want : 152 * 32);
  return launch_pdl(cache_read_kernel, dim3(grid), dim3(256), 0, stream, kq, ksc, vq, vsc, n_pool, cells, n, k16, v16,
                    status);
}

cudaError_t launch_cache_commit(int8_t* kq, __half* ksc, int8_t* vq, __half* vsc, int64_t n_pool, const int4* seqs,
                                int n_seq, const int32_t* path, const int32_t* n_path, int path_cap, int* status,
                                cudaStream_t stream) {
  return launch_pdl(cache_commit_kernel, dim3(n_seq), dim3(kCommitThreads), 0, stream, kq, ksc, vq, vsc, n_pool, seqs,
                    path, n_path, path_cap, status);
}

}  // namespace qsa
