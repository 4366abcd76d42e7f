// Operators that move cached rows without computing on them: whole-page copies (forks, copy on
// write, defragmentation) and the commit of a speculative step's accepted path.
//
// Both are bit copies inside the pool; what they cannot do without is one read and one write of
// every byte that moves (32 KiB a page; 2 KiB a token row and layer) and the index entries.
#include <cuda_runtime.h>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

// ---- kv_copy_pages ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;
constexpr int kCopyChunks = kHalfPageBytes / 16 / kCopyThreads;  // 16-byte chunks a thread moves: 4

// One CTA moves the K or the V half of one pair (16 KiB): 16384 pages take 158 us, 6.8 TB/s of reads and writes, the
// rate of one plain large copy; 512 take 5.4 us and 16, bound by the launch and two round trips, 2.2.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(
    uint8_t *__restrict__ k_base, uint8_t *__restrict__ v_base, long long page_stride, int num_pages,
    const int32_t *__restrict__ src_pages, const int32_t *__restrict__ dst_pages, int32_t *status) {
  griddep_launch_dependents();
  const long long pair = blockIdx.x >> 1;
  const int src = __ldg(src_pages + pair), dst = __ldg(dst_pages + pair);
  if (src < 0 || dst < 0) return;  // padding
  if (src >= num_pages || dst >= num_pages) {
    if (threadIdx.x == 0 && (blockIdx.x & 1) == 0) report(status, PKV_DEV_BAD_PAGE);
    return;
  }
  if (src == dst) return;
  uint8_t *base = (blockIdx.x & 1) ? v_base : k_base;
  const uint4 *from = reinterpret_cast<const uint4 *>(base + (long long)src * page_stride) + threadIdx.x;
  uint4 *to = reinterpret_cast<uint4 *>(base + (long long)dst * page_stride) + threadIdx.x;
  uint4 x[kCopyChunks];
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c) x[c] = from[c * kCopyThreads];
#pragma unroll
  for (int c = 0; c < kCopyChunks; ++c) to[c * kCopyThreads] = x[c];
}

// ---- tree_commit -----------------------------------------------------------------------------
constexpr int kCommitThreads = 2 * kKvHeads * (kRowBytes / 16);  // one thread per 16-byte chunk of a token: 128
constexpr int kCommitRows = 32;                                  // rows whose places are looked up at once
constexpr int kCommitBatch = 8;                                  // rows a thread has in flight

struct CommitArgs {
  uint8_t *k_base, *v_base;
  long long page_stride;
  int num_pages;
  const int32_t *block_tables;
  long long bt_stride, layer_stride;
  int num_layers;
  const int32_t *query_start, *context_lens, *accepted, *accept_counts;
  long long accepted_stride;
  int num_seqs, max_accept, max_context;
  int32_t *new_lens, *status;
};

// One CTA commits one (sequence, layer).  The places of up to 32 rows are looked up in parallel (path, then table
// entries: two round trips for all of them), then every thread moves one 16-byte chunk (K or V, head, chunk) of
// each row, the same chunk for every row.  The path is ascending, so path[k] >= k and path[k + 1] > path[k]: the rows
// a batch of loads reads all lie at or behind the rows its stores write, and every row a later batch reads lies
// behind them.  Each thread reads and writes its own chunk only, so loading a batch before storing it is all
// the ordering there is.
// What bounds it is latency: each CTA makes three dependent round trips (lengths, path and tables, rows), and a large batch
// is some three waves of CTAs that do so one after the other.  256 sequences x 16 layers with paths of up to 12 of 32
// nodes take 19.5 us (13.5 for the bytes; DRAM 37 %, issue slots 22 %, half the warps there), 64 with up to 8 take 4.1,
// one sequence 3.0.  (4 or 16 rows in flight: 19.4 and 23.5 us; two layers to a CTA: 20 us, and 4.4 for 64.)
__global__ void __launch_bounds__(kCommitThreads) tree_commit_kernel(const CommitArgs a) {
  __shared__ long long from[kCommitRows], to[kCommitRows];  // byte offsets in either half of the pool; to < 0: stays
  griddep_launch_dependents();
  const int s = int(blockIdx.x / unsigned(a.num_layers)), layer = int(blockIdx.x % unsigned(a.num_layers));
  const int tid = threadIdx.x;
  const int n = __ldg(a.query_start + s + 1) - __ldg(a.query_start + s);
  const int ctx = __ldg(a.context_lens + s), count = __ldg(a.accept_counts + s);
  const int base = ctx - n;
  const int32_t *path = a.accepted + (long long)s * a.accepted_stride;
  if (n < 0 || ctx < 0 || ctx > a.max_context || n > ctx) {
    if (layer == 0 && tid == 0) {
      report(a.status, PKV_DEV_BAD_CONTEXT);
      if (a.new_lens != nullptr) a.new_lens[s] = ctx;
    }
    return;
  }
  bool bad = count < 0 || count > n || count > a.max_accept;
  if (!bad)
    for (int k = tid; k < count; k += kCommitThreads) {
      const int p = __ldg(path + k);
      bad |= p >= n || p <= (k > 0 ? __ldg(path + k - 1) : -1);
    }
  bad = __syncthreads_or(bad) != 0;
  if (layer == 0 && tid == 0) {
    if (bad) report(a.status, PKV_DEV_BAD_PATH);
    if (a.new_lens != nullptr) a.new_lens[s] = bad ? ctx : base + count;
  }
  if (bad) return;
  const int32_t *table = a.block_tables + (long long)s * a.bt_stride + (long long)layer * a.layer_stride;
  const int is_v = tid / (kCommitThreads / 2), g = (tid / 8) % kKvHeads, c = tid % 8;
  uint8_t *half = (is_v ? a.v_base : a.k_base) + g * kPageTokens * kRowBytes + c * 16;
  for (int k0 = 0; k0 < count; k0 += kCommitRows) {
    const int rows = min(kCommitRows, count - k0);
    if (k0 > 0) __syncthreads();  // (the places before have been used)
    if (tid < rows) {
      const int k = k0 + tid, p = __ldg(path + k);
      to[tid] = -1;
      if (p != k) {
        const int src = base + p, dst = base + k;
        const int src_page = __ldg(table + src / kPageTokens), dst_page = __ldg(table + dst / kPageTokens);
        if (src_page < 0 || src_page >= a.num_pages || dst_page < 0 || dst_page >= a.num_pages) {
          report(a.status, PKV_DEV_BAD_PAGE);
        } else {
          from[tid] = src_page * a.page_stride + (src % kPageTokens) * kRowBytes;
          to[tid] = dst_page * a.page_stride + (dst % kPageTokens) * kRowBytes;
        }
      }
    }
    __syncthreads();
    for (int r0 = 0; r0 < rows; r0 += kCommitBatch) {
      uint4 x[kCommitBatch];
#pragma unroll
      for (int j = 0; j < kCommitBatch; ++j)
        if (r0 + j < rows && to[r0 + j] >= 0) x[j] = *reinterpret_cast<const uint4 *>(half + from[r0 + j]);
#pragma unroll
      for (int j = 0; j < kCommitBatch; ++j)
        if (r0 + j < rows && to[r0 + j] >= 0) *reinterpret_cast<uint4 *>(half + to[r0 + j]) = x[j];
    }
  }
}

// Whether [p, p + np) and [q, q + nq) share a byte (element counts of int32).
bool overlap32(const void *p, long long np, const void *q, long long nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + uintptr_t(nq) * 4u && b < a + uintptr_t(np) * 4u;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_kv_copy_pages(const pkv_pool *pool, const int32_t *src_pages, const int32_t *dst_pages,
                                 int num_copies, int32_t *device_status, void *stream) {
  const int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_copies < 0 || num_copies > 0x3fffffff) return PKV_ERR_SHAPE;
  if (num_copies == 0) return PKV_OK;
  if (src_pages == nullptr || dst_pages == nullptr) return PKV_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(src_pages) & 3u) || (reinterpret_cast<uintptr_t>(dst_pages) & 3u))
    return PKV_ERR_ALIGN;
  pkv::kv_copy_pages_kernel<<<unsigned(num_copies) * 2u, pkv::kCopyThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint8_t *>(pool->k_base), static_cast<uint8_t *>(pool->v_base), pool->page_stride_bytes,
      pool->num_pages, src_pages, dst_pages, device_status);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}

extern "C" int pkv_tree_commit(const pkv_pool *pool, const int32_t *block_tables, int64_t block_table_stride,
                               int64_t layer_stride, int num_layers, const int32_t *query_start,
                               const int32_t *context_lens, const int32_t *accepted, int64_t accepted_stride,
                               const int32_t *accept_counts, int num_seqs, int max_accept, int max_context,
                               int32_t *new_context_lens, int32_t *device_status, void *stream) {
  const int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_seqs < 0 || num_layers < 1 || max_accept < 0 || max_context < 0 || block_table_stride < 0 ||
      layer_stride < 0 || accepted_stride < max_accept || (long long)num_seqs * num_layers > 0x7fffffffLL)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  if (block_tables == nullptr || query_start == nullptr || context_lens == nullptr || accept_counts == nullptr ||
      (accepted == nullptr && max_accept > 0))
    return PKV_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(query_start) |
       reinterpret_cast<uintptr_t>(context_lens) | reinterpret_cast<uintptr_t>(accepted) |
       reinterpret_cast<uintptr_t>(accept_counts) | reinterpret_cast<uintptr_t>(new_context_lens)) & 3u)
    return PKV_ERR_ALIGN;
  // every layer's CTA of a sequence reads the lengths and the path while layer 0's writes the new lengths
  if (new_context_lens != nullptr &&
      (pkv::overlap32(new_context_lens, num_seqs, context_lens, num_seqs) ||
       pkv::overlap32(new_context_lens, num_seqs, query_start, (long long)num_seqs + 1) ||
       pkv::overlap32(new_context_lens, num_seqs, accept_counts, num_seqs) ||
       pkv::overlap32(new_context_lens, num_seqs, accepted, (num_seqs - 1) * accepted_stride + max_accept)))
    return PKV_ERR_SHAPE;
  pkv::CommitArgs a;
  a.k_base = static_cast<uint8_t *>(pool->k_base);
  a.v_base = static_cast<uint8_t *>(pool->v_base);
  a.page_stride = pool->page_stride_bytes;
  a.num_pages = pool->num_pages;
  a.block_tables = block_tables;
  a.bt_stride = block_table_stride;
  a.layer_stride = layer_stride;
  a.num_layers = num_layers;
  a.query_start = query_start;
  a.context_lens = context_lens;
  a.accepted = accepted;
  a.accept_counts = accept_counts;
  a.accepted_stride = accepted_stride;
  a.num_seqs = num_seqs;
  a.max_accept = max_accept;
  a.max_context = max_context;
  a.new_lens = new_context_lens;
  a.status = device_status;
  pkv::tree_commit_kernel<<<unsigned(num_seqs * num_layers), pkv::kCommitThreads, 0,
                            static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
