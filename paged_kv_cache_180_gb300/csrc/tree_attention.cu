// Attention of a tree of drafted tokens per sequence over its paged K/V.
//
//   out[i][h] = sum_{t in A_i} softmax_t(scale * q[i][h] . K_t[h/4]) V_t[h/4],
//   A_i = the committed prefix (t < base_s) and the nodes base_s + j whose bit j is set in row i's mask
//
// One pass over a sequence's pages with the running maximum and sum of the softmax; a masked key is
// skipped, so whatever its K and V hold (NaN included) never meets a row that may not see it.
//
// One CTA = (sequence, K/V head, 4 nodes): the 16 rows (4 nodes x 4 query heads) share each page's
// K and V rows, staged in shared memory.  Eight threads share a row, 8 dims each.
#include <cuda_runtime.h>

#include <math.h>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kTreeTok = 32;                      // nodes per tile of the workspace's accounting
constexpr int kTreeRows = kTreeTok * kGroup;
constexpr int kTreeMaxCtas = 320;
constexpr size_t kTreeSlotBytes = size_t(kTreeRows) * (kHeadDim + 2) * sizeof(float);
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kSimpleNodes = 4;
constexpr int kSimpleThreads = 128;

struct TreeArgs {
  const uint8_t *k_base, *v_base;
  long long page_stride;
  int num_pages;
  void *out;
  const uint16_t *q;
  int num_q_rows;
  const int32_t *query_start;
  const uint32_t *mask;
  long long mask_stride;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int num_seqs, max_query, max_context;
  float scale_log2;
  int out_bf16;
  int32_t *status;
};

__global__ void __launch_bounds__(kSimpleThreads) tree_attention_kernel(const TreeArgs a) {
  __shared__ uint4 ks[kPageTokens * 8], vs[kPageTokens * 8];
  const int tid = threadIdx.x;
  const int s = int(blockIdx.x), g = int(blockIdx.y), j0 = int(blockIdx.z) * kSimpleNodes;
  const int q0 = __ldg(a.query_start + s), n = __ldg(a.query_start + s + 1) - q0, ctx = __ldg(a.context_lens + s);
  const bool bad = n < 0 || n > a.max_query || ctx < 0 || ctx > a.max_context || n > ctx || q0 < 0 ||
                   q0 > a.num_q_rows - n;
  if (bad && g == 0 && j0 == 0 && tid == 0 && n != 0) report(a.status, PKV_DEV_BAD_CONTEXT);
  const int r = tid >> 3, c = tid & 7, node = j0 + (r >> 2), h = g * kGroup + (r & 3);
  auto write = [&](long long row, const float (&o)[8]) {
    const long long at = (row * kQHeads + h) * kHeadDim + c * 8;
    if (a.out_bf16) {
      *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) =
          make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]), pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    } else {
      float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
      dst[0] = make_float4(o[0], o[1], o[2], o[3]);
      dst[1] = make_float4(o[4], o[5], o[6], o[7]);
    }
  };
  if (bad) {
    const float zero[8] = {};
    for (long long j = node; j < n; j += (long long)gridDim.z * kSimpleNodes) {
      const long long row = (long long)q0 + j;
      if (row >= 0 && row < a.num_q_rows) write(row, zero);
    }
    return;
  }
  if (j0 >= n) return;
  const bool real = node < n;
  const int base = ctx - n;
  float q[8], o[8];
  {
    const uint4 x = real ? *reinterpret_cast<const uint4 *>(a.q + ((long long)(q0 + node) * kQHeads + h) * kHeadDim + c * 8)
                         : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      q[2 * i] = bf16_lo(w[i]);
      q[2 * i + 1] = bf16_hi(w[i]);
      o[2 * i] = o[2 * i + 1] = 0.f;
    }
  }
  const uint32_t *mask = a.mask + (long long)(q0 + (real ? node : 0)) * a.mask_stride;
  const int32_t *table = a.block_tables + (long long)s * a.bt_stride;
  float m = -INFINITY, l = 0.f;
  for (int p = 0; p * kPageTokens < ctx; ++p) {
    const int page = __ldg(table + p);
    if (page < 0 || page >= a.num_pages) {
      if (tid == 0) report(a.status, PKV_DEV_BAD_PAGE);
      continue;
    }
    const long long at = (long long)page * a.page_stride + g * kPageTokens * kRowBytes;
    __syncthreads();
    ks[tid] = reinterpret_cast<const uint4 *>(a.k_base + at)[tid];
    vs[tid] = reinterpret_cast<const uint4 *>(a.v_base + at)[tid];
    __syncthreads();
    for (int t = 0; t < kPageTokens && p * kPageTokens + t < ctx; ++t) {
      const uint4 kx = ks[t * 8 + c];
      const uint32_t kw[4] = {kx.x, kx.y, kx.z, kx.w};
      float x = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) x += q[2 * i] * bf16_lo(kw[i]) + q[2 * i + 1] * bf16_hi(kw[i]);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      const int j = p * kPageTokens + t - base;
      if (j >= 0 && !((__ldg(mask + (j >> 5)) >> (j & 31)) & 1u)) continue;
      x *= a.scale_log2;
      const float mn = fmaxf(m, x), keep = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(x - mn);
      m = mn;
      l = l * keep + w;
      const uint4 vx = vs[t * 8 + c];
      const uint32_t vw[4] = {vx.x, vx.y, vx.z, vx.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[2 * i] = o[2 * i] * keep + w * bf16_lo(vw[i]);
        o[2 * i + 1] = o[2 * i + 1] * keep + w * bf16_hi(vw[i]);
      }
    }
  }
  if (!real) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] *= inv;
  write((long long)q0 + node, o);
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int num_seqs, int max_query, int num_q_heads, int head_dim) {
  if (num_seqs < 0 || max_query < 0 || num_q_heads != pkv::kQHeads || head_dim != pkv::kHeadDim) return 0;
  const size_t tiles = (size_t(max_query) + pkv::kTreeTok - 1) / pkv::kTreeTok;
  const size_t counters = (size_t(num_seqs) * tiles * pkv::kKvHeads * sizeof(int32_t) + 127) / 128 * 128;
  return counters + 2 * size_t(pkv::kTreeMaxCtas) * pkv::kTreeSlotBytes;
}

extern "C" int pkv_paged_tree_attention(const pkv_pool *pool, void *out, const void *q, int num_q_heads,
                                        int num_q_rows, const int32_t *query_start, const uint32_t *tree_mask,
                                        int64_t mask_stride, const int32_t *block_tables, int64_t block_table_stride,
                                        const int32_t *context_lens, int num_seqs, int max_query, int max_context,
                                        float scale, void *workspace, size_t workspace_bytes, int32_t *device_status,
                                        unsigned flags, void *stream) {
  if (flags & ~unsigned(PKV_OVERLAP_PREVIOUS | PKV_OUT_BF16)) return PKV_ERR_SHAPE;
  const int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_q_heads != pkv::kQHeads) return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || max_query < 0 || max_context < 0 || block_table_stride < 0 || num_q_rows < 0 ||
      mask_stride < 0 || mask_stride > (1 << 24) || mask_stride * 32 < max_query)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || max_query == 0 || num_q_rows == 0) return PKV_OK;
  const long long tiles = (max_query + pkv::kSimpleNodes - 1) / pkv::kSimpleNodes;
  if (tiles > 65535) return PKV_ERR_SHAPE;
  if (out == nullptr || q == nullptr || query_start == nullptr || tree_mask == nullptr || block_tables == nullptr ||
      context_lens == nullptr || workspace == nullptr)
    return PKV_ERR_NULL;
  if (!isfinite(scale)) return PKV_ERR_SCALE;
  if (!pkv::aligned16(q) || !pkv::aligned16(out) || !pkv::aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(query_start) | reinterpret_cast<uintptr_t>(tree_mask) |
        reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens)) & 3u))
    return PKV_ERR_ALIGN;
  if (workspace_bytes < pkv_tree_workspace_bytes(num_seqs, max_query, num_q_heads, pkv::kHeadDim))
    return PKV_ERR_WORKSPACE;
  pkv::TreeArgs a;
  a.k_base = static_cast<const uint8_t *>(pool->k_base);
  a.v_base = static_cast<const uint8_t *>(pool->v_base);
  a.page_stride = pool->page_stride_bytes;
  a.num_pages = pool->num_pages;
  a.out = out;
  a.q = static_cast<const uint16_t *>(q);
  a.num_q_rows = num_q_rows;
  a.query_start = query_start;
  a.mask = tree_mask;
  a.mask_stride = mask_stride;
  a.block_tables = block_tables;
  a.bt_stride = block_table_stride;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.max_query = max_query;
  a.max_context = max_context;
  a.scale_log2 = scale * pkv::kLog2e;
  a.out_bf16 = (flags & PKV_OUT_BF16) ? 1 : 0;
  a.status = device_status;
  const dim3 grid(unsigned(num_seqs), pkv::kKvHeads, unsigned(tiles));
  pkv::tree_attention_kernel<<<grid, pkv::kSimpleThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_LAUNCH;
}
