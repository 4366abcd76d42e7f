// Eviction: per sequence, layer and K/V head the cached tokens with the largest weight sums are kept, with the first few
// and the most recent ones, and their rows move together at the front of the sequence, in order and in place.
//
// What is kept of ctx tokens with B = min(budget, ctx):  the first a = min(sinks, B), the last r = min(recent, B - a), and of
// the tokens between them the B - a - r with the largest sums; of equal sums the earlier token.
//
// A unit is one (sequence, layer, K/V head); it belongs to one CTA or one cluster of CTAs.
//  * Selection: sums are mapped to 32-bit keys of the same order and the key of rank B - a - r is found digit by digit from
//    the top (8 bits a pass, a histogram in shared memory, summed over the cluster); the passes end early once a digit's
//    bin is needed whole.  Then every warp counts what its share of the tokens keeps, in order, and writes the kept
//    positions, ascending.
//  * Moving: kept[k] >= k, ascending, so the rows that round i of the move writes (positions i R .. (i + 1) R - 1) lie at or
//    before everything that later rounds read, and a barrier between a round's loads and its stores is all the order there
//    has to be.  A row's K and V (2 x 128 B) are moved by 16 threads, 16 bytes each; the next round's places are
//    looked up while this round's loads are under way.
#include <cuda_runtime.h>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvMaxCluster = 8;
constexpr int kEvRows = 128;                                  // rows of a round and CTA
constexpr int kEvChunks = 2 * kRowBytes / 16;                 // 16-byte chunks of a row's K and V: 16
constexpr int kEvLoads = kEvRows * kEvChunks / kEvThreads;    // chunks a thread has in flight: 8
constexpr int kDigitBits = 8, kBins = 1 << kDigitBits;
static_assert(kBins == kEvThreads, "a thread owns one bin");

struct EvictArgs {
  uint8_t *k_base, *v_base;
  long long page_stride;
  int num_pages;
  const int32_t *block_tables;
  long long bt_stride, layer_stride;
  int num_layers;
  const int32_t *context_lens, *budgets;
  int max_context, max_budget, sinks, recent;
  const float *sums;
  float *new_sums;
  long long sums_seq, sums_layer, sums_head;
  int32_t *kept;
  long long kept_stride;
  int32_t *new_lens, *status;
  int cluster;
};

struct EvictSmem {
  unsigned hist[2][kBins];
  int warp_part[kEvWarps];
  int2 warp_count[kEvWarps];          // (kept for certain, equal to the threshold) of a warp's share
  int2 rank_count[kEvMaxCluster];     // the same of every CTA of the cluster
  long long from[2][kEvRows], to[2][kEvRows];  // byte offsets of a round's rows in either half of the pool; from < 0: stays
  unsigned digit, need;
  int whole;
};

// Order-preserving map of a sum to 32 bits: NaN below everything, the two zeros equal.
__device__ __forceinline__ unsigned sum_key(float f) {
  const unsigned u = __float_as_uint(f == 0.f ? 0.f : f);
  return f != f ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ unsigned ld_cluster_u32(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_cluster_s2(uint32_t addr, int2 v) {
  asm volatile("st.shared::cluster.v2.s32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

__global__ void __launch_bounds__(kEvThreads) kv_evict_kernel(const EvictArgs a) {
  __shared__ EvictSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.cluster, rank = int(blockIdx.x) % C;
  const unsigned unit = blockIdx.x / unsigned(C);
  const int g = int(unit % kKvHeads), layer = int(unit / kKvHeads % unsigned(a.num_layers));
  const int s = int(unit / kKvHeads / unsigned(a.num_layers));
  griddep_launch_dependents();
  auto barrier = [&]() {
    if (C > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  const int ctx = __ldg(a.context_lens + s), budget = __ldg(a.budgets + s);
  const bool bad_ctx = ctx < 0 || ctx > a.max_context, bad_budget = budget < 0 || min(budget, ctx) > a.max_budget;
  const bool first = layer == 0 && g == 0 && rank == 0 && tid == 0;
  if (bad_ctx || bad_budget) {
    if (first) {
      report(a.status, bad_ctx ? PKV_DEV_BAD_CONTEXT : PKV_DEV_BAD_BUDGET);
      if (a.new_lens != nullptr) a.new_lens[s] = ctx;
    }
    return;  // every CTA of the cluster
  }
  const int B = min(budget, ctx);
  if (first && a.new_lens != nullptr) a.new_lens[s] = B;
  const long long at = (long long)s * a.sums_seq + (long long)layer * a.sums_layer + (long long)g * a.sums_head;
  const float *sums = a.sums + at;
  float *new_sums = a.new_sums + at;
  int32_t *kept = a.kept + (((long long)s * a.num_layers + layer) * kKvHeads + g) * a.kept_stride;
  const int head = min(a.sinks, B), tail = ctx - min(a.recent, B - head);  // candidates: head <= t < tail
  const int p0 = int((long long)rank * ctx / C), p1 = int((long long)(rank + 1) * ctx / C);  // this CTA's tokens

  // ---- threshold: kept are the candidates whose key is above T, and the first `ties` whose key is T ----
  unsigned T = 0xffffffffu, ties = 0;
  unsigned need = unsigned(B - head - (ctx - tail));
  if (need >= unsigned(tail - head)) {
    T = 0;  // all of them
    ties = need;
  } else if (need > 0) {
    const int c0 = max(p0, head), c1 = min(p1, tail);
    unsigned prefix = 0;
    sm.hist[0][tid] = 0;
    __syncthreads();
#pragma unroll 1
    for (int pass = 0; pass < 32 / kDigitBits; ++pass) {
      const int shift = 32 - kDigitBits * (pass + 1);
      unsigned *hist = sm.hist[pass & 1];
      for (int t0 = c0 + warp * 32; t0 < c1; t0 += kEvThreads) {
        const int t = t0 + lane;
        bool in = t < c1;
        const unsigned key = in ? sum_key(sums[t]) : 0u;
        in = in && (pass == 0 || key >> (shift + kDigitBits) == prefix);
        const unsigned bin = in ? key >> shift & (kBins - 1) : kBins;
        const unsigned same = __match_any_sync(0xffffffffu, bin);
        if (in && lane == __ffs(same) - 1) atomicAdd(&hist[bin], unsigned(__popc(same)));
      }
      barrier();
      sm.hist[(pass & 1) ^ 1][tid] = 0;  // the next pass's: every CTA has read what the pass before left there
      unsigned mine = 0;                 // of bin tid, over the cluster
      if (C > 1) {
        const uint32_t addr = smem_addr(&hist[tid]);
        for (int r = 0; r < C; ++r) mine += ld_cluster_u32(cluster_map(addr, uint32_t(r)));
      } else {
        mine = hist[tid];
      }
      // keys in the bins above this one
      unsigned up = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_down_sync(0xffffffffu, up, o);
        if (lane + o < 32) up += y;
      }
      if (lane == 0) sm.warp_part[warp] = int(up);
      __syncthreads();
      for (int w = warp + 1; w < kEvWarps; ++w) up += unsigned(sm.warp_part[w]);
      const unsigned above = up - mine;
      if (above < need && need <= up) {
        sm.digit = unsigned(tid);
        sm.need = need - above;
        sm.whole = need == up;
      }
      __syncthreads();
      prefix = prefix << kDigitBits | sm.digit;
      need = sm.need;
      if (sm.whole) {  // every key with this prefix is kept
        T = (prefix << shift) - 1u;
        ties = 0;
        break;
      }
      T = prefix;
      ties = need;
    }
  }

  // ---- kept positions, ascending: a warp's share is a run of tokens ----
  const int share = (p1 - p0 + kEvWarps - 1) / kEvWarps;
  const int w0 = min(p0 + warp * share, p1), w1 = min(w0 + share, p1);
  auto classify = [&](int t, bool &sure, bool &equal) {
    const bool in = t < w1, fixed = in && (t < head || t >= tail);
    const unsigned key = in && !fixed ? sum_key(sums[t]) : 0u;
    sure = fixed || (in && key > T);
    equal = in && !fixed && key == T;
  };
  int2 count = make_int2(0, 0);
  for (int t0 = w0; t0 < w1; t0 += 32) {
    bool sure, equal;
    classify(t0 + lane, sure, equal);
    count.x += __popc(__ballot_sync(0xffffffffu, sure));
    count.y += __popc(__ballot_sync(0xffffffffu, equal));
  }
  if (lane == 0) sm.warp_count[warp] = count;
  __syncthreads();
  if (C > 1) {
    if (tid < C) {
      int2 all = make_int2(0, 0);
      for (int w = 0; w < kEvWarps; ++w) {
        all.x += sm.warp_count[w].x;
        all.y += sm.warp_count[w].y;
      }
      st_cluster_s2(cluster_map(smem_addr(&sm.rank_count[rank]), uint32_t(tid)), all);
    }
    cluster_sync();
  }
  int2 before = make_int2(0, 0);
  for (int r = 0; r < rank; ++r) {
    before.x += sm.rank_count[r].x;
    before.y += sm.rank_count[r].y;
  }
  for (int w = 0; w < warp; ++w) {
    before.x += sm.warp_count[w].x;
    before.y += sm.warp_count[w].y;
  }
  const unsigned below = (1u << lane) - 1u;
  for (int t0 = w0; t0 < w1; t0 += 32) {
    bool sure, equal;
    classify(t0 + lane, sure, equal);
    const unsigned ms = __ballot_sync(0xffffffffu, sure), me = __ballot_sync(0xffffffffu, equal);
    const int eq = before.y + __popc(me & below);
    if (sure || (equal && unsigned(eq) < ties))
      __stcg(kept + before.x + __popc(ms & below) + min(unsigned(eq), ties), t0 + lane);
    before.x += __popc(ms);
    before.y += __popc(me);
  }
  barrier();  // the list is complete, and nobody reads sums for the selection any more

  // ---- the rows move ----
  const int32_t *table = a.block_tables + (long long)s * a.bt_stride + (long long)layer * a.layer_stride;
  const long long in_page = (long long)g * kPageTokens * kRowBytes;
  const int rounds = (B + kEvRows * C - 1) / (kEvRows * C);
  float w_now = 0.f, w_next = 0.f;
  auto look_up = [&](int i, float &w) {  // places of round i's rows, by threads 0 .. kEvRows - 1
    const int k = (i * C + rank) * kEvRows + tid;
    long long from = -1, to = -1;
    if (k < B) {
      const int src = __ldcg(kept + k);
      w = sums[src];
      if (src != k) {
        const int sp = __ldg(table + src / kPageTokens), dp = __ldg(table + k / kPageTokens);
        if (unsigned(sp) >= unsigned(a.num_pages) || unsigned(dp) >= unsigned(a.num_pages)) {
          report(a.status, PKV_DEV_BAD_PAGE);
        } else {
          from = sp * a.page_stride + in_page + (src % kPageTokens) * kRowBytes;
          to = dp * a.page_stride + in_page + (k % kPageTokens) * kRowBytes;
        }
      }
    }
    sm.from[i & 1][tid] = from;
    sm.to[i & 1][tid] = to;
  };
  uint8_t *half = ((tid & 8) ? a.v_base : a.k_base) + (tid & 7) * 16;
  if (tid < kEvRows) look_up(0, w_now);
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    uint4 x[kEvLoads];
#pragma unroll
    for (int j = 0; j < kEvLoads; ++j) {
      const long long from = sm.from[i & 1][j * (kEvThreads / kEvChunks) + tid / kEvChunks];
      if (from >= 0) x[j] = *reinterpret_cast<const uint4 *>(half + from);
    }
    if (i + 1 < rounds && tid < kEvRows) look_up(i + 1, w_next);
    barrier();  // every row of the round, and every sum up to the next round's, is in registers
#pragma unroll
    for (int j = 0; j < kEvLoads; ++j) {
      const int r = j * (kEvThreads / kEvChunks) + tid / kEvChunks;
      if (sm.from[i & 1][r] >= 0) *reinterpret_cast<uint4 *>(half + sm.to[i & 1][r]) = x[j];
    }
    const int k = (i * C + rank) * kEvRows + tid;
    if (tid < kEvRows && k < B) new_sums[k] = w_now;
    w_now = w_next;
    __syncthreads();  // the places have been read
  }
  for (int t = B + rank * kEvThreads + tid; t < ctx; t += C * kEvThreads) new_sums[t] = 0.f;
}

// Whether two ranges of bytes share one.
bool ranges_overlap(const void *p, unsigned long long np, const void *q, unsigned long long nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_kv_evict(const pkv_pool *pool, const int32_t *block_tables, int64_t block_table_stride,
                            int64_t layer_stride, int num_layers, const int32_t *context_lens, const int32_t *budgets,
                            int num_seqs, int max_context, int max_budget, int sinks, int recent,
                            const float *weight_sums, float *new_weight_sums, int64_t sums_seq_stride,
                            int64_t sums_layer_stride, int64_t sums_head_stride, int32_t *kept, int64_t kept_stride,
                            int32_t *new_context_lens, int32_t *device_status, void *stream) {
  const int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_seqs < 0 || num_layers < 1 || max_context < 0 || max_context > (1 << 30) || max_budget < 0 || sinks < 0 ||
      recent < 0 || block_table_stride < 0 || layer_stride < 0 || kept_stride < max_budget ||
      sums_head_stride < max_context || sums_layer_stride < 0 || sums_seq_stride < 0 ||
      (long long)num_seqs * num_layers > 0x7fffffffLL / (pkv::kKvHeads * pkv::kEvMaxCluster))
    return PKV_ERR_SHAPE;
  // a row of sums belongs to one (sequence, layer, head)
  const long long heads = pkv::kKvHeads * sums_head_stride;
  const bool layers_inside = (num_layers == 1 || sums_layer_stride >= heads) &&
                             (num_seqs <= 1 || sums_seq_stride >= (num_layers == 1 ? heads : num_layers * sums_layer_stride));
  const bool seqs_inside = (num_seqs <= 1 || sums_seq_stride >= heads) &&
                           (num_layers == 1 || sums_layer_stride >= (num_seqs <= 1 ? heads : num_seqs * sums_seq_stride));
  if (num_seqs > 0 && !layers_inside && !seqs_inside) return PKV_ERR_SHAPE;
  if (num_seqs == 0 || max_context == 0) return PKV_OK;
  if (block_tables == nullptr || context_lens == nullptr || budgets == nullptr || weight_sums == nullptr ||
      new_weight_sums == nullptr || (kept == nullptr && max_budget > 0))
    return PKV_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens) |
       reinterpret_cast<uintptr_t>(budgets) | reinterpret_cast<uintptr_t>(weight_sums) |
       reinterpret_cast<uintptr_t>(new_weight_sums) | reinterpret_cast<uintptr_t>(kept) |
       reinterpret_cast<uintptr_t>(new_context_lens)) & 3u)
    return PKV_ERR_ALIGN;
  // what the call writes may not lie where other units still read
  const unsigned long long lens = 4ull * num_seqs;
  const unsigned long long sums = 4ull * ((num_seqs - 1) * sums_seq_stride + (num_layers - 1) * sums_layer_stride +
                                          (pkv::kKvHeads - 1) * sums_head_stride + max_context);
  const unsigned long long list = 4ull * num_seqs * num_layers * pkv::kKvHeads * kept_stride;
  if (new_weight_sums != weight_sums && pkv::ranges_overlap(new_weight_sums, sums, weight_sums, sums))
    return PKV_ERR_SHAPE;
  if (new_context_lens != nullptr && (pkv::ranges_overlap(new_context_lens, lens, context_lens, lens) ||
                                      pkv::ranges_overlap(new_context_lens, lens, budgets, lens)))
    return PKV_ERR_SHAPE;
  for (const void *p : {static_cast<const void *>(context_lens), static_cast<const void *>(budgets)})
    if (pkv::ranges_overlap(kept, list, p, lens) || pkv::ranges_overlap(new_weight_sums, sums, p, lens))
      return PKV_ERR_SHAPE;
  if (pkv::ranges_overlap(kept, list, weight_sums, sums) || pkv::ranges_overlap(kept, list, new_weight_sums, sums))
    return PKV_ERR_SHAPE;
  pkv::EvictArgs a;
  a.k_base = static_cast<uint8_t *>(pool->k_base);
  a.v_base = static_cast<uint8_t *>(pool->v_base);
  a.page_stride = pool->page_stride_bytes;
  a.num_pages = pool->num_pages;
  a.block_tables = block_tables;
  a.bt_stride = block_table_stride;
  a.layer_stride = layer_stride;
  a.num_layers = num_layers;
  a.context_lens = context_lens;
  a.budgets = budgets;
  a.max_context = max_context;
  a.max_budget = max_budget;
  a.sinks = sinks;
  a.recent = recent;
  a.sums = weight_sums;
  a.new_sums = new_weight_sums;
  a.sums_seq = sums_seq_stride;
  a.sums_layer = sums_layer_stride;
  a.sums_head = sums_head_stride;
  a.kept = kept;
  a.kept_stride = kept_stride;
  a.new_lens = new_context_lens;
  a.status = device_status;
  const long long units = (long long)num_seqs * num_layers * pkv::kKvHeads;
  const int sms = pkv::device_sm_count();
  const long long slots = 4ll * (sms > 0 ? sms : 148);
  a.cluster = 1;
  while (a.cluster < pkv::kEvMaxCluster && units * a.cluster * 2 <= slots && max_context >= a.cluster * 2 * pkv::kEvRows)
    a.cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * a.cluster));
  cfg.blockDim = dim3(pkv::kEvThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(a.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, pkv::kv_evict_kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_LAUNCH;
  }
  return PKV_OK;
}
