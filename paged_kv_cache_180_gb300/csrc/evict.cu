// Eviction: per sequence, layer and K/V head the cached tokens with the largest weight sums are kept, with the first few
// and the most recent ones, and their rows move together at the front of the sequence, in order and in place.
//
// What is kept of ctx tokens with B = min(budget, ctx):  the first a = min(sinks, B), the last r = min(recent, B - a), and
// of the tokens between them the B - a - r with the largest sums; of equal sums the earlier token.
//
// A unit is one (sequence, layer, K/V head); it belongs to one CTA or one cluster of CTAs, each of which holds the sums of
// an equal run of the tokens in shared memory (where they fit).
//  * Selection: sums are mapped to 32-bit keys of the same order and the key of rank B - a - r is found digit by digit from
//    the top (11, 11 and 10 bits, a histogram in shared memory, added up over the cluster); the passes end once a bin is
//    needed whole, which is after the second where the sums differ.  A prefix sum over the tokens then gives every kept one
//    its place, and its position and sum are written there.
//  * Moving: kept[k] >= k, ascending, so the rows that round i of the move writes (positions i R .. (i + 1) R - 1) lie at
//    or before everything that later rounds read, and a barrier between a round's loads and its stores is all the order
//    there has to be.  A row's K and V (2 x 128 B) are moved by 16 threads, 16 bytes each, through a ring in shared memory
//    (cp.async), each thread storing what it loaded itself.
//
// What bounds it: large batches HBM, 64 sequences of 1024 .. 2048 tokens in 16 layers cut to 60 % in 626 us (3.95 GB, 6.3
// TB/s, 93 % of the copy rate); few units the chain before the first row moves.  One sequence's 16 layers of 2048 tokens:
// 20 us, of them 9 until the first rows have landed (launch and lengths 0.8, sums 0.8, selection 2.6, list 1.5, first rows
// 1.9) and 10 at the rate of HBM.  Two long documents, 57000 tokens cut to a quarter: 57 us, of them 20 selection and list
// (a cluster barrier and what is read behind it take 0.7) and 20 to 26 the rows, in 27 to 30 rounds.
//  * Passes over digits, because a sort moves what selection only counts; 11 bits in a CTA of its own, as the exponent
//    decides little. In a cluster the range of the keys is found first: without it the first pass, of a few bins, decided
//    next to nothing.
//  * Rows go through shared memory rather than registers, so that four to six rounds are in flight.
#include <cuda_runtime.h>

#include <mutex>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kEvMaxCluster = 8;
constexpr int kEvChunks = 2 * kRowBytes / 16;  // 16-byte chunks of a row's K and V: 16
constexpr int kEvLook = 512;                   // rows of a CTA whose old positions are fetched at once
constexpr int kMaxBins = 2048;                 // of a digit of 11 bits, or of one of 9 bits in four copies
constexpr int kClusterBins = 512;
constexpr int kRun = 4;                        // tokens of a thread in one step of the list
constexpr int kStep = 32 * kRun;               // tokens of a warp in one
constexpr int kEvMaxPages = 4096;              // block-table entries that a CTA may hold (16 KiB)
constexpr size_t kEvMaxSmem = 200 * 1024;      // dynamic shared memory of a CTA at the most

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
  int sums_bytes;   // of the CTA's sums in shared memory, in front of the histograms
  int pages_bytes;  // of the unit's block-table entries behind the buffer, 0 where they are read from global memory
  int buffer_bytes;  // rows in flight; before that sums and histograms
};

template <int kThreads>
struct EvictSmem {
  unsigned warp_part[2][kThreads / 32];
  int2 warp_count[kThreads / 32];  // (kept for certain, equal to the threshold) of a warp's tokens
  int2 count;                      // of the CTA's tokens
  int from[2][kEvLook];            // old positions of the CTA's next rows
  // cluster: the CTA's counts of a pass; what the CTAs have in the bins that this one adds up; the sums; those of each 32
  // bins
  unsigned bins[kClusterBins], part[kClusterBins], share[kClusterBins], group[kClusterBins / 32];
  uint2 range;                     // cluster: smallest and largest key of the CTA's candidates
  unsigned digit, need;
  int whole;
};

// Order-preserving map of a sum to 32 bits: NaN below everything, the two zeros equal.
__device__ __forceinline__ unsigned sum_key(float f) {
  const unsigned u = __float_as_uint(f + 0.f);  // (-0 + 0 = 0)
  return f != f ? 0u : u ^ (unsigned(int(u) >> 31) | 0x80000000u);
}

// Asynchronous copies from global to shared memory (one group per commit).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}

__device__ __forceinline__ unsigned ld_cluster_u32(uint32_t addr) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// kRows: rows of a round and CTA; kRing: rounds whose rows are held or on their way; kStaged: sums in shared memory.
template <int kThreads, int kRows, int kRing, bool kStaged, bool kCluster>
__global__ void __launch_bounds__(kThreads) kv_evict_kernel(const EvictArgs a) {
  // digits: 11, 11 and 10 bits in a CTA of its own; 9 bits each in a cluster, where every CTA reads every other's bins
  constexpr int kDigit = kCluster ? 9 : 11, kBins = 1 << kDigit, kCopies = kMaxBins / kBins;
  static_assert(!kCluster || (kBins == kClusterBins && kBins == kThreads), "");
  constexpr int kWarps = kThreads / 32, kThreadBins = kBins > kThreads ? kBins / kThreads : 1;
  constexpr int kRowStep = kThreads / kEvChunks, kLoads = kRows / kRowStep, kRounds = kEvLook / kRows;
  static_assert(kRounds >= kRing && kLoads >= 1, "");
  __shared__ EvictSmem<kThreads> sm;
  extern __shared__ __align__(16) uint8_t buffer[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = kCluster ? a.cluster : 1, rank = kCluster ? int(blockIdx.x) % C : 0;
  const unsigned unit = blockIdx.x / unsigned(C);
  const int g = int(unit % kKvHeads), layer = int(unit / kKvHeads % unsigned(a.num_layers));
  const int s = int(unit / kKvHeads / unsigned(a.num_layers));
  griddep_launch_dependents();
  auto barrier = [&]() {
    if (kCluster)
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
  const int32_t *table = a.block_tables + (long long)s * a.bt_stride + (long long)layer * a.layer_stride;
  const int head = min(a.sinks, B), tail = ctx - min(a.recent, B - head);  // candidates: head <= t < tail
  const int p0 = int((long long)rank * ctx / C), p1 = int((long long)(rank + 1) * ctx / C);  // this CTA's tokens

  // ---- this CTA's sums and the unit's block-table entries into shared memory, where they fit ----
  const float *own = reinterpret_cast<const float *>(buffer);
  unsigned *hists = reinterpret_cast<unsigned *>(buffer + a.sums_bytes);
  const int32_t *pages = table;
  if (kStaged)
    for (int t = p0 + tid; t < p1; t += kThreads) cp_async4(smem_addr(own + (t - p0)), sums + t);
  if (a.pages_bytes > 0) {
    pages = reinterpret_cast<const int32_t *>(buffer + a.buffer_bytes);
    const int blocks = (ctx + kPageTokens - 1) / kPageTokens;
    for (int i = tid; i < blocks; i += kThreads) cp_async4(smem_addr(pages + i), table + i);
  }
  cp_async_commit();
  const int bin0 = tid * kThreadBins;
  const bool has_bins = kBins >= kThreads || tid < kBins;
  for (int i = tid; i < kBins * kCopies; i += kThreads) hists[i] = 0u;
  cp_async_wait<0>();
  __syncthreads();
  auto sum_at = [&](int t) { return kStaged ? own[t - p0] : sums[t]; };

  // ---- threshold: kept are the candidates whose key is above T, and the first `ties` whose key is T ----
  unsigned T = 0xffffffffu, ties = 0;
  unsigned need = unsigned(B - head - (ctx - tail));
  if (need >= unsigned(tail - head)) {
    T = 0;  // all of them
    ties = need;
  } else if (need > 0) {
    const int c0 = max(p0, head), c1 = min(p1, tail);
    unsigned lo = 0;  // keys looked at: lo <= key < lo + 2^(shift + kDigit)
    int shift = 32 - kDigit;
    if (kCluster) {
      // many keys of nearly the same exponent: the digits divide the range that there is
      unsigned least = ~0u, most = 0u;
#pragma unroll 4
      for (int t = c0 + tid; t < c1; t += kThreads) {
        const unsigned key = sum_key(sum_at(t));
        least = min(least, key);
        most = max(most, key);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      if (lane == 0) sm.warp_part[0][warp] = least, sm.warp_part[1][warp] = most;
      __syncthreads();
      if (tid < 32) {
        least = __reduce_min_sync(0xffffffffu, tid < kWarps ? sm.warp_part[0][tid] : ~0u);
        most = __reduce_max_sync(0xffffffffu, tid < kWarps ? sm.warp_part[1][tid] : 0u);
        if (tid == 0) sm.range = make_uint2(least, most);
      }
      cluster_sync();
      const uint32_t there = cluster_map(smem_addr(&sm.range), uint32_t((lane + rank) % C));
      least = __reduce_min_sync(0xffffffffu, ld_cluster_u32(there));
      most = __reduce_max_sync(0xffffffffu, ld_cluster_u32(there + 4));
      lo = least;
      shift = max(0, 32 - __clz(int(most - least)) - kDigit);
    }
    int bits = kDigit;
#pragma unroll 1
    for (int pass = 0;; ++pass) {
#pragma unroll 4
      for (int t = c0 + tid; t < c1; t += kThreads) {
        const unsigned d = (sum_key(sum_at(t)) - lo) >> shift;
        if (d < 1u << bits) atomicAdd(&hists[d * kCopies + lane % kCopies], 1u);
      }
      __syncthreads();
      unsigned c[kThreadBins] = {};  // this thread's bins; the next pass starts from 0
      if (has_bins) {
#pragma unroll
        for (int i = 0; i < kThreadBins * kCopies; ++i) {
          c[i / kCopies] += hists[bin0 * kCopies + i];
          hists[bin0 * kCopies + i] = 0u;
        }
      }
      if (kCluster) {
        // Every CTA adds up its share of the bins over the cluster, and the sums of each 32 of them; the sums say which 32
        // hold the key of rank `need`.  (Every CTA reading all bins of all others took 5000 cycles a pass.)
        const int slice = kBins / C;
        sm.bins[tid] = c[0];
        cluster_sync();
        sm.part[tid] = ld_cluster_u32(cluster_map(smem_addr(&sm.bins[rank * slice + tid % slice]), uint32_t(tid / slice)));
        __syncthreads();
        if (tid < slice) {
          unsigned x = 0;
          for (int r = 0; r < C; ++r) x += sm.part[r * slice + tid];
          sm.share[tid] = x;
          x = __reduce_add_sync(0xffffffffu, x);
          if (lane == 0) sm.group[warp] = x;
        }
        cluster_sync();
        if (warp == 0) {
          auto from_top = [&](unsigned x) {  // sum of the lanes from this one on
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned y = __shfl_down_sync(0xffffffffu, x, o);
              if (lane + o < 32) x += y;
            }
            return x;
          };
          const int groups = slice / 32;
          const uint32_t there = cluster_map(smem_addr(&sm.group[lane % groups]), uint32_t(lane % (kBins / 32) / groups));
          const unsigned x = lane < kBins / 32 ? ld_cluster_u32(there) : 0u;
          unsigned up = from_top(x);
          const int at = 31 - __clz(int(__ballot_sync(0xffffffffu, up >= need)));  // the group
          const unsigned above = __shfl_sync(0xffffffffu, up - x, at);
          const unsigned y = ld_cluster_u32(cluster_map(smem_addr(&sm.share[at % groups * 32 + lane]), uint32_t(at / groups)));
          up = from_top(y) + above;
          if (up - y < need && need <= up) {
            sm.digit = unsigned(at * 32 + lane);
            sm.need = need - (up - y);
            sm.whole = need == up;
          }
        }
      } else {
        unsigned mine = 0;
#pragma unroll
        for (int i = 0; i < kThreadBins; ++i) mine += c[i];
        unsigned up = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const unsigned y = __shfl_down_sync(0xffffffffu, up, o);
          if (lane + o < 32) up += y;
        }
        if (lane == 0) sm.warp_part[pass & 1][warp] = up;
        __syncthreads();
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const unsigned x = sm.warp_part[pass & 1][w];
          if (w > warp) up += x;
        }
        if (up - mine < need && need <= up) {  // the bin of the key of rank `need` is one of this thread's
          unsigned above = up - mine;
          bool found = false;
#pragma unroll
          for (int i = kThreadBins - 1; i >= 0; --i) {
            if (!found && above + c[i] >= need) {
              found = true;
              sm.digit = unsigned(bin0 + i);
              sm.need = need - above;
              sm.whole = need == above + c[i];
            }
            above += c[i];
          }
        }
      }
      __syncthreads();
      lo += sm.digit << shift;
      need = sm.need;
      if (sm.whole) {  // every key from lo on is kept
        T = lo - 1u;
        break;
      }
      if (shift == 0) {
        T = lo;
        ties = need;
        break;
      }
      bits = min(kDigit, shift);
      shift -= bits;
    }
  }

  // ---- kept positions, ascending ----
  // every warp looks at an equal run of the CTA's tokens, twice: to count, and to write
  const int run = ((p1 - p0 + kWarps - 1) / kWarps + kRun - 1) / kRun * kRun;
  const int w0 = p0 + warp * run, w1 = min(p1, w0 + run);
  float v[kRun];
  unsigned sure, equal;  // bit j: token t + j
  auto look = [&](int t) {
    if (kStaged) {  // (the buffer goes on behind p1; what lies there is not used)
      *reinterpret_cast<float4 *>(v) = *reinterpret_cast<const float4 *>(own + (t - p0));
    } else {
#pragma unroll
      for (int j = 0; j < kRun; ++j) v[j] = t + j < w1 ? sums[t + j] : 0.f;
    }
    sure = equal = 0;
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool in = t + j < w1, fixed = unsigned(t + j - head) >= unsigned(tail - head);
      const unsigned key = sum_key(v[j]);
      sure |= unsigned(in && (fixed || key > T)) << j;
      equal |= unsigned(in && !fixed && key == T) << j;
    }
  };
  int2 before = make_int2(0, 0);  // (kept for certain, equal to T) in front of this warp's tokens
#pragma unroll 2
  for (int base = w0; base < w1; base += kStep) {
    look(base + lane * kRun);
    before.x += __popc(sure);
    before.y += __popc(equal);
  }
  before.x = __reduce_add_sync(0xffffffffu, before.x);
  before.y = __reduce_add_sync(0xffffffffu, before.y);
  if (lane == 0) sm.warp_count[warp] = before;
  __syncthreads();
  before = make_int2(0, 0);
  int2 all = make_int2(0, 0);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int2 c = sm.warp_count[w];
    if (w < warp) before.x += c.x, before.y += c.y;
    all.x += c.x;
    all.y += c.y;
  }
  if (kCluster) {
    if (tid == 0) sm.count = all;
    cluster_sync();
    int2 c = make_int2(0, 0);  // of the CTAs in front
    if (lane < rank) {
      const uint32_t there = cluster_map(smem_addr(&sm.count), uint32_t(lane));
      c = make_int2(int(ld_cluster_u32(there)), int(ld_cluster_u32(there + 4)));
    }
    before.x += __reduce_add_sync(0xffffffffu, c.x);
    before.y += __reduce_add_sync(0xffffffffu, c.y);
  }
  // (sums held here are written over from now on: the barriers above followed the last CTA's copy of them)
#pragma unroll 2
  for (int base = w0; base < w1; base += kStep) {
    const int t = base + lane * kRun;
    look(t);
    const unsigned mine = unsigned(__popc(sure)) | unsigned(__popc(equal)) << 16;
    unsigned upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    unsigned x = unsigned(before.x) + ((upto - mine) & 0xffffu), y = unsigned(before.y) + ((upto - mine) >> 16);
#pragma unroll
    for (int j = 0; j < kRun; ++j) {
      const bool is = sure >> j & 1, eq = equal >> j & 1;
      if (is || (eq && y < ties)) {
        const unsigned k = x + min(y, ties);
        if (k < unsigned(B)) {  // (always, unless somebody else writes the sums meanwhile)
          __stcg(kept + k, t + j);
          if (kStaged) new_sums[k] = v[j];
        }
      }
      x += is;
      y += eq;
    }
    const unsigned step = __shfl_sync(0xffffffffu, upto, 31);
    before.x += int(step & 0xffffu);
    before.y += int(step >> 16);
  }
  barrier();  // the list is complete, and nobody reads sums for the selection any more
  if (!kStaged) {
    // the kept sums move as the rows do: a barrier between a round's loads and its stores
    for (int k0 = 0; k0 < B; k0 += C * kThreads) {
      const int k = k0 + rank * kThreads + tid;
      const float v = k < B ? sums[min(unsigned(__ldcg(kept + k)), unsigned(ctx - 1))] : 0.f;
      barrier();
      if (k < B) new_sums[k] = v;
    }
    barrier();
  }

  // ---- the rows move ----
  const int rounds = (B + kRows * C - 1) / (kRows * C);
  auto row = [&](int i, int r) { return (i * C + rank) * kRows + r; };  // row r of this CTA in round i
  auto look_up = [&](int j) {  // old positions of the rows of rounds j kRounds .. (j + 1) kRounds - 1
#pragma unroll
    for (int r = tid; r < kEvLook; r += kThreads) {
      const int k = row(j * kRounds + r / kRows, r % kRows);
      int src = k < B ? __ldcg(kept + k) : k;
      if (unsigned(src) >= unsigned(ctx)) src = k;
      sm.from[j & 1][r] = src;  // (a row that stays where it is does not move)
    }
  };
  // a thread moves the same 16-byte chunk of every kRowStep-th row
  uint8_t *half = ((tid & 8) ? a.v_base : a.k_base) + (long long)g * kPageTokens * kRowBytes + (tid & 7) * 16;
  const int r0 = tid / kEvChunks;
  auto moves = [&](int i, int r, int &sp, int &dp, int &src, int &k) {
    k = row(i, r);
    src = sm.from[i / kRounds & 1][i % kRounds * kRows + r];
    if (src == k) return false;
    sp = pages[src / kPageTokens];
    dp = pages[k / kPageTokens];
    return unsigned(sp) < unsigned(a.num_pages) && unsigned(dp) < unsigned(a.num_pages);
  };
  auto load = [&](int i) {
    if (i < rounds) {
      if (i % kRounds == 0) {
        look_up(i / kRounds);
        __syncthreads();
      }
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        int sp, dp, src, k;
        if (moves(i, j * kRowStep + r0, sp, dp, src, k))
          cp_async16(smem_addr(buffer) + (((i % kRing) * kLoads + j) * kThreads + tid) * 16,
                     half + sp * a.page_stride + (src % kPageTokens) * kRowBytes);
        else if (src != k && tid % kEvChunks == 0)
          report(a.status, PKV_DEV_BAD_PAGE);
      }
    }
    cp_async_commit();
  };
  auto store = [&](int i) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      int sp, dp, src, k;
      if (moves(i, j * kRowStep + r0, sp, dp, src, k))
        *reinterpret_cast<uint4 *>(half + dp * a.page_stride + (k % kPageTokens) * kRowBytes) =
            *reinterpret_cast<const uint4 *>(buffer + (((i % kRing) * kLoads + j) * kThreads + tid) * 16);
    }
  };
  // Round i's stores come a step after its loads have landed in every CTA of the cluster, so that the barrier's latency
  // passes under other rounds' copies.  (What the barrier orders is loads that have landed before stores that follow: it
  // need not publish the stores before it.)
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) load(i);
  for (int t = B + rank * kThreads + tid; t < ctx; t += C * kThreads) new_sums[t] = 0.f;  // (under the first copies)
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    cp_async_wait<kRing - 2>();
    if (kCluster) {
      __syncwarp();
      if (i > 0) cluster_wait();
      cluster_arrive_relaxed();
    } else {
      __syncthreads();
    }
    if (i > 0) store(i - 1);
    load(i + kRing - 1);
  }
  if (rounds > 0) {
    __syncwarp();
    if (kCluster) cluster_wait();
    store(rounds - 1);
  }
}

using EvictKernel = void (*)(EvictArgs);
constexpr EvictKernel kEvictMany = kv_evict_kernel<256, 32, 4, true, false>;
constexpr EvictKernel kEvictFew = kv_evict_kernel<512, 64, 6, true, false>;
constexpr EvictKernel kEvictCluster = kv_evict_kernel<512, 64, 5, true, true>;
constexpr EvictKernel kEvictLong = kv_evict_kernel<512, 64, 5, false, true>;

// Shared-memory limits of the kernels on the current device.
int setup_evict_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    for (EvictKernel kernel : {kEvictMany, kEvictFew, kEvictCluster, kEvictLong})
      if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kEvMaxSmem)) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
      }
    done[dev] = true;
  }
  return PKV_OK;
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
  // (no array has 2^38 elements; what is computed from the strides below stays within 64 bits)
  constexpr int64_t kFar = int64_t(1) << 38;
  if (kept_stride > kFar >> 7 || sums_head_stride > kFar || sums_layer_stride > kFar || sums_seq_stride > kFar ||
      (num_seqs > 1 && (num_seqs - 1) * sums_seq_stride > kFar) || (num_layers - 1) * sums_layer_stride > kFar)
    return PKV_ERR_SHAPE;
  // a row of sums belongs to one (sequence, layer, head)
  const long long heads = pkv::kKvHeads * sums_head_stride;
  const bool layers_inside = (num_layers == 1 || sums_layer_stride >= heads) &&
                             (num_seqs <= 1 || sums_seq_stride >= (num_layers == 1 ? heads : num_layers * sums_layer_stride));
  const bool seqs_inside = (num_seqs <= 1 || sums_seq_stride >= heads) &&
                           (num_layers == 1 || sums_layer_stride >= (num_seqs <= 1 ? heads : num_seqs * sums_seq_stride));
  if (num_seqs > 0 && !layers_inside && !seqs_inside) return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  // (without cached tokens there are no sums, and without a budget there is no list; the new lengths are written all the
  // same)
  if (block_tables == nullptr || context_lens == nullptr || budgets == nullptr ||
      ((weight_sums == nullptr || new_weight_sums == nullptr) && max_context > 0) || (kept == nullptr && max_budget > 0))
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
  if (new_context_lens != nullptr &&
      (pkv::ranges_overlap(new_context_lens, lens, kept, list) || pkv::ranges_overlap(new_context_lens, lens, weight_sums, sums) ||
       pkv::ranges_overlap(new_context_lens, lens, new_weight_sums, sums)))
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
  int sms = pkv::device_sm_count();
  if (sms <= 0) sms = 148;
  // CTAs to a unit: as many as find SMs, with a thousand tokens for each two of them.  Two sequences of 57000 tokens, one
  // layer (16 units), take 225 / 69 / 57 / 59 us with 1 / 4 / 8 / 16 of them; one of 2048 tokens (8 units) 15.9 us with 2,
  // 13.2 with 4 and 12.4 with 8, but two layers of it 13.4 with 4 and 15.8 with 8; one of 1024 tokens 10.7 with 1, 13.0
  // with 2, 11.7 with 4 or 8.
  a.cluster = 1;
  while (a.cluster < pkv::kEvMaxCluster && units * a.cluster * 2 <= sms && max_context >= (a.cluster < 2 ? 2 : a.cluster) * 1024)
    a.cluster *= 2;
  const int pages = (max_context + pkv::kPageTokens - 1) / pkv::kPageTokens;
  a.pages_bytes = pages <= pkv::kEvMaxPages ? (pages * 4 + 15) / 16 * 16 : 0;
  // Many units: small CTAs, several to an SM, so that one selects while others move: 64 x 16 layers 626 us, with the large
  // ones 652; 16 layers of one sequence (128 units) 26.7 us with the small ones, 19.3 with the large ones.
  pkv::EvictKernel kernel = a.cluster > 1 ? pkv::kEvictCluster : units > 2 * sms ? pkv::kEvictMany : pkv::kEvictFew;
  int threads = 512, ring = a.cluster > 1 ? 5 * 64 : 6 * 64;
  if (a.cluster == 1 && units > 2 * sms) {
    threads = 256;
    ring = 4 * 32;
  }
  const size_t hists = pkv::kMaxBins * sizeof(unsigned), tile = size_t(threads) * pkv::kRun;
  size_t buffer = size_t(ring) * 2 * pkv::kRowBytes;
  size_t sums_bytes = ((size_t(max_context) + a.cluster - 1) / a.cluster + tile - 1) / tile * tile * 4;
  if (sums_bytes + hists + a.pages_bytes > pkv::kEvMaxSmem) {
    kernel = pkv::kEvictLong;
    threads = 512;
    buffer = size_t(5 * 64) * 2 * pkv::kRowBytes;
    sums_bytes = 0;
  }
  if (sums_bytes + hists > buffer) buffer = sums_bytes + hists;
  a.sums_bytes = int(sums_bytes);
  a.buffer_bytes = int(buffer);
  if (pkv::setup_evict_attributes() != PKV_OK) return PKV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * a.cluster));
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = buffer + a.pages_bytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(a.cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_LAUNCH;
  }
  return PKV_OK;
}
