// Decode attention by units of one sequence and one K/V head: the two decode operators that bound a cache.
//
//  * window decode: the query attends to the first `sinks` tokens and the last `window` tokens,
//      out[s][h] = sum_{t in A} w_t V_t[h/4],  w = softmax_{t in A}(scale q[s][h] . K_t[h/4]),
//      A = { t < ctx : t < sinks or t >= ctx - window };
//  * decode with weight sums: plain decode attention that also adds up, for every cached token and K/V head g, the
//    weight it received from the head's four query heads,
//      sums[s][g][t] = decay sums[s][g][t] + sum_{h in group g} w_{h,t}.
//
// Both need the final softmax state of a unit inside the launch that reads it: the second one to normalise what it adds
// up.  So a unit belongs to one CTA or to one cluster of CTAs, which exchange their states through distributed shared
// memory: no workspace, no atomics, and results that do not depend on timing.
//
//  * The pages a unit sees are numbered v = 0 .. n - 1: the sinks' pages, then those from the window's first token on
//    (a page both reach into counts once).  CTA r of C takes [r n / C, (r + 1) n / C), its warp w every eighth of them
//    from w on.  A page is two TMA boxes (K and V rows of the head, 2 KiB each) in the warp's own ring: a warp issues
//    its own copies and waits for nobody else until its pages are done.
//  * Scores and products run on mma.sync m16n8k16.  The four query heads fill rows 0-3 and again rows 4-7 of Q, so that
//    rows 4-7 hold the same weights at no cost.  P V takes them as three bf16 terms (24 bits): the high term in rows
//    0-3, the middle one in rows 8-11, the low one in rows 4-7.  Each page's product starts from zero and is added to the
//    fp32 accumulators by ordinary additions, so that the tensor core's truncation does not build up over the pages.
//  * Tokens outside A get score -infinity and their V fragments are zeroed: what a page holds there, NaN included, reaches
//    nothing.
//  * With weight sums the scores (base 2, fp32) wait in shared memory, 16 bytes a token, until the unit's maximum and sum
//    are known; where a CTA's share does not fit (more than kChipPages pages), in the workspace.
//
// What bounds it: large batches HBM, 256 windows of 2032 tokens in 155 us (1.08 GB at 6.9 TB/s), 256 x 2048 with weight
// sums in 166 to 171 (1.11 GB at 6.5 to 6.7 TB/s); ragged batches the last CTAs, 64 windows of up to 1000 in 24.2 us and
// weight sums of 64 x 1 .. 2048 in 23.7, 5.2 to 5.4 TB/s; one sequence the latencies of one pass, 4.1 and 5.9 us (table
// entry, pages, states exchanged).
#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <mutex>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kUnitWarps = 8;
constexpr int kUnitThreads = kUnitWarps * 32;
constexpr int kDeepRing = 3, kShallowRing = 2;               // pages a warp has in flight
constexpr int kMaxCluster = 16;                              // CTAs that share a unit at the most
constexpr int kFarCluster = 8;                               // the same where they need an SM each
constexpr int kBoxBytes = kPageTokens * kRowBytes;           // one head's K (or V) rows of a page: 2 KiB
constexpr int kUnitOut = kGroup * kHeadDim;                  // output values of a unit: 256
constexpr int kScorePage = kPageTokens * int(sizeof(float4));  // scores of a page: 256 B
constexpr int kChipPages = 448;                              // pages of a CTA whose scores fit on chip beside a ring
constexpr int kSumsAhead = 8;                                // sums of a thread fetched before they are needed
constexpr int kMaxSorted = 128;                              // sequences that a CTA ranks by length
constexpr int kMinPages = 4;                                 // pages a CTA of a cluster gets at the least
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kUnitOut == kUnitThreads, "a thread owns one output value");

struct UnitArgs {
  CUtensorMap tmap_k, tmap_v;  // boxes of one head's 16 rows of one page
  int num_pages;
  const uint32_t *q;  // [num_seqs][32][64] bf16 as packed pairs
  void *out;          // [num_seqs][32][64] fp32 or bf16
  int out_bf16;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int max_context;
  int window, sinks;
  float scale_log2;  // scale * log2(e)
  int cluster;       // CTAs to a unit
  int sort;          // number of sequences where the longest go first, else 0
  float *sums;       // [num_seqs][8][tokens] at seq_stride, head_stride
  long long seq_stride, head_stride;
  float decay;
  float4 *scores;           // workspace: [unit][score_pages][16], null where shared memory holds the scores
  long long score_pages;
  int32_t *status;
};

template <int kStages>
struct __align__(1024) UnitSmem {
  uint8_t kv[kUnitWarps][kStages][2][kBoxBytes];  // 128-byte swizzled
  float acc[kUnitWarps][kGroup][kHeadDim];            // the warps' states
  float2 ml[kUnitWarps][kGroup];                      // (maximum in log2 units, sum)
  float recv_acc[kUnitOut];                           // this CTA's slice of the outputs from every CTA of the cluster
  float2 recv_ml[kMaxCluster][kGroup];
  float2 fin[kGroup];                                 // (maximum, 1 / sum) of the unit
  int seq;
  uint64_t full[kUnitWarps][kStages];
};

// D = A B with a zero accumulator.
__device__ __forceinline__ void mma_16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void st_cluster_f1(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// A maximum that exponents may be taken against: -infinity (no key, or none of finite score) becomes 0.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.f : m; }

template <bool kWeights, int kStages>
__global__ void __launch_bounds__(kUnitThreads, 2) unit_decode_kernel(const __grid_constant__ UnitArgs a) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = UnitSmem<kStages>;
  Smem &sm = *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = a.cluster, rank = int(blockIdx.x) % C;
  const unsigned unit = blockIdx.x / unsigned(C);
  const int g = int(unit % kKvHeads);
  int s = int(unit / kKvHeads);
  if (a.sort) {
    // the s-th longest sequence
    int *len = reinterpret_cast<int *>(&sm.acc[0][0][0]);
    int mine = 0;
    if (tid < a.sort) {
      const int c = __ldg(a.context_lens + tid);
      mine = c > a.max_context ? 0 : c;
      len[tid] = mine;
    }
    __syncthreads();
    int before = 0;
    for (int i = 0; i < a.sort; ++i) before += len[i] > mine || (len[i] == mine && i < tid);
    if (tid < a.sort && before == s) sm.seq = tid;
    __syncthreads();
    s = sm.seq;
  }
  const int ctx = __ldg(a.context_lens + s);
  const long long out_at = ((long long)s * kQHeads + g * kGroup) * kHeadDim;
  auto store = [&](int i, float v) {
    if (a.out_bf16)
      static_cast<uint16_t *>(a.out)[out_at + i] = uint16_t(pack_bf16x2(v, 0.f));
    else
      static_cast<float *>(a.out)[out_at + i] = v;
  };
  if (ctx <= 0 || ctx > a.max_context) {
    griddep_wait();
    griddep_launch_dependents();
    if (rank == 0) {
      if (ctx != 0 && g == 0 && tid == 0) report(a.status, PKV_DEV_BAD_CONTEXT);
      store(tid, 0.f);
    }
    return;  // every CTA of the cluster
  }
  // ---- the unit's pages, and this CTA's of them ----
  const int lo = max(0, ctx - a.window);      // first token of the window
  const int sink = min(a.sinks, lo);          // tokens before it that stay visible
  const int front = (sink + kPageTokens - 1) / kPageTokens;
  const int skip = max(lo / kPageTokens, front) - front;  // pages between that nobody sees
  const int n = (ctx + kPageTokens - 1) / kPageTokens - skip;
  const int pa = int((long long)rank * n / C), pb = int((long long)(rank + 1) * n / C);
  const int cnt = pb - pa > warp ? (pb - pa - warp + kUnitWarps - 1) / kUnitWarps : 0;
  const int32_t *table = a.block_tables + (long long)s * a.bt_stride;
  auto logical = [&](int i) {  // block of this warp's page i
    const int v = pa + warp + i * kUnitWarps;
    return v < front ? v : v + skip;
  };
  auto entry = [&](int i) { return i < cnt ? __ldg(table + logical(i)) : -1; };
  int ent = entry(lane), ent_next = entry(32 + lane);  // of the 32 pages being issued, and of the next 32
  // Q: rows 0-3 the group's query heads, rows 4-7 the same again
  uint32_t qa[4][2];
  {
    const uint32_t *row = a.q + ((long long)s * kQHeads + g * kGroup + ((lane >> 2) & 3)) * (kHeadDim / 2);
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      qa[ks][0] = __ldg(row + ks * 8 + (lane & 3));
      qa[ks][1] = __ldg(row + ks * 8 + 4 + (lane & 3));
    }
  }
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&sm.full[warp][i], 1);
    mbar_init_fence();
    if (warp == 0) {
      prefetch_tensormap(&a.tmap_k);
      prefetch_tensormap(&a.tmap_v);
    }
  }
  __syncwarp();
  // no CTA writes into another's shared memory before that one has started: this arrival, waited for before the push
  if (C > 1) cluster_arrive_relaxed();
  griddep_wait();  // pages and sums may have been written by the kernel before this one
  // (not before the wait: what the next kernel reads at once may come from a kernel before this one)
  griddep_launch_dependents();

  const uint64_t policy = policy_evict_first();
  int issued = 0, ist = 0;  // pages issued, stage of the next one
  unsigned bad = 0;         // bit st: the page in stage st has an invalid id
  auto issue = [&]() {
    if (issued > 0 && (issued & 31) == 0) {
      ent = ent_next;
      ent_next = entry(issued + 32 + lane);
    }
    const int page = __shfl_sync(0xffffffffu, ent, issued & 31);
    const bool ok = unsigned(page) < unsigned(a.num_pages);
    bad = ok ? bad & ~(1u << ist) : bad | (1u << ist);
    if (lane == 0) {
      if (ok) {
        mbar_arrive_expect_tx(&sm.full[warp][ist], 2 * kBoxBytes);
        tma_load_3d(sm.kv[warp][ist][0], &a.tmap_k, 0, g * kPageTokens, page, &sm.full[warp][ist], policy);
        tma_load_3d(sm.kv[warp][ist][1], &a.tmap_v, 0, g * kPageTokens, page, &sm.full[warp][ist], policy);
      } else {
        report(a.status, PKV_DEV_BAD_PAGE);
        mbar_arrive(&sm.full[warp][ist]);
      }
    }
    __syncwarp();
    ++issued;
    if (++ist == kStages) ist = 0;
  };
  for (int i = 0; i < kStages && i < cnt; ++i) issue();

  float4 *sc = nullptr;  // scores of this CTA's pages, [page - pa][token], one value for each of the four query heads
  if (kWeights)
    sc = a.scores != nullptr ? a.scores + ((long long)unit * a.score_pages + pa) * kPageTokens
                             : reinterpret_cast<float4 *>(reinterpret_cast<uint8_t *>(&sm) + sizeof(Smem));

  const int quad = lane & 3, hrow = lane >> 2;
  const int mi = lane >> 3, ri = lane & 7;  // ldmatrix: lane i addresses row i % 8 of matrix i / 8
  const uint32_t krow = uint32_t((((mi >> 1) << 3) + ri) * kRowBytes);
  const uint32_t kchunk = uint32_t(mi & 1);
  const uint32_t vrow = uint32_t((((mi & 1) << 3) + ri) * kRowBytes);
  const uint32_t vchunk = uint32_t(mi >> 1);
  float m_run = -INFINITY, l_run = 0.f;
  float acc[8][2];
#pragma unroll
  for (int nd = 0; nd < 8; ++nd) acc[nd][0] = acc[nd][1] = 0.f;

  int st = 0;
  uint32_t parity = 0;
  for (int i = 0; i < cnt; ++i) {
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp][st], parity))) {
      // give up: what is in flight lands (bounded again) before the CTA may end
      report(a.status, PKV_DEV_TIMEOUT);
      if (lane == 0)
        for (int j = i; j < issued; ++j) mbar_wait(&sm.full[warp][j % kStages], uint32_t(j / kStages) & 1);
      __syncwarp();
      break;
    }
    const int t0 = logical(i) * kPageTokens;
    float x[2][2] = {{-INFINITY, -INFINITY}, {-INFINITY, -INFINITY}};
    if (!((bad >> st) & 1)) {
      const uint32_t kbase = smem_addr(sm.kv[warp][st][0]), vbase = smem_addr(sm.kv[warp][st][1]);
      // ---- S = Q K^T: two n-tiles of 8 tokens, four k-steps of 16 dims ----
      float sv[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        uint32_t b00, b01, b10, b11;
        ldmatrix_x4(kbase + krow + (((2 * ks + kchunk) ^ ri) << 4), b00, b01, b10, b11);
        mma_16816(sv[0], qa[ks][0], 0u, qa[ks][1], 0u, b00, b01);
        mma_16816(sv[1], qa[ks][0], 0u, qa[ks][1], 0u, b10, b11);
      }
      // visible tokens of the page; this lane's are 8 nt + 2 quad + j
      const int to = min(kPageTokens, ctx - t0);
      unsigned vis = (1u << to) - 1u;
      if (t0 < lo) {
        const unsigned before = lo - t0 >= kPageTokens ? 0xffffu : (1u << (lo - t0)) - 1u;
        const unsigned sinks = sink - t0 >= kPageTokens ? 0xffffu : sink > t0 ? (1u << (sink - t0)) - 1u : 0u;
        vis &= ~before | sinks;
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if ((vis >> (8 * nt + 2 * quad + j)) & 1) x[nt][j] = sv[nt][j] * a.scale_log2;
      float mx = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float m_new = fmaxf(m_run, mx), m_use = finite_max(m_new);
      const float alpha = ex2_approx(m_run - m_use);
      float p[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) p[nt][j] = ex2_approx(x[nt][j] - m_use);
      l_run = l_run * alpha + ((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]));
      m_run = m_new;
      // the weights as three bf16 terms; rows 0-3 carry the high and (8-11) the middle one, rows 4-7 the low one
      uint32_t pa0[2], pa1[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const uint32_t hi = pack_bf16x2(p[nt][0], p[nt][1]);
        const float r0 = p[nt][0] - bf16_lo(hi), r1 = p[nt][1] - bf16_hi(hi);
        const uint32_t mid = pack_bf16x2(r0, r1);
        const uint32_t low = pack_bf16x2(r0 - bf16_lo(mid), r1 - bf16_hi(mid));
        pa0[nt] = hrow < kGroup ? hi : low;
        pa1[nt] = hrow < kGroup ? mid : 0u;
      }
      // V fragments hold tokens 2 quad (+1) and 8 + 2 quad (+1): zero those that are not visible
      const unsigned v_lo = vis >> (2 * quad), v_hi = vis >> (8 + 2 * quad);
      const uint32_t mask_lo = ((v_lo & 1) ? 0x0000ffffu : 0u) | ((v_lo & 2) ? 0xffff0000u : 0u);
      const uint32_t mask_hi = ((v_hi & 1) ? 0x0000ffffu : 0u) | ((v_hi & 2) ? 0xffff0000u : 0u);
      // ---- O = alpha O + P V: eight n-tiles of 8 dims, one k-step of 16 tokens ----
#pragma unroll
      for (int nd = 0; nd < 8; nd += 2) {
        uint32_t v0, v1, v2, v3;
        ldmatrix_x4_trans(vbase + vrow + (((nd + vchunk) ^ ri) << 4), v0, v1, v2, v3);
        float d0[4], d1[4];
        mma_16816_zero(d0, pa0[0], pa1[0], pa0[1], pa1[1], v0 & mask_lo, v1 & mask_hi);
        mma_16816_zero(d1, pa0[0], pa1[0], pa0[1], pa1[1], v2 & mask_lo, v3 & mask_hi);
        acc[nd][0] = fmaf(acc[nd][0], alpha, d0[0] + d0[2]);
        acc[nd][1] = fmaf(acc[nd][1], alpha, d0[1] + d0[3]);
        acc[nd + 1][0] = fmaf(acc[nd + 1][0], alpha, d1[0] + d1[2]);
        acc[nd + 1][1] = fmaf(acc[nd + 1][1], alpha, d1[1] + d1[3]);
      }
    }
    if (kWeights && hrow < kGroup) {
      float *dst = reinterpret_cast<float *>(sc + (warp + i * kUnitWarps) * kPageTokens) + hrow;
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) dst[(8 * nt + 2 * quad + j) * kGroup] = x[nt][j];
    }
    __syncwarp();  // the stage has been read by every lane
    if (issued < cnt) issue();
    if (++st == kStages) {
      st = 0;
      parity ^= 1;
    }
  }

  // ---- the CTA's state: thread i owns output value i = 64 head + dim ----
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 1);
  l_run += __shfl_xor_sync(0xffffffffu, l_run, 2);
#pragma unroll
  for (int nd = 0; nd < 8; ++nd) {
    const float v0 = acc[nd][0] + __shfl_xor_sync(0xffffffffu, acc[nd][0], 16);  // the low term of the same head
    const float v1 = acc[nd][1] + __shfl_xor_sync(0xffffffffu, acc[nd][1], 16);
    if (hrow < kGroup) *reinterpret_cast<float2 *>(&sm.acc[warp][hrow][8 * nd + 2 * quad]) = make_float2(v0, v1);
  }
  if (hrow < kGroup && quad == 0) sm.ml[warp][hrow] = make_float2(m_run, l_run);
  // the sums of the CTA's first tokens, on their way while the states are merged
  const int first = pa * kPageTokens, behind = int(min((long long)ctx, (long long)pb * kPageTokens));
  float *sums = kWeights ? a.sums + (long long)s * a.seq_stride + (long long)g * a.head_stride : nullptr;
  float old[kSumsAhead];
  if (kWeights) {
#pragma unroll
    for (int i = 0; i < kSumsAhead; ++i) {
      const int t = first + tid + i * kUnitThreads;
      old[i] = t < behind && a.decay != 0.f ? sums[t] : 0.f;
    }
  }
  __syncthreads();
  const int h = tid / kHeadDim, d = tid % kHeadDim;
  float M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
  for (int w = 0; w < kUnitWarps; ++w) M = fmaxf(M, sm.ml[w][h].x);
#pragma unroll
  for (int w = 0; w < kUnitWarps; ++w) {
    const float2 ml = sm.ml[w][h];
    const float f = ex2_approx(ml.x - finite_max(M));
    L = fmaf(ml.y, f, L);
    A = fmaf(sm.acc[w][h][d], f, A);
  }
  if (C == 1) {
    store(tid, L != 0.f ? A / L : 0.f);
    if (kWeights && d == 0) sm.fin[h] = make_float2(finite_max(M), L != 0.f ? 1.f / L : 0.f);
    if (kWeights) __syncthreads();
  } else {
    // CTA r of the cluster finishes the output values [r 256 / C, (r + 1) 256 / C): it gets that slice from every CTA, and
    // every CTA gets every maximum and sum
    const int slice = kUnitOut / C;
    cluster_wait();
    st_cluster_f1(cluster_map(smem_addr(&sm.recv_acc[rank * slice + tid % slice]), uint32_t(tid / slice)), A);
    if (d < C) st_cluster_f2(cluster_map(smem_addr(&sm.recv_ml[rank][h]), uint32_t(d)), make_float2(M, L));
    cluster_sync();
    if (tid < slice || (kWeights && tid < kGroup)) {
      const int i = rank * slice + tid;
      const bool outs = tid < slice;
      // (with weight sums threads 0-3 look after heads 0-3 as well; a slice holds 16 values or more)
#pragma unroll 1
      for (int k = outs ? 0 : 1; k < (kWeights && tid < kGroup ? 2 : 1); ++k) {
        const int hh = k == 0 ? i / kHeadDim : tid;
        float m = -INFINITY, l = 0.f, o = 0.f;
        for (int c = 0; c < C; ++c) m = fmaxf(m, sm.recv_ml[c][hh].x);
        m = finite_max(m);
        for (int c = 0; c < C; ++c) {
          const float2 ml = sm.recv_ml[c][hh];
          const float f = ex2_approx(ml.x - m);
          l = fmaf(ml.y, f, l);
          if (k == 0) o = fmaf(sm.recv_acc[c * slice + tid], f, o);
        }
        if (k == 0)
          store(i, l != 0.f ? o / l : 0.f);
        else
          sm.fin[hh] = make_float2(m, l != 0.f ? 1.f / l : 0.f);
      }
    }
    if (kWeights) __syncthreads();
  }
  if (kWeights) {
    const float2 f0 = sm.fin[0], f1 = sm.fin[1], f2 = sm.fin[2], f3 = sm.fin[3];
    auto add = [&](int t, float before) {
      const float4 x = sc[t - first];
      const float w = (ex2_approx(x.x - f0.x) * f0.y + ex2_approx(x.y - f1.x) * f1.y) +
                      (ex2_approx(x.z - f2.x) * f2.y + ex2_approx(x.w - f3.x) * f3.y);
      sums[t] = a.decay == 0.f ? w : fmaf(a.decay, before, w);
    };
#pragma unroll
    for (int i = 0; i < kSumsAhead; ++i) {
      const int t = first + tid + i * kUnitThreads;
      if (t < behind) add(t, old[i]);
    }
#pragma unroll 4
    for (int t = first + tid + kSumsAhead * kUnitThreads; t < behind; t += kUnitThreads)
      add(t, a.decay == 0.f ? 0.f : sums[t]);
  }
}

template <int kStages>
constexpr size_t unit_smem_bytes() { return sizeof(UnitSmem<kStages>) + 1024; }
constexpr size_t kPairSmem = 227 * 1024 / 2 - 1024;  // shared memory of a CTA that shares its SM with another one
constexpr int kPairPages = int((kPairSmem - unit_smem_bytes<kShallowRing>()) / kScorePage);  // whose scores fit then: 150

// Shared-memory limits of the kernels on the current device.
int setup_unit_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    const struct {
      void (*kernel)(UnitArgs);
      size_t bytes;
    } all[] = {{unit_decode_kernel<false, kDeepRing>, unit_smem_bytes<kDeepRing>()},
               {unit_decode_kernel<true, kDeepRing>, unit_smem_bytes<kDeepRing>() + kChipPages * kScorePage},
               {unit_decode_kernel<true, kShallowRing>, unit_smem_bytes<kShallowRing>() + kChipPages * kScorePage}};
    for (const auto &k : all)
      if (cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(k.bytes)) != cudaSuccess ||
          cudaFuncSetAttribute(k.kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
      }
    done[dev] = true;
  }
  return PKV_OK;
}

// Pages that a unit sees at the most, given the bound on the lengths.
long long max_unit_pages(int max_context, int window, int sinks) {
  const long long all = ((long long)max_context + kPageTokens - 1) / kPageTokens;
  const long long seen = ((long long)sinks + kPageTokens - 1) / kPageTokens +
                         ((long long)window + kPageTokens - 2) / kPageTokens + 1;
  return all < seen ? all : seen;
}

// CTAs to a unit: as many as fill the SMs with two each, as long as each gets a few pages.  1 / 2 / 4 / 8 of them: one
// sequence, window of 512 (34 pages), 5.4 / 5.2 / 4.5 / 4.0 us; weight sums of one sequence of 2048, 14.9 / 10.3 / 7.4 /
// 5.8; 64 windows of up to 1000 (512 units) 24.4 / 31.2 / 38.6 / 63.2; 256 windows of 2032 157 / 166 / 202 / 296.  16 (a
// cluster of them takes most of a GPC, so no more than one for each) where there are twice as many pages still: windows of
// 32768 19.0 us for 23.7, of 4096 5.7 for 6.5, of 1000 4.3 for 4.0; two sequences, windows of 8192, 12.4 for 10.7.
int unit_cluster(long long units, long long pages, int most) {
  const int sms = device_sm_count();
  const long long slots = 2ll * (sms > 0 ? sms : 148);
  int c = 1;
  while (c < kFarCluster && units * c * 2 <= slots && pages >= 2ll * c * kMinPages) c *= 2;
  if (c == kFarCluster && most > c && units * most * 2 <= slots && pages >= 2ll * most * kMinPages) c = most;
  return c;
}

// Common part of the two entry points; `sums` null: window decode.
int unit_decode(const pkv_pool *pool, void *out, const void *q, const int32_t *block_tables, int64_t bt_stride,
                const int32_t *context_lens, int num_seqs, int max_context, float scale, int window, int sinks, float *sums,
                int64_t seq_stride, int64_t head_stride, float decay, void *workspace, int32_t *device_status,
                unsigned flags, void *stream) {
  UnitArgs a;
  int rc = pool_tensor_maps(pool, kPageTokens, &a.tmap_k, &a.tmap_v);
  if (rc != PKV_OK) return rc;
  rc = setup_unit_attributes();
  if (rc != PKV_OK) return rc;
  const long long units = (long long)num_seqs * kKvHeads;
  const long long pages = max_unit_pages(max_context, window, sinks);
  a.num_pages = pool->num_pages;
  a.q = static_cast<const uint32_t *>(q);
  a.out = out;
  a.out_bf16 = (flags & PKV_OUT_BF16) ? 1 : 0;
  a.block_tables = block_tables;
  a.bt_stride = bt_stride;
  a.context_lens = context_lens;
  a.max_context = max_context;
  a.window = window;
  a.sinks = sinks;
  a.scale_log2 = scale * kLog2e;
  const bool paired = sums == nullptr || pages <= kMaxCluster * kPairPages;  // two CTAs find room on an SM
  a.cluster = unit_cluster(units, pages, paired ? kMaxCluster : kFarCluster);
  // More units than are resident at once, but not many times as many, and lengths that may differ: the longest first, so
  // that no long one is left at the end (weight sums of 64 sequences of 1 .. 2048 tokens: 23.5 us for 25.2).  Windows of
  // 1000 over 1 .. 8192 tokens, most of them full, take 26.1 us so and 24.2 without; batches of many rounds gain nothing.
  const int sms = device_sm_count();
  const bool whole = (long long)window + sinks >= max_context;
  a.sort = a.cluster == 1 && whole && units > 2ll * (sms > 0 ? sms : 148) && num_seqs <= kMaxSorted ? num_seqs : 0;
  a.sums = sums;
  a.seq_stride = seq_stride;
  a.head_stride = head_stride;
  a.decay = decay;
  a.scores = nullptr;
  a.score_pages = pages;
  a.status = device_status;
  void (*kernel)(UnitArgs) = unit_decode_kernel<false, kDeepRing>;
  size_t smem = unit_smem_bytes<kDeepRing>();
  if (sums != nullptr) {
    kernel = unit_decode_kernel<true, kDeepRing>;
    // Shares small enough for two CTAs to an SM, where clusters of 8 get that far: 32 sequences of 16384 tokens take 190 us
    // (220 with one), 8 of them 47 (57), 64 of 4096 101 (110), 64 of 1 .. 8192 110 (114), 40 of 1 .. 4096 36.8 (36.3).
    // Else shares that fit at all (the workspace takes as long, 217 us for 219, but needs 256 bytes a page).
    const int most = paired ? kPairPages : kChipPages;
    while (a.cluster < (paired ? kMaxCluster : kFarCluster) && (pages + a.cluster - 1) / a.cluster > most) a.cluster *= 2;
    const long long share = (pages + a.cluster - 1) / a.cluster;
    if (share <= kChipPages) {
      const size_t scores = size_t(share) * kScorePage;
      // the ring of two stages where it brings a second CTA to the SM: 256 sequences of 2048 tokens 177 us (210 with three
      // stages)
      if (smem + scores > kPairSmem && unit_smem_bytes<kShallowRing>() + scores <= kPairSmem) {
        kernel = unit_decode_kernel<true, kShallowRing>;
        smem = unit_smem_bytes<kShallowRing>();
      }
      smem += scores;
    } else {
      a.scores = static_cast<float4 *>(workspace);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(units * a.cluster));
  cfg.blockDim = dim3(kUnitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  int n_attr = 0;
  if (a.cluster > 1) {
    attr[n_attr].id = cudaLaunchAttributeClusterDimension;
    attr[n_attr].val.clusterDim.x = unsigned(a.cluster);
    attr[n_attr].val.clusterDim.y = 1;
    attr[n_attr].val.clusterDim.z = 1;
    ++n_attr;
  }
  if (flags & PKV_OVERLAP_PREVIOUS) {
    attr[n_attr].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n_attr].val.programmaticStreamSerializationAllowed = 1;
    ++n_attr;
  }
  cfg.attrs = attr;
  cfg.numAttrs = unsigned(n_attr);
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, a);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_LAUNCH;
  }
  return PKV_OK;
}

// Checks that both entry points make; num_seqs = 0 is left to the caller.
int check_unit_call(const pkv_pool *pool, const void *out, const void *q, int num_q_heads, const int32_t *block_tables,
                    int64_t bt_stride, const int32_t *context_lens, int num_seqs, int max_context, float scale,
                    unsigned flags) {
  if (flags & ~unsigned(PKV_OVERLAP_PREVIOUS | PKV_OUT_BF16)) return PKV_ERR_SHAPE;
  const int rc = check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_q_heads != kQHeads) return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_seqs > (1 << 24) || max_context < 0 || max_context > kMaxTokens || bt_stride < 0)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  if (out == nullptr || q == nullptr || block_tables == nullptr || context_lens == nullptr) return PKV_ERR_NULL;
  if (!isfinite(scale) || !isfinite(scale * kLog2e)) return PKV_ERR_SCALE;
  if (!aligned16(q) || !aligned16(out) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
      (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return PKV_ERR_ALIGN;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_paged_window_decode_attention(const pkv_pool *pool, void *out, const void *q, int num_q_heads,
                                                 const int32_t *block_tables, int64_t block_table_stride,
                                                 const int32_t *context_lens, int num_seqs, int max_context,
                                                 float scale, int window, int sinks, int32_t *device_status,
                                                 unsigned flags, void *stream) {
  const int rc = pkv::check_unit_call(pool, out, q, num_q_heads, block_tables, block_table_stride, context_lens,
                                      num_seqs, max_context, scale, flags);
  if (rc != PKV_OK) return rc;
  if (window < 1 || sinks < 0) return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  return pkv::unit_decode(pool, out, q, block_tables, block_table_stride, context_lens, num_seqs, max_context, scale,
                          window, sinks, nullptr, 0, 0, 0.f, nullptr, device_status, flags, stream);
}

extern "C" size_t pkv_weights_workspace_bytes(int num_seqs, int max_context) {
  if (num_seqs < 0 || num_seqs > (1 << 24) || max_context < 0 || max_context > (1 << 30)) return 0;
  const long long pages = ((long long)max_context + pkv::kPageTokens - 1) / pkv::kPageTokens;
  if (pages <= (long long)pkv::kFarCluster * pkv::kChipPages) return 0;
  return size_t(num_seqs) * pkv::kKvHeads * size_t(pages) * pkv::kScorePage;
}

extern "C" int pkv_paged_decode_attention_weights(const pkv_pool *pool, void *out, const void *q, int num_q_heads,
                                                  const int32_t *block_tables, int64_t block_table_stride,
                                                  const int32_t *context_lens, int num_seqs, int max_context,
                                                  float scale, float *weight_sums, int64_t seq_stride,
                                                  int64_t head_stride, float decay, void *workspace,
                                                  size_t workspace_bytes, int32_t *device_status, unsigned flags,
                                                  void *stream) {
  const int rc = pkv::check_unit_call(pool, out, q, num_q_heads, block_tables, block_table_stride, context_lens,
                                      num_seqs, max_context, scale, flags);
  if (rc != PKV_OK) return rc;
  if (!(decay >= 0.f && decay <= 1.f)) return PKV_ERR_SCALE;
  constexpr int64_t kFar = int64_t(1) << 38;  // (no array has as many elements; a stride times a count stays within 64 bits)
  if (max_context > (1 << 30) || seq_stride > kFar || head_stride > kFar) return PKV_ERR_SHAPE;
  // heads, and sequences, may not share a row of sums
  const bool heads_inside = head_stride >= max_context && (num_seqs <= 1 || seq_stride >= pkv::kKvHeads * head_stride);
  const bool seqs_inside = num_seqs > 1 && seq_stride >= max_context && head_stride >= seq_stride * num_seqs;
  if (head_stride < 0 || seq_stride < 0 || (!heads_inside && !seqs_inside)) return PKV_ERR_SHAPE;
  if (num_seqs == 0) return PKV_OK;
  if (weight_sums == nullptr && max_context > 0) return PKV_ERR_NULL;
  if (reinterpret_cast<uintptr_t>(weight_sums) & 3u) return PKV_ERR_ALIGN;
  const size_t need = pkv_weights_workspace_bytes(num_seqs, max_context);
  if (need > 0 && workspace == nullptr) return PKV_ERR_NULL;
  if (need > 0 && !pkv::aligned16(workspace)) return PKV_ERR_ALIGN;
  if (workspace_bytes < need) return PKV_ERR_WORKSPACE;
  return pkv::unit_decode(pool, out, q, block_tables, block_table_stride, context_lens, num_seqs, max_context, scale,
                          0x7fffffff, 0, weight_sums, seq_stride, head_stride, decay, workspace, device_status, flags,
                          stream);
}
