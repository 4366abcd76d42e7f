// Paged prefill attention with a sliding window and sinks: the last n_s tokens of each sequence attend to the `window`
// tokens up to and including their own position and to the first `sinks` tokens of the sequence,
//
//   out[i][h] = sum_{t in A} w_t V_t[h/4],  w = softmax_{t in A}(scale q[i][h] . K_t[h/4]),
//   A = { t <= p : t < sinks or t > p - window },  p = context_lens[s] - n_s + (i - query_start[s]).
//
// tcgen05 tensor cores, accumulators in tensor memory:
//  * An item is 64 query tokens of a sequence against one K/V head: two tiles of 32 tokens, 128 rows each (row = 4 * token
//    + head in group).  Both tiles use each K/V block that is loaded, or one of them where the other sees nothing of it.
//    The pages that the item's rows see (the sinks' and those from the first row's window on; none between) are numbered
//    without the gap and go eight to a block of 128 keys, so that the sinks cost a page and not a block.  Where there are
//    fewer items than half the SMs, they have one tile.  Where no sequence has more than 32 query tokens, and there are
//    more sequences than fill the SMs, an item is one tile's tokens against two K/V heads, a tile each.
//  * The grid is persistent, one CTA to an SM; the items that there are (a prefix sum over the sequences' lengths, made by
//    every CTA) are dealt in a snake, each sequence's latest first.
//  * A block's S_t = Q_t K^T is computed in two halves of 64 keys, into TMEM buffers of their own; P goes back over its half
//    and is the TMEM A operand of O_t += P V.  So while the softmax works on one half the tensor core has P V of the other and
//    its next S.  With bf16 output P has one bf16 term, and Q stays in tensor memory (its rows' own threads put it there), so
//    that shared memory feeds the tensor core K and V alone.  With fp32 output P has three bf16 terms, 24 bits (with two,
//    the weights' rounding alone is 1.7e-6 of the output's norm); the third ones take Q's place and more, and Q lies in
//    shared memory.  Row sums are added up in registers.
//  * The exponents of a row refer to the largest score of some keys of its tile's first block, seen by the row or by another
//    one of the item, and stay there: weights are floats, so they may well be far from 1.  A row whose sum leaves
//    [2^-90, 2^112] is computed again.
//  * The tensor core truncates what it adds up.  O is therefore taken out after every run of 256 keys (fp32 output) or 16384
//    keys (bf16 output: one run over 2^24 equal weights lost 15 %), and runs are added up, with rounding, in shared memory.
//    fp32 output, windows of 128 / 1000 / 15000: runs of 128 keys have errors of 3.0e-7 / 5.0e-7 / 6.8e-7 of the output's norm,
//    of 256 4.4e-7 / 8.5e-7 / 9.6e-7, of 1024 4.4e-7 / 2.9e-6 / 3.1e-6; fp32 arithmetic in torch 2.6e-7 / 6.3e-7 / 2.2e-6.
//    128 instead of 256 keys take 6 % more time for windows of 128 and 11 % for long ones, 1024 save 6 % there.
//  * A warp's finished rows go through the same shared memory and a TMA store: stored by their threads, 256 bytes apart, they
//    took 3400 cycles a tile.  (The last few tokens of a sequence, where a box would reach into the next one, are stored
//    directly.)
//  * Keys that a row does not see get weight 0.  Their V meets that weight in the product all the same, so a NaN or an
//    infinity in it would reach rows that do not see it: a row whose output is not finite is computed again at the end,
//    from the keys that it sees alone, by its own thread (slowly).
//  * Warps 0-3 and 4-7 own a row of tile 0 and 1 a thread.  Warp 8 loads by TMA; warps 9 and 10 issue the MMAs of a tile
//    each.
//  * Every mbarrier wait is bounded (about 2 s): on expiry the CTA reports PKV_DEV_TIMEOUT, stops issuing work, waits
//    (bounded) for what is in flight, frees its tensor memory and exits.
//
// What bounds it: 4 x 2048 queries, windows of 2000, bf16 output, take 143 us (135 GFLOP, 946 TFLOP/s, half of the measured
// bf16 peak): tensor pipe 42 %, exponentials 40 %, issue slots 45 %, so nothing is full; two softmax warps a scheduler wait
// for S, exponentials and stores in turn, and registers (168 a thread) and tensor memory (all 512 columns are taken) leave
// no room for a third.  Built and slower: two CTAs to an SM with one S buffer a tile (151 to 161 us), one issuing warp for
// both tiles (62 cycles a product), softmax warps that issue for themselves (166).  With fp32 output P V is
// three times the products and a weight 2.5 times the instructions: 2048 queries, windows of 4096, 154 us for 77 (121 with two
// terms and runs of 1024 keys).  Short windows: 16 x 300..512 queries, windows of 128, fp32 in 41 us, some 13000 cycles an item
// of two blocks, of them 2000 waiting for its S, 1800 taking out the O before it, the rest four masked halves.  200 queries
// of one sequence: 11.2 to 11.6 us, the latencies of one item (lists and set-up 2, first K/V 2, blocks and output the rest).
#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <mutex>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kWpTok = 32;                             // query tokens of a tile
constexpr int kWpTiles = 2;                            // tiles of an item
constexpr int kWpItemTok = kWpTok * kWpTiles;
constexpr int kWpRows = kWpTok * kGroup;               // M = 128
constexpr int kWpKeys = 128;                           // keys of a block
constexpr int kWpPagesPerBlock = kWpKeys / kPageTokens;
constexpr unsigned kWpStages = 4;                      // K/V blocks in flight
constexpr int kWpThreads = kWpTiles * kWpRows + 96;    // softmax groups, loader, issuers
constexpr int kWpLoader = kWpTiles * 4, kWpIssuers = kWpLoader + 1;  // warps
constexpr int kWpHalf = kWpKeys / 2;                   // keys of an S buffer
template <bool kBf16>
constexpr int kWpMaxItems = kBf16 ? 64 : 32;           // items a CTA walks (its table in shared memory)
constexpr int kWpBox = kPageTokens * kRowBytes;        // one head's rows of one page: 2 KiB
constexpr int kWpTileBytes = kWpKeys * kRowBytes;      // K (or V) of one block: 16 KiB
template <bool kBf16>
constexpr int kWpRun = kBf16 ? 128 : 2;                // blocks that O adds up at once
constexpr int kWpSumRun = 8;                           // blocks whose weights are added up at once
constexpr int kWpStretch = 16;                         // pages that a row computed again adds up at once
constexpr uint32_t kWpTmemCols = 512;
// columns of S_0, S_1 (128 each) and of O_0, O_1 (64); then with bf16 output of Q_0, Q_1 (32), with fp32 output of the third
// terms of P_0, P_1 (64)
constexpr uint32_t kColS = 0, kColO = kWpTiles * kWpKeys, kColQ = kColO + kWpTiles * kHeadDim, kColLow = kColQ;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kSumMin = 8.077935669463161e-28f, kSumMax = 5.192296858534828e33f;  // 2^-90, 2^112

constexpr uint32_t kIdescS = idesc_bf16(kWpRows, kWpHalf, false);   // B = K rows (K-major)
constexpr uint32_t kIdescPV = idesc_bf16(kWpRows, kHeadDim, true);  // B = V (MN-major)

// A box from shared memory to global memory, in the thread's bulk group.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int x, int y, int z, const void *smem_src) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
               "r"(y), "r"(z), "r"(smem_addr(smem_src))
               : "memory");
}

struct WindowArgs {
  CUtensorMap tmap_k;  // boxes of one head's 16 rows of one page
  CUtensorMap tmap_v;
  CUtensorMap tmap_q;  // with fp32 output: boxes of 8 query rows x one group's 4 heads
  CUtensorMap tmap_o;  // boxes of 8 output rows x one group's 4 heads x 128 bytes
  int num_pages;
  void *out;       // [total][32][64] fp32 or bf16
  const uint16_t *q;
  const uint8_t *k_base, *v_base;
  long long page_stride;
  int window, sinks;
  const int32_t *query_start;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int num_seqs;
  int num_q_rows;
  int max_context;
  int max_query;
  int item_tok;       // query tokens of an item: 64, or 32 (its first tile alone)
  int items_per_seq;  // of max_query query tokens and one K/V head
  int most_items;     // num_seqs * items_per_seq * 8, or 4 where the tiles take a K/V head each
  float scale_log2;  // scale * log2(e)
  int32_t *status;
};

// One item: item_tok query tokens of sequence s (from t0) against K/V head g.
struct WpItem {
  int s, g, t0, n, q0, ctx, nblocks;
  int npages;  // pages its rows see
  int front;   // of them the sinks' pages before the window
  int skip;    // pages between that no row sees
  int run;      // valid lengths
  int invalid;  // invalid ones: its rows are zeroed
};

template <bool kBf16>
struct __align__(1024) WpSmem {
  uint8_t k[kWpStages][kWpTileBytes];  // 128 keys x 128 B per stage, 128-byte swizzled
  uint8_t v[kWpStages][kWpTileBytes];
  uint8_t q[kBf16 ? 0 : kWpTiles][kWpRows * kRowBytes];  // with fp32 output: Q, 128-byte swizzled
  uint8_t rows[kWpTiles * 4][2][32 * 128];  // a warp's rows, 128 bytes of each at a time, swizzled: sums of runs, then the output
  uint64_t q_full[kWpTiles];  // the tile's Q is there (in tensor memory: a warp arrives once)
  uint64_t kv_full[kWpStages], kv_empty[kWpStages];
  uint64_t s_full[kWpTiles][2];  // S of the half of the tile's next block is there, and its bad pages are known
  uint64_t p_full[kWpTiles][2];  // every row of P of it (a warp arrives once), and O has been read where it starts anew
  uint64_t o_full[kWpTiles];  // the P V that ends a run, or the item, is done
  uint64_t mma_done[kWpTiles];
  int kv_bad[kWpStages];  // bit pp set when page pp of the block is invalid (loaded as zeros)
  WpItem items[kWpMaxItems<kBf16>];  // this CTA's, in walking order
  int warp_sum[kWpThreads / 32];
  uint32_t tmem_base;
  int abort;
};
template <bool kBf16>
constexpr size_t kWpSmemBytes = sizeof(WpSmem<kBf16>) + 1024;
static_assert(kWpSmemBytes<false> <= 227 * 1024 && kWpSmemBytes<true> <= 227 * 1024, "");

// What an item of sequence s (query tokens t0 .. of n from row q0 on, ctx cached tokens) has to know.
__device__ __forceinline__ WpItem wp_item(const WindowArgs &a, int s, int g, int t0, int q0, int n, int ctx) {
  WpItem t;
  t.s = s;
  t.g = g;
  t.t0 = t0;
  t.q0 = q0;
  t.n = n;
  t.ctx = ctx;
  t.invalid = n > a.max_query || ctx < 0 || ctx > a.max_context || n > ctx || q0 < 0 || n > a.num_q_rows - q0;
  t.run = !t.invalid;
  const int first_pos = t.run ? ctx - n + t0 : 0, last_pos = t.run ? ctx - n + min(t0 + a.item_tok, n) - 1 : 0;
  const int lo = max(0, first_pos - a.window + 1), sink = min(a.sinks, lo);
  t.front = (sink + kPageTokens - 1) / kPageTokens;
  t.skip = max(lo / kPageTokens, t.front) - t.front;
  t.npages = last_pos / kPageTokens + 1 - t.skip;
  t.nblocks = (t.npages + kWpPagesPerBlock - 1) / kWpPagesPerBlock;
  return t;
}

// Block-table index of page v of an item.
__device__ __forceinline__ int logical_page(const WpItem &t, int v) { return v < t.front ? v : v + t.skip; }

// The blocks of an item that a tile uses: those with a key in [0, sinks) (j < sinks) or [first row's window, last row's
// position] (first <= j <= last).
struct WpTile {
  int sinks, first, last;  // last < 0: the tile has no queries
  __device__ __forceinline__ int begin() const { return sinks > 0 ? 0 : first; }
  __device__ __forceinline__ int next(int j) const { return j + 1 < first && j + 1 >= sinks ? first : j + 1; }
};
__device__ __forceinline__ WpTile tile_of(const WindowArgs &a, const WpItem &t, int tile) {
  const int t0 = t.t0 + tile * kWpTok, pos = t.ctx - t.n + t0;
  auto present = [&](int page) {  // number of the page, or of the next one that is there
    return page < t.front ? page : max(page - t.skip, t.front);
  };
  WpTile w;
  w.first = present(max(0, pos - a.window + 1) / kPageTokens) / kWpPagesPerBlock;
  w.last = -1;
  if (t0 < t.n && tile * kWpTok < a.item_tok)
    w.last = present((t.ctx - t.n + min(t0 + kWpTok, t.n) - 1) / kPageTokens) / kWpPagesPerBlock;
  w.sinks = (present(a.sinks / kPageTokens + (a.sinks % kPageTokens != 0)) + kWpPagesPerBlock - 1) / kWpPagesPerBlock;
  return w;
}

// Bounded wait of a whole warp that gives up once another role has; one answer for all lanes.  Returns true when the
// phase completed.
template <class Smem>
__device__ __forceinline__ bool wp_wait(Smem &sm, uint64_t *bar, uint32_t parity, int32_t *status) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_ns();
  while (!__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) {
    const bool late = global_ns() - t0 > kWaitLimitNs;
    if (__any_sync(0xffffffffu, late || *reinterpret_cast<volatile int *>(&sm.abort) != 0)) {
      if (__any_sync(0xffffffffu, late)) {
        *reinterpret_cast<volatile int *>(&sm.abort) = 1;
        report(status, PKV_DEV_TIMEOUT);
      }
      return false;
    }
  }
  return true;
}

// Bits [0, n) of 32.
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// Of 32 keys from `key` on, `gone` pages behind those that an item's numbering gives them: the ones in [0, pos] that lie at or
// past lo, or before `sinks` (where pages are left out, the sinks lie before them and the window behind).  Bits 0, 1 of `bad`:
// the keys' first, second page is invalid.
__device__ __forceinline__ uint32_t seen_keys(int key, int gone, int lo, int pos, int sinks, int bad) {
  const int d = gone * kPageTokens;  // (at most lo where pages are left out; key + d may pass 2^31)
  uint32_t seen = first_bits(pos + 1 - d - key) & (~first_bits(lo - d - key) | first_bits(sinks - key));
  if (bad & 1) seen &= 0xffff0000u;
  if (bad & 2) seen &= 0x0000ffffu;
  return seen;
}

// Largest (kMin: smallest) of a page's scores.
template <bool kMin>
__device__ __forceinline__ float extreme16(const uint32_t (&s)[16]) {
  auto of3 = [](float x, float y, float z) { return kMin ? min3f(x, y, z) : max3f(x, y, z); };
  float m[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    m[i] = of3(__uint_as_float(s[3 * i]), __uint_as_float(s[3 * i + 1]), __uint_as_float(s[3 * i + 2]));
  return of3(of3(m[0], m[1], m[2]), of3(m[3], m[4], __uint_as_float(s[15])), m[0]);
}

// P = 2^(s c - m) for 32 keys (with kMasked, keys whose bit in `valid` is clear get 0) as bf16 terms, stored in TMEM over the S
// that they come from, two keys to a column: one term with bf16 output; with fp32 output three (24 bits), the second ones
// behind the first, the third ones at `low`.  Complete after tmem_st_wait().  Returns the weights' sum.  (Sums of the
// rounded weights: with one term errors of 2.2e-3 for 2.3e-3, for 12 % of the time.)
template <bool kMasked, bool kBf16>
__device__ __forceinline__ float quarter_probs(const uint32_t (&s)[32], uint32_t valid, float m, float c, uint32_t taddr,
                                               uint32_t low) {
  const float2 c2 = make_float2(c, c), mc = make_float2(-m, -m);
  float2 sum[4] = {};
  constexpr int kStep = kBf16 ? 16 : 8;  // words stored at once
#pragma unroll
  for (int at = 0; at < 16; at += kStep) {
    uint32_t t0[kStep], t1[8], t2[8];
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
      const int i = at + k;
      const float2 e = fma_f32x2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c2, mc);
      float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
      if (kMasked) {
        p.x = (valid >> (2 * i)) & 1 ? p.x : 0.f;
        p.y = (valid >> (2 * i + 1)) & 1 ? p.y : 0.f;
      }
      sum[i % 4] = add_f32x2(sum[i % 4], p);
      t0[k] = pack_bf16x2(p.x, p.y);
      if constexpr (!kBf16) {
        p = sub_f32x2(p, make_float2(bf16_lo(t0[k]), bf16_hi(t0[k])));
        t1[k] = pack_bf16x2(p.x, p.y);
        p = sub_f32x2(p, make_float2(bf16_lo(t1[k]), bf16_hi(t1[k])));
        t2[k] = pack_bf16x2(p.x, p.y);
      }
    }
    if constexpr (kBf16) {
      tmem_st16_async(taddr, t0);
    } else {
      tmem_st8_async(taddr + at, t0);
      tmem_st8_async(taddr + 16 + at, t1);
      tmem_st8_async(low + at, t2);
    }
  }
  const float2 t = add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3]));
  return t.x + t.y;
}

// The same for keys that no row sees: zeros.
template <bool kBf16>
__device__ __forceinline__ void no_probs(uint32_t taddr, uint32_t low) {
  const uint32_t zero[16] = {};
  tmem_st16_async(taddr, zero);
  if (!kBf16) {
    tmem_st16_async(taddr + 16, zero);
    tmem_st16_async(low, zero);
  }
}

// 16 values of an output row from element `at` on, 16 bytes at a time.  (A store of 32 bytes, st.global.v8.f32, wrote only the
// first of its eight floats where rows are computed again, every time, whatever the row.)
template <bool kBf16Out>
__device__ __forceinline__ void store_row(void *out, long long at, const float (&v)[16]) {
  if (kBf16Out) {
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
#pragma unroll
    for (int c = 0; c < 16; c += 8)
      dst[c / 8] = make_uint4(pack_bf16x2(v[c], v[c + 1]), pack_bf16x2(v[c + 2], v[c + 3]),
                              pack_bf16x2(v[c + 4], v[c + 5]), pack_bf16x2(v[c + 6], v[c + 7]));
  } else {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
#pragma unroll
    for (int c = 0; c < 16; c += 4) dst[c / 4] = make_float4(v[c], v[c + 1], v[c + 2], v[c + 3]);
  }
}

// Row `tok` of item t, query head g * 4 + hh, from the keys that it sees alone: the maximum first, then the sums, those of
// kWpStretch pages by themselves, which are added up in the thread's 256 bytes of shared memory (in one sum over 28000 equal
// weights the additions lost 1.1e-4).
template <bool kBf16Out>
__device__ __noinline__ void recompute_row(const WindowArgs &a, const WpItem &t, int g, int tok, int hh, uint8_t *mine) {
  const int pos = t.ctx - t.n + t.t0 + tok;
  const long long row = ((long long)(t.q0 + t.t0 + tok) * kQHeads + g * kGroup + hh) * kHeadDim;
  const uint32_t *q = reinterpret_cast<const uint32_t *>(a.q + row);
  const int32_t *table = a.block_tables + (long long)t.s * a.bt_stride;
  const float scale = a.scale_log2;
  const int lo = max(0, pos - a.window + 1);
  float m = -INFINITY, l = 0.f, lost = 0.f;  // l and what its additions have lost so far
  bool nan = false;
  float o[4][16];  // the sums of the stretch
#pragma unroll
  for (int c = 0; c < 64; ++c) o[c / 16][c % 16] = 0.f;
  auto sum = [&](int c) {  // 4 c .. 4 c + 3 of the stretches before
    return reinterpret_cast<float4 *>(mine + (c / 8) * 4096 + (((c % 8) ^ (threadIdx.x & 7)) << 4));
  };
  auto add = [&](int c, float4 x) {
    float *y = &o[c / 4][c % 4 * 4];
    return make_float4(x.x + y[0], x.y + y[1], x.z + y[2], x.w + y[3]);
  };
#pragma unroll
  for (int c = 0; c < 16; ++c) *sum(c) = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && m == -INFINITY) m = 0.f;
#pragma unroll 1
    for (int v = 0; v < t.npages; ++v) {
      if (v % kWpStretch == 0) {
#pragma unroll
        for (int c = 0; c < 16; ++c) *sum(c) = add(c, *sum(c));
#pragma unroll
        for (int c = 0; c < 64; ++c) o[c / 16][c % 16] = 0.f;
      }
      const int lp = logical_page(t, v), page = __ldg(table + lp);
      if (unsigned(page) >= unsigned(a.num_pages)) continue;
      const long long at = page * a.page_stride + (long long)g * kWpBox;
#pragma unroll 1
      for (int r = 0; r < kPageTokens; ++r) {
        const int key = lp * kPageTokens + r;
        if (key > pos || (key >= a.sinks && key < lo)) continue;
        const uint4 *kr = reinterpret_cast<const uint4 *>(a.k_base + at + r * kRowBytes);
        float d = 0.f;
#pragma unroll 1
        for (int c = 0; c < 8; ++c) {
          const uint4 k4 = kr[c];
          const uint32_t kw[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t qw = __ldg(q + 4 * c + i);
            d = fmaf(bf16_lo(qw), bf16_lo(kw[i]), d);
            d = fmaf(bf16_hi(qw), bf16_hi(kw[i]), d);
          }
        }
        const float x = d * scale;
        if (pass == 0) {
          m = fmaxf(m, x);
          nan |= x != x || x == INFINITY;  // a maximum of +infinity leaves no softmax
          continue;
        }
        const float p = ex2_approx(x - m), y = p - lost, sum = l + y;
        lost = (sum - l) - y;
        l = sum;
        if (p == 0.f) continue;
        const uint4 *vr = reinterpret_cast<const uint4 *>(a.v_base + at + r * kRowBytes);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint4 v4 = vr[c];
          const uint32_t vw[4] = {v4.x, v4.y, v4.z, v4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float &o0 = o[c / 2][8 * (c % 2) + 2 * i], &o1 = o[c / 2][8 * (c % 2) + 2 * i + 1];
            o0 = fmaf(p, bf16_lo(vw[i]), o0);
            o1 = fmaf(p, bf16_hi(vw[i]), o1);
          }
        }
      }
    }
  }
  const float inv = nan ? NAN : l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int part = 0; part < 4; ++part) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const float4 x = add(4 * part + c, *sum(4 * part + c));
      o[part][4 * c] = x.x * inv;
      o[part][4 * c + 1] = x.y * inv;
      o[part][4 * c + 2] = x.z * inv;
      o[part][4 * c + 3] = x.w * inv;
    }
    store_row<kBf16Out>(a.out, row + 16 * part, o[part]);
  }
}

// Every role walks the same table of this CTA's items and skips the same items and blocks, so that their running counters
// agree.  kPair: an item is one tile's tokens against two K/V heads, a tile each; blocks alternate between them.
template <bool kBf16Out, bool kPair>
__global__ void __launch_bounds__(kWpThreads, 1) window_prefill_kernel(const __grid_constant__ WindowArgs a) {
  extern __shared__ uint8_t smem_raw[];
  WpSmem<kBf16Out> &sm = *reinterpret_cast<WpSmem<kBf16Out> *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // (the same for all lanes, and the compiler knows it)
  // Item k of this CTA: k * G + c on even rounds and k * G + (G - 1 - c) on odd ones.
  const int G = int(gridDim.x), c = int(blockIdx.x);
  auto item_index = [&](int k) { return k * G + ((k & 1) ? G - 1 - c : c); };
  int nt = 0;  // <= kWpMaxItems
  while (nt < kWpMaxItems<kBf16Out> && item_index(nt) < a.most_items) ++nt;

  if (tid < kWpMaxItems<kBf16Out>) sm.items[tid].run = sm.items[tid].invalid = 0;
  if (tid == 0) {
    for (unsigned i = 0; i < kWpStages; ++i) {
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.kv_empty[i], kPair ? 1 : kWpTiles);
    }
    for (int t = 0; t < kWpTiles; ++t) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&sm.s_full[t][h], 2);
        mbar_init(&sm.p_full[t][h], kWpRows / 32);
      }
      mbar_init(&sm.mma_done[t], 1);
      mbar_init(&sm.o_full[t], 1);
      mbar_init(&sm.q_full[t], kBf16Out ? kWpRows / 32 : 1);
    }
    sm.abort = 0;
    mbar_init_fence();
  }
  if (warp == kWpLoader) tmem_alloc(&sm.tmem_base, kWpTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  // The list of items: sequence after sequence, its tokens from the last ones to the first, 8 K/V heads each.  A thread
  // takes a sequence, counts its items and, by a prefix sum, finds which of this CTA's items they are.
  bool negative = false;  // a sequence of less than no query tokens, reported once the kernel before this one has ended
  for (int base = 0, before = 0; base < a.num_seqs; base += kWpThreads) {
    const int s = base + tid;
    int q0 = 0, n = 0, ctx = 0;
    if (s < a.num_seqs) {
      q0 = __ldg(a.query_start + s);
      n = __ldg(a.query_start + s + 1) - q0;
      ctx = __ldg(a.context_lens + s);
    }
    negative |= n < 0;
    const int count = n <= 0 ? 0 : min((n - 1) / a.item_tok + 1, a.items_per_seq);
    int upto = count;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) sm.warp_sum[warp] = upto;
    __syncthreads();
    int all = 0, first = before + upto - count;
    for (int w = 0; w < kWpThreads / 32; ++w) {
      if (w < warp) first += sm.warp_sum[w];
      all += sm.warp_sum[w];
    }
    if (count > 0)
      for (int k = 0; k < nt; ++k) {
        constexpr int kHeads = kPair ? kKvHeads / 2 : kKvHeads;
        const int i = item_index(k), u = i / kHeads - first;
        if (u >= 0 && u < count)
          sm.items[k] = wp_item(a, s, i % kHeads * (kKvHeads / kHeads), (count - 1 - u) * a.item_tok, q0, n, ctx);
      }
    before += all;
    __syncthreads();
  }
  negative = __syncthreads_or(negative);
  constexpr int kShift = kPair ? 1 : 0;  // blocks of an item: nblocks << kShift
  uint64_t redo = 0;  // softmax threads: bit k set where this thread's row of item k has to be computed again
  // index of the first running item at or after k
  auto next_run = [&](int k) {
    while (k < nt && !sm.items[k].run) ++k;
    return k;
  };

  if (warp == kWpLoader) {
    // ================= loader: K/V blocks (tiled TMA) =================
    const uint64_t policy = policy_evict_last();
    if (lane == 0) {
      prefetch_tensormap(&a.tmap_k);
      prefetch_tensormap(&a.tmap_v);
    }
    // block-table entries of an item's first 128 pages: page lp sits in lane lp % 32, slot lp / 32
    auto load_entries = [&](const WpItem &t, int (&e)[4]) {
      const int32_t *table = a.block_tables + (long long)t.s * a.bt_stride;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int lp = lane + 32 * k;
        e[k] = lp < t.npages ? __ldg(table + logical_page(t, lp)) : -1;
      }
    };
    unsigned gb = 0;   // K/V blocks issued so far
    bool ok = true;
    int k = next_run(0);
    int ent[4] = {-1, -1, -1, -1};
    if (k < nt) {
      load_entries(sm.items[k], ent);
    }
    // launched with overlap (PKV_OVERLAP_PREVIOUS), the kernel before this one (the append of the prompt's K/V) may still
    // be running: the pages are read only once it has completed
    griddep_wait();
    while (ok && k < nt) {
      const WpItem t = sm.items[k];
      const int kn = next_run(k + 1);
      int ent_next[4] = {-1, -1, -1, -1};
      if (kn < nt) load_entries(sm.items[kn], ent_next);  // in flight while this item's blocks go out
      const int32_t *table = a.block_tables + (long long)t.s * a.bt_stride;
      for (int b = 0; b < t.nblocks << kShift; ++b, ++gb) {
        const int j = b >> kShift, head = kPair ? t.g + (b & 1) : t.g;
        const unsigned st = gb % kWpStages;
        if (gb >= kWpStages) {
          if (!wp_wait(sm, &sm.kv_empty[st], (gb / kWpStages - 1) & 1, a.status)) {
            ok = false;
            break;
          }
        }
        int page[kWpPagesPerBlock], bad = 0;
        const bool near = j * kWpPagesPerBlock < 128;  // the block's entries lie in one of the registers
        const int q4 = j * kWpPagesPerBlock >> 5, some = q4 == 0 ? ent[0] : q4 == 1 ? ent[1] : q4 == 2 ? ent[2] : ent[3];
#pragma unroll
        for (int pp = 0; pp < kWpPagesPerBlock; ++pp) {
          const int lp = j * kWpPagesPerBlock + pp;
          const int e = near            ? __shfl_sync(0xffffffffu, some, lp & 31)
                        : lp < t.npages ? __ldg(table + logical_page(t, lp))
                                        : -1;
          const bool ok_id = unsigned(e) < unsigned(a.num_pages);
          page[pp] = ok_id ? e : -1;  // outside the pool: TMA fills the box with zeros
          if (!ok_id && lp < t.npages) bad |= 1 << pp;
        }
        if (elect_one()) {
          if (bad) report(a.status, PKV_DEV_BAD_PAGE);
          sm.kv_bad[st] = bad;
          mbar_arrive_expect_tx(&sm.kv_full[st], 2 * kWpTileBytes);
#pragma unroll
          for (int pp = 0; pp < kWpPagesPerBlock; ++pp)
            tma_load_3d(sm.k[st] + pp * kWpBox, &a.tmap_k, 0, head * kPageTokens, page[pp], &sm.kv_full[st], policy);
#pragma unroll
          for (int pp = 0; pp < kWpPagesPerBlock; ++pp)
            tma_load_3d(sm.v[st] + pp * kWpBox, &a.tmap_v, 0, head * kPageTokens, page[pp], &sm.kv_full[st], policy);
        }
        __syncwarp();
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) ent[q] = ent_next[q];
      k = kn;
    }
    // every copy issued has landed before the CTA exits
    if (lane == 0) {
      for (unsigned j = gb > kWpStages ? gb - kWpStages : 0; j < gb; ++j)
        mbar_wait(&sm.kv_full[j % kWpStages], (j / kWpStages) & 1);
    }
    __syncwarp();
  } else if (warp >= kWpIssuers) {
    // ================= issuers: the MMAs of a tile each (one thread issues, the warp waits) =================
    griddep_wait();  // (nothing to do before the loader; their waits are not to run out on the kernel before)
    const int tile = warp - kWpIssuers, part = kPair ? 0 : tile;  // the tile's share of the item's tokens
    const uint32_t sa = tmem + kColS + tile * kWpKeys, oa = tmem + kColO + tile * kHeadDim,
                   qa = tmem + kColQ + tile * (kHeadDim / 2), la = tmem + kColLow + tile * (kWpKeys / 2);
    const uint64_t q_desc = sw128_desc(smem_addr(sm.q) + tile * (kWpRows * kRowBytes), 16, 1024);  // (fp32 output)
    const uint64_t k_desc = sw128_desc(smem_addr(sm.k), 16, 1024), v_desc = sw128_desc(smem_addr(sm.v), 16, 1024);
    unsigned passed = 0;            // blocks given back (each tile gives back every one of them)
    unsigned qs = 0, pvs = 0;       // Q's and blocks of P taken up
    bool ok = true;
    auto pass_to = [&](unsigned block) {  // the tile uses none of the blocks before `block` that it has not given back
      while (!kPair && passed < block) {
        if (!wp_wait(sm, &sm.kv_full[passed % kWpStages], (passed / kWpStages) & 1, a.status)) return false;
        if (elect_one()) mbar_arrive(&sm.kv_empty[passed % kWpStages]);
        __syncwarp();
        ++passed;
      }
      return true;
    };
    // The blocks that the tile uses: number j of item k, which has `base` blocks before it.
    struct Cursor {
      int k, j;
      unsigned base;
      WpTile w;
    };
    auto first_block = [&](Cursor &c) {  // of the tile's first item at or behind c.k; false: there is none
      for (c.k = next_run(c.k); c.k < nt; c.k = next_run(c.k + 1)) {
        c.w = tile_of(a, sm.items[c.k], part);
        c.j = c.w.begin();
        if (c.w.last >= 0) return true;
        c.base += sm.items[c.k].nblocks << kShift;
      }
      return false;
    };
    auto block_of = [&](const Cursor &c) { return c.base + unsigned(kPair ? 2 * c.j + tile : c.j); };
    auto ready = [&](const Cursor &c, bool fresh) {  // the block has landed, and Q where it is an item's first
      const WpItem &t = sm.items[c.k];
      const int j = c.j;
      const unsigned block = block_of(c), st = block % kWpStages;
      if (!wp_wait(sm, &sm.kv_full[st], (block / kWpStages) & 1, a.status)) return false;
      if (j == t.nblocks - 1) {
        // V rows at or past the context in the sequence's last page (stale pool bytes) become zeros
        const int row0 = (t.npages - 1 - j * kWpPagesPerBlock) * kPageTokens;  // the item's last page in the block
        const int live = t.ctx - logical_page(t, t.npages - 1) * kPageTokens;
        if (live < kPageTokens) {
          uint8_t *vt = sm.v[st] + (row0 + live) * kRowBytes;
          for (int idx = lane; idx < (kPageTokens - live) * 8; idx += 32)
            *reinterpret_cast<uint4 *>(vt + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        __syncwarp();
      }
      if (fresh && !wp_wait(sm, &sm.q_full[tile], qs++ & 1, a.status)) return false;
      tc_fence_after();
      return true;
    };
    auto issue_s = [&](unsigned st, int h) {  // S of a half of the block in stage st
      if (elect_one()) {
        const uint64_t kd = k_desc + uint32_t((st * kWpTileBytes + h * (kWpTileBytes / 2)) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if constexpr (kBf16Out)
            tc_mma_tmem_a(sa + h * kWpHalf, qa + kk * 8, kd + kk * (32 >> 4), kIdescS, kk > 0 ? 1u : 0u);
          else
            tc_mma(sa + h * kWpHalf, q_desc + kk * (32 >> 4), kd + kk * (32 >> 4), kIdescS, kk > 0 ? 1u : 0u);
        }
        tc_commit(&sm.s_full[tile][h]);
        mbar_arrive(&sm.s_full[tile][h]);  // (hands on the loader's word about bad pages)
      }
      __syncwarp();
    };
    // P V of a half of the block in stage st; the block starts, or ends, a sum in O
    auto issue_pv = [&](unsigned st, int h, bool starts, bool ends) {
      if (!wp_wait(sm, &sm.p_full[tile][h], pvs & 1, a.status)) return false;
      tc_fence_after();
      if (elect_one()) {
        // P: 16 columns for each 32 keys, the second terms of the same keys behind the first ones, third terms in columns of
        // their own; the small ones first
        const uint64_t vd = v_desc + uint32_t((st * kWpTileBytes + h * (kWpTileBytes / 2)) >> 4);
        const uint32_t fresh = starts && h == 0 ? 0u : 1u;
        if constexpr (!kBf16Out) {
#pragma unroll
          for (int kk = 0; kk < kWpHalf / 16; ++kk)
            tc_mma_tmem_a(oa, la + h * (kWpHalf / 2) + kk * 8, vd + kk * (2048 >> 4), kIdescPV, kk == 0 ? fresh : 1u);
#pragma unroll
          for (int kk = 0; kk < kWpHalf / 16; ++kk)
            tc_mma_tmem_a(oa, sa + h * kWpHalf + (kk / 2) * 32 + (kk % 2) * 8 + 16, vd + kk * (2048 >> 4), kIdescPV, 1u);
        }
#pragma unroll
        for (int kk = 0; kk < kWpHalf / 16; ++kk)
          tc_mma_tmem_a(oa, sa + h * kWpHalf + (kk / 2) * 32 + (kk % 2) * 8, vd + kk * (2048 >> 4), kIdescPV,
                        kBf16Out && kk == 0 ? fresh : 1u);
        if (h == 1) {
          if (ends) tc_commit(&sm.o_full[tile]);
          tc_commit(&sm.kv_empty[st]);
        }
      }
      __syncwarp();
      return true;
    };
    Cursor c = {0, 0, 0u, {0, 0, -1}};
    bool more = first_block(c);
    if (more) {
      ok = pass_to(block_of(c)) && ready(c, true);
      if (ok) {
        issue_s(block_of(c) % kWpStages, 0);
        issue_s(block_of(c) % kWpStages, 1);
      }
    }
    int used = 0;
#pragma unroll 1
    while (ok && more) {
      const bool last = c.j == c.w.last, starts = used % kWpRun<kBf16Out> == 0;
      const bool ends = last || used % kWpRun<kBf16Out> == kWpRun<kBf16Out> - 1;
      Cursor n = c;
      if (last) {
        n.base += sm.items[c.k].nblocks << kShift;
        ++n.k;
        more = first_block(n);
      } else {
        n.j = c.w.next(c.j);
      }
      const unsigned block = block_of(c), follows = block_of(n), st = block % kWpStages, sn = follows % kWpStages;
      // The next block's S goes half by half behind P V of this one's, from one item to the next as well.  Where blocks lie
      // between that the tile does not use, this one is given back first (their copies may wait for its stage).
      // (A pair's tile uses every second block, all of those, and the other ones are not its to give back.)
      const bool near = more && (kPair || follows == block + 1);
      ok = issue_pv(st, 0, starts, ends);
      if (near) {
        ok = ok && ready(n, last);
        if (ok) issue_s(sn, 0);
      }
      ok = ok && issue_pv(st, 1, starts, ends);
      ++pvs;
      ++passed;
      if (ok && more) {
        if (!near) {
          ok = pass_to(follows) && ready(n, last);
          if (ok) issue_s(sn, 0);
        }
        if (ok) issue_s(sn, 1);
      }
      used = last ? 0 : used + 1;
      c = n;
    }
    if (ok) ok = pass_to(c.base);
    // every MMA issued has completed before the tensor memory is freed
    if (elect_one()) {
      tc_commit(&sm.mma_done[tile]);
      mbar_wait(&sm.mma_done[tile], 0);
    }
    __syncwarp();
  } else {
    // ================= softmax groups: thread = row = 4 * token + head of tile `tile` =================
    const int tile = warp >> 2, share = kPair ? 0 : tile;  // ... and its share of the item's tokens
    const int r = tid & (kWpRows - 1), tok = share * kWpTok + (r >> 2), hh = r & 3;
    auto head_of = [&](const WpItem &t) { return kPair ? t.g + tile : t.g; };
    const uint32_t lane_base = tmem + (uint32_t(32 * (warp & 3)) << 16);
    const uint32_t s_addr = lane_base + kColS + tile * kWpKeys, o_addr = lane_base + kColO + tile * kHeadDim,
                   low_addr = lane_base + kColLow + tile * (kWpKeys / 2);
    // Q of the tile's next item, once the last S of the one before is there, so that the next item's first S is computed while
    // this one's last P is (16 x 512 fp32 41.3 us for 42.8, 200 queries 10.6 for 11.1; 4 x 2048, of longer items, 141 for
    // 140).  With bf16 output every row's own thread fetches it an item ahead and puts it into tensor memory; with fp32
    // output, where the weights' third terms take those columns, it goes to shared memory by TMA.
    uint32_t qn[kBf16Out ? kHeadDim / 2 : 1];
    int q_item = -1;  // the tile's next item
    uint32_t q_sent = 0;  // boxes that this thread has asked for
    auto next_q = [&]() {
      do q_item = next_run(q_item + 1);
      while (q_item < nt && (share * kWpTok >= a.item_tok || sm.items[q_item].t0 + share * kWpTok >= sm.items[q_item].n));
    };
    auto fetch_q = [&]() {
      next_q();
      if constexpr (kBf16Out) {
        if (q_item >= nt) return;
        const WpItem &t = sm.items[q_item];
        const bool there = t.t0 + tok < t.n;
        const long long row = (long long)(t.q0 + t.t0 + tok) * kQHeads + head_of(t) * kGroup + hh;
        const uint4 *src = reinterpret_cast<const uint4 *>(a.q + row * kHeadDim);
#pragma unroll
        for (int i = 0; i < kHeadDim / 8; ++i) {
          const uint4 x = there ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
          qn[4 * i] = x.x, qn[4 * i + 1] = x.y, qn[4 * i + 2] = x.z, qn[4 * i + 3] = x.w;
        }
      }
    };
    auto hand_on_q = [&]() {  // the next item's Q
      if (q_item >= nt) return;
      if constexpr (kBf16Out) {
        tmem_st32(lane_base + kColQ + tile * (kHeadDim / 2), qn);
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(&sm.q_full[tile]);
      } else if ((warp & 3) == 0) {
        const WpItem &t = sm.items[q_item];
        if (elect_one()) {
          // (rows past the sequence's are the next one's, zeros, or what was there: computed, never written)
          const int first_tok = t.t0 + share * kWpTok, boxes = min(kWpTok / 8, (t.n - first_tok + 7) / 8);
          mbar_arrive_expect_tx(&sm.q_full[tile], boxes * (8 * kGroup * kRowBytes));
          for (int i = 0; i < boxes; ++i)
            tma_load_3d(sm.q[tile] + i * (8 * kGroup * kRowBytes), &a.tmap_q, 0, head_of(t) * kGroup, t.q0 + first_tok + 8 * i,
                        &sm.q_full[tile], policy_evict_first());
          ++q_sent;
        }
        __syncwarp();
      }
      fetch_q();
    };
    fetch_q();
    hand_on_q();
    griddep_wait();  // the first global write below comes after the kernel before this one
    // (not before the wait: what the next kernel reads at once may come from a kernel before this one)
    griddep_launch_dependents();
    if (negative && blockIdx.x == 0 && tid == 0) report(a.status, PKV_DEV_BAD_CONTEXT);
    const float scale = a.scale_log2;
    unsigned gb = 0;
    uint32_t blocks = 0, drained = 0;  // blocks of this tile so far, and times that O was taken out
    bool ok = true;
    // O to be taken out once the next P is written: 0 none, 1 a run's, 2 the item's
    int drain = 0, d_k = 0;
    float d_sum = 0.f;
    bool d_more = false;  // the sum of earlier runs lies in the warp's rows
    uint8_t *mine = sm.rows[warp][0] + lane * 128;
    auto mine_at = [&](int part, int i) {  // fp32 values part + 4 i .. + 3 of the row
      return reinterpret_cast<float4 *>(mine + (part / 32) * 4096 + (((part % 32 / 4 + i) ^ (lane & 7)) << 4));
    };
    auto o_ready = [&]() {
      if (!wp_wait(sm, &sm.o_full[tile], drained & 1, a.status)) return false;
      ++drained;
      tc_fence_after();
      return true;
    };
    auto rows_free = [&]() {  // the rows that were stored last have been read
      if (elect_one()) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
      __syncwarp();
    };
    auto values = [&](int part, float (&v)[16]) {  // of O, and of the runs before
      uint32_t o[16];
      tmem_ld16_async(o_addr + part, o);
      tmem_ld_wait(o);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(o[i]);
      if (d_more) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float4 x = *mine_at(part, i);
          v[4 * i] += x.x, v[4 * i + 1] += x.y, v[4 * i + 2] += x.z, v[4 * i + 3] += x.w;
        }
      }
    };
    auto take_run = [&]() {
      if (!o_ready()) return false;
      if (!d_more) rows_free();
#pragma unroll 1
      for (int part = 0; part < kHeadDim; part += 16) {
        float v[16];
        values(part, v);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *mine_at(part, i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
      }
      drain = 0;
      return true;
    };
    auto take_item = [&]() {
      if (!o_ready()) return false;
      const WpItem &t = sm.items[d_k];
      const bool d_row = t.t0 + tok < t.n;  // the row has a query
      const long long d_at = ((long long)(t.q0 + t.t0 + tok) * kQHeads + head_of(t) * kGroup + hh) * kHeadDim;
      float finite = 0.f;  // stays 0 where every value of the row is finite
      const float inv = d_sum != 0.f ? 1.f / d_sum : 0.f;
      // the warp's 8 tokens by TMA, where they are the sequence's own
      const int first_tok = t.t0 + share * kWpTok + 8 * (warp & 3);
      const bool boxed = first_tok + 8 <= t.n;
      if (boxed) rows_free();
#pragma unroll 1
      for (int part = 0; part < kHeadDim; part += 16) {
        float v[16];
        values(part, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          v[i] *= inv;
          finite = fmaf(v[i], 0.f, finite);
        }
        if (boxed) {
          if constexpr (kBf16Out) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              *reinterpret_cast<uint4 *>(mine + (((part / 8 + i) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16x2(v[8 * i], v[8 * i + 1]), pack_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                             pack_bf16x2(v[8 * i + 4], v[8 * i + 5]), pack_bf16x2(v[8 * i + 6], v[8 * i + 7]));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *mine_at(part, i) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        } else if (d_row) {
          store_row<kBf16Out>(a.out, d_at + part, v);
        }
      }
      if (boxed) {
        fence_proxy_async_smem();
        __syncwarp();
        if (elect_one()) {
          tma_store_3d(&a.tmap_o, 0, head_of(t) * kGroup, t.q0 + first_tok, sm.rows[warp][0]);
          if (!kBf16Out) tma_store_3d(&a.tmap_o, 32, head_of(t) * kGroup, t.q0 + first_tok, sm.rows[warp][1]);
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        __syncwarp();
      }
      if (d_row && !(finite == 0.f && d_sum >= kSumMin && d_sum <= kSumMax)) redo |= 1ull << d_k;
      drain = 0;
      return true;
    };
    auto written = [&](int h) {  // P of a half is there
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (elect_one()) mbar_arrive(&sm.p_full[tile][h]);
    };
    for (int k = 0; ok && k < nt; ++k) {
      const WpItem &t = sm.items[k];
      if (t.invalid) {
        // invalid sequence: zero this item's rows (its tokens, the query heads of its K/V heads)
        if (t.t0 == 0 && t.g == 0 && tid == 0) report(a.status, PKV_DEV_BAD_CONTEXT);
        // (the last item of more query tokens than max_query takes all that are left, as far as there are rows)
        const long long left = t.n - t.t0, at0 = (long long)t.q0 + t.t0;
        const long long toks = t.t0 + a.item_tok >= a.max_query ? left : min((long long)a.item_tok, left);
        const long long row0 = max(at0, 0ll), row1 = min(at0 + toks, (long long)a.num_q_rows);
        constexpr int kWidth = (kGroup * kHeadDim) << kShift;
        for (long long i = tid; i < (row1 - row0) * kWidth; i += kWpTiles * kWpRows) {
          const long long at = ((row0 + i / kWidth) * kQHeads + t.g * kGroup) * kHeadDim + i % kWidth;
          if (kBf16Out)
            static_cast<uint16_t *>(a.out)[at] = 0;
          else
            static_cast<float *>(a.out)[at] = 0.f;
        }
        continue;
      }
      if (!t.run) continue;
      const WpTile w = tile_of(a, t, share);
      if (w.last < 0) {
        gb += t.nblocks << kShift;
        continue;
      }
      const int pos = t.ctx - t.n + min(t.t0 + tok, t.n - 1);
      const int lo = max(0, pos - a.window + 1);
      const int skip = t.skip, nblocks = t.nblocks << kShift;
      // blocks inner0 .. inner1 - 1 hold only keys that every row of the warp sees: from the last row's window on, up to the
      // first row's position
      const int pos0 = __shfl_sync(0xffffffffu, pos, 0), lo31 = __shfl_sync(0xffffffffu, lo, 31);
      const int inner0 = ((lo31 + kPageTokens - 1) / kPageTokens - skip + kWpPagesPerBlock - 1) / kWpPagesPerBlock;
      const int inner1 = min(((pos0 + 1) / kPageTokens - skip) / kWpPagesPerBlock, w.last);
      float m = 0.f;                     // the exponents' reference, times log2(e) scale
      float sum = 0.f, run_sum = 0.f;    // of the finished runs, and of this one
      int used = 0;
      bool more = false;
      uint32_t x0[32], x1[32];  // quarters of S
      bool loaded = false;      // the next block's first one has been asked for
      auto arrived = [&]() {  // the block's first half, where it has not been asked for
        if (!loaded) {
          if (!wp_wait(sm, &sm.s_full[tile][0], blocks & 1, a.status)) return false;
          tc_fence_after();
        }
        return true;
      };
      auto end_block = [&]() {
        ++blocks;
        if (++used % kWpSumRun == 0) {
          sum += run_sum;  // row sums in two levels: equal weights round the same way at every addition
          run_sum = 0.f;
        }
        if (used % kWpRun<kBf16Out> == 0) {
          drain = 1;
          d_more = more;
          d_k = k;
          more = true;
        }
      };
      // The reference: the largest score of the first of the first block's first four pages of which every key is seen by some
      // row of the item and lies at or before the tile's last position (any finite value near the scores will do); where there
      // is no such page, of such keys of the first page, which has one.  Keys that nobody sees count for nothing: they may be
      // rows of the pool behind the context, of any value.  (The scores of an invalid page are 0.)
      {
        const int key = w.begin() * kWpKeys, p0 = t.ctx - t.n + t.t0, first = max(0, p0 - a.window + 1);
        const int p1 = t.ctx - t.n + min(t.t0 + (share + 1) * kWpTok, t.n) - 1;
        const uint32_t seen0 = seen_keys(key, skip, first, p1, a.sinks, 0), seen1 = seen_keys(key + 32, skip, first, p1, a.sinks, 0);
        const int page = (seen0 & 0xffffu) == 0xffffu   ? 0
                         : seen0 >> 16 == 0xffffu       ? 1
                         : (seen1 & 0xffffu) == 0xffffu ? 2
                         : seen1 >> 16 == 0xffffu       ? 3
                                                        : 0;
        const uint32_t keys = page == 0 ? seen0 : 0xffffu;
        ok = arrived();
        if (!ok) break;
        const float none = scale < 0.f ? INFINITY : -INFINITY;
        uint32_t y[16];
        tmem_ld16_async(s_addr + page * kPageTokens, y);
        tmem_ld_wait(y);
#pragma unroll
        for (int i = 0; i < kPageTokens; ++i) y[i] = keys >> i & 1u ? y[i] : __float_as_uint(none);
        m = (scale < 0.f ? extreme16<true>(y) : extreme16<false>(y)) * scale;
        if (!(fabsf(m) < INFINITY)) m = 0.f;
      }
#pragma unroll 1
      for (int j = w.begin();;) {
        ok = arrived();
        if (!ok) break;
        const int bad = sm.kv_bad[(gb + (kPair ? 2 * j + tile : j)) % kWpStages];
        // P overwrites the columns of the S that it comes from.  Keys outside the row's window and sinks, and the keys of
        // invalid pages (loaded as zeros), get weight 0.
        if (bad == 0 && j >= inner0 && j < inner1 && drain != 2) {
          bool plain = true;
#pragma unroll 1
          while (true) {
            // every quarter is on its way while the one before it is worked on
            if (!loaded) tmem_ld32_async(s_addr, x0);
            tmem_ld_wait(x0);
            tmem_ld32_async(s_addr + 32, x1);
            run_sum += quarter_probs<false, kBf16Out>(x0, ~0u, m, scale, s_addr, low_addr);
            tmem_ld_wait(x1);
            ok = wp_wait(sm, &sm.s_full[tile][1], blocks & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            tmem_ld32_async(s_addr + 64, x0);
            run_sum += quarter_probs<false, kBf16Out>(x1, ~0u, m, scale, s_addr + 32, low_addr + 16);
            if (drain != 0) {  // O of the run before, before the issuer starts it anew
              tmem_st_wait();
              ok = take_run();
              if (!ok) break;
            }
            written(0);
            tmem_ld_wait(x0);
            tmem_ld32_async(s_addr + 96, x1);
            run_sum += quarter_probs<false, kBf16Out>(x0, ~0u, m, scale, s_addr + 64, low_addr + 32);
            tmem_ld_wait(x1);
            loaded = j + 1 < inner1 &&
                     __all_sync(0xffffffffu, mbar_try_wait(&sm.s_full[tile][0], (blocks + 1) & 1));
            if (loaded) {
              tc_fence_after();
              tmem_ld32_async(s_addr, x0);
            }
            run_sum += quarter_probs<false, kBf16Out>(x1, ~0u, m, scale, s_addr + 96, low_addr + 48);
            written(1);
            if (j + 1 >= inner1) break;
            end_block();
            ++j;
            ok = arrived();
            if (!ok) break;
            plain = sm.kv_bad[(gb + (kPair ? 2 * j + tile : j)) % kWpStages] == 0;
            if (!plain) break;
          }
          if (!ok) break;
          if (!plain) continue;  // with a mask
        } else {
          if (loaded) tmem_ld_wait(x0);  // (asked for before the block's bad pages were known)
          loaded = false;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            if (h == 1) {
              if (!wp_wait(sm, &sm.s_full[tile][1], blocks & 1, a.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (j == w.last) hand_on_q();
            }
#pragma unroll 1
            for (int part = 0; part < 2; ++part) {
              const uint32_t valid = seen_keys(j * kWpKeys + h * kWpHalf + 32 * part, skip, lo, pos, a.sinks,
                                               bad >> (4 * h + 2 * part));
              const uint32_t to = s_addr + h * kWpHalf + 32 * part, low = low_addr + h * (kWpHalf / 2) + 16 * part;
              if (__any_sync(0xffffffffu, valid != 0u)) {
                tmem_ld32(to, x0);
                if (__all_sync(0xffffffffu, valid == ~0u))
                  run_sum += quarter_probs<false, kBf16Out>(x0, ~0u, m, scale, to, low);
                else
                  run_sum += quarter_probs<true, kBf16Out>(x0, valid, m, scale, to, low);
              } else {  // keys that none of the warp's rows sees
                no_probs<kBf16Out>(to, low);
              }
            }
            if (h == 0 && drain != 0) {
              tmem_st_wait();
              ok = drain == 1 ? take_run() : take_item();
              if (!ok) break;
            }
            written(h);
          }
        }
        if (!ok) break;
        end_block();
        if (j == w.last) break;
        j = w.next(j);
      }
      if (!ok) break;
      gb += nblocks;
      // the item's last block: what is taken out last is divided
      d_more = drain == 1 ? d_more : more;
      drain = 2;
      d_k = k;
      d_sum = sum + run_sum;
    }
    if (ok && drain != 0) take_item();
    if (q_sent > 0) mbar_wait(&sm.q_full[tile], (q_sent - 1) & 1);  // no copy is on its way
    __syncwarp();
    if (elect_one()) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // every row has been written
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWpLoader) {
    tc_fence_after();
    tmem_dealloc(tmem, kWpTmemCols);
  }
  for (int k = 0; redo != 0; ++k, redo >>= 1)
    if (redo & 1) {
      const int tile = tid >> 7;
      recompute_row<kBf16Out>(a, sm.items[k], sm.items[k].g + (kPair ? tile : 0),
                              (kPair ? 0 : tile * kWpTok) + ((tid & 127) >> 2), tid & 3, sm.rows[warp][0] + lane * 128);
    }
}

using WindowKernel = void (*)(WindowArgs);
constexpr WindowKernel kWindowKernels[] = {window_prefill_kernel<false, false>, window_prefill_kernel<true, false>,
                                           window_prefill_kernel<false, true>, window_prefill_kernel<true, true>};

// Shared-memory limits of the kernels on the current device.
int setup_window_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (!done[dev]) {
    for (int i = 0; i < 4; ++i)
      if (cudaFuncSetAttribute(kWindowKernels[i], cudaFuncAttributeMaxDynamicSharedMemorySize,
                               int(i & 1 ? kWpSmemBytes<true> : kWpSmemBytes<false>)) != cudaSuccess) {
        cudaGetLastError();
        return PKV_ERR_CUDA;
      }
    done[dev] = true;
  }
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_paged_window_prefill_attention(const pkv_pool *pool, void *out, const void *q, int num_q_heads,
                                                  int num_q_rows, const int32_t *query_start,
                                                  const int32_t *block_tables, int64_t block_table_stride,
                                                  const int32_t *context_lens, int num_seqs, int max_query,
                                                  int max_context, float scale, int window, int sinks,
                                                  int32_t *device_status, unsigned flags, void *stream) {
  if (flags & ~unsigned(PKV_OVERLAP_PREVIOUS | PKV_OUT_BF16)) return PKV_ERR_SHAPE;
  int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_q_heads != pkv::kQHeads) return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || num_seqs > (1 << 24) || max_query < 0 || max_query > (1 << 20) || max_context < 0 ||
      max_context > pkv::kMaxTokens || block_table_stride < 0 || num_q_rows < 0 || window < 1 || sinks < 0)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || max_query == 0 || num_q_rows == 0) return PKV_OK;
  if (out == nullptr || q == nullptr || query_start == nullptr || block_tables == nullptr || context_lens == nullptr)
    return PKV_ERR_NULL;
  if (!isfinite(scale) || !isfinite(scale * pkv::kLog2e)) return PKV_ERR_SCALE;
  if (!pkv::aligned16(q) || !pkv::aligned16(out) || (reinterpret_cast<uintptr_t>(query_start) & 3u) ||
      (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u))
    return PKV_ERR_ALIGN;
  const int sms = pkv::device_sm_count() > 0 ? pkv::device_sm_count() : 148;
  // Items of one tile while nearly all of them find an SM of their own: 200 queries of one sequence take 11.4 us so and
  // 13.1 in items of two tiles; 16 x 300..512 queries, ten items of one tile to an SM, 58.7 us and 40.9.
  const long long pairs = (max_query + pkv::kWpItemTok - 1) / pkv::kWpItemTok;
  // No more than 32 queries a sequence fill one tile: two heads then share the CTA, 256 x 4 queries, windows of 512, fp32
  // in 99 us (156 with the second tile idle), 64 x 16 in 34 (50), 3000 x 10 of 100 in 368 (617), 40 x 32 of 200 in 18.1
  // (20.1); bf16 74.6 (92.4), 26.7 (32.1), 296 (492), 14.7 (15.3).  While every (sequence, head) finds an SM of its own it
  // has that one.
  const bool pair = max_query <= pkv::kWpTok && (long long)num_seqs * pkv::kKvHeads > sms;
  const int item_tok = pair || (long long)num_seqs * pairs * pkv::kKvHeads * 2 <= sms ? pkv::kWpTok : pkv::kWpItemTok;
  const long long items = (max_query + item_tok - 1) / item_tok;
  if ((long long)num_seqs * items * pkv::kKvHeads > 0x3fffffffLL) return PKV_ERR_SHAPE;
  rc = pkv::setup_window_attributes();
  if (rc != PKV_OK) return rc;
  pkv::WindowArgs a;
  rc = pkv::pool_tensor_maps(pool, pkv::kPageTokens, &a.tmap_k, &a.tmap_v);
  if (rc != PKV_OK) return rc;
  rc = pkv::query_tensor_map(q, num_q_rows, pkv::kQHeads, pkv::kHeadDim, pkv::kGroup, 8, &a.tmap_q);
  if (rc != PKV_OK) return rc;
  rc = pkv::output_tensor_map(out, num_q_rows, pkv::kQHeads, pkv::kHeadDim, (flags & PKV_OUT_BF16) != 0, pkv::kGroup, 8,
                              &a.tmap_o);
  if (rc != PKV_OK) return rc;
  a.num_pages = pool->num_pages;
  a.num_q_rows = num_q_rows;
  a.out = out;
  a.q = static_cast<const uint16_t *>(q);
  a.k_base = static_cast<const uint8_t *>(pool->k_base);
  a.v_base = static_cast<const uint8_t *>(pool->v_base);
  a.page_stride = pool->page_stride_bytes;
  a.window = window;
  a.sinks = sinks;
  a.query_start = query_start;
  a.block_tables = block_tables;
  a.bt_stride = block_table_stride;
  a.context_lens = context_lens;
  a.num_seqs = num_seqs;
  a.max_context = max_context;
  a.max_query = max_query;
  a.item_tok = item_tok;
  a.items_per_seq = int(items);
  a.scale_log2 = scale * pkv::kLog2e;
  a.status = device_status;
  a.most_items = int((long long)num_seqs * items * (pair ? pkv::kKvHeads / 2 : pkv::kKvHeads));
  const bool bf16 = (flags & PKV_OUT_BF16) != 0;
  const int table = bf16 ? pkv::kWpMaxItems<true> : pkv::kWpMaxItems<false>;
  const int by_table = (a.most_items + table - 1) / table;  // items per CTA <= table
  // in whole rounds of the SMs: a few CTAs more than there are SMs would take as long as all of them (40 x 2048 queries,
  // windows of 128, bf16 320 us in 304 CTAs, 573 in 160; fp32 385 in 456, 510 in 320)
  const int g = by_table > sms ? (by_table + sms - 1) / sms * sms : sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(a.most_items < g ? a.most_items : g));
  cfg.blockDim = dim3(pkv::kWpThreads);
  cfg.dynamicSmemBytes = bf16 ? pkv::kWpSmemBytes<true> : pkv::kWpSmemBytes<false>;
  cfg.stream = static_cast<cudaStream_t>(stream);
  // programmatic stream serialization: the set-up (item table, block-table entries, the first item's Q) overlaps the
  // end of the kernel before this one
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & PKV_OVERLAP_PREVIOUS) ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, pkv::kWindowKernels[(pair ? 2 : 0) + (bf16 ? 1 : 0)], a) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_LAUNCH;
  }
  return PKV_OK;
}
