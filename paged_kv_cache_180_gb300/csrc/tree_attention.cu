// Attention of a tree of drafted tokens per sequence over its paged K/V.
//
//   out[i][h] = sum_{t in A_i} softmax_t(scale * q[i][h] . K_t[h/4]) V_t[h/4],
//   A_i = the committed prefix (t < base_s) and the nodes base_s + j whose bit j is set in row i's mask
//
// evaluated in one pass over the keys: with r a reference for the row's exponents, l = sum 2^(c s_t - r) and
// O = sum 2^(c s_t - r) V_t (c = scale log2 e); two disjoint key sets merge by
// R = max(r_a, r_b), L = sum l 2^(r - R), O = sum O 2^(r - R), out = O / L.
//
// GB300 design (tcgen05 tensor cores, accumulators in tensor memory)
//  * Unit: 32 nodes of a sequence against one K/V head g.  Its 128 rows (4 * node + head in group) share
//    every K/V row loaded: M = 128.  Keys in blocks of 64 (4 pages).
//  * Work split, two CTAs per SM.  Whole units to a CTA where that costs less than merges do: the first by the CTA's number,
//    further ones claimed from a counter in the workspace, so that nothing is cut and the CTAs end together.
//    (Over 360 uniform batches of 1 to 110 sequences, 64 to 4096 tokens and 6 to 64 nodes the rule is 1.3 % slower than the
//    better of the two would be for each, whole units for all 3.7 % and shares for all 15.6 %.)
//    Otherwise the key blocks of all units form one list, of which the CTAs take equal
//    shares, whatever the mix of lengths and trees.  A unit cut across CTAs leaves one partial
//    state (r, l, O) per CTA in the workspace, and the CTA that takes the last of its tickets (an
//    atomic counter, nobody waits) merges them.  (A merge takes 1.8 us with 24 rows and 3 to 5 us with 128.)
//  * Warp roles (384 threads): 8 softmax warps, a loader of K and one of V (tiled TMA, head g's 16 rows of
//    each page as 2 KiB boxes, into rings of 4 and 5 blocks: a K block is free once its S is there, a V block waits
//    for the softmax too), one warp that issues S and one that issues the products with V: nobody's waits hold up
//    another's work.  The K loader walks the list and loads Q too (boxes of 8 nodes x 4 heads).
//  * S = Q K^T is 4 tcgen05.mma (M 128, N 64, K 16) into one of three TMEM buffers.  The softmax warps form two
//    groups that take the blocks in turn, a thread to a row; P overwrites its S and is the TMEM A operand
//    of O += P V.  (Two threads to a row on the same block, with S buffers for two blocks, took 1650 cycles a block
//    against 1300.)
//  * What bounds it, by the time a call takes on the device (replayed from a graph; calls one after the other from a
//    program take 1.5 to 3 us more each, and up to 5 % more on some machines): with many keys a node the K/V bytes: 256
//    sequences of 2048 tokens and 8 nodes take 168 to 170 us, 6.4 to 6.5 TB/s, 95 % of a plain copy's rate.  With many
//    short units their starts and ends, each as long as 7 blocks (64 trees of 1..64 nodes over 64..2048 tokens: 51 us, 24
//    for the bytes).  With 64 nodes two tiles share the bytes, and the steps from barrier to barrier count (64 x 2048 in
//    bf16: 73 us, 45 for the bytes): leaving out all of the softmax's arithmetic took 8 % off, the loads 13 more.  The
//    smallest call (600 tokens, 6 nodes) takes 10.7 to 11.1 us: launch 2, lengths 1.5, tables and first K 1.9, ten blocks
//    4.5, the end 0.7.
//  * The reference is the row's largest exponent in the segment's first block and stays: weights are floats, so
//    it only has to keep them in range, and no maximum, rescaling or exchange between the groups is needed after
//    that.  A row whose sum leaves [2^-90, 2^112] is computed again from global memory by redo_row(), slowly (with every
//    row of 64 x 2048 tokens and 32 nodes computed again a call takes 17 ms instead of 0.08).
//  * Weights: with fp32 output P is split into bf16 hi + lo terms (16 significant bits, two products: an error of
//    2.4e-6 of the output, and 2.3e-6 from the truncating accumulator over a run; a third term with two S buffers and
//    runs of 4 blocks would give 0.9e-6 in all and take 30 to 45 % longer); with bf16 output P is one bf16 term, rounded as
//    the output will be (1.6e-3 each; with two terms 64 x 2048 and 64 nodes took 94.7 us for 74.1).  Row sums are taken in
//    fp32 registers from the unrounded weights (a sum inside the MMA would be truncated at every step).
//  * Masks: the score of a key a row may not see is replaced by an infinity, so a NaN score stays out.  V rows at or
//    past the context (stale pool bytes) are zeroed in shared memory, and so are nodes' V rows that hold a
//    NaN or an infinity (0 * NaN in the product would reach every row); the segment's rows are then
//    computed again by redo_row().
//  * Every mbarrier wait is bounded (about 2 s, without the time of rows that are computed again): on expiry the CTA
//    reports PKV_DEV_TIMEOUT, stops issuing work, waits (bounded) for what is in flight, frees its tensor memory and exits.
#include <cuda.h>
#include <cuda_runtime.h>

#include <math.h>
#include <mutex>

#include "host_common.h"
#include "pkv_device.cuh"

namespace pkv {
namespace {

constexpr int kTok = 32;                            // nodes per unit
constexpr int kRows = kTok * kGroup;                // M = 128
constexpr int kOctet = 8;                           // nodes per Q box: one warp's 32 TMEM lanes
constexpr int kKeys = 64;                           // keys per block
constexpr int kPagesPerBlock = kKeys / kPageTokens;
constexpr int kStagesK = 4, kStagesV = 5;           // K and V blocks in shared memory (V waits for the softmax)
constexpr int kScores = 3;                          // S / P buffers in tensor memory
constexpr int kSoftWarps = 8;                       // two groups of four
constexpr int kSoftThreads = kSoftWarps * 32;
constexpr int kLoadWarpK = kSoftWarps, kLoadWarpV = kSoftWarps + 1, kScoreWarp = kSoftWarps + 2,
              kValueWarp = kSoftWarps + 3;
constexpr int kThreads = kSoftThreads + 128;
constexpr int kCtasPerSm = 2;
// Registers per thread: a launch at two CTAs per SM has 80; the four loading and issuing warps give up theirs above
// 40, which raises the softmax warps' to 96: 4 * 32 * 40 + 8 * 32 * 96 < 12 * 32 * 80.
constexpr int kRegsOthers = 40, kRegsSoftmax = 96;
static_assert(kThreads == 384 && 128 * kRegsOthers + kSoftThreads * kRegsSoftmax <= kThreads * 80, "registers of a CTA");
constexpr int kMaxCtas = 320;
// Least list entries a CTA is given: 2, and up to 6 where the longest unit would be in more parts than one merge takes
// (a second level of merges takes as long as 6 blocks).
constexpr int kMinEntries = 2, kMostEntries = 6;
// What the merges of cut units cost a call, in blocks, by the octets of nodes in the longest unit (up to 4): whole units
// are taken when the longest one takes no more than that longer than a CTA's share, and, with more units than CTAs, when
// what the CTAs idle in the last round does not cost more (a block there takes 9/16 of the time, with SMs half empty).
// (6 nodes: 512 tokens 3 % slower to 5 % faster whole, 1024 tokens 15 % slower to 13 % faster, by the number of sequences;
// 32 nodes: 1024 tokens 2 % slower to 29 % faster, 2048 28 % slower to 19 % faster.)
constexpr float kMergeCost = 7.f, kMergeCostOctet = 6.f, kLastRound = 0.5625f;
// A segment's products are added up in runs of this many blocks: every MMA truncates the accumulator.  With fp32 output
// (eight MMAs a block) a row is 1.4e-7 of its size too small for each block of a run, 2.3e-6 for a whole one (where V has
// one sign 3e-7 and 4.8e-6), whatever the number of runs; in one run it was 3e-5 over 14000 keys.  With bf16 output (four)
// one run over 2^24 keys of V of one sign lost 15 %.  So a run's O goes to the segment's part in the workspace, where the
// runs are added with rounding.
template <bool kBf16>
constexpr int kRunBlocks = kBf16 ? 256 : 16;
// Row sums are added up in three levels: over a block's keys, over a run's blocks, over the runs.  Nearly equal weights, whose
// additions all round the same way, then cost at most (16 + a run's blocks / 4 + the runs / 2) 2^-24 of the sum.  (One sum over all
// keys was off by up to 8e-5 at 28000 equal ones; the levels take 0 to 1 % of a call.)
constexpr int kUnitCost = 5;                        // what a unit's start and end weigh in the list, in blocks (4, 6 and 7
                                                    // were 0 to 2 % slower or faster, each on some batches)
constexpr int kBox = kPageTokens * kRowBytes;       // one head's rows of one page: 2 KiB
constexpr int kTileBytes = kKeys * kRowBytes;       // K (or V) of one block: 8 KiB
constexpr int kOctetBytes = kOctet * kGroup * kRowBytes;  // 4 KiB
constexpr uint32_t kTmemCols = 256;
constexpr uint32_t kColO = kScores * kKeys;         // S buffers at columns 0, 64 and 128, O at 192
constexpr int kMergeGroup = 5;                      // a unit in more parts than this merges groups of them first
constexpr float kLog2e = 1.4426950408889634f;
// A row's sum may lie in [2^-90, 2^112] (the scores 77 above the first block's largest) and its O below 2^118: what a
// merge adds up, 320 parts at the most, then stays in the range of fp32.
constexpr float kSumMin = 0x1p-90f, kSumMax = 0x1p112f, kInfOverMaxO = 0x1p10f;

constexpr uint32_t kIdescS = idesc_bf16(kRows, kKeys, false);     // B = K rows (K-major)
constexpr uint32_t kIdescPV = idesc_bf16(kRows, kHeadDim, true);  // B = V rows (MN-major)

// Partial state of one (CTA, unit) pair.
struct Part {
  float4 o[kHeadDim / 4][kRows];  // [4 dims][row]: neighbouring lanes hold neighbouring rows
  float2 rl[2][kRows];            // (reference, sum) of a row, for either half of its dims
  float2 group_rl[2][kRows];      // of the merged state of the group of parts that this one is the first of
  int ticket;                     // of that group; 0 between calls
  int claimed, done, unused;      // in the first part: units claimed, CTAs that are done; 0 between calls
};

struct TreeArgs {
  CUtensorMap tmap_k;  // boxes of one head's 16 rows of one page
  CUtensorMap tmap_v;
  CUtensorMap tmap_q;  // boxes of 8 query rows x one group's 4 heads (rows past num_q_rows read as zeros)
  const uint8_t *k_base, *v_base;
  long long page_stride;
  int num_pages;
  void *out;  // [total][32][64] float32 or bf16
  const uint16_t *q;
  int num_q_rows;
  const int32_t *query_start;
  const uint32_t *mask;
  long long mask_stride;
  const int32_t *block_tables;
  long long bt_stride;
  const int32_t *context_lens;
  int num_seqs, max_query, max_context;
  int max_tiles;      // units a sequence may have per K/V head
  float2 c;           // scale * log2(e), twice
  int *tickets;       // [num_seqs * max_tiles][8 heads], 0 between calls
  Part *parts;        // [2 * kMaxCtas]
  int32_t *status;
};

// A sequence's lengths and what it asks for: tiles of 32 nodes, blocks of 64 keys.  Sequences with no
// nodes, and those whose lengths do not fit, have no blocks.
struct Seq {
  int q0, n, ctx, tiles, nb;
  __device__ void load(const TreeArgs &a, int s) {
    q0 = __ldg(a.query_start + s);
    n = __ldg(a.query_start + s + 1) - q0;
    ctx = __ldg(a.context_lens + s);
    tiles = nb = 0;
    if (n > 0 && valid(a)) {
      tiles = (n + kTok - 1) / kTok;
      nb = (ctx - 1) / kKeys + 1;
    }
  }
  __device__ bool valid(const TreeArgs &a) const {
    return n >= 0 && n <= a.max_query && ctx >= 0 && ctx <= a.max_context && n <= ctx && q0 >= 0 &&
           q0 <= a.num_q_rows - n;
  }
  // Of its tiles the even (part 0) or the odd ones, and the list entries of these.
  __device__ int part_tiles(int part) const { return (tiles + 1 - part) >> 1; }
  __device__ long long entries(int part) const { return (long long)kKvHeads * part_tiles(part) * (nb + kUnitCost); }
};

// A CTA's share of one unit: key blocks j0 .. j1 - 1 of (sequence, K/V head, tile).  A unit has kUnitCost list
// entries of weight, then its blocks.  (Without the weight, CTAs with many short units took twice as long as the
// others in a ragged batch.)  The list holds the units of all even tiles, then those of the odd ones, each
// in the order sequence, head, tile: in a batch of trees of 33 to 64 nodes the CTAs that work on a K/V head's two
// tiles are half the grid apart and there at the same time, so its pages come from memory once.  The loader walks
// the list and passes the segments on in shared memory.
struct Segment {
  int s, g, tile, j0, j1;  // s < 0: there are no more
  int q0, n, ctx, nb;      // the sequence's
  long long unit0;         // list index of the unit's block 0
};
// Places for segments.  The K loader is at most 4 blocks (and so segments) ahead of S, S 3 ahead of the products,
// these one segment ahead of the softmax warps: place k is free when segment k + 16 is written to it.
constexpr int kSegments = 16;
// s_full barriers, and places for the blocks' invalid pages.  The K loader arrives at block n's when S of block n - 4 is
// done, which was issued when the product of block n - 7 was: all softmax warps are past the place's last use, block
// n - 8.  (An even number, so that a group sees every phase of the ones it waits on.)
constexpr int kReady = 8;
static_assert(kReady >= kStagesK + kScores + 1 && kReady % 2 == 0, "places in use");

// Division of non-negative numbers; nearly always they have 32 bits.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if ((a | b) >> 32 == 0) return unsigned(a) / unsigned(b);
  return (long long)((unsigned long long)a / (unsigned long long)b);
}

// Walk over the segments of a CTA's share.  (It keeps little between segments and reads a sequence's lengths
// again for each: the loader has few registers.)
struct Walk {
  long long pos, end, first;  // list position, end of the share, first entry of sequence s in its part
  int s, part;
  // For whole units (unit()): units before sequence s of length class `part`.
  __device__ void start_units() {
    first = 0;
    s = part = 0;
  }
  // Unit u of `all` in the order length class, sequence, head, tile, looked for from sequences s .. s + 31 on, by all lanes of
  // a warp; a CTA's units come in ascending order.  The class of more than half of the longest one's blocks comes
  // first, so that the CTAs end closer together.
  __device__ bool unit(const TreeArgs &a, int u, int all, int longest, int lane, Segment &x) {
#pragma unroll 1
    for (;; s += 32) {
      if (s >= a.num_seqs) {
        s = 0;
        ++part;
      }
      if (u >= all || part == 2) {
        x.s = -1;
        return false;
      }
      Seq seq;
      seq.tiles = 0;
      if (s + lane < a.num_seqs) seq.load(a, s + lane);
      const int mine = (2 * seq.nb > longest ? 0 : 1) == part ? seq.tiles * kKvHeads : 0, before = int(first);
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned there = __ballot_sync(0xffffffffu, u - before < upto);
      if (there) {
        const int l = __ffs(there) - 1;
        const int v = u - before - __shfl_sync(0xffffffffu, upto - mine, l);
        const int tiles = __shfl_sync(0xffffffffu, seq.tiles, l);
        x.s = s + l;
        x.g = v / tiles;
        x.tile = v - x.g * tiles;
        x.q0 = __shfl_sync(0xffffffffu, seq.q0, l);
        x.n = __shfl_sync(0xffffffffu, seq.n, l);
        x.ctx = __shfl_sync(0xffffffffu, seq.ctx, l);
        x.nb = x.j1 = __shfl_sync(0xffffffffu, seq.nb, l);
        x.j0 = 0;
        return true;
      }
      first += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  // From list position `from` on: looks for its sequence, by all lanes of a warp.
  __device__ void start(const TreeArgs &a, long long from, long long to, int lane) {
    pos = from;
    end = to;
    first = 0;
    s = part = 0;
#pragma unroll 1
    for (;;) {
      Seq seq;
      seq.tiles = seq.nb = 0;
      if (s + lane < a.num_seqs) seq.load(a, s + lane);
      const long long mine = seq.entries(part);
      long long upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      const unsigned there = __ballot_sync(0xffffffffu, pos < first + upto);
      if (there) {
        const int l = __ffs(there) - 1;
        first += __shfl_sync(0xffffffffu, upto - mine, l);
        s += l;
        return;
      }
      first += __shfl_sync(0xffffffffu, upto, 31);
      s += 32;
      if (s >= a.num_seqs) {
        s = 0;
        if (++part == 2) {  // (never with lengths that stay as they are)
          part = 1;
          end = pos;
          return;
        }
      }
    }
  }
  __device__ bool next(const TreeArgs &a, Segment &x) {
    Seq seq;
    seq.load(a, s);
    while (pos < end) {
      while (pos - first >= seq.entries(part)) {
        first += seq.entries(part);
        if (++s == a.num_seqs) {
          s = 0;
          if (++part == 2) {  // (never with lengths that stay as they are)
            x.s = -1;
            return false;
          }
        }
        seq.load(a, s);
      }
      const long long len = seq.nb + kUnitCost, u = divide(pos - first, len), v0 = pos - first - u * len;
      const long long v1 = min(len, v0 + (end - pos));
      pos += v1 - v0;
      if (v1 <= kUnitCost) continue;  // nothing but the unit's weight
      const int tiles = seq.part_tiles(part);
      x.s = s;
      x.g = int(u) / tiles;  // (8 heads x at most 2^14 tiles)
      x.tile = 2 * (int(u) - x.g * tiles) + part;
      x.q0 = seq.q0;
      x.n = seq.n;
      x.ctx = seq.ctx;
      x.nb = seq.nb;
      x.unit0 = first + u * len + kUnitCost;
      x.j0 = int(max(v0 - kUnitCost, 0LL));
      x.j1 = int(v1 - kUnitCost);
      return true;
    }
    x.s = -1;
    return false;
  }
};

// T list entries over G CTAs: CTA i has those from i T / G on, rounded down, so that in a batch where every tile of a head
// has a twin CTAs i and i + G / 2 work on the same keys at the same time.  (T < 2^54: at most 2^29 units of 2^25 blocks.)
struct Shares {
  long long T;
  int G;
  __device__ long long first(int cta) const { return divide(cta * T, G); }
  // CTA that has entry p
  __device__ int owner(long long p) const { return int(divide((p + 1) * G - 1, T)); }
};

struct __align__(1024) Smem {
  uint8_t q[2][kRows * kRowBytes];
  uint8_t k[kStagesK][kTileBytes];
  uint8_t v[kStagesV][kTileBytes];
  float ref[4][kRows];       // [turn]: a row's reference, from the group with the segment's first block
  float sums[4][2][kRows];   // [turn][group]: a row's sum, of the runs so far until it is posted
  // barriers of one arrival ...
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kStagesK], v_full[kStagesV];
  uint64_t p_free[kReady];       // [block % 8]: the product of a block is done: its buffer may be written, its V replaced
  uint64_t o_full;               // a run's products are done
  uint64_t ref_full[4][2];       // per quarter of the lanes, by turn: ref is there
  uint64_t seg_full[kSegments];
  uint64_t mma_done[2];
  // ... of two ...
  uint64_t s_full[kReady];       // [block % 8]: S (its K may be replaced), and from the K loader block_bad
  uint64_t sums_full[4];         // per quarter: both sums are there
  // ... of a group's four warps: they have written their P of the buffer ...
  uint64_t p_full[kScores];
  // ... and of all softmax warps: they have read O
  uint64_t o_free;
  Segment seg[kSegments];
  Segment cuts[2];  // a share cuts at most its first and its last unit: tickets taken at the end
  int cut_first[2], cut_parts[2];  // CTA with the unit's first part; parts
  int merge[2];     // this CTA took the last ticket of the cut unit (1) or of its group of parts (2)
  int block_bad[kReady];  // [block % 8] bit pp: page pp of the block is invalid (loaded as zeros)
  int nonfinite[4];  // [segment % 4]: the last segment in which a node's V was zeroed (the softmax warps are
                     // never more than two segments apart: O is written again when all have read it)
  long long warp_entries[kThreads / 32];
  int warp_longest[kThreads / 32], warp_units[kThreads / 32];
  Shares shares;
  int whole, units, longest;  // whether whole units are claimed; units, blocks of the longest one
  uint32_t tmem_base;
  alignas(8) int abort;  // (read together)
  unsigned alive;        // the clock at redo_row()'s last sign of progress
};
constexpr size_t kSmemBytes = sizeof(Smem) + 1024;

__device__ __forceinline__ Smem &shared_memory() {
  extern __shared__ uint8_t smem_raw[];
  return *reinterpret_cast<Smem *>(smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u));
}

// Waits for a phase, at most kWaitCycles (about 2 s); true when it completed.
constexpr unsigned kWaitCycles = 3800000000u;
__device__ __forceinline__ unsigned clock32() {
  unsigned c;
  asm volatile("mov.u32 %0, %%clock;" : "=r"(c));
  return c;
}
__device__ __forceinline__ bool bounded_wait(uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned t0 = clock32();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity))
    if (clock32() - t0 > kWaitCycles) return false;
  return true;
}

// The same for a role's waits: gives up when another role has, and makes the others do so.  While a softmax warp is in
// redo_row(), which ends by itself but may take seconds on a long segment, the limit counts from that one's last sign of
// progress.  (One load for both words: with two the ragged batch took 1 % longer, with a call for expired waits 2 %.)
__device__ __forceinline__ bool wait(Smem &sm, uint64_t *bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const unsigned t0 = clock32();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    int stop;
    unsigned alive;
    asm volatile("ld.volatile.shared.v2.u32 {%0, %1}, [%2];"
                 : "=r"(stop), "=r"(alive)
                 : "r"(smem_addr(&sm.abort))
                 : "memory");
    const unsigned now = clock32();
    if (min(now - t0, now - alive) > kWaitCycles) *reinterpret_cast<volatile int *>(&sm.abort) = stop = 1;
    if (stop) return false;
  }
  return true;
}

// P = 2^(c s - r) of 16 keys as bf16 terms, two keys to a word: hi, and with fp32 output lo.  `sum` takes the
// fp32 weights.
template <bool kBf16>
__device__ __forceinline__ void weights(const uint32_t (&s)[16], float2 c, float2 minus_r, float2 &sum,
                                        uint32_t (&hi)[8], uint32_t (&lo)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 e = fma_f32x2(make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), c, minus_r);
    const float2 p = make_float2(ex2_approx(e.x), ex2_approx(e.y));
    sum = add_f32x2(sum, p);
    hi[i] = pack_bf16x2(p.x, p.y);
    if constexpr (!kBf16) {
      const float2 d = sub_f32x2(p, make_float2(bf16_lo(hi[i]), bf16_hi(hi[i])));
      lo[i] = pack_bf16x2(d.x, d.y);
    }
  }
}

// The weights of a row's 64 keys, from S to P in place: of each 16 keys, hi in the first 8 columns, lo in the others.
// (Loading the next 16 scores ahead changed nothing: other warps fill the time.)
template <bool kBf16>
__device__ __forceinline__ void block_weights(uint32_t taddr, float2 c, float2 minus_r, float2 &total) {
  float2 sum = make_float2(0.f, 0.f);  // of the block alone: few additions to a number of a few blocks' size
#pragma unroll 1
  for (int i = 0; i < 4; ++i, taddr += 16) {
    uint32_t x[16], hi[8], lo[8];
    tmem_ld16_async(taddr, x);
    tmem_ld_wait(x);
    weights<kBf16>(x, c, minus_r, sum, hi, lo);
    tmem_st8_async(taddr, hi);
    if constexpr (!kBf16) tmem_st8_async(taddr + 8, lo);
  }
  total = add_f32x2(total, sum);
  tmem_st_wait();
}

// The scores of keys a row may not see (bit clear in see0, see1: 32 keys each) become the infinity whose weight is 0.
__device__ __forceinline__ void hide_keys(uint32_t taddr, uint32_t see0, uint32_t see1, float c) {
  const uint32_t hidden = c < 0.f ? 0x7f800000u : 0xff800000u;
#pragma unroll 1
  for (int i = 0; i < 4; ++i, taddr += 16) {
    uint32_t s[16];
    tmem_ld16_async(taddr, s);
    tmem_ld_wait(s);
#pragma unroll
    for (int j = 0; j < 16; ++j) s[j] = see0 >> j & 1u ? s[j] : hidden;
    see0 = i == 1 ? see1 : see0 >> 16;
    tmem_st16_async(taddr, s);
  }
  tmem_st_wait();
}

// A row's reference: the largest exponent of a block's keys, 0 if there is none that is finite.
__device__ __forceinline__ float block_reference(uint32_t taddr, float c) {
  float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
  for (int i = 0; i < 4; ++i, taddr += 16) {
    uint32_t s[16];
    tmem_ld16_async(taddr, s);
    tmem_ld_wait(s);
#pragma unroll
    for (int j = 0; j < 16; ++j) top[j & 1] = fmaxf(top[j & 1], __uint_as_float(s[j]) * c);
  }
  const float m = fmaxf(top[0], top[1]);
  return isfinite(m) ? m : 0.f;
}

// The keys of a 32-key window starting at position key0 that a row may see: the prefix, then the nodes
// named by its mask words; nothing at or past the context.
__device__ __forceinline__ uint32_t window_bits(const uint32_t *mask, int key0, int base, int ctx, int n) {
  if (key0 >= ctx) return 0u;
  const int lim = base - key0;  // prefix keys in the window
  if (lim >= 32) return ~0u;
  uint32_t bits;
  const int off = -lim;  // node of the window's first key
  if (off >= 0) {
    const int w = off >> 5;
    const uint32_t lo = __ldg(mask + w), hi = (w + 1) * 32 < n ? __ldg(mask + w + 1) : 0u;
    bits = __funnelshift_r(lo, hi, off & 31);
  } else {
    bits = (__ldg(mask) << lim) | ((1u << lim) - 1u);
  }
  const int left = ctx - key0;
  return left >= 32 ? bits : bits & ((1u << left) - 1u);
}

// Whether a row may see any of the keys pos .. end - 1 (a sum of 0 is right if not).
__device__ __forceinline__ bool sees_any(const uint32_t *mask, int pos, int end, int base, int n) {
  if (pos < base) return true;
#pragma unroll 1
  for (; pos < end; pos += 32)
    if (window_bits(mask, pos, base, end, n)) return true;
  return false;
}

// Bits 15, 31: the low, high bf16 of a word is a NaN or an infinity (its exponent is all ones).
__device__ __forceinline__ uint32_t nonfinite(uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; }
__device__ __forceinline__ uint32_t nonfinite(const uint4 &x) {
  return nonfinite(x.x) | nonfinite(x.y) | nonfinite(x.z) | nonfinite(x.w);
}

// The weight of a state (r, l) merged under the reference R; a state that has seen no key has l = 0.
__device__ __forceinline__ float state_weight(float2 rl, float R) { return rl.y == 0.f ? 0.f : ex2_approx(rl.x - R); }

// sum + x y, either half
__device__ __forceinline__ float2 dot_bf16x2(uint32_t x, uint32_t y, float2 sum) {
  return make_float2(sum.x + bf16_lo(x) * bf16_lo(y), sum.y + bf16_hi(x) * bf16_hi(y));
}

// One row's state (r, l, 32 dims of O from dim d0) over the keys pos .. end - 1, straight from global memory with a
// running maximum: for rows whose sums left the range of the fast path or whose O is not finite, and for segments with
// nodes whose V is not finite.  A key the row does not see is skipped.  Stretches of kStretch keys are summed apart and then
// added up: of n keys that weigh the same the sums are off by at most (kStretch + n / kStretch) / 2 times 2^-24.
constexpr int kStretch = 256;
__device__ __noinline__ float2 redo_row(const uint8_t *k_base, const uint8_t *v_base, long long page_stride,
                                        int num_pages, const int32_t *table, const uint32_t *mask, const uint16_t *q,
                                        int g, int pos, int end, int base, float c, int d0, float4 *o) {
  float R = -INFINITY, l = 0.f;    // the running maximum, the stretch's sum under it
  float Rt = -INFINITY, L = 0.f;   // the same of the stretches before (Rt <= R)
  float4 y[8];                     // the stretch's O
#pragma unroll 1
  for (int i = 0; i < 8; ++i) o[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int left = kStretch; pos < end; ++pos) {
    const int page = __ldg(table + pos / kPageTokens), node = pos - base;
    if (!(page < 0 || page >= num_pages || (node >= 0 && !(__ldg(mask + (node >> 5)) >> (node & 31) & 1u)))) {
      const long long at = (long long)page * page_stride + (g * kPageTokens + pos % kPageTokens) * kRowBytes;
      const uint4 *k = reinterpret_cast<const uint4 *>(k_base + at), *x = reinterpret_cast<const uint4 *>(q);
      float2 dot = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int i = 0; i < kHeadDim / 8; ++i) {
        const uint4 u = k[i], z = x[i];
        dot = dot_bf16x2(u.w, z.w, dot_bf16x2(u.z, z.z, dot_bf16x2(u.y, z.y, dot_bf16x2(u.x, z.x, dot))));
      }
      const float e = (dot.x + dot.y) * c, Rn = fmaxf(R, e);
      if (e != -INFINITY) {  // (weight 0, and no reference)
        const float keep = R == -INFINITY ? 0.f : exp2f(R - Rn), w = exp2f(e - Rn);
        R = Rn;
        l = l * keep + w;
        const uint2 *v = reinterpret_cast<const uint2 *>(v_base + at) + d0 / 4;
#pragma unroll 2
        for (int i = 0; i < 8; ++i) {
          const uint2 u = v[i];
          const float4 z = y[i];
          y[i] = make_float4(z.x * keep + w * bf16_lo(u.x), z.y * keep + w * bf16_hi(u.x), z.z * keep + w * bf16_lo(u.y),
                             z.w * keep + w * bf16_hi(u.y));
        }
      }
    }
    if ((--left == 0 || pos == end - 1) && (R != -INFINITY || l != 0.f)) {  // (a NaN leaves R as it is)
      const float keep = Rt == -INFINITY ? 0.f : exp2f(Rt - R);
      Rt = R;
      L = L * keep + l;
#pragma unroll 1
      for (int i = 0; i < 8; ++i) {
        const float4 z = o[i], u = y[i];
        o[i] = make_float4(z.x * keep + u.x, z.y * keep + u.y, z.z * keep + u.z, z.w * keep + u.w);
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
      l = 0.f;
    }
    if (left == 0) {
      left = kStretch;
      *reinterpret_cast<volatile unsigned *>(&shared_memory().alive) = clock32();
    }
  }
  return make_float2(Rt, L);
}

// Writes kDims dims of a row.
template <bool kBf16, int kDims>
__device__ __forceinline__ void write_row(void *out, long long at, const float (&r)[kDims]) {
  if constexpr (kBf16) {
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at);
#pragma unroll
    for (int i = 0; i < kDims / 8; ++i)
      dst[i] = make_uint4(pack_bf16x2(r[8 * i], r[8 * i + 1]), pack_bf16x2(r[8 * i + 2], r[8 * i + 3]),
                          pack_bf16x2(r[8 * i + 4], r[8 * i + 5]), pack_bf16x2(r[8 * i + 6], r[8 * i + 7]));
  } else {
    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
#pragma unroll
    for (int i = 0; i < kDims / 4; ++i) dst[i] = make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
  }
}

// Zeroes the rows of sequences whose lengths do not fit, spread over the CTAs (after griddep_wait).
template <bool kBf16>
__device__ __forceinline__ void zero_rows(const TreeArgs &a, int cta, int G, int tid) {
#pragma unroll 1
  for (int s = cta; s < a.num_seqs; s += G) {
    Seq q;
    q.load(a, s);
    if (q.n == 0 || q.valid(a)) continue;
    if (tid == 0) report(a.status, PKV_DEV_BAD_CONTEXT);
    const long long r0 = max((long long)q.q0, 0LL), r1 = min((long long)q.q0 + q.n, (long long)a.num_q_rows);
    constexpr int kChunks = kQHeads * kHeadDim * (kBf16 ? 2 : 4) / 16;  // 16-byte chunks of a row
#pragma unroll 1
    for (long long i = r0 * kChunks + tid; i < r1 * kChunks; i += kThreads)
      static_cast<uint4 *>(a.out)[i] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Merges `count` partial states of a unit whose first part is CTA c0's: those of CTAs c, c + stride, ...
// Writes the unit's rows, or (dst, their first part) the merged state in its place: a thread overwrites only
// what it has read itself, and the merged (reference, sum) have a place of their own.  A thread has one of the
// rows (2^shift of them at the most) and 16 of its dims at a time, with kBatch * kVec loads of 16 bytes in flight.
template <bool kBf16>
__device__ __forceinline__ void merge_parts(const Part *parts, void *out, int c0, int c, int stride, int count, int rows,
                                         int shift, long long row0, Part *dst, int tid) {
  constexpr int kVec = 4, kBatch = 3;
  const int at = tid & ((1 << shift) - 1);
  if (at >= rows) return;
#pragma unroll 1
  for (int d0 = (tid >> shift) * kVec; d0 < kHeadDim / 4; d0 += (kSoftThreads >> shift) * kVec) {
    const int half = d0 / (kHeadDim / 8);
    float R = -INFINITY, L = 0.f;
    float r[4 * kVec];
#pragma unroll
    for (int d = 0; d < 4 * kVec; ++d) r[d] = 0.f;
#pragma unroll 1
    for (int p = 0; p < count; p += kBatch) {
      float2 rl[kBatch];
      float4 y[kBatch][kVec];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool there = p + i < count;
        const int q = c + (there ? p + i : p) * stride;
        const Part &part = parts[2 * q + (q == c0 ? 1 : 0)];
        rl[i] = __ldcg(stride > 1 ? &part.group_rl[half][at] : &part.rl[half][at]);
        if (!there) rl[i].y = 0.f;  // weight 0
#pragma unroll
        for (int d = 0; d < kVec; ++d) y[i][d] = __ldcg(&part.o[d0 + d][at]);
      }
      float Rn = R;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) Rn = rl[i].y == 0.f ? Rn : fmaxf(Rn, rl[i].x);
      const float keep = state_weight(make_float2(R, L), Rn);
      L *= keep;
#pragma unroll
      for (int d = 0; d < 4 * kVec; ++d) r[d] *= keep;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = state_weight(rl[i], Rn);
        if (rl[i].y == 0.f) continue;  // (what it holds does not count, infinities included)
        L += rl[i].y * w;
#pragma unroll
        for (int d = 0; d < kVec; ++d) {
          r[4 * d] += y[i][d].x * w;
          r[4 * d + 1] += y[i][d].y * w;
          r[4 * d + 2] += y[i][d].z * w;
          r[4 * d + 3] += y[i][d].w * w;
        }
      }
      R = Rn;
    }
    if (dst != nullptr) {
#pragma unroll
      for (int d = 0; d < kVec; ++d)
        __stcg(&dst->o[d0 + d][at], make_float4(r[4 * d], r[4 * d + 1], r[4 * d + 2], r[4 * d + 3]));
      if (d0 % (kHeadDim / 8) == 0) __stcg(&dst->group_rl[half][at], make_float2(R, L));
    } else {
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int d = 0; d < 4 * kVec; ++d) r[d] *= inv;
      write_row<kBf16>(out, (row0 + (at >> 2) * kQHeads + (at & 3)) * kHeadDim + d0 * 4, r);
    }
  }
}

template <bool kBf16>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tree_attention_kernel(const __grid_constant__ TreeArgs a) {
  Smem &sm = shared_memory();
  // the warp index by a shuffle: the compiler then knows that a role's values are the same in all lanes
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int G = int(gridDim.x), cta = int(blockIdx.x);

  // ---- what the batch asks for ----
  if (warp == kScoreWarp) tmem_alloc(&sm.tmem_base, kTmemCols);
  if (uint64_t *bar = sm.q_full + tid; bar <= &sm.o_free) {
    mbar_init(bar, bar < sm.s_full ? 1 : bar < sm.p_full ? 2 : bar < &sm.o_free ? kSoftWarps / 2 : kSoftWarps);
    mbar_init_fence();
  }
  if (tid < 4) sm.nonfinite[tid] = -1;
  if (tid == 4) {
    sm.abort = 0;
    sm.alive = clock32() - kWaitCycles - 1;  // none
  }
  // entries of the list, units, and 4 x the blocks of the longest unit + its octets of nodes less one
  long long T = 0;
  int units = 0, longest = 0;
  for (int s = tid; s < a.num_seqs; s += kThreads) {
    Seq q;
    q.load(a, s);
    T += q.entries(0) + q.entries(1);
    units += q.tiles * kKvHeads;
    if (q.tiles > 0) longest = max(longest, 4 * q.nb + (min(q.n, kTok) - 1) / kOctet);
  }
  auto sum = [&](long long x) {  // over the warp, of entries (less than 2^54 in all)
    const unsigned low = __reduce_add_sync(0xffffffffu, unsigned(x) & 0x3ffffffu);
    return ((long long)__reduce_add_sync(0xffffffffu, unsigned(x >> 26)) << 26) + low;
  };
  T = sum(T);
  units = __reduce_add_sync(0xffffffffu, units);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 0) {
    sm.warp_entries[warp] = T;
    sm.warp_units[warp] = units;
    sm.warp_longest[warp] = longest;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  T = sum(lane < kThreads / 32 ? sm.warp_entries[lane] : 0);
  units = __reduce_add_sync(0xffffffffu, lane < kThreads / 32 ? sm.warp_units[lane] : 0);
  longest = __reduce_max_sync(0xffffffffu, lane < kThreads / 32 ? sm.warp_longest[lane] : 0);
  // ---- whole units or shares of the list ----
  const float merge = kMergeCost + kMergeCostOctet * ((longest & 3) + 1);
  longest >>= 2;
  const int length = longest + kUnitCost;
  const int least = min(max(length / (2 * kMergeGroup - 1) + 1, kMinEntries), kMostEntries);
  const float rounds = __fdividef(float(units), float(G)), idle = ceilf(rounds) - rounds;
  const bool whole = length - merge <= fmaxf(__fdividef(float(T), float(G)), float(least)) &&
                     (rounds <= 1.f || idle * length * kLastRound <= merge);
  const int ctas = whole ? min(units, G) : int(min((long long)G, max(1LL, divide(T, least))));  // with anything to do
  if (T == 0 || cta >= ctas) {
    if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
    griddep_wait();
    griddep_launch_dependents();
    zero_rows<kBf16>(a, cta, G, tid);
    return;
  }
  if (tid == 0 || tid == kLoadWarpK * 32) {  // (read in these two warps)
    sm.shares.T = T;
    sm.shares.G = ctas;
    sm.whole = whole;
    sm.units = units;
    sm.longest = longest;
  }
  __syncwarp();
  // Small trees fill the lanes of one warp only: units start at another quarter of the lanes each, so
  // that the quarters (the SM's sub-partitions) share the work.
  const int turn = cta * 2 >= G ? 2 : 0;

  // The pages of a segment's blocks: table entries 32 at a time (8 blocks), the next 32 in flight.
  struct Pages {
    const int32_t *table;
    int npages, next, ent, ent_next;  // of this lane; -1: not in the pool
    unsigned bad;                     // bit i: lane i's is inside the context and not in the pool
    __device__ int entry(int p) const { return p < npages ? __ldg(table + p) : -1; }
    __device__ void check(int p, int num_pages) {
      if (ent >= num_pages) ent = -1;
      bad = __ballot_sync(0xffffffffu, ent < 0 && p < npages);
    }
    __device__ void start(const TreeArgs &a, const Segment &x, int lane) {
      table = a.block_tables + (long long)x.s * a.bt_stride;
      npages = (x.ctx - 1) / kPageTokens + 1;
      next = x.j0 * kPagesPerBlock;
      ent = entry(next + lane);
      ent_next = entry(next + 32 + lane);
    }
    // Pages of the segment's block number i (in order), -1 for what is not in the pool: TMA fills these with zeros.
    // Returns the bits of those inside the context.
    __device__ int block(int i, int num_pages, int lane, int (&page)[kPagesPerBlock]) {
      const int at = i * kPagesPerBlock & 31;
      if (at == 0 && i > 0) {
        next += 32;
        ent = ent_next;
        ent_next = entry(next + 32 + lane);
        check(next + lane, num_pages);
      }
#pragma unroll
      for (int k = 0; k < kPagesPerBlock; ++k) page[k] = __shfl_sync(0xffffffffu, ent, at + k);
      return bad >> at & ((1 << kPagesPerBlock) - 1);
    }
  };

  if (warp >= kSoftWarps) regs_dec<kRegsOthers>();
  if (warp == kLoadWarpK) {
    // ================= K loader (tiled TMA); it walks the list =================
    const uint64_t once = policy_evict_first(), again = policy_evict_last();
    const bool whole = sm.whole != 0;
    Walk walk;
    if (whole) walk.start_units();
    else walk.start(a, sm.shares.first(cta), sm.shares.first(cta + 1), lane);
    if (lane == 0) {
      prefetch_tensormap(&a.tmap_k);
      prefetch_tensormap(&a.tmap_q);
    }
    unsigned gb = 0;  // blocks issued
    int loads = 0;    // segments whose Q was asked for
    bool ok = true, waited = false;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      Segment &x = sm.seg[k % kSegments];
      bool more;  // every lane writes the same
      if (whole) {
        int u = cta;
        if (k > 0) {
          u = sm.units;
          if (u > G) {
            if (lane == 0) u = G + atomicAdd(&a.parts->claimed, 1);
            u = __shfl_sync(0xffffffffu, u, 0);
          }
        }
        more = walk.unit(a, u, sm.units, sm.longest, lane, x);
      } else {
        more = walk.next(a, x);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.seg_full[k % kSegments]);
      if (!more) break;
      Pages pages;
      pages.start(a, x, lane);
      // Q: boxes of 8 nodes x 4 heads, once the segment before the last has read its own
      if (k >= 2) {
        const bool w = wait(sm, &sm.q_empty[k & 1], uint32_t(k / 2 - 1) & 1);
        if (!__all_sync(0xffffffffu, w)) break;
      }
      if (elect_one()) {
        const int octets = (min(kTok, x.n - x.tile * kTok) + kOctet - 1) / kOctet;
        mbar_arrive_expect_tx(&sm.q_full[k & 1], uint32_t(octets * kOctetBytes));
#pragma unroll 1
        for (int o = 0; o < octets; ++o)
          tma_load_3d(sm.q[k & 1] + ((o + k + turn) & 3) * kOctetBytes, &a.tmap_q, 0, x.g * kGroup,
                      x.q0 + x.tile * kTok + o * kOctet, &sm.q_full[k & 1], once);
      }
      __syncwarp();
      ++loads;
      // launched with overlap (PKV_OVERLAP_PREVIOUS), the kernel before this one may still be writing
      // the pool: it is read only once that kernel has completed
      if (!waited) griddep_wait();
      waited = true;
      pages.check(pages.next + lane, a.num_pages);
      const uint64_t policy = x.n > kTok ? again : once;  // several tiles read the same K/V
      const int j0 = x.j0, j1 = x.j1, y = x.g * kPageTokens;
#pragma unroll 1
      for (int j = j0; j < j1; ++j, ++gb) {
        const int st = int(gb % kStagesK);
        int page[kPagesPerBlock];
        const int bad = pages.block(j - j0, a.num_pages, lane, page);
        if (gb >= kStagesK) {
          const unsigned before = gb - kStagesK;  // S of the block whose place it takes is done
          const bool w = wait(sm, &sm.s_full[before % kReady], (before / kReady) & 1);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
        }
        if (elect_one()) {
          if (bad) report(a.status, PKV_DEV_BAD_PAGE);
          sm.block_bad[gb % kReady] = bad;
          mbar_arrive(&sm.s_full[gb % kReady]);
          mbar_arrive_expect_tx(&sm.k_full[st], kTileBytes);
#pragma unroll
          for (int i = 0; i < kPagesPerBlock; ++i)
            tma_load_3d(sm.k[st] + i * kBox, &a.tmap_k, 0, y, page[i], &sm.k_full[st], policy);
        }
        __syncwarp();
      }
    }
    // every copy issued has landed before the CTA exits
    if (lane == 0)
#pragma unroll 1
      for (unsigned j = gb > kStagesK ? gb - kStagesK : 0; j < gb; ++j)
        bounded_wait(&sm.k_full[j % kStagesK], (j / kStagesK) & 1);
    if (lane == 0)
#pragma unroll 1
      for (int j = loads > 2 ? loads - 2 : 0; j < loads; ++j) bounded_wait(&sm.q_full[j & 1], uint32_t(j / 2) & 1);
    __syncwarp();
  } else if (warp == kLoadWarpV) {
    // ================= V loader =================
    const uint64_t once = policy_evict_first(), again = policy_evict_last();
    if (lane == 0) prefetch_tensormap(&a.tmap_v);
    unsigned gb = 0;
    bool ok = true, waited = false;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      bool w = wait(sm, &sm.seg_full[k % kSegments], uint32_t(k / kSegments) & 1);
      if (!__all_sync(0xffffffffu, w)) break;
      const Segment &x = sm.seg[k % kSegments];
      if (x.s < 0) break;
      Pages pages;
      pages.start(a, x, lane);
      if (!waited) griddep_wait();
      waited = true;
      pages.check(pages.next + lane, a.num_pages);
      const uint64_t policy = x.n > kTok ? again : once;
      const int j0 = x.j0, j1 = x.j1, y = x.g * kPageTokens;
#pragma unroll 1
      for (int j = j0; j < j1; ++j, ++gb) {
        const int st = int(gb % kStagesV);
        int page[kPagesPerBlock];
        pages.block(j - j0, a.num_pages, lane, page);
        if (gb >= kStagesV) {
          const unsigned before = gb - kStagesV;
          w = wait(sm, &sm.p_free[before % kReady], (before / kReady) & 1);
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
        }
        if (elect_one()) {
          mbar_arrive_expect_tx(&sm.v_full[st], kTileBytes);
#pragma unroll
          for (int i = 0; i < kPagesPerBlock; ++i)
            tma_load_3d(sm.v[st] + i * kBox, &a.tmap_v, 0, y, page[i], &sm.v_full[st], policy);
        }
        __syncwarp();
      }
    }
    if (lane == 0)
#pragma unroll 1
      for (unsigned j = gb > kStagesV ? gb - kStagesV : 0; j < gb; ++j)
        bounded_wait(&sm.v_full[j % kStagesV], (j / kStagesV) & 1);
    __syncwarp();
  } else if (warp == kScoreWarp) {
    // ================= S = Q K^T (one thread issues, the warp waits) =================
    griddep_wait();  // nothing to do before the loaders; its waits are not to run out on the kernel before
    // The next kernel may start once every CTA of this one is past its wait, so that what it reads at once is
    // complete if a kernel before this one wrote it.
    griddep_launch_dependents();
    const uint64_t q_desc = sw128_desc(smem_addr(sm.q), 16, 1024),
                   k_desc = sw128_desc(smem_addr(sm.k), 16, 1024);  // a later address adds to the low bits
    unsigned gb = 0;  // blocks issued
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      bool w = wait(sm, &sm.seg_full[k % kSegments], uint32_t(k / kSegments) & 1);
      if (!__all_sync(0xffffffffu, w)) break;
      const Segment &x = sm.seg[k % kSegments];
      if (x.s < 0) break;
      const int blocks = x.j1 - x.j0;
      w = wait(sm, &sm.q_full[k & 1], uint32_t(k / 2) & 1);
      if (!__all_sync(0xffffffffu, w)) break;
      const uint64_t qdesc = q_desc + uint32_t((k & 1) * kRows * kRowBytes >> 4);
#pragma unroll 1
      for (int j = 0; j < blocks; ++j, ++gb) {
        const int st = int(gb % kStagesK), b = int(gb % kScores);
        w = wait(sm, &sm.k_full[st], (gb / kStagesK) & 1);
        if (w && gb >= kScores) w = wait(sm, &sm.p_free[(gb - kScores) % kReady], ((gb - kScores) / kReady) & 1);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t kdesc = k_desc + uint32_t(st * kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma(tmem + b * kKeys, qdesc + kk * (32 >> 4), kdesc + kk * (32 >> 4), kIdescS, kk > 0 ? 1u : 0u);
          tc_commit(&sm.s_full[gb % kReady]);
          if (j == blocks - 1) tc_commit(&sm.q_empty[k & 1]);  // the segment's last read of its Q
        }
        __syncwarp();
      }
    }
    // every MMA issued has completed before the tensor memory is freed
    if (elect_one()) {
      tc_commit(&sm.mma_done[0]);
      bounded_wait(&sm.mma_done[0], 0);
    }
    __syncwarp();
  } else if (warp == kValueWarp) {
    // ================= O += P V (one thread issues, the warp waits) =================
    griddep_wait();
    const uint64_t v_desc = sw128_desc(smem_addr(sm.v), 16, 1024);
    unsigned gb = 0, runs = 0;  // blocks and runs issued
    bool ok = true;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      bool w = wait(sm, &sm.seg_full[k % kSegments], uint32_t(k / kSegments) & 1);
      if (!__all_sync(0xffffffffu, w)) break;
      const Segment &x = sm.seg[k % kSegments];
      if (x.s < 0) break;
      const int blocks = x.j1 - x.j0;
#pragma unroll 1
      for (int j = 0; j < blocks; ++j, ++gb) {
        const int in_run = j % kRunBlocks<kBf16>;
        const bool run_ends = j == blocks - 1 || in_run == kRunBlocks<kBf16> - 1;
        const int st = int(gb % kStagesV), b = int(gb % kScores);
        w = wait(sm, &sm.v_full[st], (gb / kStagesV) & 1) &&
            wait(sm, &sm.p_full[b], (gb / kScores) & 1);
        // a run's first product overwrites O, once every softmax warp has read the one before
        if (w && in_run == 0 && runs > 0) w = wait(sm, &sm.o_free, (runs - 1) & 1);
        if (!__all_sync(0xffffffffu, w)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vdesc = v_desc + uint32_t(st * kTileBytes >> 4);
#pragma unroll
          for (int kk = 0; kk < kKeys / 16; ++kk)
#pragma unroll
            for (int term = 0; term < (kBf16 ? 1 : 2); ++term)
              tc_mma_tmem_a(tmem + kColO, tmem + b * kKeys + kk * 16 + term * 8,
                            vdesc + kk * (2048 >> 4), kIdescPV, (in_run == 0 && kk == 0 && term == 0) ? 0u : 1u);
          tc_commit(&sm.p_free[gb % kReady]);
          if (run_ends) tc_commit(&sm.o_full);
        }
        __syncwarp();
        runs += run_ends ? 1 : 0;
      }
    }
    if (elect_one()) {
      tc_commit(&sm.mma_done[1]);
      bounded_wait(&sm.mma_done[1], 0);
    }
    __syncwarp();
  } else {
    // ================= softmax: warp = (quarter of the lanes, group), thread = row =================
    regs_inc<kRegsSoftmax>();
    griddep_wait();  // the mask and every global write come after the kernel before this one
    const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;  // half: the group, and dims 32 half .. + 31
    const uint32_t my_tmem = tmem + (uint32_t(32 * quarter) << 16);
    unsigned gb0 = 0;  // blocks before the segment
    unsigned gb = half, b = half;  // the group's next block, its S / P buffer
    int turns = 0;     // segments in which this warp has had rows (the two warps of a quarter agree)
    int cuts = 0;      // bit 0, 1: the share's first, last unit is cut
    bool ok = true;
    // A run ends while the next one's first block is under way: once that block's P is stored, end_run() takes the
    // run's O, and at a segment's end (its sums have been posted) divides and writes its rows or their partial state.
    unsigned ended = 0;            // runs this warp has ended
    unsigned runs = 0, before = 0;  // runs before the current segment, before the one before it
    // The end of a run of segment k (whose first run is `first`), its last or not, for this warp: this thread has its
    // row's dims 32 half .. + 31.
    auto end_run = [&](int k, unsigned first, bool last) {
      const Segment &x = sm.seg[k % kSegments];
      const int octet = (quarter - k - turn) & 3, base = x.ctx - x.n, pos0 = x.j0 * kKeys, pos1 = min(x.ctx, x.j1 * kKeys);
      const bool active = octet * kOctet < x.n - x.tile * kTok;
      const int node = x.tile * kTok + octet * kOctet + (lane >> 2), t = turns - 1;
      const bool real = node < x.n;
      // the segment's part; between runs it holds their sum, each thread its own row and dims
      Part &part = a.parts[2 * cta + (x.j0 == 0 ? 1 : 0)];
      const int at = octet * 32 + lane;
      float r[32];
#pragma unroll
      for (int d = 0; d < 32; ++d) r[d] = 0.f;
      // The sum of the runs before is read before o_free is arrived at: the next segment's rows have other threads, which
      // write the same part, and what orders their stores behind these loads is o_free, a product and o_full.
      if (active && ended > first) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float4 y = __ldcg(&part.o[half * 8 + i][at]);
          r[4 * i] = y.x;
          r[4 * i + 1] = y.y;
          r[4 * i + 2] = y.z;
          r[4 * i + 3] = y.w;
        }
      }
      bool w = wait(sm, &sm.o_full, ended & 1);
      ++ended;
      if (active && last) w = wait(sm, &sm.sums_full[quarter], uint32_t(t) & 1) && w;
      if (!__all_sync(0xffffffffu, w)) return false;
      if (active) {
        uint32_t u[32];
        tc_fence_after();
        tmem_ld32(my_tmem + kColO + half * 32, u);
        tc_fence_before();
#pragma unroll
        for (int d = 0; d < 32; ++d) r[d] += __uint_as_float(u[d]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_free);
      if (!active) return true;
      auto store_part = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          __stcg(&part.o[half * 8 + i][at], make_float4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]));
      };
      if (!last) {
        store_part();
        return true;
      }
      float L = sm.sums[t & 3][0][row] + sm.sums[t & 3][1][row], ref = sm.ref[t & 3][row];
      const int h = x.g * kGroup + (lane & 3);
      const long long qrow = (long long)x.q0 + node;
      float z = 0.f;  // NaN when O is too large or not finite (an infinite V: hi and lo terms make a NaN of it)
#pragma unroll
      for (int d = 0; d < 32; ++d) z += r[d] * kInfOverMaxO * 0.f;
      const bool redo = !(L >= kSumMin && L <= kSumMax) || z != 0.f;
      if (real && (redo || *reinterpret_cast<volatile int *>(&sm.nonfinite[k & 3]) == k) &&
          (L != 0.f || sees_any(a.mask + qrow * a.mask_stride, pos0, pos1, base, x.n))) {
        float4 o[8];  // (it lies in memory: few come here)
        const float2 rl = redo_row(a.k_base, a.v_base, a.page_stride, a.num_pages,
                                   a.block_tables + (long long)x.s * a.bt_stride, a.mask + qrow * a.mask_stride,
                                   a.q + (qrow * kQHeads + h) * kHeadDim, x.g, pos0, pos1, base, a.c.x, half * 32, o);
        ref = rl.x;
        L = rl.y;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          r[4 * i] = o[i].x;
          r[4 * i + 1] = o[i].y;
          r[4 * i + 2] = o[i].z;
          r[4 * i + 3] = o[i].w;
        }
      }
      if (!real) return true;
      if (x.j0 == 0 && x.j1 == x.nb) {
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int d = 0; d < 32; ++d) r[d] *= inv;
        write_row<kBf16>(a.out, (qrow * kQHeads + h) * kHeadDim + half * 32, r);
      } else {
        // a cut unit: a partial state; its ticket is taken when the share is done
        store_part();
        __stcg(&part.rl[half][at], make_float2(ref, L));
      }
      return true;
    };
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      bool w = wait(sm, &sm.seg_full[k % kSegments], uint32_t(k / kSegments) & 1);
      if (!__all_sync(0xffffffffu, w)) break;
      const Segment &x = sm.seg[k % kSegments];
      const bool more = x.s >= 0;  // if not, a round of the loop below ends the last segment
      const int octet = (quarter - k - turn) & 3, base = x.ctx - x.n, j0 = more ? x.j0 : 0, j1 = more ? x.j1 : 0;
      const bool active = more && octet * kOctet < x.n - x.tile * kTok;  // the warp has rows
      // this thread's row, valid where `real`
      const int node = x.tile * kTok + octet * kOctet + (lane >> 2);
      const bool real = active && node < x.n;
      if (real && j1 * kKeys > base)  // the mask word of the segment's first node key, needed at its end
        prefetch_l1(a.mask + (long long)(x.q0 + node) * a.mask_stride + (max(j0 * kKeys - base, 0) >> 5));
      const bool leads = int(gb0 & 1) == half;  // the segment's first block is this group's
      float2 l2 = make_float2(0.f, 0.f), minus_r = l2;  // sum of the blocks since keep_sum(), - reference, both twice
      if (active) sm.sums[turns & 3][half][row] = 0.f;
      auto keep_sum = [&]() {
        sm.sums[turns & 3][half][row] += l2.x + l2.y;
        l2 = make_float2(0.f, 0.f);
      };
      const int last_run = more ? (j1 - j0 - 1) / kRunBlocks<kBf16> : 0;
      // Blocks before `plain_end` hold no nodes, no run ends at them and the reference is there.
      int plain_end = 0;
#pragma unroll 1
      for (int j = j0 + (leads ? 0 : 1);; j += 2) {
        const uint32_t taddr = my_tmem + b * kKeys;
        bool plain = j < plain_end, has = true;
        unsigned due = 0;
        if (__builtin_expect(plain, 1)) {
          w = wait(sm, &sm.s_full[gb % kReady], (gb / kReady) & 1);
          ok = __all_sync(0xffffffffu, w);
          if (!ok) break;
          tc_fence_after();
          plain = sm.block_bad[gb % kReady] == 0;
        }
        if (__builtin_expect(!plain, 0)) {
          has = j < j1;
          // the runs to end before this block's P is handed over: all before its own; after the last block
          // all but the segment's last
          due = runs + (has ? (j - j0) / kRunBlocks<kBf16> : last_run);
          if (!has && ended == due) break;
          if (has) {
            const int key0 = j * kKeys;
            w = wait(sm, &sm.s_full[gb % kReady], (gb / kReady) & 1);
            if (w && key0 + kKeys > base) {
              // the block holds nodes: the group's threads look through V, two to a row
              const int st = int(gb % kStagesV), r = (tid & 127) >> 1, pos = key0 + r;
              w = wait(sm, &sm.v_full[st], (gb / kStagesV) & 1);  // (the phase before has been consumed)
              __syncwarp();
              uint8_t *vrow = sm.v[st] + r * kRowBytes;
              uint32_t bits = 0;
#pragma unroll
              for (int i = 0; i < 4; ++i)
                bits |= nonfinite(*reinterpret_cast<const uint4 *>(vrow + (((tid & 1) * 4 + i) ^ (r & 7)) * 16));
              bool inf = bits != 0 && pos >= base && pos < x.ctx;
              inf |= __shfl_xor_sync(0xffffffffu, int(inf), 1) != 0;
              if (pos >= x.ctx || inf) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  *reinterpret_cast<uint4 *>(vrow + (((tid & 1) * 4 + i) ^ (r & 7)) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
              if (inf) *reinterpret_cast<volatile int *>(&sm.nonfinite[k & 3]) = k;
              fence_proxy_async_smem();
            }
            if (active && j > j0 && j == j0 + 1) {  // (this group does not lead: the row's reference is the other's)
              w = wait(sm, &sm.ref_full[quarter][turns & 1], uint32_t(turns >> 1) & 1) && w;
              const float ref = sm.ref[turns & 3][row];
              minus_r = make_float2(-ref, -ref);
            }
            ok = __all_sync(0xffffffffu, w);
            if (!ok) break;
            if (active) {
              keep_sum();
              tc_fence_after();
              const int bad = sm.block_bad[gb % kReady];
              const bool masked = key0 + kKeys > base || bad != 0;  // uniform over the warp
              if (masked) {
                uint32_t see0 = ~0u, see1 = ~0u;
                if (key0 + kKeys > base) {
                  const uint32_t *mask = a.mask + (long long)(x.q0 + node) * a.mask_stride;
                  see0 = real ? window_bits(mask, key0, base, x.ctx, x.n) : 0u;
                  see1 = real ? window_bits(mask, key0 + 32, base, x.ctx, x.n) : 0u;
                }
                if (bad & 1) see0 &= 0xffff0000u;
                if (bad & 2) see0 &= 0x0000ffffu;
                if (bad & 4) see1 &= 0xffff0000u;
                if (bad & 8) see1 &= 0x0000ffffu;
                hide_keys(taddr, see0, see1, a.c.x);
              }
              if (j == j0) {
                const float ref = block_reference(taddr, a.c.x);
                minus_r = make_float2(-ref, -ref);
                sm.ref[turns & 3][row] = ref;
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.ref_full[quarter][turns & 1]);
              }
            }
          }
        }
        if (active && has) {
          block_weights<kBf16>(taddr, a.c, minus_r, l2);
          tc_fence_before();
        }
        if (__builtin_expect(!plain, 0)) {
#pragma unroll 1
          while (ok && ended != due) {
            const bool last = ended < runs;  // of the segment before
            ok = end_run(last ? k - 1 : k, last ? before : runs, last);
          }
          plain_end = min(j1, base / kKeys);
          plain_end = min(plain_end, j0 + ((j - j0) / kRunBlocks<kBf16> + 1) * kRunBlocks<kBf16>);
        }
        __syncwarp();
        if (!has) break;
        if (lane == 0) mbar_arrive(&sm.p_full[b]);
        if (!ok) break;
        gb += 2;
        b = b == 0 ? kScores - 1 : b - 1;  // + 2 modulo 3
      }
      if (!ok || !more) break;
      gb0 += unsigned(j1 - j0);
      if (j0 != 0 || j1 != x.nb) {
        const int i = j0 == 0 ? 1 : 0;  // the share's last unit goes on in the next, its first began before
        cuts |= 1 << i;
        if (tid == 0) sm.cuts[i] = x;
      }
      if (active) {
        keep_sum();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.sums_full[quarter]);
        ++turns;
      }
      before = runs;
      runs += last_run + 1;
    }
    // ---- the tickets of the cut units: the CTA that takes a unit's last one merges its parts; in a unit of
    // many parts first the parts of a group, then the CTA with the last group the groups ----
    // (every softmax warp comes here, whatever became of its waits)
    auto ticket_taken = [&](int *ticket, int before) {
      const bool last = atomic_add_acq_rel_gpu(ticket, 1) == before;
      if (last) atomicExch(ticket, 0);  // ready for the next call
      return last;
    };
    named_barrier_sync(5, kSoftThreads);
    if (tid < 2) {
      int merge = 0;
      if (cuts >> tid & 1 && *reinterpret_cast<volatile int *>(&sm.abort) == 0) {
        const Segment &u = sm.cuts[tid];
        int ends[2];
#pragma unroll 1
        for (int i = 0; i < 2; ++i) ends[i] = sm.shares.owner(u.unit0 + (i ? u.nb - 1 : 0));
        const int c0 = ends[0], parts = ends[1] - ends[0] + 1;
        sm.cut_first[tid] = c0;
        sm.cut_parts[tid] = parts;
        if (parts <= 2 * kMergeGroup) {
          merge = ticket_taken(a.tickets + ((long long)u.s * a.max_tiles + u.tile) * kKvHeads + u.g, parts - 1) ? 1 : 0;
        } else {
          const int lo = (cta - c0) / kMergeGroup * kMergeGroup, hi = min(lo + kMergeGroup, parts) - 1;
          merge = ticket_taken(&a.parts[2 * (c0 + lo) + (lo == 0 ? 1 : 0)].ticket, hi - lo) ? 2 : 0;
        }
      }
      sm.merge[tid] = merge;
    }
    named_barrier_sync(5, kSoftThreads);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      int merge = sm.merge[i];
      if (merge == 0) continue;
      const Segment &u = sm.cuts[i];
      const int c0 = sm.cut_first[i], parts = sm.cut_parts[i];
      const int rows = min(kTok, u.n - u.tile * kTok) * kGroup;
      const long long row0 = ((long long)u.q0 + u.tile * kTok) * kQHeads + u.g * kGroup;
      const int shift = rows <= 32 ? 5 : rows <= 64 ? 6 : 7;
      auto merge_rows = [&](int c, int stride, int count, Part *dst) {
        merge_parts<kBf16>(a.parts, a.out, c0, c, stride, count, rows, shift, row0, dst, tid);
      };
      int c = c0, stride = 1, count = parts;  // what to merge: all parts, or first this CTA's group of them
      Part *dst = nullptr;
      if (merge == 2) {
        const int lo = (cta - c0) / kMergeGroup * kMergeGroup;
        c = c0 + lo;
        count = min(kMergeGroup, parts - lo);
        dst = &a.parts[2 * c + (lo == 0 ? 1 : 0)];
      }
#pragma unroll 1
      for (;;) {
        merge_rows(c, stride, count, dst);
        if (dst == nullptr) break;
        c = c0;
        stride = kMergeGroup;
        count = (parts + kMergeGroup - 1) / kMergeGroup;
        dst = nullptr;
        named_barrier_sync(5, kSoftThreads);
        if (tid == 0)
          sm.merge[i] = ticket_taken(a.tickets + ((long long)u.s * a.max_tiles + u.tile) * kKvHeads + u.g, count - 1);
        named_barrier_sync(5, kSoftThreads);
        if (!sm.merge[i]) break;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && sm.abort) report(a.status, PKV_DEV_TIMEOUT);
  if (tid == 0 && sm.whole && sm.units > G && atomicAdd(&a.parts->done, 1) == G - 1) {
    atomicExch(&a.parts->claimed, 0);  // ready for the next call
    atomicExch(&a.parts->done, 0);
  }
  zero_rows<kBf16>(a, cta, G, tid);
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kMaxSeqs = 1 << 24, kMaxNodes = 1 << 20;
constexpr int kMaxContext = 0x7fffffff / kKeys * kKeys;  // the last block's end is an int too

size_t ticket_bytes(int num_seqs, int max_tiles) {
  return (size_t(num_seqs) * size_t(max_tiles) * kKvHeads * sizeof(int32_t) + 127) / 128 * 128;
}
// The partial states come first: their place does not depend on the call's shape, and tickets return to zero.
size_t workspace_size(int num_seqs, int max_tiles) {
  return 2 * size_t(kMaxCtas) * sizeof(Part) + ticket_bytes(num_seqs, max_tiles);
}

// The kernels' shared-memory limit, set once per device.
int setup_attributes() {
  static std::mutex mu;
  static bool done[64] = {false};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return PKV_OK;
  constexpr auto attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
  if (cudaFuncSetAttribute(tree_attention_kernel<false>, attr, int(kSmemBytes)) != cudaSuccess ||
      cudaFuncSetAttribute(tree_attention_kernel<true>, attr, int(kSmemBytes)) != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_CUDA;
  }
  done[dev] = true;
  return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int num_seqs, int max_query, int num_q_heads, int head_dim) {
  if (num_seqs < 0 || num_seqs > pkv::kMaxSeqs || max_query < 0 || max_query > pkv::kMaxNodes ||
      num_q_heads != pkv::kQHeads || head_dim != pkv::kHeadDim)
    return 0;
  return pkv::workspace_size(num_seqs, max_query / pkv::kTok + (max_query % pkv::kTok != 0));
}

extern "C" int pkv_paged_tree_attention(const pkv_pool *pool, void *out, const void *q, int num_q_heads,
                                        int num_q_rows, const int32_t *query_start, const uint32_t *tree_mask,
                                        int64_t mask_stride, const int32_t *block_tables, int64_t block_table_stride,
                                        const int32_t *context_lens, int num_seqs, int max_query, int max_context,
                                        float scale, void *workspace, size_t workspace_bytes, int32_t *device_status,
                                        unsigned flags, void *stream) {
  if (flags & ~unsigned(PKV_OVERLAP_PREVIOUS | PKV_OUT_BF16)) return PKV_ERR_SHAPE;
  int rc = pkv::check_pool(pool);
  if (rc != PKV_OK) return rc;
  if (num_q_heads != pkv::kQHeads) return PKV_ERR_UNSUPPORTED;
  if (num_seqs < 0 || max_query < 0 || max_context < 0 || block_table_stride < 0 || num_q_rows < 0 ||
      num_seqs > pkv::kMaxSeqs || max_query > pkv::kMaxNodes || max_context > pkv::kMaxContext || mask_stride < 0 ||
      mask_stride > (1 << 26) || mask_stride * 32 < max_query)
    return PKV_ERR_SHAPE;
  if (num_seqs == 0 || max_query == 0 || num_q_rows == 0) return PKV_OK;
  if (out == nullptr || q == nullptr || query_start == nullptr || tree_mask == nullptr || block_tables == nullptr ||
      context_lens == nullptr || workspace == nullptr)
    return PKV_ERR_NULL;
  if (!isfinite(scale * pkv::kLog2e)) return PKV_ERR_SCALE;  // the exponents' factor: infinite, a score of 0 were a NaN
  if (!pkv::aligned16(q) || !pkv::aligned16(out) || !pkv::aligned16(workspace) ||
      ((reinterpret_cast<uintptr_t>(query_start) | reinterpret_cast<uintptr_t>(tree_mask) |
        reinterpret_cast<uintptr_t>(block_tables) | reinterpret_cast<uintptr_t>(context_lens)) & 3u))
    return PKV_ERR_ALIGN;
  const int tiles = max_query / pkv::kTok + (max_query % pkv::kTok != 0);
  if (workspace_bytes < pkv::workspace_size(num_seqs, tiles)) return PKV_ERR_WORKSPACE;
  rc = pkv::setup_attributes();
  if (rc != PKV_OK) return rc;
  pkv::TreeArgs a;
  rc = pkv::pool_tensor_maps(pool, pkv::kPageTokens, &a.tmap_k, &a.tmap_v);
  if (rc != PKV_OK) return rc;
  rc = pkv::query_tensor_map(q, num_q_rows, pkv::kQHeads, pkv::kHeadDim, pkv::kGroup, pkv::kOctet, &a.tmap_q);
  if (rc != PKV_OK) return rc;
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
  a.max_tiles = tiles;
  // a scale of 0 (all weights alike) becomes one whose product with a finite score vanishes, and with an infinite one
  // (a hidden key) does not
  const float c = scale * pkv::kLog2e, least = 1e-42f;
  a.c.x = a.c.y = fabsf(c) < least ? copysignf(least, c) : c;
  a.parts = static_cast<pkv::Part *>(workspace);
  a.tickets = reinterpret_cast<int *>(static_cast<uint8_t *>(workspace) + 2 * size_t(pkv::kMaxCtas) * sizeof(pkv::Part));
  a.status = device_status;
  // no more CTAs than the list can have shares
  const double entries = double(num_seqs) * tiles * pkv::kKvHeads * (max_context / pkv::kKeys + 1 + pkv::kUnitCost);
  const int sms = pkv::device_sm_count();
  long long grid = (long long)(sms > 0 ? sms : 152) * pkv::kCtasPerSm;
  if (grid > pkv::kMaxCtas) grid = pkv::kMaxCtas;
  if (double(grid) > entries / pkv::kMinEntries) grid = (long long)(entries / pkv::kMinEntries);
  if (grid < 1) grid = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(grid));
  cfg.blockDim = dim3(pkv::kThreads);
  cfg.dynamicSmemBytes = pkv::kSmemBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (flags & PKV_OVERLAP_PREVIOUS) ? 1 : 0;
  const cudaError_t err = (flags & PKV_OUT_BF16) ? cudaLaunchKernelEx(&cfg, pkv::tree_attention_kernel<true>, a)
                                                 : cudaLaunchKernelEx(&cfg, pkv::tree_attention_kernel<false>, a);
  if (err != cudaSuccess) {
    cudaGetLastError();
    return PKV_ERR_LAUNCH;
  }
  return PKV_OK;
}
