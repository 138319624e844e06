// Attention of several new tokens a sequence over a paged KV cache, sm_103a:
// causal for prompts, by a mask of drafted tokens for trees. The operations are
// stated in include/gqa_prompt.h.
//
// Rows. For one KV head the G query heads of a sequence's new tokens form the
// rows of one matrix, token by token: a query tile is TB = 128 / G tokens
// (TB * G <= 128 rows), so a key that is read once meets 128 rows, or 256 where
// two tiles of a sequence run together, and the keys that a causal tile masks
// are few (a tile of 32 tokens at G = 4 wastes half of 32 keys, not of 128).
//
// Items and units. An item is one query tile or a pair of them; it needs the
// key tiles up to its last visible row. Long items are cut along the keys into
// units of at most a chunk where that evens the SMs out; other items are one unit
// each and write their output themselves. Units are handed out heaviest first, each for every KV head. The
// lengths live on the device, so the first CTA to arrive makes the list while
// the others set up; who was first shows in a ticket. Where an item was cut, its
// units write their unnormalised output, maximum and sum to slots, and when no
// unit is left the CTAs join each row's slots in split order: who computed what
// does not matter for the result.
//
// CTAs that wait. The list and the slots are waited for by CTAs that hold an SM,
// and nothing says that all CTAs of a launch are placed at once: other streams'
// kernels may hold SMs, and wait likewise. So a CTA owns nothing before it runs:
// the list's maker is whoever came first, and every unit, a CTA's first one too, is
// claimed from one counter. What is waited for is then done by CTAs that run.
//
// A unit runs an online softmax over tiles of KEYS keys:
//   S = Q K^T     tcgen05.mma, M = 128 rows, N = KEYS, both from shared memory
//                 (K-major, 128-byte swizzle), S in tensor memory;
//   P = 2^(S' - m) by one softmax warpgroup, a row a thread, S' = S * scale *
//                 log2 e; P goes back to tensor memory over S as 16 bits;
//   O += P V      tcgen05.mma with P as the A operand from tensor memory and V
//                 from shared memory (MN-major), O in tensor memory.
// m moves only when a row's maximum has grown by much (then O and l are rescaled),
// so O is rarely touched. A tile without masks behind a first one is not searched
// for its maximum at all: its weights are made with m as it is, and only if a row's
// sum of them reaches 2^8 are they made again, with the tile's own maximum. So
// weights stay below 2^8. They are rounded to 16 bits for the one product that makes
// O (half a step each; the sum l takes them unrounded).
//
// D <= 128: two streams (S, O and a softmax warpgroup each) work in turn, so
// the tensor core multiplies for one while the other makes weights. The
// streams take the two query tiles of a pair and share every K and V stage, or
// the even and odd key tiles of a single query tile, merged at the unit's end.
// D = 256: O fills half of the tensor memory, so there is one stream with two
// S buffers and key tiles of 64; at that width the scores' product with both
// operands in shared memory waits for it (48 cycles where it takes 32), so the
// second warpgroup, which has no stream, copies the queries to tensor memory and
// the product takes them from there.
//
// Masked places. A key that some row of a unit must not see can hold anything,
// NaN and infinities too: its score is replaced, but a weight of 0 times such a
// value would still be NaN. So a warp of its own looks through the V rows of the
// tiles that are masked, zeroes what is past the last visible row and every
// value that is not finite, and notes that it did; such values are then added
// to the rows that do see them when the unit ends (a slow path that only such
// caches take).
//
// Bounds and figures (device time of a call, bf16, blocks of 16 if not named). A
// whole prompt is the tensor cores': 16384 tokens, 32 + 8 heads of 128, 1.42 ms in
// loops of calls, 1550 TFLOP/s, where the chip's 1400 W hold it (0.82 of a matrix
// product's measured burst rate, 0.92 of its sustained one), and 1.30 ms in runs of
// five calls. The figures below are of short runs. A pair's key tile takes about 2900
// cycles for 2048 of products: of a stream's own chain, 1024 are products, about
// 1150 softmax and the rest hand-overs. D = 64 (32 + 4 heads, 4 x 4096 tokens)
// 318 us, 865 TFLOP/s: a pair tile has the same 2 x 128 x 128 weights to make for half
// of the products (which of their instructions bounds it was not measured); D = 256
// (8 + 4 heads, 4 x 4096) 231 us, 1190: one stream. Trees over a cache are HBM's: 64
// sequences of 1 to 8192 rows, up to 13 drafts, 182 us (186 in loops of calls), 5.9
// TB/s, of which 10 us pass before the first keys arrive. The smallest calls are
// chains of latencies: 61 tokens of 8 + 2 heads of 64 11 us, 7 drafts over 500 rows
// 13 us: plan 2, a record 1, table and first keys 2.5, a masked tile 1.5, cleared V
// 1.5, the unit's end 1.5.
//
// Warps: 0-3 and 4-7 softmax warpgroups (and the units' ends), 8 issues the
// MMAs from one thread, 9 hands out units and loads queries and K, 10 loads V,
// 11 clears V. Every wait is bounded (2 s): on expiry the role sets the status
// word and leaves, the others run out in turn, copies and MMAs in flight are
// waited for and tensor memory is freed.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_tc.cuh"

namespace gqa_av {

constexpr int kPtThreads = 384;
// Registers a thread: 168 at launch (65536 / 384, rounded down to 8). A softmax
// thread holds a row's 128 scores (at 184 registers it spills, which costs more than
// reading them twice), the MMA warp the state of both streams (at 104 it spills: a
// prompt of 16384 tokens 1398 us, 1343 with 120): 2 * 128 * 192 + 128 * 120 = 384 * 168.
constexpr int kPtSoftmaxRegs = 192, kPtAuxRegs = 120;
constexpr int kPtMmaWarp = 8, kPtKWarp = 9, kPtVWarp = 10, kPtCleanWarp = 11;
constexpr int kPtMaxB = 8192;          // 16 bytes of the plan's shared memory each
constexpr int kPtSegs = 2;             // unit descriptors in flight
constexpr int kPtCleans = 8;           // barriers of cleared V tiles; more than stages
constexpr int kPtSmall = 32;           // sequences and items of a small batch: a lane each
constexpr int kPtBuckets = 256;        // of unit costs
constexpr int kPtMinChunk = 4;         // key tiles
constexpr int kPtCosts = 16384;        // items whose costs the plan keeps
// Chunks that the plan tries: 1.1 of an SM's share times 2^(-0.0929 i), i < 24, so
// down to a quarter of it. In key tiles (0.75 us): a unit's start and end; 8 rows
// of a partial result, written and read; the step that joins them. Measured at
// D = 128 and used for all: a tile of the other widths takes another time.
constexpr float kPtTopChunk = 1.1f, kPtChunkStep = 0.0929f;
constexpr float kPtUnitCost = 3.0f, kPtRowCost = 0.14f, kPtJoinCost = 4.0f;
constexpr int kPtDeep = 4096;          // mean rows that make a batch deep
constexpr float kPtGrow = 8.0f;        // log2 of the growth of a maximum that is tolerated
constexpr unsigned kErrPtPlan = 8u, kErrPtLoad = 16u, kErrPtMma = 32u, kErrPtSoftmax = 64u,
                   kErrPtClean = 128u;
constexpr long long kPtTimeoutNs = 2000000000LL;   // bound of every wait; also of the last ones,
                                                   // for copies and MMAs in flight

// Set by waits that run out, read by gqa_prompt_device_status. One word a device
// for the life of the process: a workspace may be outgrown while captured graphs
// still run in it, and what they report must be found.
__device__ unsigned pt_status;

template <int D>
struct PtShape {
  static constexpr int NS = D == 256 ? 1 : 2;          // streams
  static constexpr int KEYS = D == 256 ? 64 : 128;     // keys of a tile
  static constexpr int PARTS = D / 64;                 // 64-column parts of a row
  static constexpr int STAGE = KEYS * D * 2;           // bytes of a K or V stage
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int QBUF = NS;                      // query buffers
  static constexpr int KST = D == 64 ? 5 : 2;          // stages of K, and of V, which is held longer
  static constexpr int VST = D == 64 ? 6 : 3;
  static constexpr int TILES_BYTES = QBUF * QBYTES + (KST + VST) * STAGE;
  static constexpr int MISC = D == 64 ? 2048 : 1024;   // barriers, units
  static constexpr int SMEM = TILES_BYTES + MISC + 2048;
  static constexpr uint32_t S_COL = KEYS;              // tensor-memory columns of an S buffer
  static constexpr uint32_t O_COL0 = 256;
  static constexpr uint32_t Q_COL = 128;               // queries in tensor memory (one stream)
};

// What a CTA works on at a time: key tiles t0 .. t0 + tiles - 1 for the rows of
// one or two query tiles. Prompts: token x sees rows c <= base + x; trees: rows
// c < base, and the drafted rows by its mask; both c < lim.
struct alignas(16) PtUnit {
  int b;              // sequence
  int tok, ntok;      // its tokens; ntok 0: no unit left
  int base, lim;
  int t0, tiles;
  int slot;           // of the partial result, or -1: the unit is a whole item
};
struct alignas(16) PtSplit {   // an item that was cut
  int tok, ntok, slot, splits;
};
// Zeroed when the workspace is made, and by the last CTA of each call.
struct PtHeader {
  unsigned ticket, ready, next, done, left;
  int units;                      // times KV heads
  int splits, parts;              // items that were cut, and their slots
};

struct alignas(64) PromptParams {
  CUtensorMap q_map;              // q as {D, G, Hkv, T}; box {64, G, 1, TB}
  CUtensorMap k_map, v_map;       // pools as {D, Hkv, rows}; box {64, 1, R}
  const int32_t *token_start, *cached_lens, *tree_mask, *block_table, *seq_lens;
  const void* v_pool;
  void* out;
  PtHeader* head;
  PtSplit* splits;
  PtUnit* units;
  float* part_o;                  // slots [slot][Hkv][NS][D / 4][128][4]
  float2* part_ml;                // [slot][Hkv][NS][128] (maximum in log2 units, sum)
  int B, T, Hq, Hkv, G, TB, words;
  int bs, num_blocks, max_blocks;
  unsigned bs_mul;                // c / bs = c * bs_mul >> bs_shift for c < 2^26
  int bs_shift;
  int R;                          // rows of a K or V box: gcd(bs, KEYS)
  float qscale;                   // |scale| * log2(e)
  int negate;                     // scale < 0
  int small;                      // at most kPtSmall sequences and items: no list of units
  long long timeout_ns;
  unsigned withhold_from;         // self-test: query loads from this one of a CTA on are not issued
  unsigned late_from;             // self-test: CTAs from this one on start late_ns later
  long long late_ns;
};

__device__ __forceinline__ int pt_block_of(const PromptParams& p, int c) {
  return static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(c)) * p.bs_mul) >>
                          p.bs_shift);
}

// How a unit's streams share it.
struct PtShare {
  bool pair;          // two query tiles, a stream each; else one, cut into even and odd key tiles
  int n0, n1;         // key tiles of each stream
  int full;           // rows that all tokens of the unit see
};
template <int D>
__device__ __forceinline__ PtShare pt_share(const PromptParams& p, const PtUnit& u) {
  using Shape = PtShape<D>;
  PtShare s;
  s.pair = Shape::NS == 2 && u.ntok > p.TB;
  s.full = min(p.tree_mask ? u.base : u.base + 1, u.lim);
  if (Shape::NS == 1) {
    s.n0 = u.tiles;
    s.n1 = 0;
  } else if (s.pair) {
    // The first query tile of a prompt may be done some tiles before the second.
    const int sees = p.tree_mask ? u.lim : min(u.base + p.TB, u.lim);
    s.n0 = max(min((sees + Shape::KEYS - 1) / Shape::KEYS - u.t0, u.tiles), min(1, u.tiles));
    s.n1 = u.tiles;
  } else {
    s.n0 = (u.tiles + 1) / 2;
    s.n1 = u.tiles / 2;
  }
  return s;
}

// Bits c = 0 .. n - 1 of 32.
__device__ __forceinline__ uint32_t below32(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// Which of the 32 rows from `col` on token x of a unit sees.
__device__ __forceinline__ uint32_t pt_sees(const PromptParams& p, int tok, int base, int lim, int x,
                                            int col) {
  if (!p.tree_mask) return below32(min(base + x + 1, lim) - col);
  const uint32_t old = below32(min(base, lim) - col);
  const int off = col - base;
  if (off <= -32) return old;
  const int32_t* words = p.tree_mask + static_cast<size_t>(tok + x) * p.words;
  uint32_t drafts;
  if (off < 0) {
    drafts = static_cast<uint32_t>(__ldg(words)) << -off;
  } else {
    const int i = off >> 5;
    const uint32_t a = i < p.words ? __ldg(words + i) : 0;
    const uint32_t b = i + 1 < p.words ? __ldg(words + i + 1) : 0;
    drafts = __funnelshift_r(a, b, off & 31);
  }
  return old | (drafts & below32(lim - col));
}

// ---------------------------------------------------------------- the plan
template <bool MAX>
__device__ __forceinline__ int pt_join(int a, int b) { return MAX ? max(a, b) : a + b; }
// Inclusive maxima or sums over the CTA's threads on top of `carry`, which
// becomes the last one's. `part` holds an int for each warp.
template <bool MAX>
__device__ __forceinline__ int pt_scan(int x, int* carry, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x = pt_join<MAX>(x, y);
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int before = *carry, all = *carry;
#pragma unroll 1
  for (int i = 0; i < kPtThreads / 32; ++i) {
    const int y = part[i];
    if (i < warp) before = pt_join<MAX>(before, y);
    all = pt_join<MAX>(all, y);
  }
  *carry = all;
  __syncthreads();
  return pt_join<MAX>(x, before);
}

// Pairs of query tiles, which read a key once for twice the rows, where that
// leaves an SM two items at least, or where there are few items because the keys
// are many: those are cut in any case (512 tokens behind 16384 rows, 32 + 8 heads of
// 128: 140 us, single query tiles 158; 2048 tokens alone, pairs 74 us and single
// ones 58). `rows` is the sum of the tokens' sequences' rows.
template <int D>
__device__ __forceinline__ bool pt_pairs(const PromptParams& p, int tokens, float rows) {
  const bool many = static_cast<long long>(tokens / p.TB) * p.Hkv >= 4 * gridDim.x;
  return PtShape<D>::NS == 2 && (many || rows >= static_cast<float>(tokens) * kPtDeep);
}
// Whether anything is cut: not where items are small beside what an SM gets.
__device__ __forceinline__ bool pt_worth(int top, float fair) {
  return top > kPtMinChunk && 4.0f * static_cast<float>(top) > fair;
}
// How to cut: chunks are tried from 1.1 of the fair share down to a quarter of it,
// and the one with the smallest estimate is taken. Units above half a chunk come
// in rounds, the SMs with the most of them take as many of mean size, and smaller
// units fill the others up to the fair share; then a unit's start and end, and the
// partial results' way to memory and back. (Chunks of half the share whatever the
// items: 9 sequences of up to 32768 rows, 16 + 1 heads of 256, had SMs with 117
// tiles where the mean is 84.)
__device__ __forceinline__ int pt_chunk(int no, float fair, int top) {
  return min(max(static_cast<int>(fair * kPtTopChunk * exp2f(-kPtChunkStep * no)) + 1, kPtMinChunk), top);
}
// ceil(x / c), at least 1.
__device__ __forceinline__ int pt_cuts(int x, int c) {
  int s = __float2int_rz(__fdividef(static_cast<float>(x), static_cast<float>(c)));
  s += static_cast<long long>(s) * c < x;      // the quotient is off by 1 at most
  s -= s > 0 && static_cast<long long>(s - 1) * c >= x;
  return max(s, 1);
}
struct PtTry {
  int units = 0, large = 0, big = 0, rows = 0;
  float load = 0.0f;
  __device__ __forceinline__ void add(int packed, int c) {
    const int x = packed & 0xffffff, s = pt_cuts(x, c);
    const float each = __fdividef(static_cast<float>(x), static_cast<float>(s));
    units += s;
    rows += s > 1 ? s * (packed >> 24) : 0;
    big = max(big, __float2int_ru(each));
    if (2.0f * each > static_cast<float>(c)) {
      large += s;
      load += static_cast<float>(x);
    }
  }
  __device__ __forceinline__ float estimate(float fair, int hkv) const {
    const float sms = static_cast<float>(gridDim.x), per = static_cast<float>(hkv) / sms;
    const float rounds = ceilf(static_cast<float>(large) * per - 1e-4f);
    const float most = fmaxf(__fdividef(rounds * load, static_cast<float>(max(large, 1))),
                             static_cast<float>(big));
    return fmaxf(most, fair) + (rows ? kPtJoinCost : 0.0f) +
           (kPtUnitCost * static_cast<float>(units) + kPtRowCost * static_cast<float>(rows)) * per;
  }
};
// Item k of a sequence: tokens tok .. tok + n - 1 behind c0 rows, len rows in all.
template <int D>
__device__ __forceinline__ int pt_item(const PromptParams& p, int b, int k, int TI, int tok, int n,
                                       int c0, int len, PtUnit& u) {   // its cost
  u.b = b;
  u.tok = tok + k * TI;
  u.ntok = min(TI, n - k * TI);
  u.base = p.tree_mask ? c0 : c0 + k * TI;
  u.lim = min(p.tree_mask ? c0 + n : u.base + u.ntok, len);
  u.t0 = 0;
  u.tiles = (u.lim + PtShape<D>::KEYS - 1) / PtShape<D>::KEYS;
  u.slot = -1;
  return u.tiles << (u.ntok > p.TB);
}
// A cost and the item's rows, in eights.
__device__ __forceinline__ int pt_pack(const PromptParams& p, const PtUnit& u, int cost) {
  return cost | (u.ntok * p.G + 7) / 8 << 24;
}

// The plan of a small batch, by the K warp of every CTA for itself: a lane holds a
// sequence, then an item, heaviest first. Its code runs once a call and is fetched
// cold, so it is kept short; what it saves is the way of the plan from one CTA to
// the others (13 drafts over 32768 rows, 32 + 8 heads of 128: 42 us, so 37).
template <int D>
struct PtSmallPlan {
  PtUnit u;             // this lane's item
  int cuts, upto;       // its units, and all up to it
  int units, splits, parts;

  __device__ __forceinline__ void make(const PromptParams& p) {
    const int lane = threadIdx.x & 31;
    const int cap = p.max_blocks * p.bs;
    int tok = 0, end = 0, c0 = 0, len = 0;
    if (lane < p.B) {
      tok = min(max(p.token_start[lane], 0), p.T);
      end = min(max(p.token_start[lane + 1], 0), p.T);
      c0 = p.cached_lens ? p.cached_lens[lane] : 0;
      len = p.seq_lens ? p.seq_lens[lane] : 0;
    }
    if (p.B > 1) {   // starts not below their predecessors
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, tok, o);
        if (lane >= o) tok = max(tok, y);
      }
    }
    end = max(end, tok);
    const int n = lane < p.B ? end - tok : 0;
    c0 = min(max(c0, 0), cap);
    len = min(max(p.seq_lens ? len : c0 + n, 0), cap);
    const int tokens = __reduce_add_sync(0xffffffffu, n);
    float rows = static_cast<float>(n) * static_cast<float>(len);
#pragma unroll
    for (int o = 16; o; o >>= 1) rows += __shfl_xor_sync(0xffffffffu, rows, o);
    const int TI = p.TB << pt_pairs<D>(p, tokens, rows);
    const int items = (n + TI - 1) / TI;
    const int incl = warp_incl_sum(items), total = __shfl_sync(0xffffffffu, incl, 31);
    int b = 0;
#pragma unroll 1
    for (int i = 0; i < p.B; ++i) b += __shfl_sync(0xffffffffu, incl, i) <= lane;
    const int from = b & 31, k = lane - (__shfl_sync(0xffffffffu, incl, from) - __shfl_sync(0xffffffffu, items, from));
    tok = __shfl_sync(0xffffffffu, tok, from);
    const int nb = __shfl_sync(0xffffffffu, n, from);
    c0 = __shfl_sync(0xffffffffu, c0, from);
    len = __shfl_sync(0xffffffffu, len, from);
    u.ntok = u.tiles = 0;
    int cost = 0;
    if (lane < total) cost = pt_item<D>(p, b, k, TI, tok, nb, c0, len, u);
    const int top = __reduce_max_sync(0xffffffffu, cost);
    const float fair = static_cast<float>(__reduce_add_sync(0xffffffffu, cost)) *
                       static_cast<float>(p.Hkv) / static_cast<float>(gridDim.x);
    int chunk = max(top, 1);
    if (pt_worth(top, fair)) {
      const int mine = pt_pack(p, u, cost), c = pt_chunk(min(lane, 23), fair, top);
      PtTry x;
#pragma unroll 1
      for (int i = 0; i < total; ++i) x.add(__shfl_sync(0xffffffffu, mine, i), c);
      // Estimates are positive, so their bit patterns are ordered like them.
      const unsigned est = __float_as_uint(x.estimate(fair, p.Hkv));
      const unsigned best = __reduce_min_sync(0xffffffffu, est);
      chunk = __shfl_sync(0xffffffffu, c, __ffs(__ballot_sync(0xffffffffu, est == best)) - 1);
    }
    cuts = lane < total ? pt_cuts(cost, chunk) : 0;
    if (total > 1) {   // heaviest units first: lane r takes the item of rank r
      const int each = lane < total ? cost / cuts : -1;
      int rank = 0, src = 0;
#pragma unroll 1
      for (int i = 0; i < total; ++i) {
        const int y = __shfl_sync(0xffffffffu, each, i);
        rank += y > each || (y == each && i < lane);
      }
#pragma unroll 1
      for (int i = 0; i < total; ++i) src = __shfl_sync(0xffffffffu, rank, i) == lane ? i : src;
      u.b = __shfl_sync(0xffffffffu, u.b, src);
      u.tok = __shfl_sync(0xffffffffu, u.tok, src);
      u.ntok = __shfl_sync(0xffffffffu, u.ntok, src);
      u.base = __shfl_sync(0xffffffffu, u.base, src);
      u.lim = __shfl_sync(0xffffffffu, u.lim, src);
      u.tiles = __shfl_sync(0xffffffffu, u.tiles, src);
      const int of = __shfl_sync(0xffffffffu, cuts, src);
      cuts = lane < total ? of : 0;   // other lanes have no item
    }
    upto = warp_incl_sum(cuts);
    units = __shfl_sync(0xffffffffu, upto, 31) * p.Hkv;
    const int cut = cuts > 1 ? cuts : 0, slots = warp_incl_sum(cut);
    u.slot = slots - cut;
    parts = __shfl_sync(0xffffffffu, slots, 31);
  }
  // For the joining warps: the items that were cut.
  __device__ __forceinline__ void publish(PtSplit* list, int* count) {
    const int lane = threadIdx.x & 31;
    const unsigned cut = __ballot_sync(0xffffffffu, cuts > 1);
    if (cuts > 1) list[__popc(cut & ((1u << lane) - 1u))] = {u.tok, u.ntok, u.slot, cuts};
    if (lane == 0) {
      count[0] = __popc(cut);
      count[1] = parts;
    }
  }
  // Unit rec (heads aside): words lane 0-7 of its record in each lane's return value.
  __device__ __forceinline__ int word(int rec) const {
    const int lane = threadIdx.x & 31;
    const int i = __ffs(__ballot_sync(0xffffffffu, rec < upto) | 0x80000000u) - 1;
    const int s = __shfl_sync(0xffffffffu, cuts, i);
    const int k = rec - (__shfl_sync(0xffffffffu, upto, i) - s);
    const int tiles = __shfl_sync(0xffffffffu, u.tiles, i), each = tiles / max(s, 1);
    const int more = tiles - each * s;
    const int slot = __shfl_sync(0xffffffffu, u.slot, i);
    int w = __shfl_sync(0xffffffffu, u.b, i);
    const int tok = __shfl_sync(0xffffffffu, u.tok, i), ntok = __shfl_sync(0xffffffffu, u.ntok, i);
    const int base = __shfl_sync(0xffffffffu, u.base, i), lim = __shfl_sync(0xffffffffu, u.lim, i);
    w = lane == 1 ? tok : lane == 2 ? ntok : lane == 3 ? base : lane == 4 ? lim : w;
    w = lane == 5 ? k * each + min(k, more) : lane == 6 ? each + (k < more) : w;
    return lane == 7 ? (s > 1 ? slot + k : -1) : w;
  }
};

// Made by all threads of one CTA from the lengths, in the shared memory of the
// tiles (`mem`), which nothing uses yet.
template <int D>
__device__ __noinline__ void pt_plan(const PromptParams& p, int* mem) {
  using Shape = PtShape<D>;
  const int tid = threadIdx.x;
  int* tok = mem;                      // [B + 1] first token
  int* item = tok + p.B + 1;           // [B + 1] first item
  int* cached = item + p.B + 1;        // [B]
  int* len = cached + p.B;             // [B]
  int* offs = len + p.B;               // [kPtBuckets]
  int* part = offs + kPtBuckets;       // [12]
  unsigned long long* work = reinterpret_cast<unsigned long long*>(
      (reinterpret_cast<uintptr_t>(part + kPtThreads / 32) + 7) & ~static_cast<uintptr_t>(7));
  unsigned long long* best = work + 1;   // estimate and chunk
  int* most = reinterpret_cast<int*>(work + 3);   // work[2]: tokens times rows
  int* n_slots = most + 1;
  int* n_splits = most + 2;
  int* costs = most + 3;               // [kPtCosts] of the first items
  if (tid == 0) {
    *work = 0;
    *best = ~0ull;
    work[2] = 0;
    *most = *n_slots = *n_splits = 0;
  }
  for (int i = tid; i < kPtBuckets; i += kPtThreads) offs[i] = 0;
  const int cap = p.max_blocks * p.bs;

  // Starts within the tokens and not below their predecessors.
  int carry = 0;
  for (int b0 = 0; b0 <= p.B; b0 += kPtThreads) {
    const int b = b0 + tid;
    const int x = b <= p.B ? min(max(p.token_start[b], 0), p.T) : 0;
    const int s = pt_scan<true>(x, &carry, part);
    if (b <= p.B) tok[b] = s;
  }
  __syncthreads();
  unsigned long long sum = 0;
  for (int b = tid; b < p.B; b += kPtThreads) {
    const int n = tok[b + 1] - tok[b];
    const int c0 = p.cached_lens ? min(max(p.cached_lens[b], 0), cap) : 0;
    cached[b] = c0;
    len[b] = p.seq_lens ? min(max(p.seq_lens[b], 0), cap) : min(c0 + n, cap);
    sum += static_cast<unsigned long long>(n) * len[b];
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) atomicAdd(work + 2, sum);
  __syncthreads();
  const int pairs = pt_pairs<D>(p, tok[p.B] - tok[0], static_cast<float>(work[2]));
  const int TI = p.TB << pairs;
  carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPtThreads) {
    const int b = b0 + tid;
    const int items = b < p.B ? (tok[b + 1] - tok[b] + TI - 1) / TI : 0;
    const int upto = pt_scan<false>(items, &carry, part);
    if (b < p.B) item[b] = upto - items;
  }
  if (tid == 0) item[p.B] = carry;
  __syncthreads();
  const int n_items = carry;

  auto find = [&](int i, PtUnit& u) {   // the whole item; returns its cost
    int lo = 0, hi = p.B;               // the last sequence with item[b] <= i
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (item[mid] <= i) lo = mid;
      else hi = mid;
    }
    const int k = i - item[lo];
    return pt_item<D>(p, lo, k, TI, tok[lo], tok[lo + 1] - tok[lo], cached[lo], len[lo], u);
  };
  // Work, in key tiles times query tiles.
  sum = 0;
  int top = 0;
  PtUnit u;
  for (int i = tid; i < n_items; i += kPtThreads) {
    const int c = find(i, u);
    if (i < kPtCosts) costs[i] = pt_pack(p, u, c);
    sum += c;
    top = max(top, c);
  }
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  top = __reduce_max_sync(0xffffffffu, top);
  if ((tid & 31) == 0) {
    atomicAdd(work, sum);
    atomicMax(most, top);
  }
  __syncthreads();
  auto packed = [&](int i) {
    if (i < kPtCosts) return costs[i];
    const int c = find(i, u);
    return pt_pack(p, u, c);
  };
  auto cost = [&](int i) { return packed(i) & 0xffffff; };
  top = *most;
  const float fair = static_cast<float>(*work) * static_cast<float>(p.Hkv) /
                     static_cast<float>(gridDim.x);   // of an SM
  int chunk = max(top, 1);
  if (pt_worth(top, fair)) {
    for (int k = 0; k < 2; ++k) {   // two chunks a warp
      const int c = pt_chunk(2 * (tid >> 5) + k, fair, top);
      PtTry x;
      for (int i = tid & 31; i < n_items; i += 32) x.add(packed(i), c);
      x.units = __reduce_add_sync(0xffffffffu, x.units);
      x.large = __reduce_add_sync(0xffffffffu, x.large);
      x.big = __reduce_max_sync(0xffffffffu, x.big);
      x.rows = __reduce_add_sync(0xffffffffu, x.rows);
      for (int o = 16; o; o >>= 1) x.load += __shfl_xor_sync(0xffffffffu, x.load, o);
      // Estimates are positive, so their bit patterns are ordered like them.
      if ((tid & 31) == 0)
        atomicMin(best, static_cast<unsigned long long>(__float_as_uint(x.estimate(fair, p.Hkv))) << 32 |
                            static_cast<unsigned>(c));
    }
    __syncthreads();
    chunk = static_cast<int>(*best & 0xffffffffu);
  }
  const int max_unit = max(1, min(top, chunk));
  auto cuts = [&](int c) { return pt_cuts(c, chunk); };
  auto bucket = [&](int c, int s) {     // heaviest first
    const int each = (c + s - 1) / s;
    return kPtBuckets - 1 -
           static_cast<int>(static_cast<long long>(min(each, max_unit)) * (kPtBuckets - 1) / max_unit);
  };
  for (int i = tid; i < n_items; i += kPtThreads) {
    const int c = cost(i), s = cuts(c);
    atomicAdd(&offs[bucket(c, s)], s);
  }
  __syncthreads();
  carry = 0;
  {
    const int n = tid < kPtBuckets ? offs[tid] : 0;
    const int upto = pt_scan<false>(n, &carry, part);
    if (tid < kPtBuckets) offs[tid] = upto - n;
  }
  __syncthreads();
  for (int i = tid; i < n_items; i += kPtThreads) {
    const int s = cuts(find(i, u));   // at most the tiles
    const int at = atomicAdd(&offs[bucket(cost(i), s)], s);
    if (s > 1) {
      u.slot = atomicAdd(n_slots, s);
      p.splits[atomicAdd(n_splits, 1)] = {u.tok, u.ntok, u.slot, s};
    }
    const int tiles = u.tiles, each = tiles / s, more = tiles - each * s;
    for (int k = 0; k < s; ++k) {
      u.tiles = each + (k < more);
      p.units[at + k] = u;
      u.t0 += u.tiles;
      u.slot += s > 1;
    }
  }
  __syncthreads();
  if (tid == 0) {
    p.head->units = carry * p.Hkv;
    p.head->splits = *n_splits;
    p.head->parts = *n_slots;
  }
}

// Whether 8 values of a 16-bit type have one that is not finite.
template <typename Tag>
__device__ __forceinline__ uint32_t pt_odd(uint32_t x) {   // the top bit of each such half
  constexpr uint32_t e = std::is_same<Tag, Bf16Tag>::value ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t one = std::is_same<Tag, Bf16Tag>::value ? 0x00800080u : 0x04000400u;
  return ((x & e) + one) & 0x80008000u;
}
template <typename Tag>
__device__ __forceinline__ float pt_widen(uint32_t half) {
  if constexpr (std::is_same<Tag, Bf16Tag>::value) return __uint_as_float(half << 16);
  else return __half2float(__ushort_as_half(static_cast<unsigned short>(half)));
}

template <typename Tag, int D>
__global__ void __launch_bounds__(kPtThreads, 1)
    gqa_prompt_kernel(const __grid_constant__ PromptParams p) {
  using Shape = PtShape<D>;
  constexpr int NS = Shape::NS, KEYS = Shape::KEYS, PARTS = Shape::PARTS;
  constexpr int KST = Shape::KST, VST = Shape::VST;
  // fp16 weights are scaled by 2^6 (at most 2^14 with the growth allowance), so
  // that small ones keep their bits; the sum carries the same factor.
  constexpr float kOff = std::is_same<Tag, Fp16Tag>::value ? 6.0f : 0.0f;
  constexpr float kMostSum = std::is_same<Tag, Fp16Tag>::value ? 256.0f * 64.0f : 256.0f;
  extern __shared__ __align__(1024) uint8_t pt_smem[];
  uint8_t* smem = pt_smem;
  const uint32_t base_s = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::TILES_BYTES);
  const uint32_t kfull0 = smem_addr(bars), kempty0 = kfull0 + 8 * KST;
  const uint32_t vfull0 = kempty0 + 8 * KST, vempty0 = vfull0 + 8 * VST;
  const uint32_t qfull0 = vempty0 + 8 * VST, qempty0 = qfull0 + 16;
  const uint32_t sfull0 = qempty0 + 16, pfull0 = sfull0 + 16;   // a stream's, or an S buffer's
  const uint32_t ofull0 = pfull0 + 16, ofree0 = ofull0 + 16, pvdone = ofree0 + 16;
  const uint32_t meet = pvdone + 8, drain = meet + 8, clean0 = drain + 8;
  const uint32_t issued0 = clean0 + 8 * kPtCleans;
  const uint32_t tfull = issued0 + 8 * kPtCleans, tfree = tfull + 8;   // queries in tensor memory
  const uint32_t ufull0 = tfree + 8, uempty0 = ufull0 + 8 * kPtSegs;
  constexpr int kBars = 2 * (KST + VST) + 17 + 2 * kPtCleans + 2 * kPtSegs;
  struct Seg {
    PtUnit u;
    int kv;
  };
  Seg* segs = reinterpret_cast<Seg*>(bars + ((kBars + 1) & ~1));
  // Read 16 bytes at a time: behind records of multiples of 16.
  PtSplit* cut_list = reinterpret_cast<PtSplit*>(segs + kPtSegs);   // [kPtSmall] of a small batch
  int* odd = reinterpret_cast<int*>(cut_list + kPtSmall);   // [4] unit's V held values that are not finite
  int* cut_count = odd + 4;            // items of cut_list, and their slots
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(cut_count + 2);
  unsigned* ticket = tmem_slot + 1;
  float2* ml = reinterpret_cast<float2*>(smem + Shape::TILES_BYTES + Shape::MISC);   // [2][128]
  static_assert(8 * ((kBars + 1) & ~1) + sizeof(Seg) * kPtSegs + 32 + sizeof(PtSplit) * kPtSmall <= Shape::MISC,
                "shared memory besides the tiles");
  static_assert(Shape::TILES_BYTES % 16 == 0 && sizeof(Seg) % 16 == 0 && sizeof(PtSplit) == 16 &&
                    alignof(PtSplit) == 16,
                "16-byte records");
  static_assert(kPtCleans > VST && 16 * (kPtMaxB + 1) + 4 * (kPtBuckets + kPtCosts) + 128 <= Shape::TILES_BYTES,
                "barriers of cleared tiles; the plan's memory");

  if (warp == kPtMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2 * (KST + VST); ++i) mbar_init(kfull0 + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(qfull0 + 8 * i, 1);
      mbar_init(qempty0 + 8 * i, NS == 1 ? 4 : 1);
      mbar_init(sfull0 + 8 * i, 1);
      mbar_init(pfull0 + 8 * i, 4);
      mbar_init(ofull0 + 8 * i, 1);
      mbar_init(ofree0 + 8 * i, 8);
    }
    mbar_init(pvdone, 1);
    mbar_init(tfull, 4);
    mbar_init(tfree, 1);
    mbar_init(meet, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < 2 * kPtCleans; ++i) mbar_init(clean0 + 8 * i, 1);   // and issued0
    for (int i = 0; i < kPtSegs; ++i) {
      mbar_init(ufull0 + 8 * i, 1);
      mbar_init(uempty0 + 8 * i, 11);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPtKWarp && lane < 3) {
    const CUtensorMap* m = lane == 0 ? &p.k_map : lane == 1 ? &p.v_map : &p.q_map;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (threadIdx.x == 0 && blockIdx.x >= p.late_from) {
    const uint64_t since = global_timer_ns();
    while (static_cast<long long>(global_timer_ns() - since) < p.late_ns) __nanosleep(1000);
  }
  if (threadIdx.x == 0) *ticket = p.small ? 1u : atomicAdd(&p.head->ticket, 1u);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*ticket == 0) {
    pt_plan<D>(p, reinterpret_cast<int*>(smem));
    // The plan's shared memory is the copies' from here on.
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) atomicExch(&p.head->ready, 1u);
  }
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t qbuf_s = base_s, k_s = base_s + Shape::QBUF * Shape::QBYTES;
  const uint32_t v_s = k_s + KST * Shape::STAGE;
  const bool aligned = (base_s & 1023u) == 0;   // the tiles need it; dynamic memory starts so
  if (!aligned && threadIdx.x == 0) atomicOr(&pt_status, kErrPtLoad);

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPtAuxRegs));
    if (aligned && (warp == kPtKWarp || warp == kPtVWarp)) {
      // ---------------------------------------- units, queries and K, or V
      const bool is_k = warp == kPtKWarp;
      const uint32_t leader = elect_one();
      const uint64_t policy = evict_first_policy();
      const int nch = KEYS / p.R;              // boxes of one 64-column part of a tile
      const int oob = p.num_blocks * p.bs;
      const int stages = is_k ? KST : VST;
      const uint32_t full0 = is_k ? kfull0 : vfull0, empty0 = is_k ? kempty0 : vempty0;
      const uint32_t ring_s = is_k ? k_s : v_s;
      int stage = 0;
      uint32_t parity = 0;                     // of the stage's next fill
      unsigned fills = 0, cleans = 0;
      // Lane s: 1 + parity of this warp's last copy into stage s (0: none yet);
      // lane 16 + s: into query buffer s.
      unsigned held = 0;
      bool ok = true;
      int next = 0, total = 0;
      PtSmallPlan<D> plan;
      // The first unit is claimed like the others, while the plan is made.
      if (is_k && lane == 0) next = atomicAdd(&p.head->next, 1u);
      if (is_k && p.small) {
        plan.make(p);
        plan.publish(cut_list, cut_count);
        total = plan.units;
      } else if (is_k) {
        // The plan is ready when its maker says so.
        const uint64_t since = global_timer_ns();
        while (ok && !*reinterpret_cast<volatile unsigned*>(&p.head->ready))
          ok = static_cast<long long>(global_timer_ns() - since) < p.timeout_ns;
        ok = __all_sync(0xffffffffu, ok);
        __threadfence();
        total = __ldcg(&p.head->units);
        if (!ok && lane == 0) atomicOr(&pt_status, kErrPtPlan);
      }
      next = __shfl_sync(0xffffffffu, next, 0);
      for (unsigned unit_no = 0; ok; ++unit_no) {
        const int seg = unit_no % kPtSegs;
        Seg& s = segs[seg];
        if (is_k) {
          // The record by eight lanes; heads are innermost.
          const int rec = next / p.Hkv;
          int word = 0;
          if (p.small) word = next < total ? plan.word(rec) : 0;
          else if (next < total && lane < 8) word = __ldcg(reinterpret_cast<const int*>(p.units + rec) + lane);
          if (!(ok = warp_poll(uempty0 + 8 * seg, ((unit_no / kPtSegs) & 1) ^ 1, p.timeout_ns))) break;
          if (lane < 8) reinterpret_cast<int*>(&s.u)[lane] = word;
          if (lane == 8) s.kv = next - rec * p.Hkv;
          __syncwarp();
          if (lane == 0) mbar_arrive(ufull0 + 8 * seg);
        } else {
          if (!(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPtSegs) & 1, p.timeout_ns))) break;
        }
        const PtUnit u = s.u;
        const int kv = uniform(s.kv);
        __syncwarp();
        if (!is_k && lane == 0) mbar_arrive(uempty0 + 8 * seg);
        if (u.ntok == 0) break;
        int claim = 0;
        const int n = uniform(u.tiles);
        // The next unit is taken late, so that who is ahead takes more (at the head of
        // the current one: trees of 64 sequences of 1 to 8192 rows end 25 us apart).
        const int claim_at = max(n - 2, 0);
        if (is_k && lane == 0 && n == 0) claim = atomicAdd(&p.head->next, 1u);
        const int32_t* table = p.block_table + static_cast<size_t>(u.b) * p.max_blocks;
        // The pool row of this lane's box of tile i; rows past the last visible
        // one and entries outside the pool read zeros.
        auto row_of = [&](int i) {
          const int c = (u.t0 + i) * KEYS + lane * p.R;
          if (lane >= nch || i >= n || c >= u.lim) return oob;
          const int col = pt_block_of(p, c);
          const int block = table[col];
          return block >= 0 && block < p.num_blocks ? block * p.bs + (c - col * p.bs) : oob;
        };
        int row = row_of(0);
        if (is_k && n > 0) {
          const int pair = NS == 2 && u.ntok > p.TB;
          for (int i = 0; i <= pair && ok; ++i, ++fills) {
            const int buf = fills % Shape::QBUF;
            ok = warp_poll(qempty0 + 8 * buf, ((fills / Shape::QBUF) & 1) ^ 1, p.timeout_ns);
            if (!ok) break;
            if (fills >= p.withhold_from) continue;
            const uint32_t bar = qfull0 + 8 * buf;
            if (lane == 16 + buf) held = 1 + ((fills / Shape::QBUF) & 1);
            expect_one(leader, bar, p.TB * p.G * 128 * PARTS);
            const int q0 = uniform(u.tok) + i * p.TB;
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              tma_one_4d(leader, qbuf_s + buf * Shape::QBYTES + part * 128 * 128, &p.q_map,
                         64 * part, 0, kv, q0, bar, policy);
          }
        }
        const CUtensorMap* map = is_k ? &p.k_map : &p.v_map;
        const int first_clean = uniform(pt_share<D>(p, u).full) / KEYS - uniform(u.t0);
        for (int i = 0; i < n && ok; ++i) {
          if (is_k && lane == 0 && i == claim_at) claim = atomicAdd(&p.head->next, 1u);
          const int ahead = row_of(i + 1);
          if (!(ok = warp_poll(empty0 + 8 * stage, parity ^ 1, p.timeout_ns))) break;
          const uint32_t bar = full0 + 8 * stage, dst = ring_s + stage * Shape::STAGE;
          expect_one(leader, bar, Shape::STAGE);
          if (lane == stage) held = 1 + parity;
          for (int c = 0; c < nch; ++c) {
            const int r = __shfl_sync(0xffffffffu, row, c);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              tma_one_3d(leader, dst + part * KEYS * 128 + c * p.R * 128, map, 64 * part, kv, r, bar,
                         policy);
          }
          // The clearing warp may wait for this fill of the stage from now on: its
          // phase is the current one until the tile has been cleared and used.
          if (!is_k && i >= first_clean) {
            __syncwarp();
            if (lane == 0) mbar_arrive(issued0 + 8 * (cleans % kPtCleans));
            ++cleans;
          }
          if (++stage == stages) stage = 0, parity ^= 1;
          row = ahead;
        }
        if (is_k) next = __shfl_sync(0xffffffffu, claim, 0);
      }
      if (!ok) {
        // This warp's copies in flight land before the CTA leaves.
        if (lane == 0) atomicOr(&pt_status, kErrPtLoad);
        if (held && lane < stages) mbar_wait(full0 + 8 * lane, held - 1, kPtTimeoutNs);
        if (held && lane >= 16) mbar_wait(qfull0 + 8 * (lane - 16), held - 1, kPtTimeoutNs);
        __syncwarp();
      }
    } else if (aligned && warp == kPtCleanWarp) {
      // ------------------------------------------------------ V's masked rows
      unsigned tiles = 0, cleans = 0;          // V tiles before the unit's
      bool ok = true;
      for (unsigned unit_no = 0; ok; ++unit_no) {
        const int seg = unit_no % kPtSegs;
        if (!(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPtSegs) & 1, p.timeout_ns))) break;
        const PtUnit u = segs[seg].u;
        __syncwarp();
        // Nobody looks at this entry: the softmax warps are at most two units behind.
        if (lane == 0) {
          odd[unit_no & 3] = 0;
          mbar_arrive(uempty0 + 8 * seg);
        }
        if (u.ntok == 0) break;
        const PtShare sh = pt_share<D>(p, u);
        const int n = u.tiles;
        for (int i = max(0, sh.full / KEYS - u.t0); i < n; ++i, ++cleans) {
          const unsigned stage = (tiles + i) % VST;
          ok = warp_poll(issued0 + 8 * (cleans % kPtCleans), (cleans / kPtCleans) & 1, p.timeout_ns) &&
               warp_poll(vfull0 + 8 * stage, (tiles + i) / VST & 1, p.timeout_ns);
          if (!ok) break;
          uint8_t* v = smem + (v_s - base_s) + stage * Shape::STAGE;
          const int c0 = (u.t0 + i) * KEYS;
          const int from = max(0, sh.full - c0), to = min(KEYS, u.lim - c0);   // masked for some
          bool wrote = false;
#pragma unroll 1
          for (int part = 0; part < PARTS; ++part) {
            uint4* rows = reinterpret_cast<uint4*>(v + part * KEYS * 128);
            uint32_t any = 0;
#pragma unroll 8
            for (int t = from * 8 + lane; t < to * 8; t += 32) {
              const uint4 x = rows[t];
              any |= pt_odd<Tag>(x.x) | pt_odd<Tag>(x.y) | pt_odd<Tag>(x.z) | pt_odd<Tag>(x.w);
            }
            if (__any_sync(0xffffffffu, any)) {
              wrote = true;
              uint16_t* half = reinterpret_cast<uint16_t*>(rows);
#pragma unroll 1
              for (int t = from * 64 + lane; t < to * 64; t += 32)
                if (pt_odd<Tag>(half[t])) half[t] = 0;
              if (lane == 0) odd[unit_no & 3] = 1;
            }
#pragma unroll 1
            for (int t = max(0, to) * 8 + lane; t < KEYS * 8; t += 32) {
              rows[t] = make_uint4(0u, 0u, 0u, 0u);
              wrote = true;
            }
          }
          if (wrote) asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(clean0 + 8 * (cleans % kPtCleans));
        }
        tiles += n;
      }
      if (!ok && lane == 0) atomicOr(&pt_status, kErrPtClean);
      __syncwarp();
    } else if (aligned && warp == kPtMmaWarp) {
      // ---------------------------------------------------------- MMA issue
      const uint32_t leader = elect_one();
      constexpr uint32_t qk_idesc = px_idesc<Tag>(KEYS, false), pv_idesc = px_idesc<Tag>(D, true);
      // Everything here runs in uniform registers: counters that step and wrap,
      // no division, no value out of shared memory that the warp has not agreed on.
      // (With ring positions taken modulo the stages, the code around the products
      // took longer than they did.)
      const uint64_t q_desc = smem_desc(qbuf_s, 16, 1024, 2), k_desc = smem_desc(k_s, 16, 1024, 2);
      const uint64_t v_desc = smem_desc(v_s, KEYS * 128, 1024, 2);
      int kst = 0, vst = 0;                          // stages, and the parity of their fills
      uint32_t kpar = 0, vpar = 0;
      uint32_t ppar0 = 0, ppar1 = 0;                 // of the streams' weights (or S buffers')
      int fills = 0, cleans = 0, sbuf = 0;           // one stream: the S buffer of the next scores
      // The softmax warps have run through their code once (below).
      bool ok = warp_poll(ofree0, 0, p.timeout_ns) && warp_poll(ofree0 + 8, 0, p.timeout_ns);
      for (unsigned unit_no = 0; ok; ++unit_no) {
        const int seg = unit_no % kPtSegs;
        if (!(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPtSegs) & 1, p.timeout_ns))) break;
        const PtUnit u = segs[seg].u;
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty0 + 8 * seg);
        if (u.ntok == 0) break;
        const PtShare sh = pt_share<D>(p, u);
        const int pair = uniform(sh.pair);
        const int n0 = uniform(sh.n0), n1 = uniform(sh.n1), n = uniform(u.tiles);
        const int first_clean = uniform(max(0, sh.full / KEYS - u.t0));
        // Waits of the scores' product, which come before those of the PV that goes
        // first: each takes its time even when it is over.
        auto await_k = [&](int w, int j) {
          const int fill = fills + (pair ? w : 0);
          if (j == 0)
            ok = ok && (NS == 2 ? warp_poll(qfull0 + 8 * (fill & 1), fill >> 1 & 1, p.timeout_ns)
                                : warp_poll(tfull, fill & 1, p.timeout_ns));
          if (pair && w && j < n0) return;           // the first stream's, too
          ok = ok && warp_poll(kfull0 + 8 * kst, kpar, p.timeout_ns);
        };
        auto qk = [&](int w, int j, int s_no) {
          if (!ok) return;
          const int fill = fills + (pair ? w : 0), buf = NS == 2 ? fill & 1 : 0;
          tc_fence_after();
          const uint64_t a = q_desc + static_cast<uint64_t>(buf * (Shape::QBYTES >> 4));
          const uint64_t b = k_desc + static_cast<uint64_t>(kst * (Shape::STAGE >> 4));
          const uint32_t s_tmem = tmem + Shape::S_COL * s_no;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint64_t b_kk = b + (uint64_t)((kk / 4 * KEYS * 128 + kk % 4 * 32) >> 4);
            if (NS == 1)
              mma_ts(leader, s_tmem, tmem + Shape::Q_COL + 8 * kk, b_kk, qk_idesc, kk > 0);
            else
              mma_ss(leader, s_tmem, a + (uint64_t)((kk / 4 * 128 * 128 + kk % 4 * 32) >> 4), b_kk,
                     qk_idesc, kk > 0);
          }
          commit_one(leader, sfull0 + 8 * s_no);
          // A pair's second stream is the last to use a stage: it has the more tiles.
          if (!pair || w) {
            commit_one(leader, kempty0 + 8 * kst);
            if (++kst == KST) kst = 0, kpar ^= 1;
          }
          if (pair ? j == (w ? n1 : n0) - 1 : (NS == 2 ? 2 * j + w : j) == n - 1)
            commit_one(leader, NS == 2 ? qempty0 + 8 * buf : tfree);
        };
        auto pv = [&](int w, int j, int s_no) {
          const int i = NS == 1 || pair ? j : 2 * j + w;
          if (j == 0) ok = ok && warp_poll(ofree0 + 8 * w, unit_no & 1, p.timeout_ns);
          if (!(pair && w && j < n0)) {
            ok = ok && warp_poll(vfull0 + 8 * vst, vpar, p.timeout_ns);
            if (i >= first_clean) {
              const int c = cleans + i - first_clean;
              ok = ok && warp_poll(clean0 + 8 * (c % kPtCleans), c / kPtCleans & 1, p.timeout_ns);
            }
          }
          ok = ok && warp_poll(pfull0 + 8 * s_no, s_no ? ppar1 : ppar0, p.timeout_ns);
          if (s_no) ppar1 ^= 1;
          else ppar0 ^= 1;
          if (!ok) return;
          tc_fence_after();
          const uint64_t b = v_desc + static_cast<uint64_t>(vst * (Shape::STAGE >> 4));
          const uint32_t p_tmem = tmem + Shape::S_COL * s_no, o_tmem = tmem + Shape::O_COL0 + w * D;
#pragma unroll
          for (int kk = 0; kk < KEYS / 16; ++kk)
            mma_ts(leader, o_tmem, p_tmem + 8 * kk, b + (uint64_t)(kk * (2048 >> 4)), pv_idesc,
                   j > 0 || kk > 0);
          if (!pair || w) {
            commit_one(leader, vempty0 + 8 * vst);
            if (++vst == VST) vst = 0, vpar ^= 1;
          }
          if (NS == 1) commit_one(leader, pvdone);
          if (j == (w ? n1 : n0) - 1) commit_one(leader, ofull0 + 8 * w);
        };
        // A pair's tiles j = 1 .. rounds - 1: for each stream PV of tile j, then QK of tile
        // j + 1. None is a unit's first or last, or masked, so there is less to look at
        // between the products (a prompt of 16384 tokens: 1440 us without, 1354 with).
        auto middle = [&](int rounds) {
          const int buf0 = fills & 1, buf1 = buf0 ^ 1;
#pragma unroll 1
          for (int j = 1; j < rounds && ok; ++j) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              if (w == 0)
                ok = ok && warp_poll(kfull0 + 8 * kst, kpar, p.timeout_ns) &&
                     warp_poll(vfull0 + 8 * vst, vpar, p.timeout_ns);
              ok = ok && warp_poll(pfull0 + 8 * w, w ? ppar1 : ppar0, p.timeout_ns);
              if (w) ppar1 ^= 1;
              else ppar0 ^= 1;
              if (!ok) break;
              tc_fence_after();
              const uint64_t v = v_desc + static_cast<uint64_t>(vst * (Shape::STAGE >> 4));
              const uint32_t s_tmem = tmem + Shape::S_COL * w, o_tmem = tmem + Shape::O_COL0 + w * D;
#pragma unroll
              for (int kk = 0; kk < KEYS / 16; ++kk)
                mma_ts(leader, o_tmem, s_tmem + 8 * kk, v + (uint64_t)(kk * (2048 >> 4)), pv_idesc, 1);
              const uint64_t a = q_desc + static_cast<uint64_t>((w ? buf1 : buf0) * (Shape::QBYTES >> 4));
              const uint64_t k = k_desc + static_cast<uint64_t>(kst * (Shape::STAGE >> 4));
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk)
                mma_ss(leader, s_tmem, a + (uint64_t)((kk / 4 * 128 * 128 + kk % 4 * 32) >> 4),
                       k + (uint64_t)((kk / 4 * KEYS * 128 + kk % 4 * 32) >> 4), qk_idesc, kk > 0);
              commit_one(leader, sfull0 + 8 * w);
              if (w) {   // the second stream is the last to use a stage
                commit_one(leader, vempty0 + 8 * vst);
                commit_one(leader, kempty0 + 8 * kst);
                if (++kst == KST) kst = 0, kpar ^= 1;
                if (++vst == VST) vst = 0, vpar ^= 1;
              }
            }
          }
        };
        // Every unit's phase of both ofree barriers is waited for, here or by pv.
        if (n0 == 0) ok = warp_poll(ofree0, unit_no & 1, p.timeout_ns);
        if (NS == 2 && n1 == 0) ok = ok && warp_poll(ofree0 + 8, unit_no & 1, p.timeout_ns);
        if constexpr (NS == 1) {
#pragma unroll 1
          for (int j = -1; j < n && ok; ++j) {
            if (j + 1 < n) {
              await_k(0, j + 1);
              qk(0, j + 1, sbuf);
            }
            if (j >= 0) pv(0, j, sbuf ^ 1);
            sbuf ^= 1;
          }
          sbuf ^= 1;   // n scores, n + 1 steps
        } else {
          // The streams in turn: the PV of a tile, then the QK of the next.
          int t = -2;
          const int end = 2 * max(n0, n1);
#pragma unroll 1
          for (int part = 0; part < 2 && ok; ++part) {
            const int stop = part ? end : min(end, 2);
#pragma unroll 1
            for (; t < stop && ok; ++t) {
              const int w = t & 1, j = t >> 1, cnt = w ? n1 : n0;
              if (j + 1 < cnt) await_k(w, j + 1);
              if (j >= 0 && j < cnt) pv(w, j, w);
              if (j + 1 < cnt) qk(w, j + 1, w);
            }
            if (part == 0 && ok) {
              const int rounds = pair ? min(n0 - 2, first_clean) : 0;
              if (rounds > 2) {
                middle(rounds);
                t = 2 * rounds;
              }
            }
          }
        }
        fills += n > 0 ? 1 + pair : 0;
        cleans += max(0, n - first_clean);
      }
      if (!ok) {
        if (lane == 0) atomicOr(&pt_status, kErrPtMma);
        commit_one(leader, drain);
        mbar_wait(drain, 0, kPtTimeoutNs);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPtSoftmaxRegs));
    // ------------------------------------------------- softmax, units' ends
    const int w = warp >> 2;                  // stream
    const int r = threadIdx.x & 127;          // tensor-memory lane
    const uint32_t lane_addr = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    unsigned done = 0, ends0 = 0, ends1 = 0, meets = 0, copies = 0;
    bool ok = aligned;
    // Rows of a query tile are token after token, a token's heads together.
    const int x = r / p.G, g = r - x * p.G;
    // The first round takes no unit: one key tile of whatever lies in S and a
    // unit's end without rows, run through while the plan is made, so that the
    // instructions are in the caches when the first scores arrive. Its weights go to S, which no product
    // has written yet: the MMA warp waits for all warps' ofree of this round
    // before its first one.
    for (unsigned round = 0; ok; ++round) {
      const bool dry = round == 0;
      const unsigned unit_no = round - 1;
      const int seg = unit_no % kPtSegs;
      if (!dry && !(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPtSegs) & 1, p.timeout_ns))) break;
      PtUnit u = {0, 0, 2 * p.TB, 1 << 26, 1 << 26, 0, 1, -1};
      int kv = 0;
      if (!dry) {
        u = segs[seg].u;
        kv = segs[seg].kv;
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty0 + 8 * seg);
        if (u.ntok == 0) break;
      }
      const PtShare sh = pt_share<D>(p, u);
      const int n0 = sh.n0, n1 = sh.n1;
      const int mine = w ? n1 : n0;
      const int tx = x + (sh.pair ? w * p.TB : 0);    // this row's token of the unit
      const bool live = x < p.TB && tx < u.ntok && !dry;
      // Warps without rows only keep step.
      const bool active = dry || __any_sync(0xffffffffu, live);
      // Tiles from here on hold keys that some row of this query tile must not see.
      const int seen = !p.tree_mask && sh.pair && w ? min(u.base + p.TB + 1, u.lim) : sh.full;
      if (NS == 1 && w == 1 && u.tiles > 0 && !dry) {
        // Queries from shared to tensor memory, once the last unit's scores are made.
        // A row's 16-byte pieces lie where the swizzle has put them.
        ok = warp_poll(qfull0, copies & 1, p.timeout_ns) &&
             warp_poll(tfree, (copies & 1) ^ 1, p.timeout_ns);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < PARTS; ++part) {
          uint32_t q[32];
          const uint4* src = reinterpret_cast<const uint4*>(smem + part * 128 * 128 + r * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint4 x = src[c ^ (r & 7)];
            q[4 * c] = x.x; q[4 * c + 1] = x.y; q[4 * c + 2] = x.z; q[4 * c + 3] = x.w;
          }
          tmem_st32(tmem + lane_addr + Shape::Q_COL + 32 * part, q);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tfull);
          mbar_arrive(qempty0);
        }
        ++copies;
      }
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < mine; ++j) {
        const unsigned no = done + j;
        const int sb = NS == 2 ? w : no & 1;
        if (!dry && !(ok = warp_poll(sfull0 + 8 * sb, (NS == 2 ? no : no >> 1) & 1, p.timeout_ns)))
          break;
        tc_fence_after();
        const int c_first = (u.t0 + (NS == 1 || sh.pair ? j : 2 * j + w)) * KEYS;
        if (active) {
          const uint32_t s_addr = tmem + lane_addr + Shape::S_COL * sb;
          const bool masked = c_first + KEYS > seen || p.negate || dry;
          const bool tried = j > 0 && !masked;
          bool done_with = false;
          if (tried) {
            // One pass over the scores, 64 at a time; the weights go back to tensor
            // memory once their sums are known to be small. (A pass that found the
            // maximum too was no faster than one for it and one for the weights.)
            const float shift = kOff - m, qscale = p.qscale;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            uint32_t w16[KEYS / 2];
            float s[64];
#pragma unroll
            for (int c0 = 0; c0 < KEYS; c0 += 64) {
              tmem_ld32(s_addr + c0, s);
              tmem_ld32(s_addr + c0 + 32, s + 32);
              tmem_wait_ld();
              hold<64>(s);
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                float a, b;
                fma2(s[c], s[c + 1], qscale, qscale, shift, shift, a, b);
                a = ex2(a);
                b = ex2(b);
                add2(sum[c & 2], sum[(c & 2) + 1], a, b);
                w16[(c0 + c) / 2] = pack2<Tag>(a, b);
              }
            }
            const float all = (sum[0] + sum[1]) + (sum[2] + sum[3]);
            done_with = !__any_sync(0xffffffffu, live && !(all < kMostSum));
            if (done_with) {
#pragma unroll
              for (int c0 = 0; c0 < KEYS / 2; c0 += 32) tmem_st32(s_addr + c0, w16 + c0);
              l += all;
            }
          }
          if (!done_with) {
            // Sums that were too large move the maximum however little it has grown.
            const float grow = tried ? 0.0f : kPtGrow;
            if (masked) {
              // Masked keys, and a negative scale, in S itself.
#pragma unroll 1
              for (int c0 = 0; c0 < KEYS; c0 += 32) {
                const uint32_t sees =
                    live ? pt_sees(p, u.tok, u.base, u.lim, tx, c_first + c0) : 0u;
                float s[32];
                tmem_ld32(s_addr + c0, s);
                tmem_wait_ld();
                hold<32>(s);
#pragma unroll
                for (int c = 0; c < 32; ++c)
                  s[c] = (sees >> c) & 1u ? (p.negate ? -s[c] : s[c]) : -INFINITY;
                tmem_st32(s_addr + c0, reinterpret_cast<const uint32_t*>(s));
              }
              tmem_wait_st();
            }
            float s[KEYS];
#pragma unroll
            for (int c0 = 0; c0 < KEYS; c0 += 32) tmem_ld32(s_addr + c0, s + c0);
            tmem_wait_ld();
            hold<KEYS>(s);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < KEYS; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
            if (j == 0) {
              m = top == -INFINITY ? -1e30f : top;   // nothing finite yet: weights of 0
            } else if (__any_sync(0xffffffffu, live && top > m + grow)) {
              // Each row by itself: lanes without a row hold anything, and must
              // not move the others' maxima.
              // The previous tiles' products are done: S of this tile was
              // multiplied after them, or (one stream) the wait below.
              if (NS == 1) {
                if (!(ok = warp_poll(pvdone, (no - 1) & 1, p.timeout_ns))) break;
                tc_fence_after();
              }
              const float now = top > m + grow ? top : m, a = ex2(m - now);
              m = now;
              l *= a;
              const uint32_t o_addr = tmem + lane_addr + Shape::O_COL0 + w * D;
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                float o[32];
                tmem_ld32(o_addr + c, o);
                tmem_wait_ld();
                hold<32>(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] *= a;
                tmem_st32(o_addr + c, reinterpret_cast<const uint32_t*>(o));
              }
            }
            const float shift = kOff - m, qscale = p.qscale;
            float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c0 = 0; c0 < KEYS; c0 += 64) {
              uint32_t w16[32];
#pragma unroll
              for (int c = 0; c < 64; c += 2) {
                float a, b;
                fma2(s[c0 + c], s[c0 + c + 1], qscale, qscale, shift, shift, a, b);
                a = ex2(a);
                b = ex2(b);
                add2(sum[c & 2], sum[(c & 2) + 1], a, b);
                w16[c / 2] = pack2<Tag>(a, b);
              }
              tmem_st32(s_addr + c0 / 2, w16);   // over scores that have been read
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (!dry && lane == 0) mbar_arrive(pfull0 + 8 * sb);
      }
      if (!ok) break;
      // The unit's end. A single query tile's rows are shared by the two
      // warpgroups: its streams are merged and each writes half of the columns.
      const bool merge = !sh.pair && u.tiles > 0 && !dry;
      if (!dry) {
        done += mine;
        if (n0 > 0 && (w == 0 || merge)) ok = warp_poll(ofull0, ends0 & 1, p.timeout_ns);
        if (n1 > 0 && (w == 1 || merge)) ok = ok && warp_poll(ofull0 + 8, ends1 & 1, p.timeout_ns);
        if (!ok) break;
        ends0 += n0 > 0;
        ends1 += n1 > 0;
      }
      tc_fence_after();
      float a0 = 1.0f, a1 = 0.0f;
      if (merge) {
        if (mine > 0) ml[128 * w + r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(meet);
        if (!(ok = warp_poll(meet, meets & 1, p.timeout_ns))) break;
        ++meets;
        const float2 y0 = ml[r], y1 = n1 > 0 ? ml[128 + r] : make_float2(y0.x, 0.0f);
        const float top = fmaxf(y0.x, y1.x);
        a0 = ex2(y0.x - top);
        a1 = ex2(y1.x - top);
        m = top;
        l = y0.y * a0 + y1.y * a1;
      }
      if (active) {
        const bool both = NS == 2 && merge && n1 > 0;
        const bool whole = u.slot < 0;
        const int c_begin = sh.pair ? 0 : w * (D / 2);
        const int c_end = sh.pair ? D : c_begin + D / 2;
        const uint32_t o_addr = tmem + lane_addr + Shape::O_COL0 + (sh.pair ? w * D : 0);
        const size_t tile = (static_cast<size_t>(u.slot) * p.Hkv + kv) * NS + (sh.pair ? w : 0);
        float4* dst = reinterpret_cast<float4*>(p.part_o) + tile * (D / 4) * 128 + r;
        uint4* row = reinterpret_cast<uint4*>(
            static_cast<uint16_t*>(p.out) +
            (static_cast<size_t>(u.tok + tx) * p.Hq + kv * p.G + g) * D);
        const bool empty = l == 0.0f || u.tiles == 0;
        const float inv = !whole ? 1.0f : empty ? 0.0f : 1.0f / l;
        a0 *= inv;
        a1 *= inv;
        const bool any_odd = !dry && u.tiles > 0 && odd[unit_no & 3];
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 32) {
          float o[32];
          tmem_ld32(o_addr + c, o);
          if (both) {
            float o1[32];
            tmem_ld32(o_addr + D + c, o1);
            tmem_wait_ld();
            hold<32>(o);
            hold<32>(o1);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = o[e] * a0 + o1[e] * a1;
          } else {
            tmem_wait_ld();
            hold<32>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] *= a0;
          }
          if (whole && empty) {   // tensor memory may hold anything for a unit without keys
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = l == 0.0f ? 0.0f : o[e];
          }
          if (any_odd && live) {
            // Values that are not finite, for the rows that see them.
            const int end = min((u.t0 + u.tiles) * KEYS, u.lim);
#pragma unroll 1
            for (int k = max(u.t0 * KEYS, sh.full); k < end; ++k) {
              if (!(pt_sees(p, u.tok, u.base, u.lim, tx, k) & 1u)) continue;
              const int col = pt_block_of(p, k);
              const int block = p.block_table[static_cast<size_t>(u.b) * p.max_blocks + col];
              if (block < 0 || block >= p.num_blocks) continue;
              const uint16_t* v = static_cast<const uint16_t*>(p.v_pool) +
                                  ((static_cast<size_t>(block) * p.bs + (k - col * p.bs)) * p.Hkv + kv) * D + c;
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (pt_odd<Tag>(v[e])) o[e] += pt_widen<Tag>(v[e]);
            }
          }
          if (!live) continue;
          if (whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8)
              row[(c + e) / 8] = make_uint4(pack2<Tag>(o[e], o[e + 1]), pack2<Tag>(o[e + 2], o[e + 3]),
                                            pack2<Tag>(o[e + 4], o[e + 5]), pack2<Tag>(o[e + 6], o[e + 7]));
          } else {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              __stcg(dst + static_cast<size_t>((c + e) / 4) * 128,
                     make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
          }
        }
        if (!whole && live && (sh.pair || w == 0)) __stcg(p.part_ml + tile * 128 + r, make_float2(m, l));
      }
      if (u.slot >= 0) {   // a slot is filled when eight warps have said so
        __threadfence();
        __syncwarp();
        if (lane == 0) atomicAdd(&p.head->done, 1u);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {   // 8 arrivals a barrier: all warps once, or a stream's own twice
        if (sh.pair || dry) {
          mbar_arrive(ofree0 + 8 * w);
          mbar_arrive(ofree0 + 8 * w);
        } else {
          mbar_arrive(ofree0);
          mbar_arrive(ofree0 + 8);
        }
      }
    }
    // ------------------------------------------------- rows that were cut
    const int n_splits = !ok ? 0 : p.small ? cut_count[0] : __ldcg(&p.head->splits);
    if (n_splits > 0) {
      // All slots of all items: no unit is unclaimed, so CTAs that run are about to
      // end the last ones.
      const unsigned want = (p.small ? cut_count[1] : __ldcg(&p.head->parts)) * 8u * p.Hkv;
      const uint64_t since = global_timer_ns();
      while (ok && *reinterpret_cast<volatile unsigned*>(&p.head->done) != want)
        ok = static_cast<long long>(global_timer_ns() - since) < p.timeout_ns;
      ok = __all_sync(0xffffffffu, ok);
      __threadfence();
      // A thread takes 8 columns of a row, 8 slots at a time: 16 loads of 16 bytes
      // under way, and the next task's item before this one's sums.
      constexpr int kPer = NS * 128 * (D / 8) / 256;   // tasks of an item and KV head
      constexpr int U = 8;
      const int tasks = ok ? n_splits * p.Hkv * kPer : 0;
      auto item_of = [&](int t) {
        const int i = t / (kPer * p.Hkv);
        return t >= tasks ? make_int4(0, 0, 0, 0)
               : p.small  ? *reinterpret_cast<const int4*>(cut_list + i)
                          : __ldcg(reinterpret_cast<const int4*>(p.splits + i));
      };
      int4 ahead = item_of(blockIdx.x);
#pragma unroll 1
      for (int t = blockIdx.x; t < tasks; t += gridDim.x) {
        const int4 raw = ahead;
        ahead = item_of(t + gridDim.x);
        const int pos = t % kPer, h = t / kPer % p.Hkv;
        const int tok = raw.x, slot = raw.z, splits = raw.w;
        const int rows = raw.y * p.G, at = pos * 256 + threadIdx.x;
        if (at >= rows * (D / 8)) continue;
        const int c = at / rows, row = at - c * rows;
        const int tk = row / p.G, gh = row - tk * p.G;
        const int tile = NS == 2 && tk >= p.TB;
        const int lane_row = (tk - tile * p.TB) * p.G + gh;
        const size_t first = (static_cast<size_t>(slot) * p.Hkv + h) * NS + tile;
        const size_t step = static_cast<size_t>(p.Hkv) * NS;
        const float2* ms = p.part_ml + first * 128 + lane_row;
        const float4* os = reinterpret_cast<const float4*>(p.part_o) + (first * (D / 4) + 2 * c) * 128 + lane_row;
        float top = -INFINITY, sum = 0.0f;
        float acc[8] = {};
#pragma unroll 1
        for (int s = 0; s < splits; s += U) {
          float2 mm[U];
          float4 v[2 * U];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            mm[k] = make_float2(-INFINITY, 0.0f);
            v[2 * k] = v[2 * k + 1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (s + k < splits) {
              mm[k] = __ldcg(ms + (s + k) * step * 128);
              v[2 * k] = __ldcg(os + (s + k) * step * (D / 4) * 128);
              v[2 * k + 1] = __ldcg(os + (s + k) * step * (D / 4) * 128 + 128);
            }
          }
          float now = top;
#pragma unroll
          for (int k = 0; k < U; ++k) now = fmaxf(now, mm[k].x);
          const float old = ex2(top - now);
          top = now;
          sum *= old;
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const float a = ex2(mm[k].x - now);
            sum = fmaf(a, mm[k].y, sum);
            const float* x = reinterpret_cast<const float*>(&v[2 * k]);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(a, x[e], acc[e]);
          }
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) +
                                  (static_cast<size_t>(tok + tk) * p.Hq + h * p.G + gh) * D + 8 * c) =
            make_uint4(pack2<Tag>(acc[0] * inv, acc[1] * inv), pack2<Tag>(acc[2] * inv, acc[3] * inv),
                       pack2<Tag>(acc[4] * inv, acc[5] * inv), pack2<Tag>(acc[6] * inv, acc[7] * inv));
      }
    }
    if (!ok && lane == 0) atomicOr(&pt_status, kErrPtSoftmax);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kPtMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
  // The last CTA leaves the header as it was found: all others have read it.
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicInc(&p.head->left, gridDim.x - 1) == gridDim.x - 1) {
      p.head->ticket = p.head->ready = p.head->next = p.head->done = 0;
      __threadfence();
    }
  }
}

}  // namespace gqa_av
