// Decode attention over a paged KV cache with shared prefixes, sm_103a. The
// operation is stated in include/gqa_prefix.h.
//
// Rows. For one KV head the G query heads of every sequence behind a prefix
// form the rows of one matrix: a query tile is TB = 128 / G sequences (TB * G
// <= 128 rows), so a prefix key that is read once meets 128 rows, or 256 where
// two tiles run together. A sequence's own keys meet its G rows only.
//
// Units. The work is cut into units: prefix units (group, KV head, split of
// the prefix, query tile or pair of tiles; tiles fastest, so the CTAs that
// need the same keys take them at the same time) and then the sequences' own
// units (sequence, KV head, split). A persistent CTA takes unit blockIdx.x
// first and then the next free one from a counter. A unit writes its
// unnormalised output, maximum and sum to a slot of its own, and the combine
// kernel adds a row's slots in split order: who computed a unit does not
// matter for the result.
//
// A unit runs an online softmax over tiles of KEYS keys:
//   S = Q K^T     tcgen05.mma, M = 128 rows, N = KEYS, Q and K from shared
//                 memory (K-major, 128-byte swizzle), S in tensor memory;
//   P = 2^(S' - m) by one softmax warpgroup, a row a thread, S' = S * scale *
//                 log2 e; P goes back to tensor memory over S as 16 bits;
//   O += P V      tcgen05.mma with P as the A operand from tensor memory and V
//                 from shared memory (MN-major), O in tensor memory.
// m moves only when a row's maximum has grown by more than 2^8 (then O and l
// are rescaled), so O is rarely touched; weights stay below 2^8.
// Rounding the weights to 16 bits lets one product make O (two halves of a weight
// would take two) and costs half a step a weight: against 64 bits the error is
// 1.0 to 1.4 times that of a plain form with fp32 weights, whose last rounding is
// the larger part (bf16 0.0017 to 0.0023 of the output's norm for 0.0017, most
// where many keys share the weight; fp16 0.00028 for 0.00021). l sums them
// unrounded: the roundings of many weights average out, so rounding them there
// too would only take more instructions.
//
// D <= 128: two streams (S, O and a softmax warpgroup each) work in turn, so
// the tensor core multiplies for one while the other makes weights. The
// streams take the two query tiles of a pair and share every K and V stage, or
// the even and odd key tiles of a single query tile, merged at the unit's end.
// D = 256: O fills half of the tensor memory, so there is one stream with two
// S buffers and key tiles of 64.
//
// Bounds and figures. A prefix key costs 2 * 2 * D * rows operations for 4 * D
// bytes, so about 290 rows make it as much the tensor cores' work as HBM's; own
// rows are HBM's. Measured (bf16, blocks of 16, 64 + 8 heads of 128): 256
// sequences behind 32768 rows, no own rows, 239 us, 1150 TFLOP/s (128 units of one
// query tile, so 24 of the 152 SMs idle; the others' tensor pipes are active 55 %
// of the time: within a stream scores, weights and next scores follow one another,
// 1580 cycles a key tile for 1024 of products; the combine takes 17 us); 32
// sequences of 8192 own rows 174 us, 6.15 TB/s; two sequences behind 512 rows (8 +
// 2 heads of 64) 12 us, a chain of latencies. Key tiles of 128 keep
// QK at the full rate (at N = 64 it waits for shared memory: 48 cycles where the
// product takes 32) but leave no tensor memory for a second S.
//
// Warps: 0-3 and 4-7 softmax warpgroups (and the units' ends), 8 issues the
// MMAs from one thread, 9 makes the plan, hands out units and loads queries and
// K, 10 loads V (a box of a small block costs its issuing warp some time, so K
// and V go out from two); 11 only fills the warpgroup. Every wait is bounded (2 s): on expiry the role sets
// the status word and leaves, the others run out in turn, copies and MMAs in
// flight are waited for and tensor memory is freed.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_av_mma.cuh"
#include "gqa_pack.cuh"

namespace gqa_av {

constexpr int kPxThreads = 384;
// Registers a thread: 168 at launch (65536 / 384, rounded down to 8); the last
// warpgroup gives up enough of them for the softmax warpgroups' 128 scores a
// thread: 2 * 128 * 184 + 128 * 136 = 384 * 168.
constexpr int kPxSoftmaxRegs = 184, kPxAuxRegs = 136;
constexpr int kPxMmaWarp = 8, kPxKWarp = 9, kPxVWarp = 10;
constexpr int kPxMaxGroups = 32;       // a lane of the plan each
constexpr int kPxMaxB = 4096;
constexpr int kPxSegs = 2;             // unit descriptors in flight
constexpr float kPxGrow = 8.0f;        // log2 of the growth of a maximum that is tolerated
constexpr unsigned kErrPxLoad = 16u, kErrPxMma = 32u, kErrPxSoftmax = 64u;
constexpr long long kPxTimeoutNs = 2000000000LL;   // bound of every wait; also of the last ones,
                                                   // for copies and MMAs in flight

// Set by waits that run out, read by gqa_prefix_device_status. One word a device
// for the life of the process: a workspace may be outgrown while captured graphs
// still run in it, and what they report must be found.
__device__ unsigned px_status;

template <int D>
struct PxShape {
  static constexpr int NS = D == 256 ? 1 : 2;          // streams
  static constexpr int KEYS = D == 256 ? 64 : 128;     // keys of a tile
  static constexpr int PARTS = D / 64;                 // 64-column parts of a row
  static constexpr int STAGE = KEYS * D * 2;           // bytes of a K or V stage
  static constexpr int QBYTES = 128 * D * 2;
  static constexpr int QBUF = NS;                      // query buffers
  static constexpr int STAGES = D == 64 ? 11 : 5;
  static constexpr int TILES_BYTES = QBUF * QBYTES + STAGES * STAGE;
  static constexpr int MISC = D == 64 ? 2048 : 1024;   // barriers, units, plan
  static constexpr int SMEM = TILES_BYTES + MISC + 2048;
  static constexpr uint32_t S_COL = KEYS;              // tensor-memory columns of an S buffer
  static constexpr uint32_t O_COL0 = 256;
};

// A group's part of the plan, as the combine kernel reads it.
struct PxGroup {
  int begin, end;     // sequences
  int splits;         // 0: no prefix rows
  int nq;             // units a split and KV head: query tiles, or pairs of them
  int pair;           // two query tiles a unit
  int base;           // its first unit
};
struct PxHeader {
  int next;                       // units handed out past the first of each CTA
  int own_tiles;                  // key tiles of a sequence's own unit
  PxGroup group[kPxMaxGroups];
  int own_base[kPxMaxB];          // first own unit (slot) of each sequence
};

struct alignas(64) PrefixParams {
  CUtensorMap q_tile_map;         // q as {D, G, Hkv, B}; box {64, G, 1, TB}
  CUtensorMap q_one_map;          // box {64, G, 1, 1}
  CUtensorMap k_map, v_map;       // pools as {D, Hkv, rows}; box {64, 1, R}
  const int32_t *prefix_table, *prefix_lens, *group_start, *block_table, *seq_lens;
  void* out;
  PxHeader* head;
  float* prefix_o;                // prefix slots [units][NS][D / 4][128][4]
  float2* prefix_ml;              // [units][NS][128] (maximum in log2 units, sum)
  float* own_o;                   // own slots [units][D / 4][G][4]
  float2* own_ml;                 // [units][G]
  int B, P, Hq, Hkv, G, TB;
  int bs, num_blocks, max_pblocks, max_blocks;
  unsigned bs_mul;                // c / bs = c * bs_mul >> bs_shift for c < 2^26
  int bs_shift;
  int R;                          // rows of a K or V box: gcd(bs, KEYS)
  float qscale;                   // |scale| * log2(e)
  int negate;                     // scale < 0
  int prefix_slots;               // bound on the prefix units
  float c_pair, c_tile, c_own, c_unit;   // plan: cost of a key tile of each kind and of a unit
  long long timeout_ns;
  unsigned withhold_from;         // self-test: query loads from this one of a CTA on are not issued
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]),
        "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_nowait(uint32_t taddr, float* v) {
  uint32_t* r = reinterpret_cast<uint32_t*>(v);
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Issue by one lane of a converged warp. The operands of MMAs, commits and TMA
// copies have to be in uniform registers; computed by the whole warp under
// uniform control flow they stay there, while inside a one-lane branch each
// operand is moved over for every instruction (measured: 107 cycles an MMA of
// 64, and 110 a TMA box).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t leader;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(leader));
  return leader;
}
// A value that is the same in all lanes, for uniform registers.
__device__ __forceinline__ int uniform(int x) {
  return static_cast<int>(__reduce_or_sync(0xffffffffu, static_cast<unsigned>(x)));
}
// D[tmem] (+)= A[smem] * B[smem], or A[tmem] * B[smem]: 16-bit operands of one type.
__device__ __forceinline__ void mma_ss(uint32_t leader, uint32_t d_tmem, uint64_t a, uint64_t b,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t leader, uint32_t d_tmem, uint32_t a_tmem,
                                       uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_one(uint32_t leader, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void expect_one(uint32_t leader, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_one_3d(uint32_t leader, uint32_t dst, const CUtensorMap* map,
                                           int x0, int x1, int x2, uint32_t bar, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %7, 0;\n\t"
      "@q cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x0), "r"(x1), "r"(x2), "r"(bar), "l"(policy),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ void tma_one_4d(uint32_t leader, uint32_t dst, const CUtensorMap* map,
                                           int x0, int x1, int x2, int x3, uint32_t bar,
                                           uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %8, 0;\n\t"
      "@q cp.async.bulk.tensor.4d.shared::cta.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x0), "r"(x1), "r"(x2), "r"(x3), "r"(bar),
      "l"(policy), "r"(leader)
      : "memory");
}

// kind::f16 with fp32 D, M = 128, N = n; b_mn: B is MN-major.
template <typename Tag>
__host__ __device__ constexpr uint32_t px_idesc(int n, bool b_mn) {
  return (1u << 4) | (std::is_same<Tag, Bf16Tag>::value ? ((1u << 7) | (1u << 10)) : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 multiply-adds and additions in one instruction each.
__device__ __forceinline__ void fma2(float a, float b, float x, float y, float c, float d, float& r,
                                     float& t) {
  asm("{\n\t.reg .b64 u, v, w;\n\tmov.b64 u, {%2, %3};\n\tmov.b64 v, {%4, %5};\n\t"
      "mov.b64 w, {%6, %7};\n\tfma.rn.f32x2 u, u, v, w;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "=f"(r), "=f"(t)
      : "f"(a), "f"(b), "f"(x), "f"(y), "f"(c), "f"(d));
}
__device__ __forceinline__ void add2(float& a, float& b, float x, float y) {
  asm("{\n\t.reg .b64 u, v;\n\tmov.b64 u, {%0, %1};\n\tmov.b64 v, {%2, %3};\n\t"
      "add.rn.f32x2 u, u, v;\n\tmov.b64 {%0, %1}, u;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(x), "f"(y));
}

__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

// A wait by a whole warp; the lanes agree on whether it ran out, so that they
// leave together.
__device__ __forceinline__ bool warp_poll(uint32_t bar, uint32_t parity, long long timeout_ns) {
  return __all_sync(0xffffffffu, mbar_poll(bar, parity, timeout_ns));
}

// Keeps uses of values that tcgen05.ld delivers behind its wait.
template <int N>
__device__ __forceinline__ void hold(float* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}

// One run of key tiles: keys of one table row for one KV head.
struct PxPart {
  const int32_t* table;
  int len;            // rows that the table row lists
  int t0, tiles;      // key tiles
  int last_valid;     // keys of the last one
  int kv;             // KV head
  int q0;             // first sequence
  int slot;
};
// What a CTA works on at a time.
//   kSplit: one query tile; two streams take the even and the odd key tiles.
//   kPair: two query tiles, a stream each, over the same key tiles.
//   kOwn: own units of two (sequence, KV head, split)s, a stream each.
enum { kSplit, kPair, kOwn };
struct PxUnit {
  PxPart part[2];     // kOwn: one for each stream; else the first
  int rows[2];        // rows of the query tiles
  int mode;
  int own;            // a sequence's own keys
};

// The tiles of a unit in the order of their use, i = 0 .. n - 1: tile j of
// stream w when the streams take turns until the shorter one ends.
__device__ __forceinline__ int turn(int w, int j, int n0, int n1) {
  const int m = min(n0, n1);
  return j < m ? 2 * j + w : m + j;
}
// Positions of tile i's K and V in the unit's run of 2 n stages, about the
// order of their first use: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int k_pos(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int v_pos(int i, int n) { return min(2 * i + 2, 2 * n - 1); }

__device__ __forceinline__ int warp_incl_sum(int x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// x / y for 0 <= x < 2^21 and y > 0, in fp32: the quotient of x + 1/2 is at
// least 1 / (2 y) away from an integer, further than its error. The host keeps
// tiles, units and sequences below that.
__device__ __forceinline__ int quick_div(int x, int y) {
  return __float2int_rz(__fdividef(static_cast<float>(x) + 0.5f, static_cast<float>(y)));
}

// The sequences' own part of the plan, in shared memory.
struct PxOwn {
  int upto[kPxMaxB / 32];   // units of the blocks of 32 sequences up to each
  int tiles;                // key tiles of a unit
  int units;
  float work;               // key tiles of the batch, times KV heads
  int paired;               // units are taken two at a time
};

// The plan, made from the lengths by two warps at the head of every call. Its
// code runs once a call and is fetched cold each time, at about 7 ns an
// instruction (measured: 3.2 us for one part, 1 us when run again), so it is
// kept short: 32 groups at most, no integer division, no unrolling but that of
// loads. The V warp makes the own part; the K warp the groups', a lane each,
// and finds units by it.
template <int D>
struct PxPlan {
  using Shape = PxShape<D>;
  int begin, end, len, tiles, splits, nq, pair, upto;   // this lane's group
  int prefix_units;

  static __device__ __forceinline__ int own_len(const PrefixParams& p, int b) {
    const int cap = p.max_blocks * p.bs;
    return b < p.B ? (p.seq_lens ? min(max(p.seq_lens[b], 0), cap) : cap) : 0;
  }
  static __device__ __forceinline__ int tiles_of(int len) {
    return (len + Shape::KEYS - 1) / Shape::KEYS;
  }

  // By the V warp. A unit takes so many tiles that a CTA gets about four (two
  // with one stream, whose units do not overlap: 52 us where it was 55 at 64
  // sequences behind 32768 rows, 16 + 1 heads of 256), so
  // that the last ones to end are short. The sum of the tiles is made of two
  // halves: it may pass 2^31.
  static __device__ __forceinline__ void make_own(const PrefixParams& p, PxOwn* own) {
    const int lane = threadIdx.x & 31;
    const int seqs = p.max_blocks > 0 ? p.B : 0;
    unsigned low = 0, high = 0;
    for (int b0 = 0; b0 < seqs; b0 += 256) {
      int len[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) len[k] = own_len(p, b0 + 32 * k + lane);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        low += tiles_of(len[k]) & 4095;
        high += tiles_of(len[k]) >> 12;
      }
    }
    low = __reduce_add_sync(0xffffffffu, low);
    high = __reduce_add_sync(0xffffffffu, high);
    const float work = (static_cast<float>(high) * 4096.0f + static_cast<float>(low)) *
                       static_cast<float>(p.Hkv);
    // Rounded up with a margin for the rounding of the sum: never more than
    // four units a CTA beyond one a sequence and KV head.
    const int each = __float2int_ru(
        fminf(fmaxf(1.0f, __fdividef(work * 1.00001f, static_cast<float>((Shape::NS == 1 ? 2 : 4) * gridDim.x))), 1048576.0f));
    int units = 0;
#pragma unroll 1
    for (int k0 = 0; 32 * k0 < seqs; k0 += 32) {
      int mine = 0;
#pragma unroll 2
      for (int k = 0; k < 32 && 32 * (k0 + k) < seqs; ++k) {
        const int t = tiles_of(own_len(p, 32 * (k0 + k) + lane));
        const int sum = __reduce_add_sync(0xffffffffu, quick_div(t + each - 1, each));
        mine = k == lane ? sum * p.Hkv : mine;
      }
      mine = units + warp_incl_sum(mine);
      own->upto[k0 + lane] = mine;
      units = __shfl_sync(0xffffffffu, mine, 31);
    }
    if (lane == 0) {
      own->tiles = each;
      own->units = units;
      own->work = work;
      own->paired = Shape::NS == 2 && units > static_cast<int>(gridDim.x);
    }
    __syncwarp();
  }

  // By the K warp: the groups' lengths, while the V warp reads the others.
  __device__ __forceinline__ void load_groups(const PrefixParams& p) {
    const int lane = threadIdx.x & 31;
    begin = 0;
    end = lane < p.P ? p.B : 0;
    len = 0;
    if (lane < p.P) {
      len = p.prefix_lens[lane];
      if (p.group_start) {
        begin = p.group_start[lane];
        end = p.group_start[lane + 1];
      }
    }
  }
  __device__ __forceinline__ void make_groups(const PrefixParams& p, const PxOwn* own) {
    const int lane = threadIdx.x & 31;
    const int n = gridDim.x;
    // Starts within the batch and not below their predecessors.
    begin = min(max(begin, 0), p.B);
    if (p.P > 1) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, begin, o);
        if (lane >= o) begin = max(begin, y);
      }
    }
    end = max(begin, min(end, p.B));
    len = min(max(len, 0), p.max_pblocks * p.bs);
    const int q = quick_div(end - begin + p.TB - 1, p.TB);    // query tiles
    tiles = lane < p.P && q > 0 ? tiles_of(len) : 0;
    splits = upto = prefix_units = 0;
    nq = 1;
    pair = 0;
    const int longest = __reduce_max_sync(0xffffffffu, tiles);
    if (longest == 0) return;
    // How to cut the prefixes: each lane costs one choice of pairs or single
    // query tiles and of the key tiles a split takes, from the time that the
    // units take if all CTAs stay busy, own units included, and from the CTA with
    // the most prefix units. The cuts aim at 1 to 8 units a CTA; those with more
    // units than slots (one a query tile and two a CTA) are left out, so long
    // prefixes behind few query tiles have 1 or 2 to choose from. On 51 batches,
    // listed and drawn ones, the choice is 2.6 % slower than the best choice
    // measured, on average, at worst 22 % (18.4 us for 14.9: a small batch).
    const bool pairs = Shape::NS == 2 && (lane & 1);
    float w = 0.0f;                     // key tiles x query tiles (or pairs)
    for (int g = 0; g < p.P; ++g) {
      const int t = __shfl_sync(0xffffffffu, tiles, g), m = __shfl_sync(0xffffffffu, q, g);
      w += static_cast<float>(t) * static_cast<float>(pairs ? (m + 1) / 2 : m);
    }
    w *= static_cast<float>(p.Hkv);
    int chunk = __float2int_ru(__fdividef(w, static_cast<float>(((lane >> 2) + 1) * n))) +
                ((lane >> 1) & 1);
    chunk = lane >= 30 ? longest : max(1, min(chunk, longest));   // 30, 31: no cut, always fits
    float units = 0.0f;
    for (int g = 0; g < p.P; ++g) {
      const int t = __shfl_sync(0xffffffffu, tiles, g), m = __shfl_sync(0xffffffffu, q, g);
      units += static_cast<float>(quick_div(t + chunk - 1, chunk)) *
               static_cast<float>(pairs ? (m + 1) / 2 : m);
    }
    units *= static_cast<float>(p.Hkv);
    const float c = pairs ? p.c_pair : p.c_tile;
    const float one = static_cast<float>(chunk) * c + p.c_unit;
    const float all = __fdividef(w * c + units * p.c_unit + own->work * p.c_own, static_cast<float>(n));
    const float rounds = ceilf(__fdividef(units - 0.5f, static_cast<float>(n)));
    const float est = units <= static_cast<float>(p.prefix_slots) ? fmaxf(all, rounds * one) : INFINITY;
    // Costs are positive, so their bit patterns are ordered like them.
    const unsigned best = __reduce_min_sync(0xffffffffu, __float_as_uint(est));
    const int src = __ffs(__ballot_sync(0xffffffffu, __float_as_uint(est) == best)) - 1;
    const int cut = __shfl_sync(0xffffffffu, chunk, src);
    splits = quick_div(tiles + cut - 1, cut);
    pair = Shape::NS == 2 && (src & 1) && q > 1;
    nq = max(1, pair ? (q + 1) / 2 : q);
    upto = warp_incl_sum(nq * splits * p.Hkv);
    prefix_units = __shfl_sync(0xffffffffu, upto, 31);
  }

  // Part i of t tiles cut into s equal parts (the first t % s one longer).
  static __device__ __forceinline__ void cut_out(PxPart& w, int i, int t, int s) {
    const int each = quick_div(t, s), more = t - each * s;
    w.t0 = i * each + min(i, more);
    w.tiles = each + (i < more);
    w.last_valid = i == s - 1 ? w.len - (t - 1) * Shape::KEYS : Shape::KEYS;
  }
  // Prefix unit u: counted (group, KV head, split, query tile), tiles fastest.
  __device__ __forceinline__ void find_prefix(const PrefixParams& p, int u, PxUnit& un) const {
    PxPart& w = un.part[0];
    const int g = __ffs(__ballot_sync(0xffffffffu, u < upto)) - 1;
    const int a = __shfl_sync(0xffffffffu, begin, g), e = __shfl_sync(0xffffffffu, end, g);
    const int t = __shfl_sync(0xffffffffu, tiles, g), s = __shfl_sync(0xffffffffu, splits, g);
    const int q = __shfl_sync(0xffffffffu, nq, g), pr = __shfl_sync(0xffffffffu, pair, g);
    w.len = __shfl_sync(0xffffffffu, len, g);
    const int local = u - (__shfl_sync(0xffffffffu, upto, g) - q * s * p.Hkv);
    const int outer = quick_div(local, q), i = local - outer * q;
    w.kv = quick_div(outer, s);
    cut_out(w, outer - w.kv * s, t, s);
    w.q0 = a + (i << pr) * p.TB;
    un.rows[0] = min(p.TB, e - w.q0) * p.G;
    un.rows[1] = pr ? max(0, min(p.TB, e - w.q0 - p.TB)) * p.G : 0;
    un.mode = un.rows[1] > 0 ? kPair : kSplit;
    un.own = 0;
    w.slot = u;
    w.table = p.prefix_table + static_cast<size_t>(g) * p.max_pblocks;
  }
  // Own unit v: counted (sequence, KV head, split).
  static __device__ __forceinline__ void find_own(const PrefixParams& p, const PxOwn* own, int v,
                                                  PxPart& w) {
    const int lane = threadIdx.x & 31;
    int block = 0, before = 0;
#pragma unroll 1
    for (int k0 = 0; k0 < kPxMaxB / 32; k0 += 32) {
      const int upto = own->upto[k0 + lane];
      const unsigned hit = __ballot_sync(0xffffffffu, v < upto);
      const int at = hit ? __ffs(hit) - 2 : 31;
      if (at >= 0) before = __shfl_sync(0xffffffffu, upto, at);
      block = k0 + at + 1;
      if (hit) break;
    }
    const int each = own->tiles;
    const int my_len = own_len(p, 32 * block + lane);
    const int my_splits = quick_div(tiles_of(my_len) + each - 1, each);
    const int incl = warp_incl_sum(my_splits * p.Hkv);
    const int src = __ffs(__ballot_sync(0xffffffffu, v - before < incl) | 0x80000000u) - 1;
    const int s = max(1, __shfl_sync(0xffffffffu, my_splits, src));
    w.len = __shfl_sync(0xffffffffu, my_len, src);
    const int local = v - before - (__shfl_sync(0xffffffffu, incl, src) - s * p.Hkv);
    w.kv = quick_div(local, s);
    cut_out(w, local - w.kv * s, tiles_of(w.len), s);
    w.q0 = 32 * block + src;
    w.slot = v;
    w.table = p.block_table + static_cast<size_t>(w.q0) * p.max_blocks;
  }

  // For the combine kernel (the K warp of one CTA).
  __device__ __forceinline__ void write(const PrefixParams& p, const PxOwn* own) const {
    const int lane = threadIdx.x & 31;
    const int each = own->tiles;
    if (lane == 0) p.head->own_tiles = each;
    if (lane < p.P) p.head->group[lane] = {begin, end, splits, nq, pair, upto - nq * splits * p.Hkv};
    int base = 0;
    if (p.max_blocks > 0)
#pragma unroll 1
      for (int k = 0; 32 * k < p.B; ++k) {
        const int n = quick_div(tiles_of(own_len(p, 32 * k + lane)) + each - 1, each) * p.Hkv;
        const int incl = warp_incl_sum(n);
        if (32 * k + lane < p.B) p.head->own_base[32 * k + lane] = base + incl - n;
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
  }
};

template <typename Tag, int D>
__global__ void __launch_bounds__(kPxThreads, 1)
    gqa_prefix_kernel(const __grid_constant__ PrefixParams p) {
  using Shape = PxShape<D>;
  constexpr int NS = Shape::NS, KEYS = Shape::KEYS, STAGES = Shape::STAGES, PARTS = Shape::PARTS;
  // fp16 weights are scaled by 2^6 (at most 2^14 with the growth allowance), so
  // that small ones keep their bits; the sum carries the same factor.
  constexpr float kOff = std::is_same<Tag, Fp16Tag>::value ? 6.0f : 0.0f;
  extern __shared__ __align__(1024) uint8_t px_smem[];
  uint8_t* smem = px_smem;
  const uint32_t base_s = smem_addr(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Shape::TILES_BYTES);
  const uint32_t full0 = smem_addr(bars), empty0 = full0 + 8 * STAGES;
  const uint32_t qfull0 = empty0 + 8 * STAGES, qempty0 = qfull0 + 16;
  const uint32_t sfull0 = qempty0 + 16, pfull0 = sfull0 + 16;   // a stream's, or an S buffer's
  const uint32_t ofull0 = pfull0 + 16, ofree0 = ofull0 + 16, pvdone = ofree0 + 16;
  const uint32_t meet = pvdone + 8, drain = meet + 8;
  const uint32_t ufull0 = drain + 8, uempty0 = ufull0 + 8 * kPxSegs;
  constexpr int kBars = 2 * STAGES + 15 + 2 * kPxSegs;
  PxUnit* units = reinterpret_cast<PxUnit*>(bars + kBars);
  PxOwn* own_plan = reinterpret_cast<PxOwn*>(units + kPxSegs);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(own_plan + 1);
  float2* ml = reinterpret_cast<float2*>(smem + Shape::TILES_BYTES + Shape::MISC);   // [2][128]
  static_assert(8 * kBars + sizeof(PxUnit) * kPxSegs + sizeof(PxOwn) + 4 <= Shape::MISC,
                "shared memory besides the tiles");

  if (warp == kPxMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_addr(tmem_slot)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(qfull0 + 8 * i, 1);
      mbar_init(qempty0 + 8 * i, 1);
      mbar_init(sfull0 + 8 * i, 1);
      mbar_init(pfull0 + 8 * i, 4);
      mbar_init(ofull0 + 8 * i, 1);
      mbar_init(ofree0 + 8 * i, 8);
    }
    mbar_init(pvdone, 1);
    mbar_init(meet, 8);
    mbar_init(drain, 1);
    for (int i = 0; i < kPxSegs; ++i) {
      mbar_init(ufull0 + 8 * i, 1);
      mbar_init(uempty0 + 8 * i, 10);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kPxKWarp && lane < 4) {
    const CUtensorMap* m = lane == 0 ? &p.k_map : lane == 1 ? &p.v_map : lane == 2 ? &p.q_tile_map
                                                                                   : &p.q_one_map;
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t qbuf_s = base_s, ring_s = base_s + Shape::QBUF * Shape::QBYTES;
  grid_dependency_wait();
  grid_launch_dependents();
  const bool aligned = (base_s & 1023u) == 0;   // the tiles need it; dynamic memory starts so
  if (!aligned && threadIdx.x == 0) atomicOr(&px_status, kErrPxLoad);
  // kOwn: the second stream's rows lie in lanes of other warps than the first's
  // where they fit, so that the two softmax warps sit on different schedulers.
  const int own_shift = p.G <= 32 ? 32 : p.G <= 64 ? 64 : 0;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPxAuxRegs));
    if (aligned && (warp == kPxKWarp || warp == kPxVWarp)) {
      // ----------------------------------- plan, units, queries and K, or V
      const bool is_k = warp == kPxKWarp;
      const uint32_t leader = elect_one();
      const uint64_t policy = evict_first_policy();
      const int nch = KEYS / p.R;              // boxes of one 64-column part of a tile
      const int oob = p.num_blocks * p.bs;
      unsigned base = 0, fills = 0;
      // Lane s: 1 + parity of this warp's last copy into stage s (0: none yet);
      // lane 16 + s: into query buffer s.
      unsigned held = 0;
      bool ok = true;
      PxPlan<D> plan;
      int u = blockIdx.x, prefix_units = 0, total = 0;
      if (is_k) {
        plan.load_groups(p);
        named_sync(1, 64);
        plan.make_groups(p, own_plan);
        prefix_units = uniform(plan.prefix_units);
        total = prefix_units + (own_plan->paired ? (own_plan->units + 1) / 2 : own_plan->units);
      } else {
        PxPlan<D>::make_own(p, own_plan);
        named_sync(1, 64);
      }
      for (unsigned unit_no = 0; ok; ++unit_no) {
        const int seg = unit_no % kPxSegs;
        PxUnit& un = units[seg];
        int next = 0;
        if (is_k) {
          if (!(ok = warp_poll(uempty0 + 8 * seg, ((unit_no / kPxSegs) & 1) ^ 1, p.timeout_ns))) break;
          PxUnit made;
          made.part[0].tiles = made.part[1].tiles = 0;
          if (u < total) {
            if (lane == 0) next = atomicAdd(&p.head->next, 1) + gridDim.x;
            if (u < prefix_units) {
              plan.find_prefix(p, u, made);
            } else {
              const int twice = own_plan->paired;
              const int v = (u - prefix_units) << twice;
              made.own = 1;
              made.mode = twice ? kOwn : kSplit;
              made.rows[0] = made.rows[1] = p.G;
              for (int i = 0; i <= twice; ++i)
                if (v + i < own_plan->units) {
                  PxPart w;
                  PxPlan<D>::find_own(p, own_plan, v + i, w);
                  if (i == 0) made.part[0] = w;
                  else made.part[1] = w;
                }
            }
          }
          if (lane == 0) {
            un = made;
            mbar_arrive(ufull0 + 8 * seg);
          }
          __syncwarp();
        } else {
          if (!(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPxSegs) & 1, p.timeout_ns))) break;
        }
        const PxPart part0 = un.part[0], part1 = un.part[1];
        const int mode = uniform(un.mode), own = uniform(un.own);
        __syncwarp();
        if (!is_k && lane == 0) mbar_arrive(uempty0 + 8 * seg);
        const int n0 = uniform(part0.tiles), n1 = mode == kOwn ? uniform(part1.tiles) : 0;
        const int n = n0 + n1;
        if (n0 == 0) break;
        const int kv0 = uniform(part0.kv), kv1 = uniform(part1.kv);
        const int both = 2 * min(n0, n1);      // tiles during which the streams take turns
        // Which part tile i of the unit's order is of, and the pool row of this
        // lane's box of it; rows past the length and entries outside the pool
        // read zeros.
        auto of_second = [&](int i) { return i < both ? i & 1 : n1 > n0; };
        auto row_of = [&](int i) {
          const bool second = of_second(i);
          const int tile = i < both ? i >> 1 : i - both / 2;
          const int c = ((second ? part1.t0 : part0.t0) + tile) * KEYS + lane * p.R;
          if (lane >= nch || i >= n || c >= (second ? part1.len : part0.len)) return oob;
          const int col = static_cast<int>((static_cast<unsigned long long>(static_cast<unsigned>(c)) * p.bs_mul) >> p.bs_shift);
          const int block = (second ? part1.table : part0.table)[col];
          return block >= 0 && block < p.num_blocks ? block * p.bs + (c - col * p.bs) : oob;
        };
        int row = row_of(0);
        if (is_k) {
          const int q0 = uniform(part0.q0), q1 = mode == kPair ? q0 + p.TB : uniform(part1.q0);
          const int more = mode == kPair || n1 > 0;
          for (int i = 0; i <= more && ok; ++i, ++fills) {
            const int buf = fills % Shape::QBUF;
            ok = warp_poll(qempty0 + 8 * buf, ((fills / Shape::QBUF) & 1) ^ 1, p.timeout_ns);
            if (!ok) break;
            if (fills >= p.withhold_from) continue;
            const uint32_t bar = qfull0 + 8 * buf;
            if (lane == 16 + buf) held = 1 + ((fills / Shape::QBUF) & 1);
            expect_one(leader, bar, (own ? p.G : p.TB * p.G) * 128 * PARTS);
            const uint32_t dst = qbuf_s + buf * Shape::QBYTES + (mode == kOwn && i ? own_shift * 128 : 0);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              tma_one_4d(leader, dst + part * 128 * 128, own ? &p.q_one_map : &p.q_tile_map,
                         64 * part, 0, mode == kOwn && i ? kv1 : kv0, i ? q1 : q0, bar, policy);
          }
        }
        const CUtensorMap* map = is_k ? &p.k_map : &p.v_map;
        for (int i = 0; i < n && ok; ++i) {
          const int ahead = row_of(i + 1);
          const unsigned at = base + (is_k ? k_pos(i) : v_pos(i, n)), stage = at % STAGES;
          if (!(ok = warp_poll(empty0 + 8 * stage, ((at / STAGES) & 1) ^ 1, p.timeout_ns))) break;
          const uint32_t bar = full0 + 8 * stage, dst = ring_s + stage * Shape::STAGE;
          const int kv = of_second(i) ? kv1 : kv0;
          expect_one(leader, bar, Shape::STAGE);
          if (lane == stage) held = 1 + ((at / STAGES) & 1);
          for (int c = 0; c < nch; ++c) {
            const int r = __shfl_sync(0xffffffffu, row, c);
#pragma unroll
            for (int part = 0; part < PARTS; ++part)
              tma_one_3d(leader, dst + part * KEYS * 128 + c * p.R * 128, map, 64 * part, kv, r, bar,
                         policy);
          }
          row = ahead;
        }
        base += 2 * n;
        u = __shfl_sync(0xffffffffu, next, 0);
      }
      if (is_k && blockIdx.x == gridDim.x - 1) plan.write(p, own_plan);
      if (!ok) {
        // This warp's copies in flight land before the CTA leaves (a wait for a
        // stage that the other loader has filled since takes its full 2 s).
        if (lane == 0) atomicOr(&px_status, kErrPxLoad);
        if (held && lane < STAGES) mbar_wait(full0 + 8 * lane, held - 1, kPxTimeoutNs);
        if (held && lane >= 16) mbar_wait(qfull0 + 8 * (lane - 16), held - 1, kPxTimeoutNs);
        __syncwarp();
      }
    } else if (aligned && warp == kPxMmaWarp) {
      // ---------------------------------------------------------- MMA issue
      const uint32_t leader = elect_one();
      constexpr uint32_t qk_idesc = px_idesc<Tag>(KEYS, false), pv_idesc = px_idesc<Tag>(D, true);
      unsigned base = 0, fills = 0, done0 = 0, done1 = 0;   // stages, fills, tiles of each stream
      // The softmax warps have run through their code once (below).
      bool ok = warp_poll(ofree0, 0, p.timeout_ns) && warp_poll(ofree0 + 8, 0, p.timeout_ns);
      for (unsigned unit_no = 0; ok; ++unit_no) {
        const int seg = unit_no % kPxSegs;
        if (!(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPxSegs) & 1, p.timeout_ns))) break;
        const int mode = uniform(units[seg].mode);
        const int t0 = uniform(units[seg].part[0].tiles), t1 = uniform(units[seg].part[1].tiles);
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty0 + 8 * seg);
        if (t0 == 0) break;
        const int n0 = NS == 1 || mode != kSplit ? t0 : (t0 + 1) / 2;
        const int n1 = NS == 1 ? 0 : mode == kSplit ? t0 / 2 : mode == kPair ? t0 : t1;
        const int n = mode == kPair ? t0 : n0 + n1;
        auto tile_of = [&](int w, int j) { return NS == 1 || mode == kPair ? j : turn(w, j, n0, n1); };
        auto s_of = [&](int w, unsigned tile_no) {
          return tmem + Shape::S_COL * (NS == 2 ? w : tile_no & 1);
        };
        auto qk = [&](int w, int j) {
          const int i = tile_of(w, j);
          const unsigned at = base + k_pos(i), stage = at % STAGES;
          const unsigned fill = fills + (mode != kSplit ? w : 0), buf = fill % Shape::QBUF;
          if (j == 0) ok = ok && warp_poll(qfull0 + 8 * buf, (fill / Shape::QBUF) & 1, p.timeout_ns);
          ok = ok && warp_poll(full0 + 8 * stage, (at / STAGES) & 1, p.timeout_ns);
          if (!ok) return;
          tc_fence_after();
          const unsigned no = (w ? done1 : done0) + j;
          const uint64_t a = smem_desc(qbuf_s + buf * Shape::QBYTES, 16, 1024, 2);
          const uint64_t b = smem_desc(ring_s + stage * Shape::STAGE, 16, 1024, 2);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_ss(leader, s_of(w, no), a + (uint64_t)((kk / 4 * 128 * 128 + kk % 4 * 32) >> 4),
                   b + (uint64_t)((kk / 4 * KEYS * 128 + kk % 4 * 32) >> 4), qk_idesc, kk > 0);
          if (mode != kPair || w == 1) commit_one(leader, empty0 + 8 * stage);
          if (mode == kSplit ? i == n - 1 : j == (w ? n1 : n0) - 1)
            commit_one(leader, qempty0 + 8 * buf);
          commit_one(leader, sfull0 + 8 * (NS == 2 ? w : no & 1));
        };
        auto pv = [&](int w, int j) {
          const int i = tile_of(w, j);
          const unsigned at = base + v_pos(i, n), stage = at % STAGES;
          const unsigned no = (w ? done1 : done0) + j;
          ok = ok && warp_poll(pfull0 + 8 * (NS == 2 ? w : no & 1), (NS == 2 ? no : no >> 1) & 1,
                               p.timeout_ns);
          if (j == 0) ok = ok && warp_poll(ofree0 + 8 * w, unit_no & 1, p.timeout_ns);
          ok = ok && warp_poll(full0 + 8 * stage, (at / STAGES) & 1, p.timeout_ns);
          if (!ok) return;
          tc_fence_after();
          const uint64_t b = smem_desc(ring_s + stage * Shape::STAGE, KEYS * 128, 1024, 2);
#pragma unroll
          for (int kk = 0; kk < KEYS / 16; ++kk)
            mma_ts(leader, tmem + Shape::O_COL0 + w * D, s_of(w, no) + 8 * kk,
                   b + (uint64_t)(kk * (2048 >> 4)), pv_idesc, j > 0 || kk > 0);
          if (mode != kPair || w == 1) commit_one(leader, empty0 + 8 * stage);
          if (NS == 1) commit_one(leader, pvdone);
          if (j == (w ? n1 : n0) - 1) commit_one(leader, ofull0 + 8 * w);
        };
        if constexpr (NS == 1) {
          qk(0, 0);
          for (int j = 0; j < n && ok; ++j) {
            if (j + 1 < n) qk(0, j + 1);
            pv(0, j);
          }
        } else {
          // Every unit's phase of both ofree barriers is waited for, here or by
          // pv, but for an own unit without a second stream, the call's last:
          // nothing arrives for it (below).
          if (n1 == 0 && mode == kSplit) ok = warp_poll(ofree0 + 8, unit_no & 1, p.timeout_ns);
          // The streams in turn: the PV of a tile, then the QK of the next. One
          // site for each product keeps the code small.
#pragma unroll 1
          for (int t = -2; t < 2 * max(n0, n1) && ok; ++t) {
            const int w = t & 1, j = t >> 1, cnt = w ? n1 : n0;
            if (j >= 0 && j < cnt) pv(w, j);
            if (j + 1 < cnt) qk(w, j + 1);
          }
        }
        base += 2 * n;
        fills += mode == kSplit ? 1 : 1 + (n1 > 0);
        done0 += n0;
        done1 += n1;
      }
      if (!ok) {
        if (lane == 0) atomicOr(&px_status, kErrPxMma);
        commit_one(leader, drain);
        mbar_wait(drain, 0, kPxTimeoutNs);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPxSoftmaxRegs));
    // ------------------------------------------------- softmax, units' ends
    const int w = warp >> 2;                  // stream
    const int r = threadIdx.x & 127;          // tensor-memory lane
    const uint32_t lane_addr = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    unsigned base = 0, done = 0, ends0 = 0, ends1 = 0, meets = 0;
    bool ok = aligned;
    // The first round takes no unit: one key tile of whatever lies in S, run
    // through while the plan is made, so that the instructions are in the
    // caches when the first scores arrive (2 us less for them, measured). Its
    // weights go to S, which no product has written yet: the MMA warp waits
    // for all warps' ofree of this round before its first one.
    for (unsigned round = 0; ok; ++round) {
      const bool dry = round == 0;
      const unsigned unit_no = round - 1;
      const int seg = unit_no % kPxSegs;
      if (!dry && !(ok = warp_poll(ufull0 + 8 * seg, (unit_no / kPxSegs) & 1, p.timeout_ns))) break;
      const PxUnit& un = units[seg];
      int mode = kOwn, t0 = 1, t1 = 1, rows = 128, slot = 0, own = 1, last_valid = KEYS;
      if (!dry) {
        mode = un.mode;
        t0 = un.part[0].tiles;
        t1 = un.part[1].tiles;
        const int mine = mode == kOwn ? w : 0;
        rows = un.rows[mode == kPair ? w : 0];
        slot = un.part[mine].slot;
        last_valid = un.part[mine].last_valid;
        own = un.own;
        __syncwarp();
        if (lane == 0) mbar_arrive(uempty0 + 8 * seg);
        if (t0 == 0) break;
      }
      const int n0 = NS == 1 || mode != kSplit ? t0 : (t0 + 1) / 2;
      const int n1 = NS == 1 ? 0 : mode == kSplit ? t0 / 2 : mode == kPair ? t0 : t1;
      const int n = mode == kPair ? t0 : n0 + n1;
      const int mine = w ? n1 : n0;
      const int row = r - (mode == kOwn && w && !dry ? own_shift : 0);   // of the query tile
      // Warps without rows only keep step.
      const bool active = __any_sync(0xffffffffu, row >= 0 && row < rows);
      float m = -INFINITY, l = 0.0f;
      for (int j = 0; j < mine; ++j) {
        const unsigned no = done + j;
        const int sb = NS == 2 ? w : no & 1;
        if (!dry && !(ok = warp_poll(sfull0 + 8 * sb, (NS == 2 ? no : no >> 1) & 1, p.timeout_ns)))
          break;
        tc_fence_after();
        const int i = NS == 1 || mode == kPair ? j : turn(w, j, n0, n1);
        const int valid = (mode == kSplit ? i == n - 1 : j == mine - 1) ? last_valid : KEYS;
        if (valid < KEYS && (mode != kPair || w == 0)) {
          // V rows past the length may hold NaN: zeroed before the product.
          const unsigned at = base + v_pos(i, n), stage = at % STAGES;
          if (!(ok = warp_poll(full0 + 8 * stage, (at / STAGES) & 1, p.timeout_ns))) break;
          uint8_t* v = smem + Shape::QBUF * Shape::QBYTES + stage * Shape::STAGE;
          const int line = (KEYS - valid) * 8;   // 16-byte pieces of one part
          for (int t = r; t < line * PARTS; t += 128) {
            const int part = quick_div(t, line), c = t - part * line;
            *reinterpret_cast<uint4*>(v + part * KEYS * 128 + valid * 128 + c * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        if (active) {
          const uint32_t s_addr = tmem + lane_addr + Shape::S_COL * sb;
          // Loops over 64 keys, S read twice: unrolled over 128 the code of a
          // tile is past what a scheduler's instruction cache feeds, and the
          // fetches cost more than the second read of tensor memory.
          if (valid < KEYS || p.negate) {
            // Keys past the length, and a negative scale, in S itself.
#pragma unroll 1
            for (int c0 = 0; c0 < KEYS; c0 += 16) {
              float s[16];
              tmem_ld16_nowait(s_addr + c0, s);
              tmem_wait_ld();
              hold<16>(s);
#pragma unroll
              for (int c = 0; c < 16; ++c)
                s[c] = c0 + c < valid ? (p.negate ? -s[c] : s[c]) : -INFINITY;
              tmem_st16(s_addr + c0, reinterpret_cast<const uint32_t*>(s));
            }
            tmem_wait_st();
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
          for (int c0 = 0; c0 < KEYS; c0 += 64) {
            float s[64];
            tmem_ld32(s_addr + c0, s);
            tmem_ld32(s_addr + c0 + 32, s + 32);
            tmem_wait_ld();
            hold<64>(s);
#pragma unroll
            for (int c = 0; c < 64; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], s[c + e], s[c + 4 + e]);
          }
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
          if (j == 0) {
            m = top == -INFINITY ? -1e30f : top;   // nothing finite yet: weights of 0
          } else if (__any_sync(0xffffffffu, row >= 0 && row < rows && top > m + kPxGrow)) {
            // Each row by itself: lanes without a row hold anything, and must
            // not move the others' maxima.
            // The previous tiles' products are done: S of this tile was
            // multiplied after them, or (one stream) the wait below.
            if (NS == 1) {
              if (!(ok = warp_poll(pvdone, (no - 1) & 1, p.timeout_ns))) break;
              tc_fence_after();
            }
            const float now = top > m + kPxGrow ? top : m, a = ex2(m - now);
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
#pragma unroll 1
          for (int c0 = 0; c0 < KEYS; c0 += 64) {
            float s[64];
            uint32_t w16[32];
            tmem_ld32(s_addr + c0, s);
            tmem_ld32(s_addr + c0 + 32, s + 32);
            tmem_wait_ld();
            hold<64>(s);
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              float x, y;
              fma2(s[c], s[c + 1], qscale, qscale, shift, shift, x, y);
              x = ex2(x);
              y = ex2(y);
              add2(sum[c & 2], sum[(c & 2) + 1], x, y);
              w16[c / 2] = pack2<Tag>(x, y);
            }
            tmem_st32(s_addr + c0 / 2, w16);   // over scores that have been read
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (!dry && lane == 0) mbar_arrive(pfull0 + 8 * sb);
      }
      if (!ok) break;
      // The unit's end: O, m and l to its slot. A single query tile's two
      // streams (kSplit) are merged here and each warpgroup writes half of the
      // columns; else a stream writes its own rows.
      const bool merge = NS == 2 && mode == kSplit;
      if (!dry) {
        done += mine;
        if (n0 > 0 && (w == 0 || mode == kSplit)) ok = warp_poll(ofull0, ends0 & 1, p.timeout_ns);
        if (n1 > 0 && (w == 1 || merge)) ok = ok && warp_poll(ofull0 + 8, ends1 & 1, p.timeout_ns);
        if (!ok) break;
        ends0 += n0 > 0;
        ends1 += n1 > 0;
        base += 2 * n;
      }
      tc_fence_after();
      float a0 = 1.0f, a1 = 0.0f;
      if (merge) {
        if (mine > 0) ml[128 * w + r] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(meet);
        if (!(ok = warp_poll(meet, meets & 1, p.timeout_ns))) break;
        ++meets;
        if (n1 > 0) {
          const float2 x = ml[r], y = ml[128 + r];
          const float top = fmaxf(x.x, y.x);
          a0 = ex2(x.x - top);
          a1 = ex2(y.x - top);
          m = top;
          l = x.y * a0 + y.y * a1;
        }
      }
      if (active && !dry && (mode == kSplit || mine > 0)) {
        const bool live = row >= 0 && row < rows;
        const int stride = own ? p.G : 128;
        const size_t tile = own ? slot : static_cast<size_t>(slot) * NS + (mode == kPair ? w : 0);
        float4* dst = reinterpret_cast<float4*>(own ? p.own_o : p.prefix_o) + tile * (D / 4) * stride;
        float2* dst_ml = (own ? p.own_ml : p.prefix_ml) + tile * stride;
        const int c_begin = mode == kSplit ? w * (D / 2) : 0;
        const int c_end = mode == kSplit ? c_begin + D / 2 : D;
        const uint32_t o_addr = tmem + lane_addr + Shape::O_COL0 + (mode == kSplit ? 0 : w * D);
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 32) {
          float o[32];
          tmem_ld32(o_addr + c, o);
          if (merge && n1 > 0) {
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
          }
          if (live) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              __stcg(dst + static_cast<size_t>((c + e) / 4) * stride + row,
                     make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]));
          }
        }
        if (live && (mode != kSplit || w == 0)) __stcg(dst_ml + row, make_float2(m, l));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {   // 8 arrivals a barrier: all warps once, or a stream's own twice
        if (mode == kSplit) {
          mbar_arrive(ofree0);
          mbar_arrive(ofree0 + 8);
        } else if (dry || mine > 0) {
          // Warps of a stream that has nothing to do wait for nothing. Were they
          // to arrive, they could complete this phase before the MMA warp has
          // seen the one before, and its wait, for a parity, would never end.
          mbar_arrive(ofree0 + 8 * w);
          mbar_arrive(ofree0 + 8 * w);
        }
      }
    }
    if (!ok && lane == 0) atomicOr(&px_status, kErrPxSoftmax);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kPxMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512)
                 : "memory");
  }
}

// out row = sum over its slots of 2^(m_s - M) O_s / sum of 2^(m_s - M) l_s, the
// prefix's splits first, then the sequence's own, with a running maximum. A
// CTA takes 128 of the (row, 4 columns) of one sequence and KV head, a thread
// one. A row may have dozens of slots, and a thread waits for L2 at every step:
// it takes U slots a step, 8 where all CTAs fit on the SMs at once (five an SM;
// 16 sequences behind 8192 rows: 25 us, with 4 slots 28), 4 where they come in
// waves, of which more fit then (256 behind 32768, pairs cut in 5: 295 us, with 8
// slots 299; uncut, as the plan has it now, 289 with 4).
constexpr int kPxCombineThreads = 128;

template <typename Tag, int D, int U>
__global__ void __launch_bounds__(kPxCombineThreads)
    gqa_prefix_combine_kernel(const __grid_constant__ PrefixParams p) {
  using Shape = PxShape<D>;
  const int parts = (p.G * (D / 4) + kPxCombineThreads - 1) / kPxCombineThreads;
  const int bh = blockIdx.x / parts, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int x = (blockIdx.x - bh * parts) * kPxCombineThreads + threadIdx.x;
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) p.head->next = 0;   // for the next call
  const int own_tiles = p.head->own_tiles;
  const int own_base = p.max_blocks > 0 ? p.head->own_base[b] : 0;
  const int own_len = PxPlan<D>::own_len(p, b);
  bool in = false;
  if (lane < p.P) {
    const PxGroup& g = p.head->group[lane];
    in = b >= g.begin && b < g.end && g.splits > 0;
  }
  const int group = __ffs(__ballot_sync(0xffffffffu, in)) - 1;
  if (x >= p.G * (D / 4)) return;
  const int g = x % p.G, c = x / p.G;
  float top = -INFINITY, sum = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  // The slots, prefix's first: n0 of 128 rows, `step` tiles apart, then n1 of G rows.
  const float4 *o0 = nullptr, *o1 = nullptr;
  const float2 *m0 = nullptr, *m1 = nullptr;
  int n0 = 0, n1 = 0;
  size_t step = 0;
  if (group >= 0) {
    const PxGroup gr = p.head->group[group];
    const int t = quick_div(b - gr.begin, p.TB);
    const size_t unit = gr.base + static_cast<size_t>(h) * gr.splits * gr.nq + (gr.pair ? t / 2 : t);
    const size_t tile = unit * Shape::NS + (gr.pair ? t & 1 : 0);
    const int row = (b - gr.begin - t * p.TB) * p.G + g;
    n0 = gr.splits;
    step = static_cast<size_t>(gr.nq) * Shape::NS * 128;
    o0 = reinterpret_cast<const float4*>(p.prefix_o) + (tile * (D / 4) + c) * 128 + row;
    m0 = p.prefix_ml + tile * 128 + row;
  }
  if (own_len > 0) {
    n1 = quick_div(PxPlan<D>::tiles_of(own_len) + own_tiles - 1, own_tiles);
    const size_t tile = own_base + static_cast<size_t>(h) * n1;
    o1 = reinterpret_cast<const float4*>(p.own_o) + (tile * (D / 4) + c) * p.G + g;
    m1 = p.own_ml + tile * p.G + g;
  }
  for (int s = 0; s < n0 + n1; s += U) {
    float2 m[U];
    float4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      m[i] = make_float2(-INFINITY, 0.0f);
      v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (s + i < n0 + n1) {
        const bool own = s + i >= n0;
        const size_t at = own ? static_cast<size_t>(s + i - n0) * p.G : (s + i) * step;
        m[i] = __ldcg((own ? m1 : m0) + at);
        v[i] = __ldcg((own ? o1 : o0) + at * (D / 4));
      }
    }
    float now = top;
#pragma unroll
    for (int i = 0; i < U; ++i) now = fmaxf(now, m[i].x);
    const float old = ex2(top - now);
    top = now;
    sum *= old;
    acc.x *= old; acc.y *= old; acc.z *= old; acc.w *= old;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float a = ex2(m[i].x - now);
      sum = fmaf(a, m[i].y, sum);
      acc.x = fmaf(a, v[i].x, acc.x);
      acc.y = fmaf(a, v[i].y, acc.y);
      acc.z = fmaf(a, v[i].z, acc.z);
      acc.w = fmaf(a, v[i].w, acc.w);
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const uint2 y = make_uint2(pack2<Tag>(acc.x * inv, acc.y * inv), pack2<Tag>(acc.z * inv, acc.w * inv));
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) +
                            (static_cast<size_t>(b) * p.Hq + h * p.G + g) * D + 4 * c) = y;
}

}  // namespace gqa_av
