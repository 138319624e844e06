// Kernels for the life of a paged KV cache's blocks on sm_103a: forking
// requests, keeping accepted drafts, releasing blocks. The operations are
// stated in include/gqa_kv.h.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_kv_kernel.cuh"

namespace gqa_av {

constexpr int kPagePools = 256;        // pool pointers in a launch's parameters
constexpr int kPageMaxB = 8192;        // rows of a block table, and forks

struct PoolList {
  uint8_t* at[kPagePools];
};

// ---------------------------------------------------------------------------
// Fork
// ---------------------------------------------------------------------------
constexpr int kForkThreads = kTabThreads;
constexpr int kForkPiece = 4096;       // bytes that a warp copies at a time

struct ForkParams {
  PoolList pools;
  const int32_t *parent, *child;       // [N]
  int32_t* table;                      // [B, max_blocks]
  int32_t* seq_lens;                   // [B]
  int32_t* shares;                     // [num_blocks]
  const int32_t* free_list;            // [n_free]
  const int32_t* free_count;           // [1]
  int32_t* fork_block;                 // [N]
  int32_t* free_left;                  // [1]
  long long row_bytes;
  int n_pools, N, B, max_blocks, n_free, bs, num_blocks;
};

// Every CTA goes through all forks (at most 8192) in shared memory and then
// takes its own part of the table rows and of the copies, so one launch needs
// no exchange between CTAs: rows that are read (parents') are never written.
// The rows that a partial block holds are one run of bytes in a pool, cut into
// pieces of 4 KB, a warp each, eight 16-byte loads a lane under way.
// Bound by HBM and L2 where there is something to copy (192 forks of 24 partial
// blocks, 15 rows of 2 KB each on average, in 32 pools: 44 us for 370 MB read and
// written, of which eight forks share what they read), else by latency: launch,
// lengths, table.
__global__ void __launch_bounds__(kForkThreads)
    gqa_kv_fork_kernel(const __grid_constant__ ForkParams p) {
  extern __shared__ int32_t fork_smem[];
  int32_t* first = fork_smem;          // [B] first fork that names a row as its child
  int32_t* is_parent = first + p.B;    // [B]
  int32_t* block = is_parent + p.B;    // [N] block of the copy; -1: none, -2: not served
  int32_t* lens = block + p.N;         // [N] parents' rows
  __shared__ long long part[kForkThreads / 32];
  __shared__ int taken;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) taken = 0;
  for (int b = tid; b < p.B; b += kForkThreads) {
    first[b] = p.N;
    is_parent[b] = 0;
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();
  const long long cap = static_cast<long long>(p.max_blocks) * p.bs;
  for (int f = tid; f < p.N; f += kForkThreads) {
    const int a = p.parent[f], c = p.child[f];
    if (a >= 0 && a < p.B) {
      is_parent[a] = 1;
      lens[f] = static_cast<int>(min(max(static_cast<long long>(p.seq_lens[a]), 0LL), cap));
    } else {
      lens[f] = -1;
    }
    if (c >= 0 && c < p.B) atomicMin(&first[c], f);
  }
  __syncthreads();
  const int n_free = min(max(*p.free_count, 0), p.n_free);
  long long asked = 0;
  for (int f0 = 0; f0 < p.N; f0 += kForkThreads) {
    const int f = f0 + tid;
    bool good = false;
    int need = 0;
    if (f < p.N) {
      const int c = p.child[f];
      good = lens[f] >= 0 && c >= 0 && c < p.B && first[c] == f && !is_parent[c];
      need = good && lens[f] % p.bs != 0;
    }
    long long sum;
    const long long upto = asked + block_scan(need, part, &sum);
    asked += sum;
    if (f < p.N) {
      const bool served = good && (!need || upto <= n_free);
      block[f] = !served ? -2 : need ? p.free_list[n_free - upto] : -1;
      if (served && need) atomicMax(&taken, static_cast<int>(upto));
      // A free-list entry below 0 is no block, and must not read as one of the marks.
      if (served && need && block[f] < 0) block[f] = 0x7fffffff;
    }
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0) *p.free_left = n_free - taken;

  // Table rows, a CTA each.
  for (int f = blockIdx.x; f < p.N; f += gridDim.x) {
    const int mine = block[f];
    if (tid == 0) p.fork_block[f] = mine;
    if (mine == -2) continue;
    const int a = p.parent[f], c = p.child[f], full = lens[f] / p.bs;
    const int32_t* from = p.table + static_cast<size_t>(a) * p.max_blocks;
    int32_t* to = p.table + static_cast<size_t>(c) * p.max_blocks;
    for (int j = tid; j < full; j += kForkThreads) {
      const int x = from[j];
      to[j] = x;
      if (x >= 0 && x < p.num_blocks) atomicAdd(&p.shares[x], 1);
    }
    if (tid == 0) {
      if (mine != -1) to[full] = mine;
      p.seq_lens[c] = lens[f];
    }
  }
  // Partial blocks: pieces (fork, pool, 4 KB), a warp each.
  const long long most = (static_cast<long long>(p.bs - 1) * p.row_bytes + kForkPiece - 1) / kForkPiece;
  const int pieces = static_cast<int>(max(1LL, most));
  const long long tasks = static_cast<long long>(p.N) * p.n_pools * pieces;
  const long long warps = static_cast<long long>(gridDim.x) * (kForkThreads / 32);
  for (long long t = static_cast<long long>(blockIdx.x) * (kForkThreads / 32) + (tid >> 5); t < tasks;
       t += warps) {
    const long long outer = t / pieces;
    const int piece = static_cast<int>(t - outer * pieces);
    const int pool = static_cast<int>(outer % p.n_pools), f = static_cast<int>(outer / p.n_pools);
    const int dst = block[f];
    if (dst < 0 || dst >= p.num_blocks) continue;
    const int len = lens[f], full = len / p.bs;
    const long long bytes = static_cast<long long>(len - full * p.bs) * p.row_bytes;
    const long long at = static_cast<long long>(piece) * kForkPiece;
    if (at >= bytes) continue;
    const int src = p.table[static_cast<size_t>(p.parent[f]) * p.max_blocks + full];
    if (src < 0 || src >= p.num_blocks) continue;
    const long long block_bytes = p.row_bytes * p.bs;
    const uint8_t* from = p.pools.at[pool] + src * block_bytes + at;
    uint8_t* to = p.pools.at[pool] + dst * block_bytes + at;
    const int n = static_cast<int>(min(bytes - at, static_cast<long long>(kForkPiece))) / 16;
    uint4 x[kForkPiece / 512];
#pragma unroll
    for (int i = 0; i < kForkPiece / 512; ++i)
      if (32 * i + lane < n) x[i] = reinterpret_cast<const uint4*>(from)[32 * i + lane];
#pragma unroll
    for (int i = 0; i < kForkPiece / 512; ++i)
      if (32 * i + lane < n) reinterpret_cast<uint4*>(to)[32 * i + lane] = x[i];
  }
}

// ---------------------------------------------------------------------------
// Keep
// ---------------------------------------------------------------------------
constexpr int kKeepWarps = 8;
// Rows read before they are written, and CTAs an SM: 64 paths in 48 pools of 2 KB
// rows are 1536 CTAs, two and a half waves (4 and 4: 7.4 us; 8 and 3: 8.8; 4 and 6,
// 42 registers: 8.2).
constexpr int kKeepRows = 4, kKeepCtas = 4;

struct KeepParams {
  PoolList pools;
  const int32_t* cached;               // [B]
  const int32_t* accepted;             // [B, W]
  const int32_t* count;                // [B]
  const int32_t* table;                // [B, max_blocks]
  const int32_t* seq_lens;             // [B]
  int32_t* kept;                       // [B]
  long long row_bytes;
  int n_pools, B, W, max_blocks, bs, num_blocks, parts;
};

// A warp takes 512 bytes of the rows of one request in one pool, a lane 16 of
// them, and moves them in ascending order: an accepted row never lies before
// its new place, so four rows read before they are written, and all rows after
// them, are still what they were. Lane i finds the i-th row's two places.
// Bound by latency (lengths, table, rows), or by HBM with many layers (one path in 4
// pools: 2.3 us; 64 paths in 48 pools, 22 MB moved: 7.4 us).
__global__ void __launch_bounds__(32 * kKeepWarps, kKeepCtas)
    gqa_kv_keep_kernel(const __grid_constant__ KeepParams p) {
  const int lane = threadIdx.x & 31;
  const unsigned warps = static_cast<unsigned>(p.n_pools) * p.parts;
  const long long task = static_cast<long long>(blockIdx.x) * kKeepWarps + (threadIdx.x >> 5);
  const int b = static_cast<int>(task / warps);
  grid_dependency_wait();
  grid_launch_dependents();
  if (b >= p.B) return;
  const unsigned in = static_cast<unsigned>(task - static_cast<long long>(b) * warps);
  const int pool = in / p.parts, part = in - pool * p.parts;
  const long long cap = static_cast<long long>(p.max_blocks) * p.bs;
  const long long have = min(max(static_cast<long long>(p.cached[b]), 0LL), cap);
  const long long end = min(static_cast<long long>(p.seq_lens[b]), cap);
  const int count = min(p.count[b], p.W);
  const int32_t* accepted = p.accepted + static_cast<size_t>(b) * p.W;
  const int32_t* table = p.table + static_cast<size_t>(b) * p.max_blocks;
  const long long col = static_cast<long long>(part) * 512 + lane * 16;
  const bool mine = col < p.row_bytes;
  uint8_t* base = p.pools.at[pool] + col;
  auto row_of = [&](long long c) {     // of the flattened pool, -1: none
    const int block = table[c / p.bs];
    return block >= 0 && block < p.num_blocks ? block * p.bs + static_cast<int>(c % p.bs) : -1;
  };
  int kept = 0, last = -1;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane;
    const int a = i < count ? accepted[i] : -1;
    int before = __shfl_up_sync(0xffffffffu, a, 1);
    if (lane == 0) before = last;
    last = __shfl_sync(0xffffffffu, a, 31);
    // The leading ones that ascend and have a row.
    const unsigned bad = __ballot_sync(0xffffffffu, !(i < count && a > before && have + a < end));
    const int n = bad ? __ffs(bad) - 1 : 32;
    int src = -1, dst = -1;
    if (lane < n && a != i) {
      src = row_of(have + a);
      dst = row_of(have + i);
    }
    for (int k = 0; k < n; k += kKeepRows) {
      uint4 x[kKeepRows];
      int to[kKeepRows];
#pragma unroll
      for (int e = 0; e < kKeepRows; ++e) {
        const int from = __shfl_sync(0xffffffffu, src, (k + e) & 31);
        to[e] = __shfl_sync(0xffffffffu, dst, (k + e) & 31);
        if (k + e >= n || from < 0 || !mine) to[e] = -1;
        if (to[e] >= 0) x[e] = *reinterpret_cast<const uint4*>(base + from * p.row_bytes);
      }
#pragma unroll
      for (int e = 0; e < kKeepRows; ++e)
        if (to[e] >= 0) *reinterpret_cast<uint4*>(base + to[e] * p.row_bytes) = x[e];
    }
    kept += n;
    if (n < 32) break;
  }
  if (in == 0 && lane == 0) p.kept[b] = static_cast<int>(have) + kept;
}

// ---------------------------------------------------------------------------
// Release
// ---------------------------------------------------------------------------
constexpr int kReleaseThreads = 1024;
constexpr int kReleaseEach = 4;        // entries that a thread has under way
// CTAs of one cluster where there are many entries: each gathers four bytes here
// and there, about one a cycle and SM (256 requests, 22 thousand entries: 16.8 us with
// 8 CTAs, 13.7 with 16).
constexpr int kReleaseCluster = 16, kReleasePortable = 8;
constexpr int kReleaseCache = 16384;   // block numbers that a CTA keeps in shared memory

struct ReleaseParams {
  const int32_t* table;                // [B, max_blocks]
  const int32_t *old_lens, *new_lens;  // [B]
  int32_t* shares;                     // [num_blocks] or null
  int32_t* free_list;                  // [n_free]
  const int32_t* free_count;           // [1]
  int32_t* free_left;                  // [1]
  int B, max_blocks, n_free, bs, num_blocks;
};

__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_read(const int* p, uint32_t rank) {
  uint32_t addr, x;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(addr) : "memory");
  return static_cast<int>(x);
}

// Inclusive sum over the CTA's 1024 threads on top of `carry`, which becomes the
// whole sum. `part` holds 32 ints.
__device__ __forceinline__ int release_scan(int x, int* carry, int* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int sums = part[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, sums, o);
    if (lane >= o) sums += y;
  }
  const int before = warp ? __shfl_sync(0xffffffffu, sums, (warp - 1) & 31) : 0;
  const int all = __shfl_sync(0xffffffffu, sums, 31);
  __syncthreads();
  const int incl = *carry + before + x;
  *carry += all;
  return incl;
}

// The released entries of all rows, in order e = 0 .. M - 1, are cut into one run
// a CTA of a single cluster. A block goes back when more of its owners let go
// than its share count allows, at the place of its first entry, so that the
// order does not depend on who was first:
//   1. each entry takes one off its block's count;
//   2. where that left less than 0, the block's smallest entry is found by a
//      minimum over codes that rise with the entry's number (in the count itself:
//      its value is no longer needed);
//   3. the entry that finds its own code there is the one; their places are a sum
//      over the cluster, and the count becomes 0.
// Bound by latency: five steps through L2 and the cluster's barriers between them
// (3 requests, one CTA: 6 us; 256 requests, 22 thousand entries: 13.7 us).
__global__ void __launch_bounds__(kReleaseThreads, 1)
    gqa_kv_release_kernel(const __grid_constant__ ReleaseParams p) {
  extern __shared__ int32_t release_smem[];
  int32_t* start = release_smem;               // [B + 1] first entry of each row
  int32_t* held = start + p.B + 1;             // [B] first released column
  int32_t* cache = held + p.B;                 // [kReleaseCache]
  __shared__ int part[32];
  __shared__ int winners;                      // of this CTA, read by the others
  __shared__ int sums[kReleaseEach][32];
  const int tid = threadIdx.x;
  const int rank = cluster_rank(), ctas = cluster_size();
  grid_dependency_wait();
  grid_launch_dependents();
  const int n_free = min(max(*p.free_count, 0), p.n_free);
  const long long cap = static_cast<long long>(p.max_blocks) * p.bs;
  int carry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kReleaseThreads) {
    const int b = b0 + tid;
    int n = 0, from = 0;
    if (b < p.B) {
      const long long old = min(max(static_cast<long long>(p.old_lens[b]), 0LL), cap);
      const long long now = min(max(static_cast<long long>(p.new_lens[b]), 0LL), old);
      from = static_cast<int>((now + p.bs - 1) / p.bs);
      n = static_cast<int>((old + p.bs - 1) / p.bs) - from;
    }
    const int upto = release_scan(n, &carry, part);
    if (b < p.B) {
      start[b] = upto - n;
      held[b] = from;
    }
  }
  if (tid == 0) start[p.B] = carry;
  __syncthreads();
  const int M = carry;
  const int per = (M + ctas - 1) / ctas;
  const int begin = min(rank * per, M), end = min(begin + per, M);
  auto lookup = [&](int e) {                   // entry e's block, -1: none
    if (e >= end) return -1;
    int lo = 0, hi = p.B;                      // the last row with start[b] <= e
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= e) lo = mid;
      else hi = mid;
    }
    const int x = p.table[static_cast<size_t>(lo) * p.max_blocks + held[lo] + e - start[lo]];
    return x >= 0 && x < p.num_blocks ? x : -1;
  };
  auto code = [&](int e) { return -0x40000000 - (M - e); };
  // Four entries a thread at a time, so that their loads are under way together:
  // e0, e0 + 1024, ...
  auto blocks_of = [&](int e0, int (&x)[kReleaseEach]) {
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) {
      const int e = e0 + k * kReleaseThreads;
      x[k] = e >= end ? -1 : e - begin < kReleaseCache ? cache[e - begin] : lookup(e);
    }
  };
  auto counts_of = [&](const int (&x)[kReleaseEach], int (&v)[kReleaseEach]) {
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) v[k] = x[k] >= 0 ? __ldcg(&p.shares[x[k]]) : 0;
  };
  constexpr int kWave = kReleaseEach * kReleaseThreads;
  // 1.
  for (int e0 = begin + tid; e0 < end; e0 += kWave) {
    int x[kReleaseEach];
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) x[k] = lookup(e0 + k * kReleaseThreads);
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) {
      const int e = e0 + k * kReleaseThreads;
      if (e < end && e - begin < kReleaseCache) cache[e - begin] = x[k];
      if (x[k] >= 0 && p.shares) atomicSub(&p.shares[x[k]], 1);
    }
  }
  if (p.shares) {
    __threadfence();
    cluster_barrier();
    // 2.
    for (int e0 = begin + tid; e0 < end; e0 += kWave) {
      int x[kReleaseEach], v[kReleaseEach];
      blocks_of(e0, x);
      counts_of(x, v);
#pragma unroll
      for (int k = 0; k < kReleaseEach; ++k)
        if (v[k] < 0) atomicMin(&p.shares[x[k]], code(e0 + k * kReleaseThreads));
    }
    __threadfence();
    cluster_barrier();
  }
  // 3. Bit k: the thread's k-th entry from e0 on is the one.
  auto goes = [&](int e0) {
    int x[kReleaseEach], v[kReleaseEach];
    blocks_of(e0, x);
    if (p.shares) counts_of(x, v);
    unsigned bits = 0;
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k)
      if (x[k] >= 0 && (!p.shares || v[k] == code(e0 + k * kReleaseThreads))) bits |= 1u << k;
    return bits;
  };
  int count = 0;
  unsigned bits = 0;
  for (int e0 = begin + tid; e0 < end; e0 += kWave) {
    bits = goes(e0);
    count += __popc(bits);
  }
  carry = 0;
  release_scan(count, &carry, part);
  if (tid == 0) winners = carry;
  cluster_barrier();
  const int lane = tid & 31, warp = tid >> 5;
  const int n = lane < ctas ? cluster_read(&winners, lane) : 0;   // at most 32 CTAs
  int at = n_free + __reduce_add_sync(0xffffffffu, lane < rank ? n : 0);
  const int all = n_free + __reduce_add_sync(0xffffffffu, n);
  // Places: all entries of the first 1024, of the second, ... A count that becomes 0
  // is the code of no entry: nobody else is misled.
  const bool once = end - begin <= kWave;      // the bits are still at hand
  for (int e0 = begin; e0 < end; e0 += kWave) {
    if (!once) bits = goes(e0 + tid);
    unsigned votes[kReleaseEach];
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) {
      votes[k] = __ballot_sync(0xffffffffu, bits >> k & 1);
      if (lane == 0) sums[k][warp] = __popc(votes[k]);
    }
    __syncthreads();
    int x[kReleaseEach];
    blocks_of(e0 + tid, x);
#pragma unroll
    for (int k = 0; k < kReleaseEach; ++k) {
      const int s = sums[k][lane];
      const int to = at + __reduce_add_sync(0xffffffffu, lane < warp ? s : 0) +
                     __popc(votes[k] & ((1u << lane) - 1u));
      at += __reduce_add_sync(0xffffffffu, s);
      if (bits >> k & 1) {
        if (to < p.n_free) p.free_list[to] = x[k];
        if (p.shares) p.shares[x[k]] = 0;
      }
    }
    __syncthreads();
  }
  if (rank == 0 && tid == 0) *p.free_left = min(all, p.n_free);
  cluster_barrier();   // nobody leaves while its count may be read
}

}  // namespace gqa_av
