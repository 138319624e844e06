// Kernels that feed a paged KV cache on sm_103a (GB300): block tables and
// slots from request lengths, and norm + rotation + cache write of a step's
// tokens. The operations are stated in include/gqa_kv.h.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gqa_av_kernel.cuh"
#include "gqa_pack.cuh"

namespace gqa_av {

// ---------------------------------------------------------------------------
// Block tables and slots
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 512;
constexpr int kTabMaxB = 8192;         // requests: 12 B of shared memory each
constexpr int kTabTokensPerCta = 2048;

struct TablesParams {
  const int32_t* cached;       // [B]
  const int32_t* fresh;        // [B] new tokens
  const int32_t* pos_base;     // [B] or null
  const int32_t* free_list;    // [n_free]
  const int32_t* free_count;   // [1]
  int32_t* table;              // [B, max_blocks]
  int32_t* seq_lens;           // [B]
  int32_t* token_start;        // [B + 1]
  int32_t* slots;              // [T]
  int32_t* positions;          // [T]
  int32_t* free_left;          // [1]
  int B, T, max_blocks, n_free, bs, num_blocks;
};

__device__ __forceinline__ long long warp_scan(long long x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Inclusive sums of x over the block; `total` gets the block's sum. `part` is
// shared memory of kTabThreads / 32 entries, free for reuse on return.
__device__ __forceinline__ long long block_scan(long long x, long long* part, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long incl = warp_scan(x);
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kTabThreads / 32; ++i) {
    const long long y = part[i];
    before += i < warp ? y : 0;
    all += y;
  }
  *total = all;
  __syncthreads();
  return before + incl;
}

// Every CTA scans all requests (at most 8192, two loads each) into shared
// memory and then maps its own run of tokens, so one launch needs no exchange
// between CTAs. The token whose row opens a new block writes the table entry:
// a new block's first row is always a new token. The sums run in 64 bits.
// Bound by latency: launch, lengths, table or list entry (4.5 us a call for 256
// requests of one token, 7.2 for 96 requests with 131 thousand tokens).
__global__ void __launch_bounds__(kTabThreads) gqa_kv_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t tab_smem[];
  int32_t* start = tab_smem;                 // [B] first token of each request
  int32_t* len = start + p.B;                // [B] cached rows
  int32_t* take = len + p.B;                 // [B] free-list blocks before it, -1: not served
  __shared__ long long part[kTabThreads / 32];
  __shared__ int taken;                      // free-list blocks that served requests take
  if (threadIdx.x == 0) taken = 0;

  grid_dependency_wait();
  grid_launch_dependents();
  const int n_free = min(max(*p.free_count, 0), p.n_free);
  long long tokens = 0, blocks = 0;
  for (int b0 = 0; b0 < p.B; b0 += kTabThreads) {
    const int b = b0 + threadIdx.x;
    const bool in = b < p.B;
    const long long have = in ? max(p.cached[b], 0) : 0;
    const long long more = in ? max(p.fresh[b], 0) : 0;
    const long long held = (have + p.bs - 1) / p.bs;
    const long long want = (have + more + p.bs - 1) / p.bs;
    long long sum;
    const long long t1 = tokens + block_scan(more, part, &sum);
    tokens += sum;
    const bool fits = want <= p.max_blocks && t1 <= p.T;
    const long long need = fits ? want - held : 0;
    const long long upto = blocks + block_scan(need, part, &sum);
    blocks += sum;
    const bool served = fits && (need == 0 || upto <= n_free);
    // Served needs are a leading part of the running sum (a later request's
    // sum is larger), so list positions need no second scan, and the blocks
    // taken are the largest served sum.
    if (served && need > 0) atomicMax(&taken, static_cast<int>(upto));
    if (in) {
      const int32_t t0 = static_cast<int32_t>(min(t1 - more, 0x7fffffffLL));
      start[b] = t0;
      len[b] = static_cast<int32_t>(have);
      take[b] = served ? static_cast<int32_t>(min(upto - need, 0x7fffffffLL)) : -1;
      if (blockIdx.x == 0) {
        p.token_start[b] = t0;
        p.seq_lens[b] = static_cast<int32_t>(min(have + (served ? more : 0), 0x7fffffffLL));
      }
    }
  }
  const int32_t end = static_cast<int32_t>(min(tokens, 0x7fffffffLL));
  __syncthreads();
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    p.token_start[p.B] = end;
    *p.free_left = n_free - taken;
  }

  const int stop = min(p.T - static_cast<int>(blockIdx.x) * kTabTokensPerCta, kTabTokensPerCta);
  for (int i = threadIdx.x; i < stop; i += kTabThreads) {
    const int t = blockIdx.x * kTabTokensPerCta + i;
    int slot = -1, pos = 0;
    if (t < end) {
      int lo = 0, hi = p.B;  // the last request with start <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int b = lo;
      const int held = static_cast<int>((static_cast<long long>(len[b]) + p.bs - 1) / p.bs);
      const long long row = static_cast<long long>(len[b]) + t - start[b];
      pos = static_cast<int>(row + (p.pos_base ? p.pos_base[b] : 0));
      if (take[b] >= 0) {
        const int col = static_cast<int>(row / p.bs);
        const int in_block = static_cast<int>(row - static_cast<long long>(col) * p.bs);
        int32_t* entry = p.table + static_cast<size_t>(b) * p.max_blocks + col;
        int block;
        if (col < held) {
          block = *entry;
        } else {
          block = p.free_list[n_free - 1 - (take[b] + col - held)];
          if (in_block == 0) *entry = block;
        }
        if (block >= 0 && block < p.num_blocks) slot = block * p.bs + in_block;
      }
    }
    p.slots[t] = slot;
    p.positions[t] = pos;
  }
}

// ---------------------------------------------------------------------------
// Norm, rotation and cache write
// ---------------------------------------------------------------------------
constexpr int kRopeWarps = 8;
constexpr int kRopeMaxPairs = 128;

struct RopeParams {
  const void *q, *k, *v;        // 16-bit, token strides below
  long long q_stride, k_stride, v_stride;
  const int32_t* positions;     // [axes, T]
  const float* inv_freq;        // [pairs]
  const void *qw, *kw;          // [D] 16-bit or null
  const int32_t* slots;         // [T]
  void* q_out;                  // [T, Hq, D]
  void *k_pool, *v_pool;        // [rows, Hkv, D]
  int T, Hq, Hkv, D, pairs;
  int rows;                     // num_blocks * block_size
  int sec_end[4];               // first pair past each axis
  float eps, w_offset;
  int chunks;                   // parts that a token's heads are cut into
  int iters;                    // head steps of one part
};

// The rotation of one pair at `pos`. turn64 = inv_freq / (2 pi) modulo one
// turn in units of 2^-64 turns: the product with the position wraps in 64-bit
// integers, so the reduction is exact whatever the position. Its top 32 bits,
// as a signed fraction of a turn, round to fp32 with 2^-25 of a half-turn.
__device__ __forceinline__ void pair_rotation(unsigned long long turn64, int pos, float* c,
                                              float* s) {
  const unsigned long long x = turn64 * static_cast<unsigned long long>(static_cast<long long>(pos));
  const float half_turns = static_cast<float>(static_cast<int32_t>(x >> 32)) * 4.656612873077393e-10f;
  sincospif(half_turns, s, c);
}

// A warp takes part of a token's heads, 32 / L heads a step. A lane owns both
// elements of four pairs of a head, the same ones in every step: four and four
// elements half a rotation apart, or eight adjacent ones (interleaved), so a
// rotation needs no other lane, and cos and sin are made once a token and part.
// Elements past the rotation are dealt out the same way and left alone. The
// squares are summed by shuffles inside the head's L lanes. The loads of the
// next kAhead steps are under way while a step is worked on. Short inputs are
// bound by latency (3 us for one token), long ones by HBM and, nearly as much,
// by instruction issue (186 instructions a step of 512 bytes, 75 % of the issue
// slots). Measured at 16384 tokens of 32 + 8 + 8 heads of 128, bf16 (403 MB): 84
// us; 141 with eight adjacent elements a lane, whose mates came by shuffles, and
// one step's loads at a time. More loads ahead, next tokens' positions ahead and
// addresses kept as pointers all measured slower: each costs registers, and with
// more than 80 the third CTA of an SM (separate halves with fp32 queries take 86
// to 88 and run two).
template <typename Tag, int L, bool kInterleaved, bool kQ32>
__global__ void __launch_bounds__(32 * kRopeWarps) gqa_kv_rope_kernel(const RopeParams p) {
  __shared__ unsigned long long turn[kRopeMaxPairs];
  constexpr int kHeads = 32 / L;                // heads a step
  constexpr int kAhead = 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int li = lane % L, sub = lane / L;
  grid_dependency_wait();
  grid_launch_dependents();
  for (int i = threadIdx.x; i < p.pairs; i += blockDim.x) {
    const double f = static_cast<double>(p.inv_freq[i]) * 0.15915494309189534561;  // 1 / (2 pi)
    turn[i] = static_cast<unsigned long long>((f - floor(f)) * 18446744073709551616.0);
  }
  // Elements e0 .. e0 + 3 and e1 .. e1 + 3; of pairs 4 li .. 4 li + 3 where rotated.
  const bool live = 8 * li < p.D;
  const bool rot = 4 * li < p.pairs;
  int e0 = 8 * li, e1 = e0 + 4;
  if (!kInterleaved) {
    e0 = rot ? 4 * li : p.pairs + 4 * li;
    e1 = rot ? p.pairs + 4 * li : e0 + p.D / 2 - p.pairs;
  }
  const int all = p.Hq + 2 * p.Hkv;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  auto load8 = [&](const void* base, size_t at) {   // at: the head's first element
    const char* src = static_cast<const char*>(base) + 2 * at;
    if constexpr (kInterleaved) return __ldcs(reinterpret_cast<const uint4*>(src + 2 * e0));
    const uint2 a = __ldcs(reinterpret_cast<const uint2*>(src + 2 * e0));
    const uint2 b = __ldcs(reinterpret_cast<const uint2*>(src + 2 * e1));
    return make_uint4(a.x, a.y, b.x, b.y);
  };
  uint4 qw = make_uint4(0u, 0u, 0u, 0u), kw = qw;
  if (live && p.qw) qw = load8(p.qw, 0);
  if (live && p.kw) kw = load8(p.kw, 0);
  __syncthreads();

  const long long jobs = static_cast<long long>(p.T) * p.chunks;
  for (long long job = static_cast<long long>(blockIdx.x) * kRopeWarps + warp; job < jobs;
       job += static_cast<long long>(gridDim.x) * kRopeWarps) {
    const int t = static_cast<int>(job / p.chunks);
    const int first = static_cast<int>(job - static_cast<long long>(t) * p.chunks) * p.iters;
    const int last = min(first + p.iters, (all + kHeads - 1) / kHeads);
    auto fetch = [&](int it) {
      const int h = it * kHeads + sub;
      uint4 raw = make_uint4(0u, 0u, 0u, 0u);
      if (live && h < all && it < last) {
        const bool is_q = h < p.Hq, is_k = h < p.Hq + p.Hkv;
        const int head = is_q ? h : h - p.Hq - (is_k ? 0 : p.Hkv);
        raw = load8(is_q ? p.q : is_k ? p.k : p.v,
                    (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride) * t +
                        static_cast<long long>(head) * p.D);
      }
      return raw;
    };
    uint4 next[kAhead];
#pragma unroll
    for (int a = 0; a < kAhead; ++a) next[a] = fetch(first + a);
    const int slot = p.slots[t];
    const bool keep = slot >= 0 && slot < p.rows;
    float c[4], s[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      c[e] = 1.0f;
      s[e] = 0.0f;
      if (rot) {
        const int i = 4 * li + e;
        const int axis = (i >= p.sec_end[0]) + (i >= p.sec_end[1]) + (i >= p.sec_end[2]);
        pair_rotation(turn[i], p.positions[static_cast<size_t>(axis) * p.T + t], &c[e], &s[e]);
      }
    }
    for (int it0 = first; it0 < last; it0 += kAhead) {
      uint4 now[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        now[a] = next[a];
        next[a] = fetch(it0 + kAhead + a);
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int it = it0 + a;
        if (it >= last) break;
        const int h = it * kHeads + sub;
        const bool is_q = h < p.Hq;
        const bool is_k = !is_q && h < p.Hq + p.Hkv;
        uint4 raw = now[a];
        // Steps of values only (the last ones) are copied as they are.
        if (it * kHeads < p.Hq + p.Hkv) {
          float x[8];
          widen8(Tag{}, raw, x);
          if (p.qw || p.kw) {
            float ss = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (is_q ? p.qw != nullptr : p.kw != nullptr) {
              const float r = rsqrtf(fmaf(ss, inv_d, p.eps));
              float g[8];
              widen8(Tag{}, is_q ? qw : kw, g);
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] = x[e] * r * (g[e] + p.w_offset);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& u = x[kInterleaved ? 2 * e : e];
            float& v = x[kInterleaved ? 2 * e + 1 : e + 4];
            const float y = u * c[e] - v * s[e];
            v = v * c[e] + u * s[e];
            u = y;
          }
          if (kQ32 && is_q && live) {
            float* dst = static_cast<float*>(p.q_out) + (static_cast<size_t>(t) * p.Hq + h) * p.D;
            *reinterpret_cast<float4*>(dst + e0) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(dst + e1) = make_float4(x[4], x[5], x[6], x[7]);
          }
          if (is_q || is_k)
            raw = make_uint4(pack2<Tag>(x[0], x[1]), pack2<Tag>(x[2], x[3]), pack2<Tag>(x[4], x[5]),
                             pack2<Tag>(x[6], x[7]));
        }
        if (live && h < all && (is_q ? !kQ32 : keep)) {
          char* base = static_cast<char*>(is_q ? p.q_out : is_k ? p.k_pool : p.v_pool);
          const size_t row = is_q ? static_cast<size_t>(t) * p.Hq + h
                                  : static_cast<size_t>(slot) * p.Hkv + (h - p.Hq - (is_k ? 0 : p.Hkv));
          char* dst = base + 2 * row * p.D;
          if constexpr (kInterleaved) {
            *reinterpret_cast<uint4*>(dst + 2 * e0) = raw;
          } else {
            *reinterpret_cast<uint2*>(dst + 2 * e0) = make_uint2(raw.x, raw.y);
            *reinterpret_cast<uint2*>(dst + 2 * e1) = make_uint2(raw.z, raw.w);
          }
        }
      }
    }
  }
}

}  // namespace gqa_av
