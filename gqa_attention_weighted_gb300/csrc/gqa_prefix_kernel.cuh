// Decode attention over a paged KV cache with shared prefixes, sm_103a. The
// operation is stated in include/gqa_prefix.h.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "gqa_av_kernel.cuh"
#include "gqa_pack.cuh"

namespace gqa_av {

struct PrefixParams {
  const void *q, *k_pool, *v_pool;
  const int32_t *prefix_table, *prefix_lens, *group_start, *block_table, *seq_lens;
  void* out;
  int B, P, Hq, Hkv, G;
  int bs, num_blocks, max_pblocks, max_blocks;
  float qscale;                 // scale * log2(e)
};

// One CTA per (sequence, query head): its warps take every fourth key, a lane
// D / 32 elements of it, with a running maximum and sum; the warps' results
// are merged at the end. fp32 throughout, the weights not rounded.
template <typename Tag, int D>
__global__ void __launch_bounds__(128) gqa_prefix_simple_kernel(const PrefixParams p) {
  constexpr int E = D / 32;
  __shared__ float s_m[4], s_l[4], s_o[4][D];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, kv = h / p.G;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_launch_dependents();
  auto load = [&](const void* base, size_t at, float (&x)[E]) {
    const uint16_t* src = static_cast<const uint16_t*>(base) + at + E * lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint16_t v = src[e];
      if constexpr (std::is_same<Tag, Bf16Tag>::value) x[e] = __uint_as_float(uint32_t(v) << 16);
      else x[e] = __half2float(__ushort_as_half(v));
    }
  };
  int group = -1, first = 0;
  for (int g = 0; g < p.P; ++g) {
    const int a = max(first, p.group_start ? min(max(p.group_start[g], 0), p.B) : 0);
    const int e = max(a, p.group_start ? min(max(p.group_start[g + 1], 0), p.B) : p.B);
    if (b >= a && b < e) group = g;
    first = a;
  }
  const int plen = group < 0 ? 0 : min(max(p.prefix_lens[group], 0), p.max_pblocks * p.bs);
  const int cap = p.max_blocks * p.bs;
  const int len = p.seq_lens ? min(max(p.seq_lens[b], 0), cap) : cap;
  float q[E], o[E], m = -INFINITY, l = 0.0f;
  load(p.q, (static_cast<size_t>(b) * p.Hq + h) * D, q);
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.0f;
  for (int c = warp; c < plen + len; c += 4) {
    const int row = c < plen ? c : c - plen;
    const int block = c < plen ? p.prefix_table[static_cast<size_t>(group) * p.max_pblocks + row / p.bs]
                               : p.block_table[static_cast<size_t>(b) * p.max_blocks + row / p.bs];
    const bool in = block >= 0 && block < p.num_blocks;
    const size_t at = ((static_cast<size_t>(in ? block : 0) * p.bs + row % p.bs) * p.Hkv + kv) * D;
    float k[E], v[E], s = 0.0f;
    load(p.k_pool, at, k);
    load(p.v_pool, at, v);
#pragma unroll
    for (int e = 0; e < E; ++e) s = fmaf(q[e], in ? k[e] : 0.0f, s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= p.qscale;
    const float top = fmaxf(m, s), a = m == top ? 1.0f : exp2f(m - top), w = exp2f(s - top);
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * (in ? v[e] : 0.0f);
    m = top;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_o[warp][E * lane + e] = o[e];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 128) {
    const float top = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float sum = 0.0f, x = 0.0f;
    for (int w = 0; w < 4; ++w) {
      const float a = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - top);
      sum += a * s_l[w];
      x += a == 0.0f ? 0.0f : a * s_o[w][d];
    }
    const float y = sum == 0.0f ? 0.0f : x / sum;
    static_cast<uint16_t*>(p.out)[(static_cast<size_t>(b) * p.Hq + h) * D + d] =
        static_cast<uint16_t>(pack2<Tag>(y, 0.0f) & 0xffffu);
  }
}

}  // namespace gqa_av
