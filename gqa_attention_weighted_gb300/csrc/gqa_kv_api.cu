// Host side of the C ABI declared in include/gqa_kv.h: argument checks and
// dispatch of the block-table, the norm + rotation + cache-write and the fork,
// keep and release kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gqa_kv.h"
#include "gqa_kv_kernel.cuh"
#include "gqa_kv_pages.cuh"

namespace gqa_av {
namespace {

thread_local char g_kv_error[512];   // no allocation: nothing here can throw

int kfail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_kv_error, sizeof g_kv_error, fmt, ap);
  va_end(ap);
  return status;
}

int kfail_cuda(cudaError_t e, const char* what) {
  return kfail(GQA_AV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

int check_pool(int block_size, int num_blocks) {
  if (block_size <= 0 || num_blocks <= 0)
    return kfail(GQA_AV_ERR_INVALID, "block_size=%d and num_blocks=%d must be positive", block_size,
                 num_blocks);
  if (static_cast<long long>(block_size) * num_blocks > 0x7fffffffLL)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "num_blocks * block_size = %lld does not fit 31 bits",
                 static_cast<long long>(block_size) * num_blocks);
  return GQA_AV_OK;
}

cudaError_t launch(const void* fn, int grid, int block, size_t smem, cudaStream_t stream,
                   void** args, int cluster = 1) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

// A run of n bytes of device memory, by name.
struct Range {
  const char* name;
  const void* at;
  unsigned long long n;
};
bool meet(const Range& a, const Range& b) {
  return a.at && b.at && a.n && b.n && addr(a.at) < addr(b.at) + b.n && addr(b.at) < addr(a.at) + a.n;
}

// Pools of one layout, given by their rows' bytes.
int check_pools(void* const* pools, int n_pools, int64_t row_bytes, int block_size, int num_blocks) {
  if (n_pools < 0 || row_bytes <= 0 || (n_pools && !pools))
    return kfail(GQA_AV_ERR_INVALID, "n_pools=%d must not be negative, row_bytes=%lld positive and "
                 "pools given", n_pools, static_cast<long long>(row_bytes));
  if (n_pools > kPagePools)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "n_pools=%d is above %d", n_pools, kPagePools);
  if (row_bytes % 16 || row_bytes > (1 << 20))
    return kfail(GQA_AV_ERR_UNSUPPORTED, "row_bytes=%lld must be a multiple of 16, at most 2^20",
                 static_cast<long long>(row_bytes));
  const int rc = check_pool(block_size, num_blocks);
  if (rc) return rc;
  for (int i = 0; i < n_pools; ++i) {
    if (!pools[i]) return kfail(GQA_AV_ERR_INVALID, "pools[%d] is NULL", i);
    if (addr(pools[i]) & 15u)
      return kfail(GQA_AV_ERR_UNSUPPORTED, "pools[%d] must be 16-byte aligned", i);
  }
  // Rows that are moved twice would be lost.
  uintptr_t at[kPagePools];
  for (int i = 0; i < n_pools; ++i) at[i] = addr(pools[i]);
  std::sort(at, at + n_pools);
  const unsigned long long bytes = static_cast<unsigned long long>(row_bytes) * block_size * num_blocks;
  for (int i = 1; i < n_pools; ++i)
    if (at[i] - at[i - 1] < bytes) return kfail(GQA_AV_ERR_INVALID, "two pools overlap");
  return GQA_AV_OK;
}

// Tables and lengths of the calls below: their sizes.
int check_rows(int B, int max_blocks, int block_size) {
  if (B <= 0 || max_blocks <= 0)
    return kfail(GQA_AV_ERR_INVALID, "B=%d and max_blocks=%d must be positive", B, max_blocks);
  if (B > kPageMaxB) return kfail(GQA_AV_ERR_UNSUPPORTED, "B=%d is above %d", B, kPageMaxB);
  if (block_size > 0 && static_cast<long long>(max_blocks) * block_size > 0x7fffffffLL)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "a table row of 2^31 or more cache rows");
  return GQA_AV_OK;
}

// The largest cluster that the release kernel can have on a device: 16 where it
// allows that many, 8 is within every device's. Found once a device.
int release_cluster(const void* fn, int dev) {
  static std::atomic<int> known[64];
  int n = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n) return n;
  n = kReleasePortable;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kReleaseCluster);
    cfg.blockDim = dim3(kReleaseThreads);
    cfg.dynamicSmemBytes = 4 * (2 * kPageMaxB + 1 + kReleaseCache);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kReleaseCluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int fit = 0;
    if (cudaOccupancyMaxActiveClusters(&fit, fn, &cfg) == cudaSuccess && fit > 0) n = kReleaseCluster;
  }
  cudaGetLastError();   // of a query that was refused
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

using RopeKernel = void (*)(RopeParams);

template <typename Tag, int L>
RopeKernel pick_rope(bool interleaved, bool q32) {
  if (interleaved)
    return q32 ? gqa_kv_rope_kernel<Tag, L, true, true> : gqa_kv_rope_kernel<Tag, L, true, false>;
  return q32 ? gqa_kv_rope_kernel<Tag, L, false, true> : gqa_kv_rope_kernel<Tag, L, false, false>;
}

template <typename Tag>
RopeKernel pick_rope(int lanes, bool interleaved, bool q32) {
  switch (lanes) {
    case 4: return pick_rope<Tag, 4>(interleaved, q32);
    case 8: return pick_rope<Tag, 8>(interleaved, q32);
    case 16: return pick_rope<Tag, 16>(interleaved, q32);
    default: return pick_rope<Tag, 32>(interleaved, q32);
  }
}

}  // namespace
}  // namespace gqa_av

using namespace gqa_av;

extern "C" int gqa_kv_tables(const int32_t* cached_lens, const int32_t* new_lens,
                             const int32_t* pos_base, const int32_t* free_list,
                             const int32_t* free_count, int32_t* block_table, int32_t* seq_lens,
                             int32_t* token_start, int32_t* slots, int32_t* positions,
                             int32_t* free_left, int B, int T, int max_blocks, int n_free,
                             int block_size, int num_blocks, void* stream) {
  g_kv_error[0] = 0;
  if (B <= 0 || T < 0 || max_blocks <= 0 || n_free < 0)
    return kfail(GQA_AV_ERR_INVALID,
                 "B=%d and max_blocks=%d must be positive, T=%d and n_free=%d not negative", B,
                 max_blocks, T, n_free);
  if (!cached_lens || !new_lens || !free_count || !block_table || !seq_lens || !token_start ||
      !free_left || (n_free && !free_list) || (T && (!slots || !positions)))
    return kfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(cached_lens) | addr(new_lens) | addr(pos_base) | addr(free_list) | addr(free_count) |
       addr(block_table) | addr(seq_lens) | addr(token_start) | addr(slots) | addr(positions) |
       addr(free_left)) & 3u)
    return kfail(GQA_AV_ERR_INVALID, "pointers must be 4-byte aligned");
  int rc = check_pool(block_size, num_blocks);
  if (rc) return rc;
  if (B > kTabMaxB) return kfail(GQA_AV_ERR_UNSUPPORTED, "B=%d is above %d", B, kTabMaxB);
  // Every CTA reads the inputs, at any time while others write.
  const struct { const char* name; const int32_t* at; long long n; }
      ins[] = {{"cached_lens", cached_lens, B}, {"new_lens", new_lens, B}, {"pos_base", pos_base, B},
               {"free_list", free_list, n_free}, {"free_count", free_count, 1}},
      outs[] = {{"block_table", block_table, static_cast<long long>(B) * max_blocks},
                {"seq_lens", seq_lens, B}, {"token_start", token_start, B + 1LL},
                {"slots", slots, T}, {"positions", positions, T}, {"free_left", free_left, 1}};
  for (const auto& i : ins)
    for (const auto& o : outs)
      if (i.at && o.at && i.n && o.n && addr(i.at) < addr(o.at) + 4 * static_cast<uintptr_t>(o.n) &&
          addr(o.at) < addr(i.at) + 4 * static_cast<uintptr_t>(i.n))
        return kfail(GQA_AV_ERR_INVALID, "%s overlaps %s", o.name, i.name);

  TablesParams p;
  p.cached = cached_lens; p.fresh = new_lens; p.pos_base = pos_base;
  p.free_list = free_list; p.free_count = free_count; p.table = block_table;
  p.seq_lens = seq_lens; p.token_start = token_start; p.slots = slots; p.positions = positions;
  p.free_left = free_left;
  p.B = B; p.T = T; p.max_blocks = max_blocks; p.n_free = n_free; p.bs = block_size;
  p.num_blocks = num_blocks;
  const size_t smem = static_cast<size_t>(B) * 12;
  const void* fn = reinterpret_cast<const void*>(gqa_kv_tables_kernel);
  cudaError_t e = cudaSuccess;
  if (smem > 40960) {   // within the default limit otherwise
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kTabMaxB * 12);
    if (e != cudaSuccess) return kfail_cuda(e, "cudaFuncSetAttribute");
  }
  const int grid = std::max(1, T / kTabTokensPerCta + (T % kTabTokensPerCta != 0));
  void* args[] = {&p};
  e = launch(fn, grid, kTabThreads, smem, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return kfail_cuda(e, "block-table kernel launch");
  return GQA_AV_OK;
}

extern "C" int gqa_kv_norm_rope_append(
    const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, const int32_t* positions, const int32_t* sections, int n_axes,
    const float* inv_freq, const void* q_weight, const void* k_weight, float eps,
    float weight_offset, int interleaved, const int32_t* slots, void* q_out, int q_out_dtype,
    void* k_pool, void* v_pool, int T, int Hq, int Hkv, int D, int rot_dim, int kv_dtype,
    int block_size, int num_blocks, void* stream) {
  g_kv_error[0] = 0;
  if (T < 0 || Hq <= 0 || Hkv <= 0 || D <= 0)
    return kfail(GQA_AV_ERR_INVALID, "T=%d must not be negative and Hq=%d Hkv=%d D=%d positive", T,
                 Hq, Hkv, D);
  if (kv_dtype != GQA_AV_BF16 && kv_dtype != GQA_AV_FP16)
    return kfail(GQA_AV_ERR_INVALID, "kv_dtype=%d must be GQA_AV_BF16 or GQA_AV_FP16", kv_dtype);
  if (q_out_dtype != kv_dtype && q_out_dtype != GQA_KV_F32)
    return kfail(GQA_AV_ERR_INVALID, "q_out_dtype=%d must be kv_dtype or GQA_KV_F32", q_out_dtype);
  int rc = check_pool(block_size, num_blocks);
  if (rc) return rc;
  if (D % 8 || D > 256)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "D=%d must be a multiple of 8, at most 256", D);
  if (rot_dim < 0 || rot_dim > D)
    return kfail(GQA_AV_ERR_INVALID, "rot_dim=%d outside 0..%d", rot_dim, D);
  if (rot_dim % (interleaved ? 8 : 16))
    return kfail(GQA_AV_ERR_UNSUPPORTED, "rot_dim=%d must be a multiple of %d", rot_dim,
                 interleaved ? 8 : 16);
  if (n_axes < 1 || n_axes > 4 || (n_axes > 1 && !sections))
    return kfail(GQA_AV_ERR_INVALID, "n_axes=%d must be 1..4, with sections when above 1", n_axes);
  if (sections && rot_dim) {
    long long sum = 0;
    for (int a = 0; a < n_axes; ++a) {
      if (sections[a] < 0) return kfail(GQA_AV_ERR_INVALID, "sections[%d]=%d < 0", a, sections[a]);
      sum += sections[a];
    }
    if (sum != rot_dim / 2)
      return kfail(GQA_AV_ERR_INVALID, "sections sum to %lld, not rot_dim / 2 = %d", sum, rot_dim / 2);
  }
  if (!(std::isfinite(eps) && eps >= 0.0f) || !std::isfinite(weight_offset))
    return kfail(GQA_AV_ERR_INVALID, "eps must be finite and not negative, weight_offset finite");
  if (T == 0) return GQA_AV_OK;
  if (!q || !k || !v || !slots || !q_out || !k_pool || !v_pool ||
      (rot_dim && (!positions || !inv_freq)))
    return kfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(positions) | addr(slots) | addr(inv_freq)) & 3u)
    return kfail(GQA_AV_ERR_INVALID, "positions, slots and inv_freq must be 4-byte aligned");
  if ((addr(q) | addr(k) | addr(v) | addr(q_out) | addr(k_pool) | addr(v_pool) | addr(q_weight) |
       addr(k_weight)) & 15u)
    return kfail(GQA_AV_ERR_UNSUPPORTED,
                 "q, k, v, q_out, the pools and the weights must be 16-byte aligned");
  if (T == 1) q_stride = k_stride = v_stride = 0;   // of no meaning for a single token
  if ((q_stride | k_stride | v_stride) & 7)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "token strides must be multiples of 8 elements");
  if (T > 1 && (q_stride < static_cast<int64_t>(Hq) * D || k_stride < static_cast<int64_t>(Hkv) * D ||
                v_stride < static_cast<int64_t>(Hkv) * D))
    return kfail(GQA_AV_ERR_INVALID, "token strides are smaller than a token's heads");

  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return kfail_cuda(e, "cudaGetDevice");

  RopeParams p;
  p.q = q; p.k = k; p.v = v;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.positions = positions; p.inv_freq = inv_freq;
  p.qw = q_weight; p.kw = k_weight; p.slots = slots;
  p.q_out = q_out; p.k_pool = k_pool; p.v_pool = v_pool;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.D = D; p.pairs = rot_dim / 2;
  p.rows = block_size * num_blocks;
  for (int a = 0, at = 0; a < 4; ++a) {
    at += sections && rot_dim && a < n_axes ? sections[a] : 0;
    p.sec_end[a] = a < n_axes - 1 ? at : 0x7fffffff;
  }
  p.eps = eps; p.w_offset = weight_offset;
  int lanes = 4;
  while (lanes * 8 < D) lanes *= 2;
  const int steps = (Hq + 2 * Hkv + 32 / lanes - 1) / (32 / lanes);
  // A token's heads go to one warp when there are tokens for 8 CTAs of 8 warps an
  // SM; with fewer they are cut into parts, down to one step a warp, since a
  // single warp's chain of loads is all latency. That is more than fit at a time:
  // registers leave 3 CTAs an SM (2 with separate halves and fp32 queries), so
  // mid-size calls run in waves (4097 tokens of 16 + 1 + 1 heads: 1025 CTAs, 2.2
  // waves, 24.5 us).
  const long long room = static_cast<long long>(sms) * 8 * kRopeWarps;
  p.chunks = static_cast<int>(std::min<long long>(steps, std::max<long long>(1, room / T)));
  p.iters = (steps + p.chunks - 1) / p.chunks;
  p.chunks = (steps + p.iters - 1) / p.iters;
  const long long ctas = (static_cast<long long>(T) * p.chunks + kRopeWarps - 1) / kRopeWarps;
  const int grid = static_cast<int>(std::min<long long>(ctas, static_cast<long long>(sms) * 8));
  const bool q32 = q_out_dtype == GQA_KV_F32;
  RopeKernel fn = kv_dtype == GQA_AV_BF16 ? pick_rope<Bf16Tag>(lanes, interleaved != 0, q32)
                                          : pick_rope<Fp16Tag>(lanes, interleaved != 0, q32);
  void* args[] = {&p};
  e = launch(reinterpret_cast<const void*>(fn), grid, 32 * kRopeWarps, 0,
             static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return kfail_cuda(e, "norm and rotation kernel launch");
  return GQA_AV_OK;
}

extern "C" int gqa_kv_fork(void* const* pools, int n_pools, int64_t row_bytes,
                           const int32_t* parent, const int32_t* child, int32_t* block_table,
                           int32_t* seq_lens, int32_t* shares, const int32_t* free_list,
                           const int32_t* free_count, int32_t* fork_block, int32_t* free_left,
                           int N, int B, int max_blocks, int n_free, int block_size,
                           int num_blocks, void* stream) {
  g_kv_error[0] = 0;
  if (N < 0 || n_free < 0)
    return kfail(GQA_AV_ERR_INVALID, "N=%d and n_free=%d must not be negative", N, n_free);
  int rc = check_pools(pools, n_pools, row_bytes, block_size, num_blocks);
  if (!rc) rc = check_rows(B, max_blocks, block_size);
  if (rc) return rc;
  if (N > kPageMaxB) return kfail(GQA_AV_ERR_UNSUPPORTED, "N=%d is above %d", N, kPageMaxB);
  if (!block_table || !seq_lens || !shares || !free_count || !free_left ||
      (N && (!parent || !child || !fork_block)) || (n_free && !free_list))
    return kfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(parent) | addr(child) | addr(block_table) | addr(seq_lens) | addr(shares) |
       addr(free_list) | addr(free_count) | addr(fork_block) | addr(free_left)) & 3u)
    return kfail(GQA_AV_ERR_INVALID, "pointers must be 4-byte aligned");
  // Every CTA reads the inputs, at any time while others write.
  const unsigned long long n4 = 4ull * N, rows = 4ull * B * max_blocks;
  const Range ins[] = {{"parent", parent, n4}, {"child", child, n4},
                       {"free_list", free_list, 4ull * n_free}, {"free_count", free_count, 4}};
  const Range outs[] = {{"block_table", block_table, rows}, {"seq_lens", seq_lens, 4ull * B},
                        {"shares", shares, 4ull * num_blocks}, {"fork_block", fork_block, n4},
                        {"free_left", free_left, 4}};
  constexpr int kOuts = sizeof outs / sizeof outs[0];
  for (int o = 0; o < kOuts; ++o) {
    for (const Range& i : ins)
      if (meet(i, outs[o])) return kfail(GQA_AV_ERR_INVALID, "%s overlaps %s", outs[o].name, i.name);
    for (int q = 0; q < o; ++q)
      if (meet(outs[q], outs[o]))
        return kfail(GQA_AV_ERR_INVALID, "%s overlaps %s", outs[o].name, outs[q].name);
  }

  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return kfail_cuda(e, "cudaGetDevice");
  ForkParams p;
  std::copy(pools, pools + n_pools, reinterpret_cast<void**>(p.pools.at));
  p.parent = parent; p.child = child; p.table = block_table; p.seq_lens = seq_lens;
  p.shares = shares; p.free_list = free_list; p.free_count = free_count;
  p.fork_block = fork_block; p.free_left = free_left;
  p.row_bytes = row_bytes; p.n_pools = n_pools; p.N = N; p.B = B; p.max_blocks = max_blocks;
  p.n_free = n_free; p.bs = block_size; p.num_blocks = num_blocks;
  const size_t smem = 8 * (static_cast<size_t>(B) + N);
  const void* fn = reinterpret_cast<const void*>(gqa_kv_fork_kernel);
  if (smem > 40960) {   // within the default limit otherwise
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, 16 * kPageMaxB);
    if (e != cudaSuccess) return kfail_cuda(e, "cudaFuncSetAttribute");
  }
  // Two CTAs an SM where every warp has a piece to copy, fewer with fewer pieces.
  const long long pieces =
      ((block_size - 1) * static_cast<long long>(row_bytes) + kForkPiece - 1) / kForkPiece;
  const long long ctas = (static_cast<long long>(N) * n_pools * pieces + 15) / 16;
  const int grid = static_cast<int>(std::min<long long>(2LL * sms, std::max<long long>(1, std::max<long long>(N, ctas))));
  void* args[] = {&p};
  e = launch(fn, grid, kForkThreads, smem, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return kfail_cuda(e, "fork kernel launch");
  return GQA_AV_OK;
}

extern "C" int gqa_kv_keep(void* const* pools, int n_pools, int64_t row_bytes,
                           const int32_t* cached_lens, const int32_t* accepted,
                           const int32_t* accepted_count, const int32_t* block_table,
                           const int32_t* seq_lens, int32_t* kept_lens, int B, int W,
                           int max_blocks, int block_size, int num_blocks, void* stream) {
  g_kv_error[0] = 0;
  if (W < 0) return kfail(GQA_AV_ERR_INVALID, "W=%d must not be negative", W);
  int rc = check_pools(pools, n_pools, row_bytes, block_size, num_blocks);
  if (!rc) rc = check_rows(B, max_blocks, block_size);
  if (rc) return rc;
  if (!n_pools) return kfail(GQA_AV_ERR_INVALID, "no pools");
  if (W > (1 << 20)) return kfail(GQA_AV_ERR_UNSUPPORTED, "W=%d is above 2^20", W);
  if (!cached_lens || !accepted_count || !block_table || !seq_lens || !kept_lens || (W && !accepted))
    return kfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(cached_lens) | addr(accepted) | addr(accepted_count) | addr(block_table) |
       addr(seq_lens) | addr(kept_lens)) & 3u)
    return kfail(GQA_AV_ERR_INVALID, "pointers must be 4-byte aligned");
  const Range out = {"kept_lens", kept_lens, 4ull * B};
  for (const Range& i : {Range{"cached_lens", cached_lens, 4ull * B},
                         Range{"accepted", accepted, 4ull * B * W},
                         Range{"accepted_count", accepted_count, 4ull * B},
                         Range{"block_table", block_table, 4ull * B * max_blocks},
                         Range{"seq_lens", seq_lens, 4ull * B}})
    if (meet(i, out)) return kfail(GQA_AV_ERR_INVALID, "kept_lens overlaps %s", i.name);

  KeepParams p;
  std::copy(pools, pools + n_pools, reinterpret_cast<void**>(p.pools.at));
  p.cached = cached_lens; p.accepted = accepted; p.count = accepted_count; p.table = block_table;
  p.seq_lens = seq_lens; p.kept = kept_lens;
  p.row_bytes = row_bytes; p.n_pools = n_pools; p.B = B; p.W = W; p.max_blocks = max_blocks;
  p.bs = block_size; p.num_blocks = num_blocks;
  p.parts = static_cast<int>((row_bytes + 511) / 512);
  const long long tasks = static_cast<long long>(B) * n_pools * p.parts;
  const long long grid = (tasks + kKeepWarps - 1) / kKeepWarps;
  if (grid > 0x7fffffffLL)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "B=%d requests in %d pools of rows of %lld bytes are too many",
                 B, n_pools, static_cast<long long>(row_bytes));
  void* args[] = {&p};
  cudaError_t e = launch(reinterpret_cast<const void*>(gqa_kv_keep_kernel), static_cast<int>(grid),
                         32 * kKeepWarps, 0, static_cast<cudaStream_t>(stream), args);
  if (e != cudaSuccess) return kfail_cuda(e, "keep kernel launch");
  return GQA_AV_OK;
}

extern "C" int gqa_kv_release(const int32_t* block_table, const int32_t* old_lens,
                              const int32_t* new_lens, int32_t* shares, int32_t* free_list,
                              const int32_t* free_count, int32_t* free_left, int B,
                              int max_blocks, int n_free, int block_size, int num_blocks,
                              void* stream) {
  g_kv_error[0] = 0;
  if (n_free < 0) return kfail(GQA_AV_ERR_INVALID, "n_free=%d must not be negative", n_free);
  int rc = check_pool(block_size, num_blocks);
  if (!rc) rc = check_rows(B, max_blocks, block_size);
  if (rc) return rc;
  const long long most = static_cast<long long>(B) * max_blocks;
  if (most >= 1 << 30)
    return kfail(GQA_AV_ERR_UNSUPPORTED, "B * max_blocks = %lld must be below 2^30", most);
  if (!block_table || !old_lens || !new_lens || !free_count || !free_left || (n_free && !free_list))
    return kfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(block_table) | addr(old_lens) | addr(new_lens) | addr(shares) | addr(free_list) |
       addr(free_count) | addr(free_left)) & 3u)
    return kfail(GQA_AV_ERR_INVALID, "pointers must be 4-byte aligned");
  const Range ins[] = {{"block_table", block_table, 4ull * B * max_blocks},
                       {"old_lens", old_lens, 4ull * B}, {"new_lens", new_lens, 4ull * B},
                       {"free_count", free_count, 4}};
  const Range outs[] = {{"shares", shares, 4ull * num_blocks}, {"free_list", free_list, 4ull * n_free},
                        {"free_left", free_left, 4}};
  for (int o = 0; o < 3; ++o) {
    for (const Range& i : ins)
      if (meet(i, outs[o])) return kfail(GQA_AV_ERR_INVALID, "%s overlaps %s", outs[o].name, i.name);
    for (int q = 0; q < o; ++q)
      if (meet(outs[q], outs[o]))
        return kfail(GQA_AV_ERR_INVALID, "%s overlaps %s", outs[o].name, outs[q].name);
  }

  ReleaseParams p;
  p.table = block_table; p.old_lens = old_lens; p.new_lens = new_lens; p.shares = shares;
  p.free_list = free_list; p.free_count = free_count; p.free_left = free_left;
  p.B = B; p.max_blocks = max_blocks; p.n_free = n_free; p.bs = block_size;
  p.num_blocks = num_blocks;
  const void* fn = reinterpret_cast<const void*>(gqa_kv_release_kernel);
  const size_t smem = 4 * (2 * static_cast<size_t>(B) + 1 + kReleaseCache);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       4 * (2 * kPageMaxB + 1 + kReleaseCache));
  if (e != cudaSuccess) return kfail_cuda(e, "cudaFuncSetAttribute");
  int dev = 0, ctas = 1;
  if (most > kReleaseEach * kReleaseThreads) {   // more than one CTA's entries at a time
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return kfail_cuda(e, "cudaGetDevice");
    ctas = release_cluster(fn, dev);
  }
  void* args[] = {&p};
  e = launch(fn, ctas, kReleaseThreads, smem, static_cast<cudaStream_t>(stream), args, ctas);
  if (e != cudaSuccess) return kfail_cuda(e, "release kernel launch");
  return GQA_AV_OK;
}

extern "C" const char* gqa_kv_last_error(void) { return g_kv_error; }
