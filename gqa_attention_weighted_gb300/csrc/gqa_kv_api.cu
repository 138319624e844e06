// Host side of the C ABI declared in include/gqa_kv.h: argument checks and
// dispatch of the block-table and the norm + rotation + cache-write kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "gqa_kv.h"
#include "gqa_kv_kernel.cuh"

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
                   void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
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

extern "C" const char* gqa_kv_last_error(void) { return g_kv_error; }
