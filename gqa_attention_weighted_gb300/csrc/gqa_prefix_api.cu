// Host side of the C ABI declared in include/gqa_prefix.h: argument checks and
// dispatch.
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "gqa_prefix.h"
#include "gqa_prefix_kernel.cuh"

namespace gqa_av {
namespace {

thread_local std::string g_px_error;

int pfail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_px_error = buf;
  return status;
}

int pfail_cuda(cudaError_t e, const char* what) {
  return pfail(GQA_AV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

int check_args(const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
               const int32_t* prefix_lens, const int32_t* group_start, const int32_t* block_table,
               const int32_t* seq_lens, const void* out, int B, int P, int Hq, int Hkv, int D,
               int kv_dtype, int block_size, int num_blocks, int max_prefix_blocks, int max_blocks,
               float scale) {
  if (B <= 0 || P < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || block_size <= 0 || num_blocks <= 0)
    return pfail(GQA_AV_ERR_INVALID,
                 "sizes must be positive (B=%d Hq=%d Hkv=%d D=%d block_size=%d num_blocks=%d) and "
                 "P=%d not negative",
                 B, Hq, Hkv, D, block_size, num_blocks, P);
  if (Hq % Hkv) return pfail(GQA_AV_ERR_INVALID, "Hq=%d is not a multiple of Hkv=%d", Hq, Hkv);
  if (kv_dtype != GQA_AV_BF16 && kv_dtype != GQA_AV_FP16)
    return pfail(GQA_AV_ERR_INVALID, "kv_dtype=%d must be GQA_AV_BF16 or GQA_AV_FP16", kv_dtype);
  if (max_blocks < 0 || max_prefix_blocks < 0 || (P && max_prefix_blocks == 0))
    return pfail(GQA_AV_ERR_INVALID, "max_blocks=%d or max_prefix_blocks=%d out of range",
                 max_blocks, max_prefix_blocks);
  if (!std::isfinite(scale)) return pfail(GQA_AV_ERR_INVALID, "scale must be finite");
  if (!q || !k_pool || !v_pool || !out || (P && (!prefix_table || !prefix_lens)) ||
      (max_blocks && !block_table))
    return pfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if (P > 1 && !group_start)
    return pfail(GQA_AV_ERR_INVALID, "group_start may be NULL only with P <= 1");
  if ((addr(prefix_table) | addr(prefix_lens) | addr(group_start) | addr(block_table) |
       addr(seq_lens)) & 3u)
    return pfail(GQA_AV_ERR_INVALID, "tables and lengths must be 4-byte aligned");
  if (D != 64 && D != 128 && D != 256)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "D=%d must be 64, 128 or 256", D);
  if (Hq / Hkv > 128)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "Hq / Hkv = %d is above 128", Hq / Hkv);
  if (block_size % 8)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "block_size=%d must be a multiple of 8", block_size);
  if (B > 4096 || P > 128)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "B=%d is above 4096 or P=%d above 128", B, P);
  const long long most = 0x7fffffffLL / block_size;
  if (num_blocks > most || max_blocks > most || max_prefix_blocks > most)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "a pool or a table row of 2^31 or more cache rows");
  if ((addr(q) | addr(k_pool) | addr(v_pool) | addr(out)) & 15u)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "q, the pools and out must be 16-byte aligned");
  return GQA_AV_OK;
}

using SimpleKernel = void (*)(PrefixParams);

template <typename Tag>
SimpleKernel pick_simple(int D) {
  return D == 64 ? gqa_prefix_simple_kernel<Tag, 64>
                 : D == 128 ? gqa_prefix_simple_kernel<Tag, 128> : gqa_prefix_simple_kernel<Tag, 256>;
}

}  // namespace
}  // namespace gqa_av

using namespace gqa_av;

extern "C" int gqa_prefix_attn_decode(
    const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
    const int32_t* prefix_lens, const int32_t* group_start, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int P, int Hq, int Hkv, int D, int kv_dtype,
    int block_size, int num_blocks, int max_prefix_blocks, int max_blocks, float scale,
    void* stream_) {
  g_px_error.clear();
  int rc = check_args(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table,
                      seq_lens, out, B, P, Hq, Hkv, D, kv_dtype, block_size, num_blocks,
                      max_prefix_blocks, max_blocks, scale);
  if (rc) return rc;
  PrefixParams p;
  p.q = q; p.k_pool = k_pool; p.v_pool = v_pool;
  p.prefix_table = prefix_table; p.prefix_lens = prefix_lens; p.group_start = group_start;
  p.block_table = block_table; p.seq_lens = seq_lens; p.out = out;
  p.B = B; p.P = P; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv;
  p.bs = block_size; p.num_blocks = num_blocks;
  p.max_pblocks = max_prefix_blocks; p.max_blocks = max_blocks;
  p.qscale = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);  // log2(e)
  cudaStream_t stream = static_cast<cudaStream_t>(stream_);
  SimpleKernel k = kv_dtype == GQA_AV_BF16 ? pick_simple<Bf16Tag>(D) : pick_simple<Fp16Tag>(D);
  k<<<B * Hq, 128, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return pfail_cuda(e, "attention kernel launch");
  return GQA_AV_OK;
}

extern "C" int gqa_prefix_device_status(void* stream_, int clear) {
  (void)clear;
  g_px_error.clear();
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream_));
  if (e != cudaSuccess) return pfail_cuda(e, "cudaStreamSynchronize");
  return GQA_AV_OK;
}

extern "C" const char* gqa_prefix_last_error(void) { return g_px_error.c_str(); }
