// Host side of the C ABI declared in include/gqa_prefix.h: argument checks, the
// call's workspace, tensor maps and dispatch to the attention and combine
// kernels.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <new>

#include "gqa_paged_host.h"
#include "gqa_prefix.h"
#include "gqa_prefix_kernel.cuh"

namespace gqa_av {
namespace {

thread_local char g_px_error[512];

int pfail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_px_error, sizeof g_px_error, fmt, ap);
  va_end(ap);
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
  if (B > kPxMaxB || P > kPxMaxGroups)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "B=%d is above %d or P=%d above %d", B, kPxMaxB, P,
                 kPxMaxGroups);
  if (Hkv > (1 << 14) || static_cast<long long>(B) * Hkv > (1 << 20))
    return pfail(GQA_AV_ERR_UNSUPPORTED, "Hkv=%d is above 2^14 or B * Hkv = %lld above 2^20", Hkv,
                 static_cast<long long>(B) * Hkv);
  const long long most = 0x7fffffffLL / block_size, longest = (1LL << 26) / block_size;
  if (num_blocks > most || max_blocks > longest || max_prefix_blocks > longest)
    return pfail(GQA_AV_ERR_UNSUPPORTED,
                 "a pool of 2^31 or more cache rows, or a table row of more than 2^26");
  if ((addr(q) | addr(k_pool) | addr(v_pool) | addr(out)) & 15u)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "q, the pools and out must be 16-byte aligned");
  return GQA_AV_OK;
}

using PrefixKernel = void (*)(PrefixParams);

template <typename Tag>
PrefixKernel pick_main(int D) {
  return D == 64 ? gqa_prefix_kernel<Tag, 64>
                 : D == 128 ? gqa_prefix_kernel<Tag, 128> : gqa_prefix_kernel<Tag, 256>;
}
template <typename Tag, int U>
PrefixKernel pick_combine(int D) {
  return D == 64 ? gqa_prefix_combine_kernel<Tag, 64, U>
                 : D == 128 ? gqa_prefix_combine_kernel<Tag, 128, U>
                            : gqa_prefix_combine_kernel<Tag, 256, U>;
}
template <typename Tag>
PrefixKernel pick_combine(int D, bool waves) {
  return waves ? pick_combine<Tag, 4>(D) : pick_combine<Tag, 8>(D);
}
int smem_bytes(int D) {
  return D == 64 ? PxShape<64>::SMEM : D == 128 ? PxShape<128>::SMEM : PxShape<256>::SMEM;
}

using PrefixWorkspaces = Workspaces<sizeof(PxHeader), pfail>;

int encode_maps(PrefixParams* p, const void* q, const void* k_pool, const void* v_pool, int D) {
  const cuuint64_t d = D, G = p->G, Hkv = p->Hkv, rows = static_cast<cuuint64_t>(p->bs) * p->num_blocks;
  const cuuint64_t qd[4] = {d, G, Hkv, static_cast<cuuint64_t>(p->B)};
  const cuuint64_t qs[3] = {d * 2, G * d * 2, Hkv * G * d * 2};
  const cuuint32_t tile[4] = {64, static_cast<cuuint32_t>(p->G), 1, static_cast<cuuint32_t>(p->TB)};
  const cuuint32_t one[4] = {64, static_cast<cuuint32_t>(p->G), 1, 1};
  const cuuint64_t kd[3] = {d, Hkv, rows};
  const cuuint64_t ks[2] = {d * 2, Hkv * d * 2};
  const cuuint32_t kb[3] = {64, 1, static_cast<cuuint32_t>(p->R)};
  int rc = encode_map(pfail, &p->q_tile_map, q, 4, qd, qs, tile, "q");
  if (!rc) rc = encode_map(pfail, &p->q_one_map, q, 4, qd, qs, one, "q");
  if (!rc) rc = encode_map(pfail, &p->k_map, k_pool, 3, kd, ks, kb, "K");
  if (!rc) rc = encode_map(pfail, &p->v_map, v_pool, 3, kd, ks, kb, "V");
  return rc;
}

int decode(const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
           const int32_t* prefix_lens, const int32_t* group_start, const int32_t* block_table,
           const int32_t* seq_lens, void* out, int B, int P, int Hq, int Hkv, int D, int kv_dtype,
           int block_size, int num_blocks, int max_prefix_blocks, int max_blocks, float scale,
           long long wait_ns, unsigned withhold_from, cudaStream_t stream) try {
  int rc = check_args(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table,
                      seq_lens, out, B, P, Hq, Hkv, D, kv_dtype, block_size, num_blocks,
                      max_prefix_blocks, max_blocks, scale);
  if (rc) return rc;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return pfail_cuda(e, "cudaGetDevice");

  PrefixParams p;
  p.prefix_table = prefix_table; p.prefix_lens = prefix_lens; p.group_start = group_start;
  p.block_table = block_table; p.seq_lens = seq_lens; p.out = out;
  p.B = B; p.P = P; p.Hq = Hq; p.Hkv = Hkv; p.G = Hq / Hkv; p.TB = 128 / p.G;
  p.bs = block_size; p.num_blocks = num_blocks;
  p.max_pblocks = max_prefix_blocks; p.max_blocks = max_blocks;
  block_divisor(block_size, &p.bs_mul, &p.bs_shift);
  const int keys = D == 256 ? PxShape<256>::KEYS : PxShape<128>::KEYS;
  for (p.R = 8; p.R < keys && block_size % (2 * p.R) == 0;) p.R *= 2;
  // log2(e) in the scale; a scale of 0 becomes the smallest normal number, which
  // leaves every finite score at 0 and keeps masked ones at -inf.
  const double s2 = std::fabs(static_cast<double>(scale)) * 1.4426950408889634;
  if (s2 > FLT_MAX) return pfail(GQA_AV_ERR_UNSUPPORTED, "scale=%g is too large", (double)scale);
  p.qscale = std::max(static_cast<float>(s2), FLT_MIN);
  p.negate = scale < 0.0f;
  // Costs of the plan, in SM cycles. Prefix key tiles as measured on 256
  // sequences behind 32768 rows, 64 + 8 heads, one unit a CTA of all key tiles:
  // 0.83 us a tile at D = 128 (1.63 for two query tiles), 0.76 (1.50) at D = 64,
  // 0.78 at D = 256 (tiles of 64 keys), at 1.9 GHz; the products of one take
  // 1024. Own tiles come from HBM, all SMs together: 64 KiB in 2800 (32 KiB at
  // D = 64). A unit's start and end cost about 2 us beyond its tiles.
  p.c_pair = D == 64 ? 2850.0f : 3100.0f;
  p.c_tile = D == 64 ? 1450.0f : D == 128 ? 1580.0f : 1480.0f;
  p.c_own = D == 64 ? 1400.0f : 2800.0f;
  p.c_unit = 4000.0f;
  p.timeout_ns = wait_ns;
  p.withhold_from = withhold_from;

  const int ns = D == 256 ? 1 : 2;
  const size_t q_tiles = static_cast<size_t>((B + p.TB - 1) / p.TB + std::min(P, B)) * Hkv;
  const size_t prefix_slots = P ? q_tiles + 2 * static_cast<size_t>(sms) : 0;
  const size_t own_slots = max_blocks ? static_cast<size_t>(B) * Hkv + 4 * static_cast<size_t>(sms) : 0;
  p.prefix_slots = static_cast<int>(prefix_slots);
  const size_t at_po = up256(sizeof(PxHeader));
  const size_t at_pm = at_po + prefix_slots * ns * 128 * D * 4;
  const size_t at_oo = at_pm + prefix_slots * ns * 128 * 8;
  const size_t at_om = at_oo + up256(own_slots * p.G * D * 4);
  bool capturing = false;
  Workspace* ws = nullptr;
  if ((rc = PrefixWorkspaces::find(dev, stream, &capturing, &ws))) return rc;
  std::lock_guard<std::mutex> lk(ws->mu);
  if ((rc = PrefixWorkspaces::grow(ws, capturing, at_om + own_slots * p.G * 8, stream))) return rc;
  char* base = ws->base;
  p.head = reinterpret_cast<PxHeader*>(base);
  p.prefix_o = reinterpret_cast<float*>(base + at_po);
  p.prefix_ml = reinterpret_cast<float2*>(base + at_pm);
  p.own_o = reinterpret_cast<float*>(base + at_oo);
  p.own_ml = reinterpret_cast<float2*>(base + at_om);
  if ((rc = encode_maps(&p, q, k_pool, v_pool, D))) return rc;

  const bool bf = kv_dtype == GQA_AV_BF16;
  const void* k = reinterpret_cast<const void*>(bf ? pick_main<Bf16Tag>(D) : pick_main<Fp16Tag>(D));
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(D));
  if (e != cudaSuccess) return pfail_cuda(e, "cudaFuncSetAttribute");
  void* args[] = {&p};
  e = launch_pdl(k, sms, kPxThreads, smem_bytes(D), stream, args);
  if (e != cudaSuccess) return pfail_cuda(e, "attention kernel launch");
  const int parts = (p.G * (D / 4) + kPxCombineThreads - 1) / kPxCombineThreads;
  const bool waves = static_cast<long long>(B) * Hkv * parts > 5LL * sms;
  k = reinterpret_cast<const void*>(bf ? pick_combine<Bf16Tag>(D, waves)
                                       : pick_combine<Fp16Tag>(D, waves));
  e = launch_pdl(k, B * Hkv * parts, kPxCombineThreads, 0, stream, args);
  if (e != cudaSuccess) {
    cudaMemsetAsync(&p.head->next, 0, sizeof p.head->next, stream);   // the combine's job
    return pfail_cuda(e, "combine kernel launch");
  }
  return GQA_AV_OK;
} catch (const std::bad_alloc&) {
  return pfail(GQA_AV_ERR_NOMEM, "out of host memory");
}

}  // namespace
}  // namespace gqa_av

using namespace gqa_av;

extern "C" int gqa_prefix_attn_decode(
    const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
    const int32_t* prefix_lens, const int32_t* group_start, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int P, int Hq, int Hkv, int D, int kv_dtype,
    int block_size, int num_blocks, int max_prefix_blocks, int max_blocks, float scale,
    void* stream) {
  g_px_error[0] = 0;
  return decode(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table, seq_lens,
                out, B, P, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_prefix_blocks,
                max_blocks, scale, kPxTimeoutNs, ~0u, static_cast<cudaStream_t>(stream));
}

// The K warp issues no query load from number `withhold_from` of each CTA on
// (nothing of it is in flight), so the MMA warp's wait for it runs out, and
// then the others' waits; all leave as on any timeout.
extern "C" int gqa_prefix_selftest_wait_timeout(
    const void* q, const void* k_pool, const void* v_pool, const int32_t* prefix_table,
    const int32_t* prefix_lens, const int32_t* group_start, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int P, int Hq, int Hkv, int D, int kv_dtype,
    int block_size, int num_blocks, int max_prefix_blocks, int max_blocks, float scale,
    long long wait_ns, int withhold_from, void* stream) {
  g_px_error[0] = 0;
  if (wait_ns < 100000 || wait_ns > kPxTimeoutNs || withhold_from < 0)
    return pfail(GQA_AV_ERR_INVALID, "wait_ns=%lld must be in [100000, %lld], withhold_from=%d not "
                 "negative", wait_ns, kPxTimeoutNs, withhold_from);
  return decode(q, k_pool, v_pool, prefix_table, prefix_lens, group_start, block_table, seq_lens,
                out, B, P, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_prefix_blocks,
                max_blocks, scale, wait_ns, static_cast<unsigned>(withhold_from),
                static_cast<cudaStream_t>(stream));
}

extern "C" int gqa_prefix_device_status(void* stream_, int clear) {
  g_px_error[0] = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return pfail_cuda(e, "cudaGetDevice");
  e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream_));
  if (e != cudaSuccess) return pfail_cuda(e, "cudaStreamSynchronize");
  unsigned word = 0;
  e = cudaMemcpyFromSymbol(&word, px_status, sizeof word);
  if (e != cudaSuccess) return pfail_cuda(e, "reading the status word");
  if (word && clear) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(px_status, &zero, sizeof zero);
    if (e != cudaSuccess) return pfail_cuda(e, "clearing the status word");
  }
  if (word)
    return pfail(GQA_AV_ERR_DEVICE_TIMEOUT, "a bounded wait in the attention kernel ran out (0x%x)",
                 word);
  return GQA_AV_OK;
}

extern "C" int gqa_prefix_release_graph_workspaces(void) {
  g_px_error[0] = 0;
  return PrefixWorkspaces::release_captured();
}

extern "C" const char* gqa_prefix_last_error(void) { return g_px_error; }
