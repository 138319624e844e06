// Host side of the C ABI declared in include/gqa_prefix.h: argument checks, the
// call's workspace, tensor maps and dispatch to the attention and combine
// kernels.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <map>
#include <memory>
#include <mutex>
#include <new>
#include <tuple>
#include <vector>

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

// Workspaces. A call's units, plan and partial results lie in device memory
// until its combine has run, so calls that may run at the same time must not
// share a buffer. One belongs to each stream of uncaptured calls (which the
// stream orders), and one to each stream of a capture into a graph: replays of
// a graph follow one another, but may overlap with anything else. The latter
// are kept until the caller says that the graphs are gone: a graph that owns
// its buffer as a user object tells so by itself, but then each of its launches
// holds the host up until the one before has ended (measured: 2 us a replay
// become 13 to 45).
struct Owner {
  int dev;
  const void* stream;
  unsigned long long capture;    // 0: uncaptured
  bool operator<(const Owner& o) const {
    return std::tie(dev, stream, capture) < std::tie(o.dev, o.stream, o.capture);
  }
};
struct Workspace {
  std::mutex mu;                 // held until a call's kernels are launched: the stream's order
  char* base = nullptr;
  size_t bytes = 0;
  std::vector<char*> outgrown;   // by a capture, whose earlier calls use them
};
std::mutex g_px_mu;
std::map<Owner, std::unique_ptr<Workspace>> g_px_ws;

// Allocation is allowed while a stream is capturing in this mode of the thread.
struct RelaxedCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Grows a workspace, whose lock is held, to `need` bytes. The new one's header
// is zeroed on return.
int grow(Workspace* w, bool capturing, size_t need, cudaStream_t stream) {
  if (w->bytes >= need) return GQA_AV_OK;
  const size_t bytes = capturing ? need : std::max(need, w->bytes + w->bytes / 2);
  w->outgrown.reserve(w->outgrown.size() + 1);
  RelaxedCapture relaxed;
  void* p = nullptr;
  cudaError_t e = cudaMalloc(&p, bytes);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return pfail(GQA_AV_ERR_NOMEM, "cudaMalloc(%zu) failed: %s", bytes, cudaGetErrorString(e));
  }
  cudaStream_t own = nullptr;    // not the legacy stream: others may be capturing
  e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
  if (e == cudaSuccess) {
    e = cudaMemsetAsync(p, 0, sizeof(PxHeader), own);
    if (e == cudaSuccess) e = cudaStreamSynchronize(own);
    cudaStreamDestroy(own);
  }
  if (e == cudaSuccess && w->base && !capturing) {
    e = cudaStreamSynchronize(stream);   // calls under way use the old one
    if (e == cudaSuccess) cudaFree(w->base);
  }
  if (e != cudaSuccess) {
    cudaFree(p);
    return pfail_cuda(e, "setting the workspace up");
  }
  if (w->base && capturing) w->outgrown.push_back(w->base);
  w->base = static_cast<char*>(p);
  w->bytes = bytes;
  return GQA_AV_OK;
}

// The workspace that a call on `stream` uses. Those of uncaptured calls are
// never taken away, so a thread remembers its last one.
int find_workspace(int dev, cudaStream_t stream, bool* capturing, Workspace** out) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  cudaError_t e = cudaStreamIsCapturing(stream, &cs);
  if (e == cudaSuccess && cs == cudaStreamCaptureStatusInvalidated)
    e = cudaErrorStreamCaptureInvalidated;
  if (e != cudaSuccess) return pfail_cuda(e, "cudaStreamIsCapturing");
  *capturing = cs == cudaStreamCaptureStatusActive;
  static thread_local char per_thread;   // each thread's default stream has the same handle
  const void* key = stream == cudaStreamPerThread ? static_cast<const void*>(&per_thread)
                    : stream == cudaStreamLegacy  ? nullptr
                                                  : static_cast<const void*>(stream);
  static thread_local Owner last{-1, nullptr, 0};
  static thread_local Workspace* last_ws = nullptr;
  if (!*capturing && last.dev == dev && last.stream == key) {
    *out = last_ws;
    return GQA_AV_OK;
  }
  unsigned long long id = 0;
  if (*capturing) {
    e = cudaStreamGetCaptureInfo(stream, &cs, &id, nullptr, nullptr, nullptr, nullptr);
    if (e != cudaSuccess) return pfail_cuda(e, "cudaStreamGetCaptureInfo");
  }
  const Owner owner{dev, key, id};
  std::lock_guard<std::mutex> lk(g_px_mu);
  std::unique_ptr<Workspace>& w = g_px_ws[owner];
  if (!w) w = std::make_unique<Workspace>();
  *out = w.get();
  if (!*capturing) {
    last = owner;
    last_ws = w.get();
  }
  return GQA_AV_OK;
}

// A map over 16-bit elements: `rank` dimensions, boxes 64 elements wide in the
// 128-byte swizzle. What lies outside reads as zeros.
int encode(CUtensorMap* m, const void* x, int rank, const cuuint64_t* dims,
           const cuuint64_t* strides, const cuuint32_t* box, const char* what) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode_tiled = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                     cudaEnableDefault, &q);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(
        e == cudaSuccess && q == cudaDriverEntryPointSuccess ? f : nullptr);
  }();
  if (!encode_tiled)
    return pfail(GQA_AV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void*>(x), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return pfail(GQA_AV_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled (%s) failed (%d)", what, (int)r);
  return GQA_AV_OK;
}

int encode_maps(PrefixParams* p, const void* q, const void* k_pool, const void* v_pool, int D) {
  const cuuint64_t d = D, G = p->G, Hkv = p->Hkv, rows = static_cast<cuuint64_t>(p->bs) * p->num_blocks;
  const cuuint64_t qd[4] = {d, G, Hkv, static_cast<cuuint64_t>(p->B)};
  const cuuint64_t qs[3] = {d * 2, G * d * 2, Hkv * G * d * 2};
  const cuuint32_t tile[4] = {64, static_cast<cuuint32_t>(p->G), 1, static_cast<cuuint32_t>(p->TB)};
  const cuuint32_t one[4] = {64, static_cast<cuuint32_t>(p->G), 1, 1};
  const cuuint64_t kd[3] = {d, Hkv, rows};
  const cuuint64_t ks[2] = {d * 2, Hkv * d * 2};
  const cuuint32_t kb[3] = {64, 1, static_cast<cuuint32_t>(p->R)};
  int rc = encode(&p->q_tile_map, q, 4, qd, qs, tile, "q");
  if (!rc) rc = encode(&p->q_one_map, q, 4, qd, qs, one, "q");
  if (!rc) rc = encode(&p->k_map, k_pool, 3, kd, ks, kb, "K");
  if (!rc) rc = encode(&p->v_map, v_pool, 3, kd, ks, kb, "V");
  return rc;
}

cudaError_t launch_pdl(const void* fn, int grid, int block, size_t smem, cudaStream_t stream,
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

size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

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
  // Division by the block size as a product: with shift = 28 + ceil(log2(bs)) the
  // rounded-up factor is below 2^30 and off by less than 2^-28 bs, relatively to
  // 2^shift, which a dividend below 2^26 does not notice.
  for (p.bs_shift = 28; (1LL << (p.bs_shift - 28)) < block_size;) ++p.bs_shift;
  p.bs_mul = static_cast<unsigned>(((1ULL << p.bs_shift) + block_size - 1) / block_size);
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
  if ((rc = find_workspace(dev, stream, &capturing, &ws))) return rc;
  std::lock_guard<std::mutex> lk(ws->mu);
  if ((rc = grow(ws, capturing, at_om + own_slots * p.G * 8, stream))) return rc;
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
  std::lock_guard<std::mutex> lk(g_px_mu);
  RelaxedCapture relaxed;
  cudaError_t first = cudaSuccess;
  for (auto it = g_px_ws.begin(); it != g_px_ws.end();) {
    if (!it->first.capture) {
      ++it;
      continue;
    }
    cudaError_t e = cudaFree(it->second->base);
    if (first == cudaSuccess) first = e;
    for (char* p : it->second->outgrown) cudaFree(p);
    it = g_px_ws.erase(it);
  }
  return first == cudaSuccess ? GQA_AV_OK : pfail_cuda(first, "cudaFree");
}

extern "C" const char* gqa_prefix_last_error(void) { return g_px_error; }
