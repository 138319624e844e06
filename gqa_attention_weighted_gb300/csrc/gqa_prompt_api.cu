// Host side of the C ABI declared in include/gqa_prompt.h: argument checks, the
// calls' workspace, tensor maps and dispatch.
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <mutex>
#include <new>

#include "gqa_paged_host.h"
#include "gqa_prompt.h"
#include "gqa_prompt_kernel.cuh"

namespace gqa_av {
namespace {

thread_local char g_pt_error[512];

int ptfail(int status, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_pt_error, sizeof g_pt_error, fmt, ap);
  va_end(ap);
  return status;
}

int ptfail_cuda(cudaError_t e, const char* what) {
  return ptfail(GQA_AV_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

uintptr_t addr(const void* p) { return reinterpret_cast<uintptr_t>(p); }

constexpr int kMaxTokens = 1 << 20, kMaxHeads = 1 << 10, kMaxWords = 1 << 15;

struct Call {
  const void *q, *k_pool, *v_pool;
  int64_t q_stride;
  const int32_t *token_start, *cached_lens, *tree_mask, *block_table, *seq_lens;
  void* out;
  int words, B, T, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_blocks;
  float scale;
};

int check(const Call& c, bool tree) {
  if (c.B <= 0 || c.T < 0 || c.Hq <= 0 || c.Hkv <= 0 || c.D <= 0 || c.block_size <= 0 ||
      c.num_blocks <= 0 || c.max_blocks <= 0)
    return ptfail(GQA_AV_ERR_INVALID,
                  "sizes must be positive (B=%d Hq=%d Hkv=%d D=%d block_size=%d num_blocks=%d "
                  "max_blocks=%d) and T=%d not negative",
                  c.B, c.Hq, c.Hkv, c.D, c.block_size, c.num_blocks, c.max_blocks, c.T);
  if (c.Hq % c.Hkv) return ptfail(GQA_AV_ERR_INVALID, "Hq=%d is not a multiple of Hkv=%d", c.Hq, c.Hkv);
  if (c.kv_dtype != GQA_AV_BF16 && c.kv_dtype != GQA_AV_FP16)
    return ptfail(GQA_AV_ERR_INVALID, "kv_dtype=%d must be GQA_AV_BF16 or GQA_AV_FP16", c.kv_dtype);
  if (!std::isfinite(c.scale)) return ptfail(GQA_AV_ERR_INVALID, "scale must be finite");
  if (tree && c.words <= 0) return ptfail(GQA_AV_ERR_INVALID, "words=%d must be positive", c.words);
  if (!c.k_pool || !c.v_pool || !c.token_start || !c.block_table ||
      (c.T && (!c.q || !c.out || (tree && !c.tree_mask))) || (tree && !c.cached_lens))
    return ptfail(GQA_AV_ERR_INVALID, "a required pointer is NULL");
  if ((addr(c.token_start) | addr(c.cached_lens) | addr(c.tree_mask) | addr(c.block_table) |
       addr(c.seq_lens)) & 3u)
    return ptfail(GQA_AV_ERR_INVALID, "tables, masks and lengths must be 4-byte aligned");
  if (c.D != 64 && c.D != 128 && c.D != 256)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "D=%d must be 64, 128 or 256", c.D);
  if (c.Hq / c.Hkv > 128)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "Hq / Hkv = %d is above 128", c.Hq / c.Hkv);
  if (c.block_size % 8)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "block_size=%d must be a multiple of 8", c.block_size);
  if (c.B > kPtMaxB || c.T > kMaxTokens || c.Hkv > kMaxHeads || c.words > kMaxWords)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "B=%d is above %d, T=%d above %d, Hkv=%d above %d or "
                  "words=%d above %d", c.B, kPtMaxB, c.T, kMaxTokens, c.Hkv, kMaxHeads, c.words,
                  kMaxWords);
  const long long most = 0x7fffffffLL / c.block_size, longest = (1LL << 26) / c.block_size;
  if (c.num_blocks > most || c.max_blocks > longest)
    return ptfail(GQA_AV_ERR_UNSUPPORTED,
                  "a pool of 2^31 or more cache rows, or a table row of more than 2^26");
  if ((addr(c.q) | addr(c.k_pool) | addr(c.v_pool) | addr(c.out)) & 15u)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "q, the pools and out must be 16-byte aligned");
  if (c.T > 1 && c.q_stride < static_cast<int64_t>(c.Hq) * c.D)
    return ptfail(GQA_AV_ERR_INVALID, "q_stride=%lld is smaller than a token's heads",
                  static_cast<long long>(c.q_stride));
  if (c.T > 1 && (c.q_stride & 7 || c.q_stride >= 1LL << 38))
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "q_stride=%lld must be a multiple of 8 below 2^38",
                  static_cast<long long>(c.q_stride));
  // Units write their rows while others still read.
  const unsigned long long row = 2ull * c.Hq * c.D, pool = 2ull * c.num_blocks * c.block_size * c.Hkv * c.D;
  const unsigned long long q = c.T > 1 ? 2ull * c.q_stride * (c.T - 1) + row : row, b4 = 4ull * c.B;
  const struct { const char* name; const void* at; unsigned long long n; } ins[] = {
      {"q", c.q, q}, {"k_pool", c.k_pool, pool}, {"v_pool", c.v_pool, pool},
      {"token_start", c.token_start, b4 + 4}, {"cached_lens", c.cached_lens, b4},
      {"tree_mask", c.tree_mask, 4ull * c.T * c.words}, {"seq_lens", c.seq_lens, b4},
      {"block_table", c.block_table, b4 * c.max_blocks}};
  for (const auto& i : ins)
    if (c.T && i.at && addr(i.at) < addr(c.out) + row * c.T && addr(c.out) < addr(i.at) + i.n)
      return ptfail(GQA_AV_ERR_INVALID, "out overlaps %s", i.name);
  return GQA_AV_OK;
}

using PromptKernel = void (*)(PromptParams);

template <typename Tag>
PromptKernel pick(int D) {
  return D == 64 ? gqa_prompt_kernel<Tag, 64>
                 : D == 128 ? gqa_prompt_kernel<Tag, 128> : gqa_prompt_kernel<Tag, 256>;
}
int smem_bytes(int D) {
  return D == 64 ? PtShape<64>::SMEM : D == 128 ? PtShape<128>::SMEM : PtShape<256>::SMEM;
}

using PromptWorkspaces = Workspaces<sizeof(PtHeader), ptfail>;

int encode_maps(PromptParams* p, const Call& c) {
  const cuuint64_t d = c.D, G = p->G, Hkv = p->Hkv;
  const cuuint64_t rows = static_cast<cuuint64_t>(p->bs) * p->num_blocks;
  const cuuint64_t qd[4] = {d, G, Hkv, static_cast<cuuint64_t>(p->T)};
  const cuuint64_t stride = c.T > 1 ? static_cast<cuuint64_t>(c.q_stride) : d * G * Hkv;
  const cuuint64_t qs[3] = {d * 2, G * d * 2, stride * 2};
  const cuuint32_t tile[4] = {64, static_cast<cuuint32_t>(p->G), 1, static_cast<cuuint32_t>(p->TB)};
  const cuuint64_t kd[3] = {d, Hkv, rows};
  const cuuint64_t ks[2] = {d * 2, Hkv * d * 2};
  const cuuint32_t kb[3] = {64, 1, static_cast<cuuint32_t>(p->R)};
  int rc = encode_map(ptfail, &p->q_map, c.q, 4, qd, qs, tile, "q");
  if (!rc) rc = encode_map(ptfail, &p->k_map, c.k_pool, 3, kd, ks, kb, "K");
  if (!rc) rc = encode_map(ptfail, &p->v_map, c.v_pool, 3, kd, ks, kb, "V");
  return rc;
}

// What the self-tests change.
struct Trial {
  long long wait_ns = kPtTimeoutNs;
  unsigned withhold_from = ~0u, late_from = ~0u;
  long long late_ns = 0;
};

int attend(const Call& c, bool tree, cudaStream_t stream, const Trial& trial = {}) try {
  int rc = check(c, tree);
  if (rc) return rc;
  if (c.T == 0) return GQA_AV_OK;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return ptfail_cuda(e, "cudaGetDevice");

  PromptParams p;
  p.token_start = c.token_start; p.cached_lens = c.cached_lens;
  p.tree_mask = tree ? c.tree_mask : nullptr;
  p.block_table = c.block_table; p.seq_lens = c.seq_lens;
  p.v_pool = c.v_pool; p.out = c.out;
  p.B = c.B; p.T = c.T; p.Hq = c.Hq; p.Hkv = c.Hkv; p.G = c.Hq / c.Hkv; p.TB = 128 / p.G;
  p.words = c.words;
  p.bs = c.block_size; p.num_blocks = c.num_blocks; p.max_blocks = c.max_blocks;
  block_divisor(c.block_size, &p.bs_mul, &p.bs_shift);
  const int keys = c.D == 256 ? PtShape<256>::KEYS : PtShape<128>::KEYS;
  for (p.R = 8; p.R < keys && c.block_size % (2 * p.R) == 0;) p.R *= 2;
  // log2(e) in the scale; a scale of 0 becomes the smallest normal number, which
  // leaves every finite score at 0 and keeps masked ones at -inf.
  const double s2 = std::fabs(static_cast<double>(c.scale)) * 1.4426950408889634;
  if (s2 > FLT_MAX) return ptfail(GQA_AV_ERR_UNSUPPORTED, "scale=%g is too large", (double)c.scale);
  p.qscale = std::max(static_cast<float>(s2), FLT_MIN);
  p.negate = c.scale < 0.0f;
  p.timeout_ns = trial.wait_ns;
  p.withhold_from = trial.withhold_from;
  p.late_from = trial.late_from;
  p.late_ns = trial.late_ns;

  // Items: query tiles, one more a sequence than its tokens fill. Slots: a chunk is
  // at least a quarter of an SM's share of the work, so all chunks are at most 4 an
  // SM, and an item that is cut has more than one and takes less than one more. A
  // chunk is also at least kPtMinChunk key tiles, so a query tile of t key tiles has at
  // most ceil(t / kPtMinChunk) slots, and a pair, which counts 2 t, at most twice that.
  const int ns = c.D == 256 ? 1 : 2;
  const long long items = (c.T + p.TB - 1) / p.TB + std::min(c.B, c.T);
  p.small = c.B <= kPtSmall && items <= kPtSmall;
  const long long slots = std::min(8LL * sms, 4LL * sms + items * c.Hkv);
  const long long tiles = (static_cast<long long>(c.max_blocks) * c.block_size + keys - 1) / keys;
  const long long few = std::min(slots, items * c.Hkv * ((tiles + kPtMinChunk - 1) / kPtMinChunk));
  if ((items + 8LL * sms) * c.Hkv > 0x7fffffffLL)
    return ptfail(GQA_AV_ERR_UNSUPPORTED, "T=%d tokens of %d KV heads are too many for one call",
                  c.T, c.Hkv);
  const size_t at_splits = up256(sizeof(PtHeader));
  const size_t at_units = at_splits + up256(8 * static_cast<size_t>(sms) * sizeof(PtSplit));
  const size_t at_ml = at_units + up256(static_cast<size_t>(items + 8 * sms) * sizeof(PtUnit));
  bool capturing = false;
  Workspace* ws = nullptr;
  if ((rc = PromptWorkspaces::find(dev, stream, &capturing, &ws))) return rc;
  std::lock_guard<std::mutex> lk(ws->mu);
  // A stream's workspace, of which there are few, is made large enough for any
  // lengths at once. A capture's holds what its calls can need (7 drafts of 2 heads of
  // 64 over tables of 512 rows: 0.3 MB where a stream's has 41): a server keeps one a
  // graph. If a later call of the capture needs more, it at least doubles, because
  // what was outgrown stays, up to what a stream would have.
  const size_t slot = static_cast<size_t>(ns) * 128 * (c.D + 2) * 4, all = at_ml + slots * slot;
  size_t need = capturing ? at_ml + few * slot : all;
  if (ws->bytes < need && ws->bytes) need = std::max(need, std::min(all, 2 * ws->bytes));
  if ((rc = PromptWorkspaces::grow(ws, capturing, need, stream))) return rc;
  const size_t at_o = at_ml + static_cast<size_t>(capturing ? few : slots) * ns * 128 * 8;
  char* base = ws->base;
  p.head = reinterpret_cast<PtHeader*>(base);
  p.splits = reinterpret_cast<PtSplit*>(base + at_splits);
  p.units = reinterpret_cast<PtUnit*>(base + at_units);
  p.part_ml = reinterpret_cast<float2*>(base + at_ml);
  p.part_o = reinterpret_cast<float*>(base + at_o);
  if ((rc = encode_maps(&p, c))) return rc;

  const void* k = reinterpret_cast<const void*>(
      c.kv_dtype == GQA_AV_BF16 ? pick<Bf16Tag>(c.D) : pick<Fp16Tag>(c.D));
  static std::atomic<unsigned long long> allowed[6];   // of each kernel
  e = allow_smem(k, smem_bytes(c.D), dev,
                 &allowed[(c.D == 64 ? 0 : c.D == 128 ? 2 : 4) + (c.kv_dtype == GQA_AV_FP16)]);
  if (e != cudaSuccess) return ptfail_cuda(e, "cudaFuncSetAttribute");
  void* args[] = {&p};
  e = launch_pdl(k, sms, kPtThreads, smem_bytes(c.D), stream, args);
  if (e != cudaSuccess) return ptfail_cuda(e, "attention kernel launch");
  return GQA_AV_OK;
} catch (const std::bad_alloc&) {
  return ptfail(GQA_AV_ERR_NOMEM, "out of host memory");
}

}  // namespace
}  // namespace gqa_av

using namespace gqa_av;

extern "C" int gqa_prompt_attn(const void* q, int64_t q_stride, const void* k_pool,
                               const void* v_pool, const int32_t* token_start,
                               const int32_t* cached_lens, const int32_t* block_table,
                               const int32_t* seq_lens, void* out, int B, int T, int Hq, int Hkv,
                               int D, int kv_dtype, int block_size, int num_blocks, int max_blocks,
                               float scale, void* stream) {
  g_pt_error[0] = 0;
  const Call c = {q, k_pool, v_pool, q_stride, token_start, cached_lens, nullptr, block_table,
                  seq_lens, out, 0, B, T, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_blocks,
                  scale};
  return attend(c, false, static_cast<cudaStream_t>(stream));
}

extern "C" int gqa_tree_attn(const void* q, int64_t q_stride, const void* k_pool,
                             const void* v_pool, const int32_t* token_start,
                             const int32_t* cached_lens, const int32_t* tree_mask, int words,
                             const int32_t* block_table, const int32_t* seq_lens, void* out, int B,
                             int T, int Hq, int Hkv, int D, int kv_dtype, int block_size,
                             int num_blocks, int max_blocks, float scale, void* stream) {
  g_pt_error[0] = 0;
  const Call c = {q, k_pool, v_pool, q_stride, token_start, cached_lens, tree_mask, block_table,
                  seq_lens, out, words, B, T, Hq, Hkv, D, kv_dtype, block_size, num_blocks,
                  max_blocks, scale};
  return attend(c, true, static_cast<cudaStream_t>(stream));
}

// The K warp issues no query load from number `withhold_from` of each CTA on
// (nothing of it is in flight), so the MMA warp's wait for it runs out, and
// then the others' waits; all leave as on any timeout.
extern "C" int gqa_prompt_selftest_wait_timeout(
    const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
    const int32_t* token_start, const int32_t* cached_lens, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int T, int Hq, int Hkv, int D, int kv_dtype,
    int block_size, int num_blocks, int max_blocks, float scale, long long wait_ns,
    int withhold_from, void* stream) {
  g_pt_error[0] = 0;
  if (wait_ns < 100000 || wait_ns > kPtTimeoutNs || withhold_from < 0)
    return ptfail(GQA_AV_ERR_INVALID, "wait_ns=%lld must be in [100000, %lld], withhold_from=%d not "
                  "negative", wait_ns, kPtTimeoutNs, withhold_from);
  const Call c = {q, k_pool, v_pool, q_stride, token_start, cached_lens, nullptr, block_table,
                  seq_lens, out, 0, B, T, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_blocks,
                  scale};
  Trial t;
  t.wait_ns = wait_ns;
  t.withhold_from = static_cast<unsigned>(withhold_from);
  return attend(c, false, static_cast<cudaStream_t>(stream), t);
}

extern "C" int gqa_prompt_selftest_late_start(
    const void* q, int64_t q_stride, const void* k_pool, const void* v_pool,
    const int32_t* token_start, const int32_t* cached_lens, const int32_t* block_table,
    const int32_t* seq_lens, void* out, int B, int T, int Hq, int Hkv, int D, int kv_dtype,
    int block_size, int num_blocks, int max_blocks, float scale, long long wait_ns, int late_from,
    long long late_ns, void* stream) {
  g_pt_error[0] = 0;
  if (wait_ns < 100000 || wait_ns > kPtTimeoutNs || late_from < 0 || late_ns < 0 || late_ns > kPtTimeoutNs)
    return ptfail(GQA_AV_ERR_INVALID, "wait_ns=%lld must be in [100000, %lld], late_from=%d not negative "
                  "and late_ns=%lld in [0, %lld]", wait_ns, kPtTimeoutNs, late_from, late_ns, kPtTimeoutNs);
  const Call c = {q, k_pool, v_pool, q_stride, token_start, cached_lens, nullptr, block_table,
                  seq_lens, out, 0, B, T, Hq, Hkv, D, kv_dtype, block_size, num_blocks, max_blocks,
                  scale};
  Trial t;
  t.wait_ns = wait_ns;
  t.late_from = static_cast<unsigned>(late_from);
  t.late_ns = late_ns;
  return attend(c, false, static_cast<cudaStream_t>(stream), t);
}

extern "C" int gqa_prompt_device_status(void* stream_, int clear) {
  g_pt_error[0] = 0;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return ptfail_cuda(e, "cudaGetDevice");
  e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream_));
  if (e != cudaSuccess) return ptfail_cuda(e, "cudaStreamSynchronize");
  unsigned word = 0;
  e = cudaMemcpyFromSymbol(&word, pt_status, sizeof word);
  if (e != cudaSuccess) return ptfail_cuda(e, "reading the status word");
  if (word && clear) {
    const unsigned zero = 0;
    e = cudaMemcpyToSymbol(pt_status, &zero, sizeof zero);
    if (e != cudaSuccess) return ptfail_cuda(e, "clearing the status word");
  }
  if (word)
    return ptfail(GQA_AV_ERR_DEVICE_TIMEOUT, "a bounded wait in the attention kernel ran out (0x%x)",
                  word);
  return GQA_AV_OK;
}

extern "C" int gqa_prompt_release_graph_workspaces(void) {
  g_pt_error[0] = 0;
  return PromptWorkspaces::release_captured();
}

extern "C" const char* gqa_prompt_last_error(void) { return g_pt_error; }
