// Host side that the calls over paged pools share: workspaces by stream and
// capture, tensor maps, launches behind a programmatic dependency.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <map>
#include <memory>
#include <mutex>
#include <tuple>
#include <vector>

#include "gqa_av.h"

namespace gqa_av {

// Records a formatted message and returns the status: each call's own.
using FailFn = int (*)(int status, const char* fmt, ...);

// Workspaces. A call's units, plan and partial results lie in device memory
// until its last kernel has run, so calls that may run at the same time must not
// share a buffer. One belongs to each stream of uncaptured calls (which the
// stream orders), and one to each stream of a capture into a graph: replays of
// a graph follow one another, but may overlap with anything else. The latter
// are kept until the caller says that the graphs are gone: a graph that owns
// its buffer as a user object tells so by itself, but then each of its launches
// holds the host up until the one before has ended (measured: 2 us a replay
// become 13 to 45).
struct WorkspaceOwner {
  int dev;
  const void* stream;
  unsigned long long capture;    // 0: uncaptured
  bool operator<(const WorkspaceOwner& o) const {
    return std::tie(dev, stream, capture) < std::tie(o.dev, o.stream, o.capture);
  }
};
struct Workspace {
  std::mutex mu;                 // held until a call's kernels are launched: the stream's order
  char* base = nullptr;
  size_t bytes = 0;
  std::vector<char*> outgrown;   // by a capture, whose earlier calls use them
};

// Allocation is allowed while a stream is capturing in this mode of the thread.
struct RelaxedCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~RelaxedCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// One call's workspaces. `header` bytes at the head of each are zeroed when it
// is made.
template <size_t header, FailFn fail>
class Workspaces {
 public:
  // Grows a workspace, whose lock is held, to `need` bytes.
  static int grow(Workspace* w, bool capturing, size_t need, cudaStream_t stream) {
    if (w->bytes >= need) return GQA_AV_OK;
    const size_t bytes = capturing ? need : std::max(need, w->bytes + w->bytes / 2);
    w->outgrown.reserve(w->outgrown.size() + 1);
    RelaxedCapture relaxed;
    void* p = nullptr;
    cudaError_t e = cudaMalloc(&p, bytes);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(GQA_AV_ERR_NOMEM, "cudaMalloc(%zu) failed: %s", bytes, cudaGetErrorString(e));
    }
    cudaStream_t own = nullptr;    // not the legacy stream: others may be capturing
    e = cudaStreamCreateWithFlags(&own, cudaStreamNonBlocking);
    if (e == cudaSuccess) {
      e = cudaMemsetAsync(p, 0, header, own);
      if (e == cudaSuccess) e = cudaStreamSynchronize(own);
      cudaStreamDestroy(own);
    }
    if (e == cudaSuccess && w->base && !capturing) {
      e = cudaStreamSynchronize(stream);   // calls under way use the old one
      if (e == cudaSuccess) cudaFree(w->base);
    }
    if (e != cudaSuccess) {
      cudaFree(p);
      return fail(GQA_AV_ERR_CUDA, "setting the workspace up: %s", cudaGetErrorString(e));
    }
    if (w->base && capturing) w->outgrown.push_back(w->base);
    w->base = static_cast<char*>(p);
    w->bytes = bytes;
    return GQA_AV_OK;
  }

  // The workspace that a call on `stream` uses. Those of uncaptured calls are
  // never taken away, so a thread remembers its last one.
  static int find(int dev, cudaStream_t stream, bool* capturing, Workspace** out) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    cudaError_t e = cudaStreamIsCapturing(stream, &cs);
    if (e == cudaSuccess && cs == cudaStreamCaptureStatusInvalidated)
      e = cudaErrorStreamCaptureInvalidated;
    if (e != cudaSuccess)
      return fail(GQA_AV_ERR_CUDA, "cudaStreamIsCapturing: %s", cudaGetErrorString(e));
    *capturing = cs == cudaStreamCaptureStatusActive;
    static thread_local char per_thread;   // each thread's default stream has the same handle
    const void* key = stream == cudaStreamPerThread ? static_cast<const void*>(&per_thread)
                      : stream == cudaStreamLegacy  ? nullptr
                                                    : static_cast<const void*>(stream);
    static thread_local WorkspaceOwner last{-1, nullptr, 0};
    static thread_local Workspace* last_ws = nullptr;
    if (!*capturing && last.dev == dev && last.stream == key) {
      *out = last_ws;
      return GQA_AV_OK;
    }
    unsigned long long id = 0;
    if (*capturing) {
      e = cudaStreamGetCaptureInfo(stream, &cs, &id, nullptr, nullptr, nullptr, nullptr);
      if (e != cudaSuccess)
        return fail(GQA_AV_ERR_CUDA, "cudaStreamGetCaptureInfo: %s", cudaGetErrorString(e));
    }
    const WorkspaceOwner owner{dev, key, id};
    std::lock_guard<std::mutex> lk(mu_);
    std::unique_ptr<Workspace>& w = all_[owner];
    if (!w) w = std::make_unique<Workspace>();
    *out = w.get();
    if (!*capturing) {
      last = owner;
      last_ws = w.get();
    }
    return GQA_AV_OK;
  }

  // Frees the workspaces of all captures.
  static int release_captured() {
    std::lock_guard<std::mutex> lk(mu_);
    RelaxedCapture relaxed;
    cudaError_t first = cudaSuccess;
    for (auto it = all_.begin(); it != all_.end();) {
      if (!it->first.capture) {
        ++it;
        continue;
      }
      cudaError_t e = cudaFree(it->second->base);
      if (first == cudaSuccess) first = e;
      for (char* p : it->second->outgrown) cudaFree(p);
      it = all_.erase(it);
    }
    return first == cudaSuccess
               ? GQA_AV_OK
               : fail(GQA_AV_ERR_CUDA, "cudaFree: %s", cudaGetErrorString(first));
  }

 private:
  static inline std::mutex mu_;
  static inline std::map<WorkspaceOwner, std::unique_ptr<Workspace>> all_;
};

// A map over 16-bit elements: `rank` dimensions, boxes 64 elements wide in the
// 128-byte swizzle. What lies outside reads as zeros.
inline int encode_map(FailFn fail, CUtensorMap* m, const void* x, int rank, const cuuint64_t* dims,
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
    return fail(GQA_AV_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT16, rank, const_cast<void*>(x), dims,
                           strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(GQA_AV_ERR_UNSUPPORTED, "cuTensorMapEncodeTiled (%s) failed (%d)", what, (int)r);
  return GQA_AV_OK;
}

inline cudaError_t launch_pdl(const void* fn, int grid, int block, size_t smem, cudaStream_t stream,
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

// Lets a kernel have `bytes` of dynamic shared memory, once a device (`done`: a
// bit each, the kernel's own).
inline cudaError_t allow_smem(const void* fn, int bytes, int dev, std::atomic<unsigned long long>* done) {
  const unsigned long long bit = 1ull << (dev & 63);
  if (dev < 64 && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Division by a block size as a product: with shift = 28 + ceil(log2(bs)) the
// rounded-up factor is below 2^30 and off by less than 2^-28 bs, relatively to
// 2^shift, which a dividend below 2^26 does not notice.
inline void block_divisor(int block_size, unsigned* mul, int* shift) {
  for (*shift = 28; (1LL << (*shift - 28)) < block_size;) ++*shift;
  *mul = static_cast<unsigned>(((1ULL << *shift) + block_size - 1) / block_size);
}

}  // namespace gqa_av
