// host.cuh -- host-side helpers shared by the two halves of the C ABI (la_api.cu, block_api.cu).
#pragma once
#include <atomic>
#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "la.h"

namespace la {

// Kernels queued by the last successful entry point on this host thread (la_last_launch_count).
extern thread_local int g_last_launches;

// Reads and clears block_api.cu's copy of the device error word (each translation unit has its own).
cudaError_t take_block_error(unsigned int* value);

inline bool aligned16(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15u) == 0; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The current device's SM count (asked once per device: it does not change).
inline int current_sm_count(int* sm) {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return LA_ERR_CUDA;
  if (dev < 64 && (*sm = known[dev].load(std::memory_order_relaxed)) > 0) return LA_OK;
  if (cudaDeviceGetAttribute(sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return LA_ERR_CUDA;
  if (dev < 64) known[dev].store(*sm, std::memory_order_relaxed);
  return LA_OK;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult qr;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &qr) == cudaSuccess &&
        qr == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// Encodes a tensor map (the arguments are cuTensorMapEncodeTiled's).  A driver call needs a context that
// is current in the calling thread, and a host thread has none before its first runtime call that needs
// one: that of its current device is made current then.
template <typename... Args>
bool encode_tiled(const Args&... args) {
  const EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  CUresult r = enc(args...);
  int dev = 0;
  if ((r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED) && cudaGetDevice(&dev) == cudaSuccess &&
      cudaSetDevice(dev) == cudaSuccess)
    r = enc(args...);
  return r == CUDA_SUCCESS;
}

inline int launched_ok() { return cudaGetLastError() == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

// Launches `kern`; with `pdl` it may start while the previous kernel in the stream is still
// running (programmatic stream serialization).  Only kernels whose predecessor in the stream is
// one of this library's own kernels get `pdl`, and each of them calls pdl_wait() before reading
// anything produced before it; what they read earlier (K, V, G) was produced before the first
// kernel of the call, which is launched normally.
template <typename... KArgs, typename... Args>
int launch_k(void (*kern)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, bool pdl,
             const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(args)...) == cudaSuccess ? LA_OK : LA_ERR_CUDA;
}

template <typename F>
int set_smem(F* kern, size_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes)) == cudaSuccess
             ? LA_OK
             : LA_ERR_CUDA;
}

// What the driver has been told (dynamic shared memory) or has said (registers) of a kernel on a
// device, so that a call need not go to it again: a small open-addressed table, filled as kernels are
// first used.  A full table costs only the driver calls.
class KernelTable {
 public:
  // set_smem(), unless at least as many bytes are set already.
  template <typename F>
  int smem(F* kern, size_t bytes) {
    Entry* e = find(reinterpret_cast<const void*>(kern));
    if (e && e->bytes.load(std::memory_order_acquire) >= int(bytes)) return LA_OK;
    std::lock_guard<std::mutex> lock(mutex_);  // (two threads: the larger value has to be the last one set)
    if (e && e->bytes.load(std::memory_order_acquire) >= int(bytes)) return LA_OK;
    if (set_smem(kern, bytes)) return LA_ERR_CUDA;
    if (e) e->bytes.store(int(bytes), std::memory_order_release);
    return LA_OK;
  }
  // Whether the kernel's launch grants at least `regs` registers a thread.
  template <typename F>
  bool regs(F* kern, uint32_t regs) {
    Entry* e = find(reinterpret_cast<const void*>(kern));
    if (e && e->regs.load(std::memory_order_relaxed) > 0) return uint32_t(e->regs.load(std::memory_order_relaxed)) >= regs;
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) != cudaSuccess) return false;
    if (e) e->regs.store(at.numRegs, std::memory_order_relaxed);
    return uint32_t(at.numRegs) >= regs;
  }

 private:
  struct Entry {
    std::atomic<uintptr_t> key{0};
    std::atomic<int> bytes{0}, regs{0};
  };
  static constexpr size_t SIZE = 1024;
  Entry table_[SIZE];
  std::mutex mutex_;

  Entry* find(const void* kern) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    // (host stubs are at least 4 bytes apart and below 2^56, devices below 256)
    const uintptr_t key = (reinterpret_cast<uintptr_t>(kern) << 8) | uintptr_t(dev & 255);
    for (size_t i = 0, at = (key * 0x9E3779B97F4A7C15ull) >> 54; i < 16; ++i) {
      Entry& e = table_[(at + i) % SIZE];
      uintptr_t k = e.key.load(std::memory_order_acquire);
      if (k == key) return &e;
      if (k == 0 && (e.key.compare_exchange_strong(k, key) || k == key)) return &e;
    }
    return nullptr;
  }
};

}  // namespace la
