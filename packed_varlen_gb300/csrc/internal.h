// Internal interface between the C-ABI layer (api.cu) and the kernel
// translation units.  Not installed, not part of the ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "packedattn.h"

namespace pa {

// Everything an attention launch needs; filled and validated by api.cu and
// prompt_attn.cu.
struct VarlenArgs {
  const void *q, *k, *v;
  void *out;
  const int32_t *cu_q, *cu_k;
  int32_t batch, total_q, total_k, max_q, max_k, H, D;
  float scale;
  int32_t *status;  // device address of the per-device status word
  int num_sms;
  int32_t Hkv, causal;                     // K/V heads, causal order
  int64_t q_stride, k_stride, v_stride;    // elements from one token to the next
};

struct BlockWindowArgs {
  const void *q, *k, *v;
  void *out;
  int32_t batch, n, block, look_back, look_ahead, H, D;
  float scale;
  int32_t *status;
  int num_sms;
};

// A paged K/V cache as the C ABI receives it.
struct PagedCacheArgs {
  void *k, *v;
  uint8_t *k_exp, *v_exp;
  const int32_t *table;
  int32_t num_pages, page_size, table_pages;
  int64_t page_stride;
  int32_t Hkv, D, format;
};
struct PagedCache;   // paged.cuh

// The checks every entry point over a paged cache makes; fills `c` on PA_OK.
pa_status check_cache(const PagedCacheArgs &a, PagedCache &c);

inline bool aligned_to(const void *p, uintptr_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
}

// Raises a kernel's dynamic shared-memory limit once per device (the
// attribute persists; setting it on every launch costs host time between
// back-to-back launches).  `done` is the caller's per-kernel device bitmask.
inline cudaError_t set_smem_once(const void *kernel, int smem, unsigned long long &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  if (__atomic_load_n(&done, __ATOMIC_ACQUIRE) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) __atomic_fetch_or(&done, bit, __ATOMIC_ACQ_REL);
  return e;
}

// Launches `kernel` so that it may set itself up (barriers, TMEM, descriptors)
// while the kernel before it on the stream ends: it must execute griddep_wait()
// before its first access to global memory, and griddep_launch_dependents() lets
// the next one do the same.
template <typename... P, typename... A>
cudaError_t launch_beside(void (*kernel)(P...), dim3 grid, int threads, int smem,
                          cudaStream_t stream, const A &...args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Device address of the per-device status word and the SM count of the
// current device (api.cu).
cudaError_t device_context(int32_t **status, int *num_sms);

// Maps a CUDA error to a pa_status and remembers it for pa_last_cuda_error.
pa_status from_cuda(cudaError_t e);

// Launchers (launch_varlen_attn takes the kernel of the head dim): return cudaSuccess or the launch error.
cudaError_t launch_varlen_attn(const VarlenArgs &a, cudaStream_t stream);
cudaError_t launch_varlen_attn_pair(const VarlenArgs &a, cudaStream_t stream);   // D = 128
cudaError_t launch_block_window_attn(const BlockWindowArgs &a, cudaStream_t stream);

}  // namespace pa
