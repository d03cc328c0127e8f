// What the library's host files share: the per-device error word and the
// argument checks of the operators around the recurrence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "gdn_qdq.h"

namespace gdn {
// Device address of the current device's error word (kErr* bits, read and
// cleared by gdn_last_error()).
gdn_status error_word(unsigned **out);

inline bool aligned_to(const void *p, uintptr_t a) {
  return reinterpret_cast<uintptr_t>(p) % a == 0;
}
inline size_t elem_bytes(gdn_dtype dt) { return dt == GDN_DTYPE_BF16 ? 2 : 4; }
inline bool known_dtype(gdn_dtype dt) { return dt == GDN_DTYPE_BF16 || dt == GDN_DTYPE_F32; }
// Allows `kern` its dynamic shared memory on the current device, once for
// each device (`done`: one flag a device, a static of the kernel's launcher).
template <typename K>
bool allow_smem(K kern, int bytes, std::atomic<uint64_t> &done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done.fetch_or(bit, std::memory_order_release);
  return true;
}
inline gdn_status launched() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
}  // namespace gdn
