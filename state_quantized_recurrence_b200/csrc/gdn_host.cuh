// What the library's host files share: the per-device error word and the
// argument checks of the operators around the recurrence.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

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
inline gdn_status launched() { return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA; }
}  // namespace gdn
