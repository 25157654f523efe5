// Host-side helpers shared by the translation units that implement C entry
// points: the calling thread's error text, the device check, and the driver's
// tensor-map encoder. Defined in flce_api.cu.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "flce.h"

namespace flce {
namespace host {

// Records the text that flce_last_error() returns; returns `s`.
flce_status fail(flce_status s, const char* fmt, ...);
flce_status cuda_fail(cudaError_t e, const char* what);
void clear_error();

// The current device is sm_103a; its number of SMs.
flce_status check_device(int* sms);
// The caller's workspace holds `need` bytes and is 256-byte aligned.
flce_status check_workspace(void* ws, size_t have, size_t need);

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// cuTensorMapEncodeTiled, or null where the driver has none.
EncodeTiledFn tensor_map_encoder();

inline bool aligned_to(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace host
}  // namespace flce
