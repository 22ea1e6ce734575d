// Host-side helpers shared by the translation units behind the C ABI: the
// calling thread's error message, the status macros and the driver's
// tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <new>

#include "wan_vae.h"

namespace wan {

// Records the calling thread's error message (printf format) and returns s.
wan_status fail(wan_status s, const char* fmt, ...);

// The driver's cuTensorMapEncodeTiled, looked up once; null (and an error
// recorded) if the driver lacks it.
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

}  // namespace wan

#define CUDA_TRY(expr)                                                                                     \
  do {                                                                                                     \
    cudaError_t e_ = (expr);                                                                               \
    if (e_ != cudaSuccess)                                                                                 \
      return ::wan::fail(e_ == cudaErrorMemoryAllocation ? WAN_ERR_OOM : WAN_ERR_CUDA, "%s: %s (%s:%d)", #expr, \
                         cudaGetErrorString(e_), __FILE__, __LINE__);                                      \
  } while (0)
#define WAN_TRY(expr)                 \
  do {                                \
    wan_status s_ = (expr);           \
    if (s_ != WAN_OK) return s_;      \
  } while (0)
#define API_GUARD(...)                                                      \
  try {                                                                     \
    __VA_ARGS__                                                             \
  } catch (const std::bad_alloc&) {                                         \
    return ::wan::fail(WAN_ERR_OOM, "host allocation failed");              \
  } catch (...) {                                                           \
    return ::wan::fail(WAN_ERR_INTERNAL, "unexpected C++ exception");       \
  }
