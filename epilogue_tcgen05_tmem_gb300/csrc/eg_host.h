// eg_host.h -- host-side helpers the entry points share: the thread-local
// error detail and the driver's tensor-map encoder.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/eg.h"

namespace eg {

// Record a printf-style description for eg_last_error_detail(); returns s.
eg_status host_fail(eg_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
eg_status host_cuda_fail(cudaError_t e, const char* what);

// EG_OK when the current device is one the kernels are built for; its index and
// its multiprocessors (what does not change is asked of the driver once).
eg_status host_check_device(int* dev, int* sms = nullptr);
// Allow `fn` its dynamic shared memory on device `dev`; asked once for each
// function and device that `done` (one bit a device) has not seen.
eg_status host_allow_smem(const void* fn, int bytes, int dev, std::atomic<uint64_t>* done);

// cuTensorMapEncodeTiled through the runtime's driver entry point, or NULL.
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn host_encode_tiled();

// Bound on any in-kernel wait (EG_WAIT_CAP_MS, default 2 s).
uint64_t host_wait_limit_ns();

}  // namespace eg
