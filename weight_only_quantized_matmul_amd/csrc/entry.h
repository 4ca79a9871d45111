// What the C entry points of the operators share: the caller's device kept, status codes, alignment.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "wqmm.h"

namespace {

struct DeviceScope { // makes `dev` current, restoring the caller's device after
    int prev = -1;
    bool switched = false;
    explicit DeviceScope(int dev) {
        if (hipGetDevice(&prev) == hipSuccess && prev != dev) switched = hipSetDevice(dev) == hipSuccess;
    }
    ~DeviceScope() {
        if (switched) (void)hipSetDevice(prev);
    }
};

inline int status(hipError_t e) {
    return e == hipSuccess ? WQ_OK : e == hipErrorOutOfMemory ? WQ_E_OOM : e == hipErrorNotSupported ? WQ_E_UNSUPPORTED : WQ_E_HIP;
}

inline bool float_type(int t) { return t >= WQ_DT_F32 && t <= WQ_DT_F16; }

inline int size_of(int t) { return t == WQ_DT_F32 ? 4 : t == WQ_DT_I8 ? 1 : 2; }

inline bool aligned(const void *p, long a) { return ((uintptr_t)p & (uintptr_t)(a - 1)) == 0; }

} // namespace
