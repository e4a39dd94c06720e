// Argument checks that the C-ABI translation units of the serving-step operators share.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "pa.h"
#include "pa_internal.h"

namespace pa {

namespace {

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool fits_int(long long x) { return x < (1ll << 31); }
inline int bytes_of(int dtype) { return dtype == PA_F32 ? 4 : 2; }

// Whether [p, p + n) and [q, q + m) share a byte.
inline bool overlap(const void* p, long long n, const void* q, long long m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

inline int launch_failed(cudaError_t e, const char* what) {
    return fail(PA_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

}  // namespace

}  // namespace pa
