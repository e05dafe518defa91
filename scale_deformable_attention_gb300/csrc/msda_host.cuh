// msda_host.cuh -- host helpers that the translation units beside msda_api.cu
// share: error messages, pointer checks, the kernel trace, per-device facts.
// Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "msda_internal.h"

namespace msda {

// Trace slot of a launch about to be made on `st` (-1: not traced), and its end.
int trace_begin(cudaStream_t st);
void trace_end(int slot, cudaStream_t st, int kernel, int64_t work);

struct TraceSpan {
    cudaStream_t st;
    int slot;
    explicit TraceSpan(cudaStream_t s) : st(s), slot(trace_begin(s)) {}
    void end(int kernel, int64_t work) {
        if (slot >= 0) trace_end(slot, st, kernel, work);
    }
};

// Device address of the error word on the current device (its bits are those
// of msda_device_errors()).
msda_status error_word(unsigned** err);

// SMs that the dense operators' grids and splits are planned for, those of a
// GB300 whatever the device has: a workspace's size and the order of a sum
// then depend on the call alone.
constexpr int kPlanSms = 152;

// Sets a kernel's limit of dynamic shared memory, once a device context
// (`seen`: one a kernel; a device reset gives a new context and sets it again).
struct SmemSeen {
    std::atomic<unsigned long long> ctx[64] = {};
};
cudaError_t allow_smem(const void* kernel, size_t bytes, SmemSeen& seen);

// cuTensorMapEncodeTiled, or null where the driver does not give it.
void* tensor_map_encoder();

inline msda_status failf(msda_status s, const char* fmt, ...) {
    char buf[480];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return set_error(s, buf);
}

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }
inline bool mul_fits(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }

inline msda_status need_ptr(const void* p, bool needed, size_t align, const char* name) {
    if (!needed) return MSDA_OK;
    if (!p) return failf(MSDA_ERR_INVALID_ARG, "%s is NULL", name);
    if (!aligned_to(p, align)) return failf(MSDA_ERR_MISALIGNED, "%s is not aligned to %zu bytes", name, align);
    return MSDA_OK;
}

}  // namespace msda
