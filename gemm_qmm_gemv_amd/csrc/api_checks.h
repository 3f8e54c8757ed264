// api_checks.h -- what the entry points of layer_api.hip and moe_api.hip share:
// the form of a check, the device's compute units, a launch's status.  Internal
// to the library; not installed.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/qmm.h"

namespace qmm {

// Sets the calling thread's qmm_last_error text and returns st (qmm_api.hip).
qmm_status report(qmm_status st, const char* fmt, ...);

#define CHECK(cond, status, ...)                        \
    do {                                                \
        if (!(cond)) return report(status, __VA_ARGS__); \
    } while (0)

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Compute units of the current device, asked for once per device.
inline std::atomic<int> g_cus[64];

inline qmm_status current_cus(int* cus) {
    int dev = 0;
    if (hipGetDevice(&dev) == hipSuccess) {
        std::atomic<int>* known = dev >= 0 && dev < 64 ? &g_cus[dev] : nullptr;
        if (known && (*cus = known->load(std::memory_order_relaxed)) > 0) return QMM_OK;
        if (hipDeviceGetAttribute(cus, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess && *cus > 0) {
            if (known) known->store(*cus, std::memory_order_relaxed);
            return QMM_OK;
        }
    }
    (void)hipGetLastError();
    return report(QMM_ERR_DEVICE, "no HIP device available");
}

inline qmm_status launched(hipError_t e, const char* what) {
    if (e != hipSuccess) return report(QMM_ERR_DEVICE, "%s launch failed: %s", what, hipGetErrorString(e));
    return report(QMM_OK, "");
}

}  // namespace qmm
