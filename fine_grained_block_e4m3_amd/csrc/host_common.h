// host_common.h -- host-side helpers shared by the translation units of
// libfp8gemm.so: argument checks, the device's compute units, launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

#include "../../include/fp8gemm.h"

namespace fp8h {

constexpr int64_t kMaxDim = (int64_t)1 << 31;     // rows/cols fit int32 tile math
constexpr int kMaxDevices = 64;
// Per-lane operand offsets inside a tile are 32-bit: 256 rows * K < 2^31.
constexpr int64_t kMaxGemmK = (int64_t)1 << 22;

// Per-device compute-unit count, filled once per device.
inline std::atomic<int> g_cu_count[kMaxDevices];
inline std::once_flag g_cu_once[kMaxDevices];

inline fp8_status current_device_cus(int* cus) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) {
        (void)hipGetLastError();
        return FP8_ERR_NO_DEVICE;
    }
    std::call_once(g_cu_once[dev], [dev]() {
        int n = 0;
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess)
            n = 0;
        g_cu_count[dev].store(n);
    });
    const int n = g_cu_count[dev].load();
    if (n <= 0) {
        (void)hipGetLastError();
        return FP8_ERR_NO_DEVICE;
    }
    *cus = n;
    return FP8_OK;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline fp8_status launch_status() {
    return hipGetLastError() == hipSuccess ? FP8_OK : FP8_ERR_LAUNCH;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool dims_ok(int64_t a) { return a >= 0 && a < kMaxDim; }

}  // namespace fp8h
