// Host-side queries of the current device, for every entry point: the gfx950
// gate and the compute-unit count, cached per device.
#pragma once

#include <atomic>
#include <cstdlib>

#include <hip/hip_runtime.h>

#include "gemm_f16.h"

namespace gemm_f16 {

// Per-device caches below: host threads may call the library at the same
// time, so the entries are atomics; a first call on a device in two threads
// at once computes the same value twice and stores it twice.

// Compute units of the current device (0 if unknown), cached per device.
inline int device_cus() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 0;
    int n = cached[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n <= 0) return 0;
        cached[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// "gfx950", optionally followed by ":" and target features.
inline bool is_gfx950(const char *arch) {
    return arch[0] == 'g' && arch[1] == 'f' && arch[2] == 'x' && arch[3] == '9' && arch[4] == '5' &&
           arch[5] == '0' && (arch[6] == '\0' || arch[6] == ':');
}

// Test hook: when the environment variable GEMM_F16_TEST_ARCH is set as the
// library loads, its value stands in for every device's architecture name
// in the gate below (no device is queried), so the refusal path can be
// exercised on any host.
inline const char *const kTestArch = std::getenv("GEMM_F16_TEST_ARCH");

// gfx950 check, cached per device.
inline int check_device() {
    if (kTestArch) return is_gfx950(kTestArch) ? GEMM_F16_OK : GEMM_F16_EDEVICE;
    static std::atomic<int> cached[64];  // 0 = unknown, 1 = gfx950, -1 = other
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return GEMM_F16_EHIP;
    if (dev < 0 || dev >= 64) return GEMM_F16_EDEVICE;
    int state = cached[dev].load(std::memory_order_relaxed);
    if (state == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_F16_EHIP;
        state = is_gfx950(prop.gcnArchName) ? 1 : -1;
        cached[dev].store(state, std::memory_order_relaxed);
    }
    return state == 1 ? GEMM_F16_OK : GEMM_F16_EDEVICE;
}

}  // namespace gemm_f16
