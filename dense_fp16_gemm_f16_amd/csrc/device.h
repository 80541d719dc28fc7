// Host-side queries of the current device for the segmented products' entry
// points: the gfx950 gate and the compute-unit count, cached per device.  (The
// dense products' gate is in gemm_f16.hip; both follow the same rules.)
#pragma once

#include <atomic>
#include <cstdlib>
#include <cstring>

#include <hip/hip_runtime.h>

#include "gemm_f16.h"

namespace gemm_f16 {

// "gfx950", optionally followed by ":" and target features.
inline bool arch_is_gfx950(const char *arch) {
    return std::strncmp(arch, "gfx950", 6) == 0 && (arch[6] == '\0' || arch[6] == ':');
}

// Test hook: the environment variable GEMM_F16_TEST_ARCH, read as the library
// loads, stands in for the architecture's name (no device is queried).
inline const char *const kSegTestArch = std::getenv("GEMM_F16_TEST_ARCH");

// Status of the current device, and its compute units (256 if unknown).
// Threads may race on a first call: they store the same values.
inline int current_device(int *cus) {
    static std::atomic<int> state[64], units[64];  // state: 0 unknown, 1 gfx950, -1 other
    *cus = 256;
    if (kSegTestArch) return arch_is_gfx950(kSegTestArch) ? GEMM_F16_OK : GEMM_F16_EDEVICE;
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess) return GEMM_F16_EHIP;
    if (dev < 0 || dev >= 64) return GEMM_F16_EDEVICE;
    if (state[dev].load(std::memory_order_acquire) == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return GEMM_F16_EHIP;
        units[dev].store(prop.multiProcessorCount, std::memory_order_relaxed);
        state[dev].store(arch_is_gfx950(prop.gcnArchName) ? 1 : -1, std::memory_order_release);
    }
    if (units[dev].load(std::memory_order_relaxed) > 0) *cus = units[dev].load(std::memory_order_relaxed);
    return state[dev].load(std::memory_order_acquire) == 1 ? GEMM_F16_OK : GEMM_F16_EDEVICE;
}

}  // namespace gemm_f16
