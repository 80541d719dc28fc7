// What the entry points' host sides share: checks of sizes and pointers, the status of a launch, and
// the choice of a block tile.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "gemm_f16.h"

namespace gemm_f16 {

// One buffer of a call, for the checks on pointers.
struct Buffer {
    const void *p;
    int64_t bytes;
    int align;
    bool out;
};

// Null, alignment and overlap: outputs (and the workspace) against every
// other buffer.
template <int N>
inline int check_buffers(const Buffer (&bufs)[N]) {
    for (const Buffer &b : bufs)
        if (b.bytes > 0 && !b.p) return GEMM_F16_ENULL;
    for (const Buffer &b : bufs)
        if (b.bytes > 0 && ((uintptr_t)b.p % (uintptr_t)b.align) != 0) return GEMM_F16_EALIGN;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            if (i == j || !bufs[i].out || bufs[i].bytes <= 0 || bufs[j].bytes <= 0) continue;
            const uintptr_t a0 = (uintptr_t)bufs[i].p, a1 = a0 + (uintptr_t)bufs[i].bytes;
            const uintptr_t b0 = (uintptr_t)bufs[j].p, b1 = b0 + (uintptr_t)bufs[j].bytes;
            if (a0 < b1 && b0 < a1) return GEMM_F16_EOVERLAP;
        }
    return GEMM_F16_OK;
}

inline bool below(int64_t limit, int64_t a, int64_t b, int64_t c = 1) {
    // a, b, c >= 0 and below 2^31: a * b cannot wrap
    if (a == 0 || b == 0 || c == 0) return true;
    return a * b < limit && a * b <= (limit - 1) / c;
}

// The dense products' block tile on a device of `cus` compute units (gemm_f16.hip).
int auto_tile(int64_t m, int64_t n, int64_t k, int cus);

inline int status(hipError_t e) { return e == hipSuccess ? GEMM_F16_OK : e == hipErrorInvalidValue ? GEMM_F16_EINVAL : GEMM_F16_EHIP; }

}  // namespace gemm_f16
