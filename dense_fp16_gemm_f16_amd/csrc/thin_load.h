// Loads of the few-row kernels: weights from memory to registers in the MFMA's layout.
#pragma once

#include "kernels.h"

namespace gemm_f16 {

typedef int int4u __attribute__((ext_vector_type(4), aligned(2)));

// Up to N steps of a row (K >= 8), 32 elements each, `count` of them from
// step top - 1 downwards; 8 elements at kl of each.  The first one, where
// `partial`, reaches past K: its chunks past K become zeros, and the chunk
// across K is loaded from the row's last 8 elements and shifted, so every
// load stays inside the row.
template <int N>
__device__ __forceinline__ void thin_load(half8 (&v)[N], const _Float16 *row, int top, int count, bool partial,
                                          int kl, int k_elems) {
    const int k0 = 32 * (top - 1) + kl;
#pragma unroll
    for (int s = 0; s < N; ++s) {
        if (s >= count) continue;
        const int k = s == 0 && partial ? min(k0, k_elems - 8) : k0 - 32 * s;
        v[s] = __builtin_bit_cast(half8, (int4v)*reinterpret_cast<const int4u *>(row + k));
    }
    if (partial) {
        const int past = 8 - (k_elems - k0);  // elements to shift out
        unsigned __int128 w = __builtin_bit_cast(unsigned __int128, v[0]);
        if (past > 0) w = past < 8 ? w >> (16 * past) : 0;
        v[0] = __builtin_bit_cast(half8, w);
    }
}

}  // namespace gemm_f16
