// Grouping of rows by an id: a stable counting sort of ids in [0, groups),
// any other id sorting behind them.
//
// One workgroup sorts a chunk of consecutive rows, each of its waves a
// contiguous part of it.  A wave takes 64 rows at a time: the lanes that
// share a key find each other with one ballot per key bit, so a row's place
// is the count of its key before the wave's 64 rows plus the set bits below
// its lane.  Nothing depends on the order in which atomics land.
//
// Up to kGroupOneBlock rows one workgroup does it all.  Beyond that a first
// launch counts each chunk's keys, and in the second every workgroup sums
// the counts of the chunks before its own.  Bound by launches and the chain
// of dependent reads, not by bytes: 128 rows of 8 groups 2.9 us, 131072 rows of
// 64 groups 2.6 and 6.3 us.
#include <algorithm>

#include "segments.h"

namespace gemm_f16 {

// Waves whose counters of every key, and two more arrays, fit 64 KB of LDS.
static int group_waves(int groups) {
    const int keys = groups + 1;
    return 18 * keys * 4 <= 65536 ? 16 : 10 * keys * 4 <= 65536 ? 8 : 4;
}

static int group_chunk(int64_t rows) {
    if (rows <= kGroupOneBlock) return (int)std::max<int64_t>(1024, (rows + 1023) / 1024 * 1024);
    // at most 256 chunks: each workgroup reads the counts of all before it
    const int64_t chunk = std::max<int64_t>(1024, (rows + 255) / 256);
    return (int)((chunk + 1023) / 1024 * 1024);
}

int64_t group_blocks(int64_t rows) {
    const int64_t chunk = group_chunk(rows);
    return std::max<int64_t>(1, (rows + chunk - 1) / chunk);
}

struct GroupParams {
    const void *ids;
    int32_t *order, *inverse, *offsets, *counts;
    int32_t rows, groups, chunk, blocks, bits;
};

template <class Id>
__device__ __forceinline__ int group_key(const void *ids, int r, int groups) {
    const Id v = static_cast<const Id *>(ids)[r];
    return v >= 0 && v < (Id)groups ? (int)v : groups;
}

template <class Id>
__global__ __launch_bounds__(1024) void group_count_kernel(const GroupParams p) {
    extern __shared__ int count[];
    const int keys = p.groups + 1, tid = threadIdx.x, threads = blockDim.x;
    for (int k = tid; k < keys; k += threads) count[k] = 0;
    __syncthreads();
    const int first = (int)blockIdx.x * p.chunk, last = min(p.rows, first + p.chunk);
    for (int r = first + tid; r < last; r += threads) atomicAdd(&count[group_key<Id>(p.ids, r, p.groups)], 1);
    __syncthreads();
    for (int k = tid; k < keys; k += threads) p.counts[(int64_t)blockIdx.x * keys + k] = count[k];
}

template <class Id>
__global__ __launch_bounds__(1024) void group_place_kernel(const GroupParams p) {
    extern __shared__ int lds[];
    const int keys = p.groups + 1, tid = threadIdx.x, threads = blockDim.x;
    const int waves = threads / kWave, wave = tid / kWave, lane = tid % kWave;
    int *const start = lds;          // [keys] rows of each key, then its first place
    int *const before = lds + keys;  // [keys] rows of each key in the chunks before
    int *const mine = before + keys; // [waves][keys] counts, then next places
    for (int x = tid; x < (waves + 2) * keys; x += threads) lds[x] = 0;
    __syncthreads();
    const int first = (int)blockIdx.x * p.chunk, last = min(p.rows, first + p.chunk);
    // a wave's part: a whole number of 64-row steps
    const int part = ((p.chunk + waves * kWave - 1) / (waves * kWave)) * kWave;
    const int w0 = min(last, first + wave * part), w1 = min(last, w0 + part);
    for (int r = w0 + lane; r < w1; r += kWave) atomicAdd(&mine[wave * keys + group_key<Id>(p.ids, r, p.groups)], 1);
    if (p.blocks > 1) {
        // totals of each key, and the rows of it before this chunk: the
        // threads share the chunks, so that few loads follow each other
        // (one thread per key took 9.8 us over 128 chunks)
        const int shares = max(1, threads / keys);
        for (int x = tid; x < shares * keys; x += threads) {
            const int k = x % keys;
            int total = 0, below = 0;
#pragma unroll 8
            for (int b = x / keys; b < p.blocks; b += shares) {
                const int v = p.counts[(int64_t)b * keys + k];
                total += v;
                below += b < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&start[k], total);
            atomicAdd(&before[k], below);
        }
    }
    __syncthreads();
    for (int k = tid; k < keys; k += threads) {
        // each wave's first place, relative to the key's first
        int at = before[k];
        for (int w = 0; w < waves; ++w) {
            const int v = mine[w * keys + k];
            mine[w * keys + k] = at;
            at += v;
        }
        if (p.blocks == 1) start[k] = at;
    }
    __syncthreads();
    // exclusive scan of the totals over the keys
    if (wave == 0) {
        int carry = 0;
        for (int base = 0; base < keys; base += kWave) {
            const int k = base + lane, v = k < keys ? start[k] : 0;
            const int s = wave_scan(v, lane);
            if (k < keys) start[k] = carry + s - v;
            carry += __builtin_amdgcn_readlane(s, kWave - 1);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)  // keys 0 .. groups: the last is where the rows of no group start
        for (int k = tid; k < keys; k += threads) p.offsets[k] = start[k];
    volatile int *const next = mine + wave * keys;  // this wave's alone
    for (int r0 = w0; r0 < w1; r0 += kWave) {
        const int r = r0 + lane;
        const bool live = r < w1;
        const int key = live ? group_key<Id>(p.ids, r, p.groups) : 0;
        uint64_t same = __ballot(live);
        for (int b = 0; b < p.bits; ++b) {
            const uint64_t set = __ballot((key >> b) & 1);
            same &= ((key >> b) & 1) ? set : ~set;
        }
        if (live) {
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int at = next[key];
            const int place = start[key] + at + rank;
            // the last lane of each key moves its place on, after every lane
            // has read it (one wave: its LDS operations stay in order)
            __builtin_amdgcn_wave_barrier();
            if ((same >> lane) == 1) next[key] = at + rank + 1;
            p.order[place] = r;
            p.inverse[r] = place;
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <class Id>
static hipError_t launch_group(GroupParams p, hipStream_t s) {
    const int keys = p.groups + 1, waves = group_waves(p.groups);
    void *args[] = {&p};
    if (p.blocks > 1) {
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(group_count_kernel<Id>), dim3(p.blocks),
                                             dim3(waves * kWave), args, (size_t)keys * 4, s);
        if (e != hipSuccess) return e;
    }
    return hipLaunchKernel(reinterpret_cast<const void *>(group_place_kernel<Id>), dim3(p.blocks), dim3(waves * kWave),
                           args, (size_t)(waves + 2) * keys * 4, s);
}

hipError_t launch_group_rows(int64_t rows, int groups, const void *ids, int id_bytes, int32_t *order, int32_t *inverse,
                             int32_t *offsets, int32_t *counts, hipStream_t s) {
    GroupParams p;
    p.ids = ids;
    p.order = order;
    p.inverse = inverse;
    p.offsets = offsets;
    p.counts = counts;
    p.rows = (int32_t)rows;
    p.groups = groups;
    p.chunk = group_chunk(rows);
    p.blocks = (int32_t)group_blocks(rows);
    p.bits = 1;
    while ((groups >> p.bits) != 0) ++p.bits;  // keys 0 .. groups
    return id_bytes == 8 ? launch_group<int64_t>(p, s) : launch_group<int32_t>(p, s);
}

}  // namespace gemm_f16
