// What the kernels on a cache's pages share: the block table and sums over a block.
#pragma once

#include <stdint.h>

#include "kda.h"

namespace kda {
namespace cache {

constexpr int kThreads = 1024;  // of a block of the calls that choose pages

// An entry of a block table whose page the row has given back; the entries behind it keep their places.
constexpr int kPageGone = KDA_PAGE_GONE;
__device__ __forceinline__ bool in_use(int entry) { return entry >= 0 || entry == kPageGone; }

struct Table {
    int32_t *entries;
    int64_t ld;
    int32_t rows, cols;
    __device__ __forceinline__ int32_t *row(int r) const { return entries + (size_t)r * ld; }
};

// Exclusive prefix of x over a block of WARPS warps; total gets the sum. Converged block.
template <int WARPS = kThreads / 32>
__device__ __forceinline__ int block_exclusive(int x, int *warp_sums, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // warp_sums is free
    if (lane == 31) warp_sums[warp] = incl;
    __syncthreads();
    const int mine = lane < WARPS ? warp_sums[lane] : 0;
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    total = __shfl_sync(0xffffffffu, sum, 31);
    const int before = __shfl_sync(0xffffffffu, sum - mine, warp);
    return before + incl - x;
}

}  // namespace cache
}  // namespace kda
