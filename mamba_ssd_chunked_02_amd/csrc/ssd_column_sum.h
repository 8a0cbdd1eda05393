// Sum of a column over the rows of partial sums, for the gradients that
// workgroups sum each for itself.  The order is fixed by the row count.
//
// A few thousand rows at most, read once from the cache: the work is spread
// thin so that its latency is short.  A workgroup takes 16 columns (64 bytes of a
// row); 64 lanes share a column and take every 64th row, then their sums are
// added.  1024 rows of 2560 columns: 26 us with 64 columns and 16 lanes a column,
// 6 us so.
#pragma once

#include <hip/hip_runtime.h>

namespace ssd {

constexpr int kSumCols = 16, kSumStrips = 64, kSumThreads = kSumCols * kSumStrips;

// at(row): the lane's column (blockIdx.x * kSumCols + threadIdx.x % kSumCols)
// in that row, 0 if there is no such column.  The sum is returned in the first
// kSumCols lanes.
template <typename F>
__device__ inline float column_sum(int64_t n, F at) {
    __shared__ float s_s[kSumStrips][kSumCols];
    const int c = threadIdx.x % kSumCols, strip = threadIdx.x / kSumCols;
    float s = 0.f;
#pragma unroll 8
    for (int64_t t = strip; t < n; t += kSumStrips) s += at(t);
    s_s[strip][c] = s;
    __syncthreads();
    if (strip < 8) {
        s = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) s += s_s[strip * 8 + j][c];
    }
    __syncthreads();
    if (strip < 8) s_s[strip][c] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += s_s[j][c];
    return s;
}

}  // namespace ssd
