// sscan_rowsum.cuh -- column sums of a small fp32 matrix of partial sums, in a fixed
// order: how backward kernels turn one partial row per tile into a parameter's gradient
// without atomics, so that two runs give the same bits.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "sscan_check.cuh"

namespace sscan {

constexpr int kSumGroups = 32;

// put(c, sum over r of src[r * cols + c]): 32 columns by kSumGroups row groups per block;
// group g adds rows g, g + kSumGroups, ... in order, then the groups are added in order.  256 rows of
// 4608 columns: 5.0-5.5 us.
template <typename Put>
__global__ void __launch_bounds__(32 * kSumGroups) rowsum_kernel(const float* __restrict__ src, int64_t rows,
                                                                int64_t cols, Put put) {
    __shared__ float part[kSumGroups][33];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int64_t r = grp; r < rows; r += kSumGroups) s += in_range(r * cols + c, rows * cols) ? __ldg(src + r * cols + c) : 0.f;
    }
    part[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && c < cols) {
        s = 0.f;
#pragma unroll
        for (int g = 0; g < kSumGroups; ++g) s += part[g][lane];
        put(c, s);
    }
}

template <typename Put>
void launch_rowsum(const float* src, int64_t rows, int64_t cols, const Put& put, cudaStream_t st) {
    rowsum_kernel<<<(unsigned)((cols + 31) / 32), 32 * kSumGroups, 0, st>>>(src, rows, cols, put);
}

}  // namespace sscan
