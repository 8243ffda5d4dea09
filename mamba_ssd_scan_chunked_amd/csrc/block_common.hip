// Small kernels shared by the operators around the scan.
#include "block_common.hpp"

namespace ssd {

// Sums over the rows of a partial-sum array.  A workgroup takes 64 columns; its 16
// waves take every 16th row (64 consecutive columns each, so every load is a whole
// 256-byte line) and meet in LDS.  Latency-bound: eight loads in flight per wave, then a
// fixed-order sum.  With wide rows there are some hundred rows (5 us); narrow norms and
// convolutions of few channels leave thousands, which few workgroups walk: norm gradients of
// 78125 rows of 256 channels 16 us of 73, 312500 of 64 (one workgroup, 20480 rows of parts)
// 57 of 114, 1250000 of 16 (40960) 116 of 198; a convolution of 16384 tokens of 100 channels
// (2731) 11 of 26.
__global__ __launch_bounds__(1024) void column_sums_kernel(ColumnSums c) {
    __shared__ float acc[16][64];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    for (int64_t first = (int64_t)blockIdx.x * 64; first < c.cols; first += (int64_t)gridDim.x * 64) {
        const int64_t col = first + lane;
        float sum = 0.f;
        if (col < c.cols) {
            int64_t r = w;
            for (; r + 7 * 16 < c.rows; r += 8 * 16) {
                float v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) v[k] = c.part[(r + 16 * k) * c.cols + col];
#pragma unroll
                for (int k = 0; k < 8; ++k) sum += v[k];
            }
            for (; r < c.rows; r += 16) sum += c.part[r * c.cols + col];
        }
        acc[w][lane] = sum;
        __syncthreads();
        if (w == 0 && col < c.cols) {
            float total = 0.f;
#pragma unroll
            for (int k = 0; k < 16; ++k) total += acc[k][lane];
            if (col < c.split) {
                if (c.out) c.out[col] = total;
            } else if (col < c.split2) {
                if (c.out2) c.out2[col - c.split] = total;
            } else if (c.out3) {
                c.out3[col - c.split2] = total;
            }
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(256) void fill_kernel(float* p, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.f;
}
__global__ __launch_bounds__(256) void copy_kernel(float* dst, const float* src, int64_t n) {
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) dst[i] = src[i];
}

hipError_t launch_column_sums(const ColumnSums& c, hipStream_t s) {
    if (c.cols <= 0) return hipSuccess;
    const int64_t blocks = (c.cols + 63) / 64;
    hipLaunchKernelGGL(column_sums_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(1024), 0, s, c);
    return hipGetLastError();
}
static unsigned grid_of(int64_t n) {
    const int64_t g = (n + 255) / 256;
    return (unsigned)(g < 4096 ? g : 4096);
}
hipError_t launch_fill(float* p, int64_t n, hipStream_t s) {
    if (!p || n <= 0) return hipSuccess;
    hipLaunchKernelGGL(fill_kernel, dim3(grid_of(n)), dim3(256), 0, s, p, n);
    return hipGetLastError();
}
hipError_t launch_copy(float* dst, const float* src, int64_t n, hipStream_t s) {
    if (!src) return launch_fill(dst, n, s);
    if (!dst || n <= 0) return hipSuccess;
    hipLaunchKernelGGL(copy_kernel, dim3(grid_of(n)), dim3(256), 0, s, dst, src, n);
    return hipGetLastError();
}

}  // namespace ssd
