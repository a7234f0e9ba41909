// Sums of the columns of a matrix of partial results: the second step of the
// gradients that are summed over tokens or channels.  Order and grouping depend
// on the sizes alone, so results repeat bit for bit.
//
// A block owns 32 neighbouring columns; warp w sums rows w, w + 8, ... in order,
// then warp 0 adds the 8 sums in order.  Bound by the read of the matrix.
#include "ssd_common.cuh"
#include "ssd_internal.h"

namespace ssd {

template <typename T>
__global__ void __launch_bounds__(256)
column_sum_kernel(const float* __restrict__ part, int64_t rows, int64_t stride, int64_t cols, T* __restrict__ out,
                  int64_t cols1, T* __restrict__ out2) {
    __shared__ float sums[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols) {
#pragma unroll 4
        for (int64_t r = warp; r < rows; r += 8) s += part[r * stride + c];
    }
    sums[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int w = 1; w < 8; ++w) s += sums[w][lane];
        if (c < cols1) out[c] = from_f32<T>(s);
        else if (out2) out2[c - cols1] = from_f32<T>(s);
    }
}

cudaError_t launch_column_sum(const float* part, int64_t rows, int64_t stride, int64_t cols, void* out, bool out_bf16,
                              cudaStream_t s) {
    if (cols == 0) return cudaSuccess;
    const unsigned grid = (unsigned)((cols + 31) / 32);
    if (out_bf16) column_sum_kernel<bf16><<<grid, 256, 0, s>>>(part, rows, stride, cols, (bf16*)out, cols, nullptr);
    else column_sum_kernel<float><<<grid, 256, 0, s>>>(part, rows, stride, cols, (float*)out, cols, nullptr);
    return cudaGetLastError();
}

cudaError_t launch_column_sum2(const float* part, int64_t rows, int64_t cols, float* out, int64_t cols1, float* out2,
                               cudaStream_t s) {
    if (cols == 0) return cudaSuccess;
    column_sum_kernel<float><<<(unsigned)((cols + 31) / 32), 256, 0, s>>>(part, rows, cols, cols, out, cols1, out2);
    return cudaGetLastError();
}

}  // namespace ssd
