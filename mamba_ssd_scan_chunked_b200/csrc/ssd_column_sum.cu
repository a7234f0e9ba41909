// Sums of the columns of matrices of partial results: the second step of the
// gradients that are summed over tokens or channels.  Order and grouping depend
// on the sizes alone, so results repeat bit for bit.
//
// A block owns 32 neighbouring columns of one matrix; warp w sums rows w, w + 8,
// ... in order, then warp 0 adds the 8 sums in order.  Bound by the read of the
// matrices; a call's sums share one launch, most of which are too short alone.
#include "ssd_common.cuh"
#include "ssd_internal.h"

namespace ssd {

struct ColumnSums {
    ColumnSum job[kMaxColumnSums];
    unsigned first[kMaxColumnSums];      // a job's first block
    int n;
};

__global__ void __launch_bounds__(256)
column_sum_kernel(const ColumnSums all) {
    __shared__ float sums[8][32];
    int j = 0;
#pragma unroll
    for (int k = 1; k < kMaxColumnSums; ++k)
        if (k < all.n && blockIdx.x >= all.first[k]) j = k;
    const ColumnSum& s = all.job[j];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)(blockIdx.x - all.first[j]) * 32 + lane;
    float v = 0.f;
    if (c < s.cols) {
#pragma unroll 4
        for (int64_t r = warp; r < s.rows; r += 8) v += s.part[r * s.stride + c];
    }
    sums[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < s.cols) {
#pragma unroll
        for (int w = 1; w < 8; ++w) v += sums[w][lane];
        void* out = c < s.cols1 ? s.out : s.out2;
        const int64_t at = c < s.cols1 ? c : c - s.cols1;
        if (!out) return;
        if (s.out_bf16) ((bf16*)out)[at] = from_f32<bf16>(v);
        else ((float*)out)[at] = v;
    }
}

cudaError_t launch_column_sums(const ColumnSum* sums, int n, cudaStream_t s) {
    ColumnSums all{};
    unsigned blocks = 0;
    for (int i = 0; i < n; ++i) {
        if (sums[i].cols == 0) continue;
        all.job[all.n] = sums[i];
        all.first[all.n++] = blocks;
        blocks += (unsigned)((sums[i].cols + 31) / 32);
    }
    if (blocks == 0) return cudaSuccess;
    column_sum_kernel<<<blocks, 256, 0, s>>>(all);
    return cudaGetLastError();
}

}  // namespace ssd
