// Group normalisation of rows of channels, channels last, with a SiLU
// activation or gate, and its backward pass.  Per row and group of n channels,
//
//   u = x  or  x silu(z);   c = u - m, m = mean(u) (0 for the root mean square form)
//   r = 1 / sqrt(mean(c^2) + eps);   nrm = c r;   v = nrm w + bias
//   y = v, silu(v) or v silu(z)
//   dv = dy, dy silu'(v) or dy silu(z);   dn = dv w
//   du = r (dn - [mean(dn)] - nrm mean(dn nrm));   dw = sum_rows dv nrm;   db = sum_rows dv
//
// A stream bound by HBM: a row's group is read once and kept in registers over
// its sums (the mean first and then the squares of the differences, not their
// expanded form, which cancels).  Items, the pairs (row, group) in memory order,
// go to slots: `lanes` neighbouring threads each, up to a warp, or the whole
// block.  The number of slots is a multiple of the groups, so that a slot meets
// one group only and keeps its weights, and the sums of dw and db, in registers.
#include "ssd_internal.h"
#include "ssd_vec.cuh"

namespace ssd {

constexpr int kNone = 0, kSilu = 1, kAfter = 2, kBefore = 3;   // ssd_norm_activation_t

struct NormShape {
    int gs;          // channels of a group
    int lanes;       // threads of a slot
    int threads;     // of a block
    int per_block;   // slots of a block
    int64_t blocks, items;
};

// sum over the slot's threads; every thread gets it
template <bool BLOCK>
__device__ __forceinline__ float slot_sum(float v, int lanes, float* red) {
    const int span = BLOCK ? 32 : lanes;
    for (int o = span >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (BLOCK) {
        const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
        __syncthreads();                       // red may still be read by the sum before
        if ((threadIdx.x & 31) == 0) red[warp] = v;
        __syncthreads();
        v = 0.f;
        for (int w = 0; w < nw; ++w) v += red[w];
    }
    return v;
}

// Loads one item and forms nrm (in u), r and silu(z)'s factors.
template <typename XT, typename IoT, int NV, bool BLOCK>
struct Item {
    float u[NV][8];

    __device__ __forceinline__ float normalise(const GroupNormArgs& a, const NormShape& sh, int64_t item, bool live,
                                               int lane, float* red, float (&x)[NV][8], float (&z)[NV][8]) {
        const int64_t row = item / a.G, g = item % a.G;
        const XT* xp = (const XT*)a.x + item * sh.gs;
        const IoT* zp = (const IoT*)a.z + row * a.zs + g * sh.gs;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (lane + q * sh.lanes) * 8;
            const bool ok = live && i < sh.gs;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[q][j] = z[q][j] = 0.f;
            if (ok) {
                load8(xp + i, x[q]);
                if (a.act >= kAfter) load8(zp + i, z[q]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                u[q][j] = a.act == kBefore ? x[q][j] * (z[q][j] * sigmoid_f32(z[q][j])) : x[q][j];
                s += u[q][j];
            }
        }
        const float inv = 1.f / (float)sh.gs;
        if (a.center) {
            const float m = slot_sum<BLOCK>(s, sh.lanes, red) * inv;
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const bool ok = (lane + q * sh.lanes) * 8 < sh.gs;
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] = ok ? u[q][j] - m : 0.f;
            }
        }
        float ss = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(u[q][j], u[q][j], ss);
        const float r = 1.f / sqrtf(slot_sum<BLOCK>(ss, sh.lanes, red) * inv + a.eps);
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) u[q][j] *= r;
        return r;
    }
};

template <typename XT, typename IoT, typename YT, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128)
group_norm_fwd_kernel(const GroupNormArgs a, const NormShape sh) {
    __shared__ float red[32];
    const int slot = BLOCK ? 0 : (int)threadIdx.x / sh.lanes, lane = BLOCK ? (int)threadIdx.x : (int)threadIdx.x % sh.lanes;
    const int64_t first = (int64_t)blockIdx.x * sh.per_block + slot, step = sh.blocks * sh.per_block;
    const int64_t base = (first % a.G) * sh.gs;
    float w[NV][8], bias[NV][8];
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int i = (lane + q * sh.lanes) * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) { w[q][j] = 1.f; bias[q][j] = 0.f; }
        if (i < sh.gs) {
            if (a.w) load8(a.w + base + i, w[q]);
            if (a.bias) load8(a.bias + base + i, bias[q]);
        }
    }
    // every thread of a warp takes part in its sums, with or without an item
    for (int64_t it0 = (int64_t)blockIdx.x * sh.per_block; it0 < sh.items; it0 += step) {
        const int64_t item = it0 + slot;
        const bool live = item < sh.items;
        Item<XT, IoT, NV, BLOCK> t;
        float x[NV][8], z[NV][8];
        t.normalise(a, sh, item, live, lane, red, x, z);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (lane + q * sh.lanes) * 8;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float v = fmaf(t.u[q][j], w[q][j], bias[q][j]);
                y[j] = a.act == kSilu ? v * sigmoid_f32(v) : a.act == kAfter ? v * (z[q][j] * sigmoid_f32(z[q][j])) : v;
            }
            if (live && i < sh.gs) store8((YT*)a.y + item * sh.gs + i, y);
        }
    }
}

template <typename XT, typename IoT, typename GT, int NV, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 1024 : 128)
group_norm_bwd_kernel(const GroupNormArgs a, const NormShape sh) {
    __shared__ float red[32];
    const int slot = BLOCK ? 0 : (int)threadIdx.x / sh.lanes, lane = BLOCK ? (int)threadIdx.x : (int)threadIdx.x % sh.lanes;
    const int64_t first = (int64_t)blockIdx.x * sh.per_block + slot, step = sh.blocks * sh.per_block;
    const int64_t base = (first % a.G) * sh.gs;
    const float inv = 1.f / (float)sh.gs;
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[q][j] = db[q][j] = 0.f;
    for (int64_t it0 = (int64_t)blockIdx.x * sh.per_block; it0 < sh.items; it0 += step) {
        const int64_t item = it0 + slot;
        const bool live = item < sh.items;
        Item<XT, IoT, NV, BLOCK> t;
        float x[NV][8], z[NV][8], dn[NV][8];
        const float r = t.normalise(a, sh, item, live, lane, red, x, z);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (lane + q * sh.lanes) * 8;
            const bool ok = live && i < sh.gs;
            float w[8], bias[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) { dn[q][j] = 0.f; w[j] = 1.f; bias[j] = 0.f; }
            if (ok) {
                load8((const IoT*)a.dy + item * sh.gs + i, dn[q]);
                if (a.w) load8(a.w + base + i, w);
                if (a.bias) load8(a.bias + base + i, bias);
            }
            float dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float dv = dn[q][j];
                const float v = fmaf(t.u[q][j], w[j], bias[j]);
                if (a.act == kSilu) {
                    dv *= silu_grad(v, sigmoid_f32(v));
                } else if (a.act == kAfter) {
                    dz[j] = dv * v * silu_grad(z[q][j], sigmoid_f32(z[q][j]));
                    dv *= z[q][j] * sigmoid_f32(z[q][j]);
                }
                dw[q][j] = fmaf(dv, t.u[q][j], dw[q][j]);
                db[q][j] += dv;
                dn[q][j] = dv * w[j];
                s0 += dn[q][j];
                s1 = fmaf(dn[q][j], t.u[q][j], s1);
            }
            if (a.act == kAfter && ok) store8((GT*)a.dz + item * sh.gs + i, dz);
        }
        s1 = slot_sum<BLOCK>(s1, sh.lanes, red) * inv;
        s0 = a.center ? slot_sum<BLOCK>(s0, sh.lanes, red) * inv : 0.f;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (lane + q * sh.lanes) * 8;
            float dx[8], dz[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float du = r * (dn[q][j] - s0 - t.u[q][j] * s1);
                dx[j] = du;
                if (a.act == kBefore) {
                    dx[j] = du * (z[q][j] * sigmoid_f32(z[q][j]));
                    dz[j] = du * x[q][j] * silu_grad(z[q][j], sigmoid_f32(z[q][j]));
                }
            }
            if (live && i < sh.gs) {
                store8((GT*)a.dx + item * sh.gs + i, dx);
                if (a.act == kBefore) store8((GT*)a.dz + item * sh.gs + i, dz);
            }
        }
    }
    // slot q's sums: row q / G of [slots / G][C]
    float* part = a.ws + first * sh.gs;
    const int64_t all = step * sh.gs;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int i = (lane + q * sh.lanes) * 8;
        if (i >= sh.gs) continue;
        if (a.dw) store8(part + i, dw[q]);
        if (a.db) store8(part + all + i, db[q]);
    }
}

__global__ void group_norm_zero_kernel(float* dw, float* db, int64_t n) {
    const int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x;
    if (i < n) {
        if (dw) dw[i] = 0.f;
        if (db) db[i] = 0.f;
    }
}

// Slots: one vector of 8 channels a lane up to 32 lanes, then 4 a lane in a
// warp, then a block with 2 a lane.
static NormShape norm_shape(int64_t rows, int64_t C, int64_t G, int* nv, bool* block) {
    NormShape sh{};
    sh.gs = (int)(C / G);
    const int vecs = sh.gs / 8;
    if (vecs <= 128) {
        *nv = vecs <= 32 ? 1 : 4;
        *block = false;
        sh.lanes = 1;
        while (sh.lanes < 32 && sh.lanes < vecs) sh.lanes *= 2;
        sh.threads = 128;
        sh.per_block = 128 / sh.lanes;
    } else {
        *nv = 2;
        *block = true;
        sh.lanes = (vecs / 2 + 31) / 32 * 32;
        while (sh.lanes * 2 < vecs) sh.lanes += 32;
        sh.threads = sh.lanes;
        sh.per_block = 1;
    }
    sh.items = rows * G;
    // blocks: a multiple of `unit`, so that all slots together are a multiple of G
    int64_t x = G, y = sh.per_block;
    while (y) { const int64_t m = x % y; x = y; y = m; }
    const int64_t unit = G / x, want = (sh.items + sh.per_block - 1) / sh.per_block;
    const int64_t most = (int64_t)148 * (2048 / sh.threads);
    const int64_t n = want < most ? want : most;
    sh.blocks = (n + unit - 1) / unit * unit;
    if (sh.blocks < unit) sh.blocks = unit;
    return sh;
}

size_t group_norm_bwd_workspace(int64_t rows, int64_t C, int64_t G) {
    int nv; bool block;
    const NormShape sh = norm_shape(rows, C, G, &nv, &block);
    return rows ? (size_t)sh.blocks * sh.per_block * sh.gs * 2 * sizeof(float) : 0;
}

template <template <typename, typename, typename> class F>
static void dispatch_types(const GroupNormArgs& a, const NormShape& sh, int nv, bool block, cudaStream_t s) {
    if (a.x_bf16) {
        if (a.io_bf16) { if (a.y_bf16) F<bf16, bf16, bf16>::go(a, sh, nv, block, s); else F<bf16, bf16, float>::go(a, sh, nv, block, s); }
        else { if (a.y_bf16) F<bf16, float, bf16>::go(a, sh, nv, block, s); else F<bf16, float, float>::go(a, sh, nv, block, s); }
    } else {
        if (a.io_bf16) { if (a.y_bf16) F<float, bf16, bf16>::go(a, sh, nv, block, s); else F<float, bf16, float>::go(a, sh, nv, block, s); }
        else { if (a.y_bf16) F<float, float, bf16>::go(a, sh, nv, block, s); else F<float, float, float>::go(a, sh, nv, block, s); }
    }
}

template <typename X, typename I, typename Y> struct Fwd {
    static void go(const GroupNormArgs& a, const NormShape& sh, int nv, bool block, cudaStream_t s) {
        const unsigned grid = (unsigned)sh.blocks;
        if (block) group_norm_fwd_kernel<X, I, Y, 2, true><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (nv == 1) group_norm_fwd_kernel<X, I, Y, 1, false><<<grid, sh.threads, 0, s>>>(a, sh);
        else group_norm_fwd_kernel<X, I, Y, 4, false><<<grid, sh.threads, 0, s>>>(a, sh);
    }
};
template <typename X, typename I, typename Y> struct Bwd {
    static void go(const GroupNormArgs& a, const NormShape& sh, int nv, bool block, cudaStream_t s) {
        const unsigned grid = (unsigned)sh.blocks;
        if (block) group_norm_bwd_kernel<X, I, Y, 2, true><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (nv == 1) group_norm_bwd_kernel<X, I, Y, 1, false><<<grid, sh.threads, 0, s>>>(a, sh);
        else group_norm_bwd_kernel<X, I, Y, 4, false><<<grid, sh.threads, 0, s>>>(a, sh);
    }
};

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t s) {
    int nv; bool block;
    const NormShape sh = norm_shape(a.rows, a.C, a.G, &nv, &block);
    dispatch_types<Fwd>(a, sh, nv, block, s);
    return cudaGetLastError();
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, cudaStream_t s) {
    if (a.rows == 0) {
        if (!a.dw && !a.db) return cudaSuccess;
        group_norm_zero_kernel<<<(unsigned)((a.C + 255) / 256), 256, 0, s>>>(a.dw, a.db, a.C);
        return cudaGetLastError();
    }
    int nv; bool block;
    const NormShape sh = norm_shape(a.rows, a.C, a.G, &nv, &block);
    dispatch_types<Bwd>(a, sh, nv, block, s);
    cudaError_t e = cudaGetLastError();
    const int64_t rows = sh.blocks * sh.per_block / a.G;
    if (e == cudaSuccess && a.dw) e = launch_column_sum(a.ws, rows, a.C, a.C, a.dw, false, s);
    if (e == cudaSuccess && a.db) e = launch_column_sum(a.ws + rows * a.C, rows, a.C, a.C, a.db, false, s);
    return e;
}

}  // namespace ssd
