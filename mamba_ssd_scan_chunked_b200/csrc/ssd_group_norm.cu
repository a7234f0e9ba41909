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
// go to slots of `lanes` neighbouring threads, each with NV vectors of 8
// channels: part of a warp, or several warps.  A slot's next item is loaded
// while its present one is summed.  Where a slot has more than one item the
// number of slots is a multiple of the groups, so that a slot meets one group only
// and keeps the sums of dw and db in registers.  Without the mean the backward's two
// sums, of c^2 and of dn c, are formed at once (mean(dn nrm) = r mean(dn c)): one
// exchange a row.
//
// Measured, 8192 rows x 4096 channels, fp32 in, bf16 gate and out, a B200 (6568 GB/s
// copy): forward 48 us (5620 GB/s), backward in 8 groups 84 us (4820 GB/s); 8 rows
// 4 us.  Loads two rows ahead were slower (60 and 105 us against 57 and 98 us then),
// none ahead too (66 and 133 us).
#include "ssd_internal.h"
#include "ssd_vec.cuh"

namespace ssd {

constexpr int kSilu = 1, kAfter = 2, kBefore = 3;   // ssd_norm_activation_t (0: none)

// blocks an SM: 64 registers a thread forward, 128 backward (64 with 1024 threads)
constexpr int norm_blocks_per_sm(bool backward, int threads) {
    return threads >= 1024 ? 1 : (backward ? 512 : 1024) / threads;
}

struct NormShape {
    int gs;          // channels of a group
    int lanes;       // threads of a slot
    int threads;     // of a block
    int per_block;   // slots of a block
    int64_t blocks, items;
};

// rows of the backward's partial sums: of the slots, or of x where a slot has one item at most
__host__ __device__ __forceinline__ int64_t norm_parts(const NormShape& sh, int64_t rows, int64_t G) {
    const int64_t slots = sh.blocks * sh.per_block;
    return slots < sh.items ? slots / G : rows;
}

// Where a thread stands, and its way through the sums over its slot: within a
// warp, then, across the slot's warps, through shared memory, whose two halves take
// turns, so that one barrier an exchange is enough.
template <bool WARP> struct Place {
    int slot, lane;
    int64_t first, step;     // the slot's first item, from one of its items to the next
    int width;               // of the last exchange: a power of two of lanes
    float (*own)[2];         // this warp's place in red
    float (*from)[2];        // the place that this lane reads (nullptr: none)
    __device__ __forceinline__ Place(const NormShape& sh, float (*red)[32][2]) {
        slot = (int)threadIdx.x / sh.lanes;
        lane = (int)threadIdx.x % sh.lanes;
        first = (int64_t)blockIdx.x * sh.per_block + slot;
        step = sh.blocks * sh.per_block;
        width = sh.lanes;
        if constexpr (!WARP) {
            const int warp = threadIdx.x >> 5, per = sh.lanes >> 5, w0 = slot * per;
            width = per <= 2 ? 2 : per <= 4 ? 4 : per <= 8 ? 8 : per <= 16 ? 16 : 32;
            const int k = threadIdx.x & (width - 1);
            own = red[0] + warp;
            from = k < per ? red[0] + w0 + k : nullptr;
        }
    }
    // sums K values; every thread of the slot gets them
    template <int K> __device__ __forceinline__ void sum(float (&v)[K], int& turn) const {
        if constexpr (WARP) {
            for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        } else {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
            if ((threadIdx.x & 31) == 0)
#pragma unroll
                for (int k = 0; k < K; ++k) own[turn][k] = v[k];
            __syncthreads();
#pragma unroll
            for (int k = 0; k < K; ++k) v[k] = from ? from[turn][k] : 0.f;
            turn ^= 32;
            for (int o = width >> 1; o > 0; o >>= 1)
#pragma unroll
                for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
        }
    }
};

// r and nrm (in the place of u) from u; masked channels of u are 0
template <int NV, bool WARP>
__device__ __forceinline__ float normalise(const GroupNormArgs& a, const NormShape& sh, const Place<WARP>& at,
                                           float (&u)[NV][8], int& turn) {
    const float inv = 1.f / (float)sh.gs;
    if (a.center) {
        float s[1] = {0.f};
#pragma unroll
        for (int q = 0; q < NV; ++q)
#pragma unroll
            for (int j = 0; j < 8; ++j) s[0] += u[q][j];
        at.sum(s, turn);
        const float m = s[0] * inv;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if ((at.lane + q * sh.lanes) * 8 < sh.gs)
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] -= m;
    }
    float ss[1] = {0.f};
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss[0] = fmaf(u[q][j], u[q][j], ss[0]);
    at.sum(ss, turn);
    const float r = rsqrtf(ss[0] * inv + a.eps);
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) u[q][j] *= r;
    return r;
}

template <typename XT, typename IoT, typename YT, int NV, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS, norm_blocks_per_sm(false, THREADS))
group_norm_fwd_kernel(const GroupNormArgs a, const NormShape sh) {
    __shared__ float red[2][32][2];
    const Place<WARP> at(sh, red);
    const int64_t base = (at.first % a.G) * sh.gs;
    int turn = 0;
    Raw8<XT> nx[NV];
    Raw8<IoT> nz[NV];
    // a slot's items lie step apart, whole rows
    const int64_t xstep = at.step * sh.gs, zstep = at.step / a.G * a.zs;
    const XT* xp = (const XT*)a.x + at.first * sh.gs;
    const IoT* zp = (const IoT*)a.z + at.first / a.G * a.zs + base;
    YT* yp = (YT*)a.y + at.first * sh.gs;
    auto load = [&](int64_t item) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (at.lane + q * sh.lanes) * 8;
            nx[q].zero();
            nz[q].zero();
            if (item < sh.items && i < sh.gs) {
                nx[q].load(xp + i);
                if (a.act >= kAfter) nz[q].load(zp + i);
            }
        }
        xp += xstep;
        zp += zstep;
    };
    load(at.first);
    // every thread of a block takes part in its sums, with or without an item
    for (int64_t it0 = (int64_t)blockIdx.x * sh.per_block; it0 < sh.items; it0 += at.step) {
        const int64_t item = it0 + at.slot;
        float u[NV][8], gate[NV][8];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            nx[q].get(u[q]);
            if (a.act >= kAfter) {
                nz[q].get(gate[q]);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 v = f2_get(f2_silu(f2_pack(gate[q][j], gate[q][j + 1])));
                    gate[q][j] = v.x;
                    gate[q][j + 1] = v.y;
                }
                if (a.act == kBefore)
#pragma unroll
                    for (int j = 0; j < 8; ++j) u[q][j] *= gate[q][j];
            }
        }
        load(item + at.step);
        normalise<NV, WARP>(a, sh, at, u, turn);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (at.lane + q * sh.lanes) * 8;
            if (item >= sh.items || i >= sh.gs) continue;
            if (a.w) {
                float w[8];
                load8(a.w + base + i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] *= w[j];
            }
            if (a.bias) {
                float w[8];
                load8(a.bias + base + i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] += w[j];
            }
            if (a.act == kAfter) {
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] *= gate[q][j];
            } else if (a.act == kSilu) {
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const float2 v = f2_get(f2_silu(f2_pack(u[q][j], u[q][j + 1])));
                    u[q][j] = v.x;
                    u[q][j + 1] = v.y;
                }
            }
            store8(yp + i, u[q]);
        }
        yp += xstep;
    }
}

template <typename XT, typename IoT, typename GT, int NV, bool WARP, int THREADS>
__global__ void __launch_bounds__(THREADS, norm_blocks_per_sm(true, THREADS))
group_norm_bwd_kernel(const GroupNormArgs a, const NormShape sh) {
    __shared__ float red[2][32][2];
    const Place<WARP> at(sh, red);
    const int64_t base = (at.first % a.G) * sh.gs;
    const float inv = 1.f / (float)sh.gs;
    int turn = 0;
    float dw[NV][8], db[NV][8];
#pragma unroll
    for (int q = 0; q < NV; ++q)
#pragma unroll
        for (int j = 0; j < 8; ++j) dw[q][j] = db[q][j] = 0.f;
    Raw8<XT> nx[NV];
    Raw8<IoT> nz[NV], ny[NV];
    const int64_t xstep = at.step * sh.gs, zstep = at.step / a.G * a.zs;
    const XT* xp = (const XT*)a.x + at.first * sh.gs;
    const IoT* yp = (const IoT*)a.dy + at.first * sh.gs;
    const IoT* zp = (const IoT*)a.z + at.first / a.G * a.zs + base;
    GT* dxp = (GT*)a.dx + at.first * sh.gs;
    GT* dzp = (GT*)a.dz + at.first * sh.gs;
    auto load = [&](int64_t item) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (at.lane + q * sh.lanes) * 8;
            nx[q].zero();
            nz[q].zero();
            ny[q].zero();
            if (item < sh.items && i < sh.gs) {
                nx[q].load(xp + i);
                ny[q].load(yp + i);
                if (a.act >= kAfter) nz[q].load(zp + i);
            }
        }
        xp += xstep;
        yp += xstep;
        zp += zstep;
    };
    load(at.first);
    for (int64_t it0 = (int64_t)blockIdx.x * sh.per_block; it0 < sh.items; it0 += at.step) {
        const int64_t item = it0 + at.slot;
        // s: silu(z); t: what dz takes beside du (x silu'(z)) or beside v (dy silu'(z))
        float u[NV][8], dn[NV][8], s[NV][8], t[NV][8], r, s0 = 0.f, s1;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            nx[q].get(u[q]);
            ny[q].get(dn[q]);
            if (a.act >= kAfter) {
                float z[8];
                nz[q].get(z);
#pragma unroll
                for (int j = 0; j < 8; j += 2) {
                    const f32x2 zz = f2_pack(z[j], z[j + 1]), g = f2_sigmoid(zz);
                    const float2 sv = f2_get(f2_mul(zz, g)), tv = f2_get(f2_silu_grad(zz, g));
                    s[q][j] = sv.x;
                    s[q][j + 1] = sv.y;
                    t[q][j] = tv.x;
                    t[q][j + 1] = tv.y;
                }
                if (a.act == kBefore) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        t[q][j] *= u[q][j];
                        u[q][j] *= s[q][j];
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        t[q][j] *= dn[q][j];
                        dn[q][j] *= s[q][j];                // dv
                    }
                }
            }
        }
        load(item + at.step);
        if (!a.center && a.act != kSilu) {
            float sums[2] = {0.f, 0.f};
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int i = (at.lane + q * sh.lanes) * 8;
                float w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = 1.f;
                if (a.w && i < sh.gs) load8(a.w + base + i, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sums[0] = fmaf(u[q][j], u[q][j], sums[0]);
                    sums[1] = fmaf(dn[q][j] * w[j], u[q][j], sums[1]);
                }
            }
            at.sum(sums, turn);
            r = rsqrtf(sums[0] * inv + a.eps);
            s1 = r * sums[1] * inv;
#pragma unroll
            for (int q = 0; q < NV; ++q)
#pragma unroll
                for (int j = 0; j < 8; ++j) u[q][j] *= r;
        } else {
            r = normalise<NV, WARP>(a, sh, at, u, turn);
            float sums[2] = {0.f, 0.f};
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int i = (at.lane + q * sh.lanes) * 8;
                float w[8], bias[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) { w[j] = 1.f; bias[j] = 0.f; }
                if (a.w && i < sh.gs) load8(a.w + base + i, w);
                if (a.bias && a.act == kSilu && i < sh.gs) load8(a.bias + base + i, bias);
                if (a.act == kSilu) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float v = fmaf(u[q][j], w[j], bias[j]);
                        dn[q][j] *= silu_grad(v, sigmoid_f32(v));
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sums[0] = fmaf(dn[q][j], w[j], sums[0]);
                    sums[1] = fmaf(dn[q][j] * w[j], u[q][j], sums[1]);
                }
            }
            at.sum(sums, turn);
            s0 = a.center ? sums[0] * inv : 0.f;
            s1 = sums[1] * inv;
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int i = (at.lane + q * sh.lanes) * 8;
            if (item >= sh.items || i >= sh.gs) continue;
            float w[8], g[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = 1.f;
            if (a.w) load8(a.w + base + i, w);
            if (a.act == kAfter) {
                float bias[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) bias[j] = 0.f;
                if (a.bias) load8(a.bias + base + i, bias);
#pragma unroll
                for (int j = 0; j < 8; ++j) g[j] = t[q][j] * fmaf(u[q][j], w[j], bias[j]);
                store8(dzp + i, g);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) dw[q][j] = fmaf(dn[q][j], u[q][j], dw[q][j]);
            if (a.db)
#pragma unroll
                for (int j = 0; j < 8; ++j) db[q][j] += dn[q][j];
            const float rs0 = r * s0, rs1 = r * s1;
#pragma unroll
            for (int j = 0; j < 8; ++j) g[j] = fmaf(-rs1, u[q][j], fmaf(dn[q][j] * r, w[j], -rs0));          // du
            if (a.act == kBefore) {
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    t[q][j] *= g[j];
                    g[j] *= s[q][j];
                }
            }
            store8(dxp + i, g);
            if (a.act == kBefore) store8(dzp + i, t[q]);
        }
        dxp += xstep;
        dzp += xstep;
    }
    // slot q's sums: row q / G of [norm_parts][C]
    if (at.first >= sh.items) return;
    float* part = a.ws + at.first * sh.gs;
    const int64_t all = norm_parts(sh, a.rows, a.G) * a.C;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int i = (at.lane + q * sh.lanes) * 8;
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

// Slots: one vector of 8 channels a lane, up to 32 lanes of a warp, then whole
// warps, as many slots a block as make 512 threads; two vectors a lane beyond 8192
// channels (backward: beyond 4096, whose sums and terms take 128 registers a lane).
enum class NormClass { kWarp, kBlock512, kBlock1024, kBlock2 };

static NormShape norm_shape(int64_t rows, int64_t C, int64_t G, bool backward, NormClass* cls) {
    NormShape sh{};
    sh.gs = (int)(C / G);
    const int vecs = sh.gs / 8;
    if (vecs <= 32) {
        *cls = NormClass::kWarp;
        sh.lanes = 1;
        while (sh.lanes < vecs) sh.lanes *= 2;
        sh.threads = 256;
        sh.per_block = 256 / sh.lanes;
    } else {
        *cls = vecs <= 512 ? NormClass::kBlock512 : vecs <= 1024 ? NormClass::kBlock1024 : NormClass::kBlock2;
        const int per_lane = *cls == NormClass::kBlock2 || (backward && *cls == NormClass::kBlock1024) ? 2 : 1;
        sh.lanes = ((vecs + per_lane - 1) / per_lane + 31) / 32 * 32;
        sh.per_block = sh.lanes <= 512 ? 512 / sh.lanes : 1;
        sh.threads = sh.lanes * sh.per_block;
    }
    sh.items = rows * G;
    // blocks: one item a slot where that is few; else a multiple of `unit`, so that all slots together are
    // a multiple of G, and as many as fit on the machine at once, so that each keeps its next item's loads in
    // flight (fewer than `want` of them: every slot has an item)
    int64_t x = G, y = sh.per_block;
    while (y) { const int64_t m = x % y; x = y; y = m; }
    const int64_t unit = G / x, want = (sh.items + sh.per_block - 1) / sh.per_block;
    const bool half = *cls == NormClass::kBlock512 || (backward && *cls == NormClass::kBlock1024);
    const int64_t most = (int64_t)148 * norm_blocks_per_sm(backward, *cls == NormClass::kWarp ? 256 : half ? 512 : 1024);
    sh.blocks = want < most || want <= unit ? want : most / unit > 0 ? most / unit * unit : unit;
    return sh;
}

size_t group_norm_bwd_workspace(int64_t rows, int64_t C, int64_t G) {
    NormClass cls;
    const NormShape sh = norm_shape(rows, C, G, true, &cls);
    return (size_t)norm_parts(sh, rows, G) * C * 2 * sizeof(float);
}

template <typename X, typename I, typename Y> struct NormFwd {
    static void go(const GroupNormArgs& a, const NormShape& sh, NormClass cls, cudaStream_t s) {
        const unsigned grid = (unsigned)sh.blocks;
        if (cls == NormClass::kWarp) group_norm_fwd_kernel<X, I, Y, 1, true, 256><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (cls == NormClass::kBlock512) group_norm_fwd_kernel<X, I, Y, 1, false, 512><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (cls == NormClass::kBlock1024) group_norm_fwd_kernel<X, I, Y, 1, false, 1024><<<grid, sh.threads, 0, s>>>(a, sh);
        else group_norm_fwd_kernel<X, I, Y, 2, false, 1024><<<grid, sh.threads, 0, s>>>(a, sh);
    }
};
template <typename X, typename I, typename Y> struct NormBwd {
    static void go(const GroupNormArgs& a, const NormShape& sh, NormClass cls, cudaStream_t s) {
        const unsigned grid = (unsigned)sh.blocks;
        if (cls == NormClass::kWarp) group_norm_bwd_kernel<X, I, Y, 1, true, 256><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (cls == NormClass::kBlock512) group_norm_bwd_kernel<X, I, Y, 1, false, 512><<<grid, sh.threads, 0, s>>>(a, sh);
        else if (cls == NormClass::kBlock1024) group_norm_bwd_kernel<X, I, Y, 2, false, 512><<<grid, sh.threads, 0, s>>>(a, sh);
        else group_norm_bwd_kernel<X, I, Y, 2, false, 1024><<<grid, sh.threads, 0, s>>>(a, sh);
    }
};

template <template <typename, typename, typename> class F>
static void dispatch_types(const GroupNormArgs& a, const NormShape& sh, NormClass cls, cudaStream_t s) {
    if (a.x_bf16) {
        if (a.io_bf16) { if (a.y_bf16) F<bf16, bf16, bf16>::go(a, sh, cls, s); else F<bf16, bf16, float>::go(a, sh, cls, s); }
        else { if (a.y_bf16) F<bf16, float, bf16>::go(a, sh, cls, s); else F<bf16, float, float>::go(a, sh, cls, s); }
    } else {
        if (a.io_bf16) { if (a.y_bf16) F<float, bf16, bf16>::go(a, sh, cls, s); else F<float, bf16, float>::go(a, sh, cls, s); }
        else { if (a.y_bf16) F<float, float, bf16>::go(a, sh, cls, s); else F<float, float, float>::go(a, sh, cls, s); }
    }
}

cudaError_t launch_group_norm_fwd(const GroupNormArgs& a, cudaStream_t s) {
    NormClass cls;
    const NormShape sh = norm_shape(a.rows, a.C, a.G, false, &cls);
    dispatch_types<NormFwd>(a, sh, cls, s);
    return cudaGetLastError();
}

cudaError_t launch_group_norm_bwd(const GroupNormArgs& a, cudaStream_t s) {
    if (a.rows == 0) {
        if (!a.dw && !a.db) return cudaSuccess;
        group_norm_zero_kernel<<<(unsigned)((a.C + 255) / 256), 256, 0, s>>>(a.dw, a.db, a.C);
        return cudaGetLastError();
    }
    NormClass cls;
    const NormShape sh = norm_shape(a.rows, a.C, a.G, true, &cls);
    dispatch_types<NormBwd>(a, sh, cls, s);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || (!a.dw && !a.db)) return e;
    const int64_t parts = norm_parts(sh, a.rows, a.G);
    const ColumnSum sums[] = {{a.ws, parts, a.C, a.dw ? a.C : 0, a.dw, a.C, nullptr, false},
                              {a.ws + parts * a.C, parts, a.C, a.db ? a.C : 0, a.db, a.C, nullptr, false}};
    return launch_column_sums(sums, 2, s);
}

}  // namespace ssd
