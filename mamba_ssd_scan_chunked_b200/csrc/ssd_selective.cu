// Selective scan: the recurrence with a decay for each channel and state,
//
//   dt_t = softplus(dt_raw_t + dt_bias);   h_t[n] = exp(dt_t A[n]) h_{t-1}[n] + dt_t x_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
//
// and its single-token step.  With a decay of its own for every state there is
// no matrix to contract (the chunked scan's L has one entry per head and pair
// of tokens), so each state of each token costs one exponential and three
// fp32 operations: with 16 states or more the scan is bound by the special
// function units (16 results a clock and SM), below HBM's time otherwise.
#include "ssd_selective_common.cuh"

namespace ssd {

constexpr int kSelWarps = 4, kSelThreads = kSelWarps * 32, kSelTile = 32;

// Tiles of kSelTile tokens: the block forms dt and dt x once per token and
// channel in shared memory (with B and C in fp32), walks over the tile, each
// warp on its own channels, and then gates and stores the tile's y.
template <typename IoT, typename YT, int S>
__global__ void __launch_bounds__(kSelThreads)
selective_fwd_kernel(const SelectiveArgs a, const SelShape sh) {
    extern __shared__ float4 smem4[];
    constexpr int T = kSelTile;
    const int CT = sh.CT, Np = sh.Np, K = sh.K;
    float* sdt = (float*)smem4;              // [T][CT / 2][dt, dt, dt x, dt x]
    float* sB = sdt + T * CT * 2;            // [T][Np]
    float* sC = sB + T * Np;
    float* sy = sC + T * Np;                 // [T][CT]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = (int)(blockIdx.x % (unsigned)sh.tiles);
    const int64_t bg = blockIdx.x / (unsigned)sh.tiles;
    const int64_t b = bg / a.G, g = bg % a.G;
    const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;   // channels of the group here
    const int64_t d0 = g * sh.Dg + c0;
    int64_t p = a.pad_left ? a.pad_left[b] : 0;
    p = p < 0 ? 0 : p > a.L ? a.L : p;

    const int pair = warp * (32 / K) + lane / K, n0 = (lane % K) * S;
    const int ch = pair * 2;                 // channel in the block
    float A2[2][S], h[2][S];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool ok = ch + e < nc && n0 + s < a.N;
            const int64_t i = (d0 + ch + e) * a.N + n0 + s;
            A2[e][s] = ok ? a.A[i] * kLog2e : 0.f;
            h[e][s] = 0.f;
            if (ok && a.init) {
                const int64_t k = b * a.D * a.N + i;
                h[e][s] = a.state_bf16 ? to_f32(((const bf16*)a.init)[k]) : ((const float*)a.init)[k];
            }
        }
    const int64_t tok0 = b * a.L;
    for (int64_t t0 = 0; t0 < a.L; t0 += T) {
        __syncthreads();                     // the tile before has been read
        for (int i = tid; i < T * (CT / 8); i += kSelThreads) {
            const int t = i / (CT / 8), c = (i % (CT / 8)) * 8;
            const int64_t tt = t0 + t;
            float x[8], dt[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = dt[j] = 0.f;
            if (tt >= p && tt < a.L && c < nc) {
                load8((const IoT*)a.x + (tok0 + tt) * a.D + d0 + c, x);
                load8((const IoT*)a.dt_raw + (tok0 + tt) * a.D + d0 + c, dt);
#pragma unroll
                for (int j = 0; j < 8; ++j) dt[j] = softplus_f32(dt[j] + (a.dt_bias ? a.dt_bias[d0 + c + j] : 0.f));
            }
            float4* out = (float4*)(sdt + (t * CT + c) * 2);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[j] = make_float4(dt[2 * j], dt[2 * j + 1], dt[2 * j] * x[2 * j], dt[2 * j + 1] * x[2 * j + 1]);
        }
        for (int i = tid; i < T * Np; i += kSelThreads) {
            const int t = i / Np, n = i % Np;
            const int64_t tt = t0 + t;
            float bv = 0.f, cv = 0.f;
            if (tt >= p && tt < a.L && n < a.N) {
                const int64_t k = ((tok0 + tt) * a.G + g) * a.N + n;
                bv = to_f32(((const IoT*)a.B)[k]);
                cv = to_f32(((const IoT*)a.C)[k]);
            }
            sB[i] = bv;
            sC[i] = cv;
        }
        __syncthreads();
        const int nt = a.L - t0 < T ? (int)(a.L - t0) : T;
#pragma unroll 2
        for (int t = 0; t < nt; ++t) {
            const float4 d = *(const float4*)(sdt + t * CT * 2 + pair * 4);
            float B[S], C[S], y[2] = {0.f, 0.f};
#pragma unroll
            for (int s = 0; s < S; s += 4) {
                Vec16<float>::load(sB + t * Np + n0 + s, B + s);
                Vec16<float>::load(sC + t * Np + n0 + s, C + s);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float dt = e ? d.y : d.x, dx = e ? d.w : d.z;
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    h[e][s] = fmaf(exp2_approx(dt * A2[e][s]), h[e][s], dx * B[s]);
                    y[e] = fmaf(C[s], h[e][s], y[e]);
                }
            }
            for (int o = 1; o < K; o <<= 1) {
                y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
                y[1] += __shfl_xor_sync(0xffffffffu, y[1], o);
            }
            if (n0 == 0) *(float2*)(sy + t * CT + ch) = make_float2(y[0], y[1]);
        }
        __syncthreads();
        for (int i = tid; i < nt * (CT / 8); i += kSelThreads) {
            const int t = i / (CT / 8), c = (i % (CT / 8)) * 8;
            if (c >= nc) continue;
            const int64_t tt = t0 + t, at = (tok0 + tt) * a.D + d0 + c;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = 0.f;
            if (tt >= p) {
                float x[8];
                load8((const IoT*)a.x + at, x);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(a.Dv ? a.Dv[d0 + c + j] : 0.f, x[j], sy[t * CT + c + j]);
                if (a.z) {
                    float z[8];
                    load8((const IoT*)a.z + (tok0 + tt) * a.zs + d0 + c, z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= z[j] * sigmoid_f32(z[j]);
                }
            }
            store8((YT*)a.y + at, y);
        }
    }
    if (a.final_state) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (ch + e < nc && n0 + s < a.N) {
                    const int64_t k = b * a.D * a.N + (d0 + ch + e) * a.N + n0 + s;
                    if (a.state_bf16) ((bf16*)a.final_state)[k] = from_f32<bf16>(h[e][s]);
                    else ((float*)a.final_state)[k] = h[e][s];
                }
    }
}

// One token: K lanes hold a channel's states, 4 neighbouring ones each (8 with
// more than 128 states, in two rounds of 4).
template <typename StateT, typename IoT, typename YT>
__global__ void __launch_bounds__(128)
selective_update_kernel(const SelectiveArgs a, int K, int per_block) {
    const int lane = threadIdx.x % K, slot = threadIdx.x / K;
    const int64_t bd = (int64_t)blockIdx.x * per_block + slot, all = a.batch * a.D;
    const bool live = bd < all;               // every lane takes part in the sums
    const int64_t b = live ? bd / a.D : 0, d = live ? bd % a.D : 0;
    const int64_t g = d / (a.D / a.G);
    const float dt = softplus_f32(to_f32(((const IoT*)a.dt_raw)[b * a.D + d]) + (a.dt_bias ? a.dt_bias[d] : 0.f));
    const float x = to_f32(((const IoT*)a.x)[b * a.D + d]);
    float y = 0.f;
    for (int n = lane * 4; n < a.N; n += K * 4) {
        const float4 A = *(const float4*)(a.A + d * a.N + n);
        const float Av[4] = {A.x, A.y, A.z, A.w};
        StateT* hp = (StateT*)a.final_state + (b * a.D + d) * a.N + n;
        const IoT* Bp = (const IoT*)a.B + (b * a.G + g) * a.N + n;
        const IoT* Cp = (const IoT*)a.C + (b * a.G + g) * a.N + n;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const float h = fmaf(exp2_approx(dt * (Av[s] * kLog2e)), to_f32(hp[s]), dt * x * to_f32(Bp[s]));
            y = fmaf(to_f32(Cp[s]), h, y);
            if (live) hp[s] = from_f32<StateT>(h);
        }
    }
    for (int o = 1; o < K; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (live && lane == 0) {
        y = fmaf(a.Dv ? a.Dv[d] : 0.f, x, y);
        if (a.z) {
            const float z = to_f32(((const IoT*)a.z)[b * a.zs + d]);
            y *= z * sigmoid_f32(z);
        }
        ((YT*)a.y)[b * a.D + d] = from_f32<YT>(y);
    }
}

size_t selective_workspace(int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

int64_t selective_blocks(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t) {
    return batch * (L / 8 + 1) * (D / 8) * ((N + 15) / 16);
}

template <typename IoT, typename YT, int S>
static cudaError_t launch_fwd_t(const SelectiveArgs& a, cudaStream_t s) {
    const SelShape sh = sel_shape<S>(a.D, a.N, a.G, kSelWarps);
    const int smem = (int)sizeof(float) * kSelTile * (3 * sh.CT + 2 * sh.Np);
    const auto kern = selective_fwd_kernel<IoT, YT, S>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    kern<<<(unsigned)(a.batch * a.G * sh.tiles), kSelThreads, smem, s>>>(a, sh);
    return cudaGetLastError();
}

template <typename IoT, typename YT>
static cudaError_t launch_fwd_s(const SelectiveArgs& a, cudaStream_t s) {
    return a.N > 128 ? launch_fwd_t<IoT, YT, 8>(a, s) : launch_fwd_t<IoT, YT, 4>(a, s);
}

cudaError_t launch_selective_fwd(const SelectiveArgs& a, cudaStream_t s) {
    if (a.io_bf16) return a.y_bf16 ? launch_fwd_s<bf16, bf16>(a, s) : launch_fwd_s<bf16, float>(a, s);
    return a.y_bf16 ? launch_fwd_s<float, bf16>(a, s) : launch_fwd_s<float, float>(a, s);
}

template <typename StateT, typename IoT>
static void launch_update_t(const SelectiveArgs& a, cudaStream_t s) {
    int K = 1;
    while (K < 32 && K * 4 < a.N) K *= 2;
    const int per = 128 / K;
    const unsigned grid = (unsigned)((a.batch * a.D + per - 1) / per);
    if (a.y_bf16) selective_update_kernel<StateT, IoT, bf16><<<grid, 128, 0, s>>>(a, K, per);
    else selective_update_kernel<StateT, IoT, float><<<grid, 128, 0, s>>>(a, K, per);
}

cudaError_t launch_selective_update(const SelectiveArgs& a, cudaStream_t s) {
    if (a.state_bf16) {
        if (a.io_bf16) launch_update_t<bf16, bf16>(a, s); else launch_update_t<bf16, float>(a, s);
    } else {
        if (a.io_bf16) launch_update_t<float, bf16>(a, s); else launch_update_t<float, float>(a, s);
    }
    return cudaGetLastError();
}

}  // namespace ssd
