// Backward pass of the selective scan.  With the adjoint of the state carried
// back in time, G_t = C_t g_t + a_{t+1} G_{t+1}, a_t = exp(dt_t A), g = dy silu(z):
//
//   dC_t[n] = sum_d g h_t[n];          dB_t[n] = sum_d G_t[n] dt x
//   dx = dt sum_n G_t B_t + D g;       d dt = sum_n G_t (B_t x + A a_t h_{t-1})
//   dA[n] = sum_t G_t a_t h_{t-1} dt;  dD = sum_t g x;  dz = dy (sum_n C h + D x) silu'(z)
//
// in chunks of T tokens that run in parallel:
//  1. summaries: one walk over each chunk gives its end state from h = 0, and
//     the adjoint at its start from 0 at its end, sum_s (a_0 .. a_s) C_s g_s
//     (the running product serves the adjoint in forward order, so one
//     exponential serves both);
//  2. recombination over the chunks: the state that enters each chunk, the
//     adjoint that leaves it (decay of a chunk: exp(A sum dt));
//  3. per chunk: the states forward, kept in shared memory, then the adjoint
//     back over them.  A block goes over several tiles of channels and adds dB
//     and dC up in shared memory; blocks' sums are added in a fixed order last.
#include "ssd_selective_common.cuh"

namespace ssd {

constexpr int kSbWarps = 4, kSbThreads = kSbWarps * 32;

struct SbShape {
    int K;            // lanes of a channel
    int CT;           // channels of a block
    int Dg, tiles;    // channels of a group, blocks that cover them
    int Np;           // K * S
};

template <int S>
inline SbShape sel_shape(int64_t D, int64_t N, int64_t G, int warps) {
    SbShape sh{};
    sh.K = 1;
    while (sh.K * S < N) sh.K *= 2;
    sh.Np = sh.K * S;
    sh.CT = warps * (32 / sh.K) * 2;
    sh.Dg = (int)(D / G);
    sh.tiles = (sh.Dg + sh.CT - 1) / sh.CT;
    return sh;
}

struct SbLayout {
    int T;                       // tokens of a chunk
    int nch;                     // chunks of a sequence
    int split;                   // blocks that share a chunk's tiles of channels
    size_t off_h, off_g;         // fp32 [b][nch][D][N] chunk states, then adjoints
    size_t off_dt;               // fp32 [b][nch][D] sum of dt
    size_t off_dA;               // fp32 [b][nch][D][N]
    size_t off_par;              // fp32 [b][nch][2][D]: d dt_bias, dD
    size_t off_dB, off_dC;       // fp32 [split][b][L][G][N]
    size_t total;
};

static int sb_states(int64_t N) { return N > 128 ? 8 : 4; }

static SbLayout sb_layout(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    SbLayout l{};
    const SbShape sh = sb_states(N) == 8 ? sel_shape<8>(D, N, G, kSbWarps) : sel_shape<4>(D, N, G, kSbWarps);
    l.T = sb_states(N) == 8 ? 8 : 16;
    l.nch = (int)((L + l.T - 1) / l.T);
    const int64_t chunks = batch * l.nch * G, want = 148 * 6;
    l.split = (int)(chunks >= want || chunks == 0 ? 1 : (want + chunks - 1) / chunks);
    if (l.split > sh.tiles) l.split = sh.tiles;
    const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    const size_t bn = (size_t)batch * l.nch, st = bn * D * N * sizeof(float);
    l.off_h = 0;
    l.off_g = up(l.off_h + st);
    l.off_dt = up(l.off_g + st);
    l.off_dA = up(l.off_dt + bn * D * sizeof(float));
    l.off_par = up(l.off_dA + st);
    l.off_dB = up(l.off_par + bn * 2 * D * sizeof(float));
    const size_t bc = (size_t)l.split * batch * L * G * N * sizeof(float);
    l.off_dC = up(l.off_dB + bc);
    l.total = up(l.off_dC + bc);
    return l;
}

size_t selective_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    return batch == 0 || L == 0 ? 0 : sb_layout(batch, L, D, N, G).total;
}

// Stages dt, x, g (fp32, zero past the sequence and the group's channels) and B, C of a chunk.
template <typename IoT>
__device__ __forceinline__ void sb_stage(const SelectiveArgs& a, const SbShape& sh, int T, int64_t b, int64_t g,
                                         int64_t t0, int nt, int64_t d0, int nc, float* sdt, float* sx, float* sg,
                                         float* sB, float* sC) {
    const int CT = sh.CT, Np = sh.Np;
    const int64_t tok0 = b * a.L + t0;
    for (int i = threadIdx.x; i < T * (CT / 8); i += kSbThreads) {
        const int t = i / (CT / 8), c = (i % (CT / 8)) * 8;
        float x[8], dt[8], gy[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = dt[j] = gy[j] = 0.f;
        if (t < nt && c < nc) {
            const int64_t at = (tok0 + t) * a.D + d0 + c;
            load8((const IoT*)a.x + at, x);
            load8((const IoT*)a.dt_raw + at, dt);
            load8((const IoT*)a.dy + at, gy);
#pragma unroll
            for (int j = 0; j < 8; ++j) dt[j] = softplus_f32(dt[j] + (a.dt_bias ? a.dt_bias[d0 + c + j] : 0.f));
            if (a.z) {
                float z[8];
                load8((const IoT*)a.z + (tok0 + t) * a.zs + d0 + c, z);
#pragma unroll
                for (int j = 0; j < 8; ++j) gy[j] *= z[j] * sigmoid_f32(z[j]);
            }
        }
        store8(sdt + t * CT + c, dt);
        store8(sx + t * CT + c, x);
        store8(sg + t * CT + c, gy);
    }
    if (!sB) return;
    for (int i = threadIdx.x; i < T * Np; i += kSbThreads) {
        const int t = i / Np, n = i % Np;
        float bv = 0.f, cv = 0.f;
        if (t < nt && n < a.N) {
            const int64_t k = ((tok0 + t) * a.G + g) * a.N + n;
            bv = to_f32(((const IoT*)a.B)[k]);
            cv = to_f32(((const IoT*)a.C)[k]);
        }
        sB[i] = bv;
        sC[i] = cv;
    }
}

// loads the lane's A (times log2 e) of 2 channels
template <int S>
__device__ __forceinline__ void load_A(const SelectiveArgs& a, int64_t d, bool ok, int n0, float (&A2)[2][S]) {
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 0; s < S; ++s) A2[e][s] = ok && n0 + s < a.N ? a.A[(d + e) * a.N + n0 + s] * kLog2e : 0.f;
}

template <typename IoT, int S>
__global__ void __launch_bounds__(kSbThreads)
selective_bwd_summary_kernel(const SelectiveArgs a, const SbShape sh, const SbLayout l) {
    extern __shared__ float4 smem4[];
    const int T = l.T, CT = sh.CT, Np = sh.Np, K = sh.K;
    float* sdt = (float*)smem4;
    float* sx = sdt + T * CT;
    float* sg = sx + T * CT;
    float* sB = sg + T * CT;
    float* sC = sB + T * Np;
    const int tile = (int)(blockIdx.x % (unsigned)sh.tiles);
    int64_t r = blockIdx.x / (unsigned)sh.tiles;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % l.nch, b = r / l.nch, t0 = ck * l.T;
    const int nt = a.L - t0 < T ? (int)(a.L - t0) : T;
    const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;
    const int64_t d0 = g * sh.Dg + c0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pair = warp * (32 / K) + lane / K, n0 = (lane % K) * S, ch = pair * 2;
    const bool ok = ch < nc;
    sb_stage<IoT>(a, sh, T, b, g, t0, nt, d0, nc, sdt, sx, sg, sB, sC);
    float A2[2][S], h[2][S], P[2][S], Gs[2][S], sum[2] = {0.f, 0.f};
    load_A<S>(a, d0 + ch, ok, n0, A2);
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 0; s < S; ++s) { h[e][s] = Gs[e][s] = 0.f; P[e][s] = 1.f; }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
        float B[S], C[S];
#pragma unroll
        for (int s = 0; s < S; s += 4) {
            Vec16<float>::load(sB + t * Np + n0 + s, B + s);
            Vec16<float>::load(sC + t * Np + n0 + s, C + s);
        }
        const float2 dt2 = *(const float2*)(sdt + t * CT + ch), x2 = *(const float2*)(sx + t * CT + ch);
        const float2 g2 = *(const float2*)(sg + t * CT + ch);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float dt = e ? dt2.y : dt2.x, dx = dt * (e ? x2.y : x2.x), gy = e ? g2.y : g2.x;
            sum[e] += dt;
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const float av = exp2_approx(dt * A2[e][s]);
                h[e][s] = fmaf(av, h[e][s], dx * B[s]);
                P[e][s] *= av;
                Gs[e][s] = fmaf(P[e][s], C[s] * gy, Gs[e][s]);
            }
        }
    }
    float* wh = (float*)(a.ws + l.off_h);
    float* wg = (float*)(a.ws + l.off_g);
    const int64_t bc = b * l.nch + ck;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        if (!ok) continue;
        if (n0 == 0) ((float*)(a.ws + l.off_dt))[bc * a.D + d0 + ch + e] = sum[e];
#pragma unroll
        for (int s = 0; s < S; ++s)
            if (n0 + s < a.N) {
                const int64_t k = (bc * a.D + d0 + ch + e) * a.N + n0 + s;
                wh[k] = h[e][s];
                wg[k] = Gs[e][s];
            }
    }
}

// Thread = one state: the chunks' end states become the states that enter them,
// their adjoints the ones that leave them.
__global__ void __launch_bounds__(128)
selective_bwd_chunks_kernel(const SelectiveArgs a, const SbLayout l) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, DN = a.D * a.N;
    if (i >= a.batch * DN) return;
    const int64_t b = i / DN, dn = i % DN, d = dn / a.N;
    const float A2 = a.A[dn] * kLog2e;
    float* wh = (float*)(a.ws + l.off_h) + b * l.nch * DN + dn;
    float* wg = (float*)(a.ws + l.off_g) + b * l.nch * DN + dn;
    const float* wdt = (const float*)(a.ws + l.off_dt) + b * l.nch * a.D + d;
    float h = 0.f, w = 0.f;
    if (a.init) h = a.state_bf16 ? to_f32(((const bf16*)a.init)[i]) : ((const float*)a.init)[i];
    if (a.dfinal) w = a.state_bf16 ? to_f32(((const bf16*)a.dfinal)[i]) : ((const float*)a.dfinal)[i];
    for (int64_t c = 0; c < l.nch; ++c) {
        const float end = wh[c * DN];
        wh[c * DN] = h;
        h = fmaf(exp2_approx(wdt[c * a.D] * A2), h, end);
    }
    for (int64_t c = l.nch - 1; c >= 0; --c) {
        const float start = wg[c * DN];
        wg[c * DN] = w;
        w = fmaf(exp2_approx(wdt[c * a.D] * A2), w, start);
    }
    if (a.dinit) {
        if (a.state_bf16) ((bf16*)a.dinit)[i] = from_f32<bf16>(w);
        else ((float*)a.dinit)[i] = w;
    }
}

template <typename IoT, typename GT, int S>
__global__ void __launch_bounds__(kSbThreads)
selective_bwd_main_kernel(const SelectiveArgs a, const SbShape sh, const SbLayout l) {
    extern __shared__ float4 smem4[];
    const int T = l.T, CT = sh.CT, Np = sh.Np, K = sh.K;
    float4* hs = smem4;                                // [T][2 S / 4][threads]
    float* acc = (float*)(hs + T * (S / 2) * kSbThreads);   // [warps][T][dB, dC][Np]
    float* sdt = acc + kSbWarps * T * 2 * Np;
    float* sx = sdt + T * CT;
    float* sg = sx + T * CT;
    float* so = sg + T * CT;                           // [3][T][CT]: sum C h, sum G B, sum G A a h
    float* sB = so + 3 * T * CT;
    float* sC = sB + T * Np;
    const int sp = (int)(blockIdx.x % (unsigned)l.split);
    int64_t r = blockIdx.x / (unsigned)l.split;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % l.nch, b = r / l.nch, t0 = ck * l.T;
    const int nt = a.L - t0 < T ? (int)(a.L - t0) : T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pair = warp * (32 / K) + lane / K, n0 = (lane % K) * S, ch = pair * 2;
    const int64_t bc = b * l.nch + ck, tok0 = b * a.L + t0;
    for (int i = tid; i < kSbWarps * T * 2 * Np; i += kSbThreads) acc[i] = 0.f;
    float* wacc = acc + warp * T * 2 * Np;

    for (int tile = sp; tile < sh.tiles; tile += l.split) {
        const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;
        const int64_t d0 = g * sh.Dg + c0;
        const bool ok = ch < nc;
        __syncthreads();                               // the tile before has been read
        sb_stage<IoT>(a, sh, T, b, g, t0, nt, d0, nc, sdt, sx, sg, tile == sp ? sB : nullptr, sC);
        float A2[2][S], h[2][S], w[2][S], dA[2][S];
        load_A<S>(a, d0 + ch, ok, n0, A2);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int s = 0; s < S; ++s) {
                const bool in = ok && n0 + s < a.N;
                const int64_t k = (bc * a.D + d0 + ch + e) * a.N + n0 + s;
                h[e][s] = in ? ((const float*)(a.ws + l.off_h))[k] : 0.f;
                w[e][s] = in ? ((const float*)(a.ws + l.off_g))[k] : 0.f;
                dA[e][s] = 0.f;
            }
        __syncthreads();
        for (int t = 0; t < nt; ++t) {
            float B[S], C[S], y[2] = {0.f, 0.f}, dC[S];
#pragma unroll
            for (int s = 0; s < S; s += 4) {
                Vec16<float>::load(sB + t * Np + n0 + s, B + s);
                Vec16<float>::load(sC + t * Np + n0 + s, C + s);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) dC[s] = 0.f;
            const float2 dt2 = *(const float2*)(sdt + t * CT + ch), x2 = *(const float2*)(sx + t * CT + ch);
            const float2 g2 = *(const float2*)(sg + t * CT + ch);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float dt = e ? dt2.y : dt2.x, dx = dt * (e ? x2.y : x2.x), gy = e ? g2.y : g2.x;
#pragma unroll
                for (int s = 0; s < S; s += 4)
                    hs[(t * (S / 2) + e * (S / 4) + s / 4) * kSbThreads + tid] =
                        make_float4(h[e][s], h[e][s + 1], h[e][s + 2], h[e][s + 3]);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    h[e][s] = fmaf(exp2_approx(dt * A2[e][s]), h[e][s], dx * B[s]);
                    y[e] = fmaf(C[s], h[e][s], y[e]);
                    dC[s] = fmaf(gy, h[e][s], dC[s]);
                }
            }
            for (int o = 1; o < K; o <<= 1) {
                y[0] += __shfl_xor_sync(0xffffffffu, y[0], o);
                y[1] += __shfl_xor_sync(0xffffffffu, y[1], o);
            }
            if (n0 == 0) *(float2*)(so + t * CT + ch) = make_float2(y[0], y[1]);
            for (int o = K; o < 32; o <<= 1)
#pragma unroll
                for (int s = 0; s < S; ++s) dC[s] += __shfl_xor_sync(0xffffffffu, dC[s], o);
            if (lane < K)
#pragma unroll
                for (int s = 0; s < S; ++s) wacc[(t * 2 + 1) * Np + n0 + s] += dC[s];
        }
        for (int t = nt - 1; t >= 0; --t) {
            float B[S], C[S], wB[2] = {0.f, 0.f}, wA[2] = {0.f, 0.f}, dB[S];
#pragma unroll
            for (int s = 0; s < S; s += 4) {
                Vec16<float>::load(sB + t * Np + n0 + s, B + s);
                Vec16<float>::load(sC + t * Np + n0 + s, C + s);
            }
#pragma unroll
            for (int s = 0; s < S; ++s) dB[s] = 0.f;
            const float2 dt2 = *(const float2*)(sdt + t * CT + ch), x2 = *(const float2*)(sx + t * CT + ch);
            const float2 g2 = *(const float2*)(sg + t * CT + ch);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float dt = e ? dt2.y : dt2.x, dx = dt * (e ? x2.y : x2.x), gy = e ? g2.y : g2.x;
#pragma unroll
                for (int s4 = 0; s4 < S; s4 += 4) {
                    const float4 hv = hs[(t * (S / 2) + e * (S / 4) + s4 / 4) * kSbThreads + tid];
                    const float hp[4] = {hv.x, hv.y, hv.z, hv.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int s = s4 + q;
                        const float av = exp2_approx(dt * A2[e][s]);
                        w[e][s] = fmaf(C[s], gy, w[e][s]);
                        wB[e] = fmaf(w[e][s], B[s], wB[e]);
                        dB[s] = fmaf(w[e][s], dx, dB[s]);
                        w[e][s] *= av;                     // the adjoint one token back
                        const float wah = w[e][s] * hp[q];
                        wA[e] = fmaf(wah, A2[e][s], wA[e]);
                        dA[e][s] = fmaf(wah, dt, dA[e][s]);
                    }
                }
            }
            for (int o = 1; o < K; o <<= 1) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    wB[e] += __shfl_xor_sync(0xffffffffu, wB[e], o);
                    wA[e] += __shfl_xor_sync(0xffffffffu, wA[e], o);
                }
            }
            if (n0 == 0) {
                *(float2*)(so + (T + t) * CT + ch) = make_float2(wB[0], wB[1]);
                *(float2*)(so + (2 * T + t) * CT + ch) = make_float2(wA[0] * (1.f / kLog2e), wA[1] * (1.f / kLog2e));
            }
            for (int o = K; o < 32; o <<= 1)
#pragma unroll
                for (int s = 0; s < S; ++s) dB[s] += __shfl_xor_sync(0xffffffffu, dB[s], o);
            if (lane < K)
#pragma unroll
                for (int s = 0; s < S; ++s) wacc[t * 2 * Np + n0 + s] += dB[s];
        }
        float* wdA = (float*)(a.ws + l.off_dA);
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (ok && n0 + s < a.N) wdA[(bc * a.D + d0 + ch + e) * a.N + n0 + s] = dA[e][s];
        __syncthreads();
        // per channel and token: dx, d dt_raw, dz; d dt_raw and g x stay for their sums over the tokens
        for (int i = tid; i < nt * (CT / 8); i += kSbThreads) {
            const int t = i / (CT / 8), c = (i % (CT / 8)) * 8;
            if (c >= nc) continue;
            const int64_t at = (tok0 + t) * a.D + d0 + c;
            float raw[8], dx[8], ddt[8];
            load8((const IoT*)a.dt_raw + at, raw);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = t * CT + c + j;
                const float wB = so[T * CT + k], Dv = a.Dv ? a.Dv[d0 + c + j] : 0.f;
                dx[j] = fmaf(sdt[k], wB, Dv * sg[k]);
                ddt[j] = fmaf(sx[k], wB, so[2 * T * CT + k]) * sigmoid_f32(raw[j] + (a.dt_bias ? a.dt_bias[d0 + c + j] : 0.f));
            }
            store8((GT*)a.dx + at, dx);
            store8((GT*)a.ddt + at, ddt);
            if (a.z) {
                float z[8], dy[8], dz[8];
                load8((const IoT*)a.z + (tok0 + t) * a.zs + d0 + c, z);
                load8((const IoT*)a.dy + at, dy);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int k = t * CT + c + j;
                    const float q = sigmoid_f32(z[j]);
                    dz[j] = dy[j] * fmaf(a.Dv ? a.Dv[d0 + c + j] : 0.f, sx[k], so[k]) * q * fmaf(z[j], 1.f - q, 1.f);
                }
                store8((GT*)a.dz + at, dz);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int k = t * CT + c + j;
                so[T * CT + k] = ddt[j];
                so[k] = sg[k] * sx[k];
            }
        }
        __syncthreads();
        for (int c = tid; c < nc; c += kSbThreads) {
            float s0 = 0.f, s1 = 0.f;
            for (int t = 0; t < nt; ++t) { s0 += so[(T + t) * CT + c]; s1 += so[t * CT + c]; }
            float* par = (float*)(a.ws + l.off_par) + bc * 2 * a.D + d0 + c;
            par[0] = s0;
            par[a.D] = s1;
        }
    }
    __syncthreads();
    for (int i = tid; i < nt * 2 * Np; i += kSbThreads) {
        const int n = i % Np, which = (i / Np) & 1, t = i / (2 * Np);
        if (n >= a.N) continue;
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kSbWarps; ++q) s += acc[q * T * 2 * Np + i];
        float* out = (float*)(a.ws + (which ? l.off_dC : l.off_dB));
        out[((int64_t)sp * a.batch * a.L + tok0 + t) * a.G * a.N + g * a.N + n] = s;
    }
}

// batch or seqlen 0: parameter gradients 0, dinit = dfinal
__global__ void selective_bwd_empty_kernel(const SelectiveArgs a) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x, DN = a.D * a.N;
    if (i < DN) a.dA[i] = 0.f;
    if (i < a.D) {
        if (a.ddt_bias) a.ddt_bias[i] = 0.f;
        if (a.dD) a.dD[i] = 0.f;
    }
    if (a.dinit && i < a.batch * DN) {
        if (a.state_bf16) ((bf16*)a.dinit)[i] = a.dfinal ? ((const bf16*)a.dfinal)[i] : from_f32<bf16>(0.f);
        else ((float*)a.dinit)[i] = a.dfinal ? ((const float*)a.dfinal)[i] : 0.f;
    }
}

template <typename IoT, typename GT, int S>
static cudaError_t launch_bwd_t(const SelectiveArgs& a, cudaStream_t s) {
    const SbShape sh = sel_shape<S>(a.D, a.N, a.G, kSbWarps);
    const SbLayout l = sb_layout(a.batch, a.L, a.D, a.N, a.G);
    const int smem1 = (int)sizeof(float) * l.T * (3 * sh.CT + 2 * sh.Np);
    const int smem3 = (int)sizeof(float) * l.T * (2 * S * kSbThreads + kSbWarps * 2 * sh.Np + 6 * sh.CT + 2 * sh.Np);
    const auto k1 = selective_bwd_summary_kernel<IoT, S>;
    const auto k3 = selective_bwd_main_kernel<IoT, GT, S>;
    cudaError_t e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, smem1);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(k3, cudaFuncAttributeMaxDynamicSharedMemorySize, smem3);
    if (e != cudaSuccess) return e;
    const int64_t chunks = a.batch * l.nch * a.G;
    k1<<<(unsigned)(chunks * sh.tiles), kSbThreads, smem1, s>>>(a, sh, l);
    selective_bwd_chunks_kernel<<<(unsigned)((a.batch * a.D * a.N + 127) / 128), 128, 0, s>>>(a, l);
    k3<<<(unsigned)(chunks * l.split), kSbThreads, smem3, s>>>(a, sh, l);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t bn = a.batch * l.nch, DN = a.D * a.N, M = a.batch * a.L * a.G * a.N;
    const bool gb = sizeof(GT) == 2;
    const float* par = (const float*)(a.ws + l.off_par);
    e = launch_column_sum((const float*)(a.ws + l.off_dA), bn, DN, DN, a.dA, false, s);
    if (e == cudaSuccess && a.ddt_bias) e = launch_column_sum(par, bn, 2 * a.D, a.D, a.ddt_bias, false, s);
    if (e == cudaSuccess && a.dD) e = launch_column_sum(par + a.D, bn, 2 * a.D, a.D, a.dD, false, s);
    if (e == cudaSuccess) e = launch_column_sum((const float*)(a.ws + l.off_dB), l.split, M, M, a.dB, gb, s);
    if (e == cudaSuccess) e = launch_column_sum((const float*)(a.ws + l.off_dC), l.split, M, M, a.dC, gb, s);
    return e;
}

template <typename IoT, typename GT>
static cudaError_t launch_bwd_s(const SelectiveArgs& a, cudaStream_t s) {
    return sb_states(a.N) == 8 ? launch_bwd_t<IoT, GT, 8>(a, s) : launch_bwd_t<IoT, GT, 4>(a, s);
}

cudaError_t launch_selective_bwd(const SelectiveArgs& a, cudaStream_t s) {
    if (a.batch == 0 || a.L == 0) {
        int64_t n = a.D * a.N * (a.batch > 1 ? a.batch : 1);
        selective_bwd_empty_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    if (a.io_bf16) return a.y_bf16 ? launch_bwd_s<bf16, bf16>(a, s) : launch_bwd_s<bf16, float>(a, s);
    return a.y_bf16 ? launch_bwd_s<float, bf16>(a, s) : launch_bwd_s<float, float>(a, s);
}

}  // namespace ssd
