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

// A block owns CT channels of a group and walks over a run of tokens in tiles of
// T.  A tile's raw inputs are loaded while the tile before is computed; dt and
// dt x are formed once per token and channel into shared memory, B and C widened
// beside them (two buffers); each warp then walks over the tile on its own
// channels, and the block gates and stores the tile's y with whole vectors.
//
// Where batch and channels are too few for the machine the sequence is cut into
// nch chunks: SUMMARY is the pass that finds the end state of every chunk but
// the last from 0 and the sum of its dt, selective_chunks_kernel the state that
// enters each, and the main pass starts from it.
template <typename IoT, typename YT, class Tile, int T, bool SUMMARY>
__global__ void __launch_bounds__(Tile::W * 32, Tile::W == 4 ? 4 : 2)
selective_fwd_kernel(const SelectiveArgs a, const SelShape sh, float* __restrict__ wstate, float* __restrict__ wdt) {
    constexpr int K = Tile::K, S = Tile::S, Np = Tile::Np, P = Tile::P, CT = Tile::CT, THREADS = Tile::W * 32;
    constexpr int V = CT / 8;                                   // 8-channel vectors of a token here
    constexpr int IT = (T * V + THREADS - 1) / THREADS;         // of a thread in a tile
    constexpr int BN = T * Np / 8;                              // 8-state vectors of a tile's B
    constexpr int IB = ((SUMMARY ? 1 : 2) * BN + THREADS - 1) / THREADS;
    constexpr int YS = CT % 32 == 0 ? CT + 16 : CT;             // row of y: no bank conflict between 4 tokens
    extern __shared__ float4 smem4[];
    float4* sd = smem4;                                         // [2][T][CT / 2]: dt, dt, dt x, dt x
    float* sB = (float*)(sd + 2 * T * (CT / 2));                // [2][T][Np]
    float* sC = sB + 2 * T * Np;                                // [2][T][Np]
    float* sy = sC + (SUMMARY ? 0 : 2 * T * Np);                // [T][YS]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t nch = SUMMARY ? sh.nch - 1 : sh.nch;
    int64_t r = blockIdx.x;
    const int tile = (int)(r % sh.tiles);
    r /= sh.tiles;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % nch, b = r / nch;
    const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;   // channels of the group here
    const int64_t d0 = g * sh.Dg + c0;
    const int64_t tb = ck * sh.clen, te = tb + sh.clen < a.L ? tb + sh.clen : a.L;
    int64_t p = a.pad_left ? a.pad_left[b] : 0;
    p = p < 0 ? 0 : p > a.L ? a.L : p;

    const int pair = warp * P + lane % P, n0 = (lane / P) * S, ch = pair * 2;
    const int slot = pair ^ ((pair >> 3) & 7);                  // where the pair lies in a row of sd (see stage)
    float A2[2][S], h[2][S], sum[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const bool ok = ch + e < nc && n0 + s < a.N;
            const int64_t i = (d0 + ch + e) * a.N + n0 + s;
            A2[e][s] = ok ? a.A[i] * kLog2e : 0.f;
            h[e][s] = 0.f;
            if (!SUMMARY && ok) {
                const int64_t k = b * a.D * a.N + i;
                if (ck > 0) h[e][s] = wstate[(b * (nch - 1) + ck - 1) * a.D * a.N + i];
                else if (a.init) h[e][s] = a.state_bf16 ? to_f32(((const bf16*)a.init)[k]) : ((const float*)a.init)[k];
            }
        }

    const int64_t tok0 = b * a.L;
    const int vt = tid / V, vc = (tid % V) * 8;                 // this thread's first token and its channels
    const bool vok = vc < nc;
    float bias[8], Dv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) bias[j] = Dv[j] = 0.f;
    if (vok) {
        if (a.dt_bias) load8(a.dt_bias + d0 + vc, bias);
        if (!SUMMARY && a.Dv) load8(a.Dv + d0 + vc, Dv);
    }
    Raw8<IoT> rx[IT], rdt[IT], rb[IB], rz[IT], nx[IT];

    // raw x, dt, B, C of the tile at t0; tokens before the sequence's first and past the run are absent
    auto load = [&](int64_t t0) {
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int t = vt + q * (THREADS / V);
            const int64_t tt = t0 + t;
            nx[q].zero();
            rdt[q].zero();
            if (vok && t < T && tt >= p && tt < te) {
                nx[q].load((const IoT*)a.x + (tok0 + tt) * a.D + d0 + vc);
                rdt[q].load((const IoT*)a.dt_raw + (tok0 + tt) * a.D + d0 + vc);
            }
        }
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            int i = tid + q * THREADS;
            const bool second = !SUMMARY && i >= BN;
            i -= second ? BN : 0;
            const int t = i / (Np / 8), n = (i % (Np / 8)) * 8;
            const int64_t tt = t0 + t;
            rb[q].zero();
            if (i < BN && n < a.N && tt >= p && tt < te)
                rb[q].load((const IoT*)(second ? a.C : a.B) + ((tok0 + tt) * a.G + g) * a.N + n);
        }
    };
    auto stage = [&](int64_t t0, int buf) {
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int t = vt + q * (THREADS / V);
            if (t >= T) continue;
            const int64_t tt = t0 + t;
            float x[8], dt[8];
            nx[q].get(x);
            rdt[q].get(dt);
            const bool live = vok && tt >= p && tt < te;
#pragma unroll
            for (int j = 0; j < 8; ++j) dt[j] = live ? softplus_poly(dt[j] + bias[j]) : 0.f;
            // pair k lies at k ^ (k >> 3): 8 threads' vectors, 4 pairs apart, then meet all banks
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = vc / 2 + j;
                sd[(buf * T + t) * (CT / 2) + (k ^ ((k >> 3) & 7))] =
                    make_float4(dt[2 * j], dt[2 * j + 1], dt[2 * j] * x[2 * j], dt[2 * j + 1] * x[2 * j + 1]);
            }
        }
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            int i = tid + q * THREADS;
            const bool second = !SUMMARY && i >= BN;
            i -= second ? BN : 0;
            if (i >= BN) continue;
            float v[8];
            rb[q].get(v);
            store8((second ? sC : sB) + buf * T * Np + i * 8, v);
        }
    };

    if (tb < te) {
        load(tb);
        stage(tb, 0);
        __syncthreads();
    }
    int buf = 0;
    for (int64_t t0 = tb; t0 < te; t0 += T, buf ^= 1) {
#pragma unroll
        for (int q = 0; q < IT; ++q) rx[q] = nx[q];
        if (!SUMMARY && a.z) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int t = vt + q * (THREADS / V);
                rz[q].zero();
                if (vok && t < T && t0 + t >= p && t0 + t < te)
                    rz[q].load((const IoT*)a.z + (tok0 + t0 + t) * a.zs + d0 + vc);
            }
        }
        if (t0 + T < te) load(t0 + T);
        // tokens past the end have dt = 0 and leave the state alone
        const int nt = te - t0 < T ? (int)(te - t0) : T;
        const float4* pd = sd + buf * T * (CT / 2) + slot;
        const float *pB = sB + buf * T * Np + n0, *pC = sC + buf * T * Np + n0;
        for (int t = 0; t < nt; t += 4) {
            float y[8];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const float4 d = pd[(t + u) * (CT / 2)];
                float B[S], C[S];
#pragma unroll
                for (int s = 0; s < S; s += 4) {
                    Vec16<float>::load(pB + (t + u) * Np + s, B + s);
                    if (!SUMMARY) Vec16<float>::load(pC + (t + u) * Np + s, C + s);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float dt = e ? d.y : d.x, dx = e ? d.w : d.z;
                    float ys = 0.f;
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        h[e][s] = fmaf(exp2_approx(dt * A2[e][s]), h[e][s], dx * B[s]);
                        if (!SUMMARY) ys = fmaf(C[s], h[e][s], ys);
                    }
                    y[u * 2 + e] = ys;
                    if (SUMMARY) sum[e] += dt;
                }
            }
            if constexpr (!SUMMARY) {
                // lane group 8 / K values further: value 2 u + e is token u, channel e
                const int first = sum_over_states<K>(y, lane);
                float* out = sy + (t + first / 2) * YS + ch;
                if constexpr (K == 1) {
#pragma unroll
                    for (int u = 0; u < 4; ++u) *(float2*)(out + u * YS) = make_float2(y[2 * u], y[2 * u + 1]);
                } else if constexpr (K == 2) {
                    *(float2*)out = make_float2(y[0], y[1]);
                    *(float2*)(out + YS) = make_float2(y[2], y[3]);
                } else if constexpr (K == 4) {
                    *(float2*)out = make_float2(y[0], y[1]);
                } else {
                    if (lane < 8 * P) out[first & 1] = y[0];
                }
            }
        }
        __syncthreads();                                        // sy is complete, this tile's buffer free
        if constexpr (!SUMMARY) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int t = vt + q * (THREADS / V);
                const int64_t tt = t0 + t;
                if (!vok || t >= T || tt >= te) continue;
                float x[8], y[8];
                rx[q].get(x);
                load8(sy + t * YS + vc, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(Dv[j], x[j], y[j]);
                if (a.z) {
                    float z[8];
                    rz[q].get(z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= z[j] * sigmoid_f32(z[j]);
                }
                if (tt < p)
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = 0.f;
                store8((YT*)a.y + (tok0 + tt) * a.D + d0 + vc, y);
            }
        }
        if (t0 + T < te) stage(t0 + T, buf ^ 1);
        __syncthreads();                                        // the next tile is ready, sy free
    }
    if (SUMMARY) {
        const int64_t bc = b * nch + ck;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (ch + e >= nc) continue;
            if (n0 == 0) wdt[bc * a.D + d0 + ch + e] = sum[e];
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (n0 + s < a.N) wstate[(bc * a.D + d0 + ch + e) * a.N + n0 + s] = h[e][s];
        }
    } else if (a.final_state && ck == nch - 1) {
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

// wstate[b][c]: from the end state of chunk c started at 0 to the state that
// leaves it, c < nch - 1
__global__ void __launch_bounds__(128)
selective_chunks_kernel(const SelectiveArgs a, int nch, float* __restrict__ wstate, const float* __restrict__ wdt) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, DN = a.D * a.N;
    if (i >= a.batch * DN) return;
    const int64_t b = i / DN, dn = i % DN, d = dn / a.N;
    const float A2 = a.A[dn] * kLog2e;
    float h = 0.f;
    if (a.init) h = a.state_bf16 ? to_f32(((const bf16*)a.init)[i]) : ((const float*)a.init)[i];
    float* w = wstate + b * (nch - 1) * DN + dn;
    const float* dt = wdt + b * (nch - 1) * a.D + d;
    for (int c = 0; c < nch - 1; ++c) {
        h = fmaf(exp2_approx(dt[c * a.D] * A2), h, w[c * DN]);
        w[c * DN] = h;
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

// Tiles by the number of states: 4 states a lane (8 beyond 128), and more warps a
// block where a warp covers few channels, so that a token's row stays whole vectors.
constexpr int kSelMaxChunks = 64;

static int tile_channels(int64_t N) { return N <= 8 ? 128 : N <= 16 ? 64 : N <= 32 ? 32 : N <= 64 ? 32 : 16; }
static int tile_tokens(int64_t N) { return N > 128 ? 16 : 32; }

// A block's warps each keep one of the SM's four special function units busy, two
// blocks an SM saturate them.  Cutting the sequence costs a second exponential per
// state and token, so it pays once four or more chunks run in the time of one:
// from 60 blocks down (1 x 16384 tokens, 2048 channels, state 16: 32 blocks, see
// the launch below for its times).
static SelShape sel_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    SelShape sh{};
    const int CT = tile_channels(N), T = tile_tokens(N);
    sh.Dg = (int)(D / G);
    sh.tiles = (sh.Dg + CT - 1) / CT;
    const int64_t blocks = batch * G * sh.tiles, ntile = (L + T - 1) / T;
    int64_t nch = 1;
    if (blocks > 0 && blocks <= 60) nch = 296 / blocks;
    if (nch > kSelMaxChunks) nch = kSelMaxChunks;
    if (nch > ntile / 2) nch = ntile / 2;
    if (nch < 4) nch = 1;
    const int64_t per = nch > 1 ? (ntile + nch - 1) / nch : (ntile ? ntile : 1);
    sh.clen = (int)(per * T);
    sh.nch = (int)(nch > 1 ? (ntile + per - 1) / per : 1);
    return sh;
}

static size_t chunk_state_bytes(int64_t batch, int64_t D, int64_t N, int nch) {
    return ((size_t)batch * (nch - 1) * D * N * sizeof(float) + 255) & ~(size_t)255;
}

size_t selective_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    const SelShape sh = sel_shape(batch, L, D, N, G);
    if (sh.nch == 1) return 0;
    return chunk_state_bytes(batch, D, N, sh.nch) + (size_t)batch * (sh.nch - 1) * D * sizeof(float);
}

int64_t selective_blocks(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t) {
    return batch * (L / 8 + 1) * (D / 8) * ((N + 15) / 16);
}

template <typename IoT, typename YT, class Tile, int T>
static cudaError_t launch_fwd_t(const SelectiveArgs& a, cudaStream_t s) {
    constexpr int CT = Tile::CT, Np = Tile::Np, THREADS = Tile::W * 32;
    const SelShape sh = sel_shape(a.batch, a.L, a.D, a.N, a.G);
    constexpr int YS = CT % 32 == 0 ? CT + 16 : CT;
    constexpr int smem = (int)sizeof(float) * T * (4 * CT + 4 * Np + YS), smem1 = (int)sizeof(float) * T * (4 * CT + 2 * Np);
    const auto main = selective_fwd_kernel<IoT, YT, Tile, T, false>;
    const auto summary = selective_fwd_kernel<IoT, YT, Tile, T, true>;
    cudaError_t e = cudaSuccess;
    if (smem > 48 * 1024) e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess && smem1 > 48 * 1024)
        e = cudaFuncSetAttribute(summary, cudaFuncAttributeMaxDynamicSharedMemorySize, smem1);
    if (e != cudaSuccess) return e;
    float* wstate = (float*)a.ws;
    float* wdt = (float*)(a.ws + chunk_state_bytes(a.batch, a.D, a.N, sh.nch));
    const int64_t blocks = a.batch * a.G * sh.tiles;
    if (sh.nch > 1) {
        summary<<<(unsigned)(blocks * (sh.nch - 1)), THREADS, smem1, s>>>(a, sh, wstate, wdt);
        selective_chunks_kernel<<<(unsigned)((a.batch * a.D * a.N + 127) / 128), 128, 0, s>>>(a, sh.nch, wstate, wdt);
    }
    main<<<(unsigned)(blocks * sh.nch), THREADS, smem, s>>>(a, sh, wstate, wdt);
    return cudaGetLastError();
}

template <typename IoT, typename YT>
static cudaError_t launch_fwd_s(const SelectiveArgs& a, cudaStream_t s) {
    if (a.N <= 8) return launch_fwd_t<IoT, YT, SelTile<2, 4, 4>, 32>(a, s);
    if (a.N <= 16) return launch_fwd_t<IoT, YT, SelTile<4, 4, 4>, 32>(a, s);
    if (a.N <= 32) return launch_fwd_t<IoT, YT, SelTile<8, 4, 4>, 32>(a, s);
    if (a.N <= 64) return launch_fwd_t<IoT, YT, SelTile<16, 4, 8>, 32>(a, s);
    if (a.N <= 128) return launch_fwd_t<IoT, YT, SelTile<32, 4, 8>, 32>(a, s);
    return launch_fwd_t<IoT, YT, SelTile<32, 8, 8>, 16>(a, s);
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
