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
//
// Measured, bf16, gated, state 16, a B200: 4 x 2048 tokens x 4096 channels 234 us
// (the states' exponentials alone 119 us), 1 x 16384 x 2048 374 us; a token of
// 256 sequences x 8192 channels over an fp32 state 54 us (5290 GB/s of 6568).
#include "ssd_selective_common.cuh"

namespace ssd {

// A block owns CT channels of a group and walks over a run of tokens in tiles of
// T.  A tile's raw inputs are loaded while the tile before is computed; dt and
// dt x are formed once per token and channel into shared memory, B and C widened
// beside them (two buffers); each warp then walks over the tile on its own
// channels, and the block gates and stores the tile's y with whole vectors.
//
// Where batch and channels are too few for the machine the sequence is cut into
// nch chunks and takes two launches of nch - 1 of them: the first walks over chunk 0
// and, for each of the others but the last, finds its end state from 0 and the sum
// of its dt (SUMMARY); selective_chunks_kernel forms the state that enters each; the
// second launch walks over chunks 1 to nch - 1.
template <typename IoT, typename YT, class Tile, int T, bool SUMMARY, bool DEEP>
__device__ __forceinline__ void selective_walk(const SelectiveArgs& a, const SelShape& sh, int tile, int64_t g, int64_t ck,
                                               int64_t b, float* __restrict__ wstate, float* __restrict__ wdt) {
    constexpr int K = Tile::K, S = Tile::S, Np = Tile::Np, P = Tile::P, CT = Tile::CT, THREADS = Tile::W * 32;
    constexpr int V = CT / 8;                                   // 8-channel vectors of a token here
    constexpr int IT = (T * V + THREADS - 1) / THREADS;         // of a thread in a tile
    constexpr int BN = T * Np / 8;                              // 8-state vectors of a tile's B
    constexpr int IB = ((SUMMARY ? 1 : 2) * BN + THREADS - 1) / THREADS;
    constexpr int YS = CT + 4;                                  // row of y: 8 tokens' values meet all banks
    extern __shared__ float4 smem4[];
    float4* sd = smem4;                                         // [2][T][CT / 2]: (dt, dt x) of two channels
    float* sB = (float*)(sd + 2 * T * (CT / 2));                // [2][T][Np]
    float* sC = sB + 2 * T * Np;                                // [2][T][Np]
    float* sy = sC + (SUMMARY ? 0 : 2 * T * Np);                // [8 + T][YS]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t nch = sh.nch;
    const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;   // channels of the group here
    const int64_t d0 = g * sh.Dg + c0;
    const int64_t tb = ck == 0 ? 0 : sh.len0 + (ck - 1) * sh.clen, to = ck == 0 ? sh.len0 : tb + sh.clen;
    const int64_t te = to < a.L ? to : a.L;
    int64_t p = a.pad_left ? a.pad_left[b] : 0;
    p = p < 0 ? 0 : p > a.L ? a.L : p;

    const int ch = warp * P + lane % P, n0 = (lane / P) * S;
    const bool cok = ch < nc;
    const int slot = (ch >> 1) ^ ((ch >> 4) & 7);               // where its pair lies in a row of sd (see stage)
    f32x2 A2[S / 2], h[S / 2];                                  // states s, s + 1
    float sum = 0.f;
#pragma unroll
    for (int s2 = 0; s2 < S / 2; ++s2) {
        float Av[2] = {0.f, 0.f}, hv[2] = {0.f, 0.f};
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int s = 2 * s2 + q;
            const int64_t i = (d0 + ch) * a.N + n0 + s;
            if (cok && n0 + s < a.N) {
                Av[q] = decay_rate(a.A[i]);
                const int64_t k = b * a.D * a.N + i;
                if (SUMMARY) continue;
                if (ck > 0) hv[q] = wstate[(b * (nch - 1) + ck - 1) * a.D * a.N + i];
                else if (a.init) hv[q] = a.state_bf16 ? to_f32(((const bf16*)a.init)[k]) : ((const float*)a.init)[k];
            }
        }
        A2[s2] = f2_pack(Av[0], Av[1]);
        h[s2] = f2_pack(hv[0], hv[1]);
    }

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

    // addresses of this thread's first token; a tile's tokens of it are STEP apart
    constexpr int STEP = THREADS / V;
    const int64_t tok = b * a.L + tb + vt;
    const IoT* px = (const IoT*)a.x + tok * a.D + d0 + vc;
    const IoT* pdt = (const IoT*)a.dt_raw + tok * a.D + d0 + vc;
    const IoT* pz = (const IoT*)a.z + tok * a.zs + d0 + vc;
    YT* py = (YT*)a.y + tok * a.D + d0 + vc;
    // and of its vectors of B and C (the halves of a tile's 2 BN vectors)
    const IoT* pbc[IB];
    int bct[IB];                                                // token in the tile, or out of every run
#pragma unroll
    for (int q = 0; q < IB; ++q) {
        int i = tid + q * THREADS;
        const bool second = !SUMMARY && i >= BN;
        i -= second ? BN : 0;
        const int t = i / (Np / 8), n = (i % (Np / 8)) * 8;
        bct[q] = i < BN && n < a.N ? t : 1 << 30;
        pbc[q] = (const IoT*)(second ? a.C : a.B) + ((b * a.L + tb + t) * a.G + g) * a.N + n;
    }

    // raw x, dt, B, C of the tile that starts `at` tokens into the run; absent tokens (padding, or past
    // the run) get x = 0 and dt_raw = -inf, so dt = 0
    const int len = (int)(te - tb), lead = p <= tb ? 0 : p - tb < len ? (int)(p - tb) : len;
    auto load = [&](int at) {
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int t = vt + q * STEP;
            nx[q].zero();
            rdt[q].minus_inf();
            if (vok && t < T && at + t >= lead && at + t < len) {
                nx[q].load(px + (int64_t)(at + q * STEP) * a.D);
                rdt[q].load(pdt + (int64_t)(at + q * STEP) * a.D);
            }
        }
#pragma unroll
        for (int q = 0; q < IB; ++q) {
            rb[q].zero();
            if (at + bct[q] >= lead && at + bct[q] < len) rb[q].load(pbc[q] + (int64_t)at * (a.G * a.N));
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int t = vt + q * STEP;
            if (t >= T) continue;
            float x[8], z[8];
            nx[q].get(x);
            rdt[q].get(z);
            // pair k lies at k ^ (k >> 3): 8 threads' vectors, 4 pairs apart, then meet all banks
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = vc / 2 + j;
                const float2 dt = f2_get(softplus2(z[2 * j] + bias[2 * j], z[2 * j + 1] + bias[2 * j + 1]));
                sd[(buf * T + t) * (CT / 2) + (k ^ ((k >> 3) & 7))] =
                    make_float4(dt.x, dt.x * x[2 * j], dt.y, dt.y * x[2 * j + 1]);
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

    if (len > 0) {
        load(0);
        stage(0);
        __syncthreads();
    }
    int buf = 0;
    for (int at = 0; at < len; at += T, buf ^= 1) {
#pragma unroll
        for (int q = 0; q < IT; ++q) rx[q] = nx[q];
        if (!SUMMARY && a.z) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int t = vt + q * STEP;
                rz[q].zero();
                if (vok && t < T && at + t >= lead && at + t < len) rz[q].load(pz + (int64_t)(at + q * STEP) * a.zs);
            }
        }
        if (at + T < len) load(at + T);
        // tokens past the end have dt = 0 and leave the state alone
        const int nt = len - at < T ? len - at : T;
        const float2* pd = (const float2*)(sd + buf * T * (CT / 2) + slot) + (ch & 1);
        const float *pB = sB + buf * T * Np + n0, *pC = sC + buf * T * Np + n0;
        // 8 tokens a round; the sums over the states of a round are formed in the next one, beside its
        // exponentials (the first round's stand-in goes to the 8 rows before the tile's)
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = 0.f;
        auto reduce = [&](int t) {
            const int first = sum_over_states<K>(y, lane);
            float* out = sy + (t + 8 + first) * YS + ch;
            if (K > 8 && lane >= 8 * P) return;
#pragma unroll
            for (int i = 0; i < (K >= 8 ? 1 : 8 / K); ++i) out[i * YS] = y[i];
        };
#pragma unroll DEEP ? 2 : 1
        for (int t = 0; t < nt; t += 8) {
            float yn[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const float2 d = pd[(t + u) * CT];
                f32x2 B[S / 2], C[S / 2];
                f2_load<S>(pB + (t + u) * Np, B);
                if (!SUMMARY) f2_load<S>(pC + (t + u) * Np, C);
                const f32x2 dt = f2_pack(d.x, d.x), dx = f2_pack(d.y, d.y);
                f32x2 ys = 0;
#pragma unroll
                for (int s = 0; s < S / 2; ++s) {
                    h[s] = f2_fma(f2_exp2(f2_mul(dt, A2[s])), h[s], f2_mul(dx, B[s]));
                    if (!SUMMARY) ys = s ? f2_fma(C[s], h[s], ys) : f2_mul(C[s], h[s]);
                }
                const float2 yy = f2_get(ys);
                yn[u] = yy.x + yy.y;
                if (SUMMARY) sum += d.x;
            }
            if constexpr (!SUMMARY) {
                reduce(t - 8);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = yn[i];
            }
        }
        if constexpr (!SUMMARY) reduce((nt - 1) & ~7);
        __syncthreads();                                        // sy is complete, this tile's buffer free
        if constexpr (!SUMMARY) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int t = vt + q * STEP;
                if (!vok || t >= T || at + t >= len) continue;
                float x[8], y[8];
                rx[q].get(x);
                load8(sy + (t + 8) * YS + vc, y);
#pragma unroll
                for (int j = 0; j < 8; ++j) y[j] = fmaf(Dv[j], x[j], y[j]);
                if (a.z) {
                    float z[8];
                    rz[q].get(z);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] *= z[j] * sigmoid_f32(z[j]);
                }
                if (at < lead && at + t < lead) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = 0.f;
                }
                store8(py + (int64_t)(at + q * STEP) * a.D, y);
            }
        }
        if (at + T < len) stage(buf ^ 1);
        __syncthreads();                                        // the next tile is ready, sy free
    }
    if (!cok) return;
    // what leaves a summary, or chunk 0, goes to the workspace
    const int64_t bc = b * (nch - 1) + ck;
    const bool keep = SUMMARY || ck < nch - 1;
    if (SUMMARY && n0 == 0) wdt[bc * a.D + d0 + ch] = sum;
    if (keep ? ck > 0 && !SUMMARY : !a.final_state) return;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (n0 + s >= a.N) continue;
        const float2 hv = f2_get(h[s / 2]);
        const float v = s & 1 ? hv.y : hv.x;
        const int64_t i = (d0 + ch) * a.N + n0 + s;
        if (keep) wstate[bc * a.D * a.N + i] = v;
        else if (a.state_bf16) ((bf16*)a.final_state)[b * a.D * a.N + i] = from_f32<bf16>(v);
        else ((float*)a.final_state)[b * a.D * a.N + i] = v;
    }
}

// DEEP: for blocks of 4 warps of which an SM has two at most, registers for two
// rounds side by side (4 x 2048 x 4096: 245 us with one round in the registers of
// three blocks an SM, 248 us with two rounds in them, 232 us with two in those of two)
template <typename IoT, typename YT, class Tile, int T, bool FIRST, bool DEEP>
__global__ void __launch_bounds__(Tile::W * 32, Tile::W == 4 && !DEEP ? 3 : Tile::W <= 8 ? 2 : 1)
selective_fwd_kernel(const SelectiveArgs a, const SelShape sh, float* __restrict__ wstate, float* __restrict__ wdt) {
    const int64_t here = sh.nch > 1 ? sh.nch - 1 : 1;            // chunks of this launch
    int64_t r = blockIdx.x;
    const int tile = (int)(r % sh.tiles);
    r /= sh.tiles;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % here + (FIRST || sh.nch == 1 ? 0 : 1), b = r / here;
    if constexpr (FIRST) {
        if (ck > 0) {
            selective_walk<IoT, YT, Tile, T, true, DEEP>(a, sh, tile, g, ck, b, wstate, wdt);
            return;
        }
    }
    selective_walk<IoT, YT, Tile, T, false, DEEP>(a, sh, tile, g, ck, b, wstate, wdt);
}

// wstate[b][c]: from the end state of chunk c started at 0 to the state that
// leaves it, 0 < c < nch - 1 (chunk 0's is there)
__global__ void __launch_bounds__(128)
selective_chunks_kernel(const SelectiveArgs a, int nch, float* __restrict__ wstate, const float* __restrict__ wdt) {
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x, DN = a.D * a.N;
    if (i >= a.batch * DN) return;
    const int64_t b = i / DN, dn = i % DN, d = dn / a.N;
    const float A2 = decay_rate(a.A[dn]);
    float* w = wstate + b * (nch - 1) * DN + dn;
    const float* dt = wdt + b * (nch - 1) * a.D + d;
    float h = w[0];
#pragma unroll 4
    for (int c = 1; c < nch - 1; ++c) {
        h = fmaf(exp2_approx(dt[c * a.D] * A2), h, w[c * DN]);
        w[c * DN] = h;
    }
}

// One token: a stream of the states, each read and written once with 16-byte
// vectors.  K lanes cover a channel's states (R rounds of a vector each) for NB <= K
// sequences of the batch, whose loads are all in flight before the first is used:
// A is fetched once for NB states.  Of a channel's scalars lane u of the K takes
// sequence u's: it loads x, dt_raw and z, forms dt and the gate, passes dt and dt x
// to the others and stores sequence u's y.
template <typename StateT, typename IoT, typename YT, int R, int NB>
__global__ void __launch_bounds__(128)
selective_update_kernel(const SelectiveArgs a, int K, int cblocks, int Dg) {
    constexpr int VS = Vec16<StateT>::N;
    const int lane = threadIdx.x % K, slot = threadIdx.x / K;
    const int d = (int)(blockIdx.x % (unsigned)cblocks) * (128 / K) + slot;
    const int b0 = (int)(blockIdx.x / (unsigned)cblocks) * NB;
    const int nb = d >= a.D ? 0 : a.batch - b0 < NB ? (int)(a.batch - b0) : NB;   // every lane takes part in the sums
    const int N = (int)a.N;
    StateT* hp = (StateT*)a.final_state + (b0 * a.D + d) * N;
    const IoT* pb = (const IoT*)a.B + ((int64_t)b0 * a.G + d / Dg) * N;
    const IoT* pc = (const IoT*)a.C + ((int64_t)b0 * a.G + d / Dg) * N;
    const int64_t hstep = a.D * N, bstep = a.G * N;
    uint4 hr[NB][R];
    Raw4<IoT> Br[NB][R][VS / 4], Cr[NB][R][VS / 4];
#pragma unroll
    for (int u = 0; u < NB; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int n = (lane + r * K) * VS;
            hr[u][r] = make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int q = 0; q < VS / 4; ++q) {
                Br[u][r][q].zero();
                Cr[u][r][q].zero();
            }
            if (u < nb && n < N) {
                hr[u][r] = __ldcs((const uint4*)(hp + u * hstep + n));
#pragma unroll
                for (int q = 0; q < VS / 4; ++q) {
                    Br[u][r][q].load(pb + u * bstep + n + 4 * q);
                    Cr[u][r][q].load(pc + u * bstep + n + 4 * q);
                }
            }
        }
    const int own = lane % NB;
    const int64_t at = (int64_t)(b0 + own) * a.D + d;
    float x = 0.f, raw = 0.f, z = 0.f, bias = 0.f, Dv = 0.f;
    if (own < nb) {
        x = to_f32(((const IoT*)a.x)[at]);
        raw = to_f32(((const IoT*)a.dt_raw)[at]);
        if (a.z) z = to_f32(((const IoT*)a.z)[(b0 + own) * a.zs + d]);
        if (a.dt_bias) bias = a.dt_bias[d];
        if (a.Dv) Dv = a.Dv[d];
    }
    float A2[R][VS];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = (lane + r * K) * VS;
#pragma unroll
        for (int s = 0; s < VS; ++s) A2[r][s] = 0.f;
        if (nb > 0 && n < N)
#pragma unroll
            for (int s = 0; s < VS; s += 4) {
                Vec16<float>::load(a.A + (int64_t)d * N + n + s, A2[r] + s);
#pragma unroll
                for (int q = 0; q < 4; ++q) A2[r][s + q] = decay_rate(A2[r][s + q]);
            }
    }
    const float dt = f2_get(softplus2(raw + bias, raw + bias)).x, dx = dt * x;
    float mine = 0.f;
#pragma unroll
    for (int u = 0; u < NB; ++u) {
        const int from = (int)(threadIdx.x & 31) - lane + u;          // the lane of this channel that has sequence u
        const float dtu = __shfl_sync(0xffffffffu, dt, from), dxu = __shfl_sync(0xffffffffu, dx, from);
        float y = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int n = (lane + r * K) * VS;
            float h[VS], B[VS], C[VS];
            Vec16<StateT>::unpack(hr[u][r], h);
#pragma unroll
            for (int q = 0; q < VS / 4; ++q) {
                Br[u][r][q].get(B + 4 * q);
                Cr[u][r][q].get(C + 4 * q);
            }
#pragma unroll
            for (int s = 0; s < VS; ++s) {
                h[s] = fmaf(exp2_approx(dtu * A2[r][s]), h[s], dxu * B[s]);
                y = fmaf(C[s], h[s], y);
            }
            if (u < nb && n < N) __stcs((uint4*)(hp + u * hstep + n), Vec16<StateT>::pack(h));
        }
        for (int o = 1; o < K; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
        if (own == u) mine = y;
    }
    if (lane < nb) {
        mine = fmaf(Dv, x, mine);
        if (a.z) mine *= z * sigmoid_f32(z);
        ((YT*)a.y)[at] = from_f32<YT>(mine);
    }
}

// Tiles by the number of states: 8 states a lane from 9 to 32 states and beyond 128
// (half the loads and sums of 4 for each state: 246 against 251 us at 4 x 2048 x
// 4096, state 16, with half the warps), 4 otherwise; more warps a block where a warp
// covers few channels, so that a token's row stays whole vectors.  Of 33 to 128 states
// 4 a lane is the slower side, at 4 x 2048 tokens x 2048 channels, bf16, gated: 64
// states 443 us against 425 with 8 a lane and half the warps, 128 states 1039 us
// against 855.  8 states 200 us (4096 channels), 256 states 1438 us (2 x 2048 x 2048).
constexpr int kSelMaxChunks = 64;

static int tile_channels(int64_t N) { return N <= 8 ? 128 : N <= 16 ? 64 : N <= 32 ? 32 : 16; }
static int tile_tokens(int64_t N) { return N > 128 ? 16 : 32; }

// Cutting the sequence costs a second exponential per state and token, and pays while
// there are blocks for two SMs in three at most: from 100 blocks down, into as many
// chunks as make three blocks an SM.  Cut against whole, bf16, gated, state 16:
// 1 x 16384 tokens, 32 blocks 372 and 1179 us; 1 x 4096 tokens, 64 blocks 192 and 299
// us, 80 blocks 228 and 299, 100 blocks 267 and 299, 128 blocks 334 and 300.  Four
// chunks (three a launch) at least: 1 x 256 tokens, 32 blocks, 22.9 and 22.7 us in
// four, 1 x 512 tokens 28.5 and 41.0 us in eight; a short sequence of many channels
// loses by it (1 x 320 tokens, 100 blocks: 36.7 and 27.6 us).  3 x 777 x 520 fp32,
// state 24: 38 and 52 us.
static SelShape sel_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    SelShape sh{};
    const int CT = tile_channels(N), T = tile_tokens(N);
    sh.Dg = (int)(D / G);
    sh.tiles = (sh.Dg + CT - 1) / CT;
    const int64_t blocks = batch * G * sh.tiles, ntile = (L + T - 1) / T;
    int64_t nch = 1;
    if (blocks > 0 && blocks <= 100) nch = 444 / blocks + 1;
    if (nch > kSelMaxChunks) nch = kSelMaxChunks;
    if (nch > ntile / 2) nch = ntile / 2;
    if (nch < 4) {
        sh.nch = 1;
        sh.len0 = sh.clen = (int)((ntile ? ntile : 1) * T);
        return sh;
    }
    // chunk 0, walked over in full while the others are summed up, has three quarters of their tiles: a
    // summary's tile takes that much of a full one's time
    int64_t per = (ntile + nch - 1) / nch;
    while (3 * per / 4 + (nch - 1) * per < ntile) ++per;
    const int64_t per0 = 3 * per / 4 > 0 ? 3 * per / 4 : 1;
    sh.len0 = (int)(per0 * T);
    sh.clen = (int)(per * T);
    sh.nch = (int)(1 + (ntile - per0 + per - 1) / per);
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

int64_t selective_blocks(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    const SelShape sh = sel_shape(batch, L, D, N, G);
    const int64_t walk = batch * G * sh.tiles * (sh.nch > 1 ? sh.nch - 1 : 1);
    const int64_t join = sh.nch > 1 ? (batch * D * N + 127) / 128 : 0, token = batch * ((D + 3) / 4);   // K <= 32
    return walk > join ? (walk > token ? walk : token) : (join > token ? join : token);
}

template <typename IoT, typename YT, class Tile, int T>
static cudaError_t launch_fwd_t(const SelectiveArgs& a, cudaStream_t s) {
    constexpr int CT = Tile::CT, Np = Tile::Np, THREADS = Tile::W * 32;
    const SelShape sh = sel_shape(a.batch, a.L, a.D, a.N, a.G);
    constexpr int YS = CT + 4;
    constexpr int smem = (int)sizeof(float) * (T * (4 * CT + 4 * Np + YS) + 8 * YS);
    const unsigned grid = (unsigned)(a.batch * a.G * sh.tiles * (sh.nch > 1 ? sh.nch - 1 : 1));
    const bool deep = Tile::W == 4 && sh.nch == 1 && grid <= 296;
    const auto main = deep ? selective_fwd_kernel<IoT, YT, Tile, T, false, Tile::W == 4>
                           : selective_fwd_kernel<IoT, YT, Tile, T, false, false>;
    const auto first = selective_fwd_kernel<IoT, YT, Tile, T, true, false>;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e == cudaSuccess) e = cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    float* wstate = (float*)a.ws;
    float* wdt = (float*)(a.ws + chunk_state_bytes(a.batch, a.D, a.N, sh.nch));
    if (sh.nch > 1) {
        first<<<grid, THREADS, smem, s>>>(a, sh, wstate, wdt);
        selective_chunks_kernel<<<(unsigned)((a.batch * a.D * a.N + 127) / 128), 128, 0, s>>>(a, sh.nch, wstate, wdt);
    }
    main<<<grid, THREADS, smem, s>>>(a, sh, wstate, wdt);
    return cudaGetLastError();
}

template <typename IoT, typename YT>
static cudaError_t launch_fwd_s(const SelectiveArgs& a, cudaStream_t s) {
    if (a.N <= 8) return launch_fwd_t<IoT, YT, SelTile<2, 4, 8>, 32>(a, s);
    if (a.N <= 16) return launch_fwd_t<IoT, YT, SelTile<2, 8, 4>, 32>(a, s);
    if (a.N <= 32) return launch_fwd_t<IoT, YT, SelTile<4, 8, 4>, 32>(a, s);
    if (a.N <= 64) return launch_fwd_t<IoT, YT, SelTile<16, 4, 8>, 32>(a, s);
    if (a.N <= 128) return launch_fwd_t<IoT, YT, SelTile<32, 4, 16>, 32>(a, s);
    return launch_fwd_t<IoT, YT, SelTile<32, 8, 16>, 16>(a, s);
}

cudaError_t launch_selective_fwd(const SelectiveArgs& a, cudaStream_t s) {
    if (a.io_bf16) return a.y_bf16 ? launch_fwd_s<bf16, bf16>(a, s) : launch_fwd_s<bf16, float>(a, s);
    return a.y_bf16 ? launch_fwd_s<float, bf16>(a, s) : launch_fwd_s<float, float>(a, s);
}

template <typename StateT, typename IoT, typename YT, int R>
static void launch_update_r(const SelectiveArgs& a, int K, cudaStream_t s) {
    const int cblocks = (int)((a.D + 128 / K - 1) / (128 / K)), Dg = (int)(a.D / a.G);
    // as many sequences a thread as lanes, up to 4, once that still leaves 1024 threads an SM
    const int64_t quads = (a.batch + 3) / 4 * cblocks, twos = (a.batch + 1) / 2 * cblocks;
    if (R == 1 && K >= 4 && quads >= 148 * 8)
        selective_update_kernel<StateT, IoT, YT, R, R == 1 ? 4 : 1><<<(unsigned)quads, 128, 0, s>>>(a, K, cblocks, Dg);
    else if (R == 1 && K >= 2 && twos >= 148 * 8)
        selective_update_kernel<StateT, IoT, YT, R, R == 1 ? 2 : 1><<<(unsigned)twos, 128, 0, s>>>(a, K, cblocks, Dg);
    else
        selective_update_kernel<StateT, IoT, YT, R, 1><<<(unsigned)(a.batch * cblocks), 128, 0, s>>>(a, K, cblocks, Dg);
}

template <typename StateT, typename IoT>
static void launch_update_t(const SelectiveArgs& a, cudaStream_t s) {
    constexpr int VS = Vec16<StateT>::N;
    int K = 1;
    while (K < 32 && K * VS < a.N) K *= 2;
    if (K * VS < a.N) {
        if (a.y_bf16) launch_update_r<StateT, IoT, bf16, 2>(a, K, s);
        else launch_update_r<StateT, IoT, float, 2>(a, K, s);
    } else {
        if (a.y_bf16) launch_update_r<StateT, IoT, bf16, 1>(a, K, s);
        else launch_update_r<StateT, IoT, float, 1>(a, K, s);
    }
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
