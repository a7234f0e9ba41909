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
//  3. per chunk: the states forward, every GT-th kept in shared memory, then the
//     adjoint back in groups of GT tokens, whose decays serve the group's states
//     and its adjoint.  A block goes over several tiles of channels and adds
//     their dB and dC up; blocks' sums are added in a fixed order last.
//
// Three exponentials for each state of each token and some 150 instructions for
// every four: bound by the instruction rate, shared memory and the exchanges of the
// sums, then the special function units.  Measured, 2 x 2048 tokens x 4096 channels,
// state 16, bf16, gated, a B200: 563 us (summaries 112, recombination 35, third step
// 415: 54 % of the issue slots, 62 % of the shared and exchange path).  Chunks of 16
// tokens instead of 32 take 697 us: the chunk states' traffic doubles.
#include "ssd_selective_common.cuh"

namespace ssd {

// A lane holds S states of 2 neighbouring channels, a warp 32 / K pairs of them: B
// and C are read for both at once, and half of the sums of dB and dC over the
// channels are formed in registers.
template <int K_, int S_, int T_, int GT_>
struct SbTile {
    static constexpr int K = K_;             // lanes of a channel
    static constexpr int S = S_;             // states of a lane
    static constexpr int T = T_;             // tokens of a chunk
    static constexpr int GT = GT_;           // tokens of a group of the way back
    static constexpr int W = 4;              // warps of a block
    static constexpr int THREADS = W * 32;
    static constexpr int Np = K * S;
    static constexpr int P = 32 / K;         // pairs of channels of a warp
    static constexpr int CT = W * P * 2;     // channels of a block
    static constexpr int YS = CT + 8;        // row of sy: 4 tokens' pairs meet all banks
    static constexpr int ACC = (T * Np + THREADS - 1) / THREADS;   // of the chunk's sums of dB (dC) a thread
    static constexpr int SMEM = (int)sizeof(float) * (T * CT * 3 + T * YS + (T / GT - 1) * 2 * S * THREADS +
                                                      2 * T * Np + W * T * Np);
};

struct SbShape {
    int Dg, tiles;               // channels of a group, tiles that cover them
    int nch;                     // chunks of a sequence
    int split;                   // blocks that share a chunk's tiles of channels
    size_t off_h, off_g;         // fp32 [b][nch][D][N] chunk states, then adjoints
    size_t off_dt;               // fp32 [b][nch][D] sum of dt
    size_t off_dA;               // fp32 [b][nch][D][N]
    size_t off_par;              // fp32 [b][nch][2][D]: d dt_bias, dD
    size_t off_dBC;              // fp32 [split][dB, dC][b][L][G][N]
    size_t total;
};

// Tokens of a chunk: as many as leave three blocks an SM their shared memory.  Beyond 32
// states, 2 x 2048 tokens x 2048 channels, bf16, gated: 64 states 1214 us (1208 with 32
// tokens and two blocks an SM), 128 states 2490 us (3182 with 8 tokens), and 256 states
// on 1024 channels 3249 us.
static int sb_tokens(int64_t N) { return N <= 8 ? 16 : N <= 32 ? 32 : N <= 128 ? 16 : 8; }
static int sb_channels(int64_t N) { return N <= 8 ? 128 : N <= 16 ? 64 : N <= 32 ? 32 : N <= 64 ? 16 : 8; }

static SbShape sb_shape(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    SbShape l{};
    const int T = sb_tokens(N), CT = sb_channels(N);
    l.Dg = (int)(D / G);
    l.tiles = (l.Dg + CT - 1) / CT;
    l.nch = (int)((L + T - 1) / T);
    // 3 blocks an SM; several rounds of them, so that the last one does not leave most SMs idle
    const int64_t chunks = batch * l.nch * G, want = 148 * 3 * 8;
    int64_t split = chunks ? (want + chunks - 1) / chunks : 1;
    if (split > l.tiles) split = l.tiles;
    l.split = (int)split;
    const auto up = [](size_t v) { return (v + 255) & ~(size_t)255; };
    const size_t bn = (size_t)batch * l.nch, st = bn * D * N * sizeof(float);
    l.off_h = 0;
    l.off_g = up(l.off_h + st);
    l.off_dt = up(l.off_g + st);
    l.off_dA = up(l.off_dt + bn * D * sizeof(float));
    l.off_par = up(l.off_dA + st);
    l.off_dBC = up(l.off_par + bn * 2 * D * sizeof(float));
    l.total = up(l.off_dBC + (size_t)l.split * 2 * batch * L * G * N * sizeof(float));
    return l;
}

size_t selective_bwd_workspace(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    return batch == 0 || L == 0 ? 0 : sb_shape(batch, L, D, N, G).total;
}

int64_t selective_bwd_blocks(int64_t batch, int64_t L, int64_t D, int64_t N, int64_t G) {
    const SbShape sh = sb_shape(batch, L, D, N, G);
    const int64_t walk = batch * sh.nch * G * sh.tiles, join = 2 * ((batch * D * N + 127) / 128);
    const int64_t sums = (2 * batch * L * G * N + 31) / 32 + (D * N + 31) / 32 + (2 * D + 31) / 32;
    return walk > join ? (walk > sums ? walk : sums) : (join > sums ? join : sums);
}

// B and C of a chunk in fp32, zero past the sequence
template <typename IoT, int T, int Np, int THREADS>
__device__ __forceinline__ void stage_bc(const SelectiveArgs& a, int64_t b, int64_t g, int64_t t0, int nt, float* sB,
                                         float* sC) {
    for (int i = threadIdx.x; i < 2 * T * Np / 8; i += THREADS) {
        const bool second = i >= T * Np / 8;
        const int k = (second ? i - T * Np / 8 : i) * 8, t = k / Np, n = k % Np;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.f;
        if (t < nt && n < a.N) load8((const IoT*)(second ? a.C : a.B) + ((b * a.L + t0 + t) * a.G + g) * a.N + n, v);
        store8((second ? sC : sB) + k, v);
    }
}

// 8 channels of a token as they lie in memory, and x, dt and g of them
template <typename IoT> struct TokenRaw {
    Raw8<IoT> x, dt, dy, z;
    __device__ __forceinline__ void load(const SelectiveArgs& a, int64_t tok, int64_t d) {
        x.load((const IoT*)a.x + tok * a.D + d);
        dt.load((const IoT*)a.dt_raw + tok * a.D + d);
        dy.load((const IoT*)a.dy + tok * a.D + d);
        if (a.z) z.load((const IoT*)a.z + tok * a.zs + d);
    }
    __device__ __forceinline__ void get(const SelectiveArgs& a, int64_t d, float (&xv)[8], float (&dtv)[8],
                                        float (&g)[8]) const {
        float raw[8], bias[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) bias[j] = 0.f;
        if (a.dt_bias) load8(a.dt_bias + d, bias);
        x.get(xv);
        dt.get(raw);
        dy.get(g);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 v = f2_get(softplus2(raw[j] + bias[j], raw[j + 1] + bias[j + 1]));
            dtv[j] = v.x;
            dtv[j + 1] = v.y;
        }
        if (a.z) {
            float zv[8];
            z.get(zv);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 v = f2_get(f2_mul(f2_pack(g[j], g[j + 1]), f2_silu(f2_pack(zv[j], zv[j + 1]))));
                g[j] = v.x;
                g[j + 1] = v.y;
            }
        }
    }
};

// The S floats of a lane's states n0 .. of row `i` of a matrix [..][N] (zero past N)
template <int S>
__device__ __forceinline__ void load_states(const float* p, int64_t i, int64_t N, int n0, bool ok, f32x2 (&v)[S / 2]) {
#pragma unroll
    for (int s = 0; s < S / 2; ++s) v[s] = 0;
    if (!ok) return;
#pragma unroll
    for (int s = 0; s < S; s += 4)
        if (n0 + s < N) {
            const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(p + i * N + n0 + s);
            v[s / 2] = r.x;
            v[s / 2 + 1] = r.y;
        }
}
template <int S>
__device__ __forceinline__ void store_states(float* p, int64_t i, int64_t N, int n0, bool ok, const f32x2 (&v)[S / 2]) {
    if (!ok) return;
#pragma unroll
    for (int s = 0; s < S; s += 4)
        if (n0 + s < N) *reinterpret_cast<ulonglong2*>(p + i * N + n0 + s) = make_ulonglong2(v[s / 2], v[s / 2 + 1]);
}
template <int S>
__device__ __forceinline__ void decay_rates(f32x2 (&v)[S / 2]) {
#pragma unroll
    for (int s = 0; s < S / 2; ++s) {
        const float2 A = f2_get(v[s]);
        v[s] = f2_pack(decay_rate(A.x), decay_rate(A.y));
    }
}

// Step 1.
template <typename IoT, class Tile>
__global__ void __launch_bounds__(Tile::THREADS)
selective_bwd_summary_kernel(const SelectiveArgs a, const SbShape sh) {
    constexpr int S = Tile::S, Np = Tile::Np, CT = Tile::CT, P = Tile::P, T = Tile::T, THREADS = Tile::THREADS, V = CT / 8;
    extern __shared__ float4 smem4[];
    float4* sd = smem4;                                  // [T][CT / 2]: dt, dt, dt x, dt x
    float2* sg = (float2*)(sd + T * (CT / 2));           // [T][CT / 2]: g, g
    float* sB = (float*)(sg + T * (CT / 2));
    float* sC = sB + T * Np;
    const int tile = (int)(blockIdx.x % (unsigned)sh.tiles);
    int64_t r = blockIdx.x / (unsigned)sh.tiles;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % sh.nch, b = r / sh.nch, t0 = ck * T, bc = b * sh.nch + ck;
    const int nt = a.L - t0 < T ? (int)(a.L - t0) : T;
    const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;
    const int64_t d0 = g * sh.Dg + c0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pair = warp * P + lane % P, n0 = (lane / P) * S, ch = pair * 2;
    const bool ok = ch < nc;
    f32x2 A2[2][S / 2], h[2][S / 2], Pr[2][S / 2], Gs[2][S / 2];
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        load_states<S>(a.A, d0 + ch + e, a.N, n0, ok, A2[e]);
        decay_rates<S>(A2[e]);
#pragma unroll
        for (int s = 0; s < S / 2; ++s) {
            h[e][s] = Gs[e][s] = 0;
            Pr[e][s] = f2_pack(1.f, 1.f);
        }
    }
    for (int i = threadIdx.x; i < T * V; i += THREADS) {
        const int t = i / V, c = (i % V) * 8;
        float x[8], dt[8], gy[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = dt[j] = gy[j] = 0.f;
        if (t < nt && c < nc) {
            TokenRaw<IoT> raw;
            raw.load(a, b * a.L + t0 + t, d0 + c);
            raw.get(a, d0 + c, x, dt, gy);
        }
        // pair k lies at k ^ (k >> 3): the vectors of 8 threads then meet all banks
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int k = c / 2 + j;
            sd[t * (CT / 2) + (k ^ ((k >> 3) & 7))] =
                make_float4(dt[2 * j], dt[2 * j + 1], dt[2 * j] * x[2 * j], dt[2 * j + 1] * x[2 * j + 1]);
            sg[t * (CT / 2) + k] = make_float2(gy[2 * j], gy[2 * j + 1]);
        }
    }
    stage_bc<IoT, T, Np, THREADS>(a, b, g, t0, nt, sB, sC);
    __syncthreads();
    const float4* pd = sd + (pair ^ ((pair >> 3) & 7));
    const float2* pg = sg + pair;
#pragma unroll 4
    for (int t = 0; t < T; ++t) {                        // tokens past the end have dt = 0 and g = 0
        const float4 d = pd[t * (CT / 2)];
        const float2 g2 = pg[t * (CT / 2)];
        f32x2 B[S / 2], C[S / 2];
        f2_load<S>(sB + t * Np + n0, B);
        f2_load<S>(sC + t * Np + n0, C);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float dt1 = e ? d.y : d.x, dx1 = e ? d.w : d.z, g1 = e ? g2.y : g2.x;
            const f32x2 dt = f2_pack(dt1, dt1), dx = f2_pack(dx1, dx1), gy = f2_pack(g1, g1);
            sum[e] += dt1;
#pragma unroll
            for (int s = 0; s < S / 2; ++s) {
                const f32x2 av = f2_exp2(f2_mul(dt, A2[e][s]));
                h[e][s] = f2_fma(av, h[e][s], f2_mul(dx, B[s]));
                Pr[e][s] = f2_mul(Pr[e][s], av);
                Gs[e][s] = f2_fma(Pr[e][s], f2_mul(C[s], gy), Gs[e][s]);
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        store_states<S>((float*)(a.ws + sh.off_h), bc * a.D + d0 + ch + e, a.N, n0, ok, h[e]);
        store_states<S>((float*)(a.ws + sh.off_g), bc * a.D + d0 + ch + e, a.N, n0, ok, Gs[e]);
        if (ok && n0 == 0) ((float*)(a.ws + sh.off_dt))[bc * a.D + d0 + ch + e] = sum[e];
    }
}

// Step 2, a thread a state: the first half of the blocks turns the chunks' end
// states into the states that enter them, the second their adjoints into the
// ones that leave them.  8 chunks' loads at a time.
__global__ void __launch_bounds__(128)
selective_bwd_chunks_kernel(const SelectiveArgs a, const SbShape sh, int half) {
    const bool back = (int)blockIdx.x >= half;
    const int64_t i = (int64_t)(blockIdx.x - (back ? half : 0)) * 128 + threadIdx.x, DN = a.D * a.N;
    if (i >= a.batch * DN) return;
    const int64_t b = i / DN, dn = i % DN, d = dn / a.N;
    const float A2 = decay_rate(a.A[dn]);
    float* w = (float*)(a.ws + (back ? sh.off_g : sh.off_h)) + b * sh.nch * DN + dn;
    const float* wdt = (const float*)(a.ws + sh.off_dt) + b * sh.nch * a.D + d;
    const void* from = back ? a.dfinal : a.init;
    float v = 0.f;
    if (from) v = a.state_bf16 ? to_f32(((const bf16*)from)[i]) : ((const float*)from)[i];
    const int64_t last = sh.nch - 1;
    for (int64_t c0 = 0; c0 < sh.nch; c0 += 8) {
        float own[8], dt[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t c = back ? last - c0 - q : c0 + q;
            own[q] = dt[q] = 0.f;
            if (c0 + q < sh.nch) {
                own[q] = w[c * DN];
                dt[q] = wdt[c * a.D];
            }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int64_t c = back ? last - c0 - q : c0 + q;
            if (c0 + q >= sh.nch) break;
            w[c * DN] = v;
            v = fmaf(exp2_approx(dt[q] * A2), v, own[q]);
        }
    }
    if (back && a.dinit) {
        if (a.state_bf16) ((bf16*)a.dinit)[i] = from_f32<bf16>(v);
        else ((float*)a.dinit)[i] = v;
    }
}

// Sums v[i] over the P lanes (neighbours) that hold the same states of other
// channels; the lane ends up with the sums of values first .. first + max(8 / P, 1).
template <int P>
__device__ __forceinline__ int sum_over_channels(float (&v)[8], int lane) {
    int first = 0;
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        if ((1 << step) >= P) break;
        const int half = 4 >> step;
        const bool up = lane & (1 << step);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= half) break;
            const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 1 << step);
        }
        first += up ? half : 0;
    }
#pragma unroll
    for (int o = 8; o < P; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return first;
}

// Writes a round's values of the lane's states, [8 / S tokens][S] (S = 8: one
// token), summed over the warp's channels, to the warp's rows of the chunk's sums.
template <class Tile>
__device__ __forceinline__ void put_sums(float (&v)[8], int lane, float* row) {
    constexpr int P = Tile::P, S = Tile::S, Np = Tile::Np, LEFT = P >= 8 ? 1 : 8 / P;
    const int first = sum_over_channels<P>(v, lane);
    if (P > 8 && (lane & 8)) return;
#pragma unroll
    for (int i = 0; i < LEFT; ++i) {
        const int k = first + i;
        row[(k / S) * Np + k % S] = v[i];
    }
}

// Step 3.
template <typename IoT, typename GT_, class Tile>
__global__ void __launch_bounds__(Tile::THREADS, 3)
selective_bwd_main_kernel(const SelectiveArgs a, const SbShape sh) {
    constexpr int K = Tile::K, S = Tile::S, T = Tile::T, GT = Tile::GT, W = Tile::W, THREADS = Tile::THREADS;
    constexpr int Np = Tile::Np, P = Tile::P, CT = Tile::CT, YS = Tile::YS, V = CT / 8, ACC = Tile::ACC;
    constexpr int IT = (T * V + THREADS - 1) / THREADS;        // 8-channel vectors of a tile a thread
    constexpr int R = 8 / S;                                   // tokens of a round of sums over the channels
    extern __shared__ float4 smem4[];
    float4* sd = smem4;                                        // [T][CT / 2]: dt, dt, x, x; later dx, dx, d dt, d dt
    float4* hs = sd + T * (CT / 2);                            // [T / GT - 1][2 S / 4][THREADS]
    float2* sg = (float2*)(hs + (T / GT - 1) * (S / 2) * THREADS);   // [T][CT / 2]: g, g; later g x
    float* sy = (float*)(sg + T * (CT / 2));                   // [T][YS]
    float* sB = sy + T * YS;                                   // [T][Np]
    float* sC = sB + T * Np;
    float* acc = sC + T * Np;                                  // [W][T][Np]
    const int sp = (int)(blockIdx.x % (unsigned)sh.split);
    int64_t r = blockIdx.x / (unsigned)sh.split;
    const int64_t g = r % a.G;
    r /= a.G;
    const int64_t ck = r % sh.nch, b = r / sh.nch, t0 = ck * T;
    const int nt = a.L - t0 < T ? (int)(a.L - t0) : T;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pair = warp * P + lane % P, n0 = (lane / P) * S, ch = pair * 2;
    const int slot = pair ^ ((pair >> 3) & 7);                 // where the pair lies in a row of sd
    const int64_t bc = b * sh.nch + ck, tok0 = b * a.L + t0;
    const float* wh = (const float*)(a.ws + sh.off_h);
    const float* wg = (const float*)(a.ws + sh.off_g);
    float* wrow = acc + warp * T * Np + n0;
    float accB[ACC], accC[ACC];
#pragma unroll
    for (int i = 0; i < ACC; ++i) accB[i] = accC[i] = 0.f;
    stage_bc<IoT, T, Np, THREADS>(a, b, g, t0, nt, sB, sC);

    for (int tile = sp; tile < sh.tiles; tile += sh.split) {
        const int c0 = tile * CT, nc = sh.Dg - c0 < CT ? sh.Dg - c0 : CT;
        const int64_t d0 = g * sh.Dg + c0;
        const bool ok = ch < nc;
        f32x2 A2[2][S / 2], h[2][S / 2], w[2][S / 2], dA[2][S / 2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            load_states<S>(a.A, d0 + ch + e, a.N, n0, ok, A2[e]);
            decay_rates<S>(A2[e]);
            load_states<S>(wh, bc * a.D + d0 + ch + e, a.N, n0, ok, h[e]);
            load_states<S>(wg, bc * a.D + d0 + ch + e, a.N, n0, ok, w[e]);
#pragma unroll
            for (int s = 0; s < S / 2; ++s) dA[e][s] = 0;
        }
        for (int i = tid; i < T * V; i += THREADS) {
            const int t = i / V, c = (i % V) * 8;
            float x[8], dt[8], gy[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = dt[j] = gy[j] = 0.f;
            if (t < nt && c < nc) {
                TokenRaw<IoT> raw;
                raw.load(a, tok0 + t, d0 + c);
                raw.get(a, d0 + c, x, dt, gy);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = c / 2 + j;
                sd[t * (CT / 2) + (k ^ ((k >> 3) & 7))] = make_float4(dt[2 * j], dt[2 * j + 1], x[2 * j], x[2 * j + 1]);
                sg[t * (CT / 2) + k] = make_float2(gy[2 * j], gy[2 * j + 1]);
            }
        }
        // the next tile's inputs come into L2 while this one is computed
        if (tile + sh.split < sh.tiles) {
            const int64_t dn = d0 + (int64_t)sh.split * CT;
            const int nn = sh.Dg - (tile + sh.split) * CT < CT ? sh.Dg - (tile + sh.split) * CT : CT;
            constexpr int LINE = 128 / (int)sizeof(IoT), LINES = (CT + LINE - 1) / LINE;
            for (int i = tid; i < 4 * nt * LINES; i += THREADS) {
                const int which = i % 4, c = (i / 4) % LINES * LINE;
                const int64_t tok = tok0 + i / 4 / LINES;
                if (c >= nn || (which == 3 && !a.z)) continue;
                const IoT* p = (const IoT*)(which == 0 ? a.x : which == 1 ? a.dt_raw : which == 2 ? a.dy : a.z);
                prefetch_l2(p + tok * (which == 3 ? a.zs : a.D) + dn + c);
            }
        }
        const float Dv0 = ok && a.Dv ? a.Dv[d0 + ch] : 0.f, Dv1 = ok && a.Dv ? a.Dv[d0 + ch + 1] : 0.f;
        __syncthreads();

        // the states, every GT-th kept; y and dC
        for (int tg = 0; tg < T / GT; ++tg) {
            if (tg > 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int s = 0; s < S / 2; s += 2)
                        ((ulonglong2*)hs)[((tg - 1) * (S / 2) + e * (S / 4) + s / 2) * THREADS + tid] =
                            make_ulonglong2(h[e][s], h[e][s + 1]);
            }
            float y[2 * GT];                                   // token u, channel e
#pragma unroll
            for (int r0 = 0; r0 < GT; r0 += R) {
                float dC[8];
#pragma unroll
                for (int u = 0; u < R; ++u) {
                    const int t = tg * GT + r0 + u;
                    const float4 d = sd[t * (CT / 2) + slot];
                    const float2 g2 = sg[t * (CT / 2) + pair];
                    f32x2 B[S / 2], C[S / 2];
                    f2_load<S>(sB + t * Np + n0, B);
                    f2_load<S>(sC + t * Np + n0, C);
                    f32x2 c[S / 2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float dt1 = e ? d.y : d.x, dx1 = dt1 * (e ? d.w : d.z), g1 = e ? g2.y : g2.x;
                        const f32x2 dt = f2_pack(dt1, dt1), dx = f2_pack(dx1, dx1), gy = f2_pack(g1, g1);
                        f32x2 ys = 0;
#pragma unroll
                        for (int s = 0; s < S / 2; ++s) {
                            h[e][s] = f2_fma(f2_exp2(f2_mul(dt, A2[e][s])), h[e][s], f2_mul(dx, B[s]));
                            ys = s ? f2_fma(C[s], h[e][s], ys) : f2_mul(C[s], h[e][s]);
                            c[s] = e ? f2_fma(gy, h[e][s], c[s]) : f2_mul(gy, h[e][s]);
                        }
                        const float2 yy = f2_get(ys);
                        y[(r0 + u) * 2 + e] = yy.x + yy.y;
                    }
#pragma unroll
                    for (int s = 0; s < S / 2; ++s) {
                        const float2 v = f2_get(c[s]);
                        dC[u * S + 2 * s] = v.x;
                        dC[u * S + 2 * s + 1] = v.y;
                    }
                }
                put_sums<Tile>(dC, lane, wrow + (tg * GT + r0) * Np);
            }
            if (a.z) {
                float* out = sy + tg * GT * YS + ch;
                if constexpr (GT == 4 && K <= 4) {
                    const int first = sum_over_states<K>(y, lane);
#pragma unroll
                    for (int i = 0; i < 4 / K; ++i) *(float2*)(out + (first / 2 + i) * YS) = make_float2(y[2 * i], y[2 * i + 1]);
                } else {
#pragma unroll
                    for (int i = 0; i < 2 * GT; ++i) {
#pragma unroll
                        for (int o = P; o < 32; o <<= 1) y[i] += __shfl_xor_sync(0xffffffffu, y[i], o);
                    }
                    if (n0 == 0) {
#pragma unroll
                        for (int u = 0; u < GT; ++u) *(float2*)(out + u * YS) = make_float2(y[2 * u], y[2 * u + 1]);
                    }
                }
            }
        }
        // dz; its inputs are loaded on this side of the barrier
        Raw8<IoT> rz[IT], ry[IT], rx[IT];
        if (a.z) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int i = tid + q * THREADS, t = i / V, c = (i % V) * 8;
                if (t >= nt || c >= nc) continue;
                const int64_t at = (tok0 + t) * a.D + d0 + c;
                rz[q].load((const IoT*)a.z + (tok0 + t) * a.zs + d0 + c);
                ry[q].load((const IoT*)a.dy + at);
                rx[q].load((const IoT*)a.x + at);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
            const int k = tid + i * THREADS;
            if (k < T * Np) {
#pragma unroll
                for (int q = 0; q < W; ++q) accC[i] += acc[q * T * Np + k];
            }
        }
        if (a.z) {
#pragma unroll
            for (int q = 0; q < IT; ++q) {
                const int i = tid + q * THREADS, t = i / V, c = (i % V) * 8;
                if (t >= nt || c >= nc) continue;
                const int64_t at = (tok0 + t) * a.D + d0 + c;
                float z[8], dy[8], x[8], dz[8], Dv[8];
                rz[q].get(z);
                ry[q].get(dy);
                rx[q].get(x);
#pragma unroll
                for (int j = 0; j < 8; ++j) Dv[j] = 0.f;
                if (a.Dv) load8(a.Dv + d0 + c, Dv);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float q = sigmoid_f32(z[j]);
                    dz[j] = dy[j] * fmaf(Dv[j], x[j], sy[t * YS + c + j]) * silu_grad(z[j], q);
                }
                store8((GT_*)a.dz + at, dz);
            }
        }
        __syncthreads();                                       // acc is free again

        // the adjoint back over the groups
        for (int tg = T / GT - 1; tg >= 0; --tg) {
            f32x2 av[GT][2][S / 2], hp[GT][2][S / 2];          // decay of token u, state before it
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                if (tg == 0) {
                    load_states<S>(wh, bc * a.D + d0 + ch + e, a.N, n0, ok, hp[0][e]);
                } else {
#pragma unroll
                    for (int s = 0; s < S / 2; s += 2) {
                        const ulonglong2 v = ((const ulonglong2*)hs)[((tg - 1) * (S / 2) + e * (S / 4) + s / 2) * THREADS + tid];
                        hp[0][e][s] = v.x;
                        hp[0][e][s + 1] = v.y;
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < GT; ++u) {
                const int t = tg * GT + u;
                const float4 d = sd[t * (CT / 2) + slot];
                f32x2 B[S / 2];
                if (u + 1 < GT) f2_load<S>(sB + t * Np + n0, B);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float dt1 = e ? d.y : d.x, dx1 = dt1 * (e ? d.w : d.z);
#pragma unroll
                    for (int s = 0; s < S / 2; ++s) {
                        av[u][e][s] = f2_exp2(f2_mul(f2_pack(dt1, dt1), A2[e][s]));
                        if (u + 1 < GT)
                            hp[u + 1][e][s] = f2_fma(av[u][e][s], hp[u][e][s], f2_mul(f2_pack(dx1, dx1), B[s]));
                    }
                }
            }
            float vB[2 * GT], vA[2 * GT];                      // sums over the states, token u, channel e
#pragma unroll
            for (int r0 = GT - R; r0 >= 0; r0 -= R) {
                float dB[8];
#pragma unroll
                for (int q = R - 1; q >= 0; --q) {
                    const int u = r0 + q, t = tg * GT + u;
                    const float4 d = sd[t * (CT / 2) + slot];
                    const float2 g2 = sg[t * (CT / 2) + pair];
                    f32x2 B[S / 2], C[S / 2], c[S / 2];
                    f2_load<S>(sB + t * Np + n0, B);
                    f2_load<S>(sC + t * Np + n0, C);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float dt1 = e ? d.y : d.x, dx1 = dt1 * (e ? d.w : d.z), g1 = e ? g2.y : g2.x;
                        const f32x2 dt = f2_pack(dt1, dt1), dx = f2_pack(dx1, dx1), gy = f2_pack(g1, g1);
                        f32x2 sb = 0, sa = 0;
#pragma unroll
                        for (int s = 0; s < S / 2; ++s) {
                            w[e][s] = f2_fma(C[s], gy, w[e][s]);
                            sb = s ? f2_fma(w[e][s], B[s], sb) : f2_mul(w[e][s], B[s]);
                            c[s] = e ? f2_fma(w[e][s], dx, c[s]) : f2_mul(w[e][s], dx);
                            w[e][s] = f2_mul(w[e][s], av[u][e][s]);         // the adjoint one token back
                            const f32x2 wah = f2_mul(w[e][s], hp[u][e][s]);
                            sa = s ? f2_fma(wah, A2[e][s], sa) : f2_mul(wah, A2[e][s]);
                            dA[e][s] = f2_fma(wah, dt, dA[e][s]);
                        }
                        const float2 b2 = f2_get(sb), a2 = f2_get(sa);
                        vB[u * 2 + e] = b2.x + b2.y;
                        vA[u * 2 + e] = a2.x + a2.y;
                    }
#pragma unroll
                    for (int s = 0; s < S / 2; ++s) {
                        const float2 v = f2_get(c[s]);
                        dB[q * S + 2 * s] = v.x;
                        dB[q * S + 2 * s + 1] = v.y;
                    }
                }
                put_sums<Tile>(dB, lane, wrow + (tg * GT + r0) * Np);
            }
            // dx and sum_n of d dt in the place of dt and x, whose last use this was
            auto finish = [&](int u, float b0, float b1, float a0, float a1) {
                const int t = tg * GT + u;
                const float4 d = sd[t * (CT / 2) + slot];
                const float2 g2 = sg[t * (CT / 2) + pair];
                constexpr float ln2 = 0.6931471805599453f;     // A2 = A log2 e
                sd[t * (CT / 2) + slot] = make_float4(fmaf(d.x, b0, Dv0 * g2.x), fmaf(d.y, b1, Dv1 * g2.y),
                                                      fmaf(d.z, b0, a0 * ln2), fmaf(d.w, b1, a1 * ln2));
                sg[t * (CT / 2) + pair] = make_float2(g2.x * d.z, g2.y * d.w);
            };
            if constexpr (GT == 4 && K <= 4) {
                const int first = sum_over_states<K>(vB, lane);
                sum_over_states<K>(vA, lane);
                __syncwarp();                                  // the group's tokens have been read
#pragma unroll
                for (int i = 0; i < 4 / K; ++i) finish(first / 2 + i, vB[2 * i], vB[2 * i + 1], vA[2 * i], vA[2 * i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < 2 * GT; ++i) {
#pragma unroll
                    for (int o = P; o < 32; o <<= 1) {
                        vB[i] += __shfl_xor_sync(0xffffffffu, vB[i], o);
                        vA[i] += __shfl_xor_sync(0xffffffffu, vA[i], o);
                    }
                }
                __syncwarp();
                if (n0 == 0) {
#pragma unroll
                    for (int u = 0; u < GT; ++u) finish(u, vB[2 * u], vB[2 * u + 1], vA[2 * u], vA[2 * u + 1]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e)
            store_states<S>((float*)(a.ws + sh.off_dA), bc * a.D + d0 + ch + e, a.N, n0, ok, dA[e]);
        Raw8<IoT> rdt[IT];
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int i = tid + q * THREADS, t = i / V, c = (i % V) * 8;
            if (t < nt && c < nc) rdt[q].load((const IoT*)a.dt_raw + (tok0 + t) * a.D + d0 + c);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ACC; ++i) {
            const int k = tid + i * THREADS;
            if (k < T * Np) {
#pragma unroll
                for (int q = 0; q < W; ++q) accB[i] += acc[q * T * Np + k];
            }
        }
#pragma unroll
        for (int q = 0; q < IT; ++q) {
            const int i = tid + q * THREADS, t = i / V, c = (i % V) * 8;
            if (t >= nt || c >= nc) continue;
            const int64_t at = (tok0 + t) * a.D + d0 + c;
            float raw[8], bias[8], dx[8], ddt[8];
            rdt[q].get(raw);
#pragma unroll
            for (int j = 0; j < 8; ++j) bias[j] = 0.f;
            if (a.dt_bias) load8(a.dt_bias + d0 + c, bias);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = c / 2 + j;
                float4* p = sd + t * (CT / 2) + (k ^ ((k >> 3) & 7));
                float4 v = *p;
                v.z *= sigmoid_f32(raw[2 * j] + bias[2 * j]);
                v.w *= sigmoid_f32(raw[2 * j + 1] + bias[2 * j + 1]);
                dx[2 * j] = v.x;
                dx[2 * j + 1] = v.y;
                ddt[2 * j] = v.z;
                ddt[2 * j + 1] = v.w;
                *p = v;
            }
            store8((GT_*)a.dx + at, dx);
            store8((GT_*)a.ddt + at, ddt);
        }
        __syncthreads();
        for (int i = tid; i < 2 * nc; i += THREADS) {          // sums over the chunk's tokens: d dt_raw, g x
            const int which = i >= nc, c = which ? i - nc : i, k = c >> 1, e = c & 1;
            const float* p = which ? (const float*)(sg + k) + e : (const float*)(sd + (k ^ ((k >> 3) & 7))) + 2 + e;
            const int step = which ? CT : 2 * CT;
            float s = 0.f;
#pragma unroll 8
            for (int t = 0; t < nt; ++t) s += p[t * step];
            ((float*)(a.ws + sh.off_par))[(bc * 2 + which) * a.D + d0 + c] = s;
        }
        __syncthreads();                                       // the next tile is staged over these
    }
#pragma unroll
    for (int i = 0; i < ACC; ++i) {
        const int k = tid + i * THREADS, t = k / Np, n = k % Np;
        if (k >= T * Np || t >= nt || n >= a.N) continue;
        const int64_t all = a.batch * a.L * a.G * a.N;
        float* out = (float*)(a.ws + sh.off_dBC) + 2 * sp * all + ((tok0 + t) * a.G + g) * a.N + n;
        out[0] = accB[i];
        out[all] = accC[i];
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

template <typename IoT, typename GT, class Tile>
static cudaError_t launch_bwd_t(const SelectiveArgs& a, cudaStream_t s) {
    const SbShape sh = sb_shape(a.batch, a.L, a.D, a.N, a.G);
    constexpr int smem1 = (int)sizeof(float) * Tile::T * (3 * Tile::CT + 2 * Tile::Np), smem3 = Tile::SMEM;
    const auto k1 = selective_bwd_summary_kernel<IoT, Tile>;
    const auto k3 = selective_bwd_main_kernel<IoT, GT, Tile>;
    cudaError_t e = cudaSuccess;
    if (smem1 > 48 * 1024) e = cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, smem1);
    if (e == cudaSuccess && smem3 > 48 * 1024)
        e = cudaFuncSetAttribute(k3, cudaFuncAttributeMaxDynamicSharedMemorySize, smem3);
    if (e != cudaSuccess) return e;
    const int64_t chunks = a.batch * sh.nch * a.G;
    const int half = (int)((a.batch * a.D * a.N + 127) / 128);
    k1<<<(unsigned)(chunks * sh.tiles), Tile::THREADS, smem1, s>>>(a, sh);
    selective_bwd_chunks_kernel<<<(unsigned)(2 * half), 128, 0, s>>>(a, sh, half);
    k3<<<(unsigned)(chunks * sh.split), Tile::THREADS, smem3, s>>>(a, sh);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t bn = a.batch * sh.nch, DN = a.D * a.N, M = a.batch * a.L * a.G * a.N;
    const ColumnSum sums[] = {{(const float*)(a.ws + sh.off_dBC), sh.split, 2 * M, 2 * M, a.dB, M, a.dC, sizeof(GT) == 2},
                              {(const float*)(a.ws + sh.off_dA), bn, DN, DN, a.dA, DN, nullptr, false},
                              {(const float*)(a.ws + sh.off_par), bn, 2 * a.D, 2 * a.D, a.ddt_bias, a.D, a.dD, false}};
    return launch_column_sums(sums, a.ddt_bias || a.dD ? 3 : 2, s);
}

template <typename IoT, typename GT>
static cudaError_t launch_bwd_s(const SelectiveArgs& a, cudaStream_t s) {
    if (a.N <= 8) return launch_bwd_t<IoT, GT, SbTile<2, 4, 16, 4>>(a, s);
    if (a.N <= 16) return launch_bwd_t<IoT, GT, SbTile<4, 4, 32, 4>>(a, s);
    if (a.N <= 32) return launch_bwd_t<IoT, GT, SbTile<8, 4, 32, 4>>(a, s);
    if (a.N <= 64) return launch_bwd_t<IoT, GT, SbTile<16, 4, 16, 4>>(a, s);
    if (a.N <= 128) return launch_bwd_t<IoT, GT, SbTile<32, 4, 16, 4>>(a, s);
    return launch_bwd_t<IoT, GT, SbTile<32, 8, 8, 2>>(a, s);
}

cudaError_t launch_selective_bwd(const SelectiveArgs& a, cudaStream_t s) {
    if (a.batch == 0 || a.L == 0) {
        const int64_t n = a.D * a.N * (a.batch > 1 ? a.batch : 1);
        selective_bwd_empty_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(a);
        return cudaGetLastError();
    }
    if (a.io_bf16) return a.y_bf16 ? launch_bwd_s<bf16, bf16>(a, s) : launch_bwd_s<bf16, float>(a, s);
    return a.y_bf16 ? launch_bwd_s<float, bf16>(a, s) : launch_bwd_s<float, float>(a, s);
}

}  // namespace ssd
