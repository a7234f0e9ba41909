// Short causal convolution along the tokens (2 to 4 taps per channel), its
// single-token step and its backward pass.
//
//   v_t[c] = bias[c] + sum_{k < W} w[c][k] x_{t-W+1+k}[c];   y = v or silu(v)
//   dv = dy silu'(v);  dx_s = sum_k w[k] dv_{s+W-1-k};  dw[k] = sum_t dv_t x_{t-W+1+k};  db = sum_t dv_t
//
// Every kernel is a stream bound by HBM: a thread owns a few neighbouring
// channels, walks over a run of tokens with the last W - 1 inputs in registers,
// and so reads each input once (and W - 1 more per run).  The inputs stand in a
// ring of 4 slots by token mod 4, which unrolled rounds of 4 tokens turn into fixed
// registers: nothing is moved.
//
// Measured, bf16, 4 taps, SiLU, a B200 (6568 GB/s copy): 4 x 2048 tokens x 4352
// channels forward 36 us (3950 GB/s), backward 64 us (3340 GB/s); a token of 256
// sequences x 10240 channels 12 us.  SiLU's two special functions an element are
// 16 us of the forward by themselves.
#include "ssd_internal.h"
#include "ssd_vec.cuh"

namespace ssd {

constexpr int VEC = 4;    // channels of a thread: 8 or 16 bytes a token

// the kept inputs, whose dtype is known at run time only
__device__ __forceinline__ void load_state(const void* p, bool is_bf16, int64_t i, float* v) {
    if (is_bf16) load4((const bf16*)p + i, v);
    else load4((const float*)p + i, v);
}
__device__ __forceinline__ void store_state(void* p, bool is_bf16, int64_t i, const float* v) {
    if (is_bf16) store4((bf16*)p + i, v);
    else store4((float*)p + i, v);
}

// weight [D][W] of channels c .. c + VEC as w[k][i]
template <int W>
__device__ __forceinline__ void load_taps(const float* w, int64_t c, float (&out)[W][VEC]) {
    float raw[W * VEC];
#pragma unroll
    for (int i = 0; i < W * VEC / 4; ++i) Vec16<float>::load(w + c * W + 4 * i, raw + 4 * i);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
#pragma unroll
        for (int k = 0; k < W; ++k) out[k][i] = raw[i * W + k];
}

// where channel c lies in the split tensors: tensor index, its row length and c's place in the row
__device__ __forceinline__ int split_of(const Conv1dArgs& a, int64_t c, int64_t* ld, int64_t* at) {
    if (c < a.part[0]) { *ld = a.part[0]; *at = c; return 0; }
    c -= a.part[0];
    if (c < a.part[1]) { *ld = a.part[1]; *at = c; return 1; }
    *ld = a.part[2]; *at = c - a.part[1];
    return 2;
}

// the W - 1 inputs before token t0 of a sequence that starts at token p: kept
// inputs where they lie before p (t0 < p: as of token p)
template <typename IoT, int W>
__device__ __forceinline__ void load_window(const Conv1dArgs& a, int64_t b, int64_t c, int64_t t0, int64_t p,
                                            float (&win)[W][VEC]) {
    const int64_t from = t0 < p ? p : t0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int64_t s = from - (W - 1) + j;
        if (s >= p) {
            load4((const IoT*)a.x + (b * a.L + s) * a.xs + c, win[j]);
        } else if (a.init) {
            load_state(a.init, a.state_bf16, (b * (W - 1) + (W - 1) + (s - p)) * a.D + c, win[j]);
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) win[j][i] = 0.f;
        }
    }
}

// filter and bias of channels c .. c + VEC
template <int W>
__device__ __forceinline__ void load_filter(const Conv1dArgs& a, int64_t c, f32x2 (&w)[W][VEC / 2], f32x2 (&bias)[VEC / 2]) {
    float wf[W][VEC];
    load_taps<W>(a.w, c, wf);
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) w[k][i] = f2_pack(wf[k][2 * i], wf[k][2 * i + 1]);
    }
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) bias[i] = a.bias ? f2_pack(a.bias[c + 2 * i], a.bias[c + 2 * i + 1]) : 0;
}

// the inputs before the first token of a run (of token `lead` of it, when its
// first tokens are absent) at their places in the ring
template <typename IoT, int W>
__device__ __forceinline__ void load_ring(const Conv1dArgs& a, int64_t b, int64_t c, int64_t t0, int64_t p,
                                          f32x2 (&ring)[4][VEC / 2]) {
    float win[W][VEC] = {};
    load_window<IoT, W>(a, b, c, t0, p, win);
    const int shift = t0 < p ? (int)((p - t0) & 3) : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) ring[q][i] = 0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int slot = (4 - (W - 1) + j + shift) & 3;
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < VEC / 2; ++i)
                if (slot == q) ring[q][i] = f2_pack(win[j][2 * i], win[j][2 * i + 1]);
    }
}

// The forward: kFwdRound tokens' loads are in flight while the round before is
// computed.  A run of 32 tokens reads 3 / 32 of its inputs twice and its filter
// once for 256 (fp32: 512) bytes of input; where there are fewer threads than keep
// an SM's loads in flight, runs of 8.  64 registers, 8 blocks an SM: 37 us at 4 x
// 2048 x 4352, 39 us with 80 registers, 43 us with 8 channels a thread.
constexpr int kFwdThreads = 128, kFwdRound = 4;

template <typename IoT, typename YT, int W>
__global__ void __launch_bounds__(kFwdThreads, 8)
conv1d_fwd_kernel(const Conv1dArgs a, int cblocks, int nseg, int run) {
    constexpr int H = VEC / 2, U = kFwdRound;
    const int64_t c = ((int64_t)(blockIdx.x % (unsigned)cblocks) * kFwdThreads + threadIdx.x) * VEC;
    const int64_t bs = blockIdx.x / (unsigned)cblocks;
    const int64_t b = bs / nseg, seg = bs % nseg;
    if (c >= a.D) return;
    int64_t p = a.pad_left ? a.pad_left[b] : 0;
    p = p < 0 ? 0 : p > a.L ? a.L : p;
    const int64_t t0 = seg * run;
    const int64_t t1 = t0 + run < a.L ? t0 + run : a.L;
    int64_t ld, at;
    const int which = split_of(a, c, &ld, &at);
    YT* y = (YT*)a.y[which] + (b * a.L + t0) * ld + at;
    const IoT* x = (const IoT*)a.x + (b * a.L + t0) * a.xs + c;
    const int len = (int)(t1 - t0), lead = t0 < p ? (int)((p < t1 ? p : t1) - t0) : 0;   // lead: absent tokens

    Raw4<IoT> next[U];
    auto load = [&](int t) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u >= lead && t + u < len) next[u].load(x + (int64_t)(t + u) * a.xs);
    };
    load(0);
    // the input of token t (from t0 on) lies in slot t mod 4 of the ring
    f32x2 w[W][H], ring[4][H], bias[H];
    load_filter<W>(a, c, w, bias);
    load_ring<IoT, W>(a, b, c, t0, p, ring);
    auto token = [&](int t, int u) {
        float out[VEC];
        next[u].get2(ring[u]);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            f32x2 v = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) v = f2_fma(w[k][i], ring[(u + 4 - (W - 1) + k) % 4][i], v);
            const float2 r = f2_get(a.silu ? f2_silu(v) : v);
            out[2 * i] = r.x;
            out[2 * i + 1] = r.y;
        }
        store4(y + (int64_t)(t + u) * ld, out);
    };
    int t = 0;
    // absent tokens: y = 0; the ring holds the inputs before token `lead`, at its own place
    for (; t + U <= lead; t += U) {
        float zero[VEC] = {};
#pragma unroll
        for (int u = 0; u < U; ++u) store4(y + (int64_t)(t + u) * ld, zero);
    }
    if (t > 0) load(t);
    for (; t < len; t += U) {
        if (t >= lead && t + U <= len) {
            Raw4<IoT> ahead[U];
#pragma unroll
            for (int u = 0; u < U; ++u) ahead[u] = next[u];
            const bool more = t + 2 * U <= len;
            if (more) {
#pragma unroll
                for (int u = 0; u < U; ++u) ahead[u].load(x + (int64_t)(t + U + u) * a.xs);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) token(t, u);
#pragma unroll
            for (int u = 0; u < U; ++u) next[u] = ahead[u];
            if (!more) load(t + U);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= len) break;
                if (t + u >= lead) {
                    token(t, u);
                } else {
                    float zero[VEC] = {};
                    store4(y + (int64_t)(t + u) * ld, zero);
                }
            }
            load(t + U);
        }
    }
    if (a.final_state && seg == nseg - 1) {
        // the last W - 1 inputs: of the tokens before `end`
        const int end = len > lead ? len : lead;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            float f[VEC];
            const int slot = (end + 4 - (W - 1) + j) & 3;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const f32x2 lo = slot & 1 ? ring[1][i] : ring[0][i], hi = slot & 1 ? ring[3][i] : ring[2][i];
                const float2 r = f2_get(slot & 2 ? hi : lo);
                f[2 * i] = r.x;
                f[2 * i + 1] = r.y;
            }
            store_state(a.final_state, a.state_bf16, (b * (W - 1) + j) * a.D + c, f);
        }
    }
}

// One token: a thread owns VEC channels of NB sequences, whose state is read and
// written by no other thread; all loads are in flight before the first is used, and
// the filter, larger than a sequence's inputs, is fetched once for NB of them.
template <typename IoT, typename YT, int W, int NB>
__global__ void __launch_bounds__(kFwdThreads)
conv1d_update_kernel(const Conv1dArgs a, int cblocks) {
    const int64_t c = ((int64_t)(blockIdx.x % (unsigned)cblocks) * kFwdThreads + threadIdx.x) * VEC;
    const int64_t b0 = (int64_t)(blockIdx.x / (unsigned)cblocks) * NB;
    if (c >= a.D) return;
    float win[NB][W][VEC] = {};
#pragma unroll
    for (int u = 0; u < NB; ++u) {
        if (b0 + u >= a.batch) break;
        load4((const IoT*)a.x + (b0 + u) * a.xs + c, win[u][W - 1]);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            load_state(a.final_state, a.state_bf16, ((b0 + u) * (W - 1) + j) * a.D + c, win[u][j]);
    }
    float w[W][VEC], bias[VEC] = {};
    load_taps<W>(a.w, c, w);
    if (a.bias) Vec16<float>::load(a.bias + c, bias);
    int64_t ld, at;
    const int which = split_of(a, c, &ld, &at);
#pragma unroll
    for (int u = 0; u < NB; ++u) {
        if (b0 + u >= a.batch) break;
        float out[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            float v = bias[i];
#pragma unroll
            for (int k = 0; k < W; ++k) v = fmaf(w[k][i], win[u][k][i], v);
            out[i] = a.silu ? v * sigmoid_f32(v) : v;
        }
        store4((YT*)a.y[which] + (b0 + u) * ld + at, out);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
            store_state(a.final_state, a.state_bf16, ((b0 + u) * (W - 1) + j) * a.D + c, win[u][j + 1]);
    }
}

// Backward.  A block is 32 lanes (4 channels each) x 4 warps; warp q walks over
// the tokens of its run and the W - 1 after it (whose dv its last dx need), loads a
// round ahead.  dx of a token is complete W - 1 tokens later.  The
// block's sums of dw and db go to one row of the partial sums.
constexpr int kBwdWarps = 4, kBwdRound = 4;

template <typename IoT, typename GT, int W>
__global__ void __launch_bounds__(kBwdWarps * 32, 4)
conv1d_bwd_kernel(const Conv1dArgs a, int cblocks, int nseg, int run) {
    constexpr int H = VEC / 2, U = kBwdRound;
    __shared__ float sums[kBwdWarps][(W + 1) * VEC][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = ((int64_t)(blockIdx.x % (unsigned)cblocks) * 32 + lane) * VEC;
    const int64_t bs = blockIdx.x / (unsigned)cblocks;
    const int64_t b = bs / nseg, seg = bs % nseg;
    const int64_t t0 = (seg * kBwdWarps + warp) * run;
    f32x2 dw[W][H], db[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
        db[i] = 0;
#pragma unroll
        for (int k = 0; k < W; ++k) dw[k][i] = 0;
    }
    if (c < a.D && (t0 < a.L || t0 == 0)) {
        int64_t ld, at;
        const int which = split_of(a, c, &ld, &at);
        const IoT* dy = (const IoT*)a.dy[which] + (b * a.L + t0) * ld + at;
        const IoT* x = (const IoT*)a.x + (b * a.L + t0) * a.xs + c;
        GT* dx = (GT*)a.dx + (b * a.L + t0) * a.dxs + c;
        const int left = a.L - t0 < (1 << 20) ? (int)(a.L - t0) : 1 << 20;   // tokens from t0 on
        const int len = left < run ? left : run;
        Raw4<IoT> nx[U], ny[U];
        auto load = [&](int t) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u < left && t + u < len + W - 1) {
                    nx[u].load(x + (int64_t)(t + u) * a.xs);
                    ny[u].load(dy + (int64_t)(t + u) * ld);
                }
        };
        load(0);
        // inputs, and the gradients of inputs that later tokens still add to, in rings by token mod 4
        f32x2 w[W][H], ring[4][H], pend[4][H], bias[H];
        load_filter<W>(a, c, w, bias);
        load_ring<IoT, W>(a, b, c, t0, 0, ring);
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int i = 0; i < H; ++i) pend[q][i] = 0;
        // token u of a round adds its dv to the gradients (mine: to dw and db too)
        auto token = [&](int u, const Raw4<IoT>& xr, const Raw4<IoT>& yr, bool mine) {
            f32x2 dv[H];
            xr.get2(ring[u]);
            yr.get2(dv);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                if (a.silu) {
                    f32x2 v = bias[i];
#pragma unroll
                    for (int k = 0; k < W; ++k) v = f2_fma(w[k][i], ring[(u + 4 - (W - 1) + k) % 4][i], v);
                    dv[i] = f2_mul(dv[i], f2_silu_grad(v, f2_sigmoid(v)));
                }
                if (mine) {
                    db[i] = f2_fma(dv[i], f2_pack(1.f, 1.f), db[i]);
#pragma unroll
                    for (int k = 0; k < W; ++k) dw[k][i] = f2_fma(dv[i], ring[(u + 4 - (W - 1) + k) % 4][i], dw[k][i]);
                }
#pragma unroll
                for (int k = 0; k < W - 1; ++k) {
                    f32x2& q = pend[(u + 4 - (W - 1) + k) % 4][i];
                    q = f2_fma(w[k][i], dv[i], q);
                }
                pend[u][i] = f2_mul(w[W - 1][i], dv[i]);
            }
        };
        auto ready = [&](int u, float (&g)[VEC]) {        // the gradient that token u completes
#pragma unroll
            for (int i = 0; i < H; ++i) {
                const float2 r = f2_get(pend[(u + 4 - (W - 1)) % 4][i]);
                g[2 * i] = r.x;
                g[2 * i + 1] = r.y;
            }
        };
        for (int t = 0; t < len + W - 1; t += U) {
            Raw4<IoT> xr[U], yr[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                xr[u] = nx[u];
                yr[u] = ny[u];
            }
            if (t >= U && t + 2 * U <= len) {             // all tokens and their inputs inside the run
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    nx[u].load(x + (int64_t)(t + U + u) * a.xs);
                    ny[u].load(dy + (int64_t)(t + U + u) * ld);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float g[VEC];
                    token(u, xr[u], yr[u], true);
                    ready(u, g);
                    store4(dx + (int64_t)(t + u - (W - 1)) * a.dxs, g);
                }
                continue;
            }
            load(t + U);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (t + u >= len + W - 1) break;
                if (t + u < left) {
                    token(u, xr[u], yr[u], t + u < len);
                } else {
#pragma unroll
                    for (int i = 0; i < H; ++i) pend[u][i] = 0;
                }
                const int s = t + u - (W - 1);            // the input (from t0 on) whose gradient is now complete
                if (s >= 0 || t0 == 0) {
                    float g[VEC];
                    ready(u, g);
                    if (a.dfinal && s >= left - (W - 1)) {
                        float f[VEC];
                        load_state(a.dfinal, a.state_bf16, (b * (W - 1) + s - left + W - 1) * a.D + c, f);
#pragma unroll
                        for (int i = 0; i < VEC; ++i) g[i] += f[i];
                    }
                    if (s >= 0) store4(dx + (int64_t)s * a.dxs, g);
                    else if (a.dinit) store_state(a.dinit, a.state_bf16, (b * (W - 1) + s + W - 1) * a.D + c, g);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < H; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) {
            const float2 r = f2_get(dw[k][i]);
            sums[warp][2 * i * W + k][lane] = r.x;
            sums[warp][(2 * i + 1) * W + k][lane] = r.y;
        }
        const float2 r = f2_get(db[i]);
        sums[warp][W * VEC + 2 * i][lane] = r.x;
        sums[warp][W * VEC + 2 * i + 1][lane] = r.y;
    }
    __syncthreads();
    float* row = a.ws + bs * (a.D * (W + 1));
    for (int e = warp; e < (W + 1) * VEC; e += kBwdWarps) {
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < kBwdWarps; ++q) s += sums[q][e][lane];
        if (c < a.D) row[e < W * VEC ? c * W + e : a.D * W + c + (e - W * VEC)] = s;
    }
}

// batch or seqlen 0: parameter gradients 0 (the batch 0 case)
__global__ void conv1d_zero_kernel(float* dw, float* db, int64_t nw, int64_t nb) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < nw + nb; i += (int64_t)gridDim.x * blockDim.x) {
        if (i < nw) dw[i] = 0.f;
        else if (db) db[i - nw] = 0.f;
    }
}

// tokens a thread walks over: 32 from 512 threads an SM on
static int fwd_run(int64_t batch, int64_t L, int64_t vecs) { return batch * ((L + 31) / 32) * vecs >= 148 * 512 ? 32 : 8; }

static int64_t fwd_segments(int64_t L, int run) { return L > 0 ? (L + run - 1) / run : 1; }

// tokens a warp of the backward walks over: the longest run that leaves 384 threads
// an SM (4 x 2048 tokens x 4352 channels: 128 tokens 62 us, 64 tokens 68 us)
static int bwd_run(int64_t batch, int64_t L, int64_t D) {
    for (int run = 128; run > 16; run /= 2)
        if (batch * ((L + run - 1) / run) * (D / VEC) >= 148 * 384) return run;
    return 16;
}

static int64_t bwd_segments(int64_t L, int run) {
    return L > 0 ? (L + kBwdWarps * run - 1) / (kBwdWarps * run) : 1;
}

int64_t conv1d_bwd_segments(int64_t batch, int64_t L, int64_t D) { return batch * bwd_segments(L, bwd_run(batch, L, D)); }

int64_t conv1d_blocks(int64_t batch, int64_t L, int64_t D) {
    return batch * fwd_segments(L, 8) * ((D / 4 + 31) / 32);
}

// calls f<IoT, OutT, W>() for the types and taps of a
#define CONV1D_DISPATCH(FN)                                                                    \
    do {                                                                                       \
        if (a.io_bf16) {                                                                       \
            if (a.y_bf16) { if (a.W == 2) FN(bf16, bf16, 2); else if (a.W == 3) FN(bf16, bf16, 3); else FN(bf16, bf16, 4); } \
            else { if (a.W == 2) FN(bf16, float, 2); else if (a.W == 3) FN(bf16, float, 3); else FN(bf16, float, 4); } \
        } else {                                                                               \
            if (a.y_bf16) { if (a.W == 2) FN(float, bf16, 2); else if (a.W == 3) FN(float, bf16, 3); else FN(float, bf16, 4); } \
            else { if (a.W == 2) FN(float, float, 2); else if (a.W == 3) FN(float, float, 3); else FN(float, float, 4); } \
        }                                                                                      \
    } while (0)

cudaError_t launch_conv1d_fwd(const Conv1dArgs& a, cudaStream_t s) {
    const int run = fwd_run(a.batch, a.L, a.D / VEC);
    const int cblocks = (int)((a.D / VEC + kFwdThreads - 1) / kFwdThreads), nseg = (int)fwd_segments(a.L, run);
    const unsigned grid = (unsigned)(a.batch * nseg * cblocks);
#define FN(IO, Y, W_) conv1d_fwd_kernel<IO, Y, W_><<<grid, kFwdThreads, 0, s>>>(a, cblocks, nseg, run)
    CONV1D_DISPATCH(FN);
#undef FN
    return cudaGetLastError();
}

cudaError_t launch_conv1d_update(const Conv1dArgs& a, cudaStream_t s) {
    const int cblocks = (int)((a.D / VEC + kFwdThreads - 1) / kFwdThreads);
    // four sequences a thread once that still leaves 512 threads an SM
    const int64_t quads = (a.batch + 3) / 4 * cblocks;
    if (quads >= 148 * 4) {
#define FN(IO, Y, W_) conv1d_update_kernel<IO, Y, W_, 4><<<(unsigned)quads, kFwdThreads, 0, s>>>(a, cblocks)
        CONV1D_DISPATCH(FN);
#undef FN
    } else {
#define FN(IO, Y, W_) conv1d_update_kernel<IO, Y, W_, 1><<<(unsigned)(a.batch * cblocks), kFwdThreads, 0, s>>>(a, cblocks)
        CONV1D_DISPATCH(FN);
#undef FN
    }
    return cudaGetLastError();
}

cudaError_t launch_conv1d_bwd(const Conv1dArgs& a, cudaStream_t s) {
    const int64_t nw = a.D * a.W;
    if (a.batch == 0) {
        conv1d_zero_kernel<<<(unsigned)((nw + a.D + 255) / 256), 256, 0, s>>>(a.dw, a.db, nw, a.D);
        return cudaGetLastError();
    }
    const int cblocks = (int)((a.D / VEC + 31) / 32), run = bwd_run(a.batch, a.L, a.D);
    const int nseg = (int)bwd_segments(a.L, run);
    const unsigned grid = (unsigned)(a.batch * nseg * cblocks);
#define FN(IO, G_, W_) conv1d_bwd_kernel<IO, G_, W_><<<grid, kBwdWarps * 32, 0, s>>>(a, cblocks, nseg, run)
    CONV1D_DISPATCH(FN);
#undef FN
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const ColumnSum sum = {a.ws, a.batch * nseg, nw + a.D, nw + a.D, a.dw, nw, a.db, false};
    return launch_column_sums(&sum, 1, s);
}

}  // namespace ssd
