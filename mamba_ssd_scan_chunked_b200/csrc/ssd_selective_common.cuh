// What the selective scan's kernels share (ssd_selective.cu, ssd_selective_bwd.cu).
//
// A lane holds S neighbouring states; K lanes, a power of two, cover the N states,
// padded with A = B = C = 0, which keep a state at 0.  The padding is paid for in
// exponentials: lanes cover 8, 16, 32, 64, 128 or 256 states, so 24 cost as much as
// 32 and 40 as much as 64 (4 x 2048 tokens x 2048 channels, bf16, gated, a B200:
// 208 us with 24 states, 208 us with 32).
#pragma once

#include "ssd_internal.h"
#include "ssd_vec.cuh"

namespace ssd {

__device__ __forceinline__ f32x2 f2_exp2(f32x2 v) {
    const float2 t = f2_get(v);
    return f2_pack(exp2_approx(t.x), exp2_approx(t.y));
}
// A log2 e, what exp2(dt . ) takes, with the lowest fp32 value in the place of -inf (a
// state that forgets at once): absent tokens and padding have dt = 0, and 0 times
// infinity is NaN where the decay is 1.  NaN stays.
__device__ __forceinline__ float decay_rate(float A) {
    const float v = A * kLog2e;
    return v < -3.402823466e38f ? -3.402823466e38f : v;
}
// S consecutive floats (16-byte aligned) as S / 2 pairs
template <int S> __device__ __forceinline__ void f2_load(const float* p, f32x2 (&v)[S / 2]) {
#pragma unroll
    for (int i = 0; i < S / 4; ++i) {
        const ulonglong2 r = *reinterpret_cast<const ulonglong2*>(p + 4 * i);
        v[2 * i] = r.x;
        v[2 * i + 1] = r.y;
    }
}

// softplus(z) = max(z, 0) + log(1 + e), e = exp(-|z|) in [0, 1], of two values.
// log(1 + e) / e is the polynomial of degree 9 that is best in relative error
// over [0, 1] (Remez exchange: 4.7e-9; 2.3e-8 with its coefficients rounded to fp32
// and the last one to 1, 1.1e-7 evaluated in fp32; softplus itself, with the
// exponential, 4.2e-7 at most), which keeps the whole relative precision where dt
// is small; a difference of logarithms would not.  Against log1pf(expf(z)) it saves one special function and a branch.
// -inf gives 0, NaN stays NaN.
__device__ __forceinline__ f32x2 softplus2(float z0, float z1) {
    const f32x2 v = f2_pack(-fminf(fabsf(z0), 200.f), -fminf(fabsf(z1), 200.f));
    // exp(v) = 2^(v log2 e) with the rounding error of that product put back
    const f32x2 L = f2_pack(kLog2e, kLog2e), hi = f2_mul(v, L);
    const f32x2 err = f2_fma(v, L, f2_mul(hi, f2_pack(-1.f, -1.f)));
    const f32x2 lo = f2_fma(v, f2_pack(1.9259629911266175e-8f, 1.9259629911266175e-8f), err);   // log2 e - fl(log2 e)
    const f32x2 e0 = f2_exp2(hi);
    const f32x2 e = f2_fma(e0, f2_mul(lo, f2_pack(0.6931471805599453f, 0.6931471805599453f)), e0);
    constexpr float c[9] = {0.019851457327604294f, -0.056959524750709534f, 0.10603653639554977f,
                            -0.15305592119693756f, 0.1967593878507614f,    -0.24954134225845337f,
                            0.3332996368408203f,   -0.4999990165233612f,   1.f};
    f32x2 p = f2_pack(-0.003244024235755205f, -0.003244024235755205f);
#pragma unroll
    for (int i = 0; i < 9; ++i) p = f2_fma(p, e, f2_pack(c[i], c[i]));
    float m0, m1;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m0) : "f"(z0));
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(m1) : "f"(z1));
    return f2_fma(p, e, f2_pack(m0, m1));
}

// Lanes and channels of the forward: a lane holds S states of one channel, a warp
// 32 / K channels.  lane = state group * (32 / K) + channel, so that the lanes that
// read the same B and C are neighbours (a 16-byte shared load then takes 2 cycles of an
// SM; 4 when every fourth lane reads the same, measured).
template <int K_, int S_, int W_>
struct SelTile {
    static constexpr int K = K_;             // lanes of a channel
    static constexpr int S = S_;             // states of a lane
    static constexpr int W = W_;             // warps of a block
    static constexpr int Np = K * S;         // states with padding
    static constexpr int P = 32 / K;         // channels of a warp
    static constexpr int CT = W * P;         // channels of a block
};

struct SelShape {
    int Dg, tiles;           // channels of a group, blocks that cover them
    int nch, len0, clen;     // chunks of a sequence, tokens of chunk 0 and of the others
};

// Sums v[i] over the K lanes of a channel (xor distances P, 2 P, .. 16); lane
// group k of the K ends up with the sums of values first(k) .. first(k) + 8 / K
// (8 / K >= 1), or, with K > 8, each value is on several lanes.
template <int K>
__device__ __forceinline__ int sum_over_states(float (&v)[8], int lane) {
    constexpr int P = 32 / K;
    int first = 0;
    if constexpr (K >= 2) {
        const bool up = lane & P;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float send = up ? v[i] : v[i + 4], keep = up ? v[i + 4] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, P);
        }
        first += up ? 4 : 0;
    }
    if constexpr (K >= 4) {
        const bool up = lane & (2 * P);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float send = up ? v[i] : v[i + 2], keep = up ? v[i + 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, 2 * P);
        }
        first += up ? 2 : 0;
    }
    if constexpr (K >= 8) {
        const bool up = lane & (4 * P);
        const float send = up ? v[0] : v[1], keep = up ? v[1] : v[0];
        v[0] = keep + __shfl_xor_sync(0xffffffffu, send, 4 * P);
        first += up ? 1 : 0;
    }
#pragma unroll
    for (int o = 8 * P; o < 32; o <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return first;
}

}  // namespace ssd
