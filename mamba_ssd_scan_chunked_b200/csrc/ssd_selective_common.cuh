// What the selective scan's kernels share (ssd_selective.cu, ssd_selective_bwd.cu).
//
// A lane holds S neighbouring states of 2 neighbouring channels; K lanes, a
// power of two, cover the N states (padded with A = B = C = 0, which keep a
// state at 0), and a warp covers 32 / K pairs of channels.
#pragma once

#include "ssd_common.cuh"
#include "ssd_internal.h"

namespace ssd {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

struct SelShape {
    int K;            // lanes of a channel
    int CT;           // channels of a block
    int Dg, tiles;    // channels of a group, blocks that cover them
    int Np;           // K * S
};

template <int S>
inline SelShape sel_shape(int64_t D, int64_t N, int64_t G, int warps) {
    SelShape sh{};
    sh.K = 1;
    while (sh.K * S < N) sh.K *= 2;
    sh.Np = sh.K * S;
    sh.CT = warps * (32 / sh.K) * 2;
    sh.Dg = (int)(D / G);
    sh.tiles = (sh.Dg + sh.CT - 1) / sh.CT;
    return sh;
}

}  // namespace ssd
