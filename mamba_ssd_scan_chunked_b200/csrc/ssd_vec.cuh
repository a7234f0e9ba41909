// Device-side helpers of the operators around the scan: vectors of 8 elements,
// approximations of the special functions, pairs of fp32 operations.
#pragma once

#include <type_traits>

#include "ssd_common.cuh"

namespace ssd {

// 8 consecutive elements (16-byte aligned) to and from fp32.
__device__ __forceinline__ void load8(const bf16* p, float* v) { Vec16<bf16>::load(p, v); }
__device__ __forceinline__ void load8(const float* p, float* v) {
    Vec16<float>::load(p, v);
    Vec16<float>::load(p + 4, v + 4);
}
__device__ __forceinline__ void store8(bf16* p, const float* v) { Vec16<bf16>::store(p, v); }
__device__ __forceinline__ void store8(float* p, const float* v) {
    Vec16<float>::store(p, v);
    Vec16<float>::store(p + 4, v + 4);
}
// asks for the 128-byte line at p to be brought into L2
__device__ __forceinline__ void prefetch_l2(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// 4 consecutive elements (aligned to their size) to and from fp32.
__device__ __forceinline__ void load4(const bf16* p, float* v) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(r.x << 16); v[1] = __uint_as_float(r.x & 0xffff0000u);
    v[2] = __uint_as_float(r.y << 16); v[3] = __uint_as_float(r.y & 0xffff0000u);
}
__device__ __forceinline__ void load4(const float* p, float* v) { Vec16<float>::load(p, v); }
__device__ __forceinline__ void store4(bf16* p, const float* v) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void store4(float* p, const float* v) { Vec16<float>::store(p, v); }

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + e^-v).  e^-v overflows to infinity below v = -88, where the result
// is 0 in fp32.  The two approximations are within 2 units in the last place each;
// the roundings of -v log2 e add 7.3e-8 |v| to the relative error of e^-v, so the
// sigmoid of a negative v loses some 8 units at -20 and 31 at -80, where it is 2e-9
// and 2e-35: nothing beside v or 1, which it is multiplied by or added to.
__device__ __forceinline__ float sigmoid_f32(float v) { return rcp_approx(1.f + exp2_approx(-kLog2e * v)); }
// d silu(v) / dv from g = sigmoid(v)
__device__ __forceinline__ float silu_grad(float v, float g) { return g * fmaf(v, 1.f - g, 1.f); }

// Two fp32 operations in one instruction (neighbouring states or channels of a lane): the
// rate of the arithmetic is the same, the issue slots are halved.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 f2_pack(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 f2_get(f32x2 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f32x2 f2_mul(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 f2_fma(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// 1 / (1 + e^-v) of both, v / (1 + e^-v) of both, and the latter's derivative from the former
__device__ __forceinline__ f32x2 f2_sigmoid(f32x2 v) {
    const float2 t = f2_get(f2_mul(v, f2_pack(-kLog2e, -kLog2e)));
    const f32x2 one = f2_pack(1.f, 1.f);
    const float2 q = f2_get(f2_fma(f2_pack(exp2_approx(t.x), exp2_approx(t.y)), one, one));
    return f2_pack(rcp_approx(q.x), rcp_approx(q.y));
}
__device__ __forceinline__ f32x2 f2_silu(f32x2 v) { return f2_mul(v, f2_sigmoid(v)); }
__device__ __forceinline__ f32x2 f2_silu_grad(f32x2 v, f32x2 g) {
    const f32x2 one = f2_pack(1.f, 1.f), rest = f2_fma(g, f2_pack(-1.f, -1.f), one);
    return f2_mul(g, f2_fma(v, rest, one));
}

// 8 elements as they lie in memory, widened when they are used
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
    uint4 r;
    __device__ __forceinline__ void load(const bf16* p) { r = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void minus_inf() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    __device__ __forceinline__ void get(float* v) const { Vec16<bf16>::unpack(r, v); }
};
template <> struct Raw8<float> {
    uint4 r[2];
    __device__ __forceinline__ void load(const float* p) {
        r[0] = *reinterpret_cast<const uint4*>(p);
        r[1] = *reinterpret_cast<const uint4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { r[0] = r[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void minus_inf() {
        r[0] = r[1] = make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
    }
    __device__ __forceinline__ void get(float* v) const {
        Vec16<float>::unpack(r[0], v);
        Vec16<float>::unpack(r[1], v + 4);
    }
};

// the same for 4 elements; get2 gives them as pairs
template <typename T> struct Raw4 {
    typename std::conditional<sizeof(T) == 4, uint4, uint2>::type r;
    __device__ __forceinline__ void load(const T* p) { r = *reinterpret_cast<const decltype(r)*>(p); }
    __device__ __forceinline__ void zero() { r = decltype(r){}; }
    __device__ __forceinline__ void get(float* v) const {
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) v[i] = __uint_as_float(w[i]);
            else v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        }
    }
    __device__ __forceinline__ void get2(f32x2 (&v)[2]) const {
        float f[4];
        get(f);
        v[0] = f2_pack(f[0], f[1]);
        v[1] = f2_pack(f[2], f[3]);
    }
};

}  // namespace ssd
