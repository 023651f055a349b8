// gated_scan.cuh -- the arithmetic of the recurrence in gated_scan.cu.
//
// A gate g is held as one signed number c: its smaller sigmoid s = 1 / (1 +
// e^|g|), negative where the state is kept rather than dropped (g >= 0):
//     g >= 0:  1 - a = s = -c,  a v = v + c v
//     g <  0:      a = s =  c,  a v = c v
// Both a and 1 - a then have all their digits: a itself, rounded to fp32, says
// too little of 1 - a for memories of thousands of tokens (2^-25 an error of
// the same sign at every token of a constant gate).  g = -inf is c = +0, g =
// +inf is c = -0.
#pragma once

#include "osdn_device.cuh"

namespace osdn {
namespace gs {

template <int M>
struct Mix {
    static constexpr int value = M;
};

__device__ __forceinline__ float gate_coefficient(float g) {
    float e, r;
    // the hardware's base-2 exponential and reciprocal (2 ulp each); e = 0 from |g| = 87.4
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fabsf(g) * -1.4426950408889634f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return __uint_as_float(__float_as_uint(e * r) | (~__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ bool keeps(float c) { return (int)__float_as_uint(c) < 0; }
__device__ __forceinline__ bool forgets(float c) { return __float_as_uint(c) == 0u; }        // a = 0
__device__ __forceinline__ bool passes(float c) { return __float_as_uint(c) == 0x80000000u; }  // 1 - a = 0

// c v, where a factor that is exactly zero hides v whatever it holds.
__device__ __forceinline__ float hide(float c, float v) { return c == 0.0f ? 0.0f : c * v; }

// Z: some factor may be exactly zero, and then hides what it multiplies.  Without Z there is none
// (the callers look), and the selections are saved.
template <bool Z>
__device__ __forceinline__ float decay(float c, float v) {
    if (Z && forgets(c)) return 0.0f;
    return fmaf(c, v, keeps(c) ? v : 0.0f);
}
template <int MIX>
__device__ __forceinline__ float weight(float c) {
    if (MIX == OSDN_MIX_SUM) return 1.0f;
    if (MIX == OSDN_MIX_MEAN) return keeps(c) ? -c : 1.0f - c;
    // 1 - a^2 = s (2 - s), or 1 - s^2
    float w;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(w) : "f"(fmaf(-c, c, keeps(c) ? -2.0f * c : 1.0f)));
    return w;
}
// w(a) x
template <int MIX, bool Z>
__device__ __forceinline__ float weighted(float c, float x) {
    if (MIX == OSDN_MIX_SUM) return x;
    if (Z && passes(c)) return 0.0f;
    return weight<MIX>(c) * x;
}
// With r the cotangent of the state after a token and v the state before it: the gradients w r of x
// and r (a b v + w' x) = r a b (v - k x) of g, where k is 0, 1 or a / w.  (w' = -a / w times a b,
// and k a b = a^2 sqrt((1 - a) / (1 + a)) goes to zero where w does.)
template <int MIX, bool Z>
__device__ __forceinline__ void gradients(float c, float r, float v, float x, float &dx, float &dg) {
    const float s = fabsf(c), ab = fmaf(-s, s, s);
    float d = v;
    if (MIX == OSDN_MIX_SUM) dx = r;
    if (MIX == OSDN_MIX_MEAN) {
        dx = weight<MIX>(c) * r;
        d -= x;
    }
    if (MIX == OSDN_MIX_UNIT) {
        const float q = fmaf(-c, c, keeps(c) ? -2.0f * c : 1.0f);   // w^2
        float inv;
        asm("rsqrt.approx.f32 %0, %1;" : "=f"(inv) : "f"(fmaxf(q, 1e-37f)));
        dx = q * inv * r;
        d = fmaf(-(keeps(c) ? 1.0f + c : c) * inv, x, d);
    }
    dg = Z && ab == 0.0f ? 0.0f : r * ab * d;
}

}  // namespace gs
}  // namespace osdn
