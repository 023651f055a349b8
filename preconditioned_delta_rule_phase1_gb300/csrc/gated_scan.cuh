// gated_scan.cuh -- the arithmetic of the recurrence in gated_scan.cu.
//
// Two forms.  The exact one holds a gate g as one signed number c: its smaller
// sigmoid s = 1 / (1 + e^|g|), negative where the state is kept rather than
// dropped (g >= 0):
//     g >= 0:  1 - a = s = -c,  a v = v + c v
//     g <  0:      a = s =  c,  a v = c v
// Both a and 1 - a then have all their digits.
//
// The short one, for bf16 I/O and |g| <= kPlainGate, multiplies with a rounded
// to fp32, within the run of at most 16 tokens that a thread holds: instructions
// are what costs most there, and a state is off by 16 roundings (2^-23 of it each)
// for that, whatever the gate.  How a state passes from run to run is taken from
// 1 - A with its digits in both forms (gated_scan_walk.cuh): a rounded a, taken
// 2^16 times, would be off by 1e-3 at a gate of 11, and keep all from a gate of 17
// on.  The weight of x reads 1 - a as e^-g a, with its digits, in both forms.
#pragma once

#include "osdn_device.cuh"

namespace osdn {
namespace gs {

template <int M>
struct Mix {
    static constexpr int value = M;
};

// A thread's two channels; arithmetic goes through packed instructions.
template <int V>
struct Vec {
    static_assert(V == 2, "two channels a thread");
    float v[V];
};
template <int V>
__device__ __forceinline__ Vec<V> fill(float x) {
    return {{x, x}};
}
template <int V>
__device__ __forceinline__ Vec<V> mul(const Vec<V> &a, const Vec<V> &b) {
    const float2 x = __fmul2_rn(make_float2(a.v[0], a.v[1]), make_float2(b.v[0], b.v[1]));
    return {{x.x, x.y}};
}
template <int V>
__device__ __forceinline__ Vec<V> add(const Vec<V> &a, const Vec<V> &b) {
    const float2 x = __fadd2_rn(make_float2(a.v[0], a.v[1]), make_float2(b.v[0], b.v[1]));
    return {{x.x, x.y}};
}
template <int V>
__device__ __forceinline__ Vec<V> fma(const Vec<V> &a, const Vec<V> &b, const Vec<V> &c) {
    const float2 x = __ffma2_rn(make_float2(a.v[0], a.v[1]), make_float2(b.v[0], b.v[1]), make_float2(c.v[0], c.v[1]));
    return {{x.x, x.y}};
}

__device__ __forceinline__ float exp2_fast(float x) {   // the hardware's, 2 ulp, zero below 2^-126
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
__device__ __forceinline__ float rcp_fast(float x) {    // 1 ulp
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float sqrt_fast(float x) {   // 3 ulp
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rsqrt_fast(float x) {
    float r;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------- the exact form
// In kinds, X, by what the callers have looked at:
//   kPlain  no gate beyond kPlainGate, so that no factor leaves fp32's normal range;
//   kEnds   or gates of -inf (c = +0) and +inf (c = -0): factors that are exactly zero;
//   kAny    any gate.  One above kPlainGate is held as c = -g: 1 - a is less than 2^-115, nothing beside any v
//           of the same channel, and what is formed of it comes from e^-g or e^(-g / 2) as it is needed.
// A factor that is exactly zero hides what it multiplies.  Only kAny says so: where v is finite it makes no
// difference, and an infinite v becomes NaN in the others, which the recurrence then carries to its end; the
// callers look there, and do it again.
enum { kPlain, kEnds, kAny };
constexpr float kPlainGate = 80.0f;   // e^80 and its reciprocal are normal numbers
constexpr float kPasses = -INFINITY;  // c of a gate of +inf
__device__ __forceinline__ float exp2_whole(float x) {   // with what lies below 2^-126
    float e;
    asm("ex2.approx.f32 %0, %1;" : "=f"(e) : "f"(x));
    return e;
}
template <int X>
__device__ __forceinline__ float gate_coefficient(float g) {
    if (X == kAny && g > kPlainGate) return -g;
    const float t = fabsf(g) * -kLog2e, e = X == kAny ? exp2_whole(t) : exp2_fast(t);
    return __uint_as_float(__float_as_uint(e * rcp_fast(1.0f + e)) | (~__float_as_uint(g) & 0x80000000u));
}
__device__ __forceinline__ bool keeps(float c) { return (int)__float_as_uint(c) < 0; }
__device__ __forceinline__ bool forgets(float c) { return __float_as_uint(c) == 0u; }   // a = 0
__device__ __forceinline__ bool open(float c) { return c < -1.0f; }                      // c is minus the gate

// a v
template <int X>
__device__ __forceinline__ float decay(float c, float v) {
    if (X == kAny && forgets(c)) return 0.0f;
    if (X == kAny && (open(c) || (c <= 0.0f && fabsf(v) == INFINITY))) return v;   // (a NaN is neither)
    return fmaf(c, v, keeps(c) ? v : 0.0f);
}
// 1 - A, with its digits, as A becomes a A
template <int X>
__device__ __forceinline__ float decay_rest(float c, float A, float D) {
    if (X == kAny && open(c)) return D;
    return fmaf(-c, A, keeps(c) ? D : 1.0f);
}
template <int V>
__device__ __forceinline__ bool finite(const Vec<V> &a) {
    return fabsf(a.v[0]) < INFINITY && fabsf(a.v[1]) < INFINITY;
}
// w(a)^2 = 1 - a^2 = s (2 - s), or 1 - s^2
__device__ __forceinline__ float unit_square(float c) { return fmaf(-c, c, keeps(c) ? -2.0f * c : 1.0f); }
template <int MIX, int X>
__device__ __forceinline__ float weight(float c) {
    if (MIX == OSDN_MIX_SUM) return 1.0f;
    if (X == kAny && open(c))   // e^-g, or sqrt(2) e^(-g / 2)
        return MIX == OSDN_MIX_MEAN ? exp2_whole(c * kLog2e) : 1.41421356f * exp2_whole(c * (0.5f * kLog2e));
    if (MIX == OSDN_MIX_MEAN) return keeps(c) ? -c : 1.0f - c;
    return sqrt_fast(unit_square(c));
}
// w(a) x
template <int MIX, int X>
__device__ __forceinline__ float weighted(float c, float x) {
    if (MIX == OSDN_MIX_SUM) return x;
    const float w = weight<MIX, X>(c);
    return X == kAny && w == 0.0f ? 0.0f : w * x;
}
// the gate from which on e^-g, or e^(-g / 2) where that counts, is zero in fp32
template <int MIX>
__device__ __forceinline__ constexpr float zero_from() { return MIX == OSDN_MIX_UNIT ? 208.0f : 104.0f; }
// With v the state before a token, the factor that turns R into the gradient of g is a b v + w' x =
// a b (v - k x), where k is 0, 1 or a / w.  (w' = -a / w times a b, and k a b = a^2 sqrt((1 - a) /
// (1 + a)) goes to zero where w does.)  Here a b and k a b:
template <int MIX, int X>
__device__ __forceinline__ void slope_factors(float c, float &ab, float &kab) {
    const float s = fabsf(c);
    if (X == kAny && open(c)) {
        ab = c > -104.0f ? exp2_whole(c * kLog2e) : 0.0f;
        if (c <= -zero_from<MIX>()) { kab = 0.0f; return; }
        kab = MIX == OSDN_MIX_UNIT ? 0.70710678f * exp2_whole(c * (0.5f * kLog2e)) : MIX == OSDN_MIX_MEAN ? ab : 0.0f;
        return;
    }
    ab = fmaf(-s, s, s);
    // (k a b first: k alone can be large, and with a large x leave fp32)
    kab = MIX == OSDN_MIX_UNIT ? (keeps(c) ? 1.0f + c : c) * (ab * rsqrt_fast(X == kEnds ? fmaxf(unit_square(c), 1e-37f) : unit_square(c)))
                               : MIX == OSDN_MIX_MEAN ? ab : 0.0f;
}
template <int MIX, int X>
__device__ __forceinline__ float slope_of(float c, float v, float x) {
    float ab, kab;
    slope_factors<MIX, X>(c, ab, kab);
    if (MIX == OSDN_MIX_MEAN) return X == kAny && ab == 0.0f ? 0.0f : ab * (v - x);
    if (X == kAny) {
        const float y = kab == 0.0f ? 0.0f : -kab * x;
        return ab == 0.0f ? y : fmaf(ab, v, y);
    }
    return MIX == OSDN_MIX_SUM ? ab * v : fmaf(ab, v, -kab * x);
}
// whether the gradient of g is zero whatever R is
template <int MIX>
__device__ __forceinline__ bool no_slope(float c) { return c == 0.0f || c <= -zero_from<MIX>(); }

// ------------------------------------------------------------- the short form
// e^-g, and from it a and b = 1 - a
template <int V>
__device__ __forceinline__ Vec<V> exponentials(const Vec<V> &g) {
    Vec<V> e = mul(g, fill<V>(-kLog2e));
#pragma unroll
    for (int i = 0; i < V; ++i) e.v[i] = exp2_fast(e.v[i]);
    return e;
}
template <int V>
__device__ __forceinline__ void sigmoids(const Vec<V> &e, Vec<V> &a, Vec<V> &b) {
    a = add(e, fill<V>(1.0f));
#pragma unroll
    for (int i = 0; i < V; ++i) a.v[i] = rcp_fast(a.v[i]);
    b = mul(e, a);
}
template <int MIX, int V>
__device__ __forceinline__ Vec<V> weight(const Vec<V> &a, const Vec<V> &b) {
    if (MIX == OSDN_MIX_SUM) return fill<V>(1.0f);
    if (MIX == OSDN_MIX_MEAN) return b;
    Vec<V> w = fma(a, b, b);   // 1 - a^2
#pragma unroll
    for (int i = 0; i < V; ++i) w.v[i] = sqrt_fast(w.v[i]);
    return w;
}
// The same factor; v becomes the state after the token.
template <int MIX, int V>
__device__ __forceinline__ Vec<V> slope_and_next(const Vec<V> &a, const Vec<V> &b, const Vec<V> &x, Vec<V> &v) {
    const Vec<V> ab = mul(a, b);
    Vec<V> slope;
    if (MIX == OSDN_MIX_SUM) {
        slope = mul(ab, v);
        v = fma(v, a, x);
    } else if (MIX == OSDN_MIX_MEAN) {
        slope = mul(ab, fma(x, fill<V>(-1.0f), v));
        v = fma(v, a, mul(b, x));
    } else {
        const Vec<V> q = add(ab, b);   // w^2
        Vec<V> k;
#pragma unroll
        for (int i = 0; i < V; ++i) k.v[i] = rsqrt_fast(q.v[i]);
        // (k a b and w first: 1 / w alone can be large, and with a large x leave fp32)
        const Vec<V> kab = mul(mul(ab, k), a);
        slope = fma(mul(kab, x), fill<V>(-1.0f), mul(ab, v));
        v = fma(v, a, mul(mul(q, k), x));
    }
    return slope;
}

}  // namespace gs
}  // namespace osdn
