// gated_scan.cuh -- the gate of the recurrence in gated_scan.cu: a = sigmoid(g),
// the weight w(a) of the input and their derivatives.
#pragma once

#include "osdn_device.cuh"

namespace osdn {
namespace gs {

template <int M>
struct Mix {
    static constexpr int value = M;
};

// c v, where a factor c that is exactly zero hides v whatever it holds (an infinity or NaN behind a
// gate that is shut).
__device__ __forceinline__ float hide(float c, float v) { return c == 0.0f ? 0.0f : c * v; }

// Both sigmoids come from e^-|g|, so that neither loses digits where it is small:
//     a = sigmoid(g),  b = 1 - a = sigmoid(-g),  and b (1 + a) = 1 - a^2.
struct Gate {
    float a, b;
    __device__ __forceinline__ explicit Gate(float g) {
        const float e = __expf(-fabsf(g)), large = __fdividef(1.0f, 1.0f + e), small = e * large;
        a = g >= 0.0f ? large : small;
        b = g >= 0.0f ? small : large;
        if (g != g) a = b = g;
    }
    template <int MIX>
    __device__ __forceinline__ float weight() const {
        return MIX == OSDN_MIX_SUM ? 1.0f : MIX == OSDN_MIX_MEAN ? b : sqrtf(b * (1.0f + a));
    }
    // a v: as v - b v where b is the smaller, since a rounded to fp32 says too little of 1 - a for
    // memories of thousands of tokens
    __device__ __forceinline__ float decay(float v) const { return b < a ? fmaf(-b, v, v) : hide(a, v); }
    // a s + w x
    template <int MIX>
    __device__ __forceinline__ float next(float s, float x) const {
        return decay(s) + hide(weight<MIX>(), x);
    }
    // With r the cotangent of the state after this token and s the state before it: the gradients
    // w r of x and r (a b s + w' x) of g.  w' is 0, -a b, or -a^2 sqrt(b / (1 + a)), which is
    // -a / w times a b without its division by zero at a = 1.
    template <int MIX>
    __device__ __forceinline__ void gradients(float r, float s, float x, float &dx, float &dg) const {
        dx = weight<MIX>() * r;
        float d = hide(a * b, s);
        if (MIX == OSDN_MIX_MEAN) d -= hide(a * b, x);
        if (MIX == OSDN_MIX_UNIT) d -= hide(a * a * sqrtf(b / (1.0f + a)), x);
        dg = r * d;
    }
};

}  // namespace gs
}  // namespace osdn
