// decay_attn.cuh -- shared by the kernels of linear attention with a decay
// per head: what one pass over the sequences is given, and how the passes
// split the time axis.
//
// The recurrence of one sequence (b,h), a = decay[h]:
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = S_t q_t          (S [V][K], fp32)
// Its gradients are the same recurrence on other operands: with dO the
// cotangent of o and X_t = a dL/dS_{t+1} (X_T = dL/dS_T), R_t = X_t + dO_t q_t^T,
//     dq = attend(q: dO, k: v, v: k, S0: S0^T)          forwards in time,
//     dk = attend(q: v, k: dO, v: q, S0: dS_T^T)        backwards in time,
//     dv = attend(q: k, k: q, v: dO, S0: dS_T)          backwards in time,
// where the backward direction reads R_t (the carry enters undecayed) and
// leaves dL/dS_0 = a R_1.
#pragma once

#include "osdn_device.cuh"

namespace osdn {
namespace da {

// The [V][K] fp32 state that each sequence starts from (NULL: zeros), in this
// layout or transposed ([K][V]).
struct State {
    const float *p = nullptr;
    int transposed = 0;
};

// One pass: o = attend(q, k, v), K = width of q and k, V = width of v and o.
struct Pass {
    int BH, H, T, K, V, rev;
    const void *q, *k, *v;
    const float *decay;
    State S0;
    float *ST;   // NULL: not written
    void *o;
};

// The time axis in `nch` units of `unit` tokens a sequence; the BH nch units,
// sequence by sequence, are cut into G ranges of nearly equal length, one a
// CTA.  A range that starts inside a sequence starts from the state that the
// range before it leaves: a first pass forms what each range adds to that
// state (its units of the sequence it ends in), a small kernel chains them.
// Backwards in time the units start at the sequence's last token or, with
// `natural`, are those of the forward direction in reverse order (the one
// that may be short then comes first).
struct Split {
    int unit, nch, G, natural = 0;
    __host__ __device__ long long lo(int g, int BH) const {
        return (long long)BH * nch * g / G;
    }
    // tokens before unit u of a sequence, in the pass's direction
    __device__ long long before(int u, int T, int rev) const {
        return rev && natural && u > 0 ? T - (long long)(nch - u) * unit : (long long)u * unit;
    }
};

// a^n to about 46 bits as an unevaluated sum of two fp32 (0^0 = 1), by
// repeated squaring: a state that lives through thousands of decays would
// otherwise carry their common rounding error thousands of times.
struct Pow {
    float hi, lo;
};
__device__ __forceinline__ Pow pow_mul(Pow x, Pow y) {
    const float p = x.hi * y.hi;
    const float e = fmaf(x.hi, y.hi, -p) + fmaf(x.hi, y.lo, x.lo * y.hi);
    const float h = p + e;
    return {h, e - (h - p)};
}
__device__ __forceinline__ Pow decay_pow(float a, unsigned n) {
    Pow r = {1.0f, 0.0f}, b = {a, 0.0f};
    for (; n; n >>= 1) {
        if (n & 1) r = pow_mul(r, b);
        b = pow_mul(b, b);
    }
    return r;
}
__device__ __forceinline__ bool decay_ok(float a) { return a >= 0.0f && a <= 1.0f; }

// Bytes of the ranges' states ([G][V][K] fp32; none for a single range a sequence).
inline size_t split_bytes(const Split &s, int BH, int K, int V) {
    return s.G > BH ? (size_t)s.G * K * V * 4 : 0;
}
// True if every range is one whole sequence.
inline bool unsplit(const Split &s, int BH) { return s.G == BH; }

// states[g], g = 1 .. G-1: in, what range g-1 adds to the state it was given;
// out, the state entering range g (ranges that start a sequence: untouched).
cudaError_t chain_states(const Pass &p, const Split &s, float *states, cudaStream_t stream);

// The token recurrence (fp32 I/O) and the chunked tensor-core form (bf16 I/O).
Split simt_split(int BH, int T, int K, int V);
cudaError_t attend_simt(const Pass &p, void *scratch, int *status, cudaStream_t stream);
Split tc_split(int BH, int T, int K, int V);
cudaError_t attend_tc(const Pass &p, void *scratch, int *status, cudaStream_t stream);

}  // namespace da
}  // namespace osdn
