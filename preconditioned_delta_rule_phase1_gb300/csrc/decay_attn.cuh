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

// A [rows][cols] fp32 state of each sequence at `p` (NULL: zeros, or not
// written), in this layout or transposed ([cols][rows]).
struct State {
    float *p = nullptr;
    int transposed = 0;
};

// One pass: o = attend(q, k, v), K = width of q and k, V = width of v and o.
struct Pass {
    int BH, H, T, K, V, rev;
    const void *q, *k, *v;
    const float *decay;
    State S0, ST;
    void *o;
};

// The time axis in `nch` units of `unit` tokens a sequence; the BH nch units,
// sequence by sequence, are cut into G ranges of nearly equal length, one a
// CTA.  A range that starts inside a sequence starts from the state that the
// range before it leaves: a first pass forms what each range adds to that
// state (its units of the sequence it ends in), a small kernel chains them.
struct Split {
    int unit, nch, G;
    __host__ __device__ long long lo(int g, int BH) const {
        return (long long)BH * nch * g / G;
    }
};

// a^n for n >= 0 from log2(a) (a = 0: 0^0 = 1).
__device__ __forceinline__ float decay_log2(float a) { return fmaxf(log2f(a), -1e30f); }
__device__ __forceinline__ float decay_pow(float l2, float n) { return exp2f(n * l2); }
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

Split simt_split(int BH, int T, int K, int V);
cudaError_t attend_simt(int io, const Pass &p, void *scratch, int *status, cudaStream_t stream);

}  // namespace da
}  // namespace osdn
