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
    // The states entering the ranges are in the scratch already, transposed: the pass before ran on
    // the same ranges with k and v exchanged (the same sums of v k^T, so dk can follow dv).
    int given = 0;
};

// The time axis in `nch` units of `unit` tokens a sequence; the BH nch units,
// sequence by sequence, are cut into G ranges of nearly equal length, one a
// CTA (BH nch fits 31 bits: a unit is 4 KB or more of K alone).  A range that starts inside a sequence starts from the state that the
// range before it leaves: a first pass forms what each range adds to that
// state (its units of the sequence it ends in), a small kernel chains them.
// Backwards in time the units start at the sequence's last token or, with
// `natural`, are those of the forward direction in reverse order (the one
// that may be short then comes first).
struct Split {
    int unit, nch, G, natural = 0;
    int each, more;   // range g: each units, and one more for g < more
    __host__ __device__ int lo(int g) const { return g * each + (g < more ? g : more); }
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
// a^n for a weight that is used once (an exponent of a chunk's length, so that rounding
// n log2(a) costs 1e-7 where the weight counts), from log2(a); a = 0: 0^0 = 1.
__device__ __forceinline__ float decay_log2(float a) { return fmaxf(log2f(a), -1e30f); }
__device__ __forceinline__ float weight(float l2, int n) { return exp2f(l2 * (float)n); }
__device__ __forceinline__ bool decay_ok(float a) { return a >= 0.0f && a <= 1.0f; }

// The units cut into G ranges.
inline Split make_split(int unit, int natural, int BH, int T, int G) {
    Split s;
    s.unit = unit;
    s.natural = natural;
    s.nch = (int)(((long long)T + unit - 1) / unit);
    s.G = G;
    const long long n = (long long)BH * s.nch;
    s.each = (int)(n / G);
    s.more = (int)(n % G);
    return s;
}
// Bytes of the ranges' states ([G][V][K] fp32; none for a single range a sequence).
inline size_t split_bytes(const Split &s, int BH, int K, int V) {
    return s.G > BH ? (size_t)s.G * K * V * 4 : 0;
}
// True if every range is one whole sequence.
inline bool unsplit(const Split &s, int BH) { return s.G == BH; }

// states[g], g = 1 .. G-1: in, what range g-1 adds to the state it was given;
// out, the state entering range g (ranges that start a sequence: untouched).
cudaError_t chain_states(const Pass &p, const Split &s, float *states, cudaStream_t stream);

// The three launches of a split pass overlap: each may start while the one before still runs, does
// what does not depend on it, and waits (dependency_wait) for its completion before the rest.
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dependents_may_start() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <typename... P, typename... A>
cudaError_t launch_overlapped(bool overlap, void (*kernel)(P...), dim3 grid, int block, size_t smem,
                              cudaStream_t stream, const A &...args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid;
    c.blockDim = dim3(block);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = overlap ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, args...);
}

// The token recurrence (fp32 I/O) and the chunked tensor-core form (bf16 I/O).
Split simt_split(int BH, int T, int K, int V);
cudaError_t attend_simt(const Pass &p, void *scratch, int *status, cudaStream_t stream);
Split tc_split(int BH, int T, int K, int V);
cudaError_t attend_tc(const Pass &p, void *scratch, int *status, cudaStream_t stream);

}  // namespace da
}  // namespace osdn
