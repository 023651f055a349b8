// group_norm.cu -- group norm with an activation, channels last, and its
// gradients: the norm behind a linear-attention layer.
//
// Per token and group of D channels (a group is a head),
//     m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  x^ = (x - m) r,
//     z = weight x^ + bias,   y = act(z), or z act(gate) where a gate is given
// with y and gate [B][T][G D], and x either [B][T][G D] or, as the attention
// writes it, [B][G][T][D].  Statistics belong to one token alone (the norm
// stays causal) and are taken in two steps from registers, mean first, the
// rest that its rounding leaves in x - m taken off again, so that a large
// mean costs no accuracy; all arithmetic is fp32.
//
// Gradients, with dz = dy act'(z) (no gate) or dy act(gate):
//     dgate = dy z act'(gate),   dweight = sum dz x^,   dbias = sum dz,
//     h = dz weight,   dx = r (h - mean(h) - x^ mean(h x^)).
//
// Every tensor is read and written once, so both directions are HBM-bound.
// L lanes (the power of two at or above D/8, at most 32) hold a group, eight
// channels a lane in 16-byte pieces, so a warp covers 32/L groups and its
// loads are whole 128-byte lines for D >= 64 in bf16.  In the backward pass
// a CTA keeps to one group g and walks tokens, so that a lane's channels
// stay the same and dweight and dbias add up in its registers; they are
// joined over the CTA in shared memory and over CTAs by a second kernel, in
// a fixed order (no atomics).
#include "osdn_device.cuh"

namespace osdn {
namespace gn {

enum { kNone = 0, kSilu = 1, kSigmoid = 2 };
constexpr int kThreads = 256;

struct Params {
    int B, G, T, D, heads_first, act;
    float eps;
    const void *x, *gate, *dy;
    const float *weight, *bias;
    void *y, *dx, *dgate;
    float *part;        // [splits][G][2][D]: dweight and dbias of each CTA
    long long tokens;   // B T
    int splits;
};

__device__ __forceinline__ void load8(const float *p, float (&x)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <int L>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = L / 2; m; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
    return v;
}

__device__ __forceinline__ float sigmoid(float u) { return __frcp_rn(1.0f + __expf(-u)); }
__device__ __forceinline__ float act_of(float u, int act) {
    return act == kNone ? u : act == kSilu ? u * sigmoid(u) : sigmoid(u);
}
// act(u) and its derivative
__device__ __forceinline__ void act_both(float u, int act, float &f, float &d) {
    if (act == kNone) {
        f = u;
        d = 1.0f;
        return;
    }
    const float s = sigmoid(u);
    f = act == kSilu ? u * s : s;
    d = act == kSilu ? s * (1.0f + u * (1.0f - s)) : s * (1.0f - s);
}

// Where token `tok` (b T + t) of group g starts in x; in y and gate it is
// (tok G + g) D.
__device__ __forceinline__ size_t x_at(const Params &p, long long tok, int g) {
    if (!p.heads_first) return ((size_t)tok * p.G + g) * p.D;
    const long long b = tok / p.T, t = tok - b * p.T;
    return (((size_t)b * p.G + g) * p.T + t) * p.D;
}

// A lane's N pieces of eight channels: piece n starts at channel (n L + l) 8.
template <typename io_t, int L, int N>
__global__ void __launch_bounds__(kThreads) group_norm_kernel(Params p) {
    constexpr int GPC = kThreads / L;   // groups a CTA
    const int l = threadIdx.x % L;
    const long long at = (long long)blockIdx.x * GPC + threadIdx.x / L, n_all = p.tokens * p.G;
    const bool live = at < n_all;
    // consecutive groups lie next to each other in x: by token, or by head
    long long tok;
    int g;
    if (p.heads_first) {
        const long long bg = at / p.T;
        g = (int)(bg % p.G);
        tok = bg / p.G * p.T + at % p.T;
    } else {
        tok = at / p.G;
        g = (int)(at % p.G);
    }
    const io_t *x = static_cast<const io_t *>(p.x) + (size_t)at * p.D;
    const size_t ya = ((size_t)tok * p.G + g) * p.D;
    const float inv = 1.0f / (float)p.D;
    float v[N][8], gt[N][8];
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
        const bool in = live && c < p.D;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[n][e] = gt[n][e] = 0.0f;
        if (in) load8(x + c, v[n]);
        if (in && p.gate) load8(static_cast<const io_t *>(p.gate) + ya + c, gt[n]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += v[n][e];
    }
    const float mean = group_sum<L>(sum) * inv;
    float sq = 0.0f, off = 0.0f;   // off: what rounding left of the mean
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const bool in = (n * L + l) * 8 < p.D;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[n][e] = in ? v[n][e] - mean : 0.0f;
            sq = fmaf(v[n][e], v[n][e], sq);
            off += v[n][e];
        }
    }
    off = group_sum<L>(off) * inv;
    const float r = 1.0f / sqrtf(fmaxf(fmaf(-off, off, group_sum<L>(sq) * inv), 0.0f) + p.eps);
    if (!live) return;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
        if (c >= p.D) continue;
        float w[8], b[8], y[8];
        if (p.weight) load8(p.weight + (size_t)g * p.D + c, w);
        if (p.bias) load8(p.bias + (size_t)g * p.D + c, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float z = (v[n][e] - off) * r;
            if (p.weight) z *= w[e];
            if (p.bias) z += b[e];
            y[e] = p.gate ? z * act_of(gt[n][e], p.act) : act_of(z, p.act);
        }
        store8(static_cast<io_t *>(p.y) + ya + c, y);
    }
}

template <typename io_t, int L, int N>
__global__ void __launch_bounds__(kThreads) group_norm_backward_kernel(Params p) {
    constexpr int S = kThreads / L;   // tokens a CTA holds at a time
    extern __shared__ float red[];    // [S][2][N L 8]
    const int l = threadIdx.x % L, slot = threadIdx.x / L, g = blockIdx.x;
    const float inv = 1.0f / (float)p.D;
    float w[N][8], b[N][8], aw[N][8], ab[N][8];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[n][e] = 1.0f;
            b[n][e] = aw[n][e] = ab[n][e] = 0.0f;
        }
        if (c < p.D && p.weight) load8(p.weight + (size_t)g * p.D + c, w[n]);
        if (c < p.D && p.bias) load8(p.bias + (size_t)g * p.D + c, b[n]);
    }
    const long long lo = p.tokens * blockIdx.y / p.splits, hi = p.tokens * (blockIdx.y + 1) / p.splits;
    for (long long t0 = lo; t0 < hi; t0 += S) {   // uniform over the CTA: the shuffles see whole warps
        const long long tok = t0 + slot;
        const bool live = tok < hi;
        const size_t xa = live ? x_at(p, tok, g) : 0, ya = ((size_t)tok * p.G + g) * p.D;
        float v[N][8], d[N][8], gt[N][8];
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            const bool in = live && c < p.D;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[n][e] = d[n][e] = gt[n][e] = 0.0f;
            if (in) {
                load8(static_cast<const io_t *>(p.x) + xa + c, v[n]);
                load8(static_cast<const io_t *>(p.dy) + ya + c, d[n]);
                if (p.gate) load8(static_cast<const io_t *>(p.gate) + ya + c, gt[n]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[n][e];
        }
        const float mean = group_sum<L>(sum) * inv;
        float sq = 0.0f, off = 0.0f;   // off: what rounding left of the mean
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const bool in = (n * L + l) * 8 < p.D;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[n][e] = in ? v[n][e] - mean : 0.0f;
                sq = fmaf(v[n][e], v[n][e], sq);
                off += v[n][e];
            }
        }
        off = group_sum<L>(off) * inv;
        const float r = 1.0f / sqrtf(fmaxf(fmaf(-off, off, group_sum<L>(sq) * inv), 0.0f) + p.eps);
        float hs = 0.0f, hx = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float xh = (v[n][e] - off) * r, z = fmaf(xh, w[n][e], b[n][e]);
                float f, df, dz;
                if (p.gate) {
                    act_both(gt[n][e], p.act, f, df);
                    gt[n][e] = d[n][e] * z * df;
                    dz = d[n][e] * f;
                } else {
                    act_both(z, p.act, f, df);
                    dz = d[n][e] * df;
                }
                aw[n][e] = fmaf(dz, xh, aw[n][e]);
                ab[n][e] += dz;
                const float h = dz * w[n][e];
                hs += h;
                hx = fmaf(h, xh, hx);
                v[n][e] = xh;
                d[n][e] = h;
            }
        hs = group_sum<L>(hs) * inv;
        hx = group_sum<L>(hx) * inv;
        if (!live) continue;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            if (c >= p.D) continue;
            float dx[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) dx[e] = r * (d[n][e] - hs - v[n][e] * hx);
            store8(static_cast<io_t *>(p.dx) + xa + c, dx);
            if (p.gate) store8(static_cast<io_t *>(p.dgate) + ya + c, gt[n]);
        }
    }
    if (!p.part) return;
    constexpr int W = N * L * 8;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
        store8(red + (size_t)slot * 2 * W + c, aw[n]);
        store8(red + (size_t)slot * 2 * W + W + c, ab[n]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
        const int c = i < p.D ? i : W + i - p.D;
        float s = 0.0f;
        for (int k = 0; k < S; ++k) s += red[(size_t)k * 2 * W + c];
        p.part[((size_t)blockIdx.y * p.G + g) * 2 * p.D + i] = s;
    }
}

// dweight and dbias [G D] from the CTAs' partial sums: a warp takes 32
// channels of either, eight warps share the splits.
__global__ void __launch_bounds__(256)
group_norm_join_kernel(int G, int D, int splits, const float *part, float *dweight, float *dbias) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + lane, n = 2LL * G * D;
    float s = 0.0f;
    if (i < n)
        for (int k = warp; k < splits; k += 8) s += part[(size_t)k * n + i];
    red[warp][lane] = s;
    __syncthreads();
    if (warp || i >= n) return;
#pragma unroll
    for (int k = 1; k < 8; ++k) s += red[k][lane];
    const int g = (int)(i / (2 * D)), c = (int)(i % (2 * D));
    if (c < D) {
        if (dweight) dweight[(size_t)g * D + c] = s;
    } else if (dbias) {
        dbias[(size_t)g * D + c - D] = s;
    }
}

__global__ void zero_kernel(long long n, float *a, float *b) {
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= n) return;
    if (a) a[i] = 0.0f;
    if (b) b[i] = 0.0f;
}

template <typename io_t, int L, int N>
cudaError_t forward_t(const Params &p, cudaStream_t stream) {
    const long long n = p.tokens * p.G, per = kThreads / L;
    group_norm_kernel<io_t, L, N><<<(unsigned)((n + per - 1) / per), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename io_t, int L, int N>
cudaError_t backward_t(const Params &p, cudaStream_t stream) {
    const int smem = (kThreads / L) * 2 * N * L * 8 * 4;   // 16 KB a piece
    group_norm_backward_kernel<io_t, L, N><<<dim3(p.G, p.splits), kThreads, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename io_t, bool BWD, int L, int N>
cudaError_t run_t(const Params &p, cudaStream_t stream) {
    if (BWD) return backward_t<io_t, L, N>(p, stream);
    return forward_t<io_t, L, N>(p, stream);
}
template <typename io_t, bool BWD>
cudaError_t run_d(const Params &p, cudaStream_t stream) {
    const int pieces = p.D / 8;
    if (pieces <= 1) return run_t<io_t, BWD, 1, 1>(p, stream);
    if (pieces <= 2) return run_t<io_t, BWD, 2, 1>(p, stream);
    if (pieces <= 4) return run_t<io_t, BWD, 4, 1>(p, stream);
    if (pieces <= 8) return run_t<io_t, BWD, 8, 1>(p, stream);
    if (pieces <= 16) return run_t<io_t, BWD, 16, 1>(p, stream);
    if (pieces <= 32) return run_t<io_t, BWD, 32, 1>(p, stream);
    return run_t<io_t, BWD, 32, 2>(p, stream);
}

// CTAs a group in the backward pass: enough for about four a SM over all
// groups, while each still has 64 tokens to add up.
int backward_splits(long long tokens, int G) {
    long long s = (152LL * 4 + G - 1) / G;
    if (s > (tokens + 63) / 64) s = (tokens + 63) / 64;
    return (int)(s < 1 ? 1 : s > 65535 ? 65535 : s);
}

}  // namespace gn

size_t group_norm_backward_scratch_bytes(int B, int G, int T, int D) {
    return (size_t)gn::backward_splits((long long)B * T, G) * G * 2 * D * 4;
}

cudaError_t group_norm_launch(int io, int B, int G, int T, int D, int heads_first, const void *x,
                              const float *weight, const float *bias, const void *gate, int act,
                              float eps, void *y, cudaStream_t stream) {
    gn::Params p = {};
    p.B = B; p.G = G; p.T = T; p.D = D;
    p.heads_first = heads_first;
    p.act = act;
    p.eps = eps;
    p.x = x;
    p.gate = gate;
    p.weight = weight;
    p.bias = bias;
    p.y = y;
    p.tokens = (long long)B * T;
    return io == OSDN_F32 ? gn::run_d<float, false>(p, stream)
                          : gn::run_d<__nv_bfloat16, false>(p, stream);
}

cudaError_t group_norm_backward_launch(int io, int B, int G, int T, int D, int heads_first,
                                       const void *x, const void *dy, const float *weight,
                                       const float *bias, const void *gate, int act, float eps,
                                       void *dx, void *dgate, float *dweight, float *dbias,
                                       void *scratch, cudaStream_t stream) {
    gn::Params p = {};
    p.B = B; p.G = G; p.T = T; p.D = D;
    p.heads_first = heads_first;
    p.act = act;
    p.eps = eps;
    p.x = x;
    p.gate = gate;
    p.dy = dy;
    p.weight = weight;
    p.bias = bias;
    p.dx = dx;
    p.dgate = dgate;
    p.tokens = (long long)B * T;
    const long long C = (long long)G * D;
    if (p.tokens == 0) {
        if (dweight || dbias)
            gn::zero_kernel<<<(unsigned)((C + 255) / 256), 256, 0, stream>>>(C, dweight, dbias);
        return cudaGetLastError();
    }
    p.splits = gn::backward_splits(p.tokens, G);
    p.part = (dweight || dbias) ? static_cast<float *>(scratch) : nullptr;
    cudaError_t e = io == OSDN_F32 ? gn::run_d<float, true>(p, stream)
                                   : gn::run_d<__nv_bfloat16, true>(p, stream);
    if (e != cudaSuccess || !p.part) return e;
    gn::group_norm_join_kernel<<<(unsigned)((2 * C + 31) / 32), 256, 0, stream>>>(
        G, D, p.splits, p.part, dweight, dbias);
    return cudaGetLastError();
}

}  // namespace osdn
