// group_norm.cu -- group norm with an activation, channels last, and its
// gradients: the norm behind a linear-attention layer.
//
// Per token and group of D channels (a group is a head),
//     m = mean(x),  r = 1 / sqrt(mean((x - m)^2) + eps),  x^ = (x - m) r,
//     z = weight x^ + bias,   y = act(z), or z act(gate) where a gate is given
// with y and gate [B][T][G D], and x either [B][T][G D] or, as the attention
// writes it, [B][G][T][D].  Statistics belong to one token alone (the norm
// stays causal) and are taken in two steps from registers, the mean (of the
// values less the group's first, so that a large mean costs no accuracy) and
// then the variance; all arithmetic is fp32.
//
// Gradients, with dz = dy act'(z) (no gate) or dy act(gate):
//     dgate = dy z act'(gate),   dweight = sum dz x^,   dbias = sum dz,
//     h = dz weight,   dx = r (h - mean(h) - x^ mean(h x^)).
//
// Every tensor is read and written once, so both directions are HBM-bound.
// L lanes (the power of two at or above D/8, at most 32) hold a group, eight
// channels a lane in 16-byte pieces; where a group is short, neighbouring
// groups of the token stand next to it so that 16 lanes read 256 bytes in a
// row.  A CTA keeps to its groups and walks tokens: a lane's weight and bias
// (and in the backward pass the sums of dweight and dbias) stay in registers,
// and the next token's pieces are on their way while one is computed.  The
// sums are joined over the CTA in shared memory and over CTAs by a second
// kernel, in a fixed order (no atomics).
//
// Measured (bf16, gated silu, D = 128): 43 us at 2x16x8192 (4.7 TB/s, 0.69 of
// the measured copy bandwidth; a thread per group without the walk: 85 us),
// the gradients 44 us at 3x16x2731 (3.8 TB/s, 0.56; 77 us).  In fp32 with D =
// 256 both reach 5.4 TB/s; in bf16 a byte costs twice the instructions, and
// instruction issue is what bounds it (0.70 of the issue slots forward, 0.58
// backward, at 44% and 24% of the warps: 64 and 120 registers a thread), with
// 256-byte runs of memory behind it.  Two tokens ahead in registers (50
// and 64 us), four in shared memory by asynchronous copies (43 and 43 us, but
// fp32 57 us) and whole tokens side by side (54 and 68 us) gained nothing.
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

// Eight channels as they lie in memory.
template <typename io_t>
struct Raw {
    uint4 u[sizeof(io_t) / 2];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (int)sizeof(io_t) / 2; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void load(const io_t *p) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(io_t) / 2; ++i) u[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    // in pairs: the arithmetic below is packed (two fp32 an instruction), since with an activation
    // the gradients issue more instructions than the loads take time
    __device__ __forceinline__ void wide(float2 (&x)[4]) const {
        if constexpr (sizeof(io_t) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                x[2 * i] = make_float2(__uint_as_float(u[i].x), __uint_as_float(u[i].y));
                x[2 * i + 1] = make_float2(__uint_as_float(u[i].z), __uint_as_float(u[i].w));
            }
        } else {
            const uint32_t w[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        }
    }
};
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ void load8(const float *p, float2 (&x)[4]) {
    Raw<float> r;
    r.load(p);
    r.wide(x);
}
__device__ __forceinline__ void store8(float *p, const float2 (&x)[4]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
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

// 1 / (1 + e^-u) from the hardware's base-2 exponential and reciprocal (2 ulp each; e^-u = inf: 0).
__device__ __forceinline__ float2 sigmoid(float2 u) {
    float2 e = __fmul2_rn(u, both(-1.4426950408889634f)), s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
    e = __fadd2_rn(e, both(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
    return s;
}
// act(u) for eight values, and with DER its derivative; the choice is made once for all eight.
template <bool DER>
__device__ __forceinline__ void act8(int act, const float2 (&u)[4], float2 (&f)[4], float2 (&d)[4]) {
    if (act == kNone) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f[e] = u[e];
            if (DER) d[e] = both(1.0f);
        }
    } else if (act == kSilu) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 s = sigmoid(u[e]);
            f[e] = __fmul2_rn(u[e], s);
            if (DER) d[e] = __ffma2_rn(f[e], __ffma2_rn(s, both(-1.0f), both(1.0f)), s);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 s = sigmoid(u[e]);
            f[e] = s;
            if (DER) d[e] = __fmul2_rn(s, __ffma2_rn(s, both(-1.0f), both(1.0f)));
        }
    }
}

// The walk of a thread over its CTA's tokens: slots of GPB groups of L lanes,
// 16 lanes or more a slot; a slot's token, its places in x and in y (and gate).
template <int L>
struct Walk {
    static constexpr int GPB = L < 16 ? 16 / L : 1;   // groups side by side
    static constexpr int S = kThreads / (L * GPB);    // tokens at a time
    int l, g;
    bool in_range;      // the group exists
    long long tok, hi, b;
    int t;
    __device__ __forceinline__ Walk(const Params &p) {
        l = threadIdx.x % L;
        g = blockIdx.x * GPB + threadIdx.x / L % GPB;
        in_range = g < p.G;
        tok = p.tokens * blockIdx.y / p.splits + threadIdx.x / (L * GPB);
        hi = p.tokens * (blockIdx.y + 1) / p.splits;
        b = p.heads_first ? tok / p.T : 0;
        t = p.heads_first ? (int)(tok - b * p.T) : 0;
    }
    __device__ __forceinline__ bool live() const { return in_range && tok < hi; }
    __device__ __forceinline__ size_t at_y(const Params &p) const { return ((size_t)tok * p.G + g) * p.D; }
    __device__ __forceinline__ size_t at_x(const Params &p) const {
        return p.heads_first ? (((size_t)b * p.G + g) * p.T + t) * p.D : at_y(p);
    }
    __device__ __forceinline__ void next(const Params &p) {
        tok += S;
        if (!p.heads_first) return;
        t += S;
        while (t >= p.T) {
            t -= p.T;
            ++b;
        }
    }
    // CTAs' iterations: the same for all threads, so that shuffles see whole warps
    __device__ __forceinline__ static int rounds(const Params &p) {
        const long long n = p.tokens * (blockIdx.y + 1) / p.splits - p.tokens * blockIdx.y / p.splits;
        return (int)((n + S - 1) / S);
    }
};

// 1 / sqrt(var + eps) of a group; v leaves as x - mean.  The mean is taken of x less the group's
// first value, so that rounding it is relative to the spread.
template <int L, int N>
__device__ __forceinline__ float normalise(const Params &p, int l, float2 (&v)[N][4]) {
    const float inv = 1.0f / (float)p.D;
    const float x0 = __shfl_sync(kFullMask, v[0][0].x, 0, L);
    float2 sum = both(0.0f), sq = both(0.0f);
#pragma unroll
    for (int n = 0; n < N; ++n) {   // (channels past D hold zeros, and keep them)
        const float2 m = both((n * L + l) * 8 < p.D ? -x0 : 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[n][e] = __fadd2_rn(v[n][e], m);
            sum = __fadd2_rn(sum, v[n][e]);
        }
    }
    const float mean = group_sum<L>(sum.x + sum.y) * inv;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const float2 m = both((n * L + l) * 8 < p.D ? -mean : 0.0f);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v[n][e] = __fadd2_rn(v[n][e], m);
            sq = __ffma2_rn(v[n][e], v[n][e], sq);
        }
    }
    return rsqrtf(fmaf(group_sum<L>(sq.x + sq.y), inv, p.eps));
}

// A lane's N pieces of eight channels: piece n starts at channel (n L + l) 8.
template <typename io_t, int L, int N>
__global__ void __launch_bounds__(kThreads) group_norm_kernel(Params p) {
    Walk<L> w(p);
    const int l = w.l;
    float2 wt[N][4], bs[N][4];
    Raw<io_t> rx[N], rg[N];
    auto fetch = [&] {
        const bool live = w.live();
        const io_t *x = static_cast<const io_t *>(p.x) + (live ? w.at_x(p) : 0);
        const io_t *gate = static_cast<const io_t *>(p.gate) + (live ? w.at_y(p) : 0);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            rx[n].zero();
            rg[n].zero();
            if (live && c < p.D) {
                rx[n].load(x + c);
                if (p.gate) rg[n].load(gate + c);
            }
        }
    };
    fetch();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wt[n][e] = both(1.0f);
            bs[n][e] = both(0.0f);
        }
        if (w.in_range && c < p.D && p.weight) load8(p.weight + (size_t)w.g * p.D + c, wt[n]);
        if (w.in_range && c < p.D && p.bias) load8(p.bias + (size_t)w.g * p.D + c, bs[n]);
    }
    for (int i = Walk<L>::rounds(p); i > 0; --i) {
        float2 v[N][4], gt[N][4];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            rx[n].wide(v[n]);
            rg[n].wide(gt[n]);
        }
        const bool live = w.live();
        io_t *y = static_cast<io_t *>(p.y) + (live ? w.at_y(p) : 0);
        w.next(p);
        if (i > 1) fetch();   // on its way while this token is computed
        const float r = normalise<L, N>(p, l, v);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            if (!live || c >= p.D) continue;
            float2 z[4], o[4], none[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = __ffma2_rn(__fmul2_rn(v[n][e], both(r)), wt[n][e], bs[n][e]);
            if (p.gate) {
                act8<false>(p.act, gt[n], o, none);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = __fmul2_rn(o[e], z[e]);
            } else {
                act8<false>(p.act, z, o, none);
            }
            store8(y + c, o);
        }
    }
}

template <typename io_t, int L, int N>
__global__ void __launch_bounds__(kThreads) group_norm_backward_kernel(Params p) {
    extern __shared__ float red[];    // [S][GPB][2][N L 8]
    constexpr int W = N * L * 8, S = Walk<L>::S, GPB = Walk<L>::GPB;
    Walk<L> w(p);
    const int l = w.l;
    const float inv = 1.0f / (float)p.D;
    float2 wt[N][4], bs[N][4], aw[N][4], ab[N][4];
    Raw<io_t> rx[N], rd[N], rg[N];
    auto fetch = [&] {
        const bool live = w.live();
        const size_t xa = live ? w.at_x(p) : 0, ya = live ? w.at_y(p) : 0;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            rx[n].zero();
            rd[n].zero();
            rg[n].zero();
            if (live && c < p.D) {
                rx[n].load(static_cast<const io_t *>(p.x) + xa + c);
                rd[n].load(static_cast<const io_t *>(p.dy) + ya + c);
                if (p.gate) rg[n].load(static_cast<const io_t *>(p.gate) + ya + c);
            }
        }
    };
    fetch();
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            wt[n][e] = both(1.0f);
            bs[n][e] = aw[n][e] = ab[n][e] = both(0.0f);
        }
        if (w.in_range && c < p.D && p.weight) load8(p.weight + (size_t)w.g * p.D + c, wt[n]);
        if (w.in_range && c < p.D && p.bias) load8(p.bias + (size_t)w.g * p.D + c, bs[n]);
    }
    for (int i = Walk<L>::rounds(p); i > 0; --i) {
        float2 v[N][4], d[N][4], gt[N][4];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            rx[n].wide(v[n]);
            rd[n].wide(d[n]);
            rg[n].wide(gt[n]);
        }
        const bool live = w.live();
        const size_t xa = live ? w.at_x(p) : 0, ya = live ? w.at_y(p) : 0;
        w.next(p);
        if (i > 1) fetch();   // on its way while this token is computed
        const float r = normalise<L, N>(p, l, v);
        float2 h1 = both(0.0f), h2 = both(0.0f);
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float2 z[4], f[4], df[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[n][e] = __fmul2_rn(v[n][e], both(r));
                z[e] = __ffma2_rn(v[n][e], wt[n][e], bs[n][e]);
            }
            if (p.gate) {
                act8<true>(p.act, gt[n], f, df);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    gt[n][e] = __fmul2_rn(__fmul2_rn(d[n][e], z[e]), df[e]);
                    d[n][e] = __fmul2_rn(d[n][e], f[e]);
                }
            } else {
                act8<true>(p.act, z, f, df);
#pragma unroll
                for (int e = 0; e < 4; ++e) d[n][e] = __fmul2_rn(d[n][e], df[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // d is dz here, then h
                aw[n][e] = __ffma2_rn(d[n][e], v[n][e], aw[n][e]);
                ab[n][e] = __fadd2_rn(ab[n][e], d[n][e]);
                d[n][e] = __fmul2_rn(d[n][e], wt[n][e]);
                h1 = __fadd2_rn(h1, d[n][e]);
                h2 = __ffma2_rn(d[n][e], v[n][e], h2);
            }
        }
        const float hs = group_sum<L>(h1.x + h1.y) * -inv, hx = group_sum<L>(h2.x + h2.y) * -inv;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * L + l) * 8;
            if (!live || c >= p.D) continue;
            float2 dx[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                dx[e] = __fmul2_rn(both(r), __ffma2_rn(v[n][e], both(hx), __fadd2_rn(d[n][e], both(hs))));
            store8(static_cast<io_t *>(p.dx) + xa + c, dx);
            if (p.gate) store8(static_cast<io_t *>(p.dgate) + ya + c, gt[n]);
        }
    }
    if (!p.part) return;
    float *mine = red + (size_t)(threadIdx.x / L) * 2 * W;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * L + l) * 8;
        store8(mine + c, aw[n]);
        store8(mine + W + c, ab[n]);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < GPB * 2 * p.D; i += kThreads) {
        const int gi = i / (2 * p.D), at = i % (2 * p.D), c = at < p.D ? at : W + at - p.D;
        const int g = blockIdx.x * GPB + gi;
        float s = 0.0f;
        for (int k = 0; k < S; ++k) s += red[(size_t)(k * GPB + gi) * 2 * W + c];
        if (g < p.G) p.part[((size_t)blockIdx.y * p.G + g) * 2 * p.D + at] = s;
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
    constexpr int GPB = Walk<L>::GPB;
    group_norm_kernel<io_t, L, N><<<dim3((p.G + GPB - 1) / GPB, p.splits), kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename io_t, int L, int N>
cudaError_t backward_t(const Params &p, cudaStream_t stream) {
    constexpr int GPB = Walk<L>::GPB;
    const int smem = (kThreads / L) * 2 * N * L * 8 * 4;   // 16 KB a piece
    group_norm_backward_kernel<io_t, L, N><<<dim3((p.G + GPB - 1) / GPB, p.splits), kThreads, smem, stream>>>(p);
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

// CTAs that share a block of groups' tokens: enough for `per_sm` CTAs a SM
// over all blocks, while each still has `least` tokens.
int token_splits(long long tokens, int G, int D, int per_sm, int least) {
    const int lanes = D <= 8 ? 1 : D <= 16 ? 2 : D <= 32 ? 4 : D <= 64 ? 8 : 16;
    const long long blocks = (G + 16 / lanes - 1) / (16 / lanes);
    long long s = (152LL * per_sm + blocks - 1) / blocks;
    if (s > (tokens + least - 1) / least) s = (tokens + least - 1) / least;
    return (int)(s < 1 ? 1 : s > 65535 ? 65535 : s);
}
int backward_splits(long long tokens, int G, int D) { return token_splits(tokens, G, D, 4, 64); }

}  // namespace gn

size_t group_norm_backward_scratch_bytes(int B, int G, int T, int D) {
    return (size_t)gn::backward_splits((long long)B * T, G, D) * G * 2 * D * 4;
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
    p.splits = gn::token_splits(p.tokens, G, D, 8, 16);
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
    p.splits = gn::backward_splits(p.tokens, G, D);
    p.part = (dweight || dbias) ? static_cast<float *>(scratch) : nullptr;
    cudaError_t e = io == OSDN_F32 ? gn::run_d<float, true>(p, stream)
                                   : gn::run_d<__nv_bfloat16, true>(p, stream);
    if (e != cudaSuccess || !p.part) return e;
    gn::group_norm_join_kernel<<<(unsigned)((2 * C + 31) / 32), 256, 0, stream>>>(
        G, D, p.splits, p.part, dweight, dbias);
    return cudaGetLastError();
}

}  // namespace osdn
