// layer_norm.cu -- layer norm over whole rows, with the addition to the
// residual stream in front of it, and its gradients.  Per row of C values,
//     s = x + residual,  r = 1 / sqrt(mean((s - m)^2) + eps),  x^ = (s - m) r,
//     y = weight x^ + bias
//     u = dy weight,  dx = r (u - mean(u) - x^ mean(u x^)) + ds
//     dweight = sum over rows of dy x^,   dbias = sum over rows of dy
// Rows are read and written once, so HBM bounds both directions.  A row is
// held in registers, N pieces of E neighbouring channels a thread (16 bytes
// where rows keep 16-byte boundaries, else one word or one element), by one
// warp where it is short and by up to 32 otherwise.  Statistics are taken in
// two steps, the mean of the values less the row's first, so that a large mean
// costs no accuracy, and then the variance; all arithmetic is fp32.
#include <algorithm>

#include "decay_attn.cuh"
#include "ptx.cuh"

namespace osdn {
namespace ln {

namespace {

// E neighbouring channels as they lie in memory.
template <int BYTES> struct Word;
template <> struct Word<16> { typedef uint4 type; };
template <> struct Word<4> { typedef unsigned type; };
template <> struct Word<2> { typedef unsigned short type; };

template <typename io_t, int E>
struct Piece {
    typedef typename Word<E * (int)sizeof(io_t)>::type raw_t;
    raw_t u;
    __device__ __forceinline__ void zero() { u = raw_t(); }
    __device__ __forceinline__ void load(const io_t *p) { u = *reinterpret_cast<const raw_t *>(p); }
    __device__ __forceinline__ void wide(float (&x)[E]) const {
        if constexpr (sizeof(raw_t) == 16) {
            const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (sizeof(io_t) == 4) {
                    x[i] = __uint_as_float(w[i]);
                } else {
                    x[2 * i] = __uint_as_float(w[i] << 16);
                    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        } else if constexpr (sizeof(io_t) == 4) {
            x[0] = __uint_as_float(u);
        } else {
            x[0] = __uint_as_float((unsigned)u << 16);
            if constexpr (E == 2) x[1] = __uint_as_float(u & 0xffff0000u);
        }
    }
    __device__ __forceinline__ static void store(io_t *p, const float (&x)[E]) {
        if constexpr (sizeof(io_t) == 4) {
            if constexpr (E == 4) store4(p, x); else *p = x[0];
        } else if constexpr (E == 1) {
            *p = __float2bfloat16_rn(x[0]);
        } else {
            unsigned w[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                w[i] = *reinterpret_cast<const unsigned *>(&h);
            }
            if constexpr (E == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<unsigned *>(p) = w[0];
        }
    }
};
// E values of a weight or bias [C] fp32 at c, or `other` without one
template <int E>
__device__ __forceinline__ void affine(const float *p, int c, float other, float (&x)[E]) {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = other;
    if (!p) return;
    if constexpr (E % 4 == 0) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
            const float4 v = *reinterpret_cast<const float4 *>(p + c + e);
            x[e] = v.x; x[e + 1] = v.y; x[e + 2] = v.z; x[e + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = p[c + e];
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
    return v;
}
// Sums of K values over the `warps` warps of a row, in a fixed order; `part` is the row's, of
// [warps][K], and `bar` its barrier.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int warps, int warp, float *part, int bar) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
    if (warps == 1) return;
    if (threadIdx.x % 32 == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) part[warp * K + k] = v[k];
    }
    ptx::named_bar(bar, warps * 32);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = 0.0f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += part[w * K + k];
}

struct Params {
    long long rows;
    int C, warps;          // warps a row
    float eps;
    const void *x, *residual, *dy, *ds;
    const float *weight, *bias;
    void *y, *sum, *dx;
    float *part;           // [CTAs][2][C]: shares of dweight and dbias
    bool columns;          // whether they are wanted
};

constexpr int kMaxWarps = 32;

// A row a group of p.warps warps; several groups a CTA where that is one warp.
template <typename io_t, int E, int N, bool RES>
__global__ void __launch_bounds__(N * E > 16 ? 512 : 1024) norm_kernel(Params p) {
    __shared__ float part[2][kMaxWarps];
    const int width = p.warps * 32, tid = threadIdx.x % width;
    const long long row = (long long)blockIdx.x * (blockDim.x / width) + threadIdx.x / width;
    if (row >= p.rows) return;   // (a whole warp, and then a group of one)
    const size_t at = (size_t)row * p.C;
    const io_t *x = static_cast<const io_t *>(p.x) + at, *res = static_cast<const io_t *>(p.residual) + at;
    Piece<io_t, E> px[N], pr[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * width + tid) * E;
        px[n].zero();
        pr[n].zero();
        if (c < p.C) {
            px[n].load(x + c);
            if (RES) pr[n].load(res + c);
        }
    }
    const float x0 = to_f32(x[0]) + (RES ? to_f32(res[0]) : 0.0f);
    float v[N][E], k[1] = {0.0f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * width + tid) * E;
        px[n].wide(v[n]);
        if (RES) {
            float b[E];
            pr[n].wide(b);
#pragma unroll
            for (int e = 0; e < E; ++e) v[n][e] += b[e];
            if (c < p.C) Piece<io_t, E>::store(static_cast<io_t *>(p.sum) + at + c, v[n]);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[n][e] = c < p.C ? v[n][e] - x0 : 0.0f;
            k[0] += v[n][e];
        }
    }
    const float inv = 1.0f / (float)p.C;
    row_sum(k, p.warps, tid / 32, part[0], 1);
    const float m = k[0] * inv;
    k[0] = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * width + tid) * E;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            v[n][e] = c < p.C ? v[n][e] - m : 0.0f;
            k[0] = fmaf(v[n][e], v[n][e], k[0]);
        }
    }
    row_sum(k, p.warps, tid / 32, part[1], 1);
    const float r = rsqrtf(fmaf(k[0], inv, p.eps));
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int c = (n * width + tid) * E;
        if (c >= p.C) continue;
        float w[E], b[E];
        affine<E>(p.weight, c, 1.0f, w);
        affine<E>(p.bias, c, 0.0f, b);
#pragma unroll
        for (int e = 0; e < E; ++e) v[n][e] = fmaf(v[n][e] * r, w[e], b[e]);
        Piece<io_t, E>::store(static_cast<io_t *>(p.y) + at + c, v[n]);
    }
}

// Groups of p.warps warps walk rows; the sums over rows stay with the threads that own the columns,
// in registers or (SMEM, wide rows) in shared memory, and end as one share a CTA.
template <typename io_t, int E, int N, bool SMEM>
__global__ void __launch_bounds__(512) backward_kernel(Params p) {
    extern __shared__ float sums[];   // [2][C]
    __shared__ float part[2][3 * 16];
    const int width = p.warps * 32, groups = blockDim.x / width;
    const int group = threadIdx.x / width, tid = threadIdx.x % width, warp = tid / 32;
    float *const part0 = part[0] + group * p.warps, *const part1 = part[1] + group * p.warps * 3;
    const float inv = 1.0f / (float)p.C;
    float aw[N][E], ab[N][E];
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int e = 0; e < E; ++e) aw[n][e] = ab[n][e] = 0.0f;
    for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) sums[c] = 0.0f;
    __syncthreads();
    const long long step = (long long)gridDim.x * groups;
    for (long long row = (long long)blockIdx.x * groups + group; row < p.rows; row += step) {
        const size_t at = (size_t)row * p.C;
        const io_t *x = static_cast<const io_t *>(p.x) + at, *dy = static_cast<const io_t *>(p.dy) + at;
        const io_t *ds = static_cast<const io_t *>(p.ds) + at;
        Piece<io_t, E> px[N], pd[N], ps[N];
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * width + tid) * E;
            px[n].zero();
            pd[n].zero();
            ps[n].zero();
            if (c < p.C) {
                px[n].load(x + c);
                pd[n].load(dy + c);
                if (p.ds) ps[n].load(ds + c);
            }
        }
        const float x0 = to_f32(x[0]);
        float v[N][E], k[1] = {0.0f};
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * width + tid) * E;
            px[n].wide(v[n]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[n][e] = c < p.C ? v[n][e] - x0 : 0.0f;
                k[0] += v[n][e];
            }
        }
        row_sum(k, p.warps, warp, part0, 1 + group);
        const float m = k[0] * inv;
        float q[3] = {0.0f, 0.0f, 0.0f};   // sums of v^2, u and u v
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * width + tid) * E;
            float d[E], w[E];
            pd[n].wide(d);
            if (c < p.C) affine<E>(p.weight, c, 1.0f, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                v[n][e] = c < p.C ? v[n][e] - m : 0.0f;
                const float u = c < p.C ? __fmul_rn(d[e], w[e]) : 0.0f;
                q[0] = fmaf(v[n][e], v[n][e], q[0]);
                q[1] += u;
                q[2] = fmaf(u, v[n][e], q[2]);
            }
        }
        row_sum(q, p.warps, warp, part1, 1 + group);
        const float r = rsqrtf(fmaf(q[0], inv, p.eps)), mu = q[1] * inv, mx = q[2] * inv * r * r;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int c = (n * width + tid) * E;
            if (c >= p.C) continue;
            float d[E], w[E], s[E];
            pd[n].wide(d);
            ps[n].wide(s);
            affine<E>(p.weight, c, 1.0f, w);
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // u rounded as in its mean, so that they cancel where they have to
                s[e] = fmaf(r, fmaf(-v[n][e], mx, __fmul_rn(d[e], w[e]) - mu), s[e]);
                if (SMEM) {
                    sums[c + e] = fmaf(d[e], v[n][e] * r, sums[c + e]);
                    sums[p.C + c + e] += d[e];
                } else {
                    aw[n][e] = fmaf(d[e], v[n][e] * r, aw[n][e]);
                    ab[n][e] += d[e];
                }
            }
            Piece<io_t, E>::store(static_cast<io_t *>(p.dx) + at + c, s);
        }
    }
    if (!p.columns) return;
    if (!SMEM) {
        for (int g = 0; g < groups; ++g) {
            if (g == group) {
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int c = (n * width + tid) * E;
                    if (c >= p.C) continue;
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        sums[c + e] += aw[n][e];
                        sums[p.C + c + e] += ab[n][e];
                    }
                }
            }
            __syncthreads();
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) p.part[(size_t)blockIdx.x * 2 * p.C + c] = sums[c];
}

// dweight and dbias from the CTAs' shares: eight warps take shares 0, 8, ..; 1, 9, ..; of 32 columns.
__global__ void __launch_bounds__(256) columns_kernel(int ctas, int C, const float *part, float *dweight, float *dbias) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < 2 * C)
        for (int i = warp; i < ctas; i += 8) v += part[(size_t)i * 2 * C + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp || c >= 2 * C) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) v += s[w][lane];
    if (c < C) {
        if (dweight) dweight[c] = v;
    } else if (dbias) {
        dbias[c - C] = v;
    }
}

int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return 152;
    return n;
}

// Channels a piece: 16 bytes where every row starts on such a boundary, else a word where it starts on
// one, else an element.
int piece(int io, int C) {
    const int e = io == OSDN_F32 ? 4 : 2;
    return C * e % 16 == 0 ? 16 / e : C * e % 4 == 0 ? 4 / e : 1;
}
constexpr int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// f(E tag, N tag) for M = N E values a thread
template <int X>
using Int = std::integral_constant<int, X>;
template <typename io_t, int M, typename F>
void with_pieces(int E, const F &f) {
    constexpr int wide = 16 / (int)sizeof(io_t);
    if (E == wide) f(Int<wide>(), Int<M / wide>());
    else if (sizeof(io_t) == 2 && E == 2) f(Int<sizeof(io_t) == 2 ? 2 : 1>(), Int<sizeof(io_t) == 2 ? M / 2 : M>());
    else f(Int<1>(), Int<M>());
}

template <typename io_t, int M>
cudaError_t forward(Params p, int E, cudaStream_t stream) {
    p.warps = ceil_div(p.C, 32 * M);
    const int groups = p.warps == 1 ? 4 : 1;
    const dim3 grid((unsigned)((p.rows + groups - 1) / groups));
    with_pieces<io_t, M>(E, [&](auto e, auto n) {
        constexpr int EE = decltype(e)::value, NN = decltype(n)::value;
        if (p.residual) norm_kernel<io_t, EE, NN, true><<<grid, groups * p.warps * 32, 0, stream>>>(p);
        else norm_kernel<io_t, EE, NN, false><<<grid, groups * p.warps * 32, 0, stream>>>(p);
    });
    return cudaGetLastError();
}
template <typename io_t>
cudaError_t forward_any(const Params &p, int E, cudaStream_t stream) {
    // few rows: more threads a row, so that each waits less
    const bool few = p.rows <= 1024;
    if (p.C <= 256 || (few && p.C <= 8192)) return forward<io_t, 8>(p, E, stream);
    if (p.C <= 512 || few) return forward<io_t, 16>(p, E, stream);
    return forward<io_t, 32>(p, E, stream);
}

struct Cut {
    int M, warps, groups, ctas;
    bool smem;
};
Cut cut(long long rows, int C) {
    Cut k;
    k.M = C <= 256 ? 8 : C <= 8192 ? 16 : 32;
    k.smem = k.M == 32;
    k.warps = ceil_div(C, 32 * k.M);
    k.groups = 16 / k.warps;
    k.ctas = (int)std::min<long long>(sm_count(), (rows + k.groups - 1) / k.groups);
    return k;
}

template <typename io_t, int M>
cudaError_t backward(const Params &p, const Cut &k, int E, cudaStream_t stream) {
    cudaError_t r = cudaSuccess;
    with_pieces<io_t, M>(E, [&](auto e, auto n) {
        auto *kernel = backward_kernel<io_t, decltype(e)::value, decltype(n)::value, M == 32>;
        static std::atomic<unsigned long long> done{0};
        r = smem_attr_once(reinterpret_cast<const void *>(kernel), 2 * 16384 * 4, done);
        if (r == cudaSuccess) {
            kernel<<<k.ctas, k.groups * k.warps * 32, (size_t)p.C * 8, stream>>>(p);
            r = cudaGetLastError();
        }
    });
    return r;
}

}  // namespace

size_t backward_scratch_bytes(long long rows, int C) { return (size_t)cut(rows, C).ctas * C * 8; }

cudaError_t norm_launch(int io, long long rows, int C, const void *x, const void *residual, const float *weight,
                        const float *bias, float eps, void *y, void *sum, cudaStream_t stream) {
    Params p = {};
    p.rows = rows; p.C = C; p.eps = eps;
    p.x = x; p.residual = residual; p.weight = weight; p.bias = bias;
    p.y = y; p.sum = sum;
    const int E = piece(io, C);
    return io == OSDN_F32 ? forward_any<float>(p, E, stream) : forward_any<__nv_bfloat16>(p, E, stream);
}

cudaError_t backward_launch(int io, long long rows, int C, const void *x, const void *dy, const float *weight,
                            const void *ds, float eps, void *dx, float *dweight, float *dbias, void *scratch,
                            cudaStream_t stream) {
    Params p = {};
    const Cut k = cut(rows, C);
    p.rows = rows; p.C = C; p.eps = eps; p.warps = k.warps;
    p.x = x; p.dy = dy; p.ds = ds; p.weight = weight;
    p.dx = dx;
    p.part = static_cast<float *>(scratch);
    p.columns = dweight || dbias;
    const int E = piece(io, C);
    if (rows) {
        const auto by_size = [&](auto t) {
            using io_t = decltype(t);
            return k.M == 8 ? backward<io_t, 8>(p, k, E, stream)
                            : k.M == 16 ? backward<io_t, 16>(p, k, E, stream) : backward<io_t, 32>(p, k, E, stream);
        };
        const cudaError_t r = io == OSDN_F32 ? by_size(float()) : by_size(__nv_bfloat16());
        if (r != cudaSuccess) return r;
    }
    if (p.columns)
        columns_kernel<<<(2 * C + 31) / 32, 256, 0, stream>>>(k.ctas, C, p.part, dweight, dbias);
    return cudaGetLastError();
}

}  // namespace ln
}  // namespace osdn
