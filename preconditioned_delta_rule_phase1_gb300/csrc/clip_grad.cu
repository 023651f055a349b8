// clip_grad.cu -- the global 2-norm of many tensors and their clipping by it:
//     n = sqrt(sum over all tensors of g^2),   g <- g min(1, max_norm / n)
//
// Two passes, each read- and write-bound: the first needs every element once,
// the second once more, so 3 N bytes move where an oracle that knew the norm
// would move 2 N.  The second pass walks each CTA's share backwards, so what
// the first pass read last is still in the 129 MB L2.
//
// The tensors' addresses and sizes travel in the kernel's parameters (no copy
// to the device, so the call can be captured into a graph), up to kTable of
// them a launch.  Every tensor is cut into chunks of kChunk elements; a CTA
// takes a run of chunks.
//
// The sum: a thread squares and adds 32 elements in fp32, and adds such sums
// with their rounding errors kept (an unevaluated pair of fp32).  The 32 squares
// are what rounds: ten additions deep, so the norm is within 5 * 2^-24 (3e-7)
// of one summed in 64 bits (no more than 2e-7 was met).  Squares that leave fp32's range
// (|g| above 1e15 or so, or all below 1e-14) are squared and added in fp64
// instead; infinities and NaN reach the norm, and through it every output.
// CTAs' sums are joined in a fixed order (no atomics).
//
// Measured at 340M gradients (266 tensors, out of place): 108 us for the sum
// (6.3 TB/s, 0.92 of the measured copy bandwidth) and 221 us for the scaling
// (5.9 TB/s, 0.87).
#include <cmath>

#include "osdn_device.cuh"

namespace osdn {
namespace clip {

constexpr int kThreads = 256;
constexpr int kPer = 32;                      // elements a thread a chunk
constexpr int kChunk = kThreads * kPer;
constexpr int kCtas = 152 * 4;                // CTAs of a launch at most

template <int N>
struct Table {
    int n;
    unsigned first[N + 1];       // chunks before tensor i
    const void *g[N];
    void *o[N];
    long long size[N];           // elements; bf16 tensors: minus 1 minus that
};

template <typename io_t>
__device__ __forceinline__ void load_chunk(const io_t *p, long long left, float (&x)[kPer]) {
    if (left >= kChunk) {
#pragma unroll
        for (int i = 0; i < kPer; i += 8) {
            const io_t *at = p + (threadIdx.x * 8 + i * kThreads);
            float a[4], b[4];
            if constexpr (sizeof(io_t) == 4) {
                load4(at, a);
                load4(at + 4, b);
            } else {
                const uint4 u = *reinterpret_cast<const uint4 *>(at);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
                    (e < 2 ? a : b)[2 * (e & 1)] = f.x;
                    (e < 2 ? a : b)[2 * (e & 1) + 1] = f.y;
                }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                x[i + e] = a[e];
                x[i + 4 + e] = b[e];
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = threadIdx.x + i * kThreads;
            x[i] = at < left ? to_f32(p[at]) : 0.0f;
        }
    }
}
template <typename io_t>
__device__ __forceinline__ void store_chunk(io_t *p, long long left, const float (&x)[kPer]) {
    if (left >= kChunk) {
#pragma unroll
        for (int i = 0; i < kPer; i += 8) {
            io_t *at = p + (threadIdx.x * 8 + i * kThreads);
            if constexpr (sizeof(io_t) == 4) {
                *reinterpret_cast<float4 *>(at) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                *reinterpret_cast<float4 *>(at + 4) = make_float4(x[i + 4], x[i + 5], x[i + 6], x[i + 7]);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[i + 2 * e], x[i + 2 * e + 1]);
                    w[e] = *reinterpret_cast<const uint32_t *>(&h);
                }
                *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int at = threadIdx.x + i * kThreads;
            if (at < left) from_f32(p[at], x[i]);
        }
    }
}

// The tensor that chunk c lies in.
template <int N>
__device__ __forceinline__ int find(const Table<N> &t, unsigned c) {
    int lo = 0, hi = t.n - 1;   // first[lo] <= c < first[hi + 1]
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (t.first[mid] <= c) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

__device__ __forceinline__ double cta_sum(double v) {
    __shared__ double red[kThreads / 32];
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    __syncthreads();
    return s;
}

template <int N>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ Table<N> t, double *part) {
    const unsigned all = t.first[t.n];
    const unsigned lo = (unsigned)((unsigned long long)all * blockIdx.x / gridDim.x);
    const unsigned hi = (unsigned)((unsigned long long)all * (blockIdx.x + 1) / gridDim.x);
    float sh = 0.0f, sl = 0.0f;   // their sum is the thread's
    double wide = 0.0;
    int i = lo < hi ? find(t, lo) : 0;
    for (unsigned c = lo; c < hi; ++c) {
        while (c >= t.first[i + 1]) ++i;
        const bool bf = t.size[i] < 0;
        const long long off = (long long)(c - t.first[i]) * kChunk;
        const long long left = (bf ? -1 - t.size[i] : t.size[i]) - off;
        float x[kPer];
        if (bf) load_chunk(static_cast<const __nv_bfloat16 *>(t.g[i]) + off, left, x);
        else load_chunk(static_cast<const float *>(t.g[i]) + off, left, x);
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < kPer; ++e) s4[e & 3] = fmaf(x[e], x[e], s4[e & 3]);
        const float s = (s4[0] + s4[1]) + (s4[2] + s4[3]);
        if (s < 1e30f && s > 1e-28f) {
            const float n = sh + s, b = n - sh;       // two-sum
            sl += (sh - (n - b)) + (s - b);
            sh = n;
        } else {
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) m = x[e] == 0.0f ? m : 1.0f;
            if (m != 0.0f) {
#pragma unroll 1
                for (int e = 0; e < kPer; e += 4) {
                    // (a dynamic index would put x in local memory: four at a time, rotated down)
                    wide += (double)x[0] * x[0] + (double)x[1] * x[1] + (double)x[2] * x[2] + (double)x[3] * x[3];
#pragma unroll
                    for (int f = 0; f < kPer - 4; ++f) x[f] = x[f + 4];
                }
            }
        }
    }
    const double s = cta_sum((double)sh + (double)sl + wide);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The sum of all parts, the same in every CTA.
__device__ __forceinline__ double total(const double *part, int parts) {
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) v += part[i];
    return cta_sum(v);
}

__global__ void __launch_bounds__(kThreads) join_kernel(const double *part, int parts, double *out, float *norm) {
    const double s = total(part, parts);
    if (threadIdx.x == 0) {
        if (out) *out = s;
        if (norm) *norm = (float)sqrt(s);
    }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
scale_kernel(const __grid_constant__ Table<N> t, const double *part, int parts, float max_norm,
             float *norm) {
    const double n = sqrt(total(part, parts));
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const float f = n <= (double)max_norm ? 1.0f : (float)((double)max_norm / n);   // NaN for a NaN norm
    const unsigned all = t.first[t.n];
    const unsigned lo = (unsigned)((unsigned long long)all * blockIdx.x / gridDim.x);
    const unsigned hi = (unsigned)((unsigned long long)all * (blockIdx.x + 1) / gridDim.x);
    int i = lo < hi ? find(t, hi - 1) : 0;
    for (unsigned c = hi; c-- > lo;) {
        while (c < t.first[i]) --i;
        if (f == 1.0f && t.o[i] == t.g[i]) continue;
        const bool bf = t.size[i] < 0;
        const long long off = (long long)(c - t.first[i]) * kChunk;
        const long long left = (bf ? -1 - t.size[i] : t.size[i]) - off;
        float x[kPer];
        if (bf) load_chunk(static_cast<const __nv_bfloat16 *>(t.g[i]) + off, left, x);
        else load_chunk(static_cast<const float *>(t.g[i]) + off, left, x);
#pragma unroll
        for (int e = 0; e < kPer; ++e) x[e] *= f;
        if (bf) store_chunk(static_cast<__nv_bfloat16 *>(t.o[i]) + off, left, x);
        else store_chunk(static_cast<float *>(t.o[i]) + off, left, x);
    }
}

constexpr int kTable = 1024;   // 28 KB of the 32 KB that a kernel's parameters may take

// Tensors [at, n) into the table, as many as fit; returns the first left out that is not empty
// (n: none), so that only a call without any element meets an empty table.  A launch numbers its
// chunks in 32 bits (a call has at most 2^44 elements, and 2^31 tensors).
template <int N>
int fill(Table<N> &t, int at, int n, const void *const *g, void *const *o, const long long *size,
         const int *io) {
    t.n = 0;
    t.first[0] = 0;
    unsigned long long c = 0;
    for (; at < n; ++at) {
        if (size[at] == 0) continue;
        if (t.n == N) break;
        c += (unsigned long long)((size[at] + kChunk - 1) / kChunk);
        t.g[t.n] = g[at];
        t.o[t.n] = o ? o[at] : const_cast<void *>(g[at]);
        t.size[t.n] = io[at] == OSDN_BF16 ? -1 - size[at] : size[at];
        t.first[++t.n] = (unsigned)c;
    }
    return at;
}

template <int N>
cudaError_t run(int n, const void *const *g, void *const *o, const long long *size, const int *io,
                float max_norm, float *norm, double *part, cudaStream_t stream) {
    Table<N> t;
    int parts = 0, tables = 0;
    cudaError_t e = cudaSuccess;
    for (int at = 0; at < n && e == cudaSuccess;) {
        at = fill(t, at, n, g, o, size, io);
        if (!t.n) break;
        const int ctas = t.first[t.n] < (unsigned)kCtas ? (int)t.first[t.n] : kCtas;
        sum_kernel<N><<<ctas, kThreads, 0, stream>>>(t, part + 1 + parts);
        e = cudaGetLastError();
        parts += ctas;
        ++tables;
    }
    const double *from = part + 1;
    const bool scale = o || !std::isinf(max_norm);
    if (e == cudaSuccess && (tables != 1 || !scale)) {
        join_kernel<<<1, kThreads, 0, stream>>>(from, parts, part, norm);
        e = cudaGetLastError();
        from = part;
        parts = 1;
        norm = nullptr;
    }
    if (!scale) return e;
    for (int at = 0; at < n && e == cudaSuccess;) {
        if (tables != 1) at = fill(t, at, n, g, o, size, io);
        else at = n;   // the table is still the sum's
        if (!t.n) break;
        const int ctas = t.first[t.n] < (unsigned)kCtas ? (int)t.first[t.n] : kCtas;
        scale_kernel<N><<<ctas, kThreads, 0, stream>>>(t, from, parts, max_norm, norm);
        e = cudaGetLastError();
    }
    return e;
}

}  // namespace clip

size_t clip_scratch_bytes(int n) {
    return (size_t)(1 + (size_t)clip::kCtas * ((n + clip::kTable - 1) / clip::kTable)) * 8;
}

cudaError_t clip_launch(int n, const void *const *g, void *const *o, const long long *size,
                        const int *io, float max_norm, float *norm, void *scratch,
                        cudaStream_t stream) {
    double *part = static_cast<double *>(scratch);
    // A launch copies its parameters, 1.4 or 28 KB: 48 tensors take 55.8 us a call (12 on the device),
    // 49 with the large table 60.4 (12)
    if (n <= 48) return clip::run<48>(n, g, o, size, io, max_norm, norm, part, stream);
    return clip::run<clip::kTable>(n, g, o, size, io, max_norm, norm, part, stream);
}

}  // namespace osdn
