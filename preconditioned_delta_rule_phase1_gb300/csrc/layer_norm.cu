// layer_norm.cu -- layer norm over whole rows, with the addition to the
// residual stream in front of it, and its gradients.  Per row of C values,
//     s = x + residual,  r = 1 / sqrt(mean((s - m)^2) + eps),  x^ = (s - m) r,
//     y = weight x^ + bias
//     u = dy weight,  dx = r (u - mean(u) - x^ mean(u x^)) + ds
//     dweight = sum over rows of dy x^,   dbias = sum over rows of dy
// Rows are read and written once, so HBM bounds both directions.  A row is
// held in registers, N pieces of E neighbouring channels a thread (16 bytes
// where rows keep 16-byte boundaries, else one word), by one warp where it is
// short and by up to 32 otherwise.  Differences to the row's first value come
// before any sum, so that a large mean costs no accuracy; the norm then takes
// the mean and the variance about it, two reductions, the gradients all four
// sums in one.  A row whose first value is an outlier (kFarSquare) takes them
// again about its mean.  All arithmetic is fp32.
//
// Measured (bf16): the norm 47 us at 16384 rows of 2048 with a residual (5.7
// TB/s, 0.84 of the measured copy bandwidth; 45 us among other calls), 130 us
// at rows of 2047 (words, and masks at both ends); its gradients with ds 56 us
// at 16384x2048 (0.71), where nothing is full (0.54 of the issue slots at 16
// warps an SM, 430 instructions a warp and row; 0.67 of HBM) and a row's way
// through barrier, shared memory and arithmetic is what counts, 26 us at
// 8193x1024 (0.38) and 78 us at 1024x16384 (0.25: one row ahead, sums in shared
// memory, the weight read twice a row).  Gradients with two reductions a row
// took 72 us, without loads ahead 88 us, where one reduction and three rows
// ahead took 66.
#include <algorithm>
#include <type_traits>

#include "decay_attn.cuh"
#include "ptx.cuh"

namespace osdn {
namespace ln {

namespace {

// Zeros, or the bytes at p where `there`.  Predicated rather than branched around: the compiler would
// move the first use into the branch, and wait there for one load after the other.
__device__ __forceinline__ void load_if(const void *p, bool there, uint4 &u) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\t"
                 "mov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t@q ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p), "r"((int)there));
}
__device__ __forceinline__ void load_if(const void *p, bool there, unsigned &u) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\tmov.b32 %0, 0;\n\t@q ld.global.nc.b32 %0, [%1];\n\t}"
                 : "=r"(u) : "l"(p), "r"((int)there));
}
// A word, or its lower half, or zero.
__device__ __forceinline__ void load_if(const void *p, bool whole, bool half, unsigned &u) {
    asm volatile("{\n\t.reg .pred q, r;\n\tsetp.ne.b32 q, %2, 0;\n\tsetp.ne.b32 r, %3, 0;\n\tmov.b32 %0, 0;\n\t"
                 "@q ld.global.nc.b32 %0, [%1];\n\t@r ld.global.nc.u16 %0, [%1];\n\t}"
                 : "=r"(u) : "l"(p), "r"((int)whole), "r"((int)half));
}

// How a row of C channels lies in its threads' pieces: kFull, it fills them all; kTail, some threads
// have fewer or none; kOdd (rows of an odd number of bf16, E = 2), also the row may begin in the middle
// of a word, and its first and last pieces may hold one channel.
enum { kFull, kTail, kOdd };
// A thread's N pieces of E neighbouring channels: piece n begins at channel (n width + tid) E - odd.
template <typename io_t, int E, int N, int KIND>
struct Pieces {
    static constexpr bool ODD = KIND == kOdd;
    static constexpr bool FULL = KIND == kFull;
    static constexpr int M = N * E;
    typedef typename std::conditional<E * sizeof(io_t) == 16, uint4, unsigned>::type raw_t;
    int C;
    int first, step, count, last;   // channel of piece 0, from piece to piece, pieces, and (ODD) of second channels
    __device__ __forceinline__ Pieces(int channels, int width, int tid, int odd) : C(channels) {
        first = tid * E - (ODD ? odd : 0);
        step = width * E;
        count = (C - first + step - 1) / step;   // (first is less than 32 M; C may be less)
        last = ODD ? (C - first + step - 2) / step : count;
        count = C > first ? count : 0;
        last = ODD && C <= first + 1 ? 0 : last;
    }
    // pieces n, n + 1, .. of a thread that has more
    template <int N2>
    __device__ __forceinline__ Pieces(const Pieces<io_t, E, N2, KIND> &all, int n)
        : C(all.C), first(all.first + n * all.step), step(all.step), count(all.count - n), last(all.last - n) {}
    __device__ __forceinline__ int at(int n) const { return n * step + first; }
    // whether element i (of M) is a channel of the row
    __device__ __forceinline__ bool has(int i) const {
        if (FULL) return true;
        if (!ODD) return i / E < count;
        return i % E ? i / E < last : i / E < count && (i || first >= 0);
    }
    __device__ __forceinline__ float pick(int i, float v) const { return has(i) ? v : 0.0f; }
    __device__ __forceinline__ void load(const io_t *row, raw_t (&u)[N]) const {
        const io_t *p = row + first;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (FULL) u[n] = *reinterpret_cast<const raw_t *>(p + n * step);
            else if constexpr (ODD) load_if(p + n * step, n < last, n >= last && n < count, u[n]);
            else load_if(p + n * step, n < last, u[n]);
        }
        if constexpr (ODD)
            if (first < 0) u[0] &= 0xffff0000u;
    }
    __device__ __forceinline__ static void wide(const raw_t (&u)[N], float (&x)[M]) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            unsigned w[E * sizeof(io_t) / 4];
            if constexpr (sizeof(raw_t) == 16) {
                w[0] = u[n].x; w[1] = u[n].y; w[2] = u[n].z; w[3] = u[n].w;
            } else {
                w[0] = u[n];
            }
#pragma unroll
            for (int i = 0; i < (int)(E * sizeof(io_t) / 4); ++i) {
                if constexpr (sizeof(io_t) == 4) {
                    x[n * E + i] = __uint_as_float(w[i]);
                } else {
                    x[n * E + 2 * i] = __uint_as_float(w[i] << 16);
                    x[n * E + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        }
    }
    __device__ __forceinline__ void store(io_t *row, const float (&x)[M]) const {
        io_t *p = row + first;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            io_t *q = p + n * step;
            if constexpr (sizeof(io_t) == 4) {
                if (FULL || n < count) {
                    if constexpr (E == 4)
                        *reinterpret_cast<float4 *>(q) = make_float4(x[n * E], x[n * E + 1], x[n * E + 2], x[n * E + 3]);
                    else
                        *q = x[n];
                }
            } else {
                unsigned w[E / 2];
#pragma unroll
                for (int i = 0; i < E / 2; ++i) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(x[n * E + 2 * i], x[n * E + 2 * i + 1]);
                    w[i] = *reinterpret_cast<const unsigned *>(&h);
                }
                if constexpr (E == 8) {
                    if (FULL || n < count) *reinterpret_cast<uint4 *>(q) = make_uint4(w[0], w[1], w[2], w[3]);
                } else if constexpr (!ODD) {
                    if (n < count) *reinterpret_cast<unsigned *>(q) = w[0];
                } else {
                    if (n < last && (n || first >= 0)) *reinterpret_cast<unsigned *>(q) = w[0];
                    else if (n < last) reinterpret_cast<unsigned short *>(q)[1] = (unsigned short)(w[0] >> 16);
                    else if (n < count && (n || first >= 0)) *reinterpret_cast<unsigned short *>(q) = (unsigned short)w[0];
                }
            }
        }
    }
    // of a weight or bias [C] fp32, or `other` without one
    __device__ __forceinline__ void affine(const float *p, float other, float (&x)[M]) const {
        const float *q = p + first;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            if constexpr (E % 4 == 0) {
#pragma unroll
                for (int e = 0; e < E; e += 4) {
                    float4 v = make_float4(other, other, other, other);
                    if (p && (FULL || n < count)) v = *reinterpret_cast<const float4 *>(q + n * step + e);
                    x[n * E + e] = v.x; x[n * E + e + 1] = v.y; x[n * E + e + 2] = v.z; x[n * E + e + 3] = v.w;
                }
            } else if constexpr (E == 2 && !ODD) {
                float2 v = make_float2(other, other);
                if (p && n < count) v = *reinterpret_cast<const float2 *>(q + n * step);
                x[n * E] = v.x; x[n * E + 1] = v.y;
            } else {
                // (what is no channel takes a value of another: nothing is made of it)
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    x[n * E + e] = other;
                    if (p) x[n * E + e] = p[min(max(at(n) + e, 0), C - 1)];
                }
            }
        }
    }
};

// Two values an instruction.
__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }
template <int M>
__device__ __forceinline__ float2 get2(const float (&x)[M], int i) { return make_float2(x[i], x[i + 1]); }
template <int M>
__device__ __forceinline__ void put2(float (&x)[M], int i, float2 v) {
    x[i] = v.x;
    x[i + 1] = v.y;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
    return v;
}
// Sums over the `warps` warps of a row, in a fixed order; `part` is the row's, and `bar` its barrier.
__device__ __forceinline__ float row_sum(float v, int warps, int warp, float *part, int bar) {
    v = warp_sum(v);
    if (warps == 1) return v;
    if (threadIdx.x % 32 == 0) part[warp] = v;
    ptx::named_bar(bar, warps * 32);
    v = 0.0f;
    for (int w = 0; w < warps; ++w) v += part[w];
    return v;
}
// Four at once: the first two exchanges halve what a lane carries, so that six shuffles do instead of
// twenty; lanes 0 to 3 then hold one sum each.
__device__ __forceinline__ float4 row_sum(float4 v, int warps, int warp, float4 *part, int bar) {
    const int lane = threadIdx.x & 31;
    const bool a = lane & 1, b = lane & 2;
    const float p = (a ? v.y : v.x) + __shfl_xor_sync(kFullMask, a ? v.x : v.y, 1);
    const float q = (a ? v.w : v.z) + __shfl_xor_sync(kFullMask, a ? v.z : v.w, 1);
    float s = (b ? q : p) + __shfl_xor_sync(kFullMask, b ? p : q, 2);   // lane 0: x, 1: y, 2: z, 3: w
#pragma unroll
    for (int m = 4; m < 32; m <<= 1) s += __shfl_xor_sync(kFullMask, s, m);
    if (warps == 1)
        return make_float4(__shfl_sync(kFullMask, s, 0), __shfl_sync(kFullMask, s, 1), __shfl_sync(kFullMask, s, 2),
                           __shfl_sync(kFullMask, s, 3));
    if (lane < 4) reinterpret_cast<float *>(part + warp)[lane] = s;
    ptx::named_bar(bar, warps * 32);
    float2 t = two(0.0f), u = two(0.0f);
    for (int w = 0; w < warps; ++w) {
        const float4 o = part[w];
        t = __fadd2_rn(t, make_float2(o.x, o.y));
        u = __fadd2_rn(u, make_float2(o.z, o.w));
    }
    return make_float4(t.x, t.y, u.x, u.y);
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
// A row's first value may lie this far (four standard deviations, squared) from the mean: differences to it
// are then rounded by 2^-22 of one.
constexpr float kFarSquare = 16.0f;

// A row a group of p.warps warps; several groups a CTA where that is one warp.
template <typename io_t, int E, int N, int KIND, bool RES>
__global__ void __launch_bounds__(N * E == 8 ? 1024 : N * E == 16 ? 128 : 512) norm_kernel(Params p) {
    typedef Pieces<io_t, E, N, KIND> P;
    constexpr int M = P::M;
    __shared__ float part[2][kMaxWarps];
    const int width = p.warps * 32, tid = threadIdx.x % width;
    const long long row = (long long)blockIdx.x * (blockDim.x / width) + threadIdx.x / width;
    if (row >= p.rows) return;   // (a whole warp, and then a group of one)
    const size_t at = (size_t)row * p.C;
    const io_t *x = static_cast<const io_t *>(p.x) + at, *res = static_cast<const io_t *>(p.residual) + at;
    const P g(p.C, width, tid, (int)(at & 1));
    typename P::raw_t rx[N], rr[N];
    g.load(x, rx);
    if (RES) g.load(res, rr);
    const float x0 = to_f32(x[0]) + (RES ? to_f32(res[0]) : 0.0f);
    float v[M];
    float2 sum = two(0.0f);
    P::wide(rx, v);
    if (RES) {
        float b[M];
        P::wide(rr, b);
#pragma unroll
        for (int i = 0; i < M; i += 2) put2(v, i, __fadd2_rn(get2(v, i), get2(b, i)));
        g.store(static_cast<io_t *>(p.sum) + at, v);
    }
#pragma unroll
    for (int i = 0; i < M; i += 2) {
        put2(v, i, __fadd2_rn(get2(v, i), make_float2(g.pick(i, -x0), g.pick(i + 1, -x0))));
        sum = __fadd2_rn(sum, get2(v, i));
    }
    const float inv = 1.0f / (float)p.C;
    // the mean of v off, and the variance
    const auto centre = [&](const P &g, float s, float &m) {
        m = row_sum(s, p.warps, tid / 32, part[0], 1) * inv;
        float2 q = two(0.0f);
#pragma unroll
        for (int i = 0; i < M; i += 2) {
            put2(v, i, __fadd2_rn(get2(v, i), make_float2(g.pick(i, -m), g.pick(i + 1, -m))));
            q = __ffma2_rn(get2(v, i), get2(v, i), q);
        }
        return row_sum(q.x + q.y, p.warps, tid / 32, part[1], 1) * inv;
    };
    float m, var = centre(g, sum.x + sum.y, m);
    if (!(m * m <= kFarSquare * var)) {
        // The first value lies far outside the others: the differences to it have lost their digits.  Those
        // to the mean have them all, and their mean is what that one was off by.  (The whole row sees the
        // same sums.)
        const float mean = x0 + m;
        P h = g;   // (its masks computed again: kept over the reductions, rows on words take twice the time)
        asm volatile("" : "+r"(h.first), "+r"(h.count), "+r"(h.last));
        h.load(x, rx);
        P::wide(rx, v);
        if (RES) {
            float b[M];
            h.load(res, rr);
            P::wide(rr, b);
#pragma unroll
            for (int i = 0; i < M; i += 2) put2(v, i, __fadd2_rn(get2(v, i), get2(b, i)));
        }
        sum = two(0.0f);
#pragma unroll
        for (int i = 0; i < M; i += 2) {
            put2(v, i, __fadd2_rn(get2(v, i), make_float2(h.pick(i, -mean), h.pick(i + 1, -mean))));
            sum = __fadd2_rn(sum, get2(v, i));
        }
        var = centre(h, sum.x + sum.y, m);
    }
    const float r = rsqrtf(var + p.eps);
    float w[M], b[M];
    g.affine(p.weight, 1.0f, w);
    g.affine(p.bias, 0.0f, b);
#pragma unroll
    for (int i = 0; i < M; i += 2)
        put2(v, i, __ffma2_rn(__fmul2_rn(get2(v, i), two(r)), get2(w, i), get2(b, i)));
    g.store(static_cast<io_t *>(p.y) + at, v);
}

// Groups of p.warps warps walk rows; the sums over rows stay with the threads that own the columns,
// in registers or (SMEM, wide rows) in shared memory, and end as one share a CTA.  Rows come into shared
// memory by asynchronous copies, S at a time; a thread reads only what it copied itself.  With kOdd a
// group keeps to rows of one parity, which begin in the same place of a word, so that its columns stay
// its own.
// S, by what 227 KB of shared memory hold beside the sums: three rows of up to 16 values a thread in bf16
// and 8 in fp32, of which two are under way while one is worked on; one of 32 in bf16 and 16 in fp32, whose
// copy begins when the row before it is done, so that every row waits for memory; none of 32 in fp32, which
// are read when they are needed.
template <typename io_t, int M>
struct Ahead {
    static constexpr bool kSmem = M == 32;
    static constexpr int S = sizeof(io_t) * M <= 32 ? 3 : sizeof(io_t) * M <= 64 ? 1 : 0;
    static constexpr int bytes(int threads) { return threads * M * (int)sizeof(io_t) * 3 * S; }   // of copies
    static constexpr int sum_bytes(int threads, int C) { return kSmem ? threads * M * 8 : C * 8; }
};
template <typename io_t, int E, int N, int KIND>
__global__ void __launch_bounds__(512) backward_kernel(Params p) {
    typedef Pieces<io_t, E, N, KIND> P;
    typedef typename P::raw_t raw_t;
    constexpr int M = P::M, S = Ahead<io_t, M>::S;
    constexpr bool ODD = P::ODD, SMEM = Ahead<io_t, M>::kSmem;
    constexpr int Q = E == 1 ? 2 : 1, EE = Q * E;   // pieces and values at a time
    extern __shared__ __align__(16) char sm[];      // [S][3][N][threads] pieces, sums
    __shared__ float4 part[2][16];   // (one for even and one for odd rows of a group)
    const int width = p.warps * 32, groups = blockDim.x / width;
    const int group = threadIdx.x / width, tid = threadIdx.x % width, warp = tid / 32;
    const float inv = 1.0f / (float)p.C;
    const long long first = (long long)blockIdx.x * groups + group, all = (long long)gridDim.x * groups;
    // an even number of groups with kOdd (a last one too many idles; alone it has one row)
    const long long step = !ODD ? all : all > 1 ? all & ~1ll : 2;
    const long long rows = ODD && all > 1 && first >= step ? 0 : p.rows;
    const P g(p.C, width, tid, (int)(first & 1));
    raw_t *const slot = reinterpret_cast<raw_t *>(sm) + threadIdx.x;
    float *const sums = reinterpret_cast<float *>(sm + Ahead<io_t, M>::bytes(blockDim.x));
    // tensor k (x, dy, ds) of a row into its place of stage s
    const auto place = [&](int s, int k, int n) { return slot + ((s * 3 + k) * N + n) * (int)blockDim.x; };
    const io_t *const x = static_cast<const io_t *>(p.x) + g.first, *const dy = static_cast<const io_t *>(p.dy) + g.first;
    const io_t *const ds = p.ds ? static_cast<const io_t *>(p.ds) + g.first : nullptr;
    const auto fetch = [&](const io_t *base, int s, int k, size_t at) {
        const uint32_t to = ptx::smem_u32(place(s, k, 0));
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const int bytes = P::FULL || n < g.last ? (int)sizeof(raw_t) : ODD && n < g.count ? 2 : 0;
            const io_t *q = base + at + n * g.step;
            if (!P::FULL && !bytes) q = base - g.first;
            ptx::copy_async<sizeof(raw_t)>(to + n * (unsigned)(blockDim.x * sizeof(raw_t)), q, bytes);
        }
    };
    const size_t far = (size_t)step * p.C;   // elements from a group's row to its next
    size_t at = (size_t)first * p.C;
    const auto fetch_row = [&](int s, long long row, size_t from) {
        if (S && row < rows) {
            fetch(x, s, 0, from);
            fetch(dy, s, 1, from);
            if (ds) fetch(ds, s, 2, from);
        }
        ptx::copies_commit();   // (a group even of nothing, so that waiting counts them)
    };
    const auto read = [&](int s, int k, int n, float (&v)[EE]) {
        raw_t u[Q];
        if constexpr (S == 0) {
            const void *base = k == 0 ? p.x : k == 1 ? p.dy : p.ds;
            Pieces<io_t, E, Q, KIND>(g, n).load(static_cast<const io_t *>(base) + at, u);
        } else {
#pragma unroll
            for (int i = 0; i < Q; ++i) u[i] = *place(s, k, n + i);
            if constexpr (ODD)
                if (n == 0 && g.first < 0) u[0] &= 0xffff0000u;
        }
        Pieces<io_t, E, Q, KIND>::wide(u, v);
    };
    // a row's first value: of the row in stage s, which the group's first thread has copied, or from `from`
    const auto pivot = [&](int s, long long row, size_t from) {
        if (row >= rows) return 0.0f;
        if constexpr (S <= 1) return to_f32(static_cast<const io_t *>(p.x)[from]);
        const raw_t *q = place(s, 0, 0) - tid;
        return to_f32(reinterpret_cast<const io_t *>(q)[ODD ? (int)(from & 1) : 0]);
    };
    float aw[M], ab[M], w[M];
#pragma unroll
    for (int i = 0; i < M; ++i) aw[i] = ab[i] = 0.0f;
    if (!SMEM) g.affine(p.weight, 1.0f, w);
    // (SMEM: a thread's own sums, two at a time side by side over the threads)
    float2 *const own = reinterpret_cast<float2 *>(sums) + threadIdx.x;
    if (SMEM) {
#pragma unroll
        for (int i = 0; i < M; ++i) own[i * (int)blockDim.x] = two(0.0f);
    } else {
        for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) sums[c] = 0.0f;
    }
    __syncthreads();
    float x0 = first < rows ? to_f32(static_cast<const io_t *>(p.x)[at]) : 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) fetch_row(i, first + i * step, at + i * far);
    int s = 0, odd = 0;
    for (long long row = first; row < rows; row += step, at += far, odd ^= 1) {
        const int next = s + 1 >= S ? 0 : s + 1;
        float v[M];
        float2 q[4] = {two(0.0f), two(0.0f), two(0.0f), two(0.0f)};   // sums of v, v^2, u and u v
        ptx::copies_wait<(S > 1 ? S - 2 : 0)>();   // this row's and the next one's (for its pivot)
#pragma unroll
        for (int n = 0; n < N; n += Q) {
            float t[EE], d[EE];
            read(s, 0, n, t);
            read(s, 1, n, d);
            if (SMEM) Pieces<io_t, E, Q, KIND>(g, n).affine(p.weight, 1.0f, reinterpret_cast<float (&)[EE]>(w[n * E]));
#pragma unroll
            for (int i = 0; i < EE; i += 2) {
                const int o = n * E + i;
                put2(v, o, __fadd2_rn(get2(t, i), make_float2(g.pick(o, -x0), g.pick(o + 1, -x0))));
                const float2 u = __fmul2_rn(get2(d, i), get2(w, o));
                q[0] = __fadd2_rn(q[0], get2(v, o));
                q[1] = __ffma2_rn(get2(v, o), get2(v, o), q[1]);
                q[2] = __fadd2_rn(q[2], u);
                q[3] = __ffma2_rn(u, get2(v, o), q[3]);
            }
        }
        float4 t = row_sum(make_float4(q[0].x + q[0].y, q[1].x + q[1].y, q[2].x + q[2].y, q[3].x + q[3].y), p.warps,
                           warp, part[odd] + group * p.warps, 1 + group);
        const float mu = t.z * inv;
        float m = t.x * inv, var = fmaf(-m, m, t.y * inv), uv = fmaf(-m, t.z, t.w) * inv;
        if (!(m * m <= kFarSquare * var)) {
            // the first value lies far outside the others: differences and sums are taken again, about the mean
            // (by the whole group, which sees the same sums)
            const float mean = x0 + m;
            float2 z[3] = {two(0.0f), two(0.0f), two(0.0f)};
#pragma unroll
            for (int n = 0; n < N; n += Q) {
                float c[EE], d[EE];
                read(s, 0, n, c);
                read(s, 1, n, d);
#pragma unroll
                for (int i = 0; i < EE; i += 2) {
                    const int o = n * E + i;
                    put2(v, o, __fadd2_rn(get2(c, i), make_float2(g.pick(o, -mean), g.pick(o + 1, -mean))));
                    z[0] = __fadd2_rn(z[0], get2(v, o));
                    z[1] = __ffma2_rn(get2(v, o), get2(v, o), z[1]);
                    z[2] = __ffma2_rn(__fmul2_rn(get2(d, i), get2(w, o)), get2(v, o), z[2]);
                }
            }
            if (p.warps > 1) ptx::named_bar(1 + group, width);   // all have read the sums above
            t = row_sum(make_float4(z[0].x + z[0].y, z[1].x + z[1].y, mu, z[2].x + z[2].y), p.warps, warp,
                        part[odd] + group * p.warps, 1 + group);
            m = t.x * inv;   // (what the mean was off by)
            var = fmaf(-m, m, t.y * inv);
            uv = fmaf(-m, mu, t.w * inv);
        }
        if (S > 1) {
            if (p.warps == 1) __syncwarp();
            x0 = pivot(next, row + step, at + far);   // (past a barrier that the copying thread has passed)
        } else {
            x0 = pivot(0, row + step, at + far);
        }
        // x^ = r v - r m,  dx = r u + k x^ + k0  (in v, k would have a cube of r, which may leave fp32 where dx
        // does not)
        const float r = rsqrtf(var + p.eps), rm = -r * m, kx = -uv * r * r, k0 = -r * mu;
        io_t *out = static_cast<io_t *>(p.dx) + at;
#pragma unroll
        for (int n = 0; n < N; n += Q) {
            float d[EE], e[EE];
            read(s, 1, n, d);
            if (ds) read(s, 2, n, e);
            if (SMEM) Pieces<io_t, E, Q, KIND>(g, n).affine(p.weight, 1.0f, reinterpret_cast<float (&)[EE]>(w[n * E]));
#pragma unroll
            for (int i = 0; i < EE; i += 2) {
                const int o = n * E + i;
                const float2 u = __fmul2_rn(get2(d, i), get2(w, o));
                const float2 xh = __ffma2_rn(get2(v, o), two(r), two(rm));
                float2 f = __ffma2_rn(xh, two(kx), two(k0));
                f = __ffma2_rn(u, two(r), f);
                if (ds) f = __fadd2_rn(f, get2(e, i));
                put2(e, i, f);
                if (SMEM) {
                    float2 &sw = own[(o / 2) * (int)blockDim.x], &sb = own[(M / 2 + o / 2) * (int)blockDim.x];
                    sw = __ffma2_rn(get2(d, i), xh, sw);
                    sb = __fadd2_rn(sb, get2(d, i));
                } else {
                    put2(aw, o, __ffma2_rn(get2(d, i), xh, get2(aw, o)));
                    put2(ab, o, __fadd2_rn(get2(ab, o), get2(d, i)));
                }
            }
            Pieces<io_t, E, Q, KIND>(g, n).store(out, e);
        }
        fetch_row(s, row + S * step, at + S * far);
        s = next;
    }
    if (!p.columns) return;
    da::dependents_may_start();
    float *const share = p.part + (size_t)blockIdx.x * 2 * p.C;
    if (SMEM) {   // one group
#pragma unroll
        for (int i = 0; i < M; ++i)
            if (g.has(i)) {
                const int c = g.at(i / E) + i % E;
                const float2 sw = own[(i / 2) * (int)blockDim.x], sb = own[(M / 2 + i / 2) * (int)blockDim.x];
                share[c] = i % 2 ? sw.y : sw.x;
                share[p.C + c] = i % 2 ? sb.y : sb.x;
            }
        return;
    }
    for (int o = 0; o < groups; ++o) {
        if (o == group) {
#pragma unroll
            for (int i = 0; i < M; ++i)
                if (g.has(i)) {
                    const int c = g.at(i / E) + i % E;
                    sums[c] += aw[i];
                    sums[p.C + c] += ab[i];
                }
        }
        __syncthreads();
    }
    for (int c = threadIdx.x; c < 2 * p.C; c += blockDim.x) share[c] = sums[c];
}

// dweight and dbias from the CTAs' shares, 32 columns a CTA: its 32 warps take shares 0, 32, ..; 1, 33, ..
// (all at once: at most five each), and the first adds up what they have.
constexpr int kColumnWarps = 32;
__global__ void __launch_bounds__(kColumnWarps * 32) columns_kernel(int ctas, int C, const float *part, float *dweight,
                                                                   float *dbias) {
    __shared__ float s[kColumnWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;   // C is at most 16384
    da::dependency_wait();
    float v = 0.0f;
    if (c < 2 * C)
#pragma unroll 5
        for (int i = warp; i < ctas; i += kColumnWarps) v += part[(size_t)i * 2 * C + c];
    s[warp][lane] = v;
    __syncthreads();
    if (warp || c >= 2 * C) return;
#pragma unroll
    for (int w = 1; w < kColumnWarps; ++w) v += s[w][lane];
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

// Channels a piece: 16 bytes where every row starts on such a boundary, else a word.
int piece(int io, int C) {
    const int e = io == OSDN_F32 ? 4 : 2;
    return C * e % 16 == 0 ? 16 / e : 4 / e;
}
constexpr int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

// f(E tag, N tag, KIND tag) for M = N E values a thread
template <int X>
using Int = std::integral_constant<int, X>;
template <typename io_t, int M, typename F>
void with_pieces(int C, int E, int threads, const F &f) {
    constexpr int wide = 16 / (int)sizeof(io_t), word = 4 / (int)sizeof(io_t);
    if (E == wide && C == threads * M) f(Int<wide>(), Int<M / wide>(), Int<kFull>());
    else if (E == wide) f(Int<wide>(), Int<M / wide>(), Int<kTail>());
    else if (sizeof(io_t) == 4 || C % 2 == 0) f(Int<word>(), Int<M / word>(), Int<kTail>());
    else f(Int<word>(), Int<M / word>(), Int<sizeof(io_t) == 2 ? kOdd : kTail>());
}

template <typename io_t, int M>
cudaError_t forward(Params p, int E, cudaStream_t stream) {
    p.warps = ceil_div(p.C + (p.C & 1), 32 * M);   // an odd row may begin inside a word
    const int groups = p.warps == 1 ? 4 : 1;
    const dim3 grid((unsigned)((p.rows + groups - 1) / groups));
    with_pieces<io_t, M>(p.C, E, p.warps * 32, [&](auto e, auto n, auto kind) {
        constexpr int EE = decltype(e)::value, NN = decltype(n)::value, K = decltype(kind)::value;
        if (p.residual) norm_kernel<io_t, EE, NN, K, true><<<grid, groups * p.warps * 32, 0, stream>>>(p);
        else norm_kernel<io_t, EE, NN, K, false><<<grid, groups * p.warps * 32, 0, stream>>>(p);
    });
    return cudaGetLastError();
}
template <typename io_t>
cudaError_t forward_any(const Params &p, int E, cudaStream_t stream) {
    // few rows: more threads a row, so that each waits less
    if (p.C < 256 || (p.rows <= 1024 && p.C < 8192)) return forward<io_t, 8>(p, E, stream);
    if (p.C < 512) return forward<io_t, 16>(p, E, stream);
    return forward<io_t, 32>(p, E, stream);
}

struct Cut {
    int M, warps, groups, ctas;
};
Cut cut(int io, long long rows, int C) {
    Cut k;
    // 16 values a thread halve what a row costs beside them, eight fill more threads (bf16, 8193 rows of
    // 1024: 31 and 27 us; 16384 rows of 2048: 68 and 72 us); fp32 has no room for three rows of 16
    k.M = C < (io == OSDN_F32 ? 4096 : 1536) ? 8 : C <= 8192 - (C & 1) ? 16 : 32;
    k.warps = ceil_div(C + (C & 1), 32 * k.M);
    k.groups = 16 / k.warps;
    k.ctas = (int)std::min<long long>(sm_count(), (rows + k.groups - 1) / k.groups);
    return k;
}

template <typename io_t, int M>
cudaError_t backward(const Params &p, const Cut &k, int E, cudaStream_t stream) {
    cudaError_t r = cudaSuccess;
    with_pieces<io_t, M>(p.C, E, p.warps * 32, [&](auto e, auto n, auto kind) {
        auto *kernel = backward_kernel<io_t, decltype(e)::value, decltype(n)::value, decltype(kind)::value>;
        static std::atomic<unsigned long long> done{0};
        r = smem_attr_once(reinterpret_cast<const void *>(kernel),
                           Ahead<io_t, M>::bytes(512) + Ahead<io_t, M>::sum_bytes(512, sizeof(io_t) == 2 || M == 16 ? 8192 : 4096), done);
        if (r == cudaSuccess) {
            const int threads = k.groups * k.warps * 32;
            kernel<<<k.ctas, threads, Ahead<io_t, M>::bytes(threads) + Ahead<io_t, M>::sum_bytes(threads, p.C), stream>>>(p);
            r = cudaGetLastError();
        }
    });
    return r;
}

}  // namespace

size_t backward_scratch_bytes(long long rows, int C) {   // (the shares of either I/O type)
    return (size_t)std::max(cut(OSDN_F32, rows, C).ctas, cut(OSDN_BF16, rows, C).ctas) * C * 8;
}

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
    const Cut k = cut(io, rows, C);
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
    if (!p.columns) return cudaSuccess;
    return da::launch_overlapped(rows > 0, columns_kernel, dim3((2 * C + 31) / 32), kColumnWarps * 32, 0, stream, k.ctas,
                                 C, static_cast<const float *>(p.part), dweight, dbias);
}

}  // namespace ln
}  // namespace osdn
