// gated_scan_walk.cuh -- what the recurrence (gated_scan.cu) and its gradients
// (gated_scan_backward.cu) share: the walk of a cluster over its strip of
// channels, the copies ahead into shared memory and the join of what threads,
// warps and CTAs have folded.  gated_scan.cu describes the whole.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gated_scan.cuh"
#include "ptx.cuh"

namespace osdn {
namespace gs {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;

struct Params {
    int T, C, per_seq;      // per_seq: strips of 64 channels a sequence
    int steps;              // of n kWarps R tokens
    const void *x, *gate, *h, *dh;
    const float *h0;        // (gradients)
    const float *first;     // the state that enters: h0, or dhT
    void *out, *dgate;      // h, or dx and dgate
    float *last;            // the state that leaves: hT, or dh0
};

// A lane's two neighbouring channels as they lie in memory.
template <typename io_t>
struct Raw {
    typedef typename std::conditional<sizeof(io_t) == 4, uint2, unsigned>::type type;
};
__device__ __forceinline__ Vec<2> wide(uint2 u) { return {{__uint_as_float(u.x), __uint_as_float(u.y)}}; }
__device__ __forceinline__ Vec<2> wide(unsigned u) {
    return {{__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u)}};
}
// PAIRED: rows keep the boundaries of two channels; else `second`: whether the second one exists
template <bool PAIRED, typename io_t>
__device__ __forceinline__ void put(io_t *p, const Vec<2> &x, bool second) {
    if constexpr (PAIRED) {
        store2(p, x.v);
    } else {
        from_f32(p[0], x.v[0]);
        if (second) from_f32(p[1], x.v[1]);
    }
}

// R rows (tokens) of a strip of 64 channels in shared memory, and how a warp gets them.  W: 16, 8 or 4
// bytes a copy, or 2: rows of an odd number of bf16, which start anywhere; the nine 16-byte pieces around
// a row are copied, and it begins `in` bytes into its place.
template <typename io_t, int R, int W>
struct Rows {
    typedef typename Raw<io_t>::type raw_t;
    static constexpr bool kPaired = W >= 2 * (int)sizeof(io_t);
    static constexpr int kRow = 64 * (int)sizeof(io_t);          // bytes a row
    static constexpr int kPitch = W == 2 ? kRow + 16 : kRow;     // in shared memory
    static constexpr int kBytes = R * kPitch;
    // rows 0 .. n - 1 from `src`, `pitch` bytes apart, the first `valid` bytes of each; zeros for the rest
    __device__ __forceinline__ static void fetch(uint32_t dst, const char *src, unsigned pitch, int n, int valid) {
        const int lane = threadIdx.x & 31;
        if constexpr (W == 2) {
            const char *const start = src - (reinterpret_cast<uintptr_t>(src) & 15);
            const int r0 = lane / 9, q = lane % 9 * 16;   // three rows a warp at once
#pragma unroll
            for (int r = 0; r < R; r += 3) {
                const char *row = src + (size_t)(r + r0) * pitch;
                const int in = (int)(reinterpret_cast<uintptr_t>(row) & 15);
                const int left = r + r0 < n ? in + valid - q : 0;
                if (lane < 27 && r + r0 < R)
                    ptx::copy_async<16>(dst + (r + r0) * kPitch + q, left > 0 ? row - in + q : start, max(0, min(16, left)));
            }
        } else {
            constexpr int per = kRow / W;                 // copies a row
            constexpr int many = per < 32 ? 32 / per : 1; // rows a warp at once
            constexpr int turns = per < 32 ? 1 : per / 32;
            const int r0 = lane / per, q = lane % per * W;
            const char *p = src + (size_t)r0 * pitch + q;
            if (n >= R && valid == kRow) {
#pragma unroll
                for (int r = 0; r < R; r += many)
#pragma unroll
                    for (int t = 0; t < turns; ++t)
                        ptx::copy_async<W>(dst + (r + r0) * kPitch + q + t * 32 * W, p + (size_t)r * pitch + t * 32 * W, W);
            } else {
#pragma unroll
                for (int r = 0; r < R; r += many)
#pragma unroll
                    for (int t = 0; t < turns; ++t) {
                        const bool there = r + r0 < n && q + t * 32 * W < valid;
                        ptx::copy_async<W>(dst + (r + r0) * kPitch + q + t * 32 * W,
                                      there ? p + (size_t)r * pitch + t * 32 * W : src, there ? W : 0);
                    }
            }
        }
    }
    // this lane's channels of row r; `in`: where row 0 begins in its place
    __device__ __forceinline__ static raw_t get(const char *p, int r, int in, unsigned pitch) {
        const char *at = p + r * kPitch + (threadIdx.x & 31) * sizeof(raw_t);
        if constexpr (W == 2) {
            const unsigned short *q = reinterpret_cast<const unsigned short *>(at + ((in + r * pitch) & 15));
            return (unsigned)q[0] | (unsigned)q[1] << 16;
        } else {
            return *reinterpret_cast<const raw_t *>(at);
        }
    }
};

// What a run of tokens does to a lane's channels, s <- A s + E.  A is held as one signed number c, as a gate
// is (gated_scan.cuh): -(1 - A) where that is small, with its digits, else A.  An A near 1 that is rounded to
// fp32 takes up to 2^-25 of the state with it, or adds as much, at every run, and to the same side where gates
// are constant.  (Measured, 2x8192x2048 bf16: 50 us either way, gradients 89 us either way with mean, 70
// for 68 us with sum and 87 for 85 us with unit.)
constexpr float kNear = 0.125f;   // (eight factors of 1 - kNear are still 0.34: see join)
struct alignas(16) Pair {
    Vec<2> c, E;
};
// c of A and D = 1 - A where A is near 1; never a zero with a sign, so that `c < 0` says which it is
__device__ __forceinline__ float near_one(float D) { return -fmaxf(D, 1e-38f); }
__device__ __forceinline__ Pair own_run(const Vec<2> &A, const Vec<2> &D, const Vec<2> &E) {
    Pair p = {A, E};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if (D.v[i] < 0.5f) p.c.v[i] = 1.0f - D.v[i];   // (A is a product of many)
        if (D.v[i] < kNear) p.c.v[i] = near_one(D.v[i]);
    }
    return p;
}
// 1 where c is held as -(1 - A), else 0: A = unit(c) + c
__device__ __forceinline__ Vec<2> unit(const Vec<2> &c) { return {{c.v[0] < 0.0f ? 1.0f : 0.0f, c.v[1] < 0.0f ? 1.0f : 0.0f}}; }
// A s + E, where that is finite; else the exact form: an A that is exactly zero hides s, and an infinite s
// stays as it is.
__device__ __forceinline__ Vec<2> through(const Pair &b, const Vec<2> &s) { return fma(b.c, s, fma(unit(b.c), s, b.E)); }
__device__ __forceinline__ Vec<2> through_exact(const Pair &b, const Vec<2> &s) {
    return {{decay<kAny>(b.c.v[0], s.v[0]) + b.E.v[0], decay<kAny>(b.c.v[1], s.v[1]) + b.E.v[1]}};
}

// Where a step's pairs meet; one set for even and one for odd steps, so that a step's barriers are
// enough: who writes a set again has passed the barriers of the step between.
struct Join {
    Pair warp[2][kWarps][32];
    Pair total[2][kMaxCluster][32];
    Vec<2> entered[2][32];   // the state that enters the step
};
// From every thread's own run and the state s that enters the step: the state before the thread's first
// token.  s becomes the state after the step (where a CTA walks alone, its last warp's only: that one hands it
// to the others in the next step).  `place`: the warp's turn in the recurrence.  `meanwhile()` runs while the
// cluster's CTAs wait for one another.
template <typename F>
__device__ __forceinline__ Vec<2> join(Join &j, int set, int n, int rank, int place, const Pair &own, Vec<2> &s,
                                       const F &meanwhile) {
    const int lane = threadIdx.x & 31;
    const bool last = place == kWarps - 1;
    const Vec<2> one = fill<2>(1.0f), zero = fill<2>(0.0f);
    j.warp[set][place][lane] = own;
    if (last) j.entered[set][lane] = s;
    __syncthreads();
    if (n == 1) s = j.entered[set][lane];
    // What lies before this warp in the CTA.  It goes no further than the warp's own tokens: A may be rounded.
    Vec<2> A = one, E = zero;
    Pair sum;
    if (!last) {
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w) {
            if (w >= place) break;
            const Pair b = j.warp[set][w][lane];
            const Vec<2> a = add(b.c, unit(b.c));
            E = fma(a, E, b.E);
            A = mul(a, A);
        }
    } else {
        // What the CTA does in all.  A = P + C, with P 0 or 1; with P = 1 every A is at least 1 - kNear and
        // their product at least 0.34, so that C has the digits of A as well as those of 1 - A.
        Vec<2> P = one, C = zero, T = zero;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const Pair b = w == kWarps - 1 ? own : j.warp[set][w][lane];
            const Vec<2> p = unit(b.c);
            if (w == kWarps - 1) A = add(P, C), E = T;
            T = fma(b.c, T, fma(p, T, b.E));
            C = fma(C, b.c, fma(C, p, mul(P, b.c)));
            P = mul(P, p);
        }
        sum.E = T;
        sum.c = add(P, C);
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (P.v[i] != 0.0f && -C.v[i] < kNear) sum.c.v[i] = near_one(-C.v[i]);
    }
    if (!finite(E) || (last && !finite(sum.E))) {
        // exactly; an A of zero is zero before and behind a gate of NaN, too
        E = zero;
        for (int w = 0; w < place; ++w) {
            const Pair b = j.warp[set][w][lane];
            E = through_exact(b, E);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (forgets(b.c.v[i])) A.v[i] = sum.c.v[i] = 0.0f;
        }
        if (last) {
            sum.E = through_exact(own, E);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (forgets(own.c.v[i])) sum.c.v[i] = 0.0f;
        }
    }
    Vec<2> mine = s;
    if (n > 1) {
        if (last) {   // to every CTA of the cluster
            for (int r = 0; r < n; ++r) {
                const uint32_t at = ptx::cluster_map(&j.total[set][rank][lane], r);
                ptx::cluster_store(at, make_float4(sum.c.v[0], sum.c.v[1], sum.E.v[0], sum.E.v[1]));
            }
        }
        // Only the last warp has written for the others.  What every warp has read of an earlier step
        // comes before it, by the barrier of the CTA.
        __syncwarp();
        if (last) ptx::cluster_arrive(); else ptx::cluster_arrive_relaxed();
        meanwhile();
        ptx::cluster_wait();
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < n) {
                if (r == rank) mine = s;
                s = through(j.total[set][r][lane], s);
            }
        if (!finite(s)) {
            s = j.entered[set][lane];
            for (int r = 0; r < n; ++r) {
                if (r == rank) mine = s;
                s = through_exact(j.total[set][r][lane], s);
            }
        }
    } else {
        meanwhile();
        if (last) {
            s = through(sum, s);
            if (!finite(s)) s = through_exact(sum, j.entered[set][lane]);
        }
    }
    Vec<2> q = fma(A, mine, E);
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (A.v[i] == 0.0f) q.v[i] = E.v[i];
    return q;
}

constexpr int kStages = 2;   // steps on their way into shared memory

// What the two kernels share: the place of a thread, and the copies of K tensors.
template <typename io_t, int R, int W, int K>
struct Walk {
    typedef Rows<io_t, R, W> rows;
    int n, rank, lane, warp, b, c0, c, stride, t0;
    bool live, second;   // whether this lane's two channels exist
    unsigned pitch;
    int valid;           // bytes of the strip's channels
    size_t at;           // of row t0, channel c0
    uint32_t smem;       // this warp's place
    const char *mine;
    __device__ __forceinline__ Walk(const Params &p, char *sm, bool backward) {
        n = ptx::cluster_size();
        rank = ptx::cluster_rank();
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        const int strip = blockIdx.x / n;
        b = strip / p.per_seq;
        c0 = (strip - b * p.per_seq) * 64;
        c = c0 + lane * 2;
        live = c < p.C;
        second = c + 1 < p.C;
        pitch = p.C * (unsigned)sizeof(io_t);
        valid = min(64, p.C - c0) * (int)sizeof(io_t);
        stride = n * (kWarps * R);                 // tokens a step; T is at most 2^30
        t0 = (backward ? p.steps * n - 1 - rank : rank) * (kWarps * R) + warp * R;
        at = ((size_t)b * p.T + t0) * p.C + c0;
        mine = sm + warp * (kStages * K * rows::kBytes);
        smem = ptx::smem_u32(mine);
    }
    __device__ __forceinline__ void fetch(int stage, int k, const void *base, size_t from, int tokens) const {
        // (computed where it is needed: kept over the steps, rows' offsets would take the tokens' registers)
        unsigned pitch = this->pitch;
        asm volatile("" : "+r"(pitch));
        rows::fetch(smem + (stage * K + k) * rows::kBytes,
                    reinterpret_cast<const char *>(static_cast<const io_t *>(base) + from), pitch, tokens, valid);
    }
    __device__ __forceinline__ const char *tile(int stage, int k) const { return mine + (stage * K + k) * rows::kBytes; }
    __device__ __forceinline__ int in(const void *base) const {   // where row t0 begins in its place
        return W == 2 ? (int)((reinterpret_cast<uintptr_t>(base) + at * 2) & 15) : 0;
    }
    // a state [B][C] fp32 (zeros without one)
    __device__ __forceinline__ Vec<2> load_state(const Params &p, const float *s) const {
        Vec<2> v = fill<2>(0.0f);
        if (s && live) v.v[0] = s[(size_t)b * p.C + c];
        if (s && second) v.v[1] = s[(size_t)b * p.C + c + 1];
        return v;
    }
    __device__ __forceinline__ void store_state(const Params &p, float *s, const Vec<2> &v) const {
        if (s && live) s[(size_t)b * p.C + c] = v.v[0];
        if (s && second) s[(size_t)b * p.C + c + 1] = v.v[1];
    }
};

// Values of this size and less stay finite over a warp's tokens, whatever the gates.
constexpr float kCalm = 1e36f;
__device__ __forceinline__ bool calm(const Vec<2> &a) { return fabsf(a.v[0]) <= kCalm && fabsf(a.v[1]) <= kCalm; }
// The arithmetic that a warp's tokens ask for (gated_scan.cuh): kPlain, by the gates alone; kEnds, where some
// gates are infinite or some tokens past the end, and all values calm; else kAny.  (kAny is several times the
// instructions, and one warp of it in a step holds up its cluster: 306 us at 1x65536x2048 with documents of 3000
// tokens, with kEnds 210 us.)
template <int R, typename F, typename G>
__device__ __forceinline__ int kind_of(const F &gate, const G &values, int tokens, bool live) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const Vec<2> g = gate(i);
        most = fmaxf(most, fmaxf(fabsf(g.v[0]), fabsf(g.v[1])));
    }
    if (__builtin_expect(__all_sync(kFullMask, tokens >= R && (most <= kPlainGate || !live)), 1)) return kPlain;
    bool ends = true;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const Vec<2> g = gate(i);
#pragma unroll
        for (int v = 0; v < 2; ++v) ends &= fabsf(g.v[v]) <= kPlainGate || fabsf(g.v[v]) == INFINITY;
        ends &= values(i);
    }
    return __all_sync(kFullMask, ends || !live) ? kEnds : kAny;
}
template <int X>
using Int = std::integral_constant<int, X>;

// f(type tag, mix tag) for the call's type and mix
template <typename F>
cudaError_t with_types(int io, int mix, const F &f) {
    const auto by_mix = [&](auto t) {
        if (mix == OSDN_MIX_SUM) return f(t, Mix<OSDN_MIX_SUM>());
        if (mix == OSDN_MIX_MEAN) return f(t, Mix<OSDN_MIX_MEAN>());
        return f(t, Mix<OSDN_MIX_UNIT>());
    };
    return io == OSDN_F32 ? by_mix(float()) : by_mix(__nv_bfloat16());
}

// How a call is cut: clusters of n CTAs a strip of 64 channels, R tokens a warp.
struct Plan {
    int R, W, n, steps, per_seq;
    long long strips;
};
// `most`: the most tokens a warp holds in registers (4 at least, in powers of two).
inline Plan plan(int io, int most, int B, int T, int C) {
    Plan best = {};
    const int row = C * (io == OSDN_F32 ? 4 : 2);
    Plan p = {};
    p.W = C % (io == OSDN_F32 ? 4 : 8) == 0 ? 16 : row % 8 == 0 && io == OSDN_F32 ? 8 : row % 4 == 0 ? 4 : 2;
    p.per_seq = (C + 63) / 64;
    p.strips = (long long)B * p.per_seq;
    for (p.R = 4; p.R <= most; p.R *= 2) {
        const int chunks = (T + kWarps * p.R - 1) / (kWarps * p.R);
        // two CTAs an SM, in clusters of up to eight, are about 256
        p.n = 1;
        while (p.n < kMaxCluster && 2 * p.n * p.strips <= 288 && p.n < chunks) p.n *= 2;
        p.steps = (chunks + p.n - 1) / p.n;
        // a step takes its tokens and a join that is worth about four
        if (!best.R || (long long)p.steps * (p.R + 4) <= (long long)best.steps * (best.R + 4)) best = p;
    }
    return best;
}

// K: the tensors that the kernel copies.
template <typename io_t, int R, int W, int K>
cudaError_t launch_as(void (*kernel)(Params), std::atomic<unsigned long long> &done, const Plan &pl, const Params &p,
                      cudaStream_t stream) {
    constexpr int smem = kWarps * kStages * K * Rows<io_t, R, W>::kBytes;
    const cudaError_t e = smem_attr_once(reinterpret_cast<const void *>(kernel), smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(pl.strips * pl.n));
    c.blockDim = dim3(kThreads);
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = pl.n;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    c.attrs = &at;
    c.numAttrs = pl.n > 1;
    return cudaLaunchKernelEx(&c, kernel, p);
}
// f(R tag, W tag) for a plan of at most MOST tokens a warp, of rows of odd bf16 at most ODD
template <typename io_t, int MOST, int ODD, typename F>
cudaError_t with_rows(const Plan &pl, const F &f) {
    const auto by_copy = [&](auto r) {
        constexpr bool f32 = sizeof(io_t) == 4, odd = !f32 && decltype(r)::value <= ODD;
        if (pl.W == 16) return f(r, Int<16>());
        if (f32 && pl.W == 8) return f(r, Int<f32 ? 8 : 4>());
        if (odd && pl.W == 2) return f(r, Int<odd ? 2 : 4>());
        return f(r, Int<4>());
    };
    return pl.R == 4 ? by_copy(Int<4>()) : pl.R == 8 ? by_copy(Int<8>()) : by_copy(Int<MOST>());
}

}  // namespace

}  // namespace gs
}  // namespace osdn
