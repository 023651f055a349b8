// gated_scan.cu -- a linear recurrence with a gate per token and channel, its
// single-token step and its gradients:
//     h_t = a_t h_{t-1} + w(a_t) x_t,   a_t = sigmoid(gate_t)
//     R_t = dh_t + Q_t,  Q_{t-1} = a_t R_t          (Q_T = dhT, dh0 = Q_0)
//     dx_t = w(a_t) R_t,   dgate_t = R_t (a_t (1 - a_t) h_{t-1} + w'_t x_t)
//
// Both directions are a recurrence s <- a s + e of every channel, and runs of
// it compose: (A, E) after (A', E') is (A A', A E' + E).  The tensors are read
// and written once, so HBM bounds them.  A warp holds R tokens of 32 lanes'
// channels (two a lane where rows allow) in registers, a CTA kWarps warps one
// behind the other in time, a cluster up to eight CTAs:
//   1  every thread folds its tokens to (A, E);
//   2  the warps' pairs meet in shared memory, the CTAs' totals in the cluster's
//      (distributed shared memory);
//   3  with the state that enters the cluster each thread has the state before
//      its first token, runs the recurrence over its registers and stores.
// A sequence longer than a cluster's tokens is a chain of clusters: the last CTA
// hands its state on in global memory, and the next cluster, whose loads and
// folds are done by then, waits for it.  The waiting words are set to a value
// that no state has by a small kernel in front; a state is its own flag.
// Clusters take numbers from a counter as they start, in the chain's order, so
// what one waits for has started before it; waits are bounded all the same.
// Every fold is in a fixed order: results do not depend on who waited.
#include <algorithm>
#include <type_traits>

#include "decay_attn.cuh"
#include "gated_scan.cuh"
#include "ptx.cuh"

namespace osdn {
namespace gs {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr unsigned kEmpty = 0xffffffffu;   // a NaN that no arithmetic yields
constexpr size_t kCounterBytes = 256;

// How a call is cut: clusters of n CTAs, each CTA kWarps R tokens of 32 V channels of a sequence.
struct Plan {
    int V, R, n;
    long long strips;   // columns of tiles: B times the strips of a sequence's channels
    int per_seq;        // strips a sequence
    int links;          // clusters along the time axis
    int chunk() const { return kWarps * R; }
    size_t state_bytes() const { return (size_t)(links - 1) * strips * 32 * V * 4; }
    size_t scratch_bytes() const { return links > 1 ? kCounterBytes + state_bytes() : 0; }
};

Plan plan(int B, int T, int C) {
    Plan p;
    p.V = C % 2 ? 1 : 2;
    p.per_seq = (C + 32 * p.V - 1) / (32 * p.V);
    p.strips = (long long)B * p.per_seq;
    p.R = T > kWarps * 4 * kMaxCluster ? 16 : 4;
    const int chunks = (T + p.chunk() - 1) / p.chunk();
    p.n = std::min(chunks, kMaxCluster);
    p.links = (chunks + p.n - 1) / p.n;
    return p;
}

struct Params {
    int T, C, per_seq, links;
    long long strips;
    const void *x, *gate, *h, *dh;
    const float *h0;        // (backward)
    const float *first;     // the state that enters: h0, or dhT
    void *out, *dgate;      // h, or dx and dgate
    float *last;            // the state that leaves: hT, or dh0
    unsigned *counter;
    unsigned *states;       // [links - 1][strips][32 V]
    int *status;
};

__global__ void __launch_bounds__(256) empty_kernel(uint4 *p, size_t n) {
    da::dependents_may_start();
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    const unsigned v = i < kCounterBytes / 16 ? 0u : kEmpty;
    p[i] = make_uint4(v, v, v, v);
}

template <int V>
struct Vec {
    float v[V];
};
template <int V>
__device__ __forceinline__ Vec<V> fill(float x) {
    Vec<V> r;
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = x;
    return r;
}
// V neighbouring channels as they lie in memory
template <typename io_t, int V>
struct Raw {
    typedef typename std::conditional<sizeof(io_t) * V == 8, uint2,
            typename std::conditional<sizeof(io_t) * V == 4, unsigned, unsigned short>::type>::type type;
};
template <typename io_t, int V>
__device__ __forceinline__ Vec<V> wide(typename Raw<io_t, V>::type u) {
    Vec<V> r;
    if constexpr (sizeof(io_t) == 4) {
        if constexpr (V == 2) {
            r.v[0] = __uint_as_float(u.x);
            r.v[1] = __uint_as_float(u.y);
        } else {
            r.v[0] = __uint_as_float(u);
        }
    } else {
        r.v[0] = __uint_as_float((unsigned)u << 16);
        if constexpr (V == 2) r.v[1] = __uint_as_float(u & 0xffff0000u);
    }
    return r;
}
template <typename io_t, int V>
__device__ __forceinline__ void put(io_t *p, const Vec<V> &x) {
    if constexpr (V == 2) {
        store2(p, x.v);
    } else {
        from_f32(*p, x.v[0]);
    }
}

// (A, E) pairs of V channels: s <- A s + E.
template <int V>
struct Pair {
    float2 v[V];
    __device__ __forceinline__ void apply(Vec<V> &s) const {
#pragma unroll
        for (int i = 0; i < V; ++i) s.v[i] = hide(v[i].x, s.v[i]) + v[i].y;
    }
    __device__ __forceinline__ void then(const Pair &b) {   // this one first, then b
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = make_float2(b.v[i].x * v[i].x, hide(b.v[i].x, v[i].y) + b.v[i].y);
    }
};

// What a CTA's threads share: its tile, and the join of the recurrence over warps, CTAs and clusters.
template <int V>
struct Join {
    float2 warp[kWarps][32 * V];
    float2 total[32 * V];
    float start[32 * V];
    unsigned ticket;
};

// The tile of this CTA: which strip, and which chunk of tokens, counted from the end of the sequence
// that the recurrence starts from.
struct Tile {
    long long strip;
    int link, rank, n;
};
template <int V>
__device__ __forceinline__ Tile take_tile(const Params &p, Join<V> &j) {
    Tile t;
    t.rank = ptx::cluster_rank();
    t.n = ptx::cluster_size();
    unsigned id = blockIdx.x / t.n;
    t.link = 0;
    if (p.links > 1) {
        da::dependency_wait();   // the counter and the states are set
        if (t.rank == 0 && threadIdx.x == 0) j.ticket = atomicAdd(p.counter, 1u);
        ptx::cluster_arrive();
        ptx::cluster_wait();
        id = ptx::cluster_load(ptx::cluster_map(&j.ticket, 0), 0u);
        t.link = (int)(id / p.strips);
    }
    t.strip = id - t.link * p.strips;
    return t;
}

// V words that are not empty, or zeros after `limit` looks.
template <int V>
__device__ __forceinline__ bool wait_states(const unsigned *p, unsigned limit, Vec<V> &s) {
    for (unsigned i = 0; i < limit; ++i) {
        unsigned a, b = 0;
        if constexpr (V == 2) {
            unsigned long long u;
            asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(u) : "l"(p) : "memory");
            a = (unsigned)u;
            b = (unsigned)(u >> 32);
        } else {
            asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(a) : "l"(p) : "memory");
        }
        if (a != kEmpty && b != kEmpty) {
            s.v[0] = __uint_as_float(a);
            if constexpr (V == 2) s.v[1] = __uint_as_float(b);
            return true;
        }
    }
    return false;
}
template <int V>
__device__ __forceinline__ void hand_on(unsigned *p, const Vec<V> &s) {
    unsigned u[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        u[i] = __float_as_uint(s.v[i]);
        if (u[i] == kEmpty) u[i] = 0x7fffffffu;
    }
    if constexpr (V == 2)
        asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"((unsigned long long)u[1] << 32 | u[0])
                     : "memory");
    else
        asm volatile("st.relaxed.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(u[0]) : "memory");
}

constexpr unsigned kLooks = 1u << 22;        // seconds
constexpr unsigned kLooksTest = 1u << 10;

// From each thread's (A, E) the state before its first token.  Warps are folded in the order
// `order(0), order(1), ..`: a warp's place in the recurrence.
template <int V>
__device__ __forceinline__ Vec<V> join(const Params &p, const Tile &t, Join<V> &j, const Pair<V> &own, int place,
                                       int c, size_t state) {
    const int lane = threadIdx.x & 31;
    const bool live = c < p.C;
#pragma unroll
    for (int i = 0; i < V; ++i) j.warp[place][lane * V + i] = own.v[i];
    __syncthreads();
    Pair<V> total;
    if (threadIdx.x < 32) {
#pragma unroll
        for (int i = 0; i < V; ++i) total.v[i] = j.warp[0][lane * V + i];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            Pair<V> b;
#pragma unroll
            for (int i = 0; i < V; ++i) b.v[i] = j.warp[w][lane * V + i];
            total.then(b);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) j.total[lane * V + i] = total.v[i];
    }
    if (t.n > 1) {
        ptx::cluster_arrive();
        ptx::cluster_wait();
    }
    if (threadIdx.x < 32) {
        Pair<V> before[kMaxCluster - 1];
#pragma unroll
        for (int r = 0; r < kMaxCluster - 1; ++r)
            if (r < t.rank) {
                const uint32_t a = ptx::cluster_map(&j.total[lane * V], r);
#pragma unroll
                for (int i = 0; i < V; ++i) before[r].v[i] = ptx::cluster_load(a + 8 * i, float2());
            }
        Vec<V> s = fill<V>(0.0f);
        if (t.link == 0) {
            if (p.first && live)
#pragma unroll
                for (int i = 0; i < V; ++i) s.v[i] = p.first[state + i];
        } else if (live) {
            const bool test = p.status[1] != 0;
            const size_t at = ((size_t)(t.link - 1) * p.strips + t.strip) * (32 * V) + lane * V;
            if (!wait_states<V>(p.states + at, test ? kLooksTest : kLooks, s))
                report_status(p.status, OSDN_ERR_TIMEOUT);
        }
#pragma unroll
        for (int r = 0; r < kMaxCluster - 1; ++r)
            if (r < t.rank) before[r].apply(s);
#pragma unroll
        for (int i = 0; i < V; ++i) j.start[lane * V + i] = s.v[i];
        if (t.rank == t.n - 1 && live) {
            total.apply(s);
            if (t.link < p.links - 1) {
                if (p.status[1] == 0)   // the test word: nothing is handed on, so that waits run out
                    hand_on<V>(p.states + ((size_t)t.link * p.strips + t.strip) * (32 * V) + lane * V, s);
            } else if (p.last) {
#pragma unroll
                for (int i = 0; i < V; ++i) p.last[state + i] = s.v[i];
            }
        }
    }
    __syncthreads();
    if (t.n > 1) ptx::cluster_arrive();   // this CTA has read the others' totals
    Vec<V> s;
#pragma unroll
    for (int i = 0; i < V; ++i) s.v[i] = j.start[lane * V + i];
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w)
        if (w < place) {
            Pair<V> b;
#pragma unroll
            for (int i = 0; i < V; ++i) b.v[i] = j.warp[w][lane * V + i];
            b.apply(s);
        }
    return s;
}

template <typename io_t, int V, int MIX, int R>
__global__ void __launch_bounds__(kThreads) scan_kernel(Params p) {
    typedef typename Raw<io_t, V>::type raw_t;
    __shared__ Join<V> j;
    const Tile t = take_tile(p, j);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long b = t.strip / p.per_seq;
    const int c = (int)(t.strip - b * p.per_seq) * (32 * V) + lane * V;
    const bool live = c < p.C;
    // T is at most 2^30, and a cluster's tokens a few thousand
    const int t0 = (t.link * t.n + t.rank) * (kWarps * R) + warp * R;
    const int tokens = live ? min(R, p.T - t0) : 0;
    const size_t at = ((size_t)b * p.T + t0) * p.C + c;
    const io_t *gate = static_cast<const io_t *>(p.gate) + at, *x = static_cast<const io_t *>(p.x) + at;
    float co[R][V];
    raw_t rx[R];
    {
        raw_t rg[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rg[i] = raw_t();
            rx[i] = raw_t();
            if (i < tokens) {
                rg[i] = *reinterpret_cast<const raw_t *>(gate + (size_t)i * p.C);
                rx[i] = *reinterpret_cast<const raw_t *>(x + (size_t)i * p.C);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> g = wide<io_t, V>(rg[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) co[i][v] = i < tokens ? gate_coefficient(g.v[v]) : -0.0f;
        }
    }
    float least = 1.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) least = fminf(least, fabsf(co[i][v]));
    const bool zeros = __any_sync(kFullMask, least == 0.0f);
    Pair<V> own;
    const auto fold = [&](auto z) {
        constexpr bool Z = decltype(z)::value;
#pragma unroll
        for (int v = 0; v < V; ++v) own.v[v] = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> xi = wide<io_t, V>(rx[i]);
#pragma unroll
            for (int v = 0; v < V; ++v)
                own.v[v] = make_float2(decay<Z>(co[i][v], own.v[v].x),
                                       decay<Z>(co[i][v], own.v[v].y) + weighted<MIX, Z>(co[i][v], xi.v[v]));
        }
    };
    if (zeros) fold(std::true_type()); else fold(std::false_type());
    Vec<V> s = join<V>(p, t, j, own, warp, c, (size_t)b * p.C + c);
    io_t *h = static_cast<io_t *>(p.out) + at;
    const auto run = [&](auto z) {
        constexpr bool Z = decltype(z)::value;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> xi = wide<io_t, V>(rx[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) s.v[v] = decay<Z>(co[i][v], s.v[v]) + weighted<MIX, Z>(co[i][v], xi.v[v]);
            if (i < tokens) put<io_t, V>(h + (size_t)i * p.C, s);
        }
    };
    if (zeros) run(std::true_type()); else run(std::false_type());
    if (t.n > 1) ptx::cluster_wait();   // the others have read this CTA's total
}

// Backwards in time: chunks, warps and tokens from the last to the first.  The states are recomputed
// from the row of h in front of the warp's tokens: one row in R is read again, instead of all.
template <typename io_t, int V, int MIX, int R>
__global__ void __launch_bounds__(kThreads) backward_kernel(Params p) {
    typedef typename Raw<io_t, V>::type raw_t;
    __shared__ Join<V> j;
    const Tile t = take_tile(p, j);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long b = t.strip / p.per_seq;
    const int c = (int)(t.strip - b * p.per_seq) * (32 * V) + lane * V;
    const bool live = c < p.C;
    const int t0 = (p.links * t.n - 1 - (t.link * t.n + t.rank)) * (kWarps * R) + warp * R;
    const int tokens = live ? max(0, min(R, p.T - t0)) : 0;
    const size_t state = (size_t)b * p.C + c, at = ((size_t)b * p.T + t0) * p.C + c;
    const io_t *gate = static_cast<const io_t *>(p.gate) + at, *x = static_cast<const io_t *>(p.x) + at;
    const io_t *dh = static_cast<const io_t *>(p.dh) + at;
    float co[R][V], before[R][V];
    raw_t rx[R], rd[R];
    Vec<V> s = fill<V>(0.0f);
    {
        raw_t rg[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            rg[i] = rx[i] = rd[i] = raw_t();
            if (i < tokens) {
                rg[i] = *reinterpret_cast<const raw_t *>(gate + (size_t)i * p.C);
                rx[i] = *reinterpret_cast<const raw_t *>(x + (size_t)i * p.C);
                rd[i] = *reinterpret_cast<const raw_t *>(dh + (size_t)i * p.C);
            }
        }
        if (tokens > 0 && t0 > 0) {
            s = wide<io_t, V>(*reinterpret_cast<const raw_t *>(static_cast<const io_t *>(p.h) + at - p.C));
        } else if (tokens > 0 && p.h0) {
#pragma unroll
            for (int v = 0; v < V; ++v) s.v[v] = p.h0[state + v];
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> g = wide<io_t, V>(rg[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) co[i][v] = i < tokens ? gate_coefficient(g.v[v]) : -0.0f;
        }
    }
    float least = 1.0f;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) least = fminf(least, fabsf(co[i][v]));
    const bool zeros = __any_sync(kFullMask, least == 0.0f);
    Pair<V> own;
    const auto fold = [&](auto z) {
        constexpr bool Z = decltype(z)::value;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> xi = wide<io_t, V>(rx[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                before[i][v] = s.v[v];
                s.v[v] = decay<Z>(co[i][v], s.v[v]) + weighted<MIX, Z>(co[i][v], xi.v[v]);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) own.v[v] = make_float2(1.0f, 0.0f);
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const Vec<V> d = wide<io_t, V>(rd[i]);
#pragma unroll
            for (int v = 0; v < V; ++v)
                own.v[v] = make_float2(decay<Z>(co[i][v], own.v[v].x), decay<Z>(co[i][v], d.v[v] + own.v[v].y));
        }
    };
    if (zeros) fold(std::true_type()); else fold(std::false_type());
    Vec<V> q = join<V>(p, t, j, own, kWarps - 1 - warp, c, state);
    io_t *dx = static_cast<io_t *>(p.out) + at, *dgate = static_cast<io_t *>(p.dgate) + at;
    const auto run = [&](auto z) {
        constexpr bool Z = decltype(z)::value;
#pragma unroll
        for (int i = R - 1; i >= 0; --i) {
            const Vec<V> xi = wide<io_t, V>(rx[i]), d = wide<io_t, V>(rd[i]);
            Vec<V> gx, gg;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float r = d.v[v] + q.v[v];
                gradients<MIX, Z>(co[i][v], r, before[i][v], xi.v[v], gx.v[v], gg.v[v]);
                q.v[v] = decay<Z>(co[i][v], r);
            }
            if (i < tokens) {
                put<io_t, V>(dx + (size_t)i * p.C, gx);
                put<io_t, V>(dgate + (size_t)i * p.C, gg);
            }
        }
    };
    if (zeros) run(std::true_type()); else run(std::false_type());
    if (t.n > 1) ptx::cluster_wait();
}

// One token: h and the I/O tensors are flat, four elements a thread.
template <typename io_t, int MIX>
__global__ void __launch_bounds__(128) step_kernel(long long n, const io_t *x, const io_t *gate, float *h, io_t *y) {
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) * 4;
    if (i >= n) return;
    float xv[4], gv[4], hv[4];
    const bool whole = i + 4 <= n;
    if (whole) {
        load4(x + i, xv);
        load4(gate + i, gv);
        load4(h + i, hv);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            xv[e] = gv[e] = hv[e] = 0.0f;
            if (i + e < n) {
                xv[e] = to_f32(x[i + e]);
                gv[e] = to_f32(gate[i + e]);
                hv[e] = h[i + e];
            }
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float c = gate_coefficient(gv[e]);
        hv[e] = decay<true>(c, hv[e]) + weighted<MIX, true>(c, xv[e]);
    }
    if (whole) {
        store4(h + i, hv);
        store4(y + i, hv);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) {
                h[i + e] = hv[e];
                from_f32(y[i + e], hv[e]);
            }
    }
}

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

template <typename io_t, int V, int MIX, int R>
void (*kernel_of(bool backward))(Params) {
    return backward ? backward_kernel<io_t, V, MIX, R> : scan_kernel<io_t, V, MIX, R>;
}

cudaError_t launch(int io, int mix, bool backward, int B, int T, int C, Params p, void *scratch, int *status,
                   cudaStream_t stream) {
    const Plan pl = plan(B, T, C);
    p.T = T; p.C = C;
    p.per_seq = pl.per_seq;
    p.strips = pl.strips;
    p.links = pl.links;
    p.status = status;
    p.counter = static_cast<unsigned *>(scratch);
    p.states = reinterpret_cast<unsigned *>(static_cast<char *>(scratch) + kCounterBytes);
    void (*kernel)(Params) = nullptr;
    with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        constexpr int M = decltype(m)::value;
        if (pl.V == 2)
            kernel = pl.R == 16 ? kernel_of<io_t, 2, M, 16>(backward) : kernel_of<io_t, 2, M, 4>(backward);
        else
            kernel = pl.R == 16 ? kernel_of<io_t, 1, M, 16>(backward) : kernel_of<io_t, 1, M, 4>(backward);
        return cudaSuccess;
    });
    if (pl.links > 1) {
        const size_t n = pl.scratch_bytes() / 16;   // (states come 128 bytes a strip at least)
        empty_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(static_cast<uint4 *>(scratch), n);
        if (cudaError_t e = cudaGetLastError()) return e;
    }
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(pl.strips * pl.links * pl.n));
    c.blockDim = dim3(kThreads);
    c.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = pl.n;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = at;
    c.numAttrs = pl.links > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, p);
}

}  // namespace

size_t scan_scratch_bytes(int, int B, int T, int C) { return plan(B, T, C).scratch_bytes(); }
size_t backward_scratch_bytes(int, int B, int T, int C) { return plan(B, T, C).scratch_bytes(); }

cudaError_t scan_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                        void *h, float *hT, void *scratch, int *status, cudaStream_t stream) {
    Params p = {};
    p.x = x; p.gate = gate;
    p.first = h0;
    p.out = h;
    p.last = hT;
    return launch(io, mix, false, B, T, C, p, scratch, status, stream);
}

cudaError_t step_launch(int io, int B, int C, int mix, const void *x, const void *gate, float *h, void *y,
                        cudaStream_t stream) {
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        const long long n = (long long)B * C;
        step_kernel<io_t, decltype(m)::value><<<(unsigned)((n + 511) / 512), 128, 0, stream>>>(
            n, static_cast<const io_t *>(x), static_cast<const io_t *>(gate), h, static_cast<io_t *>(y));
        return cudaGetLastError();
    });
}

cudaError_t backward_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const void *h,
                            const float *h0, const void *dh, const float *dhT, void *dx, void *dgate, float *dh0,
                            void *scratch, int *status, cudaStream_t stream) {
    Params p = {};
    p.x = x; p.gate = gate; p.h = h; p.dh = dh;
    p.h0 = h0;
    p.first = dhT;
    p.out = dx; p.dgate = dgate;
    p.last = dh0;
    return launch(io, mix, true, B, T, C, p, scratch, status, stream);
}

}  // namespace gs
}  // namespace osdn
