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
// behind the other in time.  A strip of channels belongs to a cluster of up to
// eight CTAs, which walks the sequence, each step a run of tokens a CTA:
//   1  every thread turns its tokens into factors and folds them to (A, E);
//   2  the warps' pairs meet in shared memory, and, in a cluster, the CTAs'
//      totals in distributed shared memory;
//   3  every thread folds what lies before it onto the state that entered the
//      step, runs the recurrence over its factors and stores.
// A warp's tokens of the next two steps are on their way into shared memory
// meanwhile, by asynchronous copies of 16 bytes where rows keep 16-byte
// boundaries, else of words; a warp reads only what it copied itself.
// Nothing leaves the cluster, so there is no workspace and nothing to wait for
// but its own barrier.  Every fold is in a fixed order.
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
    int T, C, per_seq;      // per_seq: strips of 32 V channels a sequence
    int steps;              // of n kWarps R tokens
    const void *x, *gate, *h, *dh;
    const float *h0;        // (gradients)
    const float *first;     // the state that enters: h0, or dhT
    void *out, *dgate;      // h, or dx and dgate
    float *last;            // the state that leaves: hT, or dh0
};

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
// `bytes` of the W bytes at src (the rest: zeros) into shared memory, asynchronously.
template <int W>
__device__ __forceinline__ void copy_async(uint32_t dst, const char *src, int bytes) {
    if constexpr (W == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {   // all but the last N groups
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// R rows (tokens) of a strip of 32 V channels in shared memory, and how a warp gets them.  W: 16 or 4
// bytes a copy, or 2: rows of an odd number of bf16, of which every other starts inside a word; the
// words around it are copied, and a row begins 0 or 2 bytes into its place.
template <typename io_t, int V, int R, int W>
struct Rows {
    typedef typename Raw<io_t, V>::type raw_t;
    static constexpr int kRow = 32 * V * (int)sizeof(io_t);      // bytes a row
    static constexpr int kPitch = W == 2 ? kRow + 16 : kRow;     // in shared memory
    static constexpr int kBytes = R * kPitch;
    // rows 0 .. n - 1 from `src`, `pitch` bytes apart, the first `valid` bytes of each; zeros for the rest
    __device__ __forceinline__ static void fetch(uint32_t dst, const char *src, unsigned pitch, int n, int valid) {
        const int lane = threadIdx.x & 31;
        if constexpr (W == 2) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const char *row = src + (size_t)r * pitch;
                const int in = (int)(reinterpret_cast<uintptr_t>(row) & 2);   // bytes into its word
                const int left = r < n ? in + valid - 4 * lane : 0;
                if (lane <= kRow / 4)
                    copy_async<4>(dst + r * kPitch + 4 * lane, left > 0 ? row - in + 4 * lane : src - ((uintptr_t)src & 2),
                                  max(0, min(4, left)));
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
                        if (many <= R || r0 < R)
                            copy_async<W>(dst + (r + r0) * kPitch + q + t * 32 * W, p + (size_t)r * pitch + t * 32 * W, W);
            } else {
#pragma unroll
                for (int r = 0; r < R; r += many)
#pragma unroll
                    for (int t = 0; t < turns; ++t) {
                        const bool there = r + r0 < n && q + t * 32 * W < valid;
                        if (many <= R || r0 < R)
                            copy_async<W>(dst + (r + r0) * kPitch + q + t * 32 * W,
                                          there ? p + (size_t)r * pitch + t * 32 * W : src, there ? W : 0);
                    }
            }
        }
    }
    // this lane's channels of row r; `odd`: whether row 0 began inside a word
    __device__ __forceinline__ static raw_t get(const char *p, int r, int odd) {
        const int at = W == 2 ? r * kPitch + ((odd + r) & 1) * 2 : r * kPitch;
        return *reinterpret_cast<const raw_t *>(p + at + (threadIdx.x & 31) * (V * (int)sizeof(io_t)));
    }
};

// (A, E) pairs of V channels: s <- A s + E.
template <int V>
struct alignas(8 * V) Pair {
    Vec<V> A, E;
    // Z: an A that is exactly zero hides s.  (Without an exactly shut gate anywhere an A of zero is an
    // underflow, and takes nothing from a finite s.)
    template <bool Z>
    __device__ __forceinline__ void apply(Vec<V> &s) const {
        const Vec<V> r = fma(A, s, E);
#pragma unroll
        for (int i = 0; i < V; ++i) s.v[i] = Z && A.v[i] == 0.0f ? E.v[i] : r.v[i];
    }
    template <bool Z>
    __device__ __forceinline__ void then(const Pair &b) {   // this one first, then b
        b.template apply<Z>(E);
        A = mul(A, b.A);
    }
};

// Where a step's pairs meet; one set for even and one for odd steps, so that a step's barriers are
// enough: who writes a set again has passed the barriers of the step between.
template <int V>
struct Join {
    Pair<V> warp[2][kWarps][32];
    Pair<V> total[2][kMaxCluster][32];
};
// From every thread's (A, E) and the state s that enters the step: the state before the thread's
// first token.  s becomes the state after the step.  `place`: the warp's turn in the recurrence;
// `zeros`: whether a factor of this warp may be exactly zero.  `meanwhile()` runs while the cluster's
// CTAs wait for one another.
template <int V, typename F>
__device__ __forceinline__ Vec<V> join(Join<V> &j, int set, int n, int rank, int place, bool zeros, const Pair<V> &own,
                                       Vec<V> &s, const F &meanwhile) {
    const int lane = threadIdx.x & 31;
    j.warp[set][place][lane] = own;
    const bool any = __syncthreads_or(zeros);
    // what lies before this warp in the CTA, and what the CTA does in all
    Pair<V> before = {fill<V>(1.0f), fill<V>(0.0f)}, total = before;
    const auto fold = [&](auto z) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == place) before = total;
            total.template then<decltype(z)::value>(j.warp[set][w][lane]);
        }
    };
    if (any) fold(std::true_type()); else fold(std::false_type());
    Vec<V> mine = s;
    if (n > 1) {
        if (place == kWarps - 1) {   // the CTA's total, to every CTA of the cluster
            for (int r = 0; r < n; ++r) {
                const uint32_t at = ptx::cluster_map(&j.total[set][rank][lane], r);
                if constexpr (V == 2)
                    ptx::cluster_store(at, make_float4(total.A.v[0], total.A.v[1], total.E.v[0], total.E.v[1]));
                else
                    ptx::cluster_store(at, make_float2(total.A.v[0], total.E.v[0]));
            }
        }
        // Only the last warp has written for the others.  What every warp has read of an earlier step
        // comes before it, by the barrier of the CTA.
        __syncwarp();
        if (place == kWarps - 1) ptx::cluster_arrive(); else ptx::cluster_arrive_relaxed();
        meanwhile();
        ptx::cluster_wait();
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
            if (r < n) {
                if (r == rank) mine = s;
                j.total[set][r][lane].template apply<true>(s);
            }
    } else {
        meanwhile();
        total.template apply<true>(s);
    }
    before.template apply<true>(mine);
    return mine;
}

constexpr int kStages = 2;   // steps on their way into shared memory

// What the two kernels share: the place of a thread, and the copies of K tensors.
template <typename io_t, int V, int R, int W, int K>
struct Walk {
    typedef Rows<io_t, V, R, W> rows;
    int n, rank, lane, warp, b, c0, c, stride, t0;
    bool live;
    unsigned pitch;
    int valid;        // bytes of the strip's channels
    size_t at;        // of row t0, channel c0
    uint32_t smem;    // this warp's place
    const char *mine;
    __device__ __forceinline__ Walk(const Params &p, char *sm, bool backward) {
        n = ptx::cluster_size();
        rank = ptx::cluster_rank();
        lane = threadIdx.x & 31;
        warp = threadIdx.x >> 5;
        const int strip = blockIdx.x / n;
        b = strip / p.per_seq;
        c0 = (strip - b * p.per_seq) * (32 * V);
        c = c0 + lane * V;
        live = c < p.C;
        pitch = p.C * (unsigned)sizeof(io_t);
        valid = min(32 * V, p.C - c0) * (int)sizeof(io_t);
        stride = n * (kWarps * R);                 // tokens a step; T is at most 2^30
        t0 = (backward ? p.steps * n - 1 - rank : rank) * (kWarps * R) + warp * R;
        at = ((size_t)b * p.T + t0) * p.C + c0;
        mine = sm + warp * (kStages * K * rows::kBytes);
        smem = ptx::smem_u32(mine);
    }
    __device__ __forceinline__ void fetch(int stage, int k, const void *base, size_t from, int tokens) const {
        rows::fetch(smem + (stage * K + k) * rows::kBytes,
                    reinterpret_cast<const char *>(static_cast<const io_t *>(base) + from), pitch, tokens, valid);
    }
    __device__ __forceinline__ const char *tile(int stage, int k) const { return mine + (stage * K + k) * rows::kBytes; }
    __device__ __forceinline__ int odd(const void *base) const {
        return W == 2 ? (int)((reinterpret_cast<uintptr_t>(base) >> 1) + at) & 1 : 0;
    }
};

template <typename io_t, int V, int MIX, int R, int W>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(Params p) {
    constexpr bool kShort = sizeof(io_t) == 2;
    extern __shared__ __align__(16) char sm[];
    __shared__ Join<V> j;
    Walk<io_t, V, R, W, 2> k(p, sm, false);
    typedef Rows<io_t, V, R, W> rows;
    if (k.n > 1) ptx::cluster_arrive();   // every CTA of the cluster has started once all have arrived
    Vec<V> s = fill<V>(0.0f);
    if (p.first && k.live)
#pragma unroll
        for (int v = 0; v < V; ++v) s.v[v] = p.first[(size_t)k.b * p.C + k.c + v];
    const size_t far = (size_t)k.stride * p.C;   // elements a step
    const auto fetch = [&](int step, int ahead) {
        if (step + ahead < p.steps) {
            const size_t from = k.at + ahead * far;
            const int tokens = p.T - k.t0 - ahead * k.stride;
            k.fetch((step + ahead) % kStages, 0, p.gate, from, tokens);
            k.fetch((step + ahead) % kStages, 1, p.x, from, tokens);
        }
        copies_commit();   // (a group a step, so that waiting counts them)
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(0, i);
    if (k.n > 1) ptx::cluster_wait();
    for (int step = 0; step < p.steps; ++step) {
        copies_wait<kStages - 1>();
        __syncwarp();
        const int tokens = p.T - k.t0, odd = k.odd(p.gate), oddx = k.odd(p.x);
        const char *gate = k.tile(step % kStages, 0), *xs = k.tile(step % kStages, 1);
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> g = wide<io_t, V>(rows::get(gate, i, odd));
#pragma unroll
            for (int v = 0; v < V; ++v) most = fmaxf(most, fabsf(g.v[v]));
        }
        // all tokens there and no factor zero, for the whole warp
        const bool usual = __all_sync(kFullMask, tokens >= R && (most <= kPlainGate || !k.live));
        Vec<V> co[R], wx[R];
        Vec<V> A = fill<V>(1.0f), E = fill<V>(0.0f);
        const auto exact = [&](auto z) {
            constexpr bool Z = decltype(z)::value;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<V> g = wide<io_t, V>(rows::get(gate, i, odd)), x = wide<io_t, V>(rows::get(xs, i, oddx));
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    // tokens past the end leave everything as it is
                    co[i].v[v] = !Z || i < tokens ? gate_coefficient(g.v[v]) : -0.0f;
                    wx[i].v[v] = !Z || i < tokens ? weighted<MIX, Z>(co[i].v[v], x.v[v]) : 0.0f;
                    A.v[v] = decay<Z>(co[i].v[v], A.v[v]);
                    E.v[v] = decay<Z>(co[i].v[v], E.v[v]) + wx[i].v[v];
                }
            }
        };
        if (!usual) {
            exact(std::true_type());
        } else if constexpr (!kShort) {
            exact(std::false_type());
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<V> f;
                const Vec<V> x = wide<io_t, V>(rows::get(xs, i, oddx));
                sigmoids(wide<io_t, V>(rows::get(gate, i, odd)), co[i], f);
                wx[i] = MIX == OSDN_MIX_SUM ? x : mul(weight<MIX>(co[i], f), x);
                A = mul(A, co[i]);
                E = fma(E, co[i], wx[i]);
            }
        }
        __syncwarp();   // the stage is read
        Vec<V> q = join<V>(j, step & 1, k.n, k.rank, k.warp, !usual, Pair<V>{A, E}, s, [&] { fetch(step, kStages); });
        char *out = reinterpret_cast<char *>(static_cast<io_t *>(p.out) + k.at + k.lane * V);
        const auto run = [&](auto z) {
            constexpr bool Z = decltype(z)::value;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (!Z && kShort) {
                    q = fma(q, co[i], wx[i]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) q.v[v] = decay<Z>(co[i].v[v], q.v[v]) + wx[i].v[v];
                }
                if (k.live && (!Z || i < tokens)) put<io_t, V>(reinterpret_cast<io_t *>(out + (size_t)i * k.pitch), q);
            }
        };
        if (!usual) run(std::true_type()); else run(std::false_type());
        k.t0 += k.stride;
        k.at += far;
    }
    if (p.last && k.live && k.rank == 0 && k.warp == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[(size_t)k.b * p.C + k.c + v] = s.v[v];
}

// Backwards in time: steps, CTAs, warps and tokens from the last to the first.  The states are
// recomputed from the row of h in front of the warp's tokens, so that one row in R of h is read.
template <typename io_t, int V, int MIX, int R, int W>
__global__ void __launch_bounds__(kThreads, 2) backward_kernel(Params p) {
    typedef typename Raw<io_t, V>::type raw_t;
    constexpr bool kShort = sizeof(io_t) == 2;
    extern __shared__ __align__(16) char sm[];
    __shared__ Join<V> j;
    Walk<io_t, V, R, W, 3> k(p, sm, true);
    typedef Rows<io_t, V, R, W> rows;
    const size_t state = (size_t)k.b * p.C + k.c;
    if (k.n > 1) ptx::cluster_arrive();   // every CTA of the cluster has started once all have arrived
    Vec<V> s = fill<V>(0.0f);
    if (p.first && k.live)
#pragma unroll
        for (int v = 0; v < V; ++v) s.v[v] = p.first[state + v];
    const size_t far = (size_t)k.stride * p.C;
    const auto fetch = [&](int step, int ahead) {
        if (step + ahead < p.steps) {
            const size_t from = k.at - ahead * far;
            const int tokens = p.T - k.t0 + ahead * k.stride;
            k.fetch((step + ahead) % kStages, 0, p.gate, from, tokens);
            k.fetch((step + ahead) % kStages, 1, p.x, from, tokens);
            k.fetch((step + ahead) % kStages, 2, p.dh, from, tokens);
        }
        copies_commit();
    };
    // the state before token t, where that is one of this lane's
    const auto before = [&](int t, size_t at) {
        raw_t u = raw_t();
        if (k.live && t > 0 && t < p.T)
            u = *reinterpret_cast<const raw_t *>(static_cast<const io_t *>(p.h) + at - p.C + k.lane * V);
        return u;
    };
    raw_t row = before(k.t0, k.at);
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(0, i);
    if (k.n > 1) ptx::cluster_wait();
    for (int step = 0; step < p.steps; ++step) {
        copies_wait<kStages - 1>();
        __syncwarp();
        const int tokens = p.T - k.t0, odd = k.odd(p.gate), oddx = k.odd(p.x), oddd = k.odd(p.dh);
        const char *gate = k.tile(step % kStages, 0), *xs = k.tile(step % kStages, 1), *ds = k.tile(step % kStages, 2);
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const Vec<V> g = wide<io_t, V>(rows::get(gate, i, odd));
#pragma unroll
            for (int v = 0; v < V; ++v) most = fmaxf(most, fabsf(g.v[v]));
        }
        const bool usual = __all_sync(kFullMask, tokens >= R && (most <= kPlainGate || !k.live));
        Vec<V> h = wide<io_t, V>(row);
        if (k.t0 == 0 && p.h0 && k.live)
#pragma unroll
            for (int v = 0; v < V; ++v) h.v[v] = p.h0[state + v];
        Vec<V> co[R], w[R], slope[R];
        raw_t d[R];
        Vec<V> A = fill<V>(1.0f), E = fill<V>(0.0f);
        const auto exact = [&](auto z) {
            constexpr bool Z = decltype(z)::value;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<V> g = wide<io_t, V>(rows::get(gate, i, odd)), x = wide<io_t, V>(rows::get(xs, i, oddx));
                d[i] = rows::get(ds, i, oddd);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    co[i].v[v] = !Z || i < tokens ? gate_coefficient(g.v[v]) : -0.0f;
                    slopes<MIX, Z>(co[i].v[v], h.v[v], x.v[v], w[i].v[v], slope[i].v[v]);
                    h.v[v] = decay<Z>(co[i].v[v], h.v[v]) + (!Z || i < tokens ? weighted<MIX, Z>(co[i].v[v], x.v[v]) : 0.0f);
                }
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const Vec<V> di = wide<io_t, V>(d[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    A.v[v] = decay<Z>(co[i].v[v], A.v[v]);
                    E.v[v] = decay<Z>(co[i].v[v], di.v[v] + E.v[v]);
                }
            }
        };
        if (!usual) {
            exact(std::true_type());
        } else if constexpr (!kShort) {
            exact(std::false_type());
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<V> f;
                const Vec<V> x = wide<io_t, V>(rows::get(xs, i, oddx));
                sigmoids(wide<io_t, V>(rows::get(gate, i, odd)), co[i], f);
                slopes<MIX>(co[i], f, h, x, w[i], slope[i]);
                h = fma(h, co[i], mul(w[i], x));
                d[i] = rows::get(ds, i, oddd);
            }
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                A = mul(A, co[i]);
                E = mul(add(wide<io_t, V>(d[i]), E), co[i]);
            }
        }
        __syncwarp();
        Vec<V> q = join<V>(j, step & 1, k.n, k.rank, kWarps - 1 - k.warp, !usual, Pair<V>{A, E}, s, [&] {
            fetch(step, kStages);
            row = before(k.t0 - k.stride, k.at - far);
        });
        char *dx = reinterpret_cast<char *>(static_cast<io_t *>(p.out) + k.at + k.lane * V);
        char *dg = reinterpret_cast<char *>(static_cast<io_t *>(p.dgate) + k.at + k.lane * V);
        const auto run = [&](auto z) {
            constexpr bool Z = decltype(z)::value;
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const Vec<V> r = add(wide<io_t, V>(d[i]), q);
                if (k.live && (!Z || i < tokens)) {
                    put<io_t, V>(reinterpret_cast<io_t *>(dx + (size_t)i * k.pitch), MIX == OSDN_MIX_SUM ? r : mul(w[i], r));
                    put<io_t, V>(reinterpret_cast<io_t *>(dg + (size_t)i * k.pitch), mul(slope[i], r));
                }
                if (!Z && kShort) {
                    q = mul(r, co[i]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) q.v[v] = decay<Z>(co[i].v[v], r.v[v]);
                }
            }
        };
        if (!usual) run(std::true_type()); else run(std::false_type());
        k.t0 -= k.stride;
        k.at -= far;
    }
    if (p.last && k.live && k.rank == 0 && k.warp == 0)
#pragma unroll
        for (int v = 0; v < V; ++v) p.last[state + v] = s.v[v];
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

// How a call is cut: clusters of n CTAs a strip of 32 V channels, R tokens a warp.
struct Plan {
    int V, R, W, n, steps, per_seq;
    long long strips;
};
constexpr int rows_a_warp(bool f32, bool backward) { return backward || f32 ? 8 : 16; }
Plan plan(int io, bool backward, int B, int T, int C) {
    Plan p;
    const int e = io == OSDN_F32 ? 4 : 2;
    p.V = C % 2 ? 1 : 2;
    p.W = p.V == 2 && C * (size_t)e % 16 == 0 ? 16 : C * (size_t)e % 4 == 0 ? 4 : 2;
    p.per_seq = (C + 32 * p.V - 1) / (32 * p.V);
    p.strips = (long long)B * p.per_seq;
    p.R = T <= kWarps * 4 ? 4 : rows_a_warp(io == OSDN_F32, backward);
    const int chunks = (T + kWarps * p.R - 1) / (kWarps * p.R);
    // two CTAs an SM, in clusters of up to eight, are about 256
    p.n = 1;
    while (p.n < kMaxCluster && 2 * p.n * p.strips <= 288 && p.n < chunks) p.n *= 2;
    p.steps = (chunks + p.n - 1) / p.n;
    return p;
}

template <bool BACKWARD, typename io_t, int V, int MIX, int R, int W>
cudaError_t launch_as(const Plan &pl, const Params &p, cudaStream_t stream) {
    void (*kernel)(Params);
    if constexpr (BACKWARD) kernel = backward_kernel<io_t, V, MIX, R, W>;
    else kernel = scan_kernel<io_t, V, MIX, R, W>;
    constexpr int smem = kWarps * kStages * (BACKWARD ? 3 : 2) * Rows<io_t, V, R, W>::kBytes;
    static std::atomic<unsigned long long> done{0};
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
template <bool BACKWARD, typename io_t, int MIX, int R>
cudaError_t launch_rows(const Plan &pl, const Params &p, cudaStream_t stream) {
    if (pl.V == 1) return launch_as<BACKWARD, io_t, 1, MIX, R, sizeof(io_t) == 4 ? 4 : 2>(pl, p, stream);
    return pl.W == 16 ? launch_as<BACKWARD, io_t, 2, MIX, R, 16>(pl, p, stream)
                      : launch_as<BACKWARD, io_t, 2, MIX, R, 4>(pl, p, stream);
}

template <bool BACKWARD>
cudaError_t launch(int io, int mix, int B, int T, int C, Params p, cudaStream_t stream) {
    const Plan pl = plan(io, BACKWARD, B, T, C);
    p.T = T; p.C = C;
    p.per_seq = pl.per_seq;
    p.steps = pl.steps;
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        constexpr int M = decltype(m)::value, R = rows_a_warp(sizeof(io_t) == 4, BACKWARD);
        return pl.R == 4 ? launch_rows<BACKWARD, io_t, M, 4>(pl, p, stream)
                         : launch_rows<BACKWARD, io_t, M, R>(pl, p, stream);
    });
}

}  // namespace

cudaError_t scan_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                        void *h, float *hT, cudaStream_t stream) {
    Params p = {};
    p.x = x; p.gate = gate;
    p.first = h0;
    p.out = h;
    p.last = hT;
    return launch<false>(io, mix, B, T, C, p, stream);
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
                            cudaStream_t stream) {
    Params p = {};
    p.x = x; p.gate = gate; p.h = h; p.dh = dh;
    p.h0 = h0;
    p.first = dhT;
    p.out = dx; p.dgate = dgate;
    p.last = dh0;
    return launch<true>(io, mix, B, T, C, p, stream);
}

}  // namespace gs
}  // namespace osdn
