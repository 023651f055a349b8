// gated_scan_backward.cu -- the gradients of the gated recurrence; gated_scan.cu
// has the formulas and the design.
//
// Measured (bf16, 2x8192x2048, five tensors of 67 MB): sum 70, unit 89, mean 90
// us (0.71, 0.56 and 0.55 of the measured copy bandwidth); fp32 67 us at
// 2x4096x2048, mean.  Neither issue (0.46 of the slots at 16 warps an SM) nor HBM
// (0.45) is full: a step's latency is what counts, its barriers first (2.2 warps
// wait there for each one that issues).  Only e^-g and the slope of the gate stay in
// registers between the two passes over a thread's tokens; with a and w kept
// too there is room for eight tokens in place of 16 (sum 93 us).
#include "gated_scan_walk.cuh"

namespace osdn {
namespace gs {

namespace {

// Backwards in time: steps, CTAs, warps and tokens from the last to the first.  The states are
// recomputed from the row of h in front of the warp's tokens, so that one row in R of h is read.  A
// thread's own (A, E) is gathered on the same way forwards: Q before its tokens is A Q + E with A the
// product of their a and E the sum of their dh, each times the product of the a up to it.
template <typename io_t, int MIX, int R, int W>
__global__ void __launch_bounds__(kThreads, 2) backward_kernel(Params p) {
    typedef typename Raw<io_t>::type raw_t;
    constexpr int V = 2;
    constexpr bool kShort = sizeof(io_t) == 2;
    extern __shared__ __align__(16) char sm[];
    __shared__ Join j;
    Walk<io_t, R, W, 3> k(p, sm, true);
    typedef Rows<io_t, R, W> rows;
    if (k.n > 1) ptx::cluster_arrive();   // every CTA of the cluster has started once all have arrived
    Vec<V> s = k.load_state(p, p.first);
    const size_t far = (size_t)k.stride * p.C;
    const auto fetch = [&](int step, int ahead) {
        if (step + ahead < p.steps) {
            const size_t from = k.at - ahead * far;
            const int tokens = p.T - k.t0 + ahead * k.stride;
            k.fetch((step + ahead) % kStages, 0, p.gate, from, tokens);
            k.fetch((step + ahead) % kStages, 1, p.x, from, tokens);
            k.fetch((step + ahead) % kStages, 2, p.dh, from, tokens);
        }
        ptx::copies_commit();
    };
    // the state before token t, where that is one of this lane's
    const auto before = [&](int t, size_t at) {
        raw_t u = raw_t();
        if (k.live && t > 0 && t < p.T) {
            const io_t *q = static_cast<const io_t *>(p.h) + at - p.C + k.lane * 2;
            if constexpr (rows::kPaired) {
                u = *reinterpret_cast<const raw_t *>(q);
            } else if constexpr (sizeof(io_t) == 4) {
                u.x = reinterpret_cast<const unsigned *>(q)[0];
                if (k.second) u.y = reinterpret_cast<const unsigned *>(q)[1];
            } else {
                u = reinterpret_cast<const unsigned short *>(q)[0];
                if (k.second) u |= (unsigned)reinterpret_cast<const unsigned short *>(q)[1] << 16;
            }
        }
        return u;
    };
    raw_t row = before(k.t0, k.at);
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(0, i);
    if (k.n > 1) ptx::cluster_wait();
    for (int step = 0; step < p.steps; ++step) {
        ptx::copies_wait<kStages - 1>();
        __syncwarp();
        const int tokens = p.T - k.t0, in = k.in(p.gate), inx = k.in(p.x), ind = k.in(p.dh);
        const char *gate = k.tile(step % kStages, 0), *xs = k.tile(step % kStages, 1), *ds = k.tile(step % kStages, 2);
        raw_t rg[R];
#pragma unroll
        for (int i = 0; i < R; ++i) rg[i] = rows::get(gate, i, in, k.pitch);
        const auto state_before = [&] { return k.t0 == 0 ? k.load_state(p, p.h0) : wide(row); };
        Vec<V> h = state_before();
        const bool calm_state = calm(h);
        int kind = kind_of<R>(
            [&](int i) { return wide(rg[i]); },
            [&](int i) { return calm_state && calm(wide(rows::get(xs, i, inx, k.pitch))) && calm(wide(rows::get(ds, i, ind, k.pitch))); },
            tokens, k.live);
        Vec<V> co[R], slope[R];   // (co: c, or e^-g in the short form)
        raw_t d[R];
        Vec<V> A = fill<V>(1.0f), D = fill<V>(0.0f), E = D;   // (D: 1 - A)
        const auto exact = [&](auto x_) {
            constexpr int X = decltype(x_)::value;
            if (X != kPlain) asm volatile("" ::: "memory");   // (the gates are read again, not kept)
            h = state_before(), A = fill<V>(1.0f), D = E = fill<V>(0.0f);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<V> g = wide(X == kPlain ? rg[i] : rows::get(gate, i, in, k.pitch));
                const Vec<V> x = wide(rows::get(xs, i, inx, k.pitch));
                const bool there = X == kPlain || i < tokens;
                d[i] = rows::get(ds, i, ind, k.pitch);
                const Vec<V> di = wide(d[i]);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    co[i].v[v] = there ? gate_coefficient<X>(g.v[v]) : X == kAny ? kPasses : -0.0f;
                    slope[i].v[v] = slope_of<MIX, X>(co[i].v[v], h.v[v], x.v[v]);
                    h.v[v] = decay<X>(co[i].v[v], h.v[v]) + (there ? weighted<MIX, X>(co[i].v[v], x.v[v]) : 0.0f);
                    D.v[v] = decay_rest<X>(co[i].v[v], A.v[v], D.v[v]);
                    if (X != kAny || A.v[v] != 0.0f) A.v[v] = decay<X>(co[i].v[v], A.v[v]);
                    E.v[v] = X == kAny && A.v[v] == 0.0f ? E.v[v] : fmaf(A.v[v], di.v[v], E.v[v]);
                }
            }
        };
        if (!kShort && kind == kPlain) {
            exact(Int<kPlain>());
            if (!__all_sync(kFullMask, finite(h) && finite(E))) kind = kAny;
        }
        if (__builtin_expect(kind == kAny, 0)) {
            exact(Int<kAny>());
        } else if (__builtin_expect(kind == kEnds, 0)) {
            exact(Int<kEnds>());
        } else if (kShort) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<V> a, f;
                const Vec<V> x = wide(rows::get(xs, i, inx, k.pitch));
                co[i] = exponentials(wide(rg[i]));
                sigmoids(co[i], a, f);
                slope[i] = slope_and_next<MIX>(a, f, x, h);
                d[i] = rows::get(ds, i, ind, k.pitch);
                D = fma(f, A, D);
                A = mul(A, a);
                E = fma(A, wide(d[i]), E);
            }
        }
        __syncwarp();
        Vec<V> q = join(j, step & 1, k.n, k.rank, kWarps - 1 - k.warp, own_run(A, D, E), s, [&] {
            fetch(step, kStages);
            row = before(k.t0 - k.stride, k.at - far);
        });
        char *dx = reinterpret_cast<char *>(static_cast<io_t *>(p.out) + k.at + k.lane * V);
        char *dg = reinterpret_cast<char *>(static_cast<io_t *>(p.dgate) + k.at + k.lane * V);
        unsigned pitch = k.pitch;
        asm volatile("" : "+r"(pitch));
        const Vec<V> behind = q;
        const auto run = [&](auto x_) {
            constexpr int X = decltype(x_)::value;
            if (!kShort) q = behind;
#pragma unroll
            for (int i = R - 1; i >= 0; --i) {
                const Vec<V> r = add(wide(d[i]), q);
                Vec<V> w;
                // a and w again, rather than kept from above: registers for more tokens are worth more
#pragma unroll
                for (int v = 0; v < V; ++v) asm volatile("" : "+f"(co[i].v[v]));
                if (kShort && X == kPlain) {
                    Vec<V> a, f;
                    sigmoids(co[i], a, f);
                    w = weight<MIX>(a, f);
                    q = mul(r, a);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        w.v[v] = weight<MIX, X>(co[i].v[v]);
                        q.v[v] = decay<X>(co[i].v[v], r.v[v]);
                    }
                }
                Vec<V> gx = MIX == OSDN_MIX_SUM ? r : mul(w, r), gg = mul(slope[i], r);
                if constexpr (X == kAny) {   // factors that are exactly zero hide r
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (w.v[v] == 0.0f) gx.v[v] = 0.0f;
                        if (no_slope<MIX>(co[i].v[v])) gg.v[v] = 0.0f;
                    }
                }
                if (k.live && (X == kPlain || i < tokens)) {
                    put<rows::kPaired>(reinterpret_cast<io_t *>(dx + (size_t)i * pitch), gx, k.second);
                    put<rows::kPaired>(reinterpret_cast<io_t *>(dg + (size_t)i * pitch), gg, k.second);
                }
            }
        };
        if (__builtin_expect(kind == kPlain, 1)) {
            run(Int<kPlain>());
            if (!kShort && !finite(q)) run(Int<kAny>());
        } else if (kind == kEnds && calm(q)) {
            run(Int<kEnds>());
        } else {
            run(Int<kAny>());
        }
        k.t0 -= k.stride;
        k.at -= far;
    }
    if (k.rank == 0 && k.warp == 0) k.store_state(p, p.last, s);   // (the last in turn)
}

}  // namespace

cudaError_t backward_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const void *h,
                            const float *h0, const void *dh, const float *dhT, void *dx, void *dgate, float *dh0,
                            cudaStream_t stream) {
    Params p = {};
    p.T = T; p.C = C;
    p.x = x; p.gate = gate; p.h = h; p.dh = dh;
    p.h0 = h0;
    p.first = dhT;
    p.out = dx; p.dgate = dgate;
    p.last = dh0;
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        // 16 tokens of OSDN_MIX_MEAN do not find room in 128 registers (2x8192x2048: 91 us either way,
        // 16x1024x2048: 87 us, with 8 tokens 79 us), nor do those of rows of odd bf16 (2x8192x2047, sum:
        // 160 us, with 8 tokens 128 us); the others do (2x8192x2048, unit and sum: 84 and 68 us, with 8
        // tokens 99 and 93 us)
        constexpr int M = decltype(m)::value, most = sizeof(io_t) == 4 || M == OSDN_MIX_MEAN ? 8 : 16;
        const Plan pl = plan(io, C % 2 ? 8 : most, B, T, C);
        p.per_seq = pl.per_seq;
        p.steps = pl.steps;
        return with_rows<io_t, most, 8>(pl, [&](auto r, auto w) {
            constexpr int R = decltype(r)::value, W = decltype(w)::value;
            static std::atomic<unsigned long long> done{0};
            return launch_as<io_t, R, W, 3>(backward_kernel<io_t, M, R, W>, done, pl, p, stream);
        });
    });
}

}  // namespace gs
}  // namespace osdn
