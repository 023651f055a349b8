// gated_scan.cu -- a linear recurrence with a gate per token and channel, its
// single-token step and its gradients:
//     h_t = a_t h_{t-1} + w(a_t) x_t,   a_t = sigmoid(gate_t)
//     R_t = dh_t + Q_t,  Q_{t-1} = a_t R_t          (Q_T = dhT, dh0 = Q_0)
//     dx_t = w(a_t) R_t,   dgate_t = R_t (a_t (1 - a_t) h_{t-1} + w'_t x_t)
//
// Both directions are a recurrence s <- a s + e of every channel, and runs of
// it compose: (A, E) after (A', E') is (A A', A E' + E), with A held so that 1 - A
// keeps its digits (gated_scan_walk.cuh).  The tensors are read and written once,
// so HBM is what they cannot do without.  A warp holds R tokens of 32 lanes'
// channels (two a lane) in registers, a CTA kWarps warps one
// behind the other in time.  A strip of channels belongs to a cluster of up to
// eight CTAs, which walks the sequence, each step a run of tokens a CTA:
//   1  every thread turns its tokens into factors and folds them to (A, E);
//   2  the warps' pairs meet in shared memory, and, in a cluster, the CTAs'
//      totals in distributed shared memory;
//   3  every thread folds what lies before it onto the state that entered the
//      step, runs the recurrence over its factors and stores.
// A warp's tokens of the next two steps are on their way into shared memory
// meanwhile, by asynchronous copies of 16 bytes where rows keep 16-byte
// boundaries or are odd numbers of bf16, else of words; a warp reads only what
// it copied itself.  Nothing leaves the cluster, so there is no workspace and
// nothing to wait for but its own barrier.  Every fold is in a fixed order.
//
// Measured (bf16, mean): 43 us at 16x1024x2048, where a CTA walks a strip alone
// (4.7 TB/s, 0.69 of the measured copy bandwidth), 52 us at 2x8192x2048 in
// clusters of four (0.57) and 193 us at 1x65536x2048 in clusters of eight
// (0.62); fp32 51 us at 2x4096x2048.  38 to 45 instructions a token and warp at
// 16 warps an SM (128 registers) take 0.43 to 0.49 of the issue slots; the rest
// is a step's latency, about 2 us in a cluster of eight that has its SMs to
// itself.  Joining through a chain of clusters in global memory took 118 us at
// 2x8192x2048, eight tokens a warp in place of 16 66 us.
#include "gated_scan_walk.cuh"

namespace osdn {
namespace gs {

namespace {

template <typename io_t, int MIX, int R, int W>
__global__ void __launch_bounds__(kThreads, 2) scan_kernel(Params p) {
    typedef typename Raw<io_t>::type raw_t;
    constexpr int V = 2;
    constexpr bool kShort = sizeof(io_t) == 2;
    extern __shared__ __align__(16) char sm[];
    __shared__ Join j;
    Walk<io_t, R, W, 2> k(p, sm, false);
    typedef Rows<io_t, R, W> rows;
    if (k.n > 1) ptx::cluster_arrive();   // every CTA of the cluster has started once all have arrived
    Vec<V> s = k.load_state(p, p.first);
    const size_t far = (size_t)k.stride * p.C;   // elements a step
    const auto fetch = [&](int step, int ahead) {
        if (step + ahead < p.steps) {
            const size_t from = k.at + ahead * far;
            const int tokens = p.T - k.t0 - ahead * k.stride;
            k.fetch((step + ahead) % kStages, 0, p.gate, from, tokens);
            k.fetch((step + ahead) % kStages, 1, p.x, from, tokens);
        }
        ptx::copies_commit();   // (a group a step, so that waiting counts them)
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(0, i);
    if (k.n > 1) ptx::cluster_wait();
    for (int step = 0; step < p.steps; ++step) {
        ptx::copies_wait<kStages - 1>();
        __syncwarp();
        const int tokens = p.T - k.t0, in = k.in(p.gate), inx = k.in(p.x);
        const char *gate = k.tile(step % kStages, 0), *xs = k.tile(step % kStages, 1);
        raw_t rg[R];
#pragma unroll
        for (int i = 0; i < R; ++i) rg[i] = rows::get(gate, i, in, k.pitch);
        int kind = kind_of<R>(
            [&](int i) { return wide(rg[i]); }, [&](int i) { return calm(wide(rows::get(xs, i, inx, k.pitch))); }, tokens, k.live);
        Vec<V> co[R], wx[R];
        Vec<V> A = fill<V>(1.0f), D = fill<V>(0.0f), E = D;   // (D: 1 - A)
        const auto exact = [&](auto x_) {
            constexpr int X = decltype(x_)::value;
            if (X != kPlain) asm volatile("" ::: "memory");   // (the gates are read again, not kept)
            A = fill<V>(1.0f), D = E = fill<V>(0.0f);
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const Vec<V> g = wide(X == kPlain ? rg[i] : rows::get(gate, i, in, k.pitch));
                const Vec<V> x = wide(rows::get(xs, i, inx, k.pitch));
                const bool there = X == kPlain || i < tokens;   // tokens past the end leave everything as it is
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    co[i].v[v] = there ? gate_coefficient<X>(g.v[v]) : X == kAny ? kPasses : -0.0f;
                    wx[i].v[v] = there ? weighted<MIX, X>(co[i].v[v], x.v[v]) : 0.0f;
                    D.v[v] = decay_rest<X>(co[i].v[v], A.v[v], D.v[v]);
                    A.v[v] = decay<X>(co[i].v[v], A.v[v]);
                    E.v[v] = decay<X>(co[i].v[v], E.v[v]) + wx[i].v[v];
                }
            }
        };
        if (!kShort && kind == kPlain) {
            exact(Int<kPlain>());
            if (!__all_sync(kFullMask, finite(E))) kind = kAny;
        }
        if (__builtin_expect(kind == kAny, 0)) {
            exact(Int<kAny>());
        } else if (__builtin_expect(kind == kEnds, 0)) {
            exact(Int<kEnds>());
        } else if (kShort) {
#pragma unroll
            for (int i = 0; i < R; ++i) {
                Vec<V> f;
                const Vec<V> x = wide(rows::get(xs, i, inx, k.pitch)), e = exponentials(wide(rg[i]));
                sigmoids(e, co[i], f);
                wx[i] = MIX == OSDN_MIX_SUM ? x : mul(weight<MIX>(co[i], f), x);
                D = fma(D, e, add(D, e));   // the product of the 1 + e, less 1: 1 / A - 1
                E = fma(E, co[i], wx[i]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A.v[v] = rcp_fast(1.0f + D.v[v]);
                D.v[v] = D.v[v] < 1.0f ? D.v[v] * A.v[v] : 1.0f;   // (own_run then takes A)
            }
        }
        __syncwarp();   // the stage is read
        Vec<V> q = join(j, step & 1, k.n, k.rank, k.warp, own_run(A, D, E), s, [&] { fetch(step, kStages); });
        char *out = reinterpret_cast<char *>(static_cast<io_t *>(p.out) + k.at + k.lane * V);
        unsigned pitch = k.pitch;
        asm volatile("" : "+r"(pitch));
        const Vec<V> before = q;
        const auto run = [&](auto x_) {
            constexpr int X = decltype(x_)::value;
            if (!kShort) q = before;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                if (kShort && X == kPlain) {
                    q = fma(q, co[i], wx[i]);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) q.v[v] = decay<X>(co[i].v[v], q.v[v]) + wx[i].v[v];
                }
                if (k.live && (X == kPlain || i < tokens)) put<rows::kPaired>(reinterpret_cast<io_t *>(out + (size_t)i * pitch), q, k.second);
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
        k.t0 += k.stride;
        k.at += far;
    }
    if (k.rank == 0 && k.warp == kWarps - 1) k.store_state(p, p.last, s);   // (the last in turn)
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
        const float c = gate_coefficient<kAny>(gv[e]);
        hv[e] = decay<kAny>(c, hv[e]) + weighted<MIX, kAny>(c, xv[e]);
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

}  // namespace

cudaError_t scan_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                        void *h, float *hT, cudaStream_t stream) {
    Params p = {};
    p.T = T; p.C = C;
    p.x = x; p.gate = gate;
    p.first = h0;
    p.out = h;
    p.last = hT;
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        constexpr int M = decltype(m)::value, most = sizeof(io_t) == 4 ? 8 : 16;   // registers
        const Plan pl = plan(io, most, B, T, C);
        p.per_seq = pl.per_seq;
        p.steps = pl.steps;
        return with_rows<io_t, most, most>(pl, [&](auto r, auto w) {
            constexpr int R = decltype(r)::value, W = decltype(w)::value;
            static std::atomic<unsigned long long> done{0};
            return launch_as<io_t, R, W, 2>(scan_kernel<io_t, M, R, W>, done, pl, p, stream);
        });
    });
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

}  // namespace gs
}  // namespace osdn
