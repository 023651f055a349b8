// gated_scan.cu -- a linear recurrence with a gate per token and channel, its
// single-token step and its gradients (include/osdn.h has the formulas).
//
// One thread a channel walks the tokens.
#include "gated_scan.cuh"

namespace osdn {
namespace gs {

namespace {

constexpr int kThreads = 128;

template <typename io_t, int MIX>
__global__ void __launch_bounds__(kThreads)
scan_kernel(long long n, int T, int C, const io_t *x, const io_t *gate, const float *h0, io_t *h, float *hT) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const long long b = i / C, c = i % C;
    float s = h0 ? h0[i] : 0.0f;
    for (long long t = 0, at = b * T * C + c; t < T; ++t, at += C) {
        const Gate g(to_f32(gate[at]));
        s = g.next<MIX>(s, to_f32(x[at]));
        from_f32(h[at], s);
    }
    if (hT) hT[i] = s;
}

template <typename io_t, int MIX>
__global__ void __launch_bounds__(kThreads)
step_kernel(long long n, const io_t *x, const io_t *gate, float *h, io_t *y) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const Gate g(to_f32(gate[i]));
    const float s = g.next<MIX>(h[i], to_f32(x[i]));
    h[i] = s;
    from_f32(y[i], s);
}

template <typename io_t, int MIX>
__global__ void __launch_bounds__(kThreads)
backward_kernel(long long n, int T, int C, const io_t *x, const io_t *gate, const io_t *h, const float *h0,
                const io_t *dh, const float *dhT, io_t *dx, io_t *dgate, float *dh0) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (i >= n) return;
    const long long b = i / C, c = i % C;
    float q = dhT ? dhT[i] : 0.0f;
    for (long long t = T - 1, at = (b * T + T - 1) * C + c; t >= 0; --t, at -= C) {
        const Gate g(to_f32(gate[at]));
        const float before = t ? to_f32(h[at - C]) : h0 ? h0[i] : 0.0f;
        const float r = to_f32(dh[at]) + q;
        float gx, gg;
        g.gradients<MIX>(r, before, to_f32(x[at]), gx, gg);
        from_f32(dx[at], gx);
        from_f32(dgate[at], gg);
        q = g.decay(r);
    }
    if (dh0) dh0[i] = q;
}

unsigned blocks(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace

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

size_t scan_scratch_bytes(int, int, int, int) { return 0; }
size_t backward_scratch_bytes(int, int, int, int) { return 0; }

cudaError_t scan_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                        void *h, float *hT, void *, int *, cudaStream_t stream) {
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        const long long n = (long long)B * C;
        scan_kernel<io_t, decltype(m)::value><<<blocks(n), kThreads, 0, stream>>>(
            n, T, C, static_cast<const io_t *>(x), static_cast<const io_t *>(gate), h0, static_cast<io_t *>(h), hT);
        return cudaGetLastError();
    });
}

cudaError_t step_launch(int io, int B, int C, int mix, const void *x, const void *gate, float *h, void *y,
                        cudaStream_t stream) {
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        const long long n = (long long)B * C;
        step_kernel<io_t, decltype(m)::value><<<blocks(n), kThreads, 0, stream>>>(
            n, static_cast<const io_t *>(x), static_cast<const io_t *>(gate), h, static_cast<io_t *>(y));
        return cudaGetLastError();
    });
}

cudaError_t backward_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const void *h,
                            const float *h0, const void *dh, const float *dhT, void *dx, void *dgate, float *dh0,
                            void *, int *, cudaStream_t stream) {
    return with_types(io, mix, [&](auto t, auto m) {
        using io_t = decltype(t);
        const long long n = (long long)B * C;
        backward_kernel<io_t, decltype(m)::value><<<blocks(n), kThreads, 0, stream>>>(
            n, T, C, static_cast<const io_t *>(x), static_cast<const io_t *>(gate), static_cast<const io_t *>(h), h0,
            static_cast<const io_t *>(dh), dhT, static_cast<io_t *>(dx), static_cast<io_t *>(dgate), dh0);
        return cudaGetLastError();
    });
}

}  // namespace gs
}  // namespace osdn
