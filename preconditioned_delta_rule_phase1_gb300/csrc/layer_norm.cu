// layer_norm.cu -- layer norm over whole rows, with the addition to the
// residual stream in front of it, and its gradients (include/osdn.h has the
// formulas).
//
// One CTA a row, one thread a column for the sums over rows.
#include "osdn_device.cuh"

namespace osdn {
namespace ln {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v) {
    __shared__ float part[kThreads / 32];
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFullMask, v, m);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += part[i];
    return s;
}

// The mean and 1 / sqrt(var + eps) of the row that get(c) reads.  Sums are of the values less the
// row's first, so that rounding them is relative to the spread.
template <typename F>
__device__ __forceinline__ void row_stats(int C, float eps, const F &get, float &x0, float &m, float &r) {
    x0 = get(0);
    float s = 0.0f;
    for (int c = threadIdx.x; c < C; c += kThreads) s += get(c) - x0;
    m = block_sum(s) / C;
    s = 0.0f;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        const float d = get(c) - x0 - m;
        s = fmaf(d, d, s);
    }
    r = rsqrtf(block_sum(s) / C + eps);
}

template <typename io_t>
__global__ void __launch_bounds__(kThreads)
norm_kernel(int C, const io_t *x, const io_t *residual, const float *weight, const float *bias, float eps,
            io_t *y, io_t *sum) {
    const size_t at = (size_t)blockIdx.x * C;
    const auto get = [&](int c) { return to_f32(x[at + c]) + (residual ? to_f32(residual[at + c]) : 0.0f); };
    float x0, m, r;
    row_stats(C, eps, get, x0, m, r);
    for (int c = threadIdx.x; c < C; c += kThreads) {
        const float v = get(c);
        from_f32(y[at + c], (v - x0 - m) * r * (weight ? weight[c] : 1.0f) + (bias ? bias[c] : 0.0f));
        if (sum) from_f32(sum[at + c], v);
    }
}

template <typename io_t>
__global__ void __launch_bounds__(kThreads)
backward_kernel(int C, const io_t *x, const io_t *dy, const float *weight, const io_t *ds, float eps, io_t *dx,
                float *stats) {
    const size_t at = (size_t)blockIdx.x * C;
    const auto get = [&](int c) { return to_f32(x[at + c]); };
    float x0, m, r;
    row_stats(C, eps, get, x0, m, r);
    float s = 0.0f, sx = 0.0f;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        const float t = to_f32(dy[at + c]) * (weight ? weight[c] : 1.0f);
        s += t;
        sx = fmaf(t, (get(c) - x0 - m) * r, sx);
    }
    const float mu = block_sum(s) / C, mx = block_sum(sx) / C;
    for (int c = threadIdx.x; c < C; c += kThreads) {
        const float t = to_f32(dy[at + c]) * (weight ? weight[c] : 1.0f);
        const float d = r * (t - mu - (get(c) - x0 - m) * r * mx);
        from_f32(dx[at + c], d + (ds ? to_f32(ds[at + c]) : 0.0f));
    }
    if (threadIdx.x == 0) {
        stats[3 * (size_t)blockIdx.x] = x0;
        stats[3 * (size_t)blockIdx.x + 1] = m;
        stats[3 * (size_t)blockIdx.x + 2] = r;
    }
}

template <typename io_t>
__global__ void __launch_bounds__(kThreads)
columns_kernel(long long rows, int C, const io_t *x, const io_t *dy, const float *stats, float *dweight,
               float *dbias) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float w = 0.0f, b = 0.0f;
    for (long long i = 0; i < rows; ++i) {
        const float d = to_f32(dy[i * C + c]);
        const float *s = stats + 3 * i;
        w = fmaf(d, (to_f32(x[i * C + c]) - s[0] - s[1]) * s[2], w);
        b += d;
    }
    if (dweight) dweight[c] = w;
    if (dbias) dbias[c] = b;
}

template <typename io_t>
cudaError_t forward(long long rows, int C, const void *x, const void *residual, const float *weight,
                    const float *bias, float eps, void *y, void *sum, cudaStream_t stream) {
    norm_kernel<io_t><<<(unsigned)rows, kThreads, 0, stream>>>(
        C, static_cast<const io_t *>(x), static_cast<const io_t *>(residual), weight, bias, eps,
        static_cast<io_t *>(y), static_cast<io_t *>(sum));
    return cudaGetLastError();
}

template <typename io_t>
cudaError_t backward(long long rows, int C, const void *x, const void *dy, const float *weight, const void *ds,
                     float eps, void *dx, float *dweight, float *dbias, void *scratch, cudaStream_t stream) {
    if (rows)
        backward_kernel<io_t><<<(unsigned)rows, kThreads, 0, stream>>>(
            C, static_cast<const io_t *>(x), static_cast<const io_t *>(dy), weight, static_cast<const io_t *>(ds),
            eps, static_cast<io_t *>(dx), static_cast<float *>(scratch));
    if (dweight || dbias)
        columns_kernel<io_t><<<(C + kThreads - 1) / kThreads, kThreads, 0, stream>>>(
            rows, C, static_cast<const io_t *>(x), static_cast<const io_t *>(dy),
            static_cast<const float *>(scratch), dweight, dbias);
    return cudaGetLastError();
}

}  // namespace

size_t backward_scratch_bytes(long long rows, int) { return (size_t)rows * 3 * sizeof(float); }

cudaError_t norm_launch(int io, long long rows, int C, const void *x, const void *residual, const float *weight,
                        const float *bias, float eps, void *y, void *sum, cudaStream_t stream) {
    return io == OSDN_F32 ? forward<float>(rows, C, x, residual, weight, bias, eps, y, sum, stream)
                          : forward<__nv_bfloat16>(rows, C, x, residual, weight, bias, eps, y, sum, stream);
}

cudaError_t backward_launch(int io, long long rows, int C, const void *x, const void *dy, const float *weight,
                            const void *ds, float eps, void *dx, float *dweight, float *dbias, void *scratch,
                            cudaStream_t stream) {
    return io == OSDN_F32
               ? backward<float>(rows, C, x, dy, weight, ds, eps, dx, dweight, dbias, scratch, stream)
               : backward<__nv_bfloat16>(rows, C, x, dy, weight, ds, eps, dx, dweight, dbias, scratch, stream);
}

}  // namespace ln
}  // namespace osdn
