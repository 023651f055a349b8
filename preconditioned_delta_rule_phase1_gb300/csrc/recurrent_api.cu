// recurrent_api.cu -- the extern "C" boundary of the gated recurrent layer
// (include/osdn.h): the gated recurrence over prompts, its single-token step
// and its gradients, and the layer norm in front of it.
#include <cmath>

#include "api_checks.cuh"

namespace osdn {
namespace gs {
cudaError_t scan_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                        void *h, float *hT, cudaStream_t stream);
cudaError_t step_launch(int io, int B, int C, int mix, const void *x, const void *gate, float *h, void *y,
                        cudaStream_t stream);
cudaError_t backward_launch(int io, int B, int T, int C, int mix, const void *x, const void *gate, const void *h,
                            const float *h0, const void *dh, const float *dhT, void *dx, void *dgate, float *dh0,
                            cudaStream_t stream);
}  // namespace gs
namespace ln {
size_t backward_scratch_bytes(long long rows, int C);
cudaError_t norm_launch(int io, long long rows, int C, const void *x, const void *residual, const float *weight,
                        const float *bias, float eps, void *y, void *sum, cudaStream_t stream);
cudaError_t backward_launch(int io, long long rows, int C, const void *x, const void *dy, const float *weight,
                            const void *ds, float eps, void *dx, float *dweight, float *dbias, void *scratch,
                            cudaStream_t stream);
}  // namespace ln
cudaError_t fill_state_launch(size_t n, const float *src, float fill, float *dst, cudaStream_t stream);
}  // namespace osdn

namespace {

using namespace osdn::api;

constexpr int kMaxWidth = 16384;   // layer norm: a row stays in one CTA's registers
constexpr long long kMaxRows = 0x7fffffff;
constexpr int kMaxChannels = 1 << 24;   // the recurrence: a row's bytes, and 16 rows' of bf16, are counted in 32 bits

bool mix_ok(int mix) { return mix >= OSDN_MIX_SUM && mix <= OSDN_MIX_UNIT; }

// A CTA, or a cluster, takes 64 channels of a sequence, and CTAs are numbered in 31 bits; the rest is
// addressed in 64 bits (2^39 elements are a terabyte in bf16, more than any device holds).
bool scan_dims_ok(int B, int T, int C) {
    if (B < 0 || T < 0 || C < 0 || T > kMaxTokens || C > kMaxChannels) return false;
    const double strips = (double)B * ((C + 63) / 64);
    return strips <= 2147483647.0 && (double)B * C * T <= 549755813888.0;
}
bool norm_dims_ok(long long rows, int C) { return rows >= 0 && rows <= kMaxRows && C >= 1 && C <= kMaxWidth; }
bool eps_ok(float eps) { return eps > 0.0f && !std::isinf(eps); }

}  // namespace

extern "C" {

int osdn_gated_scan(int io, int B, int T, int C, int mix, const void *x, const void *gate, const float *h0,
                    void *h, float *hT, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!scan_dims_ok(B, T, C)) return OSDN_ERR_DIMS;
    if (!mix_ok(mix)) return OSDN_ERR_ARG;
    const size_t states = (size_t)B * C, n = states * T * io_bytes(io);
    if (states == 0) return OSDN_OK;
    if (n && (!x || !gate || !h)) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {gate, n, false}, {h0, states * 4, false}, {h, n, true},
                        {hT, states * 4, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return done(osdn::fill_state_launch(hT ? states : 0, h0, 0.0f, hT, st));
    return done(osdn::gs::scan_launch(io, B, T, C, mix, x, gate, h0, h, hT, st));
}

int osdn_gated_scan_step(int io, int B, int C, int mix, const void *x, const void *gate, float *h, void *y,
                         void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!scan_dims_ok(B, 1, C)) return OSDN_ERR_DIMS;
    if (!mix_ok(mix)) return OSDN_ERR_ARG;
    const size_t states = (size_t)B * C, n = states * io_bytes(io);
    if (states == 0) return OSDN_OK;
    if (!x || !gate || !h || !y) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {gate, n, false}, {h, states * 4, true}, {y, n, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::gs::step_launch(io, B, C, mix, x, gate, h, y, (cudaStream_t)stream));
}

int osdn_gated_scan_backward(int io, int B, int T, int C, int mix, const void *x, const void *gate, const void *h,
                             const float *h0, const void *d_h, const float *d_hT, void *dx, void *dgate,
                             float *dh0, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!scan_dims_ok(B, T, C)) return OSDN_ERR_DIMS;
    if (!mix_ok(mix)) return OSDN_ERR_ARG;
    const size_t states = (size_t)B * C, n = states * T * io_bytes(io);
    if (states == 0) return OSDN_OK;
    if (n && (!x || !gate || !h || !d_h || !dx || !dgate)) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {gate, n, false}, {h, n, false}, {h0, states * 4, false}, {d_h, n, false},
                        {d_hT, states * 4, false}, {dx, n, true}, {dgate, n, true}, {dh0, states * 4, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return done(osdn::fill_state_launch(dh0 ? states : 0, d_hT, 0.0f, dh0, st));
    return done(osdn::gs::backward_launch(io, B, T, C, mix, x, gate, h, h0, d_h, d_hT, dx, dgate, dh0, st));
}

int osdn_layer_norm(int io, long long rows, int C, const void *x, const void *residual, const float *weight,
                    const float *bias, float eps, void *y, void *sum, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!norm_dims_ok(rows, C)) return OSDN_ERR_DIMS;
    if (!eps_ok(eps)) return OSDN_ERR_ARG;
    const size_t n = (size_t)rows * C * io_bytes(io), w = (size_t)C * 4;
    if (n == 0) return OSDN_OK;
    if (!x || !y || !residual != !sum) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {residual, n, false}, {weight, w, false}, {bias, w, false}, {y, n, true},
                        {sum, n, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::ln::norm_launch(io, rows, C, x, residual, weight, bias, eps, y, sum, (cudaStream_t)stream));
}

size_t osdn_layer_norm_backward_workspace_bytes(long long rows, int C) {
    if (!norm_dims_ok(rows, C)) return kStatusBytes;
    return kStatusBytes + osdn::ln::backward_scratch_bytes(rows, C);
}

int osdn_layer_norm_backward(int io, long long rows, int C, const void *x, const void *dy, const float *weight,
                             const void *d_sum, float eps, void *dx, float *dweight, float *dbias,
                             void *workspace, size_t workspace_bytes, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!norm_dims_ok(rows, C)) return OSDN_ERR_DIMS;
    if (!eps_ok(eps)) return OSDN_ERR_ARG;
    if (!workspace || workspace_bytes < osdn_layer_norm_backward_workspace_bytes(rows, C))
        return OSDN_ERR_WORKSPACE;
    const size_t n = (size_t)rows * C * io_bytes(io), w = (size_t)C * 4;
    if (n && (!x || !dy || !dx)) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {dy, n, false}, {weight, w, false}, {d_sum, n, false}, {dx, n, true},
                        {dweight, w, true}, {dbias, w, true}, {workspace, workspace_bytes, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::ln::backward_launch(io, rows, C, x, dy, weight, d_sum, eps, dx, dweight, dbias,
                                          static_cast<char *>(workspace) + kStatusBytes, (cudaStream_t)stream));
}

}  // extern "C"
