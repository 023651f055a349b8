// layer_api.cu -- the extern "C" boundary of the decayed linear-attention
// layer (include/osdn.h): attention over prompts, its single-token step and
// its gradients, the group norm behind it, and gradient clipping.
#include <algorithm>
#include <cmath>
#include <stdint.h>

#include "api_checks.cuh"
#include "decay_attn.cuh"

namespace osdn {
namespace da {
cudaError_t decay_step_launch(int io, int BH, int H, int K, int V, const void *q, const void *k,
                              const void *v, const float *decay, float *S, void *o, int *status,
                              cudaStream_t stream);
}
cudaError_t fill_state_launch(size_t n, const float *src, float fill, float *dst,
                              cudaStream_t stream);
size_t group_norm_backward_scratch_bytes(int B, int G, int T, int D);
cudaError_t group_norm_launch(int io, int B, int G, int T, int D, int heads_first, const void *x,
                              const float *weight, const float *bias, const void *gate, int act,
                              float eps, void *y, cudaStream_t stream);
cudaError_t group_norm_backward_launch(int io, int B, int G, int T, int D, int heads_first,
                                       const void *x, const void *dy, const float *weight,
                                       const float *bias, const void *gate, int act, float eps,
                                       void *dx, void *dgate, float *dweight, float *dbias,
                                       void *scratch, cudaStream_t stream);
size_t clip_scratch_bytes(int n);
cudaError_t clip_launch(int n, const void *const *g, void *const *o, const long long *size,
                        const int *io, float max_norm, float *norm, void *scratch,
                        cudaStream_t stream);
}  // namespace osdn

namespace {

using namespace osdn::api;

constexpr size_t kMaxSeqs = size_t(1) << 24;

bool width_ok(int x) { return x == 64 || x == 128; }
bool dims_ok(int B, int H, int T) {
    return B >= 0 && H >= 0 && T >= 0 && T <= kMaxTokens && (size_t)B * (size_t)H <= kMaxSeqs;
}

// Units of the attention's time axis over all sequences, numbered in 31 bits (2^31 of the smallest
// ones are 8 TB of K).
size_t units(size_t BH, int T) { return BH * (((size_t)T + 15) / 16); }

// An address range, and whether the call writes it; in a sorted list `any`
// and `written` are the furthest ends up to there of all and of written ones.
struct Span {
    uintptr_t lo, any, written;
};
// True if, of the spans at(0) .. at(n - 1) (empty ones: lo == any; read ones:
// written == 0), a written one overlaps another.  The library allocates no
// host memory, so they are sorted kSpans at a time on the stack, and the later
// ones looked up in each such list.
constexpr long long kSpans = 1024;
template <typename At>
bool overlap(long long n, const At &at) {
    Span s[kSpans];
    for (long long from = 0; from < n; from += kSpans) {
        const long long to = std::min(n, from + kSpans);
        int m = 0;
        for (long long i = from; i < to; ++i) {
            s[m] = at(i);
            m += s[m].lo != s[m].any;
        }
        std::sort(s, s + m, [](const Span &a, const Span &b) { return a.lo < b.lo; });
        for (int i = 1; i < m; ++i) {
            if (s[i].lo < (s[i].written ? s[i - 1].any : s[i - 1].written)) return true;
            s[i].any = std::max(s[i].any, s[i - 1].any);
            s[i].written = std::max(s[i].written, s[i - 1].written);
        }
        for (long long i = to; i < n; ++i) {
            const Span x = at(i);
            const int before = (int)(std::lower_bound(s, s + m, x.any, [](const Span &a, uintptr_t end) { return a.lo < end; }) - s);
            if (x.lo != x.any && before && x.lo < (x.written ? s[before - 1].any : s[before - 1].written)) return true;
        }
    }
    return false;
}

osdn::da::Pass make_pass(int BH, int H, int T, int K, int V, const void *q, const void *k,
                         const void *v, const float *decay, osdn::da::State S0, void *o,
                         float *ST, int rev) {
    osdn::da::Pass p;
    p.BH = BH; p.H = H; p.T = T; p.K = K; p.V = V;
    p.rev = rev;
    p.q = q; p.k = k; p.v = v;
    p.decay = decay;
    p.S0 = S0;
    p.ST = ST;
    p.o = o;
    return p;
}
osdn::da::State state(const float *p, int transposed = 0) {
    osdn::da::State s;
    s.p = p;
    s.transposed = transposed;
    return s;
}

size_t attend_bytes(int io, int BH, int T, int K, int V) {
    using namespace osdn::da;
    return split_bytes(io == OSDN_F32 ? simt_split(BH, T, K, V) : tc_split(BH, T, K, V), BH, K, V);
}
cudaError_t attend(int io, const osdn::da::Pass &p, void *scratch, int *status, cudaStream_t stream) {
    return io == OSDN_F32 ? osdn::da::attend_simt(p, scratch, status, stream)
                          : osdn::da::attend_tc(p, scratch, status, stream);
}

}  // namespace

extern "C" {

size_t osdn_decay_attn_workspace_bytes(int io, int B, int H, int T, int K, int V) {
    if (!io_ok(io) || !dims_ok(B, H, T) || !width_ok(K) || !width_ok(V) || T == 0 || B * H == 0 ||
        units((size_t)B * H, T) > 0x7fffffff)
        return kStatusBytes;
    return kStatusBytes + attend_bytes(io, B * H, T, K, V);
}

int osdn_decay_attn(int io, int B, int H, int T, int K, int V, const void *q, const void *k,
                    const void *v, const float *decay, const float *S0, void *o, float *ST,
                    void *workspace, size_t workspace_bytes, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!dims_ok(B, H, T) || !width_ok(K) || !width_ok(V)) return OSDN_ERR_DIMS;
    if (!workspace || workspace_bytes < osdn_decay_attn_workspace_bytes(io, B, H, T, K, V))
        return OSDN_ERR_WORKSPACE;
    const size_t BH = (size_t)B * H, e = io_bytes(io);
    if (BH == 0) return OSDN_OK;
    if (T > 0 && (!q || !k || !v || !decay || !o)) return OSDN_ERR_NULL;
    if (units(BH, T) > 0x7fffffff) return OSDN_ERR_DIMS;
    const size_t kb = BH * T * K * e, vb = BH * T * V * e, sb = BH * V * K * 4;
    const Buf bufs[] = {{q, kb, false}, {k, kb, false}, {v, vb, false}, {decay, (size_t)H * 4, false},
                        {S0, sb, false}, {o, vb, true}, {ST, sb, true}, {workspace, workspace_bytes, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return done(osdn::fill_state_launch(ST ? sb / 4 : 0, S0, 0.0f, ST, st));
    const auto p = make_pass((int)BH, H, T, K, V, q, k, v, decay, state(S0), o, ST, 0);
    return done(attend(io, p, static_cast<char *>(workspace) + kStatusBytes,
                       static_cast<int *>(workspace), st));
}

int osdn_decay_attn_step(int io, int B, int H, int K, int V, const void *q, const void *k,
                         const void *v, const float *decay, float *S, void *o, void *workspace,
                         size_t workspace_bytes, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!dims_ok(B, H, 0) || !width_ok(K) || !width_ok(V)) return OSDN_ERR_DIMS;
    if (!workspace || workspace_bytes < kStatusBytes) return OSDN_ERR_WORKSPACE;
    const size_t BH = (size_t)B * H, e = io_bytes(io);
    if (BH == 0) return OSDN_OK;
    if (!q || !k || !v || !decay || !S || !o) return OSDN_ERR_NULL;
    const Buf bufs[] = {{q, BH * K * e, false}, {k, BH * K * e, false}, {v, BH * V * e, false},
                        {decay, (size_t)H * 4, false}, {S, BH * V * K * 4, true}, {o, BH * V * e, true},
                        {workspace, workspace_bytes, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::da::decay_step_launch(io, (int)BH, H, K, V, q, k, v, decay, S, o,
                                            static_cast<int *>(workspace), (cudaStream_t)stream));
}

size_t osdn_decay_attn_backward_workspace_bytes(int io, int B, int H, int T, int K, int V) {
    if (!io_ok(io) || !dims_ok(B, H, T) || !width_ok(K) || !width_ok(V) || T == 0 || B * H == 0 ||
        units((size_t)B * H, T) > 0x7fffffff)
        return kStatusBytes;
    const size_t a = attend_bytes(io, B * H, T, K, V), b = attend_bytes(io, B * H, T, V, K);
    return kStatusBytes + (a > b ? a : b);
}

int osdn_decay_attn_backward(int io, int B, int H, int T, int K, int V, const void *q,
                             const void *k, const void *v, const float *decay, const float *S0,
                             const void *d_o, const float *d_ST, void *dq, void *dk, void *dv,
                             float *dS0, void *workspace, size_t workspace_bytes, void *stream) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!dims_ok(B, H, T) || !width_ok(K) || !width_ok(V)) return OSDN_ERR_DIMS;
    if (!workspace || workspace_bytes < osdn_decay_attn_backward_workspace_bytes(io, B, H, T, K, V))
        return OSDN_ERR_WORKSPACE;
    const size_t BH = (size_t)B * H, e = io_bytes(io);
    if (BH == 0) return OSDN_OK;
    if (T > 0 && (!q || !k || !v || !decay || !d_o || !dq || !dk || !dv)) return OSDN_ERR_NULL;
    if (units(BH, T) > 0x7fffffff) return OSDN_ERR_DIMS;
    const size_t kb = BH * T * K * e, vb = BH * T * V * e, sb = BH * V * K * 4;
    const Buf bufs[] = {{q, kb, false}, {k, kb, false}, {v, vb, false}, {decay, (size_t)H * 4, false},
                        {S0, sb, false}, {d_o, vb, false}, {d_ST, sb, false}, {dq, kb, true},
                        {dk, kb, true}, {dv, vb, true}, {dS0, sb, true}, {workspace, workspace_bytes, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) return done(osdn::fill_state_launch(dS0 ? sb / 4 : 0, d_ST, 0.0f, dS0, st));
    void *scratch = static_cast<char *>(workspace) + kStatusBytes;
    int *status = static_cast<int *>(workspace);
    cudaError_t r = attend(io, make_pass((int)BH, H, T, V, K, d_o, v, k, decay, state(S0, 1), dq, nullptr, 0),
                           scratch, status, st);
    if (r == cudaSuccess)
        r = attend(io, make_pass((int)BH, H, T, K, V, k, q, d_o, decay, state(d_ST), dv, dS0, 1),
                   scratch, status, st);
    if (r == cudaSuccess) {
        auto p = make_pass((int)BH, H, T, V, K, v, d_o, q, decay, state(d_ST, 1), dk, nullptr, 1);
        p.given = 1;   // dv's states, transposed
        r = attend(io, p, scratch, status, st);
    }
    return done(r);
}

}  // extern "C"

namespace {

// The checks that both directions of the group norm share.
int norm_args(int io, int B, int G, int T, int D, int act, float eps) {
    if (!io_ok(io)) return OSDN_ERR_DTYPE;
    if (!dims_ok(B, G, T) || G == 0 || D < 8 || D > 512 || D % 8) return OSDN_ERR_DIMS;
    if (act < OSDN_ACT_NONE || act > OSDN_ACT_SIGMOID || !(eps > 0.0f) || std::isinf(eps))
        return OSDN_ERR_ARG;
    // a launch numbers its CTAs (at least eight groups each) in 31 bits
    if ((double)B * G * T >= 8.0 * 2147483647.0) return OSDN_ERR_DIMS;
    return OSDN_OK;
}

}  // namespace

extern "C" {

int osdn_group_norm(int io, int B, int G, int T, int D, int heads_first, const void *x,
                    const float *weight, const float *bias, const void *gate, int act, float eps,
                    void *y, void *stream) {
    if (int c = norm_args(io, B, G, T, D, act, eps)) return c;
    const size_t n = (size_t)B * G * T * D * io_bytes(io), C = (size_t)G * D * 4;
    if (n == 0) return OSDN_OK;
    if (!x || !y) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {weight, C, false}, {bias, C, false}, {gate, n, false}, {y, n, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::group_norm_launch(io, B, G, T, D, heads_first, x, weight, bias, gate, act, eps,
                                        y, (cudaStream_t)stream));
}

size_t osdn_group_norm_backward_workspace_bytes(int B, int G, int T, int D) {
    if (!dims_ok(B, G, T) || G == 0 || D < 8 || D > 512 || D % 8) return kStatusBytes;
    return kStatusBytes + osdn::group_norm_backward_scratch_bytes(B, G, T, D);
}

int osdn_group_norm_backward(int io, int B, int G, int T, int D, int heads_first, const void *x,
                             const void *dy, const float *weight, const float *bias,
                             const void *gate, int act, float eps, void *dx, void *dgate,
                             float *dweight, float *dbias, void *workspace,
                             size_t workspace_bytes, void *stream) {
    if (int c = norm_args(io, B, G, T, D, act, eps)) return c;
    if (!workspace || workspace_bytes < osdn_group_norm_backward_workspace_bytes(B, G, T, D))
        return OSDN_ERR_WORKSPACE;
    const size_t n = (size_t)B * G * T * D * io_bytes(io), C = (size_t)G * D * 4;
    if (n && (!x || !dy || !dx || (gate && !dgate))) return OSDN_ERR_NULL;
    const Buf bufs[] = {{x, n, false}, {dy, n, false}, {weight, C, false}, {bias, C, false},
                        {gate, n, false}, {dx, n, true}, {gate ? dgate : nullptr, n, true},
                        {dweight, C, true}, {dbias, C, true}, {workspace, workspace_bytes, true}};
    if (int c = check_bufs(bufs)) return c;
    if (int c = check_device()) return c;
    return done(osdn::group_norm_backward_launch(
        io, B, G, T, D, heads_first, x, dy, weight, bias, gate, act, eps, dx, dgate, dweight, dbias,
        static_cast<char *>(workspace) + kStatusBytes, (cudaStream_t)stream));
}

size_t osdn_clip_grad_norm_workspace_bytes(int n) {
    return kStatusBytes + osdn::clip_scratch_bytes(n > 0 ? n : 1);
}

int osdn_clip_grad_norm(int n, const void *const *grads, void *const *outs,
                        const long long *sizes, const int *ios, float max_norm, float *norm,
                        void *workspace, size_t workspace_bytes, void *stream) {
    if (n < 0) return OSDN_ERR_DIMS;
    if (!(max_norm >= 0.0f)) return OSDN_ERR_ARG;
    if (!workspace || workspace_bytes < osdn_clip_grad_norm_workspace_bytes(n)) return OSDN_ERR_WORKSPACE;
    if (n > 0 && (!grads || !sizes || !ios)) return OSDN_ERR_NULL;
    if (misaligned(workspace) || (reinterpret_cast<uintptr_t>(norm) & 3u)) return OSDN_ERR_ALIGN;
    long long elements = 0;   // a launch numbers chunks of 2^13 in 32 bits
    for (int i = 0; i < n; ++i) {
        if (!io_ok(ios[i])) return OSDN_ERR_DTYPE;
        if (sizes[i] < 0 || sizes[i] > (1LL << 40)) return OSDN_ERR_DIMS;
        if ((elements += sizes[i]) > (1LL << 44)) return OSDN_ERR_DIMS;
        if (sizes[i] == 0) continue;
        if (!grads[i] || (outs && !outs[i])) return OSDN_ERR_NULL;
        if (misaligned(grads[i]) || (outs && misaligned(outs[i]))) return OSDN_ERR_ALIGN;
    }
    const bool scale = outs || !std::isinf(max_norm);
    const auto span = [&](long long k) {   // the workspace, the norm, the gradients, the outputs
        const void *p = k == 0 ? workspace : norm;
        size_t b = k == 0 ? workspace_bytes : norm ? 4 : 0;
        bool out = true;
        if (k >= 2) {
            const long long i = k - 2 < n ? k - 2 : k - 2 - n;
            const bool in_place = !outs || outs[i] == grads[i];
            p = k - 2 < n ? grads[i] : outs[i];
            b = k - 2 < n || !in_place ? (size_t)sizes[i] * io_bytes(ios[i]) : 0;
            out = k - 2 < n ? in_place && scale : true;
        }
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        return Span{lo, lo + b, out ? lo + b : 0};
    };
    if (overlap(2 + (long long)n * (outs ? 2 : 1), span)) return OSDN_ERR_ALIAS;
    if (int c = check_device()) return c;
    return done(osdn::clip_launch(n, grads, outs, sizes, ios, max_norm, norm,
                                  static_cast<char *>(workspace) + kStatusBytes, (cudaStream_t)stream));
}

}  // extern "C"
