// decay_attn.cu -- linear attention with a decay per head, the token
// recurrence in fp32 FFMA:
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a = decay[h]
// for fp32 I/O, where tensor-core operand rounding would not keep fp32
// accuracy.
//
// The rows of S evolve independently, so a CTA of 128 threads takes 64 rows
// of one range of the time axis: a thread holds four rows' columns 32m + 4p +
// {0..3} (p = lane & 7), so that k and q come from shared memory as 16-byte
// reads that serve four rows, and the four dot products are summed over the
// eight lanes together, four shuffles.  With two rows a thread those reads,
// four cycles a warp each, took twice the arithmetic's time (2x16x8192x128
// 16% longer, 1024 sequences of 256 tokens 25%).
// The decay costs no multiplication a token: over groups of eight tokens the
// state is kept as S~ = a^-n S (v is scaled instead) and multiplied by a^8
// once a group, as long as a^-8 <= 2, so that S~ leaves fp32's range only where
// S is within a factor of 2 of doing so.  Heads that forget faster (a < 0.917,
// a memory of 12 tokens) decay token by token, which takes a tenth longer
// (2x16x4096x128: 520 us with a = 0.95, 569 us with 0.9).  Groups of four and
// two tokens for those between, chosen at run time, would cost the others 6%,
// and noticing an overflow to do the tokens over 15%.
//
// Bound: 2 K V multiply-adds a token, 232 us for 262144 token-heads of 128x128
// (half as much again, for the states alone, where the time axis is cut).
// 1024 sequences of 256 tokens take 644 us, 0.36 of that rate; 2x16x8192, which
// is cut, 1020 us, 0.34.  Twelve warps a SM (160 registers a thread) issue in
// 0.54 of the slots, half of them multiply-adds: the rest is reads, sums over
// lanes and their latency.
#include "decay_attn.cuh"

#include <algorithm>

namespace osdn {
namespace da {

namespace {

constexpr int kThreads = 128;
constexpr int kRows = 64;
constexpr int kStage = 8;    // tokens staged at a time
constexpr int kGroup = 8;    // tokens between rescalings
constexpr float kGrouped = 0.917005f;   // the least decay with a^-kGroup <= 2
constexpr int kUnit = 16;    // tokens a unit of the split

struct Args {
    Pass p;
    Split s;
    float *states;   // [G][V][K], see chain_states; NULL: every range is a whole sequence
    int *status;
};

template <int K, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 3) attend_simt_kernel(Args a) {
    constexpr int M = K / 32, R = 4;   // 32s of columns, rows a thread
    __shared__ __align__(16) float ks[kStage][K], qs[STATE_ONLY ? 1 : kStage][K];
    __shared__ __align__(16) float vs[kStage][kRows];
    __shared__ Pow pows[kGroup + 1];     // a^n
    __shared__ float2 updown[kGroup];   // a^-x and a^x after a group's n-th token
    const Pass &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int pc = lane & 7, row = warp * 16 + (lane >> 3) * R, row0 = blockIdx.x * kRows;
    const int g = blockIdx.y + gridDim.y * blockIdx.z;
    if (g >= a.s.G) return;
    int lo = a.s.lo(g);
    const int hi = a.s.lo(g + 1);
    if (STATE_ONLY) {   // only the sequence that this range leaves unfinished
        dependents_may_start();
        if (g + 1 >= a.s.G || hi % a.s.nch == 0) return;
        lo = max(lo, hi / a.s.nch * a.s.nch);
    } else if (a.states) {
        dependency_wait();
    }
    const float *q = static_cast<const float *>(p.q), *k = static_cast<const float *>(p.k);
    const float *v = static_cast<const float *>(p.v);
    float *o = static_cast<float *>(p.o);

    constexpr int NK = kStage * K / (kThreads * 4), NV = kStage * kRows / (kThreads * 4);
    float rk[NK][4], rq[STATE_ONLY ? 1 : NK][4], rv[NV][4];
    for (int at = lo; at < hi;) {
        const int seq = at / a.s.nch, u0 = at - seq * a.s.nch, u1 = min(a.s.nch, u0 + (hi - at));
        const int tbeg = u0 * kUnit, tend = min(p.T, u1 * kUnit);
        at += u1 - u0;
        const float dec = p.decay[seq % p.H];
        if (!decay_ok(dec) && tid == 0) report_status(a.status, OSDN_ERR_DEVICE);
        const bool grouped = dec >= kGrouped;
        const size_t kb = (size_t)seq * p.T * K, vb = (size_t)seq * p.T * p.V + row0;
        auto fetch = [&](int t0) {   // the stage's tokens, in the pass's direction
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const int idx = (tid + n * kThreads) * 4, t = t0 + idx / K;
                const size_t r = kb + (size_t)(p.rev ? p.T - 1 - t : t) * K + idx % K;
#pragma unroll
                for (int e = 0; e < 4; ++e) rk[n][e] = 0.0f;
                if (t < tend) load4(k + r, rk[n]);
                if (!STATE_ONLY) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) rq[n][e] = 0.0f;
                    if (t < tend) load4(q + r, rq[n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) {
                const int idx = (tid + n * kThreads) * 4, t = t0 + idx / kRows;
                const size_t r = vb + (size_t)(p.rev ? p.T - 1 - t : t) * p.V + idx % kRows;
#pragma unroll
                for (int e = 0; e < 4; ++e) rv[n][e] = 0.0f;
                if (t < tend) load4(v + r, rv[n]);
            }
        };
        float2 S[R][M][2];
        {
            const size_t sb = (size_t)p.K * p.V;
            const float *src = nullptr;
            bool tr = false;
            if (!STATE_ONLY && u0 > 0) {
                src = a.states + (size_t)g * sb;
                tr = p.given;
            } else if (!STATE_ONLY && p.S0.p) {
                src = p.S0.p + (size_t)seq * sb;
                tr = p.S0.transposed;
            }
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    const int c = 32 * m + 4 * pc, i = row0 + row + r;
                    if (src && !tr) load4(src + (size_t)i * K + c, x);
                    if (src && tr) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) x[e] = src[(size_t)(c + e) * p.V + i];
                    }
                    S[r][m][0] = make_float2(x[0], x[1]);
                    S[r][m][1] = make_float2(x[2], x[3]);
                }
        }
        auto scale = [&](Pow f) {
            const float2 h = make_float2(f.hi, f.hi), l = make_float2(f.lo, f.lo);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        S[r][m][e] = __ffma2_rn(h, S[r][m][e], __fmul2_rn(l, S[r][m][e]));
        };
        auto forget = [&] {   // one token's decay
            const float2 h = make_float2(dec, dec);
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m)
#pragma unroll
                    for (int e = 0; e < 2; ++e) S[r][m][e] = __fmul2_rn(h, S[r][m][e]);
        };
        __syncthreads();   // the last sequence's powers have been read
        if (tid <= kGroup) pows[tid] = decay_pow(dec, tid);
        if (tid < kGroup) {
            // S_t = a^x S~ after the token, x counted from the group's start
            const float down = grouped ? decay_pow(dec, tid + (p.rev ? 0 : 1)).hi : 1.0f;
            updown[tid] = make_float2(1.0f / down, down);
        }
        fetch(tbeg);
        for (int t0 = tbeg; t0 < tend; t0 += kStage) {
            __syncthreads();   // the last stage has been read
#pragma unroll
            for (int n = 0; n < NK; ++n) {
                const int idx = (tid + n * kThreads) * 4;
                store4(&ks[0][0] + idx, rk[n]);
                if (!STATE_ONLY) store4(&qs[0][0] + idx, rq[n]);
            }
#pragma unroll
            for (int n = 0; n < NV; ++n) store4(&vs[0][0] + (tid + n * kThreads) * 4, rv[n]);
            __syncthreads();
            if (t0 + kStage < tend) fetch(t0 + kStage);
            const int tn = min(kStage, tend - t0);
#pragma unroll 2
            for (int tt = 0; tt < tn; ++tt) {
                const int in = tt & (kGroup - 1);
                const float up = updown[in].x, down = updown[in].y;
                if (!grouped && !p.rev) forget();
                float2 w[R], dot[R];
                {
                    float vv[R];
                    load4(&vs[tt][row], vv);
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        w[r] = make_float2(up * vv[r], up * vv[r]);
                        dot[r] = make_float2(0.0f, 0.0f);
                    }
                }
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const float4 kk = *reinterpret_cast<const float4 *>(&ks[tt][32 * m + 4 * pc]);
                    const float2 ka = make_float2(kk.x, kk.y), kc = make_float2(kk.z, kk.w);
                    float2 qa, qc;
                    if (!STATE_ONLY) {
                        const float4 qq = *reinterpret_cast<const float4 *>(&qs[tt][32 * m + 4 * pc]);
                        qa = make_float2(qq.x, qq.y);
                        qc = make_float2(qq.z, qq.w);
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        S[r][m][0] = __ffma2_rn(w[r], ka, S[r][m][0]);
                        S[r][m][1] = __ffma2_rn(w[r], kc, S[r][m][1]);
                        if (!STATE_ONLY) dot[r] = __ffma2_rn(S[r][m][1], qc, __ffma2_rn(S[r][m][0], qa, dot[r]));
                    }
                }
                if (!STATE_ONLY) {
                    // four sums over eight lanes: each exchange halves the rows a lane still carries
                    float s[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) s[r] = dot[r].x + dot[r].y;
                    const bool b0 = pc & 1, b1 = pc & 2;
                    float s0 = (b0 ? s[2] : s[0]) + __shfl_xor_sync(kFullMask, b0 ? s[0] : s[2], 1);
                    float s1 = (b0 ? s[3] : s[1]) + __shfl_xor_sync(kFullMask, b0 ? s[1] : s[3], 1);
                    s0 = (b1 ? s1 : s0) + __shfl_xor_sync(kFullMask, b1 ? s0 : s1, 2);
                    s0 += __shfl_xor_sync(kFullMask, s0, 4);
                    const int t = t0 + tt;
                    if (pc < 4) o[vb + (size_t)(p.rev ? p.T - 1 - t : t) * p.V + row + 2 * (pc & 1) + (pc >> 1)] = down * s0;
                }
                if (!grouped && p.rev) forget();
                if (grouped && (in == kGroup - 1 || tt == tn - 1)) scale(pows[in + 1]);
            }
        }
        float *dst = nullptr;
        const size_t sb = (size_t)p.K * p.V;
        if (STATE_ONLY) {
            dst = a.states + (size_t)(g + 1) * sb;
        } else if (tend == p.T && p.ST) {
            dst = p.ST + (size_t)seq * sb;
        }
        if (dst) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int m = 0; m < M; ++m) {
                    const int c = 32 * m + 4 * pc, i = row0 + row + r;
                    const float x[4] = {S[r][m][0].x, S[r][m][0].y, S[r][m][1].x, S[r][m][1].y};
                    store4(dst + (size_t)i * K + c, x);
                }
        }
    }
}

// One thread per four state elements of a sequence: the states entering the
// sequence's ranges, one after another.  Up to kAhead ranges' states are
// loaded before the first is used, and the powers between them (thread i's
// the i-th) come first, so that the chain itself is fused multiply-adds.
constexpr int kAhead = 8;
__global__ void __launch_bounds__(256) chain_states_kernel(Pass p, Split s, float *states) {
    __shared__ Pow pows[kAhead];
    const size_t seq = grid_seq();
    if (seq >= (size_t)p.BH) return;
    const int n = p.K * p.V, tid = threadIdx.x;
    const int e = (blockIdx.x * blockDim.x + tid) * 4;
    const int beg = (int)seq * s.nch, end = beg + s.nch;
    // the first range that starts inside this sequence: the least g with lo(g) > beg
    int g = beg < s.more * (s.each + 1) ? beg / (s.each + 1) + 1 : s.more + (beg - s.more * (s.each + 1)) / s.each + 1;
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (p.S0.p && e < n) {
        const float *src = p.S0.p + seq * n;
        if (!p.S0.transposed) {
            load4(src + e, c);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = src[(size_t)(e % p.K + i) * p.V + e / p.K];
        }
    }
    const float dec = p.decay[seq % p.H];
    dependents_may_start();
    bool waited = false;
    for (; g < s.G && s.lo(g) < end; g += kAhead) {
        int m = 0;   // ranges of this round
#pragma unroll
        for (int i = 0; i < kAhead; ++i) m += g + i < s.G && s.lo(g + i) < end;
        __syncthreads();   // the last round's powers have been read
        if (tid < m) {
            const int at = s.lo(g + tid), from = max(beg, s.lo(g + tid - 1));
            pows[tid] = decay_pow(dec, (unsigned)(s.before(at - beg, p.T, p.rev) - s.before(from - beg, p.T, p.rev)));
        }
        if (!waited) dependency_wait();
        waited = true;
        float x[kAhead][4];
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (i < m && e < n) load4(states + (size_t)(g + i) * n + e, x[i]);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (i >= m) break;
            const Pow f = pows[i];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = fmaf(f.hi, c[k], fmaf(f.lo, c[k], x[i][k]));
            if (e < n) store4(states + (size_t)(g + i) * n + e, c);
        }
    }
    // this launch completes only after the one before, whatever it had to do
    if (!waited) dependency_wait();
}

template <int K>
cudaError_t launch_simt(const Args &a, cudaStream_t stream) {
    const dim3 grid = seq_grid(a.p.V / kRows, a.s.G);
    const bool split = a.states != nullptr;
    cudaError_t e = cudaSuccess;
    if (split && !a.p.given) {
        e = launch_overlapped(false, attend_simt_kernel<K, true>, grid, kThreads, 0, stream, a);
        if (e == cudaSuccess) e = chain_states(a.p, a.s, a.states, stream);
    }
    if (e != cudaSuccess) return e;
    return launch_overlapped(split && !a.p.given, attend_simt_kernel<K, false>, grid, kThreads, 0, stream, a);
}

}  // namespace

cudaError_t chain_states(const Pass &p, const Split &s, float *states, cudaStream_t stream) {
    const dim3 grid = seq_grid((p.K * p.V / 4 + 255) / 256, p.BH);
    return launch_overlapped(true, chain_states_kernel, grid, 256, 0, stream, p, s, states);
}

Split simt_split(int BH, int T, int K, int V) {
    const int nch = (int)(((long long)T + kUnit - 1) / kUnit);
    // CTAs resident at once, in ranges (the same for K and V exchanged)
    const long long slots = 152LL * 3 / (std::max(K, V) / kRows);
    const long long N = (long long)BH * nch;
    // Tokens one after another: a split pass costs up to two thirds more (half the arithmetic again,
    // 1020 us where whole sequences take 644), two launches (about 40 tokens' time) and, in
    // chain_states, about one a range of a sequence.
    const long long whole = (BH + slots - 1) / slots * T;
    long long best = whole, G = BH;
    for (long long g = std::min(N, slots); g > BH; g /= 2) {
        const long long cost = (N + g - 1) / g * kUnit * 5 / 3 + 40 + g / BH;
        if (cost < best) {
            best = cost;
            G = g;
        }
    }
    return make_split(kUnit, 0, BH, T, (int)G);
}

cudaError_t attend_simt(const Pass &p, void *scratch, int *status, cudaStream_t stream) {
    Args a;
    a.p = p;
    a.s = simt_split(p.BH, p.T, p.K, p.V);
    a.states = unsplit(a.s, p.BH) ? nullptr : static_cast<float *>(scratch);
    a.status = status;
    return p.K == 128 ? launch_simt<128>(a, stream) : launch_simt<64>(a, stream);
}

}  // namespace da
}  // namespace osdn
