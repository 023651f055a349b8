// decay_attn_tc.cu -- linear attention with a decay per head on the sm_103a
// tensor cores (tcgen05 + TMEM + TMA), bf16 I/O:
//     S_t = a S_{t-1} + v_t k_t^T,   o_t = S_t q_t,   a = decay[h]
//
// A chunk of C = 128 tokens (rows of Q, K, V; S the state entering it):
//     O  = diag(a^(i+1)) Q S^T + P V,     P_ij = a^(i-j) (q_i . k_j), j <= i
//     S' = a^L S + V^T K^,                K^_j = a^(L-1-j) k_j   (L tokens)
// Backwards in time (for the gradients, see decay_attn.cuh) the same with
// the chunk's order reversed, the carry read one power earlier.
//
// Precision.  P and the copy of S that multiplies Q are rounded to bf16: each
// is one operand rounding of the size of the output's own.  The state itself
// is an output and is carried over thousands of tokens, so it is kept in
// fp32 (in registers), and K^ enters the product as three bf16 parts
// (8 + 8 + 8 bits, exactly the fp32 product a^e k): V is exact in bf16, so
// the update has fp32 accuracy.  Powers of the decay come from repeated
// squaring in two fp32 (decay_attn.cuh).
//
// Bound.  Q, K, V in and O out are 128 KB a chunk at K = V = 128, 2.9 us at
// an SM's share of HBM; the six 128^3 products take about 1.6 us of the
// tensor pipe.  So the kernel is HBM-bound if everything overlaps, and the
// chain of chunks needs few steps: only the register update of S and the
// product Q S^T wait for the chunk before.
//
// Time axis.  Every CTA takes a range of the chunks of all sequences (one
// CTA a SM, nearly equal ranges).  A range that starts inside a sequence
// needs the state there: a first launch (STATE_ONLY: K, V and the state
// update alone) forms each range's addition to the state, chain_states joins
// them, the second launch does the work.  That reads K and V once more, so
// ranges that hold whole sequences are preferred where they fill the GPU.
//
// Roles (18 warps): 0 TMA; 1 MMA issue; 2-5 P out of TMEM, weighted, back as
// a TMEM operand, and O to global memory; 6-9 K^ in halves of 64 tokens (the
// first part over K, the others in two buffers of 16 KB); 10-17 the state.
// Every wait is bounded: one that runs out records OSDN_ERR_TIMEOUT and all
// roles leave their loops; no role waits for another in any other way.
#include <algorithm>

#include "decay_attn.cuh"
#include "tc_common.cuh"

namespace osdn {
namespace da {

namespace {

using tc::dk0;
using tc::dmn0;
using tc::drain_bar;
using tc::koff;
using tc::mnoff;
using tc::wait_bar;
using tc::wait_poll;

constexpr int C = 128;          // tokens a chunk
constexpr int kThreads = 576;
constexpr uint32_t kColP = 0;     // Q K^T, then P (bf16) over it
constexpr uint32_t kColO1 = 128;  // Q S^T
constexpr uint32_t kColO2 = 256;  // P V
constexpr uint32_t kColD = 384;   // V^T K^
constexpr uint32_t kTmemCols = 512;

template <int K, int V>
struct Lay {
    static constexpr int kK = C * K * 2, kV = C * V * 2;   // a tile of K (or Q), of V
    static constexpr int oK = 0;
    static constexpr int oV = oK + 2 * kK;
    static constexpr int oQ = oV + 2 * kV;
    static constexpr int oS = oQ + kK;               // bf16 S: V rows of K columns
    static constexpr int oM = oS + V * K * 2;        // second and third parts of half a K^
    static constexpr int oL = oM + kK / 2;
    static constexpr int kBytes = oL + kK / 2;
    static constexpr int kAlloc = kBytes + 1024;
};

struct Args {
    Pass p;
    Split s;
    float *states;   // [G][V][K], see chain_states
    int *status;     // status[1]: test word, see osdn.h
};

struct Bars {
    uint64_t fullK[2], fullV[2], emptyKV[2], fullQ, emptyQ;
    uint64_t qk_full, p_ready, o_full, o_free;
    uint64_t kh[2], h0_done, s_ready, ds_full, ds_free, done;
};

// The chunks of a range, one after another.
struct Walk {
    long long seq;
    int u, nch, T, rev;
    __device__ Walk(const Args &a, long long at) : nch(a.s.nch), T(a.p.T), rev(a.p.rev) {
        seq = at / nch;
        u = (int)(at - seq * nch);
    }
    __device__ void next() {
        if (++u == nch) {
            u = 0;
            ++seq;
        }
    }
    // first row of the chunk's tile (negative for the last chunk backwards), tokens in it
    __device__ int row() const { return rev ? T - (u + 1) * C : u * C; }
    __device__ int len() const { return min(C, T - u * C); }
};

__device__ __forceinline__ uint32_t top2(float a, float b) {   // the upper 16 bits of both
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float top(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

template <int K, int V, bool STATE_ONLY>
__global__ void __launch_bounds__(kThreads, 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, Args a) {
    using LY = Lay<K, V>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = tc::align1024(smem_raw);
    __shared__ Bars bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int s_abort;
    __shared__ float s_pow[4][32];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q4 = warp & 3;
    const int g = blockIdx.x;
    const Pass &p = a.p;
    long long lo = a.s.lo(g, p.BH);
    const long long hi = a.s.lo(g + 1, p.BH);
    if (STATE_ONLY) {   // only the sequence that this range leaves unfinished
        if (hi % a.s.nch == 0) return;
        lo = max(lo, hi / a.s.nch * a.s.nch);
    }
    const int n = (int)(hi - lo);
    int *st = a.status;
    const int stall = *reinterpret_cast<volatile int *>(st + 1);
    const uint32_t bar_limit = stall ? 64u : tc::kWaitLimit;
    const uint32_t poll_limit = stall ? (1u << 14) : (tc::kWaitLimit << 11);
    auto wait = [&](uint64_t &b, int parity) {   // by a whole warp
        return __all_sync(kFullMask, wait_bar(&b, parity & 1, &s_abort, st, bar_limit));
    };
    auto arrive = [&](uint64_t &b) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b);
    };

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars.fullK[i], 1);
            ptx::mbar_init(&bars.fullV[i], 1);
            ptx::mbar_init(&bars.emptyKV[i], 1);
            ptx::mbar_init(&bars.kh[i], 4);
        }
        uint64_t *one[] = {&bars.fullQ, &bars.emptyQ, &bars.qk_full, &bars.o_full, &bars.h0_done,
                           &bars.ds_full, &bars.done};
        for (uint64_t *b : one) ptx::mbar_init(b, 1);
        ptx::mbar_init(&bars.p_ready, 4);
        ptx::mbar_init(&bars.o_free, 4);
        ptx::mbar_init(&bars.s_ready, 8);
        ptx::mbar_init(&bars.ds_free, 8);
        ptx::fence_mbar_init();
        s_abort = 0;
    }
    if (warp == 1) {
        ptx::tmem_alloc(&tmem_base_sh, kTmemCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_sh;
    const uint32_t lane_off = static_cast<uint32_t>(32 * q4) << 16;
    auto sK = [&](int j) { return smem + LY::oK + (j & 1) * LY::kK; };
    auto sV = [&](int j) { return smem + LY::oV + (j & 1) * LY::kV; };

    if (warp == 0) {
        // ======================================================== TMA
        if (lane == 0 && !stall) {
            int last_kv = -1, last_q = -1;
            Walk w(a, lo), wq(a, lo);
            auto load_kv = [&](int j) {
                if (j >= 2 && !wait_bar(&bars.emptyKV[j & 1], ((j >> 1) - 1) & 1, &s_abort, st, bar_limit)) return false;
                ptx::mbar_arrive_expect_tx(&bars.fullK[j & 1], LY::kK);
#pragma unroll
                for (int b = 0; b < K / 64; ++b)
                    ptx::tma_load_3d(sK(j) + b * C * 128, &tm_k, &bars.fullK[j & 1], b * 64, w.row(), (int)w.seq);
                ptx::mbar_arrive_expect_tx(&bars.fullV[j & 1], LY::kV);
#pragma unroll
                for (int b = 0; b < V / 64; ++b)
                    ptx::tma_load_3d(sV(j) + b * C * 128, &tm_v, &bars.fullV[j & 1], b * 64, w.row(), (int)w.seq);
                last_kv = j;
                w.next();
                return true;
            };
            bool ok = load_kv(0);
            for (int j = 0; j < n && ok; ++j) {
                if (!STATE_ONLY) {
                    if (j >= 1 && !wait_bar(&bars.emptyQ, (j - 1) & 1, &s_abort, st, bar_limit)) break;
                    ptx::mbar_arrive_expect_tx(&bars.fullQ, LY::kK);
#pragma unroll
                    for (int b = 0; b < K / 64; ++b)
                        ptx::tma_load_3d(smem + LY::oQ + b * C * 128, &tm_q, &bars.fullQ, b * 64, wq.row(), (int)wq.seq);
                    last_q = j;
                    wq.next();
                    // the next Q waits for this buffer: bring it as far as L2 meanwhile
                    if (j + 1 < n && wq.row() >= 0) {
#pragma unroll
                        for (int b = 0; b < K / 64; ++b) ptx::tma_prefetch_3d(&tm_q, b * 64, wq.row(), (int)wq.seq);
                    }
                }
                if (j + 1 < n) ok = load_kv(j + 1);
            }
            // every copy has landed before the CTA ends, also after an abort
            for (int j = max(0, last_kv - 1); j <= last_kv; ++j) {
                drain_bar(&bars.fullK[j & 1], (j >> 1) & 1);
                drain_bar(&bars.fullV[j & 1], (j >> 1) & 1);
            }
            if (last_q >= 0) drain_bar(&bars.fullQ, last_q & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ======================================================== MMA issue
        if (lane == 0) {
            auto pw = [&](uint64_t &b, int parity) { return wait_poll(&b, parity & 1, &s_abort, st, poll_limit); };
            const uint32_t id_qk = ptx::idesc_bf16(C, C, 0, 0), id_qs = ptx::idesc_bf16(C, V, 0, 0);
            const uint32_t id_pv = ptx::idesc_bf16(C, V, 0, 1), id_d = ptx::idesc_bf16(V, K, 1, 1);
            const uint32_t q = ptx::smem_u32(smem + LY::oQ), s = ptx::smem_u32(smem + LY::oS);
            const uint32_t km = ptx::smem_u32(smem + LY::oM), kl = ptx::smem_u32(smem + LY::oL);
            for (int j = 0; j < n; ++j) {
                const uint32_t k = ptx::smem_u32(sK(j)), v = ptx::smem_u32(sV(j));
                auto add_half = [&](int h) {   // V^T K^ over the half's tokens, small parts first
#pragma unroll
                    for (int part = 2; part >= 0; --part) {
                        const uint64_t db = part == 0 ? dmn0(k, C * 128) + mnoff(4 * h)
                                                      : dmn0(part == 1 ? km : kl, C * 64);
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks)
                            ptx::umma_bf16(tmem + kColD, dmn0(v, C * 128) + mnoff(4 * h + ks), db + mnoff(ks), id_d,
                                           h > 0 || part < 2 || ks > 0);
                    }
                };
                if (!pw(bars.fullK[j & 1], j >> 1)) break;
                if (!STATE_ONLY) {
                    // P's columns are free once the last P V has completed
                    if (!pw(bars.fullQ, j) || (j && !pw(bars.o_full, j - 1))) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < K / 16; ++ks)
                        ptx::umma_bf16(tmem + kColP, dk0(q) + koff(C, ks), dk0(k) + koff(C, ks), id_qk, ks > 0);
                    ptx::umma_commit(&bars.qk_full);
                    if (!pw(bars.s_ready, j) || (j && !pw(bars.o_free, j - 1))) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < K / 16; ++ks)
                        ptx::umma_bf16(tmem + kColO1, dk0(q) + koff(C, ks), dk0(s) + koff(V, ks), id_qs, ks > 0);
                    ptx::umma_commit(&bars.emptyQ);
                }
                if (!pw(bars.fullV[j & 1], j >> 1) || !pw(bars.kh[0], j) || (j && !pw(bars.ds_free, j - 1))) break;
                ptx::tc_fence_after();
                add_half(0);
                ptx::umma_commit(&bars.h0_done);
                if (!STATE_ONLY) {
                    if (!pw(bars.p_ready, j)) break;
                    ptx::tc_fence_after();
#pragma unroll
                    for (int ks = 0; ks < C / 16; ++ks)
                        ptx::umma_bf16_ts(tmem + kColO2, tmem + kColP + 8 * ks, dmn0(v, C * 128) + mnoff(ks), id_pv,
                                          ks > 0);
                    ptx::umma_commit(&bars.o_full);
                }
                if (!pw(bars.kh[1], j)) break;
                ptx::tc_fence_after();
                add_half(1);
                ptx::umma_commit(&bars.ds_full);
                ptx::umma_commit(&bars.emptyKV[j & 1]);
            }
            // every product issued has completed before TMEM is released
            ptx::umma_commit(&bars.done);
            drain_bar(&bars.done, 0);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ======================================================== P and O
        if (!STATE_ONLY) {
            const int r = 32 * q4 + lane;   // row of the chunk
            float *tab = s_pow[warp - 2];
            float wq = 0.0f, far[3] = {0.0f, 0.0f, 0.0f};
            long long have = -1;
            Walk w(a, lo);
            for (int j = 0; j < n; ++j, w.next()) {
                if (w.seq != have) {
                    // a^m; the row's power on the carry; a^(gap to the near end of block 1, 2, 3 away)
                    const float dec = p.decay[w.seq % p.H];
                    __syncwarp();
                    tab[lane] = decay_pow(dec, lane).hi;
                    __syncwarp();
                    wq = decay_pow(dec, p.rev ? C - 1 - r : r + 1).hi;
                    const int near = p.rev ? 31 - lane : lane;
#pragma unroll
                    for (int d = 0; d < 3; ++d) far[d] = decay_pow(dec, near + 1 + 32 * d).hi;
                    have = w.seq;
                }
                if (!wait(bars.qk_full, j)) break;
                ptx::tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {   // 32 columns: keys 32 b ..
                    const int d = p.rev ? b - q4 : q4 - b;   // blocks between the row's and the keys'
                    float x[32];
                    uint32_t pk[16];
                    if (d >= 0) {
                        tc::tmem_ld32(tmem + lane_off + kColP + 32 * b, x);
                        if (d == 0) {
#pragma unroll
                            for (int m = 0; m < 32; ++m) {
                                const int gap = p.rev ? m - lane : lane - m;
                                x[m] = gap >= 0 ? x[m] * tab[max(gap, 0)] : 0.0f;
                            }
                        } else {
                            const float f = d == 1 ? far[0] : d == 2 ? far[1] : far[2];
#pragma unroll
                            for (int m = 0; m < 32; ++m) x[m] *= f * tab[p.rev ? m : 31 - m];
                        }
                    } else {
#pragma unroll
                        for (int m = 0; m < 32; ++m) x[m] = 0.0f;
                    }
                    float packed[16];
#pragma unroll
                    for (int m = 0; m < 16; ++m) {
                        pk[m] = tc::pack_bf16x2(x[2 * m], x[2 * m + 1]);
                        packed[m] = __uint_as_float(pk[m]);
                    }
                    ptx::tmem_st16(tmem + lane_off + kColP + 16 * b, packed);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                arrive(bars.p_ready);

                if (!wait(bars.o_full, j)) break;
                ptx::tc_fence_after();
                const int t = w.row() + r;
                const bool live = t >= 0 && t < p.T;
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((size_t)w.seq * p.T + max(t, 0)) * V;
#pragma unroll
                for (int c = 0; c < V; c += 32) {
                    float x[32], y[32];
                    tc::tmem_ld32(tmem + lane_off + kColO1 + c, x);
                    tc::tmem_ld32(tmem + lane_off + kColO2 + c, y);
                    if (c + 32 == V) {
                        ptx::tc_fence_before();
                        arrive(bars.o_free);
                    }
#pragma unroll
                    for (int h = 0; h < 32; h += 16) {
                        uint32_t out[8];
#pragma unroll
                        for (int m = 0; m < 8; ++m)
                            out[m] = tc::pack_bf16x2(fmaf(wq, x[h + 2 * m], y[h + 2 * m]),
                                                     fmaf(wq, x[h + 2 * m + 1], y[h + 2 * m + 1]));
                        if (live) {
                            *reinterpret_cast<uint4 *>(o + c + h) = make_uint4(out[0], out[1], out[2], out[3]);
                            *reinterpret_cast<uint4 *>(o + c + h + 8) = make_uint4(out[4], out[5], out[6], out[7]);
                        }
                    }
                }
            }
        }
    } else if (warp < 10) {
        // ======================================================== K^
        const int rt = (tid - 192) & 63, c0 = ((tid - 192) >> 6) * (K / 2);   // row of the half, first column
        float wk[2] = {0.0f, 0.0f};
        long long have = -1;
        int have_len = 0;
        Walk w(a, lo);
        for (int j = 0; j < n; ++j, w.next()) {
            const int len = w.len();
            if (w.seq != have || len != have_len) {
                const float dec = p.decay[w.seq % p.H];
                if (!decay_ok(dec)) report_status(st, OSDN_ERR_DEVICE);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    // the token's distance to the chunk's end, in the pass's direction
                    const int row = 64 * h + rt, e = p.rev ? len - C + 1 + row : len - 1 - row;
                    wk[h] = decay_pow(dec, max(e, 0)).hi;
                }
                have = w.seq;
                have_len = len;
            }
            // K as loaded has been read by Q K^T; the halves' buffers by the last chunk's update
            if (STATE_ONLY ? !wait(bars.fullK[j & 1], j >> 1) : !wait(bars.qk_full, j)) break;
            if (j && !wait(bars.ds_full, j - 1)) break;
            bool ok = true;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h && !wait(bars.h0_done, j)) {
                    ok = false;
                    break;
                }
                uint8_t *hi_row = sK(j) + (c0 >> 6) * C * 128 + (64 * h + rt) * 128;
                uint8_t *mid_row = smem + LY::oM + (c0 >> 6) * C * 64 + rt * 128;
                uint8_t *lo_row = smem + LY::oL + (c0 >> 6) * C * 64 + rt * 128;
#pragma unroll
                for (int i = 0; i < K / 16; ++i) {
                    const int off = ((((c0 & 63) >> 3) + i) ^ (rt & 7)) * 16;
                    const uint4 u = *reinterpret_cast<const uint4 *>(hi_row + off);
                    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                    uint32_t ph[4], pm[4], pl[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float x0 = __uint_as_float(in[e] << 16) * wk[h];
                        const float x1 = __uint_as_float(in[e] & 0xffff0000u) * wk[h];
                        const float m0 = x0 - top(x0), m1 = x1 - top(x1);
                        ph[e] = top2(x0, x1);
                        pm[e] = top2(m0, m1);
                        pl[e] = top2(m0 - top(m0), m1 - top(m1));
                    }
                    *reinterpret_cast<uint4 *>(hi_row + off) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                    *reinterpret_cast<uint4 *>(mid_row + off) = make_uint4(pm[0], pm[1], pm[2], pm[3]);
                    *reinterpret_cast<uint4 *>(lo_row + off) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                }
                ptx::fence_proxy_async_smem();
                arrive(bars.kh[h]);
            }
            if (!ok) break;
        }
    } else {
        // ======================================================== state
        // row i of S: TMEM lane i (V = 128) or 32 (i / 16) + i % 16 (V = 64); columns c0 ..
        constexpr int NC = K / 2;
        const int c0 = ((warp - 10) >> 2) * NC;
        const int row = V == 128 ? 32 * q4 + lane : 16 * q4 + lane;
        const bool act = V == 128 || lane < 16;
        constexpr size_t sb = (size_t)K * V;
        float S[NC];
        Pow f = {0.0f, 0.0f};
        long long have = -1;
        int have_len = 0;
        Walk w(a, lo);
        for (int j = 0; j < n; ++j, w.next()) {
            const int len = w.len();
            if (w.seq != have || len != have_len) {
                f = decay_pow(p.decay[w.seq % p.H], len);
                have = w.seq;
                have_len = len;
            }
            if (j == 0 || w.u == 0) {   // the state entering the range, or a sequence
                const float *src = nullptr;
                bool tr = false;
                if (!STATE_ONLY && w.u > 0) {
                    src = a.states + (size_t)g * sb;
                } else if (!STATE_ONLY && p.S0.p) {
                    src = p.S0.p + (size_t)w.seq * sb;
                    tr = p.S0.transposed;
                }
#pragma unroll
                for (int e = 0; e < NC; e += 4) {
                    float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    if (src && act && !tr) load4(src + (size_t)row * K + c0 + e, x);
                    if (src && act && tr) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = src[(size_t)(c0 + e + i) * V + row];
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) S[e + i] = x[i];
                }
            }
            if (!STATE_ONLY) {
                // the copy of the last chunk's state has been read by Q S^T
                if (j && !wait(bars.emptyQ, j - 1)) break;
                if (act) tc::st_row_sw128(smem + LY::oS, V, row, c0, S, NC);
                ptx::fence_proxy_async_smem();
                arrive(bars.s_ready);
            }
            if (!wait(bars.ds_full, j)) break;
            ptx::tc_fence_after();
#pragma unroll
            for (int e = 0; e < NC; e += 16) {
                float x[16];
                ptx::tmem_ld16(tmem + lane_off + kColD + c0 + e, x);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[e + i] = fmaf(f.hi, S[e + i], fmaf(f.lo, S[e + i], x[i]));
            }
            ptx::tc_fence_before();
            arrive(bars.ds_free);
            float *dst = nullptr;
            bool tr = false;
            if (STATE_ONLY) {
                if (j == n - 1) dst = a.states + (size_t)(g + 1) * sb;
            } else if (w.u == a.s.nch - 1 && p.ST.p) {
                dst = p.ST.p + (size_t)w.seq * sb;
                tr = p.ST.transposed;
            }
            if (dst && act) {
#pragma unroll
                for (int e = 0; e < NC; e += 4) {
                    const float x[4] = {S[e], S[e + 1], S[e + 2], S[e + 3]};
                    if (!tr) {
                        store4(dst + (size_t)row * K + c0 + e, x);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) dst[(size_t)(c0 + e + i) * V + row] = x[i];
                    }
                }
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int K, int V, bool STATE_ONLY>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Args &a,
                   cudaStream_t stream) {
    constexpr int smem = Lay<K, V>::kAlloc;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = smem_attr_once((const void *)attend_tc_kernel<K, V, STATE_ONLY>, smem, attr_done);
    if (e != cudaSuccess) return e;
    // no range follows the last one, so nothing needs its state
    attend_tc_kernel<K, V, STATE_ONLY><<<a.s.G - (STATE_ONLY ? 1 : 0), kThreads, smem, stream>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

template <int K, int V>
cudaError_t run(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Args &a,
                cudaStream_t stream) {
    if (!unsplit(a.s, a.p.BH)) {
        cudaError_t e = launch<K, V, true>(mq, mk, mv, a, stream);
        if (e == cudaSuccess) e = chain_states(a.p, a.s, a.states, stream);
        if (e != cudaSuccess) return e;
    }
    return launch<K, V, false>(mq, mk, mv, a, stream);
}

}  // namespace

Split tc_split(int BH, int T, int, int) {
    Split s;
    s.unit = C;
    s.nch = (T + C - 1) / C;
    s.G = BH;
    const long long slots = tc::sm_count(), N = (long long)BH * s.nch, G = std::min(N, slots);
    // chunks in a row: a split pass reads K and V twice (half as much again), and has two more
    // launches (about three chunks' time)
    const long long whole = (BH + slots - 1) / slots * s.nch;
    const long long split = (N + G - 1) / G * 3 / 2 + 3;
    if (G > BH && split < whole) s.G = (int)G;
    return s;
}

cudaError_t attend_tc(const Pass &p, void *scratch, int *status, cudaStream_t stream) {
    if (!tc::tensor_map_encoder_ready()) return cudaErrorNotSupported;
    CUtensorMap mq, mk, mv;
    if (!tc::make_map(&mq, p.q, p.BH, p.T, p.K, C) || !tc::make_map(&mk, p.k, p.BH, p.T, p.K, C) ||
        !tc::make_map(&mv, p.v, p.BH, p.T, p.V, C))
        return cudaErrorInvalidValue;
    Args a;
    a.p = p;
    a.s = tc_split(p.BH, p.T, p.K, p.V);
    a.states = static_cast<float *>(scratch);
    a.status = status;
    if (p.K == 128) return p.V == 128 ? run<128, 128>(mq, mk, mv, a, stream) : run<128, 64>(mq, mk, mv, a, stream);
    return p.V == 128 ? run<64, 128>(mq, mk, mv, a, stream) : run<64, 64>(mq, mk, mv, a, stream);
}

}  // namespace da
}  // namespace osdn
