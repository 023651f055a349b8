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
// the update has fp32 accuracy (S_T within 4e-7 of 64 bits; a plain bf16 K^
// would leave 2e-3).  Where the state is not an output two parts do.  The
// chunk's decay a^L, which a state meets hundreds of times, comes from
// repeated squaring in two fp32 (decay_attn.cuh).
//
// Time axis.  Every CTA takes a range of the chunks of all sequences (one
// CTA a SM, nearly equal ranges).  A range that starts inside a sequence
// needs the state there: a first launch (STATE_ONLY: K, V and the state
// update alone) forms each range's addition to the state, chain_states joins
// them, the second launch does the work.  That reads K and V once more (1.5
// times the unsplit bytes), so ranges that hold whole sequences are preferred
// where they fill the GPU.  The launches overlap: the second one's CTAs start
// as the first one's leave and form K^, Q K^T and P before they need a state
// (8x8x2048x128 75 -> 63 us with the cheaper numbering of ranges).
//
// Roles (15 warps): 0 TMA; 1 MMA issue for the outputs; 2-5 P out of TMEM,
// weighted, back as a TMEM operand, and O out of TMEM to global memory, a
// row a lane in whole sectors; 6-13 the state: K^ in two steps of 64 tokens
// (its first part in K's place), each multiplied while the next is formed,
// then the update of S and its bf16 copy; 14 MMA issue for the state.
// STATE_ONLY: 16 warps form K^; it takes its chunks last to first with
// weights up to the range's end, so that they add up in TMEM, four at a time
// (see kGroup), and leaves in L2 what the second launch reads first.
// 224 KB hold two tiles of K, one of V and Q, S and two parts of K^; the next
// V and Q are brought to L2 meanwhile.
//
// Bound.  At K = V = 128 a chunk is 128 KB in and out, 2.9 us at an SM's
// share of HBM; its products take 3100 cycles of the tensor pipe and, as
// their operands come from shared memory at 128 bytes a cycle, most of the
// 4700 cycles of shared-memory traffic that a chunk cannot do without (352 KB
// for the products, 160 KB for forming K^ and S, 96 KB arriving).  A chunk
// takes about 6000 cycles (3.2 us): the second launch 60 us at 2x16x8192x128,
// DRAM at 0.54 and the tensor pipe at 0.42 of their peaks, the first 33 us.
// What was measured on the way there, second launch at 2x16x8192x128: short
// role loops instead of unrolled ones, which miss the instruction cache, 124
// -> 80 us; the tile's transposition for whole-row stores of O 78 -> 68 us; K
// a chunk ahead 68 -> 60 us.  26 warps (16 for the state, 8 for P and O)
// were slower (108 us), and so were steps of 32 tokens (64 -> 70 us), P V
// ahead of Q S^T (+4 us for the three launches) and straight-line issue of
// the state's products (+5 us: they crowd K^'s traffic out).
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
constexpr int kStep = 64;       // tokens of K^ formed at a time
constexpr int kSteps = C / kStep;
// warps that form K^ (the first eight of them also hold the state), and a launch's threads
constexpr int state_warps(bool state_only) { return state_only ? 16 : 8; }
constexpr int threads(bool state_only) { return (7 + state_warps(state_only)) * 32; }
constexpr uint32_t kColP = 0;     // Q K^T, then P (bf16) over it
constexpr uint32_t kColO1 = 128;  // Q S^T
constexpr uint32_t kColO2 = 256;  // P V
constexpr uint32_t kColD = 384;   // V^T K^
constexpr uint32_t kTmemCols = 512;
// STATE_ONLY adds kGroup chunks up in TMEM before the sum goes to registers: two sets of columns in
// turn, in each one for K^'s first part and one for the others.  The tensor cores cut every sum off
// at 24 bits, so that each of the eight products a chunk with the first part costs the sum up to
// 2^-24; the others are 2^-8 as large and cost nothing where they have columns of their own.
constexpr int kGroup = 4;
__host__ __device__ constexpr uint32_t group_col(int group, int small) { return 256 * (group & 1) + 128 * small; }

template <int K, int V, bool STATE_ONLY>
struct Lay {
    static constexpr int NV = STATE_ONLY ? 2 : 1;          // tiles of V (two do not fit beside Q and S)
    static constexpr int kK = C * K * 2, kV = C * V * 2;   // a tile of K (or Q), of V
    static constexpr int oK = 0;
    static constexpr int oV = oK + 2 * kK;
    // the parts of K^: the second and third (the first takes K's place), in STATE_ONLY all three
    // (K's place is free the earlier)
    static constexpr int oP = oV + NV * kV;
    static constexpr int oQ = oP + (STATE_ONLY ? 3 : 2) * kK;
    static constexpr int oS = oQ + (STATE_ONLY ? 0 : kK);   // bf16 S: V rows of K columns
    static constexpr int kBytes = oS + (STATE_ONLY ? 0 : V * K * 2);
    static constexpr int kAlloc = kBytes + 1024;
};

struct Args {
    Pass p;
    Split s;
    float *states;   // [G][V][K], see chain_states; NULL: every range is a whole sequence
    int *status;     // status[1]: test word, see osdn.h
};

struct Bars {
    uint64_t fullK[2], emptyK[2], fullV[2], emptyV[2], fullQ, emptyQ;
    uint64_t qk_full, p_ready, o_full, o_free;
    uint64_t kq_full[kSteps], kq_free[kSteps], s_ready, ds_full, ds_free, done[2];
};

// A condition whose code is kept out of the loop's straight line.
__device__ __forceinline__ bool rare(bool c) { return __builtin_expect(c, 0); }

// The waits' loops, once in the kernel instead of at every wait.
__device__ __noinline__ bool wait_on(uint64_t *b, uint32_t parity, volatile int *abort, int *st, uint32_t limit) {
    return wait_bar(b, parity, abort, st, limit);
}
__device__ __noinline__ bool poll_on(uint64_t *b, uint32_t parity, volatile int *abort, int *st, uint32_t limit) {
    return wait_poll(b, parity, abort, st, limit);
}

// The chunks of a range, one after another.
struct Walk {
    int seq, u, nch, T, rev;
    __device__ Walk(const Args &a, int at) : nch(a.s.nch), T(a.p.T), rev(a.p.rev) {
        seq = at / nch;
        u = at - seq * nch;
    }
    __device__ void next() {
        if (++u == nch) {
            u = 0;
            ++seq;
        }
    }
    __device__ void prev() { --u; }   // within a sequence
    // the chunk's first token, and its length (a sequence's last tokens may be fewer than C)
    __device__ int row() const { return (rev ? nch - 1 - u : u) * C; }
    __device__ int len() const { return min(C, T - row()); }
};

__device__ __forceinline__ uint32_t top2(float a, float b) {   // the upper 16 bits of both
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float top(float a) { return __uint_as_float(__float_as_uint(a) & 0xffff0000u); }

// PARTS: the parts of K^.  Three where the state is an output; two (16 bits) where it only enters
// Q S^T, as bf16.
template <int K, int V, bool STATE_ONLY, int PARTS>
__global__ void __launch_bounds__(threads(STATE_ONLY), 1)
attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                 const __grid_constant__ CUtensorMap tm_v, Args a) {
    using LY = Lay<K, V, STATE_ONLY>;
    constexpr int NV = LY::NV, NW = state_warps(STATE_ONLY);
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = tc::align1024(smem_raw);
    __shared__ Bars bars;
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int s_abort;
    __shared__ __align__(16) float s_pow[4][96];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, q4 = warp & 3;
    const int g = blockIdx.x;
    const Pass &p = a.p;
    int lo = a.s.lo(g);
    const int hi = a.s.lo(g + 1);
    if (STATE_ONLY) {   // only the sequence that this range leaves unfinished
        dependents_may_start();
        if (hi % a.s.nch == 0) return;
        lo = max(lo, hi / a.s.nch * a.s.nch);
    }
    const int n = hi - lo;
    int *st = a.status;
    const int stall = *reinterpret_cast<volatile int *>(st + 1);
    const uint32_t bar_limit = stall ? 64u : tc::kWaitLimit;
    const uint32_t poll_limit = stall ? (1u << 14) : (tc::kWaitLimit << 11);
    auto wait = [&](uint64_t &b, int parity) {   // by a whole warp
        return __all_sync(kFullMask, ptx::mbar_try_wait(&b, parity & 1) || wait_on(&b, parity & 1, &s_abort, st, bar_limit));
    };
    auto poll = [&](uint64_t &b, int parity) {   // by one thread, on the critical path
        return ptx::mbar_try_wait(&b, parity & 1) || poll_on(&b, parity & 1, &s_abort, st, poll_limit);
    };
    auto arrive = [&](uint64_t &b) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&b);
    };

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&bars.fullK[i], 1);
            ptx::mbar_init(&bars.fullV[i], 1);
            // K's place: free once it has been read (STATE_ONLY) or, as K^'s first part, multiplied
            ptx::mbar_init(&bars.emptyK[i], STATE_ONLY ? NW : 1);
            ptx::mbar_init(&bars.emptyV[i], STATE_ONLY ? 1 : 2);
            ptx::mbar_init(&bars.done[i], 1);
        }
        for (int i = 0; i < kSteps; ++i) {
            ptx::mbar_init(&bars.kq_full[i], NW);
            ptx::mbar_init(&bars.kq_free[i], 1);
        }
        uint64_t *one[] = {&bars.fullQ, &bars.emptyQ, &bars.qk_full, &bars.o_full, &bars.ds_full};
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
    auto sV = [&](int j) { return smem + LY::oV + (j % NV) * LY::kV; };

    if (warp == 0) {
        // ======================================================== TMA
        if (lane == 0 && !stall) {
            // One loop over all loads, in the order in which their places fall free: K a chunk ahead,
            // (not STATE_ONLY) Q, V.
            constexpr int kinds = STATE_ONLY ? 2 : 3;
            int last[3] = {-1, -1, -1};
            Walk w(a, STATE_ONLY ? hi - 1 : lo);
#pragma unroll 1
            for (int i = 0; i < n * kinds; ++i) {
                const int j = i / kinds, kind = i % kinds;
                const bool is_k = kind == 0, is_v = kind == kinds - 1;
                const int nb = is_k ? 2 : is_v ? NV : 1, at = is_k ? j & 1 : is_v ? j % NV : 0;
                uint64_t *full = is_v ? &bars.fullV[at] : is_k ? &bars.fullK[at] : &bars.fullQ;
                uint64_t *empty = is_v ? &bars.emptyV[at] : is_k ? &bars.emptyK[at] : &bars.emptyQ;
                if (j >= nb && !wait_on(empty, (j / nb - 1) & 1, &s_abort, st, bar_limit)) break;
                const CUtensorMap *tm = is_v ? &tm_v : is_k ? &tm_k : &tm_q;
                uint8_t *dst = is_v ? sV(j) : is_k ? sK(j) : smem + LY::oQ;
                const int width = is_v ? V : K;
                ptx::mbar_arrive_expect_tx(full, C * width * 2);
#pragma unroll 1
                for (int b = 0; b < width / 64; ++b)
                    ptx::tma_load_3d(dst + b * C * 128, tm, full, b * 64, w.row(), w.seq);
                // a single place: the next tile is brought as far as L2 meanwhile
                if (!STATE_ONLY && !is_k && j + 1 < n) {
                    Walk x = w;
                    x.next();
                    ptx::bulk_prefetch_l2(static_cast<const __nv_bfloat16 *>(is_v ? p.v : p.q) +
                                              ((size_t)x.seq * p.T + x.row()) * width, x.len() * width * 2);
                }
                if (is_k) last[0] = j;
                else if (is_v) last[2] = j;
                else last[1] = j;
                if (is_v) STATE_ONLY ? w.prev() : w.next();
            }
            // every copy has landed before the CTA ends, also after an abort
            for (int j = max(0, last[0] - 1); j <= last[0]; ++j) drain_bar(&bars.fullK[j & 1], (j >> 1) & 1);
            for (int j = max(0, last[2] - NV + 1); j <= last[2]; ++j) drain_bar(&bars.fullV[j % NV], (j / NV) & 1);
            if (last[1] >= 0) drain_bar(&bars.fullQ, last[1] & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ======================================================== MMA issue: the outputs
        if (lane == 0 && !STATE_ONLY) {
            const uint32_t id_qk = ptx::idesc_bf16(C, C, 0, 0), id_qs = ptx::idesc_bf16(C, V, 0, 0);
            const uint32_t id_pv = ptx::idesc_bf16(C, V, 0, 1);
            const uint32_t q = ptx::smem_u32(smem + LY::oQ), s = ptx::smem_u32(smem + LY::oS);
#pragma unroll 1
            for (int j = 0; j < n; ++j) {
                const uint32_t k = ptx::smem_u32(sK(j)), v = ptx::smem_u32(sV(j));
                // P's columns are free once the last P V has completed; and every waiter has seen the
                // last Q K^T (the warps that form K^ show it), so that no phase of qk_full is missed
                if (!poll(bars.fullK[j & 1], j >> 1) || !poll(bars.fullQ, j) ||
                    (j && (!poll(bars.o_full, j - 1) || !poll(bars.kq_full[0], j - 1))))
                    break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < K / 64; ++b)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        ptx::umma_bf16(tmem + kColP, dk0(q + b * C * 128) + koff(C, ks), dk0(k + b * C * 128) + koff(C, ks), id_qk, b + ks > 0);
                ptx::umma_commit(&bars.qk_full);
                if (!poll(bars.s_ready, j) || (j && !poll(bars.o_free, j - 1))) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < K / 64; ++b)
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        ptx::umma_bf16(tmem + kColO1, dk0(q + b * C * 128) + koff(C, ks), dk0(s + b * V * 128) + koff(V, ks), id_qs, b + ks > 0);
                ptx::umma_commit(&bars.emptyQ);
                if (!poll(bars.fullV[j % NV], j / NV) || !poll(bars.p_ready, j)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int ks = 0; ks < C / 32; ++ks)
                        ptx::umma_bf16_ts(tmem + kColO2, tmem + kColP + 8 * (ks + b * C / 32), dmn0(v + b * C * 64, C * 128) + mnoff(ks), id_pv, b + ks > 0);
                ptx::umma_commit(&bars.o_full);
                ptx::umma_commit(&bars.emptyV[j % NV]);
            }
            // every product issued has completed before TMEM is released
            ptx::umma_commit(&bars.done[0]);
            drain_bar(&bars.done[0], 0);
        }
        __syncwarp();
    } else if (warp == 6 + NW) {
        // ======================================================== MMA issue: the state
        if (lane == 0) {
            const uint32_t id_d = ptx::idesc_bf16(V, K, 1, 1);
            const uint32_t parts = ptx::smem_u32(smem + LY::oP);
            bool ok = true;
            for (int j = 0; j < n && ok; ++j) {
                const uint32_t v = ptx::smem_u32(sV(j));
                ok = poll(bars.fullV[j % NV], j / NV) &&
                     (STATE_ONLY || !j || poll(bars.ds_free, j - 1));
#pragma unroll 1
                for (int h = 0; ok && h < kSteps; ++h) {   // V^T K^ step by step, small parts first
                    if (!(ok = poll(bars.kq_full[h], j))) break;
                    ptx::tc_fence_after();
#pragma unroll 1
                    for (int part = PARTS - 1; part >= 0; --part) {
                        const uint64_t da = dmn0(v, C * 128) + mnoff(kStep / 16 * h);
                        const uint32_t at = STATE_ONLY ? parts + part * LY::kK : part ? parts + (part - 1) * LY::kK : ptx::smem_u32(sK(j));
                        const uint64_t db = dmn0(at, C * 128) + mnoff(kStep / 16 * h);
#pragma unroll
                        for (int ks = 0; ks < kStep / 16; ++ks)
                            ptx::umma_bf16(tmem + (STATE_ONLY ? group_col(j / kGroup, part > 0) : kColD), da + mnoff(ks),
                                           db + mnoff(ks), id_d,
                                           STATE_ONLY ? j % kGroup || h || part == 1 || ks : h || part < PARTS - 1 || ks);
                    }
                    if (STATE_ONLY) ptx::umma_commit(&bars.kq_free[h]);
                }
                if (!ok) break;
                if (!STATE_ONLY || j % kGroup == kGroup - 1 || j == n - 1) ptx::umma_commit(&bars.ds_full);
                ptx::umma_commit(&bars.emptyV[j % NV]);
                if (!STATE_ONLY) ptx::umma_commit(&bars.emptyK[j & 1]);
            }
            ptx::umma_commit(&bars.done[1]);
            drain_bar(&bars.done[1], 0);
        }
        __syncwarp();
    } else if (warp < 6) {
        // ======================================================== P and O
        if (!STATE_ONLY) {
            const int r = 32 * q4 + lane;   // row of the chunk
            // Key block b (32 columns) against the row's own block, d blocks away: the weight of
            // column m is far[d-1] col[m], far from the row to the near end of the block and col
            // from there on; on the diagonal it is a^gap, read from the same table.  Scores that the
            // mask hides are put to zero, not multiplied by it: they may have overflowed.
            float *col = s_pow[warp - 2] + 32;
            const float *diag = col + (p.rev ? -lane : 31 - lane);
            const uint32_t seen = p.rev ? kFullMask << lane : kFullMask >> (31 - lane);   // columns of the diagonal block
            const bool wide = (reinterpret_cast<uintptr_t>(p.o) & 31) == 0;
            float wq = 0.0f, far[3] = {0.0f, 0.0f, 0.0f};
            int have = -1;
            int have_len = 0;
            Walk w(a, lo);
            for (int j = 0; j < n; ++j, w.next()) {
                const int len = w.len();
                if (rare(w.seq != have || len != have_len)) {
                    const float dec = p.decay[w.seq % p.H];
                    __syncwarp();
                    const float l2 = decay_log2(dec);
                    col[lane] = weight(l2, p.rev ? lane : 31 - lane);
                    col[lane - 32] = col[lane + 32] = 0.0f;
                    __syncwarp();
                    wq = weight(l2, p.rev ? max(len - 1 - r, 0) : r + 1);
#pragma unroll
                    for (int d = 0; d < 3; ++d) far[d] = weight(l2, (p.rev ? 31 - lane : lane) + 1 + 32 * d);
                    have = w.seq;
                    have_len = len;
                }
                if (!wait(bars.qk_full, j)) break;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int b = 0; b < 4; ++b) {
                    const int d = p.rev ? b - q4 : q4 - b;
                    float pk[16];
                    if (d < 0) {
#pragma unroll
                        for (int m = 0; m < 16; ++m) pk[m] = 0.0f;
                    } else {
                        float x[32];
                        tc::tmem_ld32(tmem + lane_off + kColP + 32 * b, x);
                        if (d == 0) {
#pragma unroll
                            for (int m = 0; m < 32; ++m) x[m] = seen >> m & 1 ? x[m] : 0.0f;
#pragma unroll
                            for (int m = 0; m < 16; ++m)
                                pk[m] = __uint_as_float(tc::pack_bf16x2(x[2 * m] * diag[2 * m], x[2 * m + 1] * diag[2 * m + 1]));
                        } else {
                            const float f = d == 1 ? far[0] : d == 2 ? far[1] : far[2];
                            const float2 ff = make_float2(f, f);
#pragma unroll
                            for (int m = 0; m < 16; m += 2) {
                                const float4 c = *reinterpret_cast<const float4 *>(col + 2 * m);
                                const float2 y = __fmul2_rn(__fmul2_rn(make_float2(x[2 * m], x[2 * m + 1]), ff), make_float2(c.x, c.y));
                                const float2 z = __fmul2_rn(__fmul2_rn(make_float2(x[2 * m + 2], x[2 * m + 3]), ff), make_float2(c.z, c.w));
                                pk[m] = __uint_as_float(tc::pack_bf16x2(y.x, y.y));
                                pk[m + 1] = __uint_as_float(tc::pack_bf16x2(z.x, z.y));
                            }
                        }
                    }
                    ptx::tmem_st16(tmem + lane_off + kColP + 16 * b, pk);
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                arrive(bars.p_ready);

                if (!wait(bars.o_full, j)) break;
                ptx::tc_fence_after();
                __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.o) + ((size_t)w.seq * p.T + w.row() + r) * V;
#pragma unroll 1
                for (int c = 0; c < V; c += 32) {
                    float x[2][16], y[2][16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        ptx::tmem_ld16(tmem + lane_off + kColO1 + c + 16 * h, x[h]);
                        ptx::tmem_ld16(tmem + lane_off + kColO2 + c + 16 * h, y[h]);
                    }
                    ptx::tmem_wait_ld();
                    if (c + 32 == V) {
                        ptx::tc_fence_before();
                        arrive(bars.o_free);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t out[8];
#pragma unroll
                        for (int m = 0; m < 8; ++m) {
                            const float2 u = __ffma2_rn(make_float2(wq, wq), make_float2(x[h][2 * m], x[h][2 * m + 1]),
                                                        make_float2(y[h][2 * m], y[h][2 * m + 1]));
                            out[m] = tc::pack_bf16x2(u.x, u.y);
                        }
                        if (r >= len) continue;
                        if (wide) {   // whole 32-byte sectors
                            ptx::st_global_256(o + c + 16 * h, out);
                        } else {
                            *reinterpret_cast<uint4 *>(o + c + 16 * h) = make_uint4(out[0], out[1], out[2], out[3]);
                            *reinterpret_cast<uint4 *>(o + c + 16 * h + 8) = make_uint4(out[4], out[5], out[6], out[7]);
                        }
                    }
                }
            }
        }
    } else {
        // ======================================================== K^ and the state
        // row i of S: TMEM lane i (V = 128) or 32 (i / 16) + i % 16 (V = 64); columns c0 ..
        constexpr int NC = K * 4 / NW;
        const int c0 = ((warp - 6) >> 2) * NC;
        const int row = V == 128 ? 32 * q4 + lane : 16 * q4 + lane;
        const bool act = V == 128 || lane < 16;
        constexpr size_t sb = (size_t)K * V;
        // K^: a lane takes the rows of its number in 32s, a warp NC8 pieces of eight columns (and,
        // where there are more warps than pieces, a share of the rows)
        constexpr int P8 = K / 8, NC8 = P8 > NW ? P8 / NW : 1, RG = NW > P8 ? NW / P8 : 1;
        constexpr int NR = kStep / 32 / RG;   // 32s of rows a step
        const int piece = (warp - 6) % (P8 / NC8) * NC8, rg = (warp - 6) / (P8 / NC8) * NR;
        float S[NC], wk[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        Pow f = {1.0f, 0.0f};    // the chunk's whole decay; STATE_ONLY: from the chunk's end to the range's
        Pow fc = {1.0f, 0.0f};
        int have = -1, have_len = 0;
        bool ok = true;
        Walk w(a, STATE_ONLY ? hi - 1 : lo);
        // STATE_ONLY: the group's sums into registers.  A warp does that before it forms more K^, so
        // that kq_full of the group after the next finds the columns free.
        auto add_group = [&](int group) {
            if (!wait(bars.ds_full, group)) return false;
            ptx::tc_fence_after();
#pragma unroll
            for (int e = 0; e < NC; e += 16) {
                float x[16], y[16];
                ptx::tmem_ld16(tmem + lane_off + group_col(group, 0) + c0 + e, x);
                ptx::tmem_ld16(tmem + lane_off + group_col(group, 1) + c0 + e, y);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) S[e + i] += x[i] + y[i];
            }
            ptx::tc_fence_before();
            return true;
        };
        if (STATE_ONLY) {
#pragma unroll
            for (int e = 0; e < NC; ++e) S[e] = 0.0f;
        }
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
            const int len = w.len();
            if (rare(w.seq != have || len != have_len)) {
                const float dec = p.decay[w.seq % p.H];
                if (!decay_ok(dec)) report_status(st, OSDN_ERR_DEVICE);
                const float l2 = decay_log2(dec);
#pragma unroll
                for (int qt = 0; qt < 4; ++qt) {
                    // the token's distance to the chunk's end, in the pass's direction
                    const int kr = 32 * qt + lane, e = p.rev ? kr + 1 : len - 1 - kr;
                    wk[qt] = weight(l2, max(e, 0));
                }
                fc = decay_pow(dec, len);
                if (!STATE_ONLY) f = fc;
                have = w.seq;
                have_len = len;
            }
            if (!STATE_ONLY) {
                if (rare(j == 0 || w.u == 0)) {   // the state entering the range, or a sequence
                    const float *src = nullptr;
                    bool tr = false;
                    if (w.u > 0) {
                        dependency_wait();
                        src = a.states + (size_t)g * sb;
                        tr = p.given;
                    } else if (p.S0.p) {
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
                // the copy of the last chunk's state has been read by Q S^T
                if (j && !(ok = wait(bars.emptyQ, j - 1))) break;
                if (act) tc::st_row_sw128(smem + LY::oS, V, row, c0, S, NC);
                ptx::fence_proxy_async_smem();
                arrive(bars.s_ready);
            }
            // K has arrived, and been read by Q K^T where its first part takes its place
            if (!(ok = STATE_ONLY ? wait(bars.fullK[j & 1], j >> 1) : wait(bars.qk_full, j))) break;
#pragma unroll 1
            for (int h = 0; h < kSteps; ++h) {
                // K^ of the last chunk has been read (before its state was, where that is read)
                if (STATE_ONLY && j && !(ok = wait(bars.kq_free[h], j - 1))) break;
                const float2 minus = make_float2(-1.0f, -1.0f);
#pragma unroll 2
                for (int i = 0; i < NR * NC8; ++i) {
                    const int r32 = h * (kStep / 32) + rg + i / NC8, c = piece + i % NC8;
                    float wt = r32 < 2 ? (r32 ? wk[1] : wk[0]) : (r32 == 2 ? wk[2] : wk[3]);
                    if (STATE_ONLY) wt *= f.hi;
                    const float2 ww = make_float2(wt, wt);
                    const int at = (c >> 3) * C * 128 + (32 * r32 + lane) * 128 + ((c & 7) ^ (lane & 7)) * 16;
                    const uint4 u = *reinterpret_cast<const uint4 *>(sK(j) + at);
                    const uint32_t in[4] = {u.x, u.y, u.z, u.w};
                    uint32_t ph[4], pm[4], pl[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 x = __fmul2_rn(make_float2(__uint_as_float(in[e] << 16), __uint_as_float(in[e] & 0xffff0000u)), ww);
                        const float2 m = __ffma2_rn(make_float2(top(x.x), top(x.y)), minus, x);
                        ph[e] = top2(x.x, x.y);
                        pm[e] = top2(m.x, m.y);
                        if (PARTS == 3) {
                            const float2 l = __ffma2_rn(make_float2(top(m.x), top(m.y)), minus, m);
                            pl[e] = top2(l.x, l.y);
                        }
                    }
                    uint8_t *dst = smem + LY::oP + at + (STATE_ONLY ? LY::kK : 0);
                    *reinterpret_cast<uint4 *>(STATE_ONLY ? smem + LY::oP + at : sK(j) + at) = make_uint4(ph[0], ph[1], ph[2], ph[3]);
                    *reinterpret_cast<uint4 *>(dst) = make_uint4(pm[0], pm[1], pm[2], pm[3]);
                    if (PARTS == 3)
                        *reinterpret_cast<uint4 *>(dst + LY::kK) = make_uint4(pl[0], pl[1], pl[2], pl[3]);
                }
                ptx::fence_proxy_async_smem();
                arrive(bars.kq_full[h]);
            }
            if (!ok) break;
            if (STATE_ONLY) {
                arrive(bars.emptyK[j & 1]);
                f = pow_mul(f, fc);
                w.prev();
                if (j && j % kGroup == 0 && !(ok = add_group(j / kGroup - 1))) break;
            } else {
                if (!(ok = wait(bars.ds_full, j))) break;
                ptx::tc_fence_after();
                const float2 fh = make_float2(f.hi, f.hi), fl = make_float2(f.lo, f.lo);
#pragma unroll
                for (int e = 0; e < NC; e += 32) {
                    float x[32];
                    tc::tmem_ld32(tmem + lane_off + kColD + c0 + e, x);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 s = make_float2(S[e + i], S[e + i + 1]);
                        const float2 u = __ffma2_rn(fh, s, __ffma2_rn(fl, s, make_float2(x[i], x[i + 1])));
                        S[e + i] = u.x;
                        S[e + i + 1] = u.y;
                    }
                }
                ptx::tc_fence_before();
                arrive(bars.ds_free);
                if (rare(w.u == a.s.nch - 1 && p.ST && act)) {
                    float *dst = p.ST + (size_t)w.seq * sb;
#pragma unroll
                    for (int e = 0; e < NC; e += 4) {
                        const float x[4] = {S[e], S[e + 1], S[e + 2], S[e + 3]};
                        store4(dst + (size_t)row * K + c0 + e, x);
                    }
                }
                w.next();
            }
        }
        if (STATE_ONLY && ok && add_group((n - 1) / kGroup) && act) {
            float *dst = a.states + (size_t)(g + 1) * sb + (size_t)row * K + c0;
#pragma unroll
            for (int i = 0; i < NC; i += 4) {
                const float y[4] = {S[i], S[i + 1], S[i + 2], S[i + 3]};
                store4(dst + i, y);
            }
        }
    }

    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) ptx::tmem_dealloc(tmem, kTmemCols);
}

template <int K, int V, bool STATE_ONLY, int PARTS>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Args &a,
                   cudaStream_t stream) {
    constexpr int smem = Lay<K, V, STATE_ONLY>::kAlloc;
    static std::atomic<unsigned long long> attr_done{0};
    cudaError_t e = smem_attr_once((const void *)attend_tc_kernel<K, V, STATE_ONLY, PARTS>, smem, attr_done);
    if (e != cudaSuccess) return e;
    // no range follows the last one, so nothing needs its state
    return launch_overlapped(!STATE_ONLY && a.states && !a.p.given, attend_tc_kernel<K, V, STATE_ONLY, PARTS>,
                             dim3(a.s.G - (STATE_ONLY ? 1 : 0)), threads(STATE_ONLY), smem, stream, mq, mk, mv, a);
}

template <int K, int V>
cudaError_t run(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const Args &a,
                cudaStream_t stream) {
    if (a.states && !a.p.given) {
        cudaError_t e = launch<K, V, true, 3>(mq, mk, mv, a, stream);
        if (e == cudaSuccess) e = chain_states(a.p, a.s, a.states, stream);
        if (e != cudaSuccess) return e;
    }
    if (a.p.ST) return launch<K, V, false, 3>(mq, mk, mv, a, stream);
    return launch<K, V, false, 2>(mq, mk, mv, a, stream);
}

}  // namespace

Split tc_split(int BH, int T, int, int) {
    const int nch = (int)(((long long)T + C - 1) / C);
    const long long slots = tc::sm_count(), N = (long long)BH * nch;
    // In sixths of a chunk's time: a split pass reads K and V twice (half as much again),
    // has two more launches (about two chunks' time) and chains the ranges of a sequence (four in
    // one).
    long long best = (BH + slots - 1) / slots * nch * 6, G = BH;
    for (long long g = std::min(N, slots); g > BH; g /= 2) {
        const long long cost = (N + g - 1) / g * 9 + 12 + g / BH / 4;
        if (cost < best) {
            best = cost;
            G = g;
        }
    }
    return make_split(C, 1, BH, T, (int)G);
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
    a.states = unsplit(a.s, p.BH) ? nullptr : static_cast<float *>(scratch);
    a.status = status;
    if (p.K == 128) return p.V == 128 ? run<128, 128>(mq, mk, mv, a, stream) : run<128, 64>(mq, mk, mv, a, stream);
    return p.V == 128 ? run<64, 128>(mq, mk, mv, a, stream) : run<64, 64>(mq, mk, mv, a, stream);
}

}  // namespace da
}  // namespace osdn
