// Linear attention prompts on the sm_100a tensor cores (bf16 q, k, v; any K and V that are
// multiples of 8 up to 128: the TMA boxes fill the missing columns with zeros).
//
// One CTA per (segment, key/value head, 64 columns of V) walks the segment's 128-token
// chunks with the FP32 state in the registers of eight warps:
//
//     P  = (Q K^T) o lam^(t-s), s <= t        UMMA -> TMEM, warps scale and mask, bf16 -> TMEM
//     Oi = P V                                UMMA, A from TMEM
//     Ox = Q [S_hi | S_lo]                    UMMA, N = 128; S = S_hi + S_lo, a bf16 pair
//     o  = scale (Oi + lam^(t+1) (Ox_hi + Ox_lo))
//     D  = K^T (w V), w_s = lam^(len-1-s)     UMMA, three bf16 terms of w V
//     S' = lam^len S + D                      registers
//
// Roundings to bf16 and why: the scores P (as any attention on these tensor cores; 2^-8 of a
// term, no more than the result's own rounding); S as a pair (2^-16: with slow decays nearly
// all of o comes from S, and a single bf16 would double o's error); w V as three terms (2^-24:
// the FP32 final state is an output, and two terms leave it at 2e-6 relative).
//
// R query heads that share a key/value head are units (chunk, r) of the same CTA: K, V and
// the state are read and formed once for all of them.
//
// Work split: warp 0 issues TMA loads, warp 1 the UMMAs of P, Oi and Ox, warp 2 those of D (an
// issuing warp takes its batches in order, and D's waits would hold up the outputs'); then
// groups of warps for the scores (8), the outputs (4), w V (4) and the state (8). Q, K and V are
// double-buffered; the next unit's Q K^T runs while this one's scores are formed. w V goes
// through a ring of two 32-token parts, since three terms of a whole chunk do not fit.
// Without OUT (state pass): only loads, w V, D and the state.
//
// 64 columns of V per CTA: 128 would need a single-buffered Q, K, V and S (227 KB), and twice
// the CTAs fill the SMs of small batches; the price is Q K^T once per 64 columns.
//
// TMEM columns: Q K^T [0, 128) and [128, 256) (units alternate), P of a 32-token block in the
// first 16 columns of the block's scores (read and written by the same thread), Oi [256, 320),
// Ox [320, 448), D [448, 512).
#pragma once

#include "ssd_linattn.cuh"
#include "ssd_scan_tc.cuh"

namespace ssd {
namespace la {

constexpr int kTcC = 128;                    // tokens per chunk
constexpr int kTcV = 64;                     // V columns per CTA
constexpr int kPart = 32;                    // tokens per part of w V
constexpr int kScoreWarps = 8, kOutWarps = 4, kWriteWarps = 4, kStateWarps = 8;

constexpr int kOffK = 0;                     // 2 x [2 halves][128 tokens][64] bf16
constexpr int kOffV = 65536;                 // 2 x [128 tokens][64]
constexpr int kOffW = 98304;                 // 2 parts x 3 terms x [32 tokens][64]
constexpr int kOffS = 122880;                // hi, lo: [128 k][64 v]
constexpr int kOffQ = 155648;                // 2 x [2 halves][128 tokens][64]
constexpr int kTcSmemOut = 221184 + 1024;
constexpr int kTcSmemState = kOffS + 1024;

__host__ __device__ constexpr int tc_threads(bool out) {
    return 32 * (4 + (out ? kScoreWarps + kOutWarps : 0) + kWriteWarps + kStateWarps);
}

// Registers of the calling group of four warps, all of which execute it.
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

template <bool OUT>
__global__ void __launch_bounds__(tc_threads(OUT), 1)
k_la_tc(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
        const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args a) {
    using namespace tc;
    constexpr int NT = tc_threads(OUT);
    const int nvb = (a.V + kTcV - 1) / kTcV;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg<OUT>(a, blockIdx.x / nvb / a.Hk, &sg)) return;
    const int K = a.K, V = a.V, R = a.R, v0 = vb * kTcV, nv = min(kTcV, V - v0);
    const int nt = (sg.len + kTcC - 1) / kTcC;
    const int ksteps = (K + 15) / 16, halves = (K + 63) / 64;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float pw_pad[32 + kTcC + 1];  // 32 zeros, then lam^0 .. lam^128
    __shared__ __align__(16) float rev[32];  // lam^31 .. lam^0
    __shared__ float2 lam_full, lam_tail, lam_seg;
    __shared__ uint64_t full_kv[2], empty_kv[2], full_q[2], empty_q[2], qk_done[2], p_ready[2], o_done, o_free, qs_done,
        w_ready[2], w_free[2], d_done, d_free, s_ready, tail_ready, drained[2], stall_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const float* pw = pw_pad + 32;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float gd = a.log_decay[g];
    for (int i = tid; i < 32 + kTcC + 1; i += NT) pw_pad[i] = i < 32 ? 0.f : (float)exp((double)gd * (i - 32));
    if (tid < 32) rev[tid] = (float)exp((double)gd * (31 - tid));
    if (tid == 64) lam_full = pow2f(gd, kTcC);
    if (tid == 96) lam_tail = pow2f(gd, sg.len - (nt - 1) * kTcC);
    if (tid == 128) lam_seg = pow2f(gd, a.Ls);
    if (tid == 0) {
        check_decay(gd);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_kv[i], 1);
            mbar_init(&empty_kv[i], OUT ? 2 : 1);
            mbar_init(&full_q[i], 1);
            mbar_init(&empty_q[i], 1);
            mbar_init(&qk_done[i], 1);
            mbar_init(&p_ready[i], kScoreWarps);
            mbar_init(&w_ready[i], kWriteWarps);
            mbar_init(&w_free[i], 1);
            mbar_init(&drained[i], 1);
        }
        mbar_init(&o_done, 1);
        mbar_init(&o_free, kOutWarps);
        mbar_init(&qs_done, 1);
        mbar_init(&d_done, 1);
        mbar_init(&d_free, kStateWarps);
        mbar_init(&s_ready, kStateWarps);
        mbar_init(&tail_ready, kWriteWarps);
        mbar_init(&stall_bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    constexpr int kOutAt = 4 + kScoreWarps, kWriteAt = OUT ? kOutAt + kOutWarps : 4, kStateAt = kWriteAt + kWriteWarps;
    const int64_t per_state = (int64_t)a.Hk * V * K, head = ((int64_t)g * V + v0) * K;
    const int64_t ip = a.init ? page_of(a.init_pages, a.npages, sg.seq) : -1;
    int64_t fp = -1;
    if (OUT && sg.j + 1 == sg.n && a.fin) {
        fp = page_of(a.fin_pages, a.npages, sg.seq);
        if (a.fin_pages && fp >= 0 && page_clash(a, sg.seq, fp, NT)) {
            latch_error(SSD_ERR_INVALID_ARG);
            fp = -1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_slot, tOi = tbase + 256, tOx = tbase + 320, tD = tbase + 448;
    volatile int* abort_p = &abort_flag;
    const bool has_init = OUT && (ip >= 0 || sg.j > 0);           // the first chunk meets a state
    // Chunks whose D is formed: the last one's only for a state to write, or where the chunk is
    // partial, since forming w V also zeroes the tail of V.
    const bool partial = sg.len % kTcC != 0;
    const int nd = !OUT || fp >= 0 || partial ? nt : max(0, nt - 1);
    auto len_of = [&](int c) { return min(kTcC, sg.len - c * kTcC); };
    auto parts_of = [&](int c) { return (len_of(c) + kPart - 1) / kPart; };

    // Registers: 72 a thread at launch (896 threads), moved between groups of four warps:
    // 64 + 72 + 72 + 80 + 56 + 80 + 80 = 7 * 72.
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (OUT) regs_dec<64>();
        if (lane == 0 && nt > 0) {
            prefetch_tmap(&map_k);
            prefetch_tmap(&map_v);
            if (OUT) prefetch_tmap(&map_q);
            int nkv = 0, nq = 0;             // loads of K and V, of Q issued (alternating buffers)
            bool ok = true;
            for (int c = 0; c < nt && ok; ++c) {
                const int st = c & 1, t0 = (int)(sg.start + (int64_t)c * kTcC);
                if (c >= 2 && !wait_issue(&empty_kv[st], ((c >> 1) - 1) & 1, abort_p)) break;
                mbar_arrive_expect_tx(&full_kv[st], (halves + 1) * 16384);
                for (int h = 0; h < halves; ++h)
                    tma_load_3d(sm + kOffK + st * 32768 + h * 16384, &map_k, &full_kv[st], 64 * h, g, t0);
                tma_load_3d(sm + kOffV + st * 16384, &map_v, &full_kv[st], v0, g, t0);
                ++nkv;
                for (int r = 0; OUT && r < R; ++r) {
                    const int u = c * R + r, sq = u & 1;
                    if (u >= 2 && !wait_issue(&empty_q[sq], ((u >> 1) - 1) & 1, abort_p)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(&full_q[sq], halves * 16384);
                    for (int h = 0; h < halves; ++h)
                        tma_load_3d(sm + kOffQ + sq * 32768 + h * 16384, &map_q, &full_q[sq], 64 * h, g * R + r, t0);
                    ++nq;
                }
            }
            // The last phase issued on each barrier completes once its bytes have landed (a
            // phase is issued only after the previous one has been consumed).
            for (int i = 0; i < 2; ++i) {
                if (nkv > i) mbar_wait(&full_kv[i], ((nkv - 1 - i) >> 1) & 1);
                if (nq > i) mbar_wait(&full_q[i], ((nq - 1 - i) >> 1) & 1);
            }
        }
    } else if (OUT && warp == 1) {
        // ------------------------------------------------------------ UMMA issuer: P, Oi, Ox
        regs_dec<64>();
        const uint32_t id_x = idesc_bf16(128, 128, 0, 1), id_v = idesc_bf16(128, 64, 0, 1);
        const uint64_t dQ = smem_desc(smem_u32(sm + kOffQ), 16, 1024), dK = smem_desc(smem_u32(sm + kOffK), 16, 1024);
        const uint64_t dV = smem_desc(smem_u32(sm + kOffV), 16384, 1024), dS = smem_desc(smem_u32(sm + kOffS), 16384, 1024);
        // Q K^T of unit u = (c, r): N = the chunk's tokens rounded up to a part.
        auto issue_qk = [&](int c, int r, int u) -> bool {
            if (r == 0 && !wait_issue_warp(&full_kv[c & 1], (c >> 1) & 1, abort_p)) return false;
            if (!wait_issue_warp(&full_q[u & 1], (u >> 1) & 1, abort_p)) return false;
            tc_fence_after();
            const uint32_t id = idesc_bf16(128, kPart * parts_of(c), 0, 0), d = tbase + 128 * (u & 1);
            const uint64_t dq = desc_add(dQ, (u & 1) * 32768), dk = desc_add(dK, (c & 1) * 32768);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < ksteps)
                        umma_bf16(d, desc_add(dq, kmajor_step(128, k)), desc_add(dk, kmajor_step(128, k)), id, k > 0);
                umma_commit(&qk_done[u & 1]);
            }
            __syncwarp();
            return true;
        };
        // test hook (stall): a wait that runs out
        bool ok = nt > 0 && !(a.stall && !wait_issue_warp(&stall_bar, 0, abort_p)) && issue_qk(0, 0, 0);
        int u = 0;
        for (int c = 0; c < nt && ok; ++c) {
            const bool st = c > 0 || has_init;
            for (int r = 0; r < R && ok; ++r, ++u) {
                // The buffer of the next Q K^T holds P of unit u-1 until its product is done.
                const int cn = r == R - 1 ? c + 1 : c, rn = r == R - 1 ? 0 : r + 1;
                if (u > 0 && !wait_issue_warp(&o_done, (u - 1) & 1, abort_p)) { ok = false; break; }
                if (cn < nt && !issue_qk(cn, rn, u + 1)) { ok = false; break; }
                if (u > 0 && !wait_issue_warp(&o_free, (u - 1) & 1, abort_p)) { ok = false; break; }
                if (st && r == 0 && !wait_issue_warp(&s_ready, (has_init ? c : c - 1) & 1, abort_p)) { ok = false; break; }
                tc_fence_after();
                const uint64_t dq = desc_add(dQ, (u & 1) * 32768);
                const int xsteps = st ? ksteps : 0;
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < xsteps) umma_bf16(tOx, desc_add(dq, kmajor_step(128, k)), desc_add(dS, k * kMnStep), id_x, k > 0);
                    umma_commit(&empty_q[u & 1]);
                    if (r == R - 1) umma_commit(&qs_done);
                }
                __syncwarp();
                if (!wait_issue_warp(&p_ready[u & 1], (u >> 1) & 1, abort_p)) { ok = false; break; }
                // V's rows past the last token hold zeros
                if (partial && c == nt - 1 && r == 0 && !wait_issue_warp(&tail_ready, 0, abort_p)) { ok = false; break; }
                tc_fence_after();
                const int steps = parts_of(c) * (kPart / 16);
                const uint32_t tP = tbase + 128 * (u & 1);
                const uint64_t dv = desc_add(dV, (c & 1) * 16384);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < steps) umma_bf16_ts(tOi, tP + 32 * (k >> 1) + 8 * (k & 1), desc_add(dv, k * kMnStep), id_v, k > 0);
                    umma_commit(&o_done);
                    if (r == R - 1) umma_commit(&empty_kv[c & 1]);
                }
                __syncwarp();
            }
        }
        // Every MMA issued above has completed once this commit arrives.
        if (elect_one()) umma_commit(&drained[0]);
        __syncwarp();
        mbar_wait(&drained[0], 0);
    } else if (warp == 2) {
        // ------------------------------------------------------------ UMMA issuer: D
        if (OUT) regs_dec<64>();
        const uint32_t id_d = idesc_bf16(128, 64, 1, 1);
        const uint64_t dK = smem_desc(smem_u32(sm + kOffK), 16384, 1024), dW = smem_desc(smem_u32(sm + kOffW), 16384, 1024);
        bool ok = !(!OUT && a.stall && !wait_issue_warp(&stall_bar, 0, abort_p));     // test hook, as above
        int part = 0;                        // parts of w V consumed so far
        for (int c = 0; c < nd && ok; ++c) {
            if (!wait_issue_warp(&full_kv[c & 1], (c >> 1) & 1, abort_p)) break;
            if (c > 0 && !wait_issue_warp(&d_free, (c - 1) & 1, abort_p)) break;
            const int np = parts_of(c);
            for (int i = 0; i < np; ++i, ++part) {
                if (!wait_issue_warp(&w_ready[part & 1], (part >> 1) & 1, abort_p)) { ok = false; break; }
                tc_fence_after();
                const uint64_t dk = desc_add(dK, (c & 1) * 32768 + i * (kPart / 16) * kMnStep);
                const uint64_t dw = desc_add(dW, (part & 1) * 12288);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < kPart / 16; ++k)
#pragma unroll
                        for (int t = 0; t < 3; ++t)
                            umma_bf16(tD, desc_add(dk, k * kMnStep), desc_add(dw, t * 4096 + k * kMnStep), id_d,
                                      k + t > 0 || i > 0);
                    umma_commit(&w_free[part & 1]);
                    if (i == np - 1) {
                        umma_commit(&d_done);
                        umma_commit(&empty_kv[c & 1]);
                    }
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit(&drained[1]);
        __syncwarp();
        mbar_wait(&drained[1], 0);
    } else if (warp < 4) {
        if (OUT) regs_dec<64>();
        // nothing: the groups below start at a multiple of four warps (TMEM lane quarters)
    } else if (OUT && warp < kOutAt) {
        // ------------------------------------------------------------ scores
        // Thread: token row t = 32 quarter + lane; of the four 32-wide column blocks, 0 and 3
        // (half 0) or 1 and 2 (half 1), so that every warp has about the same share of the
        // causal triangle.
        const int quarter = warp & 3, half = (warp - 4) >> 2, t = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        int u = 0;
        for (int c = 0; c < nt; ++c) {
            const int np = parts_of(c);
            for (int r = 0; r < R; ++r, ++u) {
                const uint32_t tP = tbase + 128 * (u & 1) + lanes;
                wait_abort(&qk_done[u & 1], (u >> 1) & 1, abort_p);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int b = half ? 1 + e : 3 * e;          // block of source tokens 32 b ..
                    uint32_t p[16];
                    if (b >= np || b > quarter) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = 0;
                    } else {
                        uint32_t x[32];
                        tmem_ld32(tP + 32 * b, x);
                        tmem_wait_ld();
                        if (b < quarter) {
                            // lam^(t-s) = lam^(t - 32b - 31) lam^(31 - j): both exponents >= 0
                            const float rf = pw[t - 32 * b - 31];
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(rev + i);
                                const float2 lo = fmul2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                                        fmul2(make_float2(rf, rf), make_float2(f.x, f.y)));
                                const float2 hi = fmul2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                                        fmul2(make_float2(rf, rf), make_float2(f.z, f.w)));
                                p[i / 2] = pack_bf16(lo);
                                p[i / 2 + 1] = pack_bf16(hi);
                            }
                        } else {
                            // diagonal block: s > t is dropped whatever the score holds
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float y0 = i <= lane ? __uint_as_float(x[i]) * pw[lane - i] : 0.f;
                                const float y1 = i + 1 <= lane ? __uint_as_float(x[i + 1]) * pw[lane - i - 1] : 0.f;
                                p[i / 2] = pack_bf16(y0, y1);
                            }
                        }
                    }
                    tmem_st16(tP + 32 * b, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[u & 1]);
            }
        }
    } else if (OUT && warp < kWriteAt) {
        // ------------------------------------------------------------ outputs
        regs_inc<80>();
        // Thread: token row t, the CTA's 64 columns.
        const int quarter = warp & 3, t = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        const float wx = pw[t + 1] * a.scale;
        int u = 0;
        for (int c = 0; c < nt; ++c) {
            const bool st = c > 0 || has_init, live = t < len_of(c);
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.o) +
                               ((sg.start + (int64_t)c * kTcC + t) * a.H + g * R) * (int64_t)V + v0;
            for (int r = 0; r < R; ++r, ++u, p += V) {
                wait_abort(&o_done, u & 1, abort_p);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t x[16], h[16], l[16];
                    tmem_ld16(tOi + lanes + 16 * e, x);
                    if (st) {
                        tmem_ld16(tOx + lanes + 16 * e, h);
                        tmem_ld16(tOx + lanes + 64 + 16 * e, l);
                    }
                    tmem_wait_ld();
                    if (e == 3) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_free);
                    }
                    uint32_t out[8];
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        float2 y = make_float2(__uint_as_float(x[i]) * a.scale, __uint_as_float(x[i + 1]) * a.scale);
                        if (st) {
                            y.x = fmaf(wx, __uint_as_float(h[i]) + __uint_as_float(l[i]), y.x);
                            y.y = fmaf(wx, __uint_as_float(h[i + 1]) + __uint_as_float(l[i + 1]), y.y);
                        }
                        out[i / 2] = pack_bf16(y);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (live && 16 * e + 8 * i < nv)
                            reinterpret_cast<uint4*>(p)[2 * e + i] =
                                make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                }
            }
        }
    } else if (warp < kStateAt) {
        // ------------------------------------------------------------ w V
        if (OUT) regs_dec<56>();
        // Thread: token rows wt and wt + 16 of a part, 8 columns.
        const int wi = tid - 32 * kWriteAt, wt = wi >> 3, wc = wi & 7;
        int part = 0;                        // parts written so far
        for (int c = 0; c < nd; ++c) {
            const int np = parts_of(c), len = len_of(c);
            wait_abort(&full_kv[c & 1], (c >> 1) & 1, abort_p);
            for (int i = 0; i < np; ++i, ++part) {
                const int buf = part & 1;
                if (part >= 2) wait_abort(&w_free[buf], ((part >> 1) - 1) & 1, abort_p);
#pragma unroll
                for (int n2 = 0; n2 < 2; ++n2) {
                    const int row = wt + 16 * n2, s = i * kPart + row;
                    const uint32_t vt = smem_u32(sm + kOffV) + (c & 1) * 16384 + swz(s, wc);
                    const uint32_t dst = smem_u32(sm + kOffW) + buf * 12288 + swz(row, wc);
                    if (s < len) {
                        const uint4 x = ld_shared_v4(vt);
                        const float w = pw[len - 1 - s];
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                        uint32_t y[3][4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 z = fmul2(bf16x2_to_f2(xs[e]), make_float2(w, w));
#pragma unroll
                            for (int n = 0; n < 3; ++n) {
                                y[n][e] = pack_bf16(z);
                                z = fsub2(z, bf16x2_to_f2(y[n][e]));
                            }
                        }
#pragma unroll
                        for (int n = 0; n < 3; ++n) st_shared_v4(dst + n * 4096, y[n][0], y[n][1], y[n][2], y[n][3]);
                    } else {
                        // Rows past the sequence's end (another sequence's, or nothing): zero in
                        // w V, V and K, since 0 times what they hold need not be 0.
#pragma unroll
                        for (int n = 0; n < 3; ++n) st_shared_v4(dst + n * 4096, 0, 0, 0, 0);
                        st_shared_v4(vt, 0, 0, 0, 0);
                        for (int h = 0; h < halves; ++h)
                            st_shared_v4(smem_u32(sm + kOffK) + (c & 1) * 32768 + h * 16384 + swz(s, wc), 0, 0, 0, 0);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&w_ready[buf]);
            }
            if (OUT && partial && c == nt - 1 && lane == 0) mbar_arrive(&tail_ready);
        }
    } else {
        // ------------------------------------------------------------ the state
        if (OUT) regs_inc<80>();
        // Thread: state row k = 32 quarter + lane, 32 of the 64 V columns.
        const int quarter = warp & 3, half = (warp - kStateAt) >> 2, k = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        float S[32];
        // States in memory are [V][K]: this thread's column begins at base, lanes side by side
        // along K; rows past V (and lanes past K) hold zeros.
        const int base = 32 * half * K + k, rows = k < K ? max(0, min(32, nv - 32 * half)) : 0;
        float* slots = a.slots + (int64_t)sg.slot0 * per_state + head + base;
        // S = lam S + the column at p (S = the column with FIRST); eight loads at a time, since
        // all 32 with their addresses would not fit next to S.
        auto take = [&](const float* p, bool first) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i, p += K) x[i] = 8 * e + i < rows ? *p : 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    S[8 * e + i] = first ? x[i] : fmaf(lam_seg.x, S[8 * e + i], fmaf(lam_seg.y, S[8 * e + i], x[i]));
                __syncwarp();
            }
        };
        auto put = [&](float* p) {
#pragma unroll
            for (int i = 0; i < 32; ++i, p += K)
                if (i < rows) *p = S[i];
        };
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = 0.f;
        if (ip >= 0 && (OUT || sg.j == 0)) {
            const bool own = !OUT || sg.n == 1;                   // no other CTA replaces it meanwhile
            take(own ? a.init + ip * per_state + head + base : slots, true);
        }
        if (OUT) {
            for (int j = 1; j <= sg.j; ++j) take(slots + j * per_state, false);
        } else if (sg.j == 0 && ip >= 0) {
            put(slots);                      // the copy for the output pass
#pragma unroll
            for (int i = 0; i < 32; ++i) S[i] = 0.f;
        }
        auto hand_over = [&]() {             // S as the B operand of Q S: row k, a bf16 pair
            const uint32_t base = smem_u32(sm + kOffS);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = make_float2(S[8 * i + 2 * e], S[8 * i + 2 * e + 1]);
                    h[e] = pack_bf16(x);
                    l[e] = pack_bf16(fsub2(x, bf16x2_to_f2(h[e])));
                }
                const uint32_t o = base + swz(k, 4 * half + i);
                st_shared_v4(o, h[0], h[1], h[2], h[3]);
                st_shared_v4(o + 16384, l[0], l[1], l[2], l[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_ready);
        };
        if (has_init && nt > 0) hand_over();
        for (int c = 0; c < nd; ++c) {
            wait_abort(&d_done, c & 1, abort_p);
            tc_fence_after();
            const float2 lam = c == nt - 1 ? lam_tail : lam_full;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t d[8];
                tmem_ld8(tD + lanes + 32 * half + 8 * e, d);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x = __uint_as_float(d[i]);
                    S[8 * e + i] = fmaf(lam.x, S[8 * e + i], fmaf(lam.y, S[8 * e + i], x));
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&d_free);
            if (OUT && c + 1 < nt) {         // handed to the next chunk's Q S
                wait_abort(&qs_done, c & 1, abort_p);
                hand_over();
            }
        }
        // S after the segment's last chunk: the final state, or what the segment adds.
        if (!OUT) put(slots + (sg.j + 1) * per_state);
        else if (fp >= 0) put(a.fin + fp * per_state + head + base);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tbase, 512);
}

}  // namespace la
}  // namespace ssd
