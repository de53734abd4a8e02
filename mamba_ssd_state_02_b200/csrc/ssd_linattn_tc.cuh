// Linear attention prompts on the sm_100a tensor cores (bf16 q, k, v; any K and V that are
// multiples of 8 up to 128: the TMA boxes fill the missing columns with zeros).
//
// Two passes over the segments, both with one CTA per (segment, key/value head, 64 columns of
// V), walking the segment's 128-token chunks:
//
//   state pass: the FP32 state the segment adds, S' = lam^len S + K^T (w V) from S = 0, w_s =
//       lam^(len-1-s). w V goes to the tensor cores as three bf16 terms (2^-24 of it: the
//       final state is an FP32 output, and two terms would leave it at 2e-6 relative).
//   output pass: starts from the states of the segments before it, and per chunk
//       P  = (Q K^T) o lam^(t-s), s <= t        UMMA -> TMEM, warps scale and mask, bf16 -> TMEM
//       Oi = P V                                UMMA, A from TMEM
//       Ox = Q [S_hi | S_lo]                    UMMA, N = 128; S = S_hi + S_lo, a bf16 pair
//       o  = scale (Oi + lam^(t+1) (Ox_hi + Ox_lo))
//       S' = lam^128 S + K^T (w V)              UMMA, w V rounded to bf16; FP32 in registers
//     The CTA of a sequence's last segment also writes the final state, from the states of the
//     state pass alone.
//
// Roundings to bf16 in the output pass and why: the scores P and w V, each 2^-8 of a term, no
// more than the rounding of o itself (a running state that carried w V exactly would need the
// three terms here too: three times the MMAs and the conversions, which bound this pass); S as
// a pair, 2^-16, because a single bf16 would add a third rounding of that size to o.
//
// R query heads that share a key/value head are units (chunk, r) of the same CTA: K, V and
// the state are read and formed once for all of them. 64 columns of V per CTA: 128 would need
// single-buffered operands (227 KB of shared memory), and twice the CTAs fill the SMs of small
// batches; the price is Q K^T once per 64 columns.
#pragma once

#include "ssd_linattn.cuh"
#include "ssd_scan_tc.cuh"

namespace ssd {
namespace la {

constexpr int kTcC = 128;                    // tokens per chunk
constexpr int kTcV = 64;                     // V columns per CTA
constexpr int kBlock = 32;                   // columns of a score block
constexpr int kStateWarps = 8;

// Where a state column of a thread lies: element (v, k) of a [V][K] state at v * K + k; the
// thread has k fixed and up to 32 consecutive v, lanes side by side along K.
struct Column {
    int offset, rows, K;
    __device__ __forceinline__ Column(int k, int first_v, int nv, int K_)
        : offset(first_v * K_ + k), rows(k < K_ ? max(0, min(32, nv - first_v)) : 0), K(K_) {}
};

// S = x (FIRST), or lam S + x, for the column x at p. Eight loads at a time: all 32 with their
// addresses would not fit in registers next to S.
template <bool FIRST>
__device__ __forceinline__ void take(float (&S)[32], const Column& c, const float* p, float2 lam) {
    p += c.offset;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i, p += c.K) x[i] = 8 * e + i < c.rows ? *p : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& s = S[8 * e + i];
            s = FIRST ? x[i] : fmaf(lam.x, s, fmaf(lam.y, s, x[i]));
        }
        __syncwarp();
    }
}

// Row `r` (0..127), 16-byte chunk `c` of a [128][64] bf16 tile in the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int c) { return base + tc::swz(r, c); }

// ---------------------------------------------------------------------------------
// State pass. Warp 0 issues the TMA loads, warp 2 the UMMAs; eight warps write w V, eight hold
// the state. K, V, w V and D are double-buffered by chunk, and one barrier says that a chunk's
// UMMAs are done: its K, V and w V buffers are free and its D is ready. The three terms of w V
// lie side by side as one N = 192 operand, so K is read once for them (97 cycles a step; three
// N = 64 steps take 147, bound by the reads of their operands).
constexpr int kWriteWarps = 8;
constexpr int kStateThreads = 32 * (4 + kWriteWarps + kStateWarps);
constexpr int kStateV = 65536, kStateW = 98304;          // K at 0: 2 x 32 KB; V: 2 x 16 KB; w V: 2 x 48 KB
constexpr int kStateSmem = 196608 + 1024;

__global__ void __launch_bounds__(kStateThreads, 1)
k_la_tc_state(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const __grid_constant__ Args a) {
    using namespace tc;
    const int nvb = (a.V + kTcV - 1) / kTcV;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg(a, blockIdx.x / nvb / a.Hk, true, &sg)) return;
    const int K = a.K, v0 = vb * kTcV, nv = min(kTcV, a.V - v0), halves = (K + 63) / 64;
    const int nt = (sg.len + kTcC - 1) / kTcC;
    auto len_of = [&](int c) { return min(kTcC, sg.len - c * kTcC); };
    auto steps_of = [&](int c) { return (len_of(c) + 15) / 16; };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float pw[kTcC + 1];
    __shared__ float2 lam_full, lam_tail;
    __shared__ uint64_t full[2], done[2], w_ready[2], d_free[2], drained, stall_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float gd = a.log_decay[g];
    if (tid <= kTcC) pw[tid] = (float)pow_decay(gd, tid);
    if (tid == 160) lam_full = pow2f(gd, kTcC);
    if (tid == 192) lam_tail = pow2f(gd, nt > 0 ? len_of(nt - 1) : 0);
    if (tid == 0) {
        check_decay(gd);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&done[i], 1);
            mbar_init(&w_ready[i], kWriteWarps);
            mbar_init(&d_free[i], kStateWarps);
        }
        mbar_init(&drained, 1);
        mbar_init(&stall_bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tD = tmem_slot;           // 192 columns at 0 and at 256
    volatile int* abort_p = &abort_flag;
    const int64_t per_state = (int64_t)a.Hk * a.V * K, head = ((int64_t)g * a.V + v0) * K;

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        if (lane == 0 && nt > 0) {
            prefetch_tmap(&map_k);
            prefetch_tmap(&map_v);
            int n = 0;
#pragma unroll 1
            for (int c = 0; c < nt; ++c) {
                const int b = c & 1, t0 = (int)(sg.start + (int64_t)c * kTcC);
                if (c + 1 < nt) {            // the next chunk into L2 meanwhile
#pragma unroll 1
                    for (int h = 0; h < halves; ++h) tma_prefetch_3d(&map_k, 64 * h, g, t0 + kTcC);
                    tma_prefetch_3d(&map_v, v0, g, t0 + kTcC);
                }
                if (c >= 2 && !wait_issue(&done[b], ((c >> 1) - 1) & 1, abort_p)) break;
                mbar_arrive_expect_tx(&full[b], (halves + 1) * 16384);
#pragma unroll 1
                for (int h = 0; h < halves; ++h) tma_load_3d(sm + b * 32768 + h * 16384, &map_k, &full[b], 64 * h, g, t0);
                tma_load_3d(sm + kStateV + b * 16384, &map_v, &full[b], v0, g, t0);
                ++n;
            }
            // The last phase issued on each barrier completes once its bytes have landed (a
            // phase is issued only after the previous one has been consumed).
            for (int i = 0; i < 2; ++i)
                if (n > i) mbar_wait(&full[i], ((n - 1 - i) >> 1) & 1);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ UMMA issuer
        // D (k x [v hi | v mid | v lo]) = K^T (w V): A = K, MN-major; B = w V, MN-major.
        const uint32_t id = idesc_bf16(128, 192, 1, 1);
        const uint64_t dK = smem_desc(smem_u32(sm), 16384, 1024), dW = smem_desc(smem_u32(sm + kStateW), 16384, 1024);
        bool ok = !(a.stall && !wait_issue_warp(&stall_bar, 0, abort_p));     // test hook: a wait that runs out
#pragma unroll 1
        for (int c = 0; c < nt && ok; ++c) {
            const int b = c & 1, ph = (c >> 1) & 1;
            if (!wait_issue_warp(&full[b], ph, abort_p) || !wait_issue_warp(&w_ready[b], ph, abort_p) ||
                (c >= 2 && !wait_issue_warp(&d_free[b], ph ^ 1, abort_p)))
                break;
            tc_fence_after();
            const uint64_t dk = desc_add(dK, b * 32768), dw = desc_add(dW, b * 49152);
            const uint32_t d = tD + 256 * b;
            const int steps = steps_of(c);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < steps) umma_bf16(d, desc_add(dk, k * kMnStep), desc_add(dw, k * kMnStep), id, k > 0);
                umma_commit(&done[b]);
            }
            __syncwarp();
        }
        // Every MMA issued above has completed once this commit arrives.
        if (elect_one()) umma_commit(&drained);
        __syncwarp();
        mbar_wait(&drained, 0);
    } else if (warp < 4) {
        // nothing: the groups below start at a multiple of four warps (TMEM lane quarters)
    } else if (warp < 4 + kWriteWarps) {
        // ------------------------------------------------------------ w V
        // Thread: token rows wt + 32 i of a chunk, 8 columns.
        const int wi = tid - 128, wt = wi >> 3, wc = wi & 7;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int b = c & 1, len = len_of(c), rows = 16 * steps_of(c);
            wait_abort(&full[b], (c >> 1) & 1, abort_p);
            if (c >= 2) wait_abort(&done[b], ((c >> 1) - 1) & 1, abort_p);
            const uint32_t sv = smem_u32(sm + kStateV) + b * 16384, sw = smem_u32(sm + kStateW) + b * 49152;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int s = wt + 32 * i;
                if (s >= rows) break;
                uint32_t y[3][4];
                if (s < len) {
                    const uint4 x = ld_shared_v4(tile_at(sv, s, wc));
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                    const float w = pw[len - 1 - s];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float2 z = fmul2(bf16x2_to_f2(xs[e]), make_float2(w, w));
#pragma unroll
                        for (int n = 0; n < 3; ++n) {
                            y[n][e] = pack_bf16(z);
                            z = fsub2(z, bf16x2_to_f2(y[n][e]));
                        }
                    }
                } else {
                    // Rows past the sequence's end (another sequence's, or nothing): zero in w V
                    // and in K, since 0 times what K holds there need not be 0.
#pragma unroll
                    for (int n = 0; n < 3; ++n) y[n][0] = y[n][1] = y[n][2] = y[n][3] = 0;
#pragma unroll 1
                    for (int h = 0; h < halves; ++h)
                        st_shared_v4(tile_at(smem_u32(sm) + b * 32768 + h * 16384, s, wc), 0, 0, 0, 0);
                }
#pragma unroll
                for (int n = 0; n < 3; ++n) st_shared_v4(tile_at(sw + n * 16384, s, wc), y[n][0], y[n][1], y[n][2], y[n][3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_ready[b]);
        }
    } else {
        // ------------------------------------------------------------ the state
        // Thread: state row k = 32 quarter + lane, 32 of the 64 V columns.
        const int quarter = warp & 3, half = (warp - 4 - kWriteWarps) >> 2;
        const Column col(32 * quarter + lane, 32 * half, nv, K);
        float* slots = a.slots + (int64_t)sg.slot0 * per_state + head;
        float S[32];
        if (sg.j == 0 && a.init) {
            // The output pass starts from a copy: the final state may replace the initial one.
            const int64_t ip = page_of(a.init_pages, a.npages, sg.seq);
            if (ip >= 0) {
                take<true>(S, col, a.init + ip * per_state + head, make_float2(0.f, 0.f));
                float* p = slots + col.offset;
#pragma unroll
                for (int i = 0; i < 32; ++i, p += K)
                    if (i < col.rows) *p = S[i];
            }
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = 0.f;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int b = c & 1;
            wait_abort(&done[b], (c >> 1) & 1, abort_p);
            tc_fence_after();
            const uint32_t t = tD + 256 * b + ((uint32_t)quarter << 21) + 32 * half;
            const float2 lam = c == nt - 1 ? lam_tail : lam_full;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t d[3][16];
#pragma unroll
                for (int n = 0; n < 3; ++n) tmem_ld16(t + 64 * n + 16 * e, d[n]);
                tmem_wait_ld();
                if (e == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&d_free[b]);
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float& s = S[16 * e + i];
                    const float x = __uint_as_float(d[0][i]) + (__uint_as_float(d[1][i]) + __uint_as_float(d[2][i]));
                    s = fmaf(lam.x, s, fmaf(lam.y, s, x));
                }
            }
        }
        float* p = slots + (int64_t)(sg.j + 1) * per_state + col.offset;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += K)
            if (i < col.rows) *p = S[i];
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tD, 512);
}

// ---------------------------------------------------------------------------------
// Output pass. Warp 0 issues the TMA loads, warp 1 the UMMAs of P, Oi and Ox, warp 2 those of
// the state (an issuing warp takes its batches in order, and the state's waits would hold up
// the outputs'); then three groups of eight warps: scores, outputs, and w V with the state.
// Q, K and V are double-buffered, and what they have no room for yet is brought into L2.
//
// Shared memory: K, V, Q (two buffers each), S (a bf16 pair), w V. TMEM columns: Q K^T [0, 128)
// and [128, 256) (units alternate), P of a 32-token block in the first 16 columns of the
// block's scores (read and written by the same thread), Oi [256, 320), Ox [320, 448), D
// [448, 512).

// Registers of the calling group of four warps, all of which execute it.
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

constexpr int kScoreWarps = 8, kOutWarps = 8;
constexpr int kOutThreads = 32 * (4 + kScoreWarps + kOutWarps + kStateWarps);
constexpr int kOutV = 65536, kOutQ = 98304, kOutS = 163840, kOutW = 196608;      // K at 0
constexpr int kOutSmem = 212992 + 1024;

__global__ void __launch_bounds__(kOutThreads, 1)
k_la_tc_out(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ Args a) {
    using namespace tc;
    const int nvb = (a.V + kTcV - 1) / kTcV;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg(a, blockIdx.x / nvb / a.Hk, true, &sg)) return;
    const int K = a.K, R = a.R, v0 = vb * kTcV, nv = min(kTcV, a.V - v0);
    const int nt = (sg.len + kTcC - 1) / kTcC, ksteps = (K + 15) / 16, halves = (K + 63) / 64;
    const bool partial = sg.len % kTcC != 0;                      // the last chunk
    auto len_of = [&](int c) { return min(kTcC, sg.len - c * kTcC); };
    auto blocks_of = [&](int c) { return (len_of(c) + kBlock - 1) / kBlock; };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float pw_pad[32 + kTcC + 1];  // 32 zeros, then lam^0 .. lam^128
    __shared__ __align__(16) float rev[32];  // lam^31 .. lam^0
    __shared__ float2 lam_full, lam_seg, lam_len;
    __shared__ uint64_t full_k[2], empty_k[2], full_v[2], empty_v[2], full_q[2], empty_q[2], qk_done[2], p_ready[2],
        o_done, o_free, qs_done, w_ready, d_done, s_ready, tail_ready, drained[2], stall_bar;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    const float* pw = pw_pad + 32;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float gd = a.log_decay[g];
    if (tid < 32 + kTcC + 1) pw_pad[tid] = tid < 32 ? 0.f : (float)pow_decay(gd, tid - 32);
    if (tid >= 192 && tid < 224) rev[tid - 192] = (float)pow_decay(gd, 31 - (tid - 192));
    if (tid == 256) lam_full = pow2f(gd, kTcC);
    if (tid == 288) lam_seg = pow2f(gd, a.Ls);
    if (tid == 320) lam_len = pow2f(gd, sg.len);
    if (tid == 0) {
        check_decay(gd);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&full_k[i], 1);
            mbar_init(&empty_k[i], 2);
            mbar_init(&full_v[i], 1);
            mbar_init(&empty_v[i], 2);
            mbar_init(&full_q[i], 1);
            mbar_init(&empty_q[i], 1);
            mbar_init(&qk_done[i], 1);
            mbar_init(&p_ready[i], kScoreWarps);
            mbar_init(&drained[i], 1);
        }
        mbar_init(&o_done, 1);
        mbar_init(&o_free, kOutWarps);
        mbar_init(&qs_done, 1);
        mbar_init(&w_ready, kStateWarps);
        mbar_init(&d_done, 1);
        mbar_init(&s_ready, kStateWarps);
        mbar_init(&tail_ready, kStateWarps);
        mbar_init(&stall_bar, 1);
        abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    const int64_t per_state = (int64_t)a.Hk * a.V * K, head = ((int64_t)g * a.V + v0) * K;
    const int64_t ip = a.init ? page_of(a.init_pages, a.npages, sg.seq) : -1;
    int64_t fp = -1;
    if (a.fin && sg.j + 1 == sg.n) {
        fp = page_of(a.fin_pages, a.npages, sg.seq);
        if (a.fin_pages && fp >= 0 && page_clash(a, sg.seq, fp, kOutThreads)) {
            latch_error(SSD_ERR_INVALID_ARG);
            fp = -1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = tmem_slot, tOi = tbase + 256, tOx = tbase + 320, tD = tbase + 448;
    volatile int* abort_p = &abort_flag;
    const bool has_init = ip >= 0 || sg.j > 0;                    // the first chunk meets a state

    // Registers: 72 a thread at launch (896 threads), moved between groups of four warps:
    // 56 + 2 * 72 + 2 * 72 + 2 * 80 = 7 * 72.
    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        regs_dec<56>();
        if (lane == 0 && nt > 0) {
            prefetch_tmap(&map_k);
            prefetch_tmap(&map_v);
            prefetch_tmap(&map_q);
            int nk = 0, nl = 0, nq = 0;      // loads of K, V and Q issued (alternating buffers)
            auto row = [&](int c) { return (int)(sg.start + (int64_t)c * kTcC); };
            auto load_q = [&](int c, int r) -> bool {
                const int u = c * R + r, b = u & 1;
                if (u >= 2 && !wait_issue(&empty_q[b], ((u >> 1) - 1) & 1, abort_p)) return false;
                mbar_arrive_expect_tx(&full_q[b], halves * 16384);
#pragma unroll 1
                for (int h = 0; h < halves; ++h)
                    tma_load_3d(sm + kOutQ + b * 32768 + h * 16384, &map_q, &full_q[b], 64 * h, g * R + r, row(c));
                ++nq;
                const int r2 = (r + 2) % R, c2 = c + (r + 2) / R;             // two units on, into L2
                if (c2 < nt)
#pragma unroll 1
                    for (int h = 0; h < halves; ++h) tma_prefetch_3d(&map_q, 64 * h, g * R + r2, row(c2));
                return true;
            };
            bool ok = true;
#pragma unroll 1
            for (int c = 0; c < nt && ok; ++c) {
                const int b = c & 1;
                if (c >= 2 && !wait_issue(&empty_k[b], ((c >> 1) - 1) & 1, abort_p)) break;
                mbar_arrive_expect_tx(&full_k[b], halves * 16384);
#pragma unroll 1
                for (int h = 0; h < halves; ++h)
                    tma_load_3d(sm + b * 32768 + h * 16384, &map_k, &full_k[b], 64 * h, g, row(c));
                ++nk;
                if (!load_q(c, 0)) break;
                if (c >= 2 && !wait_issue(&empty_v[b], ((c >> 1) - 1) & 1, abort_p)) break;
                mbar_arrive_expect_tx(&full_v[b], 16384);
                tma_load_3d(sm + kOutV + b * 16384, &map_v, &full_v[b], v0, g, row(c));
                ++nl;
                if (c + 2 < nt) {            // two chunks on, into L2
#pragma unroll 1
                    for (int h = 0; h < halves; ++h) tma_prefetch_3d(&map_k, 64 * h, g, row(c + 2));
                    tma_prefetch_3d(&map_v, v0, g, row(c + 2));
                }
#pragma unroll 1
                for (int r = 1; r < R && ok; ++r) ok = load_q(c, r);
            }
            // As in the state pass: wait for what is in flight.
            for (int i = 0; i < 2; ++i) {
                if (nk > i) mbar_wait(&full_k[i], ((nk - 1 - i) >> 1) & 1);
                if (nl > i) mbar_wait(&full_v[i], ((nl - 1 - i) >> 1) & 1);
                if (nq > i) mbar_wait(&full_q[i], ((nq - 1 - i) >> 1) & 1);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ UMMA issuer: P, Oi, Ox
        regs_dec<56>();
        const uint32_t id_x = idesc_bf16(128, 128, 0, 1), id_v = idesc_bf16(128, 64, 0, 1);
        const uint64_t dQ = smem_desc(smem_u32(sm + kOutQ), 16, 1024), dK = smem_desc(smem_u32(sm), 16, 1024);
        const uint64_t dV = smem_desc(smem_u32(sm + kOutV), 16384, 1024), dS = smem_desc(smem_u32(sm + kOutS), 16384, 1024);
        // Q K^T of unit u = (c, r): N = the chunk's tokens rounded up to a block.
        auto issue_qk = [&](int c, int r, int u) -> bool {
            if (r == 0 && !wait_issue_warp(&full_k[c & 1], (c >> 1) & 1, abort_p)) return false;
            if (!wait_issue_warp(&full_q[u & 1], (u >> 1) & 1, abort_p)) return false;
            tc_fence_after();
            const uint32_t id = idesc_bf16(128, kBlock * blocks_of(c), 0, 0), d = tbase + 128 * (u & 1);
            const uint64_t dq = desc_add(dQ, (u & 1) * 32768), dk = desc_add(dK, (c & 1) * 32768);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (k < ksteps)
                        umma_bf16(d, desc_add(dq, kmajor_step(128, k)), desc_add(dk, kmajor_step(128, k)), id, k > 0);
                umma_commit(&qk_done[u & 1]);
                if (r == R - 1) umma_commit(&empty_k[c & 1]);
            }
            __syncwarp();
            return true;
        };
        // test hook (stall): a wait that runs out
        bool ok = nt > 0 && !(a.stall && !wait_issue_warp(&stall_bar, 0, abort_p)) && issue_qk(0, 0, 0);
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt && ok; ++c) {
            const bool st = c > 0 || has_init;
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                ok = (u == 0 || wait_issue_warp(&o_free, (u - 1) & 1, abort_p)) &&
                     (!st || r > 0 || wait_issue_warp(&s_ready, (has_init ? c : c - 1) & 1, abort_p));
                if (!ok) break;
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
                // The buffer of the next Q K^T last held P of unit u-1, whose product is done
                // (o_free above). V's rows past the last token hold zeros (tail_ready).
                const int cn = r == R - 1 ? c + 1 : c, rn = r == R - 1 ? 0 : r + 1;
                ok = (cn == nt || issue_qk(cn, rn, u + 1)) && wait_issue_warp(&full_v[c & 1], (c >> 1) & 1, abort_p) &&
                     wait_issue_warp(&p_ready[u & 1], (u >> 1) & 1, abort_p) &&
                     (!partial || c < nt - 1 || r > 0 || wait_issue_warp(&tail_ready, 0, abort_p));
                if (!ok) break;
                tc_fence_after();
                const int steps = blocks_of(c) * (kBlock / 16);
                const uint32_t tP = tbase + 128 * (u & 1);
                const uint64_t dv = desc_add(dV, (c & 1) * 16384);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (k < steps) umma_bf16_ts(tOi, tP + 32 * (k >> 1) + 8 * (k & 1), desc_add(dv, k * kMnStep), id_v, k > 0);
                    umma_commit(&o_done);
                    if (r == R - 1) umma_commit(&empty_v[c & 1]);
                }
                __syncwarp();
            }
        }
        // Every MMA issued above has completed once this commit arrives.
        if (elect_one()) umma_commit(&drained[0]);
        __syncwarp();
        mbar_wait(&drained[0], 0);
    } else if (warp == 2) {
        // ------------------------------------------------------------ UMMA issuer: the state
        regs_dec<56>();
        // D = K^T (w V), for every chunk that another one follows (all of them full).
        const uint32_t id = idesc_bf16(128, 64, 1, 1);
        const uint64_t dK = smem_desc(smem_u32(sm), 16384, 1024), dW = smem_desc(smem_u32(sm + kOutW), 16384, 1024);
#pragma unroll 1
        for (int c = 0; c + 1 < nt; ++c) {
            // w_ready also says that the last D has been read
            if (!wait_issue_warp(&full_k[c & 1], (c >> 1) & 1, abort_p) || !wait_issue_warp(&w_ready, c & 1, abort_p)) break;
            tc_fence_after();
            const uint64_t dk = desc_add(dK, (c & 1) * 32768);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 8; ++k) umma_bf16(tD, desc_add(dk, k * kMnStep), desc_add(dW, k * kMnStep), id, k > 0);
                umma_commit(&d_done);
                umma_commit(&empty_k[c & 1]);
                umma_commit(&empty_v[c & 1]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(&drained[1]);
        __syncwarp();
        mbar_wait(&drained[1], 0);
    } else if (warp < 4) {
        regs_dec<56>();
        // nothing: the groups below start at a multiple of four warps (TMEM lane quarters)
    } else if (warp < 4 + kScoreWarps) {
        // ------------------------------------------------------------ scores
        // Thread: token row t = 32 quarter + lane; of the four 32-wide column blocks, 0 and 3
        // (half 0) or 1 and 2 (half 1), so that every warp has about the same share of the
        // causal triangle.
        const int quarter = warp & 3, half = (warp - 4) >> 2, t = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int nb = blocks_of(c);
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                const uint32_t tP = tbase + 128 * (u & 1) + lanes;
                wait_abort(&qk_done[u & 1], (u >> 1) & 1, abort_p);
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    const int b = half ? 1 + e : 3 * e;          // block of source tokens 32 b ..
                    uint32_t p[16];
                    if (b >= nb || b > quarter) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) p[i] = 0;
                    } else {
                        uint32_t x[32];
                        tmem_ld32(tP + 32 * b, x);
                        tmem_wait_ld();
                        if (b < quarter) {
                            // lam^(t-s) = lam^(t - 32b - 31) lam^(31 - j): both exponents >= 0
                            const float rf = pw[t - 32 * b - 31];
                            const float2 rf2 = make_float2(rf, rf);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(rev + i);
                                const float2 lo = fmul2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                                        fmul2(rf2, make_float2(f.x, f.y)));
                                const float2 hi = fmul2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                                        fmul2(rf2, make_float2(f.z, f.w)));
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
    } else if (warp < 4 + kScoreWarps + kOutWarps) {
        // ------------------------------------------------------------ outputs
        // Thread: token row t, 32 of the 64 columns.
        const int quarter = warp & 3, half = (warp - 4 - kScoreWarps) >> 2, t = 32 * quarter + lane;
        const uint32_t lanes = ((uint32_t)quarter << 21) + 32 * half;
        const float wx = pw[t + 1] * a.scale;
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const bool st = c > 0 || has_init;
            const int cols = t < len_of(c) ? nv - 32 * half : 0;
            __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.o) +
                               ((sg.start + (int64_t)c * kTcC + t) * a.H + g * R) * (int64_t)a.V + v0 + 32 * half;
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u, p += a.V) {
                wait_abort(&o_done, u & 1, abort_p);
                tc_fence_after();
#pragma unroll 1
                for (int e = 0; e < 2; ++e) {
                    uint32_t out[8], x[16], h[16], l[16];
                    tmem_ld16(tOi + lanes + 16 * e, x);
                    if (st) {
                        tmem_ld16(tOx + lanes + 16 * e, h);
                        tmem_ld16(tOx + lanes + 64 + 16 * e, l);
                    }
                    tmem_wait_ld();
                    if (e == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&o_free);
                    }
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
                        if (16 * e + 8 * i < cols)
                            reinterpret_cast<uint4*>(p)[2 * e + i] =
                                make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ w V and the state
        regs_inc<80>();
        // Thread: state row k = 32 quarter + lane, 32 of the 64 V columns; as a writer of w V:
        // token rows wt + 32 i, 8 columns.
        const int quarter = warp & 3, half = (warp - 4 - kScoreWarps - kOutWarps) >> 2, k = 32 * quarter + lane;
        const int wi = tid - 32 * (4 + kScoreWarps + kOutWarps), wt = wi >> 3, wc = wi & 7;
        float S[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) S[i] = 0.f;
        {
            // The state entering the segment, and the final state after the last one.
            const Column col(k, 32 * half, nv, K);
            const float* slots = a.slots + (int64_t)sg.slot0 * per_state + head;
            if (ip >= 0) take<true>(S, col, a.two_pass ? slots : a.init + ip * per_state + head, make_float2(0.f, 0.f));
#pragma unroll 1
            for (int j = 1; j <= sg.j; ++j) take<false>(S, col, slots + j * per_state, lam_seg);
            if (fp >= 0) {
                const float* add = slots + (int64_t)(sg.j + 1) * per_state + col.offset;
                float* to = a.fin + fp * per_state + head + col.offset;
#pragma unroll
                for (int i = 0; i < 32; ++i, add += K, to += K)
                    if (i < col.rows) *to = fmaf(lam_len.x, S[i], fmaf(lam_len.y, S[i], *add));
            }
        }
        auto write_w = [&](int c) {          // w V of a full chunk
            wait_abort(&full_v[c & 1], (c >> 1) & 1, abort_p);
            const uint32_t sv = smem_u32(sm + kOutV) + (c & 1) * 16384, sw = smem_u32(sm + kOutW);
#pragma unroll 2
            for (int i = 0; i < 4; ++i) {
                const int s = wt + 32 * i;
                const float w = pw[kTcC - 1 - s];
                const uint4 x = ld_shared_v4(tile_at(sv, s, wc));
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = pack_bf16(fmul2(bf16x2_to_f2(xs[e]), make_float2(w, w)));
                st_shared_v4(tile_at(sw, s, wc), y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&w_ready);
        };
        auto hand_over = [&]() {             // S as the B operand of Q S: row k, a bf16 pair
            const uint32_t base = smem_u32(sm + kOutS);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 x = make_float2(S[8 * i + 2 * e], S[8 * i + 2 * e + 1]);
                    h[e] = pack_bf16(x);
                    l[e] = pack_bf16(fsub2(x, bf16x2_to_f2(h[e])));
                }
                st_shared_v4(tile_at(base, k, 4 * half + i), h[0], h[1], h[2], h[3]);
                st_shared_v4(tile_at(base + 16384, k, 4 * half + i), l[0], l[1], l[2], l[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_ready);
        };
        if (has_init && nt > 0) hand_over();
        if (nt > 1) write_w(0);
#pragma unroll 1
        for (int c = 0; c + 1 < nt; ++c) {
            wait_abort(&d_done, c & 1, abort_p);
            tc_fence_after();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t d[16];
                tmem_ld16(tD + ((uint32_t)quarter << 21) + 32 * half + 16 * e, d);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float& s = S[16 * e + i];
                    s = fmaf(lam_full.x, s, fmaf(lam_full.y, s, __uint_as_float(d[i])));
                }
            }
            tc_fence_before();
            wait_abort(&qs_done, c & 1, abort_p);
            hand_over();
            if (c + 2 < nt) write_w(c + 1);
        }
        if (partial) {
            // Rows past the sequence's end (another sequence's, or nothing) are zeroed in V,
            // since a score of 0 times what they hold need not be 0.
            const int c = nt - 1, len = len_of(c), rows = kBlock * blocks_of(c);
            wait_abort(&full_v[c & 1], (c >> 1) & 1, abort_p);
            for (int s = len + wt; s < rows; s += 32)
                st_shared_v4(tile_at(smem_u32(sm + kOutV) + (c & 1) * 16384, s, wc), 0, 0, 0, 0);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail_ready);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tbase, 512);
}

}  // namespace la
}  // namespace ssd
