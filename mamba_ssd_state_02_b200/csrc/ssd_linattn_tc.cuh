// Linear attention prompts on the sm_100a tensor cores (bf16 q, k, v; any K and V that are
// multiples of 8 up to 128: the TMA boxes fill the missing columns with zeros).
//
// Two passes over the segments, both with one CTA per (segment, key/value head, 64 columns of
// V), walking the segment's 128-token chunks:
//
//   state pass: the FP32 state the segment adds, S' = lam^len S + K^T (w V) from S = 0, w_s =
//       lam^(len-1-s). w V goes to the tensor cores as three bf16 terms (2^-24 of it: the
//       final state is an FP32 output, and two terms would leave it at 2e-6 relative).
//   output pass: starts from the state entering the segment (the passing kernel in between
//       makes it from what the segments before add), and per chunk
//       P  = (Q K^T) o lam^(t-s), s <= t        UMMA -> TMEM, warps scale and mask, bf16 -> TMEM
//       Oi = P V                                UMMA, A from TMEM
//       Ox = Q [S_hi | S_lo]                    UMMA, N = 128; S = S_hi + S_lo, a bf16 pair
//       o  = Oi + scale lam^(t+1) (Ox_hi + Ox_lo)       (P carries scale)
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

// Bounded waits, as wait_abort and wait_issue of the scan's passes (an expired wait latches
// SSD_ERR_TIMEOUT and raises the CTA's abort flag, after which every wait returns; the issuing
// warps look at the flag after their waits and stop), but short: the passes have two dozen
// waits in loops that ten kinds of warps run at once, and once their code outgrows the
// instruction cache every one of them runs at the speed of its misses (at 107 KB of code the
// output pass took 1.3 times as long as at 40 KB). A try that fails blocks for about 4 us
// (measured), so the tries add up to about 2 s.
constexpr uint32_t kWaitTries = 1u << 19;

__device__ __forceinline__ void wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
    for (uint32_t n = 0; !tc::mbar_try_wait_sleep(bar, parity & 1) && !*abort_flag; ++n)
        if (n == kWaitTries) {
            latch_error(SSD_ERR_TIMEOUT);
            *abort_flag = 1;
        }
}

// The barrier at the start of a block: every warp has set up its part (barriers, tables, TMEM).
// Warp 0 made the barriers itself and needs nothing else, so that its first loads are on their
// way while the others still compute tables.
__device__ __forceinline__ void start_block(int warp, int threads) {
    tc::tc_fence_before();
    if (warp == 0) {
        __syncwarp();
        asm volatile("bar.arrive 15, %0;" ::"r"(threads) : "memory");
    } else {
        tc::named_barrier(15, threads);
    }
    tc::tc_fence_after();
}

// For an issuing warp, after its waits: none of them was given up.
__device__ __forceinline__ bool go_on(volatile int* abort_flag) { return __all_sync(0xffffffffu, *abort_flag == 0); }

__device__ __forceinline__ float2 fadd2(float2 x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
        "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return d;
}

// Row `r` (0..127), 16-byte chunk `c` of a [128][64] bf16 tile in the 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int r, int c) { return base + tc::swz(r, c); }

// ---------------------------------------------------------------------------------
// A matrix descriptor's low word: start address, and the distance between 64-wide blocks of an
// MN-major operand (not read for K-major ones). The high word is the same for all. In
// units of 16 bytes, a K-step of 16 advances a K-major operand by 2, the other half of its
// columns lies 1024 on, and a K-step of an MN-major operand is 128.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t block = 16384) {
    return (saddr >> 4) | (block >> 4) << 16;
}
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;          // SBO, version, 128-byte swizzle

__device__ __forceinline__ void umma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    const uint64_t hi = (uint64_t)kDescHi << 32;
    tc::umma_bf16(d, hi | a_lo, hi | b_lo, idesc, accumulate);
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate) {
    tc::umma_bf16_ts(d, a_tmem, (uint64_t)kDescHi << 32 | b_lo, idesc, accumulate);
}

// ---------------------------------------------------------------------------------
// State pass. Warp 0 issues the TMA loads, warp 2 the UMMAs; eight warps write w V, eight hold
// the state. K and V are triple-buffered; w V goes through two buffers of 64 tokens, so
// that one is written while the UMMAs read the other; D is double-buffered. The three terms of
// w V lie side by side as one N = 192 operand, so K is read once for them (97 cycles a step;
// three N = 64 steps take 147, bound by the reads of their operands). 4 x 4096 tokens, 32 heads of
// 128 x 128: 95 us (268 MB of k and v: 2.8 TB/s); tensor pipe 31%, DRAM 35%: bound by the chain
// V -> w V -> D -> state.
constexpr int kWriteWarps = 8;
constexpr int kHalf = 64;                    // tokens of a w V buffer
constexpr int kStateThreads = 32 * (4 + kWriteWarps + kStateWarps);
constexpr int kStateV = 98304, kStateW = 147456;         // K at 0: 3 x 32 KB; V: 3 x 16 KB; w V: 2 x 24 KB
constexpr int kStateSmem = 196608 + 1024;

__global__ void __launch_bounds__(kStateThreads, 1)
k_la_tc_state(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
              const __grid_constant__ Args a) {
    using namespace tc;
    const int nvb = (a.V + kTcV - 1) / kTcV;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg(a, blockIdx.x / nvb / a.Hk, true, &sg)) return;
    const int K = a.K, v0 = vb * kTcV, nv = min(kTcV, a.V - v0), tiles = (K + 63) / 64;
    const int nt = (sg.len + kTcC - 1) / kTcC, nh = (sg.len + kHalf - 1) / kHalf;

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float pw[kTcC + 1];
    __shared__ float2 lam_full, lam_tail;
    // FULL, FREE: K and V of a chunk; W_*: w V of a half; D_*: D of a chunk
    enum { FULL = 0, FREE = 3, W_READY = 6, W_FREE = 8, D_DONE = 10, D_FREE = 12, DRAINED = 14, STALL, BARS };
    __shared__ uint64_t bars[BARS];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float gd = a.log_decay[g];
    const int tt = tid - 64;                 // warps 0 and 1 have other things to set up
    if (tt >= 0 && tt <= kTcC) pw[tt] = (float)pow_decay(gd, tt);
    if (tid == 256) lam_full = pow2f(gd, kTcC);
    if (tid == 288) lam_tail = pow2f(gd, nt > 0 ? sg.len - (nt - 1) * kTcC : 0);
    if (tid < BARS) {
        const int pair = tid & ~1;
        mbar_init(&bars[tid], pair == W_READY ? kWriteWarps : pair == D_FREE ? kStateWarps : 1);
    }
    if (tid == 0) {
        check_decay(gd);
        abort_flag = 0;
    }
    fence_barrier_init();
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    start_block(warp, kStateThreads);
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
            for (int c = 0, b = 0, ph = 0; c < nt; ++c) {
                const int t0 = (int)(sg.start + (int64_t)c * kTcC);
                if (c >= 3) wait_bar(&bars[FREE + b], ph - 1, abort_p);
                if (*abort_p) break;
                mbar_arrive_expect_tx(&bars[FULL + b], (tiles + 1) * 16384);
#pragma unroll 1
                for (int t = 0; t < tiles; ++t) tma_load_3d(sm + b * 32768 + t * 16384, &map_k, &bars[FULL + b], 64 * t, g, t0);
                tma_load_3d(sm + kStateV + b * 16384, &map_v, &bars[FULL + b], v0, g, t0);
                ++n;
                if (++b == 3) {
                    b = 0;
                    ++ph;
                }
            }
            // The last phase issued on each barrier completes once its bytes have landed (a
            // phase is issued only after the previous one has been consumed).
            for (int b = 0; b < 3; ++b)
                if (n > b) mbar_wait(&bars[FULL + b], ((n - 1 - b) / 3) & 1);
        }
    } else if (warp == 2) {
        // ------------------------------------------------------------ UMMA issuer
        // D (k x [v hi | v mid | v lo]) = K^T (w V): A = K, MN-major; B = w V, MN-major.
        const uint32_t id = idesc_bf16(128, 192, 1, 1);
        const uint32_t dK = desc_lo(smem_u32(sm)), dW = desc_lo(smem_u32(sm + kStateW), 8192);
        if (a.stall) wait_bar(&bars[STALL], 0, abort_p);          // test hook: a wait that runs out
        bool ok = true;
#pragma unroll 1
        for (int c = 0, b = 0, ph = 0, h = 0; c < nt && ok; ++c) {
            wait_bar(&bars[FULL + b], ph, abort_p);
            if (c >= 2) wait_bar(&bars[D_FREE + (c & 1)], (c >> 1) - 1, abort_p);
            const uint32_t d = tD + 256 * (c & 1);
#pragma unroll 1
            for (int i = 0; i < 2 && h < nh; ++i, ++h) {
                wait_bar(&bars[W_READY + (h & 1)], h >> 1, abort_p);
                if (!(ok = go_on(abort_p))) break;
                tc_fence_after();
                const uint32_t dk = dK + b * 2048 + i * 512, dw = dW + (h & 1) * 1536;
                const int steps = min(4, (sg.len - h * kHalf + 15) / 16);
                if (elect_one()) {
#pragma unroll 1
                    for (int k = 0; k < steps; ++k) umma(d, dk + k * 128, dw + k * 128, id, i + k > 0);
                    umma_commit(&bars[W_FREE + (h & 1)]);
                    if (i == 1 || h + 1 == nh) {
                        umma_commit(&bars[D_DONE + (c & 1)]);
                        umma_commit(&bars[FREE + b]);
                    }
                }
                __syncwarp();
            }
            if (++b == 3) {
                b = 0;
                ++ph;
            }
        }
        // Every MMA issued above has completed once this commit arrives.
        if (elect_one()) umma_commit(&bars[DRAINED]);
        __syncwarp();
        mbar_wait(&bars[DRAINED], 0);
    } else if (warp < 4) {
        // nothing: the groups below start at a multiple of four warps (TMEM lane quarters)
    } else if (warp < 4 + kWriteWarps) {
        // ------------------------------------------------------------ w V
        // Thread: token rows wt and wt + 32 of a half, 8 columns. Factors and addresses are the
        // same in every full chunk.
        const int wt = (tid - 128) >> 3, wc = tid & 7;
        const uint32_t at = tile_at(smem_u32(sm), wt, wc);        // row wt + 32 i is 4096 i further
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = pw[kTcC - 1 - wt - 32 * i];
#pragma unroll 1
        for (int c = 0, b = 0, ph = 0; c < nt; ++c) {
            const int len = sg.len - c * kTcC;                    // tokens from the chunk on
            if (len < kTcC)
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = pw[max(0, len - 1 - wt - 32 * i)];
            wait_bar(&bars[FULL + b], ph, abort_p);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (i * kHalf >= len) break;
                if (c > 0) wait_bar(&bars[W_FREE + i], c - 1, abort_p);
                const uint32_t from = at + kStateV + b * 16384 + i * 8192, to = at + kStateW + i * 24576;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int left = len - i * kHalf - wt - 32 * r;
                    uint32_t y[3][4] = {};
                    if (left > 0) {
                        const uint4 x = ld_shared_v4(from + r * 4096);
                        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                        const float2 ww = make_float2(w[2 * i + r], w[2 * i + r]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 z = fmul2(bf16x2_to_f2(xs[e]), ww);
#pragma unroll
                            for (int n = 0; n < 3; ++n) {
                                y[n][e] = pack_bf16(z);
                                z = fsub2(z, bf16x2_to_f2(y[n][e]));
                            }
                        }
                    } else {
                        // Rows past the sequence's end (another sequence's, or nothing): zero in
                        // w V and in K, since 0 times what K holds need not be 0.
                        for (int t = 0; t < tiles; ++t)
                            st_shared_v4(at + b * 32768 + t * 16384 + i * 8192 + r * 4096, 0, 0, 0, 0);
                    }
#pragma unroll
                    for (int n = 0; n < 3; ++n)
                        st_shared_v4(to + r * 4096 + n * 8192, y[n][0], y[n][1], y[n][2], y[n][3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[W_READY + i]);
            }
            if (++b == 3) {
                b = 0;
                ++ph;
            }
        }
    } else {
        // ------------------------------------------------------------ the state
        // Thread: state row k = 32 quarter + lane, 32 of the 64 V columns.
        const int quarter = warp & 3, half = (warp - 4 - kWriteWarps) >> 2, k = 32 * quarter + lane;
        float* slots = a.slots + (int64_t)sg.slot0 * per_state + head;
        if (sg.j == 0 && a.init) {
            // The output pass starts from a copy: the final state may replace the initial one.
            const int64_t ip = page_of(a.init_pages, a.npages, sg.seq);
            if (ip >= 0) {
                const float* from = a.init + ip * per_state + head;
#pragma unroll 4
                for (int e = 4 * (tid - 32 * (4 + kWriteWarps)); e < nv * K; e += 128 * kStateWarps)
                    *reinterpret_cast<float4*>(slots + e) = *reinterpret_cast<const float4*>(from + e);
            }
        }
        float2 S[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) S[i] = make_float2(0.f, 0.f);
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int b = c & 1;
            wait_bar(&bars[D_DONE + b], c >> 1, abort_p);
            tc_fence_after();
            const uint32_t t = tD + 256 * b + ((uint32_t)quarter << 21) + 32 * half;
            const float2 lam = c == nt - 1 ? lam_tail : lam_full;
            const float2 hi = make_float2(lam.x, lam.x), lo = make_float2(lam.y, lam.y);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t d[3][16];
#pragma unroll
                for (int n = 0; n < 3; ++n) tmem_ld16(t + 64 * n + 16 * e, d[n]);
                tmem_wait_ld();
                if (e == 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars[D_FREE + b]);
                }
                auto two = [&](int n, int i) { return make_float2(__uint_as_float(d[n][2 * i]), __uint_as_float(d[n][2 * i + 1])); };
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2& s = S[8 * e + i];
                    s = ffma2(hi, s, ffma2(lo, s, fadd2(two(0, i), fadd2(two(1, i), two(2, i)))));
                }
            }
        }
        // lanes side by side along K
        float* p = slots + (int64_t)(sg.j + 1) * per_state + 32 * half * K + k;
        const int rows = k < K ? nv - 32 * half : 0;
#pragma unroll
        for (int i = 0; i < 32; ++i, p += K)
            if (i < rows) *p = i & 1 ? S[i / 2].y : S[i / 2].x;
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tD, 512);
}

// ---------------------------------------------------------------------------------
// Output pass. Warp 0 issues the TMA loads; warp 3 the UMMAs of Q K^T, warp 1 those of Oi and
// Ox, warp 2 those of D (an issuing warp takes its batches in order, and the waits of one
// product would hold up the others); then three groups of eight warps: scores and w V, outputs,
// and the state. Q, K and V are double-buffered. Q K^T runs one unit ahead, in the gap that the
// outputs leave in the tensor pipe while they are read. 4 x 4096 tokens, 32 heads of 128 x 128:
// 177 us (537 MB: 3.0 TB/s); tensor pipe 32%, DRAM 33%: bound by the chain scores -> P -> P V.
//
// Shared memory: K, V, Q (two buffers each), S (a bf16 pair), w V, and a tile of o on its way
// out by TMA (a thread's row of o is 64 bytes in another line than its neighbours'; stored from
// registers it took a seventh of the pass). TMEM columns: Q K^T [0, 128)
// and [128, 256) (units alternate), P of a 32-token block in the first 16 columns of the
// block's scores (read and written by the same thread), Oi [256, 320), Ox [320, 448), D
// [448, 512).

constexpr int kScoreWarps = 8, kOutWarps = 8;
constexpr int kOutThreads = 32 * (4 + kScoreWarps + kOutWarps + kStateWarps);
constexpr int kOutV = 65536, kOutQ = 98304, kOutS = 163840, kOutW = 196608, kOutO = 212992;   // K at 0
constexpr int kOutSmem = 229376 + 1024;

__global__ void __launch_bounds__(kOutThreads, 1)
k_la_tc_out(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
            const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o,
            const __grid_constant__ Args a) {
    using namespace tc;
    const int nvb = (a.V + kTcV - 1) / kTcV;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg(a, blockIdx.x / nvb / a.Hk, true, &sg)) return;
    const int K = a.K, R = a.R, v0 = vb * kTcV, nv = min(kTcV, a.V - v0);
    const int nt = (sg.len + kTcC - 1) / kTcC, halves = (K + 63) / 64;
    const bool partial = sg.len % kTcC != 0;                      // the last chunk
    auto len_of = [&](int c) { return min(kTcC, sg.len - c * kTcC); };
    auto blocks_of = [&](int c) { return (len_of(c) + kBlock - 1) / kBlock; };

    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float pw[kTcC + 1];           // lam^0 .. lam^128
    __shared__ float pws[32 + kTcC];         // 32 zeros, then scale lam^0 .. lam^127
    __shared__ __align__(16) float rev[32];  // lam^31 .. lam^0
    __shared__ float2 lam_full, lam_len;
    // pairs for the two buffers of K, V, Q and the scores, then single barriers
    enum { FULL_K = 0, EMPTY_K = 2, FULL_V = 4, EMPTY_V = 6, FULL_Q = 8, EMPTY_Q = 10, QK_DONE = 12, P_READY = 14, O_DONE = 16,
           O_FREE = 18, QS_DONE, W_READY, D_DONE, D_FREE, S_READY, TAIL_READY, DRAINED, STALL = DRAINED + 3, BARS };
    __shared__ uint64_t bars[BARS];
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float gd = a.log_decay[g];
    const int tt = tid - 64;                 // warps 0 and 1 have other things to set up
    if (tt >= 0 && tt <= kTcC) {
        const float x = (float)pow_decay(gd, tt);
        pw[tt] = x;
        if (tt < kTcC) pws[32 + tt] = a.scale * x;
        if (tt < 32) {
            pws[tt] = 0.f;
            rev[31 - tt] = x;
        }
    }
    if (tid == 256) lam_full = pow2f(gd, kTcC);
    if (tid == 320) lam_len = pow2f(gd, sg.len);
    if (tid < BARS) {
        const int pair = tid & ~1;
        mbar_init(&bars[tid], pair == EMPTY_K || pair == EMPTY_V || pair == EMPTY_Q ? 2
                              : pair == P_READY || tid == O_FREE || (tid >= D_FREE && tid <= TAIL_READY) || tid == W_READY ? 8 : 1);
    }
    static_assert(kScoreWarps == 8 && kOutWarps == 8 && kStateWarps == 8, "arrivals a group makes on a barrier");
    if (tid == 0) {
        check_decay(gd);
        abort_flag = 0;
    }
    fence_barrier_init();
    if (warp == 1) {
        tmem_alloc(&tmem_slot, 512);
        tmem_relinquish();
    }
    const int64_t per_state = (int64_t)a.Hk * a.V * K, head = ((int64_t)g * a.V + v0) * K;
    const int64_t ip = a.init ? page_of(a.init_pages, a.npages, sg.seq) : -1;
    int64_t fp = -1;
    if (a.fin && sg.j + 1 == sg.n) {
        fp = page_of(a.fin_pages, a.npages, sg.seq);
        if (fp >= 0 && __syncthreads_or(page_clash(a, sg.seq, fp, threadIdx.x, kOutThreads))) {
            latch_error(SSD_ERR_INVALID_ARG);
            fp = -1;
        }
    }
    start_block(warp, kOutThreads);
    const uint32_t tbase = tmem_slot, tOi = tbase + 256, tOx = tbase + 320, tD = tbase + 448;
    volatile int* abort_p = &abort_flag;
    const bool has_init = ip >= 0 || sg.j > 0;                    // the first chunk meets a state

    if (warp == 0) {
        // ------------------------------------------------------------ TMA producer
        // Per chunk: K, the first Q, V, the other Qs; every load waits until its buffer is free.
        // (Issuing a 16 KB box takes the thread 320 cycles, five boxes a chunk and head of 128
        // columns; bringing the next ones into L2 took 100 more each and paid nothing.)
        if (lane == 0 && nt > 0) {
            int c = 0, r = 0, job = 0, n[3] = {0, 0, 0};          // loads of K, V and Q issued
#pragma unroll 1
            while (c < nt && !*abort_p) {
                const bool k_ = job == 0, v_ = job == 2;
                const int i = k_ ? n[0] : v_ ? n[1] : n[2], b = i & 1, tiles = v_ ? 1 : halves;
                const CUtensorMap* map = k_ ? &map_k : v_ ? &map_v : &map_q;
                uint64_t* full = &bars[(k_ ? FULL_K : v_ ? FULL_V : FULL_Q) + b];
                uint8_t* dst = sm + (k_ ? b * 32768 : v_ ? kOutV + b * 16384 : kOutQ + b * 32768);
                const int x = v_ ? v0 : 0, head_ = k_ || v_ ? g : g * R + r;
                if (i >= 2) {
                    wait_bar(full + 2, (i >> 1) - 1, abort_p);    // EMPTY follows FULL
                    if (*abort_p) break;
                }
                mbar_arrive_expect_tx(full, tiles * 16384);
#pragma unroll 1
                for (int t = 0; t < tiles; ++t)
                    tma_load_3d(dst + t * 16384, map, full, x + 64 * t, head_, (int)(sg.start + (int64_t)c * kTcC));
                if (k_) ++n[0]; else if (v_) ++n[1]; else { ++n[2]; ++r; }
                if (++job == R + 2) {
                    job = r = 0;
                    ++c;
                }
            }
            // As in the state pass: wait for what is in flight.
#pragma unroll
            for (int m = 0; m < 3; ++m)
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    if (n[m] > b) mbar_wait(&bars[4 * m + b], ((n[m] - 1 - b) >> 1) & 1);
        }
    } else if (warp == 3) {
        // ------------------------------------------------------------ UMMA issuer: Q K^T
        const uint32_t dQ = desc_lo(smem_u32(sm + kOutQ)), dK = desc_lo(smem_u32(sm));
        bool ok = true;
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt && ok; ++c) {
            const uint32_t id = idesc_bf16(128, kBlock * blocks_of(c), 0, 0);          // N: whole blocks
            const uint32_t dk = dK + (c & 1) * 2048;
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                // The buffer last held P of unit u-2, whose product is done.
                if (u >= 2) wait_bar(&bars[O_DONE + (u & 1)], (u >> 1) - 1, abort_p);
                if (r == 0) wait_bar(&bars[FULL_K + (c & 1)], c >> 1, abort_p);
                wait_bar(&bars[FULL_Q + (u & 1)], u >> 1, abort_p);
                if (!(ok = go_on(abort_p))) break;
                tc_fence_after();
                const uint32_t d = tbase + 128 * (u & 1);
                const uint32_t dq = dQ + (u & 1) * 2048;
                if (elect_one()) {
#pragma unroll 1
                    for (int hf = 0; hf < halves; ++hf)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma(d, dq + hf * 1024 + 2 * k, dk + hf * 1024 + 2 * k, id, hf + k > 0);
                    umma_commit(&bars[QK_DONE + (u & 1)]);
                    umma_commit(&bars[EMPTY_Q + (u & 1)]);
                    if (r == R - 1) umma_commit(&bars[EMPTY_K + (c & 1)]);
                }
                __syncwarp();
            }
        }
        // Every MMA issued above has completed once this commit arrives.
        if (elect_one()) umma_commit(&bars[DRAINED + 0]);
        __syncwarp();
        mbar_wait(&bars[DRAINED + 0], 0);
    } else if (warp == 1) {
        // ------------------------------------------------------------ UMMA issuer: Oi, Ox
        const uint32_t id_x = idesc_bf16(128, 128, 0, 1), id_v = idesc_bf16(128, 64, 0, 1);
        const uint32_t dQ = desc_lo(smem_u32(sm + kOutQ));
        const uint32_t dV = desc_lo(smem_u32(sm + kOutV)), dS = desc_lo(smem_u32(sm + kOutS));
        // test hook (stall): a wait that runs out
        if (a.stall && nt > 0) wait_bar(&bars[STALL], 0, abort_p);
        bool ok = true;
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt && ok; ++c) {
            const bool st = c > 0 || has_init;
            const int xhalves = st ? halves : 0, nb = blocks_of(c);
            const uint32_t dv = dV + (c & 1) * 1024;
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                if (r == 0 && st) wait_bar(&bars[S_READY], has_init ? c : c - 1, abort_p);
                wait_bar(&bars[FULL_Q + (u & 1)], u >> 1, abort_p);
                if (u > 0) wait_bar(&bars[O_FREE], u - 1, abort_p);
                if (!(ok = go_on(abort_p))) break;
                tc_fence_after();
                const uint32_t dq = dQ + (u & 1) * 2048;
                if (elect_one()) {
#pragma unroll 1
                    for (int hf = 0; hf < xhalves; ++hf)
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            umma(tOx, dq + hf * 1024 + 2 * k, dS + (hf * 4 + k) * 128, id_x, hf + k > 0);
                    umma_commit(&bars[EMPTY_Q + (u & 1)]);
                    if (r == R - 1) umma_commit(&bars[QS_DONE]);
                }
                __syncwarp();
                // V's rows past the last token hold zeros (tail_ready).
                if (r == 0) wait_bar(&bars[FULL_V + (c & 1)], c >> 1, abort_p);
                if (r == 0 && partial && c == nt - 1) wait_bar(&bars[TAIL_READY], 0, abort_p);
                wait_bar(&bars[P_READY + (u & 1)], u >> 1, abort_p);
                if (!(ok = go_on(abort_p))) break;
                tc_fence_after();
                const uint32_t tP = tbase + 128 * (u & 1);
                if (elect_one()) {
#pragma unroll 1
                    for (int n = 0; n < nb; ++n)
#pragma unroll
                        for (int k = 0; k < 2; ++k) umma_ts(tOi, tP + 32 * n + 8 * k, dv + (2 * n + k) * 128, id_v, n + k > 0);
                    umma_commit(&bars[O_DONE + (u & 1)]);
                    if (r == R - 1) umma_commit(&bars[EMPTY_V + (c & 1)]);
                }
                __syncwarp();
            }
        }
        if (elect_one()) umma_commit(&bars[DRAINED + 1]);
        __syncwarp();
        mbar_wait(&bars[DRAINED + 1], 0);
    } else if (warp == 2) {
        // ------------------------------------------------------------ UMMA issuer: D
        // D = K^T (w V), for every chunk that another one follows (all of them full).
        const uint32_t id = idesc_bf16(128, 64, 1, 1);
        const uint32_t dK = desc_lo(smem_u32(sm)), dW = desc_lo(smem_u32(sm + kOutW));
#pragma unroll 1
        for (int c = 0; c + 1 < nt; ++c) {
            wait_bar(&bars[FULL_K + (c & 1)], c >> 1, abort_p);
            wait_bar(&bars[W_READY], c, abort_p);
            if (c > 0) wait_bar(&bars[D_FREE], c - 1, abort_p);
            if (!go_on(abort_p)) break;
            tc_fence_after();
            const uint32_t dk = dK + (c & 1) * 2048;
            if (elect_one()) {
#pragma unroll 1
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma(tD, dk + (4 * n + k) * 128, dW + (4 * n + k) * 128, id, n + k > 0);
                umma_commit(&bars[D_DONE]);
                umma_commit(&bars[EMPTY_K + (c & 1)]);
                umma_commit(&bars[EMPTY_V + (c & 1)]);
            }
            __syncwarp();
        }
        if (elect_one()) umma_commit(&bars[DRAINED + 2]);
        __syncwarp();
        mbar_wait(&bars[DRAINED + 2], 0);
    } else if (warp < 4 + kScoreWarps) {
        // ------------------------------------------------------------ scores and w V
        // Thread: token row t = 32 quarter + lane; of the four 32-wide column blocks, 0 and 3
        // (half 0) or 1 and 2 (half 1), so that every warp has about the same share of the
        // causal triangle. As a writer of w V: token rows wt + 32 i, 8 columns.
        const int quarter = warp & 3, half = (warp - 4) >> 2, t = 32 * quarter + lane;
        const uint32_t lanes = (uint32_t)quarter << 21;
        const int wt = (tid - 128) >> 3, wc = tid & 7;
        const uint32_t w_at = tile_at(smem_u32(sm), wt, wc);     // row wt + 32 i is 4096 i further
        auto write_w = [&](int c) {          // w V of a full chunk
            wait_bar(&bars[FULL_V + (c & 1)], c >> 1, abort_p);
            if (c > 0) wait_bar(&bars[D_DONE], c - 1, abort_p);            // its buffer has been read
            const uint32_t from = w_at + kOutV + (c & 1) * 16384, to = w_at + kOutW;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 x = ld_shared_v4(from + i * 4096);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                const float w = pw[kTcC - 1 - wt - 32 * i];
                uint32_t y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = pack_bf16(fmul2(bf16x2_to_f2(xs[e]), make_float2(w, w)));
                st_shared_v4(to + i * 4096, y[0], y[1], y[2], y[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[W_READY]);
        };
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const int nb = blocks_of(c);
            if (partial && c == nt - 1) {
                // Rows past the sequence's end (another sequence's, or nothing) are zeroed in V,
                // since a score of 0 times what they hold need not be 0.
                wait_bar(&bars[FULL_V + (c & 1)], c >> 1, abort_p);
                for (int s = len_of(c) + wt; s < kBlock * nb; s += 32)
                    st_shared_v4(tile_at(smem_u32(sm + kOutV) + (c & 1) * 16384, s, wc), 0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[TAIL_READY]);
            }
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                const uint32_t tP = tbase + 128 * (u & 1) + lanes;
                // w V first: K's buffer is free only once it has met it
                if (r == 0 && c + 1 < nt) write_w(c);
                wait_bar(&bars[QK_DONE + (u & 1)], u >> 1, abort_p);
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
                            const float rf = pws[32 + t - 32 * b - 31];
                            const float2 rf2 = make_float2(rf, rf);
#pragma unroll
                            for (int i = 0; i < 32; i += 4) {
                                const float4 f = *reinterpret_cast<const float4*>(rev + i);
                                p[i / 2] = pack_bf16(fmul2(make_float2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])),
                                                           fmul2(rf2, make_float2(f.x, f.y))));
                                p[i / 2 + 1] = pack_bf16(fmul2(make_float2(__uint_as_float(x[i + 2]), __uint_as_float(x[i + 3])),
                                                               fmul2(rf2, make_float2(f.z, f.w))));
                            }
                        } else {
                            // diagonal block: s > t is dropped whatever the score holds
                            const float* f = pws + 32 + lane;
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                const float y0 = i <= lane ? __uint_as_float(x[i]) * f[-i] : 0.f;
                                const float y1 = i + 1 <= lane ? __uint_as_float(x[i + 1]) * f[-i - 1] : 0.f;
                                p[i / 2] = pack_bf16(y0, y1);
                            }
                        }
                    }
                    tmem_st16(tP + 32 * b, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[P_READY + (u & 1)]);
            }
        }
    } else if (warp < 4 + kScoreWarps + kOutWarps) {
        // ------------------------------------------------------------ outputs
        // Thread: token row t, 32 of the 64 columns.
        const int quarter = warp & 3, half = (warp - 4 - kScoreWarps) >> 2, t = 32 * quarter + lane;
        const uint32_t lanes = ((uint32_t)quarter << 21) + 32 * half, sO = smem_u32(sm + kOutO);
        const float2 wx = make_float2(pw[t + 1] * a.scale, pw[t + 1] * a.scale);
        const bool issuer = warp == 4 + kScoreWarps && lane == 0;
        int u = 0;
#pragma unroll 1
        for (int c = 0; c < nt; ++c) {
            const bool st = c > 0 || has_init, whole = len_of(c) == kTcC;
#pragma unroll 1
            for (int r = 0; r < R; ++r, ++u) {
                wait_bar(&bars[O_DONE + (u & 1)], u >> 1, abort_p);
                tc_fence_after();
                uint32_t out[16];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t x[16], h[16], l[16];
                    tmem_ld16(tOi + lanes + 16 * e, x);
                    if (st) {
                        tmem_ld16(tOx + lanes + 16 * e, h);
                        tmem_ld16(tOx + lanes + 64 + 16 * e, l);
                    }
                    tmem_wait_ld();
                    if (e == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bars[O_FREE]);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2 z = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
                        if (st)
                            z = ffma2(wx, fadd2(make_float2(__uint_as_float(h[2 * i]), __uint_as_float(h[2 * i + 1])),
                                                make_float2(__uint_as_float(l[2 * i]), __uint_as_float(l[2 * i + 1]))), z);
                        out[8 * e + i] = pack_bf16(z);
                    }
                }
                if (whole) {
                    if (issuer) bulk_wait_read_all();             // the last tile has left
                    named_barrier(2, 32 * kOutWarps);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        st_shared_v4(tile_at(sO, t, 4 * half + i), out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                    fence_proxy_async_smem();
                    named_barrier(2, 32 * kOutWarps);
                    if (issuer && !*abort_p) {
                        tma_store_3d(&map_o, sm + kOutO, v0, g * R + r, (int)(sg.start + (int64_t)c * kTcC));
                        bulk_commit_group();
                    }
                } else if (t < len_of(c)) {
                    // a partial chunk ends inside the tile: rows one by one
                    __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.o) +
                                       ((sg.start + (int64_t)c * kTcC + t) * a.H + g * R + r) * (int64_t)a.V + v0 + 32 * half;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (8 * i < nv - 32 * half)
                            reinterpret_cast<uint4*>(p)[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
                }
            }
        }
        if (issuer) bulk_wait_all();
    } else {
        // ------------------------------------------------------------ the state
        // Thread: state row k = 32 quarter + lane, 32 of the 64 V columns.
        const int quarter = warp & 3, half = (warp - 4 - kScoreWarps - kOutWarps) >> 2, k = 32 * quarter + lane;
        // The state entering the segment, and the final state after the last one: a warp takes
        // columns of V one by one, lanes side by side along K, sixteen elements a lane in flight;
        // then through shared memory (the place of the operand S; rows of 64 floats, 16-byte
        // chunks exchanged to spread the banks) to the threads that keep them.
        const uint32_t sS = smem_u32(sm + kOutS);
        if (has_init || fp >= 0) {
            const float* slots = a.slots + (int64_t)(sg.slot0 + sg.j) * per_state + head;
            const float* from = a.two_pass ? slots : a.init + ip * per_state + head;
            float* fin = a.fin + fp * per_state + head;
            const int w8 = warp - (4 + kScoreWarps + kOutWarps);
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                float x[16];
                auto v_of = [&](int i) { return w8 + 8 * (4 * step + (i >> 2)); };
                auto k_of = [&](int i) { return lane + 32 * (i & 3); };
                auto mine = [&](int i) { return v_of(i) < nv && k_of(i) < K; };
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = has_init && mine(i) ? from[v_of(i) * K + k_of(i)] : 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int v = v_of(i), kk = k_of(i);
                    const uint32_t to = sS + kk * 256 + ((((uint32_t)v >> 2) ^ (kk & 15)) << 4) + (v & 3) * 4;
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(x[i]) : "memory");
                    // an empty sequence's state as it is: 0 times an infinity would be NaN
                    if (fp >= 0 && mine(i))
                        fin[v * K + kk] = nt == 0 ? x[i] : fmaf(lam_len.x, x[i], fmaf(lam_len.y, x[i], slots[per_state + v * K + kk]));
                }
            }
            named_barrier(1, 32 * kStateWarps);
        }
        float2 S[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (has_init) x = ld_shared_v4(sS + k * 256 + (((8 * half + i) ^ (k & 15)) << 4));
            S[2 * i] = make_float2(__uint_as_float(x.x), __uint_as_float(x.y));
            S[2 * i + 1] = make_float2(__uint_as_float(x.z), __uint_as_float(x.w));
        }
        if (has_init) named_barrier(1, 32 * kStateWarps);        // read before the operand takes the place
        // One float of lam^128 is enough here: an error of 2^-25 per chunk that the state remembers, 2^-12
        // over the longest segment (8192 chunks), beside the 2^-8 of w V's rounding.
        const float2 lam = make_float2(lam_full.x, lam_full.x);
#pragma unroll 1
        for (int c = has_init ? -1 : 0; c + 1 < nt; ++c) {        // S entering chunk c + 1
            if (c >= 0) {
                wait_bar(&bars[D_DONE], c, abort_p);
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint32_t d[8];
                    tmem_ld8(tD + ((uint32_t)quarter << 21) + 32 * half + 8 * e, d);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        S[4 * e + i] =
                            ffma2(lam, S[4 * e + i], make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1])));
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars[D_FREE]);
                wait_bar(&bars[QS_DONE], c, abort_p);
            }
            // S as the B operand of Q S: row k, a bf16 pair
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t h[4], l[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    h[e] = pack_bf16(S[4 * i + e]);
                    l[e] = pack_bf16(fsub2(S[4 * i + e], bf16x2_to_f2(h[e])));
                }
                st_shared_v4(tile_at(sS, k, 4 * half + i), h[0], h[1], h[2], h[3]);
                st_shared_v4(tile_at(sS + 16384, k, 4 * half + i), l[0], l[1], l[2], l[3]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars[S_READY]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tbase, 512);
}

}  // namespace la
}  // namespace ssd
