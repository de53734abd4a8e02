// Linear attention with a decay for each key/value head: what the prompt and the
// single-token kernels share, the CUDA-core prompt kernel, and the single-token kernel.
//
// For every sequence and key/value head g (query heads h = g*R .. g*R+R-1 share it, R =
// H/Hk), lam = exp(log_decay[g]) <= 1:
//
//     S_t = lam S_{t-1} + v_t k_t^T          FP32, stored [V][K] with K contiguous
//     o_t[h] = scale * S_t q_t[h]
//
// Prompts are evaluated in chunks of C tokens. With S the state entering a chunk of len
// tokens, t and s counted from its first token:
//
//     o_t = scale * ( sum_{s<=t} lam^(t-s) (q_t.k_s) v_s + lam^(t+1) S q_t )
//     S' = lam^len S + sum_s lam^(len-1-s) v_s k_s^T
//
// All exponents are >= 0, so nothing overflows. Powers of lam that multiply the state
// again and again (lam, lam^len) are kept as a sum of two floats: with one float the
// relative error of lam^C (2^-25) would grow with the number of chunks the state
// remembers (1 / (1 - lam^C), thousands for slow decays).
#pragma once

#include "ssd_common.cuh"

namespace ssd {
namespace la {

// ---------------------------------------------------------------------------------
// One prompt call as the kernels see it.
struct Args {
    const void* q;
    const void* k;
    const void* v;
    const float* log_decay;
    const float* init;           // [nseq or pages, Hk, V, K] or null
    const int32_t* init_pages;   // [nseq] or null
    float* fin;                  // [nseq or pages, Hk, V, K] or null
    const int32_t* fin_pages;    // [nseq] or null
    void* o;
    float* slots;                // segment states [slot][Hk][V][K]
    const ChunkEntry* table;     // packed: segment table, else null
    const int32_t* first;
    const int32_t* count;
    const int32_t* order;
    const int32_t* cu;           // packed: cu_seqlens
    int64_t q_stride, k_stride, v_stride;   // elements between tokens
    int64_t seqlen, npages;
    float scale;
    int32_t nseq, nps;           // dense: segments per sequence
    int32_t Ls;                  // tokens per segment
    int32_t least;               // packed: sequences of up to `least` tokens go token by token (-1: none do)
    int32_t H, Hk, R, K, V;
    bool two_pass;               // a state pass ran before the output pass
    bool stall;                  // test hook: a wait of the tensor-core kernel's UMMA warp runs out
};

// One segment: tokens [start, start + len) of the packed rows, number j of the n segments
// of sequence seq, whose n + 1 state slots begin at slot0. After the state pass slot slot0
// holds a copy of the sequence's initial state (the state may be replaced in place while other
// segments' CTAs still run), slot0 + i the state that segment i-1 alone adds; the passing
// kernel turns slots slot0 + 1 .. slot0 + n - 1 into the states entering segments 1 .. n-1.
struct Seg {
    int32_t seq, j, n, slot0, len;
    int64_t start;
};

// First state slot of sequence s, whose segments begin with number `first`. Sequences that go
// token by token have no segments and are many: the others then take two slots per segment.
__device__ __forceinline__ int32_t slot_of(const Args& a, int32_t first, int32_t s) {
    return a.table && a.least >= 0 ? 2 * first : first + s;
}

// Segment `i` of a pass; false where a packed call has fewer. `last`: the pass takes each
// sequence's last segment too.
__device__ __forceinline__ bool find_seg(const Args& a, int i, bool last, Seg* s) {
    if (a.table) {
        if (i >= *a.count) return false;
        const ChunkEntry e = a.table[a.order[i]];
        s->seq = e.seq;
        s->start = e.start;
        s->len = e.len;
        const int first = a.first[e.seq];
        s->slot0 = slot_of(a, first, e.seq);
        s->n = a.first[e.seq + 1] - first;
        s->j = e.pad - first;
        return last || s->j + 1 < s->n;
    }
    const int per = last ? a.nps : a.nps - 1;
    s->seq = i / per;
    s->j = i % per;
    s->n = a.nps;
    s->slot0 = s->seq * (a.nps + 1);
    s->start = (int64_t)s->seq * a.seqlen + (int64_t)s->j * a.Ls;
    s->len = (int32_t)min((int64_t)a.Ls, a.seqlen - (int64_t)s->j * a.Ls);
    return true;
}

// Where sequence s's state is in an array of states: its page, or s without a page list.
// -1 stands for "none"; a page outside the pool is an error and stands for none too.
__device__ __noinline__ int64_t page_of(const int32_t* pages, int64_t npages, int32_t s) {
    if (!pages) return s;
    const int32_t p = pages[s];
    if (p < -1 || p >= npages) {
        latch_error(SSD_ERR_INVALID_ARG);
        return -1;
    }
    return p;
}

// Whether sequence s must not write its final state to page p: an earlier sequence writes
// the same page, or another one starts from it in this call. Each of `step` threads looks
// at its share; the caller joins what they find.
__device__ __noinline__ int page_clash(const Args& a, int32_t s, int64_t p, int from, int step) {
    int bad = 0;
    const bool one_pool = a.init == a.fin;
    if (!a.fin_pages && !(a.init_pages && one_pool)) return 0;
    for (int32_t i = from; i < a.nseq; i += step) {
        if (i == s) continue;
        if (i < s && a.fin_pages && a.fin_pages[i] == p) bad = 1;
        if (one_pool && (a.init_pages ? a.init_pages[i] : i) == p) bad = 1;
    }
    return bad;
}

// lam^n in 64 bits. Not inlined: the prompt kernels take it at six places, and code that runs
// once per CTA should not crowd the instruction cache.
__device__ __noinline__ double pow_decay(float g, int64_t n) { return exp((double)g * (double)n); }

// lam^n as hi + lo; hi is lam^n rounded to float.
__device__ __forceinline__ float2 pow2f(float g, int64_t n) {
    const double e = pow_decay(g, n);
    const float hi = (float)e;
    return make_float2(hi, (float)(e - (double)hi));
}

// lam as hi + lo for a state that meets it once a token. Slow decays: 1 + expm1(g) with the
// rounding of the sum kept, an error of 2^-24 of 1 - lam, so that it stays 2^-24 over the 1 / (1 - lam)
// tokens that the state remembers. Below 1/2 that would be relative to 1 and not to lam (no digit is
// left at g = -17), and the state remembers less than two tokens: exp(g) rounded to float.
__device__ __forceinline__ float2 decay_pair(float g) {
    const float m1 = expm1f(g), hi = 1.f + m1;
    return m1 < -0.5f ? make_float2(expf(g), 0.f) : make_float2(hi, m1 - (hi - 1.f));
}

__device__ __forceinline__ void check_decay(float g) {
    if (!(g <= 0.f) || isinf(g)) latch_error(SSD_ERR_INVALID_ARG);
}

// ---------------------------------------------------------------------------------
// States entering the segments, in place: S_j = lam^Ls S_(j-1) + (what segment j-1 adds), from
// the copy of the initial state. One thread per four state elements, the loads of four
// segments in flight ahead of the chain. (Each output CTA summing the segments before it
// itself costs a pass over all their states per segment: with 64 segments the output pass took
// ten times as long.) 4 to 12 us: latency.
constexpr int kPassThreads = 256;

__global__ void __launch_bounds__(kPassThreads) k_la_passing(const __grid_constant__ Args a) {
    const int s = blockIdx.x, g = blockIdx.y;
    const int e = 4 * (blockIdx.z * kPassThreads + threadIdx.x), size = a.V * a.K;
    int first = s * a.nps, n = a.nps;
    if (a.table) {
        if (*a.count <= 0) return;                                // a bad cu_seqlens, or no segments
        first = a.first[s];
        n = a.first[s + 1] - first;
    }
    if (e >= size || n < 2) return;
    const int64_t per_state = (int64_t)a.Hk * size;
    float* p = a.slots + (int64_t)slot_of(a, first, s) * per_state + (int64_t)g * size + e;
    const float2 lam = pow2f(a.log_decay[g], a.Ls);
    const bool init = a.init && page_of(a.init_pages, a.npages, s) >= 0;
    float4 x = init ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 1; j < n; j += 4) {
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i < n) y[i] = *reinterpret_cast<const float4*>(p + (j + i) * per_state);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (j + i < n) {
                x.x = fmaf(lam.x, x.x, fmaf(lam.y, x.x, y[i].x));
                x.y = fmaf(lam.x, x.y, fmaf(lam.y, x.y, y[i].y));
                x.z = fmaf(lam.x, x.z, fmaf(lam.y, x.z, y[i].z));
                x.w = fmaf(lam.x, x.w, fmaf(lam.y, x.w, y[i].w));
                *reinterpret_cast<float4*>(p + (j + i) * per_state) = x;
            }
    }
}

// ---------------------------------------------------------------------------------
// CUDA-core prompt kernel for fp32 (FP32 arithmetic throughout; the tensor cores would round
// the inputs). One CTA per (segment, key/value head, 64 columns of V); chunks of 64 tokens in
// shared memory, the state there too as [K][64]. Without OUT: only the state that the segment
// adds. Every product runs in 4 x 4 register tiles fed by 16-byte shared loads along the
// summed index, eight for 64 FMAs. Bound by those shared loads and by the wait for a chunk's rows
// (two CTAs per SM hide each other's where their shared memory fits): 3 sequences of 1537 tokens
// take 43 us (state) and 104 us (output), a lone CTA 5.5 us per chunk at K = V = 16, 10 at 64.
constexpr int kSimtC = 64;           // tokens per chunk
constexpr int kSimtV = 64;           // V columns per CTA
constexpr int kSimtThreads = 256;

__host__ __device__ constexpr int simt_ld(int n) { return n + 4; }   // row stride: rows start in other banks
__host__ __device__ constexpr size_t simt_smem(int K, bool out) {
    return sizeof(float) * ((size_t)kSimtC * simt_ld(K) + kSimtC * kSimtV + (size_t)K * simt_ld(kSimtV) + kSimtC + 4 +
                            (out ? (size_t)kSimtC * simt_ld(K) + kSimtC * kSimtV + kSimtC * simt_ld(kSimtC) : 0));
}

// The 16-byte pieces of a chunk's [64][n] rows as the threads share them out (n a multiple of 8):
// a power of two of lanes per row, f(row, first column).
template <typename F>
__device__ __forceinline__ void simt_share(int n, F f) {
    const int bits = 32 - __clz(n / 4 - 1), c = 4 * (threadIdx.x & ((1 << bits) - 1));
    if (c >= n) return;
#pragma unroll 1
    for (int t = threadIdx.x >> bits; t < kSimtC; t += kSimtThreads >> bits) f(t, c);
}

// Rows of a [tokens][n] matrix (`stride` elements between rows) on their way into shared memory
// with row stride ld (asynchronous copies: all of a chunk's are in flight at once); rows from
// len on are zeros.
__device__ __forceinline__ void simt_rows(float* dst, int ld, const float* src, int64_t stride, int n, int len) {
    simt_share(n, [&](int t, int c) {
        if (t < len) cp_async16(dst + t * ld + c, src + t * stride + c);
        else *reinterpret_cast<float4*>(dst + t * ld + c) = make_float4(0.f, 0.f, 0.f, 0.f);
    });
}

// dst row s = f[len-1-s] times row s of src, the elements that the thread has copied itself.
__device__ __forceinline__ void simt_scale(float* dst, const float* src, int ld, int n, int len, const float* f) {
    simt_share(n, [&](int t, int c) {
        const float w = t < len ? f[len - 1 - t] : 0.f;
        const float4 x = *reinterpret_cast<const float4*>(src + t * ld + c);
        *reinterpret_cast<float4*>(dst + t * ld + c) = make_float4(w * x.x, w * x.y, w * x.z, w * x.w);
    });
}

__device__ __forceinline__ void axpy4(float4& acc, float x, const float4& y) {
    acc.x = fmaf(x, y.x, acc.x);
    acc.y = fmaf(x, y.y, acc.y);
    acc.z = fmaf(x, y.z, acc.z);
    acc.w = fmaf(x, y.w, acc.w);
}

// acc[i] += sum over n of x[row i][n] * y[n][four columns], n in steps of four up to `end`.
__device__ __forceinline__ void simt_tile(float4 (&acc)[4], const float* x, int ldx16, const float* y, int ldy, int end) {
#pragma unroll 2
    for (int n = 0; n < end; n += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i] = *reinterpret_cast<const float4*>(x + i * ldx16 + n);
            b[i] = *reinterpret_cast<const float4*>(y + (n + i) * ldy);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            axpy4(acc[i], a[i].x, b[0]);
            axpy4(acc[i], a[i].y, b[1]);
            axpy4(acc[i], a[i].z, b[2]);
            axpy4(acc[i], a[i].w, b[3]);
        }
    }
}

template <bool OUT>
__global__ void __launch_bounds__(kSimtThreads, 2) k_la_simt(const __grid_constant__ Args a) {
    constexpr int C = kSimtC, VB = kSimtV, NT = kSimtThreads, ldp = simt_ld(C), lds = simt_ld(VB);
    const int nvb = (a.V + VB - 1) / VB;
    const int vb = blockIdx.x % nvb, g = (blockIdx.x / nvb) % a.Hk;
    Seg sg;
    if (!find_seg(a, blockIdx.x / nvb / a.Hk, OUT, &sg)) return;
    const int K = a.K, V = a.V, ldk = simt_ld(K), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int v0 = vb * VB, nv = min(VB, V - v0);

    extern __shared__ __align__(16) float smem[];
    float* sk = smem;                        // [C][ldk]
    float* sw = sk + C * ldk;                // [C][VB]: w V
    float* sS = sw + C * VB;                 // [K][lds]
    float* pw = sS + K * lds;                // lam^0 .. lam^C
    float* sq = pw + C + 4;                  // [C][ldk]
    float* sv = sq + C * ldk;                // [C][VB]
    float* sP = sv + C * VB;                 // [C][ldp]
    __shared__ float2 lam_full, lam_tail;

    const float gd = a.log_decay[g];
    const int tail = sg.len - (sg.len - 1) / C * C;              // tokens of the last chunk
    if (tid <= C) pw[tid] = (float)pow_decay(gd, tid);
    if (tid == 96) lam_full = pow2f(gd, C);
    if (tid == 128) lam_tail = pow2f(gd, sg.len > 0 ? tail : 0);
    if (tid == 0) check_decay(gd);
    const int64_t per_state = (int64_t)a.Hk * V * K, head = ((int64_t)g * V + v0) * K;
    const int64_t ip = a.init ? page_of(a.init_pages, a.npages, sg.seq) : -1;
    int64_t fp = -1;
    if (OUT && sg.j + 1 == sg.n && a.fin) {
        fp = page_of(a.fin_pages, a.npages, sg.seq);
        if (fp >= 0 && __syncthreads_or(page_clash(a, sg.seq, fp, threadIdx.x, NT))) {
            latch_error(SSD_ERR_INVALID_ARG);
            fp = -1;
        }
    }
    // State entering the segment (zero without OUT); [V][K] in memory, lanes along K.
    {
        const float* from = nullptr;
        if (OUT && sg.j > 0) from = a.slots + (int64_t)(sg.slot0 + sg.j) * per_state + head;
        else if (OUT && ip >= 0) from = sg.n == 1 ? a.init + ip * per_state + head : a.slots + (int64_t)sg.slot0 * per_state + head;
        const bool copy = !OUT && sg.j == 0 && ip >= 0;          // for the output pass
#pragma unroll 4
        for (int v = warp; v < VB; v += NT / 32)
            for (int kk = lane; kk < K; kk += 32) {
                sS[kk * lds + v] = from && v < nv ? from[v * K + kk] : 0.f;
                if (copy && v < nv)
                    a.slots[(int64_t)sg.slot0 * per_state + head + v * K + kk] = a.init[ip * per_state + head + v * K + kk];
            }
    }

    const float* kp = static_cast<const float*>(a.k) + sg.start * a.k_stride + (int64_t)g * K;
    const float* vp = static_cast<const float*>(a.v) + sg.start * a.v_stride + (int64_t)g * V + v0;
    const bool need_last = !OUT || fp >= 0;
    const int tx = tid & 15, ty = tid >> 4;                      // rows ty + 16 i, columns 4 tx ..
#pragma unroll 1
    for (int c0 = 0; c0 < sg.len; c0 += C) {
        const int len = min(C, sg.len - c0), end = (len + 3) & ~3;
        __syncthreads();                     // the last chunk's readers are done (and the tables written)
        auto rows_q = [&](int r) {
            simt_rows(sq, ldk, static_cast<const float*>(a.q) + (sg.start + c0) * a.q_stride + (int64_t)(g * a.R + r) * K,
                      a.q_stride, K, len);
        };
        simt_rows(sk, ldk, kp + c0 * a.k_stride, a.k_stride, K, len);
        simt_rows(OUT ? sv : sw, VB, vp + c0 * a.v_stride, a.v_stride, nv, len);
        if (OUT) rows_q(0);
        cp_async_commit();
        cp_async_wait<0>();
        simt_scale(sw, OUT ? sv : sw, VB, nv, len, pw);
        __syncthreads();
#pragma unroll 1
        for (int r = 0; OUT && r < a.R; ++r) {
            if (r > 0) {
                __syncthreads();             // readers of sq and sP are done
                rows_q(r);
                cp_async_commit();
                cp_async_wait<0>();
                __syncthreads();
            }
            {
                float acc[4][4] = {};        // rows ty + 16 i, source tokens tx + 16 j
#pragma unroll 2
                for (int kk = 0; kk < K; kk += 4) {
                    float4 x[4], y[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[i] = *reinterpret_cast<const float4*>(sq + (ty + 16 * i) * ldk + kk);
                        y[i] = *reinterpret_cast<const float4*>(sk + (tx + 16 * i) * ldk + kk);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j <= i; ++j) {            // later blocks lie above the diagonal
                            acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
                            acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
                            acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
                            acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = ty + 16 * i, s = tx + 16 * j;
                        sP[t * ldp + s] = s <= t ? acc[i][j] * pw[t - s] : 0.f;
                    }
            }
            __syncthreads();
            float4 acc[4], inter[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = inter[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            simt_tile(acc, sP + ty * ldp, 16 * ldp, sv + 4 * tx, VB, min(end, (ty + 52) & ~3));
            simt_tile(inter, sq + ty * ldk, 16 * ldk, sS + 4 * tx, lds, K);
            float* op = static_cast<float*>(a.o) + ((sg.start + c0) * a.H + g * a.R + r) * (int64_t)V + v0 + 4 * tx;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = ty + 16 * i;
                if (t >= len || 4 * tx >= nv) continue;
                const float w = pw[t + 1];
                *reinterpret_cast<float4*>(op + (int64_t)t * a.H * V) =
                    make_float4(a.scale * fmaf(w, inter[i].x, acc[i].x), a.scale * fmaf(w, inter[i].y, acc[i].y),
                                a.scale * fmaf(w, inter[i].z, acc[i].z), a.scale * fmaf(w, inter[i].w, acc[i].w));
            }
        }
        if (OUT) __syncthreads();            // readers of the state are done
        if (c0 + C < sg.len || need_last) {
            // S = lam^len S + k^T (w V): rows 4 ty .. of 64, columns 4 tx ..
            const float2 lam = c0 + C < sg.len ? lam_full : lam_tail;
#pragma unroll 1
            for (int kb = 4 * ty; kb < K; kb += 64) {
                float4 acc[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int s = 0; s < end; ++s) {
                    const float4 x = *reinterpret_cast<const float4*>(sk + s * ldk + kb);
                    const float4 y = *reinterpret_cast<const float4*>(sw + s * VB + 4 * tx);
                    axpy4(acc[0], x.x, y);
                    axpy4(acc[1], x.y, y);
                    axpy4(acc[2], x.z, y);
                    axpy4(acc[3], x.w, y);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float4* p = reinterpret_cast<float4*>(sS + (kb + i) * lds + 4 * tx);
                    float4 s = *p;
                    s.x = fmaf(lam.x, s.x, fmaf(lam.y, s.x, acc[i].x));
                    s.y = fmaf(lam.x, s.y, fmaf(lam.y, s.y, acc[i].y));
                    s.z = fmaf(lam.x, s.z, fmaf(lam.y, s.z, acc[i].z));
                    s.w = fmaf(lam.x, s.w, fmaf(lam.y, s.w, acc[i].w));
                    *p = s;
                }
            }
        }
    }
    __syncthreads();
    float* dst = OUT ? (fp >= 0 ? a.fin + fp * per_state : nullptr) : a.slots + (int64_t)(sg.slot0 + sg.j + 1) * per_state;
    if (dst)
        for (int v = warp; v < nv; v += NT / 32)
            for (int kk = lane; kk < K; kk += 32) dst[head + v * K + kk] = sS[kk * lds + v];
}

// ---------------------------------------------------------------------------------
// Single tokens: S <- lam S + v k^T in place and o = scale * S q for one token of every
// batch row. The FP32 state (64 KiB per head at 128 x 128) is read and written once and
// is all the traffic that counts, so the kernel is an HBM stream: a state row of K floats
// is LPR lanes of 16 bytes, a warp keeps 8 rows per lane group in flight before it writes
// any, and one state serves all R query heads that share it. 256 sequences of 32 heads (1.08 GB
// of traffic): 165 us, 99% of the measured copy rate. A warp as the unit, each with its own
// search for pages named twice, was 1.7 times as fast on 16384 rows of 4 KiB states, but took
// 100 registers instead of 72 and 180 us of the case above. That search is quadratic in the batch:
// nothing to see at 256 rows, 4 us of 86 at 4096, half of the time at 16384.
constexpr int kTokThreads = 128;
constexpr int kTokRows = 8;          // state rows in flight per lane group

// Sums of kTokRows values per lane over the LPR lanes of a group. While more than one row is
// left per lane, a lane gives half of its rows to its partner (8/2, 8/4, .. shuffles instead of
// 8 per step); then plain butterflies. d[0 .. rows_left) are rows `returned` and on; with more
// than eight lanes they are in every (LPR / 8)-th lane.
__host__ __device__ constexpr int rows_left(int lpr) { return lpr >= kTokRows ? 1 : kTokRows / lpr; }

template <int LPR>
__device__ __forceinline__ int sum_rows(float (&d)[kTokRows], int c4) {
    int n = kTokRows, off = LPR / 2, mine = 0;
#pragma unroll
    for (int step = 0; step < 3; ++step) {
        if (off >= 1 && n > 1) {
            const bool up = (c4 & off) != 0;
#pragma unroll
            for (int i = 0; i < kTokRows / 2; ++i)
                if (i < n / 2) {
                    const float give = up ? d[i] : d[i + n / 2], keep = up ? d[i + n / 2] : d[i];
                    d[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
                }
            n /= 2;
            mine += up ? n : 0;
            off /= 2;
        }
    }
#pragma unroll
    for (int w = LPR / 16; w >= 1; w /= 2) d[0] += __shfl_xor_sync(0xffffffffu, d[0], w);
    return mine;
}

template <typename T, int LPR>
__global__ void __launch_bounds__(kTokThreads)
k_la_update(float* __restrict__ state, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
            const float* __restrict__ log_decay, float scale, const int32_t* __restrict__ pages, int64_t npages,
            T* __restrict__ o, int nvs, int Hk, int R, int K, int V, int64_t qs, int64_t ks, int64_t vs) {
    constexpr int GPW = 32 / LPR;                        // lane groups (rows of one load) per warp
    constexpr int U = kTokRows, WARPS = kTokThreads / 32;
    constexpr int RPB = U * GPW * WARPS;                 // state rows per CTA
    const int vsp = blockIdx.x % nvs, g = (blockIdx.x / nvs) % Hk;
    const int64_t b = blockIdx.x / nvs / Hk;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c4 = lane % LPR, grp = lane / LPR;
    int64_t page = b;
    if (pages) {
        page = pages[b];
        if (page < 0 || page >= npages) {                // -1: a padded row, left as it is
            if (page != -1 && threadIdx.x == 0) latch_error(SSD_ERR_INVALID_ARG);
            return;
        }
    }
    float* st = state + (page * Hk + g) * (int64_t)V * K;
    // this lane group's rows: r0 + u * GPW, columns 4 c4 ..
    const int r0 = vsp * RPB + warp * U * GPW + grp;
    const bool col = 4 * c4 < K;
    float4 s[U];
    float vr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = r0 + u * GPW;
        const bool ok = col && row < V;
        s[u] = ok ? __ldcs(reinterpret_cast<const float4*>(st + (int64_t)row * K + 4 * c4)) : make_float4(0, 0, 0, 0);
        vr[u] = row < V ? to_f32(v[b * vs + (int64_t)g * V + row]) : 0.f;
    }
    const float4 kv = col ? load4(k + b * ks + (int64_t)g * K + 4 * c4) : make_float4(0, 0, 0, 0);
    if (pages) {
        // A page named twice would be updated by two blocks at once: the first row keeps
        // it, the others are refused.
        int dup = 0;
        for (int64_t i = threadIdx.x; i < b; i += kTokThreads) dup |= pages[i] == page;
        if (__syncthreads_or(dup)) {
            if (threadIdx.x == 0) latch_error(SSD_ERR_INVALID_ARG);
            return;
        }
    }
    const float gd = log_decay[g];
    if (threadIdx.x == 0) check_decay(gd);
    const float2 lam = decay_pair(gd);
    const float hi = lam.x, lo = lam.y;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = r0 + u * GPW;
        s[u].x = fmaf(hi, s[u].x, fmaf(lo, s[u].x, vr[u] * kv.x));
        s[u].y = fmaf(hi, s[u].y, fmaf(lo, s[u].y, vr[u] * kv.y));
        s[u].z = fmaf(hi, s[u].z, fmaf(lo, s[u].z, vr[u] * kv.z));
        s[u].w = fmaf(hi, s[u].w, fmaf(lo, s[u].w, vr[u] * kv.w));
        if (col && row < V) __stcs(reinterpret_cast<float4*>(st + (int64_t)row * K + 4 * c4), s[u]);
    }
    const T* qb = q + b * qs + (int64_t)g * R * K;
    T* ob = o + ((b * Hk + g) * (int64_t)R) * V;
    for (int r = 0; r < R; ++r) {
        const float4 qv = col ? load4(qb + (int64_t)r * K + 4 * c4) : make_float4(0, 0, 0, 0);
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) d[u] = fmaf(s[u].x, qv.x, fmaf(s[u].y, qv.y, fmaf(s[u].z, qv.z, s[u].w * qv.w)));
        const int mine = sum_rows<LPR>(d, c4);
        if (LPR <= 8 || (c4 & (LPR / 8 - 1)) == 0) {
#pragma unroll
            for (int i = 0; i < rows_left(LPR); ++i) {
                const int row = r0 + (mine + i) * GPW;
                if (row < V) ob[(int64_t)r * V + row] = from_f32<T>(scale * d[i]);
            }
        }
    }
}

// ---------------------------------------------------------------------------------
// Short sequences of a prompt call, token by token: the same recurrence, the state in registers
// from the sequence's first token to its last, so that it crosses HBM twice however many tokens
// there are. A warp holds 8 to 64 rows of one state (a lane eight neighbouring rows, four columns) and
// needs nothing from other warps; the next token's q, k and v are on their way while one is
// computed. 4 K V FMAs a token where the chunked form has fewer and tensor cores for them, but a lone
// call of one chunk takes 17 us there (both passes; 20 with an initial state), and on a full GPU every
// CTA (64 columns of V) 8 us of the state pass and 24 of the output pass, however short its
// sequence. 256 sequences of one token (32 heads, 128 x 128): 167 us, 99% of the measured copy rate (in
// chunks 3530 us); of 16 tokens 824 us.
// Bound by instruction issue from a few tokens on (274 instructions a token and warp, 66% of the
// issue slots). Packed pairs of FMAs and batches of four tokens were no faster.
template <typename T> struct Raw;                        // elements as they are loaded
template <> struct Raw<float> {
    float4 x{};
    __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ float4 four() const { return x; }
};
template <> struct Raw<__nv_bfloat16> {
    uint2 x{};
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { x = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ float4 four() const {
        return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                           __uint_as_float(x.y & 0xffff0000u));
    }
};

template <typename T, int LPR>
__global__ void __launch_bounds__(kTokThreads) k_la_steps(const __grid_constant__ Args a, int nvs) {
    constexpr int U = kTokRows, RPW = U * (32 / LPR);
    const int lane = threadIdx.x & 31, c4 = lane % LPR, grp = lane / LPR;
    const int Hk = a.Hk, K = a.K, V = a.V, R = a.R;
    const uint32_t unit = blockIdx.x * (kTokThreads / 32) + (threadIdx.x >> 5), part = unit / (uint32_t)nvs;   // < 2^31
    const int seq = (int)(part / (uint32_t)Hk), g = (int)part - seq * Hk, row = (int)(unit - part * nvs) * RPW + grp * U;
    if (seq >= a.nseq) return;
    int64_t start = seq * a.seqlen;
    int32_t len = (int32_t)a.seqlen;
    if (a.cu) {
        if (*a.count < 0) return;                        // a bad cu_seqlens
        start = a.cu[seq];
        len = a.cu[seq + 1] - (int32_t)start;
        if (len > a.least) return;
    }
    const bool col = 4 * c4 < K, rows = row < V, mine_ = col && rows;
    const int64_t ip = a.init ? page_of(a.init_pages, a.npages, seq) : -1;
    int64_t fp = a.fin ? page_of(a.fin_pages, a.npages, seq) : -1;
    if (fp >= 0 && __any_sync(0xffffffffu, page_clash(a, seq, fp, lane, 32))) {
        if (lane == 0) latch_error(SSD_ERR_INVALID_ARG);
        fp = -1;
    }
    const int64_t at = ((int64_t)g * V + row) * K + 4 * c4, per_state = (int64_t)Hk * V * K;
    float4 s[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        s[u] = mine_ && ip >= 0 ? __ldcs(reinterpret_cast<const float4*>(a.init + ip * per_state + at + u * K)) : make_float4(0, 0, 0, 0);
    const T* qp = static_cast<const T*>(a.q) + start * a.q_stride + (int64_t)g * R * K + 4 * c4;
    const T* kp = static_cast<const T*>(a.k) + start * a.k_stride + (int64_t)g * K + 4 * c4;
    const T* vp = static_cast<const T*>(a.v) + start * a.v_stride + (int64_t)g * V + row;
    T* op = static_cast<T*>(a.o) + (start * a.H + (int64_t)g * R) * V + row;
    const float gd = a.log_decay[g];
    if (lane == 0) check_decay(gd);
    const float2 lam = decay_pair(gd);
    const float hi = lam.x, lo = lam.y;
    Raw<T> qn, kn, vn[2];
    auto load_kv = [&] {
        if (col) kn.load(kp);
        if (rows) {
            vn[0].load(vp);
            vn[1].load(vp + 4);
        }
        kp += a.k_stride;
        vp += a.v_stride;
    };
    if (len > 0) {
        load_kv();
        if (col) qn.load(qp);
    }
#pragma unroll 1
    for (int t = 0; t < len; ++t, op += (int64_t)a.H * V) {
        const float4 kv = kn.four(), va = vn[0].four(), vb = vn[1].four();
        const float v[U] = {va.x, va.y, va.z, va.w, vb.x, vb.y, vb.z, vb.w};
        if (t + 1 < len) load_kv();
#pragma unroll
        for (int u = 0; u < U; ++u) {
            s[u].x = fmaf(hi, s[u].x, fmaf(lo, s[u].x, v[u] * kv.x));
            s[u].y = fmaf(hi, s[u].y, fmaf(lo, s[u].y, v[u] * kv.y));
            s[u].z = fmaf(hi, s[u].z, fmaf(lo, s[u].z, v[u] * kv.z));
            s[u].w = fmaf(hi, s[u].w, fmaf(lo, s[u].w, v[u] * kv.w));
        }
#pragma unroll 1
        for (int r = 0; r < R; ++r) {
            const float4 qv = qn.four();
            if (r + 1 == R) qp += a.q_stride;
            if (col && (r + 1 < R || t + 1 < len)) qn.load(qp + (r + 1 < R ? (r + 1) * K : 0));
            float d[U];
#pragma unroll
            for (int u = 0; u < U; ++u) d[u] = fmaf(s[u].x, qv.x, fmaf(s[u].y, qv.y, fmaf(s[u].z, qv.z, s[u].w * qv.w)));
            const int mine = sum_rows<LPR>(d, c4);
            if (rows && (LPR <= 8 || (c4 & (LPR / 8 - 1)) == 0)) {
#pragma unroll
                for (int i = 0; i < rows_left(LPR); ++i) op[(int64_t)r * V + mine + i] = from_f32<T>(a.scale * d[i]);
            }
        }
    }
    if (mine_ && fp >= 0)
#pragma unroll
        for (int u = 0; u < U; ++u) __stcs(reinterpret_cast<float4*>(a.fin + fp * per_state + at + u * K), s[u]);
}

}  // namespace la
}  // namespace ssd
