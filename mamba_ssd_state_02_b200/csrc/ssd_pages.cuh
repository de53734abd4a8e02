// Pages of a state cache: append, fork, free, compact and copy.
//
// A pool is a set of device arrays, all with the same number of pages along their first
// dimension (a page = one state in every array: the SSM states, conv states, linear
// attention states or strict chunk caches of all layers), and int32 metadata on the device:
//   refcount [n_pages]           rows that hold the page; 0: free
//   table    [n_rows][max_pages] pages of each row (a sequence) in order, -1 past its end
//   length   [n_rows]            pages of the row
//   live     [n_rows]            the row's last page, the one its next token changes; -1: none
// Every operation is two launches without any host synchronisation: one block decides
// (checks the request, takes the lowest free pages in the order of the request, updates the
// metadata and writes the list of page moves), and a grid moves the bytes. A request that
// is not valid as a whole, or for which there are not enough free pages, is latched and
// changes nothing. The results do not depend on the order in which threads run.
#pragma once

#include "ssd_common.cuh"

namespace ssd {
namespace pages {

constexpr int kThreads = 1024;               // the deciding block
constexpr int kMaxArrays = 128;
constexpr int kMaxIndex = 1 << 20;           // pages and rows: one bit each in shared memory

struct Meta {
    int32_t* refcount;
    int32_t* table;
    int32_t* length;
    int32_t* live;
    int32_t n_pages, n_rows, max_pages;
};

// Moves of one operation, in the workspace: count, then src and dst page numbers.
struct Moves {
    int32_t* count;
    int32_t* src;
    int32_t* dst;
};

enum Op { APPEND, FORK, FREE, COPY };

// Exclusive prefix sum over the block; *total the sum. wsum: 33 shared slots.
__device__ __forceinline__ int32_t block_scan(int32_t v, int32_t* wsum, int32_t* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    int32_t x = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
    }
    __syncthreads();                         // readers of the last call's totals are done
    if (lane == 31) wsum[wid] = x;
    __syncthreads();
    if (wid == 0) {
        int32_t w = wsum[lane];
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int32_t y = __shfl_up_sync(0xffffffffu, w, off);
            if (lane >= off) w += y;
        }
        wsum[lane] = w;
    }
    __syncthreads();
    *total = wsum[31];
    return (wid ? wsum[wid - 1] : 0) + x - v;
}

__device__ __forceinline__ bool take_bit(uint32_t* bits, int32_t i) {      // true: it was set before
    return (atomicOr(&bits[i >> 5], 1u << (i & 31)) >> (i & 31)) & 1;
}
__device__ __forceinline__ bool has_bit(const uint32_t* bits, int32_t i) { return (bits[i >> 5] >> (i & 31)) & 1; }

// A row's length and pages can be trusted: in range and in use.
__device__ __forceinline__ bool row_ok(const Meta& m, int32_t r) {
    const int32_t n = m.length[r];
    return n >= 0 && n <= m.max_pages;
}
__device__ __forceinline__ bool page_ok(const Meta& m, int32_t p) {
    return p >= 0 && p < m.n_pages && m.refcount[p] > 0;
}

// One block: APPEND (a = rows), FORK (a = parents, b = children), FREE (a = rows), COPY
// (a = source pages, b = destination pages). Entries of -1 are skipped. fresh: n ints of
// workspace for the new pages. copy_last (APPEND): the new page starts as a copy of the
// row's last one.
template <Op OP>
__global__ void __launch_bounds__(kThreads)
k_pages_plan(const Meta m, const int32_t* __restrict__ a, const int32_t* __restrict__ b, int32_t n, int copy_last,
             int32_t* __restrict__ fresh, const Moves mv) {
    extern __shared__ uint32_t bits[];       // rows (pages for COPY) named so far
    __shared__ int32_t wsum[33];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int32_t range = OP == COPY ? m.n_pages : m.n_rows;
    for (int32_t i = tid; i < (range + 31) / 32; i += kThreads) bits[i] = 0;
    if (tid == 0 && OP != FREE) *mv.count = 0;
    __syncthreads();

    // -------- the request as a whole: valid indexes, nothing named twice
    int bad = 0;
    for (int32_t i = tid; i < n; i += kThreads) {
        const int32_t x = a[i], y = OP == FORK || OP == COPY ? b[i] : 0;
        if (x == -1 || y == -1) continue;
        if (x < 0 || x >= range || y < 0 || y >= range) {
            bad = 1;
            continue;
        }
        if (OP == COPY) {
            bad |= take_bit(bits, y);            // a page copied onto itself counts as a destination too
        } else if (OP == FORK) {
            bad |= take_bit(bits, y) || m.length[y] != 0 || !row_ok(m, x);
        } else {
            bad |= take_bit(bits, x) || !row_ok(m, x);
            if (OP == APPEND) bad |= m.length[x] >= m.max_pages;
            if (OP == APPEND && copy_last && m.length[x] > 0) bad |= !page_ok(m, m.table[(int64_t)x * m.max_pages + m.length[x] - 1]);
        }
    }
    bad = __syncthreads_or(bad);
    if (!bad) {
        // Sources are not destinations; the pages of rows to share or release are in use.
        if (OP == FORK || OP == COPY) {
            for (int32_t i = tid; i < n; i += kThreads) {
                const int32_t x = a[i], y = b[i];
                if (x == -1 || y == -1 || (OP == COPY && x == y)) continue;
                bad |= has_bit(bits, x);
            }
        }
        if (OP == FORK || OP == FREE) {
            for (int32_t i = wid; i < n; i += kThreads / 32) {
                const int32_t x = a[i];
                if (x == -1 || (OP == FORK && b[i] == -1)) continue;
                const int32_t len = m.length[x];
                for (int32_t j = lane; j < len; j += 32) bad |= !page_ok(m, m.table[(int64_t)x * m.max_pages + j]);
            }
        }
    }
    bad = __syncthreads_or(bad);
    if (bad) {
        if (tid == 0) latch_error(SSD_ERR_INVALID_ARG);
        return;
    }

    if (OP == FREE) {
        for (int32_t i = wid; i < n; i += kThreads / 32) {
            const int32_t x = a[i];
            if (x == -1) continue;
            int32_t* row = m.table + (int64_t)x * m.max_pages;
            const int32_t len = m.length[x];
            for (int32_t j = lane; j < len; j += 32) {
                atomicSub(&m.refcount[row[j]], 1);
                row[j] = -1;
            }
            __syncwarp();
            if (lane == 0) {
                m.length[x] = 0;
                m.live[x] = -1;
            }
        }
        return;
    }
    if (OP == COPY) {
        int32_t done = 0;
        for (int32_t i0 = 0; i0 < n; i0 += kThreads) {
            const int32_t i = i0 + tid;
            const bool go = i < n && a[i] != -1 && b[i] != -1 && a[i] != b[i];
            int32_t tot;
            const int32_t at = done + block_scan(go, wsum, &tot);
            if (go) {
                mv.src[at] = a[i];
                mv.dst[at] = b[i];
            }
            done += tot;
        }
        if (tid == 0) *mv.count = done;
        return;
    }

    // -------- how many new pages, and which: the lowest free ones
    int32_t need = 0;
    for (int32_t i0 = 0; i0 < n; i0 += kThreads) {
        const int32_t i = i0 + tid;
        const bool go = i < n && a[i] != -1 && (OP == APPEND || (b[i] != -1 && m.length[a[i]] > 0));
        need += __syncthreads_count(go);
    }
    int32_t found = 0;
    for (int32_t p0 = 0; p0 < m.n_pages && found < need; p0 += 4 * kThreads) {
        int32_t free_ = 0;
        const int32_t p = p0 + 4 * tid;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (p + k < m.n_pages && m.refcount[p + k] == 0) free_ |= 1 << k;
        int32_t tot;
        int32_t at = found + block_scan(__popc(free_), wsum, &tot);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (free_ >> k & 1) {
                if (at < need) fresh[at] = p + k;
                ++at;
            }
        found += tot;
    }
    if (found < need) {
        if (tid == 0) latch_error(SSD_ERR_NO_PAGES);
        return;
    }
    __syncthreads();                         // fresh is written

    // -------- the rows: request i takes the next new page in the order of the request
    int32_t done = 0;
    for (int32_t i0 = 0; i0 < n; i0 += kThreads) {
        const int32_t i = i0 + tid;
        const bool go = i < n && a[i] != -1 && (OP == APPEND || (b[i] != -1 && m.length[a[i]] > 0));
        int32_t tot;
        const int32_t at = done + block_scan(go, wsum, &tot);
        if (go) {
            const int32_t x = a[i], row = OP == FORK ? b[i] : x, len = m.length[x], page = fresh[at];
            const int32_t at_row = OP == FORK ? len - 1 : len;
            const bool copied = OP == FORK || (copy_last && len > 0);
            mv.src[at] = copied ? m.table[(int64_t)x * m.max_pages + len - 1] : -1;
            mv.dst[at] = page;
            m.table[(int64_t)row * m.max_pages + at_row] = page;
            m.refcount[page] = 1;
            m.live[row] = page;
            m.length[row] = at_row + 1;
        }
        done += tot;
    }
    if (tid == 0) *mv.count = done;
    if (OP == FORK) {
        // Earlier pages are shared. Parents' rows are not written above (no parent is a
        // child), and a child's entries before its last are written only here.
        for (int32_t i = wid; i < n; i += kThreads / 32) {
            const int32_t x = a[i], y = b[i];
            if (x == -1 || y == -1) continue;
            const int32_t len = m.length[x];
            for (int32_t j = lane; j < len - 1; j += 32) {
                const int32_t p = m.table[(int64_t)x * m.max_pages + j];
                m.table[(int64_t)y * m.max_pages + j] = p;
                atomicAdd(&m.refcount[p], 1);
            }
        }
    }
}

// One block: compaction. Pages in use past the new end move, in ascending order, into the
// free pages before it; remap[p] = where page p is afterwards (-1: it was free), counts =
// {pages in use, pages moved}. The table and live pages are renumbered by the moving grid.
__global__ void __launch_bounds__(kThreads)
k_pages_compact(const Meta m, int32_t* __restrict__ remap, int32_t* __restrict__ counts, const Moves mv) {
    __shared__ int32_t wsum[33];
    const int tid = threadIdx.x;
    constexpr int PER = 4;
    int32_t used = 0;
    for (int32_t p0 = 0; p0 < m.n_pages; p0 += PER * kThreads) {
        int32_t c = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int32_t p = p0 + PER * tid + k;
            c += p < m.n_pages && m.refcount[p] > 0;
        }
        int32_t tot;
        block_scan(c, wsum, &tot);
        used += tot;
    }
    int32_t ndst = 0, nsrc = 0;
    for (int32_t p0 = 0; p0 < m.n_pages; p0 += PER * kThreads) {
        int32_t holes = 0, movers = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int32_t p = p0 + PER * tid + k;
            const bool in = p < m.n_pages, u = in && m.refcount[p] > 0;
            if (in && !u && p < used) holes |= 1 << k;
            if (u && p >= used) movers |= 1 << k;
            if (in) remap[p] = u ? p : -1;
        }
        int32_t tot;
        int32_t d = ndst + block_scan(__popc(holes), wsum, &tot);
        ndst += tot;
        int32_t s = nsrc + block_scan(__popc(movers), wsum, &tot);
        nsrc += tot;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            if (holes >> k & 1) mv.dst[d++] = p0 + PER * tid + k;
            if (movers >> k & 1) mv.src[s++] = p0 + PER * tid + k;
        }
    }
    __syncthreads();                         // src and dst are written; nsrc == ndst
    for (int32_t i = tid; i < nsrc; i += kThreads) {
        const int32_t s = mv.src[i], d = mv.dst[i];
        remap[s] = d;
        m.refcount[d] = m.refcount[s];
        m.refcount[s] = 0;
    }
    if (tid == 0) {
        *mv.count = nsrc;
        counts[0] = used;
        counts[1] = nsrc;
    }
}

// The bytes. A page's bytes in all arrays are cut into tiles of kTile bytes (an array's
// last tile may be short); work item = (move, tile). Reads and writes of one call never
// touch the same page, so the tiles need no order. HBM-bound: 2 bytes of traffic per byte
// moved; a thread has kVec 16-byte loads in flight. 64 pages forked (2.19 GB of traffic): 358 us,
// 6.1 TB/s, 94% of the measured copy rate; the deciding block before it takes about 10 us, bound by the
// latency of its dependent steps.
constexpr int kMoveThreads = 256;
constexpr int kVec = 8;
constexpr int kTile = kMoveThreads * kVec * 16;          // 32 KiB

struct Arrays {
    char* base[kMaxArrays];
    int64_t bytes[kMaxArrays];               // of one page
    int32_t first[kMaxArrays + 1];           // first tile of each array within a page
    int32_t n;
};

template <typename W>
__device__ __forceinline__ void move_tile(char* dst, const char* src, int64_t bytes) {
    const int64_t n = bytes / (int64_t)sizeof(W);
    const W* s = reinterpret_cast<const W*>(src);
    W* d = reinterpret_cast<W*>(dst);
    for (int64_t i0 = 0; i0 < n; i0 += kMoveThreads * kVec) {
        W x[kVec];
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int64_t i = i0 + k * kMoveThreads + threadIdx.x;
            if (i < n) x[k] = __ldcs(s + i);
        }
#pragma unroll
        for (int k = 0; k < kVec; ++k) {
            const int64_t i = i0 + k * kMoveThreads + threadIdx.x;
            if (i < n) __stcs(d + i, x[k]);
        }
    }
}

// remap (compaction): renumber the table and the live pages.
__global__ void __launch_bounds__(kMoveThreads)
k_pages_move(const __grid_constant__ Arrays ar, const Moves mv, const Meta m, const int32_t* __restrict__ remap) {
    const int64_t per = ar.first[ar.n], items = *mv.count * per;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t i = it / per;
        const int32_t tile = (int32_t)(it % per), src = mv.src[i], dst = mv.dst[i];
        if (src < 0) continue;               // a new page that starts without a copy
        int lo = 0, hi = ar.n;               // array of the tile
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (ar.first[mid] <= tile) lo = mid; else hi = mid;
        }
        const int64_t off = (int64_t)(tile - ar.first[lo]) * kTile, bytes = ar.bytes[lo];
        const int64_t todo = bytes - off < kTile ? bytes - off : kTile;
        char* base = ar.base[lo];
        const char* s = base + (int64_t)src * bytes + off;
        char* d = base + (int64_t)dst * bytes + off;
        const uint64_t mix = reinterpret_cast<uint64_t>(base) | (uint64_t)bytes;
        // the widest access that every page of the array is aligned to
        if (mix % 16 == 0) move_tile<uint4>(d, s, todo);
        else if (mix % 4 == 0) move_tile<uint32_t>(d, s, todo);
        else move_tile<uint8_t>(d, s, todo);
    }
    if (remap) {
        const int64_t nt = (int64_t)m.n_rows * m.max_pages, stride = (int64_t)gridDim.x * kMoveThreads;
        for (int64_t i = (int64_t)blockIdx.x * kMoveThreads + threadIdx.x; i < nt + m.n_rows; i += stride) {
            int32_t* e = i < nt ? m.table + i : m.live + (i - nt);
            const int32_t p = *e;
            if (p >= 0 && p < m.n_pages) *e = remap[p];
        }
    }
}

}  // namespace pages
}  // namespace ssd
