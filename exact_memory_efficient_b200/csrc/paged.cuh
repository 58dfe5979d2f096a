// paged.cuh -- how the kernels of the paged key/value cache read a ragged
// batch: packed rows, lengths and page tables, all in device memory.
//
// Nothing in device memory can be checked on the host, so each value is
// brought into range before it is used as an index, and a value that was out
// of range is recorded in the per-device error word (MEA_DEVERR_PAGE): a bad
// table costs wrong results for its sequence, never an access outside the
// caller's buffers, and never a write to a page that the table does not name.
#pragma once

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mea {

// Sequence b of the batch: its rows [q0, q0 + n) of the packed tensors and its
// L cached keys, the n new ones last.
struct Seq {
    int q0, n, L;
};

__device__ __forceinline__ Seq load_seq(const PagedBatch& s, int b) {
    const int lo = s.cu_q ? s.cu_q[b] : 0;
    const int hi = s.cu_q ? s.cu_q[b + 1] : 0;
    const int len = s.kv_len[b];
    const int cap = s.max_pages << s.page_shift;
    Seq r;
    r.q0 = min(max(lo, 0), s.T);
    const int q1 = min(max(hi, r.q0), s.T);
    r.n = q1 - r.q0;
    r.L = min(max(len, 0), cap);
    if (r.q0 != lo || q1 != hi || r.L != len) flag_bad_page();
    return r;
}

// Entry of the sequence's keys [i << page_shift, (i + 1) << page_shift), i < max_pages,
// and the page that it names.  Apart where the entry is asked for ahead of its use.
__device__ __forceinline__ int page_entry(const PagedBatch& s, int b, int i) {
    return s.page_table[(size_t)b * s.max_pages + i];
}
__device__ __forceinline__ int page_of(const PagedBatch& s, int entry, int otherwise = 0) {
    if ((unsigned)entry < (unsigned)s.num_pages) return entry;
    flag_bad_page();
    return otherwise;
}
// For reads: an entry out of range reads page 0.
__device__ __forceinline__ int load_page(const PagedBatch& s, int b, int i) { return page_of(s, page_entry(s, b, i)); }
// For writes: an entry out of range is -1 and nothing is written (page 0 is another sequence's).
__device__ __forceinline__ int page_to_write(const PagedBatch& s, int b, int i) {
    return page_of(s, page_entry(s, b, i), -1);
}

// A tile of 128 keys of bf16 pages in shared memory, as one TMA box per page
// lays it out: groups of 8 keys, in a group the blocks of 64 head dims, in a
// block 8 rows of 128 bytes (128-byte swizzle).  Groups and blocks keep their
// distances from page to page, so a tile of any page size is one operand with
// the same descriptors; a box per page and block, with the blocks 16 KB apart,
// takes twice the TMA instructions.
template <int D>
struct PageTile {
    static constexpr int kGroupBytes = 8 * D * 2;
    static constexpr int kBytes = 128 * D * 2;
    static constexpr uint32_t kHi = desc_hi_sw128(kGroupBytes);
    // K-major operand (K): step kk of 16 head dims, in 16-byte units
    static constexpr uint32_t kmajor(int kk) { return (kk >> 2) * 64u + (kk & 3) * 2u; }
    // MN-major operand (V): blocks of 64 head dims 1 KB apart; step kk of 16 keys
    __device__ static uint32_t mn_lo(unsigned smem_addr) { return (smem_addr >> 4) | (64u << 16); }
    static constexpr uint32_t mnmajor(int kk) { return kk * 2u * (kGroupBytes >> 4); }
    // byte offset of key r, block x
    __device__ static int row(int r, int x) { return (r >> 3) * kGroupBytes + x * 1024 + (r & 7) * 128; }
};

// Packed rows are cut into tiles of `per` rows that start anew with every
// sequence.  Tile x belongs to the sequence b with start(b) <= x < start(b + 1),
// where start(b) = floor(cu_q[b] * mul / per) + b: since
// ceil(n / per) <= floor((c + n) / per) - floor(c / per) + 1, the tiles of
// different sequences never share an x, and a launch needs T * mul / per + B of
// them, which the host knows without the lengths.  Returns b, or -1 when x is
// in front of the first sequence; *tile is the tile's number in its sequence
// (it may lie behind the sequence's end: the caller leaves then).
__device__ __forceinline__ int find_tile(const PagedBatch& s, int x, int mul, int per, int* tile) {
    int lo = 0, hi = s.B - 1;   // the last b whose start is at or below x
    auto start = [&](int b) {
        return (int)((long long)min(max(s.cu_q[b], 0), s.T) * mul / per) + b;
    };
    if (x < start(0)) return -1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (start(mid) <= x) lo = mid;
        else hi = mid - 1;
    }
    *tile = x - start(lo);
    return lo;
}

// The sequence of packed row t (-1: in front of the first or behind the last).
__device__ __forceinline__ int find_row(const PagedBatch& s, int t) {
    if (t < s.cu_q[0] || t >= s.cu_q[s.B]) return -1;
    int lo = 0, hi = s.B - 1;   // the last b with cu_q[b] <= t
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s.cu_q[mid] <= t) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// x / y, and the border of share i of n, of sizes that most often fit 32 bits (a
// division of 64-bit numbers takes some 150 cycles, and shares are found before any work)
__device__ __forceinline__ long long divide(long long x, long long y) {
    return (unsigned long long)(x | y) >> 32 ? x / y : (long long)((unsigned)x / (unsigned)y);
}
__device__ __forceinline__ long long share_begin(long long W, unsigned i, unsigned n) { return divide(W * i, n); }

// The costs of all sequences as one line: calls locate(b, before, cost, W) for
// every b, with the sum of the costs in front of b and of all.  All THREADS
// threads of the block call it; a thread's cost(b) and locate(b, ...) calls
// follow one another, so that cost() may leave what locate() needs.  What locate()
// writes is seen after the block's next barrier.
template <int THREADS, typename Cost, typename Locate>
__device__ __forceinline__ void lay_out_costs(int B, long long (&warp_sum)[THREADS / 32], Cost&& cost, Locate&& locate) {
    const int tid = (int)threadIdx.x;
    const unsigned lane = lane_id(), warp = warp_id();
    // the sum in front of this thread, *all the block's
    auto scan = [&](long long x, long long* all) {
        long long upto = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= (unsigned)o) upto += y;
        }
        if (lane == 31) warp_sum[warp] = upto;
        __syncthreads();
        long long before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) {
            if (w < (int)warp) before += warp_sum[w];
            total += warp_sum[w];
        }
        __syncthreads();
        *all = total;
        return before + upto - x;
    };
    if (B <= 32) {   // one warp's work: no exchange between warps
        if (warp != 0) return;
        const long long mine = (int)lane < B ? cost((int)lane) : 0;
        long long upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= (unsigned)o) upto += y;
        }
        const long long W = __shfl_sync(0xffffffffu, upto, 31);
        if ((int)lane < B) locate((int)lane, upto - mine, mine, W);
        return;
    }
    long long W = 0, mine = 0, before = 0;
    for (int b0 = 0; b0 < B; b0 += THREADS) {
        long long all;
        mine = b0 + tid < B ? cost(b0 + tid) : 0;
        before = scan(mine, &all);
        W += all;
    }
    if (B <= THREADS) {
        if (tid < B) locate(tid, before, mine, W);
    } else {   // a second walk, now that W is known
        long long base = 0;
        for (int b0 = 0; b0 < B; b0 += THREADS) {
            long long all;
            const long long x = b0 + tid < B ? cost(b0 + tid) : 0;
            const long long at = base + scan(x, &all);
            if (b0 + tid < B) locate(b0 + tid, at, x, W);
            base += all;
        }
    }
}

}  // namespace mea
