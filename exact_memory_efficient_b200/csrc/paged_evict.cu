// paged_evict.cu -- eviction from a paged cache by accumulated attention
// weight.  Of a sequence's L > n_keep cached keys every key/value head keeps
// its n_recent last ones and, of the others, the n_keep - n_recent with the
// largest weights (equal weights: the lower slot first; NaN counts as the
// smallest).  The kept keys, values and weights move, in the order of their
// slots, to the slots 0, 1, ... of the destination pages.
//
// evict_select_kernel, a cluster of CTAs per (sequence, key/value head): finds
// the weight of the last heavy key by radix selection (8 bits a pass, most
// significant first, over order-preserving integers) and writes the kept slots
// in order to keep_idx, -1 behind them.  Each CTA of a cluster holds a
// contiguous piece of the candidates in shared memory; per pass every CTA reads
// the other CTAs' 256 counts through distributed shared memory and comes to the
// same digit, so one cluster barrier a pass is enough.
// evict_move_kernel: copies.  Into other pages every kept key is independent.
// In place (the destination table is the page table) slot j takes a key from a
// slot >= j, so a CTA that owns some bytes of every key of a head walks over
// the kept keys in rising order, in chunks: it reads chunk c from slots that no
// earlier chunk wrote, waits, and writes slots that no later chunk reads.
#include <cooperative_groups.h>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mea {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCacheMax = 48 * 1024;   // candidates of a CTA that are kept in shared memory (192 KB)
constexpr int kMaxCluster = 8;
constexpr int kLoadBatch = 8;          // weights in flight per thread

// Order-preserving integer of a weight: -0 equals 0, NaN comes last (with -inf).
__device__ __forceinline__ uint32_t order_of(float w) {
    if (isnan(w)) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int cached_max) {
    namespace cg = cooperative_groups;
    extern __shared__ uint32_t s_keys[];
    __shared__ unsigned hist[4][256];           // of this CTA's piece, one per pass
    __shared__ unsigned s_pick[2];
    __shared__ unsigned warp_gt[kSelWarps], warp_eq[kSelWarps];
    __shared__ unsigned s_total[2];             // this CTA's keys above the last heavy one, and equal to it
    cg::cluster_group cluster = cg::this_cluster();
    const unsigned ranks = cluster.num_blocks(), rank = cluster.block_rank();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int head = (int)(blockIdx.x / ranks);
    const int b = head / a.Hkv;
    const int h = head - b * a.Hkv;
    const int tid = (int)threadIdx.x;
    const unsigned lane = lane_id(), warp = warp_id();
    const Seq sq = load_seq(a.s, b);
    int* out = a.keep_idx + (size_t)head * a.n_keep;
    if (sq.L <= a.n_keep) {   // nothing to evict (the same for the whole cluster)
        for (int j = (int)rank * kSelThreads + tid; j < a.n_keep; j += (int)ranks * kSelThreads) out[j] = j < sq.L ? j : -1;
        return;
    }
    const int cand = sq.L - a.n_recent;
    const int heavy = a.n_keep - a.n_recent;   // < cand
    const int mask = (1 << a.s.page_shift) - 1;
    // this CTA's candidates [first, first + n): whole warps' pieces
    const int piece = ((cand + (int)ranks - 1) / (int)ranks + 31) & ~31;
    const int first = min(cand, (int)rank * piece);
    const int n = min(cand, first + piece) - first;
    const bool cached = n <= cached_max;
    auto fetch = [&](int j) {
        const size_t page = (size_t)load_page(a.s, b, (first + j) >> a.s.page_shift);
        return order_of(a.weights[((page * a.Hkv + h) << a.s.page_shift) + ((first + j) & mask)]);
    };
    auto key_of = [&](int j) { return cached ? s_keys[j] : fetch(j); };
    for (int i = tid; i < 4 * 256; i += kSelThreads) hist[i >> 8][i & 255] = 0;
    if (cached) {
        for (int j0 = tid; j0 < n; j0 += kLoadBatch * kSelThreads) {
            uint32_t k[kLoadBatch];
#pragma unroll
            for (int u = 0; u < kLoadBatch; ++u)
                if (j0 + u * kSelThreads < n) k[u] = fetch(j0 + u * kSelThreads);
#pragma unroll
            for (int u = 0; u < kLoadBatch; ++u)
                if (j0 + u * kSelThreads < n) s_keys[j0 + u * kSelThreads] = k[u];
        }
    }
    __syncthreads();

    // the heavy-th largest key: `prefix` holds its digits found so far
    uint32_t prefix = 0;
    unsigned need = (unsigned)heavy;   // of the keys that share the prefix, how many are still to be taken
    for (int pass = 0; pass < 4 && heavy > 0; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (shift + 8);
        for (int j0 = 0; j0 < n; j0 += kSelThreads) {
            const int j = j0 + tid;
            const uint32_t k = j < n ? key_of(j) : 0u;
            const bool in = j < n && (k & above) == prefix;
            const unsigned digit = in ? (k >> shift) & 255u : 256u;
            // a warp whose keys all share a digit (a cache of equal weights) adds
            // once; otherwise every lane adds: grouping equal digits first
            // (__match_any_sync) took longer than the collisions it saves, 2.4 us
            // of the 128 heads' 20
            const bool same = __all_sync(0xffffffffu, digit == __shfl_sync(0xffffffffu, digit, 0));
            if (in && (!same || lane == 0)) atomicAdd(&hist[pass][digit], same ? 32u : 1u);
        }
        cluster.sync();
        // digits from the largest down, one per thread: the cluster's count, and the
        // counts in front of it
        unsigned c = 0, upto = 0;
        if (tid < 256) {
#pragma unroll
            for (unsigned r = 0; r < kMaxCluster; ++r)
                if (r < ranks) c += cluster.map_shared_rank(&hist[pass][0], r)[255 - tid];
            upto = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
                if (lane >= (unsigned)o) upto += x;
            }
            if (lane == 31) warp_gt[warp] = upto;
        }
        __syncthreads();
        if (tid < 256) {
            unsigned before = upto - c;
            for (unsigned w = 0; w < warp; ++w) before += warp_gt[w];
            if (before < need && before + c >= need) {
                s_pick[0] = 255u - (unsigned)tid;
                s_pick[1] = need - before;
            }
        }
        __syncthreads();
        prefix |= s_pick[0] << shift;
        need = s_pick[1];
        __syncthreads();
    }
    // kept: keys above the heavy-th, the first `need` equal to it, and the recent
    // ones.  Every warp takes a contiguous run of the CTA's piece: it counts, the
    // counts in front of it are added up, and it writes.
    const int run = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int j_begin = min(n, (int)warp * run), j_end = min(n, j_begin + run);
    unsigned gt_mine = 0, eq_mine = 0;
    if (heavy > 0) {
        for (int j0 = j_begin; j0 < j_end; j0 += 32) {
            const int j = j0 + (int)lane;
            const uint32_t k = j < j_end ? key_of(j) : 0u;
            gt_mine += (unsigned)__popc(__ballot_sync(0xffffffffu, j < j_end && k > prefix));
            eq_mine += (unsigned)__popc(__ballot_sync(0xffffffffu, j < j_end && k == prefix));
        }
    }
    if (lane == 0) {
        warp_gt[warp] = gt_mine;
        warp_eq[warp] = eq_mine;
    }
    __syncthreads();
    unsigned g = 0, e = 0;
    {
        const unsigned x = warp_gt[lane], y = warp_eq[lane];
        const unsigned gt_all = __reduce_add_sync(0xffffffffu, x), eq_all = __reduce_add_sync(0xffffffffu, y);
        g = __reduce_add_sync(0xffffffffu, lane < warp ? x : 0u);
        e = __reduce_add_sync(0xffffffffu, lane < warp ? y : 0u);
        if (tid == 0) {
            s_total[0] = gt_all;
            s_total[1] = eq_all;
        }
    }
    cluster.sync();
    for (unsigned r = 0; r < rank; ++r) {
        const unsigned* other = cluster.map_shared_rank(&s_total[0], r);
        g += other[0];
        e += other[1];
    }
    if (heavy > 0) {
        for (int j0 = j_begin; j0 < j_end; j0 += 32) {
            const int j = j0 + (int)lane;
            const uint32_t k = j < j_end ? key_of(j) : 0u;
            const bool gt = j < j_end && k > prefix, eq = j < j_end && k == prefix;
            const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
            const unsigned below = (1u << lane) - 1u;
            const unsigned gg = g + (unsigned)__popc(bg & below), ee = e + (unsigned)__popc(be & below);
            if (gt || (eq && ee < need)) out[gg + min(ee, need)] = first + j;
            g += (unsigned)__popc(bg);
            e += (unsigned)__popc(be);
        }
    }
    for (int j = (int)rank * kSelThreads + tid; j < a.n_recent; j += (int)ranks * kSelThreads) out[heavy + j] = cand + j;
    cluster.sync();   // no CTA leaves while another reads its memory
}

constexpr int kMoveThreads = 128;

// Slot of kept key j in the destination pages.  Into other pages, one that is the
// sequence's own page at the same place (the table's contents under another
// pointer) would be overwritten while it is read: reported, not written.
__device__ __forceinline__ size_t dst_slot(const EvictArgs& a, int b, int h, int j) {
    const int i = j >> a.s.page_shift;
    int p = i < a.dst_max_pages ? a.dst_table[(size_t)b * a.dst_max_pages + i] : -1;
    if ((unsigned)p >= (unsigned)a.s.num_pages ||
        (!a.in_place && i < a.s.max_pages && a.s.page_table[(size_t)b * a.s.max_pages + i] == p)) {
        flag_bad_page();
        return ~(size_t)0;   // not written
    }
    return (((size_t)p * a.Hkv + h) << a.s.page_shift) + (size_t)(j & ((1 << a.s.page_shift) - 1));
}
__device__ __forceinline__ size_t src_slot(const EvictArgs& a, int b, int h, int j) {
    return (((size_t)load_page(a.s, b, j >> a.s.page_shift) * a.Hkv + h) << a.s.page_shift) +
           (size_t)(j & ((1 << a.s.page_shift) - 1));
}

// Into other pages: a group of `lanes` threads (16 bytes each) moves kMoveDepth
// keys of K and V at a time; grid (chunks of keys, B * Hkv).  Small CTAs with
// two keys per thread in flight carry most (128 heads of 2048 keys, 268 MB: 53 us
// with 256 threads and four keys, 46 with 128 and two; 69 with eight).
constexpr int kMoveDepth = 2;

__device__ __forceinline__ void write_length(const EvictArgs& a, int b, const int* idx) {
    int n = 0, hi = a.n_keep;   // first j with idx[j] < 0; every head keeps the same number
    while (n < hi) {
        const int mid = n + ((hi - n) >> 1);
        if (idx[mid] >= 0) n = mid + 1;
        else hi = mid;
    }
    a.kv_len_out[b] = n;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int lanes, int per_cta) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = (int)blockIdx.y / a.Hkv;
    const int h = (int)blockIdx.y - b * a.Hkv;
    const int* idx = a.keep_idx + (size_t)blockIdx.y * a.n_keep;
    const int l = (int)threadIdx.x % lanes;
    const int groups = kMoveThreads / lanes;
    const int j1 = (int)min((long long)a.n_keep, ((long long)blockIdx.x + 1) * per_cta);
    if ((int)threadIdx.x < groups * lanes) {
        for (int j0 = (int)blockIdx.x * per_cta + (int)threadIdx.x / lanes; j0 < j1; j0 += kMoveDepth * groups) {
            int from[kMoveDepth];
            size_t src[kMoveDepth], dst[kMoveDepth];
            uint4 kx[kMoveDepth], vx[kMoveDepth];
            float wx[kMoveDepth];
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) from[u] = j0 + u * groups < j1 ? idx[j0 + u * groups] : -1;
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) {
                if (from[u] < 0) continue;
                src[u] = src_slot(a, b, h, from[u]);
                dst[u] = dst_slot(a, b, h, j0 + u * groups);
            }
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) {
                if (from[u] < 0) continue;
                kx[u] = static_cast<const uint4*>(a.k)[src[u] * lanes + l];
                vx[u] = static_cast<const uint4*>(a.v)[src[u] * lanes + l];
                if (l == 0) wx[u] = a.weights[src[u]];
            }
#pragma unroll
            for (int u = 0; u < kMoveDepth; ++u) {
                if (from[u] < 0 || dst[u] == ~(size_t)0) continue;
                static_cast<uint4*>(a.k)[dst[u] * lanes + l] = kx[u];
                static_cast<uint4*>(a.v)[dst[u] * lanes + l] = vx[u];
                if (l == 0) a.weights[dst[u]] = wx[u];
            }
        }
    }
    if (a.kv_len_out != nullptr && h == 0 && blockIdx.x == 0 && threadIdx.x == 0) write_length(a, b, idx);
}

// In place: grid (slices of 16 bytes x 4 lanes of K, of V, then the weights; B * Hkv).
constexpr int kShiftThreads = 256;
constexpr int kSliceLanes = 4;
constexpr int kDepth = 4;   // keys in flight per thread

__global__ void __launch_bounds__(kShiftThreads) evict_shift_kernel(const EvictArgs a, int lanes, int slices) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int b = (int)blockIdx.y / a.Hkv;
    const int h = (int)blockIdx.y - b * a.Hkv;
    const int* idx = a.keep_idx + (size_t)blockIdx.y * a.n_keep;
    const int part = (int)blockIdx.x;
    const bool is_w = part == 2 * slices;
    const int wide = is_w ? 1 : kSliceLanes;
    const int l = (int)threadIdx.x % wide;
    const int lane16 = is_w ? 0 : (part % slices) * kSliceLanes + l;   // 16-byte column of the row
    const bool own = is_w || lane16 < lanes;
    const int groups = kShiftThreads / wide;
    const int g = (int)threadIdx.x / wide;
    uint4* rows = static_cast<uint4*>(part < slices ? a.k : a.v);
    for (int j0 = 0; j0 < a.n_keep; j0 += groups * kDepth) {
        if (idx[j0] < 0) break;
        uint4 x[kDepth];
        float w[kDepth];
        int from[kDepth];
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            const int j = j0 + u * groups + g;
            from[u] = j < a.n_keep && own ? idx[j] : -1;
            if (from[u] == j) from[u] = -1;   // already there
            if (from[u] < 0) continue;
            const size_t src = src_slot(a, b, h, from[u]);
            if (is_w) w[u] = a.weights[src];
            else x[u] = rows[src * lanes + lane16];
        }
        __syncthreads();   // the chunk is read before any of it is overwritten
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
            const int j = j0 + u * groups + g;
            if (from[u] < 0) continue;
            const size_t dst = dst_slot(a, b, h, j);
            if (dst == ~(size_t)0) continue;
            if (is_w) a.weights[dst] = w[u];
            else rows[dst * lanes + lane16] = x[u];
        }
    }
    if (a.kv_len_out != nullptr && h == 0 && part == 0 && threadIdx.x == 0) write_length(a, b, idx);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, bool bf16, int sm_count, cudaStream_t stream) {
    const long long heads = (long long)a.s.B * a.Hkv;
    if (heads > 65535) return cudaErrorInvalidValue;
    const long long cap = (long long)a.s.max_pages << a.s.page_shift;
    // CTAs per head: as many as the device holds at once, while each has a
    // thousand candidates to look at (8 heads of 16384 keys: 52 us with one, 15 us
    // with eight)
    int ranks = 1;
    while (ranks < kMaxCluster && heads * ranks * 2 <= sm_count && cap >= (long long)ranks * 2 * 1024) ranks *= 2;
    const long long piece = ((cap + ranks - 1) / ranks + 31) & ~31LL;
    const int cached = (int)(piece < kCacheMax ? piece : kCacheMax);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheMax * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(heads * ranks));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)cached * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    if ((e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, cached)) != cudaSuccess) return e;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int lanes = a.D * (bf16 ? 2 : 4) / 16;
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    if (a.in_place) {
        const int slices = (lanes + kSliceLanes - 1) / kSliceLanes;
        cfg.blockDim = dim3(kShiftThreads);
        cfg.gridDim = dim3((unsigned)(2 * slices + 1), (unsigned)heads);
        e = cudaLaunchKernelEx(&cfg, evict_shift_kernel, a, lanes, slices);
    } else {
        // keys per CTA: a whole batch for every group of lanes, and enough CTAs for a few waves
        const int batch = kMoveThreads / lanes * kMoveDepth;
        long long per = (long long)a.n_keep * heads / ((long long)sm_count * 16);
        per = per < batch ? batch : (per + batch - 1) / batch * batch;
        cfg.gridDim = dim3((unsigned)(((long long)a.n_keep + per - 1) / per), (unsigned)heads);
        e = cudaLaunchKernelEx(&cfg, evict_move_kernel, a, lanes, (int)per);
    }
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace mea
