// paged_evict.cu -- eviction from a paged cache by accumulated attention
// weight.  Of a sequence's L > n_keep cached keys every key/value head keeps
// its n_recent last ones and, of the others, the n_keep - n_recent with the
// largest weights (equal weights: the lower slot first; NaN counts as the
// smallest).  The kept keys, values and weights move, in the order of their
// slots, to the slots 0, 1, ... of the destination pages.
//
// evict_select_kernel, one CTA per (sequence, key/value head): finds the weight
// of the last heavy key by radix selection (8 bits a pass, most significant
// first, over order-preserving integers) and writes the kept slots in order to
// keep_idx, -1 behind them.
// evict_move_kernel: copies.  Into other pages every kept key is independent.
// In place (the destination table is the page table) slot j takes a key from a
// slot >= j, so a CTA that owns some bytes of every key of a head walks over
// the kept keys in rising order, in chunks: it reads chunk c from slots that no
// earlier chunk wrote, waits, and writes slots that no later chunk reads.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mea {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCacheMax = 48 * 1024;   // candidates whose keys are kept in shared memory (192 KB)

// Order-preserving integer of a weight: -0 equals 0, NaN comes last (with -inf).
__device__ __forceinline__ uint32_t order_of(float w) {
    if (isnan(w)) w = -INFINITY;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictArgs a, int cached_max) {
    extern __shared__ uint32_t s_keys[];
    __shared__ unsigned hist[256];
    __shared__ unsigned s_pick[2];
    __shared__ unsigned warp_gt[kSelWarps], warp_eq[kSelWarps];
    const int b = (int)blockIdx.x / a.Hkv;
    const int h = (int)blockIdx.x - b * a.Hkv;
    const int tid = (int)threadIdx.x;
    const unsigned lane = lane_id(), warp = warp_id();
    const Seq sq = load_seq(a.s, b);
    int* out = a.keep_idx + (size_t)blockIdx.x * a.n_keep;
    if (sq.L <= a.n_keep) {   // nothing to evict
        for (int j = tid; j < a.n_keep; j += kSelThreads) out[j] = j < sq.L ? j : -1;
        return;
    }
    const int cand = sq.L - a.n_recent;
    const int heavy = a.n_keep - a.n_recent;   // < cand
    const int mask = (1 << a.s.page_shift) - 1;
    const bool cached = cand <= cached_max;
    auto fetch = [&](int j) {
        const size_t page = (size_t)load_page(a.s, b, j >> a.s.page_shift);
        return order_of(a.weights[((page * a.Hkv + h) << a.s.page_shift) + (j & mask)]);
    };
    auto key_of = [&](int j) { return cached ? s_keys[j] : fetch(j); };
    if (cached)
        for (int j = tid; j < cand; j += kSelThreads) s_keys[j] = fetch(j);

    // the heavy-th largest key: `prefix` holds its digits found so far
    uint32_t prefix = 0;
    unsigned need = (unsigned)heavy;   // of the keys that share the prefix, how many are still to be taken
    if (heavy > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t above = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int j0 = 0; j0 < cand; j0 += kSelThreads) {
                const int j = j0 + tid;
                const uint32_t k = j < cand ? key_of(j) : 0u;
                const bool in = j < cand && (k & above) == prefix;
                const unsigned digit = in ? (k >> shift) & 255u : 256u;
                // lanes with the same digit add once
                const unsigned peers = __match_any_sync(0xffffffffu, digit);
                if (in && (unsigned)(__ffs((int)peers) - 1) == lane) atomicAdd(&hist[digit], (unsigned)__popc(peers));
            }
            __syncthreads();
            if (warp == 0) {
                // digits from the largest down: lane l holds digits 255 - 8l ... 248 - 8l
                unsigned c[8], own = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    c[i] = hist[255 - 8 * (int)lane - i];
                    own += c[i];
                }
                unsigned upto = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
                    if (lane >= (unsigned)o) upto += x;
                }
                unsigned before = upto - own;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (before < need && before + c[i] >= need) {
                        s_pick[0] = 255u - 8u * lane - (unsigned)i;
                        s_pick[1] = need - before;
                    }
                    before += c[i];
                }
            }
            __syncthreads();
            prefix |= s_pick[0] << shift;
            need = s_pick[1];
            __syncthreads();
        }
    }
    // kept: keys above the heavy-th, the first `need` equal to it, and the recent ones
    unsigned base_gt = 0, base_eq = 0;
    for (int j0 = 0; j0 < cand && heavy > 0; j0 += kSelThreads) {
        const int j = j0 + tid;
        const uint32_t k = j < cand ? key_of(j) : 0u;
        const bool gt = j < cand && k > prefix, eq = j < cand && k == prefix;
        const unsigned bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
        if (lane == 0) {
            warp_gt[warp] = (unsigned)__popc(bg);
            warp_eq[warp] = (unsigned)__popc(be);
        }
        __syncthreads();
        unsigned g = base_gt, e = base_eq;
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < (int)warp) {
                g += warp_gt[w];
                e += warp_eq[w];
            }
            base_gt += warp_gt[w];
            base_eq += warp_eq[w];
        }
        const unsigned below = (1u << lane) - 1u;
        g += (unsigned)__popc(bg & below);
        e += (unsigned)__popc(be & below);
        if (gt || (eq && e < need)) out[g + min(e, need)] = j;
        __syncthreads();
    }
    for (int j = tid; j < a.n_recent; j += kSelThreads) out[heavy + j] = cand + j;
}

constexpr int kMoveThreads = 256;

// Slot of kept key j in the destination pages.
__device__ __forceinline__ size_t dst_slot(const EvictArgs& a, int b, int h, int j) {
    const int i = j >> a.s.page_shift;
    int p = i < a.dst_max_pages ? a.dst_table[(size_t)b * a.dst_max_pages + i] : -1;
    if ((unsigned)p >= (unsigned)a.s.num_pages) {
        flag_bad_page();
        return ~(size_t)0;   // not written
    }
    return (((size_t)p * a.Hkv + h) << a.s.page_shift) + (size_t)(j & ((1 << a.s.page_shift) - 1));
}
__device__ __forceinline__ size_t src_slot(const EvictArgs& a, int b, int h, int j) {
    return (((size_t)load_page(a.s, b, j >> a.s.page_shift) * a.Hkv + h) << a.s.page_shift) +
           (size_t)(j & ((1 << a.s.page_shift) - 1));
}

// Into other pages: a group of `lanes` threads (16 bytes each) moves one key of
// K and V; grid (chunks of keys, B * Hkv).
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a, int lanes, int per_cta) {
    const int b = (int)blockIdx.y / a.Hkv;
    const int h = (int)blockIdx.y - b * a.Hkv;
    const int* idx = a.keep_idx + (size_t)blockIdx.y * a.n_keep;
    const int l = (int)threadIdx.x % lanes;
    const int groups = kMoveThreads / lanes;
    const int j1 = min(a.n_keep, ((int)blockIdx.x + 1) * per_cta);
    if ((int)threadIdx.x < groups * lanes) {
        for (int j = (int)blockIdx.x * per_cta + (int)threadIdx.x / lanes; j < j1; j += groups) {
            const int from = idx[j];
            if (from < 0) break;
            const size_t src = src_slot(a, b, h, from), dst = dst_slot(a, b, h, j);
            if (dst == ~(size_t)0) continue;
            const uint4 kx = static_cast<const uint4*>(a.k)[src * lanes + l];
            const uint4 vx = static_cast<const uint4*>(a.v)[src * lanes + l];
            static_cast<uint4*>(a.k)[dst * lanes + l] = kx;
            static_cast<uint4*>(a.v)[dst * lanes + l] = vx;
            if (l == 0) a.weights[dst] = a.weights[src];
        }
    }
    // every (sequence, head) keeps the same number of keys
    if (a.kv_len_out != nullptr && h == 0 && blockIdx.x == 0 && threadIdx.x == 0) {
        int n = 0, hi = a.n_keep;   // first j with idx[j] < 0
        while (n < hi) {
            const int mid = (n + hi) >> 1;
            if (idx[mid] >= 0) n = mid + 1;
            else hi = mid;
        }
        a.kv_len_out[b] = n;
    }
}

// In place: grid (slices of 16 bytes x 4 lanes of K, of V, then the weights; B * Hkv).
constexpr int kSliceLanes = 4;
constexpr int kDepth = 4;   // keys in flight per thread

__global__ void __launch_bounds__(kMoveThreads) evict_shift_kernel(const EvictArgs a, int lanes, int slices) {
    const int b = (int)blockIdx.y / a.Hkv;
    const int h = (int)blockIdx.y - b * a.Hkv;
    const int* idx = a.keep_idx + (size_t)blockIdx.y * a.n_keep;
    const int part = (int)blockIdx.x;
    const bool is_w = part == 2 * slices;
    const int wide = is_w ? 1 : kSliceLanes;
    const int l = (int)threadIdx.x % wide;
    const int lane16 = is_w ? 0 : (part % slices) * kSliceLanes + l;   // 16-byte column of the row
    const bool own = is_w || lane16 < lanes;
    const int groups = kMoveThreads / wide;
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
    if (a.kv_len_out != nullptr && h == 0 && part == 0 && threadIdx.x == 0) {
        int n = 0, hi = a.n_keep;
        while (n < hi) {
            const int mid = (n + hi) >> 1;
            if (idx[mid] >= 0) n = mid + 1;
            else hi = mid;
        }
        a.kv_len_out[b] = n;
    }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, bool bf16, int sm_count, cudaStream_t stream) {
    const long long heads = (long long)a.s.B * a.Hkv;
    if (heads > 65535) return cudaErrorInvalidValue;
    const long long cap = (long long)a.s.max_pages << a.s.page_shift;
    const int cached = (int)(cap < kCacheMax ? cap : kCacheMax);
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCacheMax * 4);
    if (e != cudaSuccess) return e;
    evict_select_kernel<<<(unsigned)heads, kSelThreads, (size_t)cached * 4, stream>>>(a, cached);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int lanes = a.D * (bf16 ? 2 : 4) / 16;
    if (a.in_place) {
        const int slices = (lanes + kSliceLanes - 1) / kSliceLanes;
        evict_shift_kernel<<<dim3((unsigned)(2 * slices + 1), (unsigned)heads), kMoveThreads, 0, stream>>>(a, lanes, slices);
    } else {
        // keys per CTA: enough CTAs for a few waves, at least one key per group of lanes
        const int groups = kMoveThreads / lanes;
        long long per = (long long)a.n_keep * heads / ((long long)sm_count * 16);
        per = per < groups ? groups : (per + groups - 1) / groups * groups;
        const long long chunks = ((long long)a.n_keep + per - 1) / per;
        evict_move_kernel<<<dim3((unsigned)chunks, (unsigned)heads), kMoveThreads, 0, stream>>>(a, lanes, (int)per);
    }
    return cudaGetLastError();
}

}  // namespace mea
