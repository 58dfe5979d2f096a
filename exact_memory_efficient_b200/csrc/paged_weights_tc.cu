// paged_weights_tc.cu -- the attention weight that every cached key receives
// from the rows of one call, bf16 on the tensor cores (definition and order as
// in paged_weights.cu).
//
// S^T = K Q^T puts the keys on TMEM lanes, so a thread owns one key and adds up
// its columns exp2(c s - lse log2 e) in a register: no maximum, no exchange.
// The rows that see a key are those from its own token on, so the mask is one
// first column per key.
//
// Work.  An item is 256 keys (two key tiles) of one key/value head; its units
// are the query tiles (tt tokens, tt * G <= 128 rows) from the first token that
// sees the item's first key.  As in paged_tc.cu every CTA of one launch takes
// an equal share of all units and finds it itself.  With `split` a share may
// begin and end inside an item, whose sums then go to the CTA's first or second
// workspace slot, to be added in order by weights_merge_kernel; without it (one
// query tile per item: decode) a CTA takes the items that begin in its share.
//
// Roles: warp 0 TMA producer of K (a pair of tiles per item), the last warp of Q (a
// tile per unit, with its rows' lse), warp 1 MMA issuer; of the two key tiles each
// has eight warps, four for the first 64 columns of every unit and four for the
// others, whose sums are added at the item's end (four warps with few rows).
// TMEM: two score buffers of 128 columns per key tile.
//
// Rounding: exp2 is the approximate instruction (2^-22 relative), sums are fp32, 16
// running ones per key (8 with few rows) and their sum at the item's end.
//
// Bound: decode reads K once (HBM); with many rows one exponential per score
// binds (16 per clock and SM), the tensor cores need half that time.  With four
// warps per key tile every warp waited for the same barriers at the same time
// and the exponential unit idled meanwhile.
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mea {
namespace {

constexpr int kTile = 128;
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned long long kUnitLimitNs = 16000;   // of a unit, some ten times what it takes at low clocks

// FEW: at most kFewRows rows per query tile (decode).  Q then takes 2 KB per 64
// head dims and the space goes to K: three pairs in flight instead of two at
// D = 128 (six at D = 64), since decode is bound by the bytes in flight.
constexpr int kFewRows = 16;
constexpr int kMaxPairs = 6;

template <int D, bool FEW>
struct Cfg {
    static constexpr int kHalves = FEW ? 1 : 2;                      // warps per 32 keys
    static constexpr int kQWarp = 2 + 8 * kHalves;
    static constexpr int kThreads = 32 * (kQWarp + 1);
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kQBox = FEW ? kFewRows * 128 : 128 * 128;   // 64 head dims of a query tile
    static constexpr int kQBytes = D / 64 * kQBox;
    static constexpr int kPairs = FEW ? (D == 128 ? 3 : 6) : 2;      // K pairs in flight
    static constexpr int kQStages = D == 128 && !FEW ? 2 : 4;
    static constexpr int kSmemData = 2 * kPairs * kTileBytes + kQStages * kQBytes;
    static constexpr int kLseBytes = kQStages * kTile * 4;
    static constexpr int kSumBytes = 2 * kTile * 4;          // the second halves' sums; before, the warps' costs
    static constexpr int kSmemBytes = kSmemData + kLseBytes + kSumBytes + 1024 /*barriers*/ + 1024 /*alignment slack*/;
    static_assert(kSmemBytes <= 227 * 1024 && kPairs <= kMaxPairs, "shared memory");
};

struct Barriers {
    uint64_t k_full[kMaxPairs], k_empty[kMaxPairs];
    uint64_t q_full[4], q_empty[4];
    uint64_t s_full[2][2], s_free[2][2];   // [key tile][buffer]
    uint64_t sum_full[8], sum_free[8];     // [key tile, quarter of it]
    uint64_t drain;
    unsigned tmem_base;
    int abort_flag;
    // this CTA's share: where it begins, and its units
    struct Share {
        Seq sq;
        int b, h, i, u0;
        long long units;
    } share;
};

__device__ __forceinline__ int q_tiles(const Seq& sq, int tt) { return (sq.n + tt - 1) / tt; }
__device__ __forceinline__ int items_of(const Seq& sq) { return sq.n > 0 ? (sq.L + 2 * kTile - 1) / (2 * kTile) : 0; }
// first query tile of item i: the one of the first token that sees key 256 i
__device__ __forceinline__ int first_tile(const Seq& sq, int tt, int i) {
    const int first = i * 2 * kTile - (sq.L - sq.n);
    return first < tt ? 0 : first / tt;
}
__device__ __forceinline__ int units_of(const Seq& sq, int tt, int i) { return q_tiles(sq, tt) - first_tile(sq, tt, i); }
// items that every query tile sees
__device__ __forceinline__ int full_items(const Seq& sq) {
    return sq.L < sq.n ? 0 : min(items_of(sq), (sq.L - sq.n) / (2 * kTile) + 1);
}

struct Walk {
    Seq sq;
    int b, h, i, items;
    int u0, u1, n_units;
    long long left;
    bool first, split;

    __device__ __forceinline__ void begin(const PagedWeightsTcArgs& a, const Barriers* bars) {
        sq = bars->share.sq;
        b = bars->share.b;
        h = bars->share.h;
        i = bars->share.i;
        u0 = bars->share.u0;
        left = bars->share.units;
        first = true;
        split = a.split;
        if (left <= 0) return;
        items = items_of(sq);
        n_units = units_of(sq, a.tt, i);
        u1 = split ? (int)min((long long)n_units, u0 + left) : n_units;
        if (!split && u0 > 0) next(a);   // the item belongs to the CTA in front
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const PagedWeightsTcArgs& a) {
        left -= u1 - u0;
        first = false;
        if (left <= 0) return;
        if (++i == items) {
            i = 0;
            if (++h == a.Hkv) {
                h = 0;
                do {
                    ++b;
                    if (b >= a.s.B) {
                        left = 0;
                        return;
                    }
                    sq = load_seq(a.s, b);
                    items = items_of(sq);
                } while (items == 0);
            }
        }
        n_units = units_of(sq, a.tt, i);
        u0 = 0;
        u1 = split ? (int)min((long long)n_units, left) : n_units;
    }
    __device__ __forceinline__ bool whole() const { return u0 == 0 && u1 == n_units; }
    __device__ __forceinline__ bool two() const { return i * 2 * kTile + kTile < sq.L; }   // the second key tile has keys
};

template <int THREADS>
__device__ __forceinline__ void find_share(const PagedWeightsTcArgs& a, Barriers* bars, long long (&warp_sum)[THREADS / 32]) {
    if (threadIdx.x == 0) bars->share.units = 0;
    __syncthreads();
    Seq sq;
    auto cost = [&](int b) {
        sq = load_seq(a.s, b);
        const int items = items_of(sq), full = full_items(sq);
        long long sum = (long long)full * q_tiles(sq, a.tt);
        for (int i = full; i < items; ++i) sum += units_of(sq, a.tt, i);
        return sum * a.Hkv;
    };
    auto locate = [&](int b, long long before, long long sum, long long W) {
        const long long w0 = share_begin(W, blockIdx.x, gridDim.x), w1 = share_begin(W, blockIdx.x + 1, gridDim.x);
        if (w0 < before || w0 >= before + sum || w1 <= w0) return;
        const int items = items_of(sq), full = full_items(sq), nq = q_tiles(sq, a.tt);   // sq is b's since cost(b)
        const long long per_head = divide(sum, a.Hkv);
        long long x = w0 - before;
        Barriers::Share& at = bars->share;
        at.units = w1 - w0;
        at.sq = sq;
        at.b = b;
        at.h = (int)divide(x, per_head);
        x -= at.h * per_head;
        int i = (int)min((long long)full, divide(x, nq));
        x -= (long long)i * nq;
        for (; i >= full && i + 1 < items; ++i) {
            const int n = units_of(sq, a.tt, i);
            if (x < n) break;
            x -= n;
        }
        at.i = i;
        at.u0 = (int)x;
    };
    lay_out_costs<THREADS>(a.s.B, warp_sum, cost, locate);
    __syncthreads();
}

// Pairs of fp32 in one instruction each, every lane rounded as fmaf and a sum.
__device__ __forceinline__ void scale_pair(float& d0, float& d1, float x0, float x1, float c, float a0, float a1) {
    asm("{\n\t.reg .b64 px, pc, pa, pd;\n\t"
        "mov.b64 px, {%2, %3};\n\t"
        "mov.b64 pc, {%4, %4};\n\t"
        "mov.b64 pa, {%5, %6};\n\t"
        "fma.rn.f32x2 pd, px, pc, pa;\n\t"
        "mov.b64 {%0, %1}, pd;\n\t}"
        : "=f"(d0), "=f"(d1)
        : "f"(x0), "f"(x1), "f"(c), "f"(a0), "f"(a1));
}
__device__ __forceinline__ void add_pair(float& d0, float& d1, float x0, float x1) {
    asm("{\n\t.reg .b64 px, pd;\n\t"
        "mov.b64 px, {%2, %3};\n\t"
        "mov.b64 pd, {%0, %1};\n\t"
        "add.rn.f32x2 pd, pd, px;\n\t"
        "mov.b64 {%0, %1}, pd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(x0), "f"(x1));
}

// Slot of key `key` of head h in weights, in page `page`.
__device__ __forceinline__ size_t weight_at(const PagedBatch& s, int Hkv, int page, int h, int key) {
    return (((size_t)page * Hkv + h) << s.page_shift) + (key & ((1 << s.page_shift) - 1));
}

template <int D, bool FEW>
__global__ void __launch_bounds__(Cfg<D, FEW>::kThreads, 1)
paged_weights_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const PagedWeightsTcArgs a) {
    using C = Cfg<D, FEW>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sK = smem;                                       // [pair][key tile]
    uint8_t* sQ = smem + 2 * C::kPairs * C::kTileBytes;
    float* sLse = reinterpret_cast<float*>(smem + C::kSmemData);   // [Q stage][row], times -log2 e
    float* sSum = reinterpret_cast<float*>(smem + C::kSmemData + C::kLseBytes);
    Barriers* bars = reinterpret_cast<Barriers*>(smem + C::kSmemData + C::kLseBytes + C::kSumBytes);
    static_assert(sizeof(Barriers) <= 1024, "shared memory");
    const unsigned warp = warp_id();
    const unsigned lane = lane_id();
    const int tt = a.tt;
    const int G = a.H / a.Hkv;

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::kPairs; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            for (int j = 0; j < 2; ++j) {
                mbar_init(&bars->s_full[i][j], 1);
                mbar_init(&bars->s_free[i][j], 128 * C::kHalves);
            }
        }
        for (int i = 0; i < C::kQStages; ++i) {
            mbar_init(&bars->q_full[i], 2);    // the copies, and the rows' lse
            mbar_init(&bars->q_empty[i], 1 + 256 * C::kHalves);   // both MMAs, and the readers of lse
        }
        for (int i = 0; i < 8; ++i) {
            mbar_init(&bars->sum_full[i], 32);
            mbar_init(&bars->sum_free[i], 32);
        }
        mbar_init(&bars->drain, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&bars->tmem_base, 512);
        tmem_relinquish();
        if (lane == 0) {   // kernel parameters: no need to wait for the kernel in front
            prefetch_tmap(&tm_q);
            prefetch_tmap(&tm_k);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort_flag;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_share<C::kThreads>(a, bars, *reinterpret_cast<long long(*)[C::kThreads / 32]>(sSum));

    Walk w;
    w.begin(a, bars);
    if (warp == 0) {
        // ------------------------------------------------ producer
        if (lane == 0 && a.split) {
            a.parts[2 * blockIdx.x].n_kv = 0;
            a.parts[2 * blockIdx.x + 1].n_kv = 0;
        }
        const int shift = a.s.page_shift;
        const int box_rows = min(kTile, 1 << shift);
        const int my_row = (int)lane * box_rows;         // first key of the lane's box in the tile
        const bool mine = my_row < kTile;
        const int outside = a.s.num_pages * a.Hkv;
        int li = 0;                 // items asked for
        bool ok = true;
        // K comes an item ahead, and a pair is free when all units of its item are
        // done: about 1 us each, so that a million query tiles take the whole limit
        // of a wait.  It grows with the longest item so far.
        int longest = 0;
        auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
            const int got = lane != 0 || mbar_wait(bar, parity, abort_flag, kWaitLimitNs + longest * kUnitLimitNs);
            return __shfl_sync(0xffffffffu, got, 0) != 0;
        };
        // page coordinates of the lane's boxes in an item's two key tiles, looked up
        // an item ahead: a lookup takes about half as long as the item's K
        int z[2] = {outside, outside}, z_next[2];
        auto look_up = [&](const Walk& x, int (&at)[2]) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int key = (2 * x.i + t) * kTile + my_row;
                at[t] = mine && key < x.sq.L ? load_page(a.s, x.b, key >> shift) * a.Hkv + x.h : outside;
            }
        };
        if (!w.done()) look_up(w, z);
        while (ok && !w.done()) {
            const int ks = li % C::kPairs;
            const int n_kt = w.two() ? 2 : 1;
            if (li >= C::kPairs && !(ok = wait(&bars->k_empty[ks], (li / C::kPairs - 1) & 1))) break;
            if (lane == 0) {
                if (!w.whole()) {
                    PagedPart& p = a.parts[2 * blockIdx.x + (w.first ? 0 : 1)];
                    p.b = w.b;
                    p.h = w.h;
                    p.i = w.i;
                    p.t0 = w.u0;
                    p.t1 = w.u1;
                    p.n_kv = w.n_units;
                }
                mbar_arrive_expect_tx(&bars->k_full[ks], (unsigned)(n_kt * C::kTileBytes));
            }
            __syncwarp();
            if (mine) {
                const int group = ((2 * w.i * kTile + my_row) & ((1 << shift) - 1)) >> 3;
                tma_load_5d(sK + 2 * ks * C::kTileBytes + PageTile<D>::row(my_row, 0), &tm_k, &bars->k_full[ks], 0, 0, 0,
                            group, z[0]);
                if (n_kt == 2)
                    tma_load_5d(sK + (2 * ks + 1) * C::kTileBytes + PageTile<D>::row(my_row, 0), &tm_k,
                                &bars->k_full[ks], 0, 0, 0,
                                (((2 * w.i + 1) * kTile + my_row) & ((1 << shift) - 1)) >> 3, z[1]);
            }
            longest = max(longest, w.u1 - w.u0);
            Walk ahead = w;
            ahead.next(a);
            if (!ahead.done()) look_up(ahead, z_next);
            ++li;
            w = ahead;
            z[0] = z_next[0];
            z[1] = z_next[1];
        }
        // never leave with copies in flight
        for (int i = li > C::kPairs ? li - C::kPairs : 0; i < li; ++i)
            mbar_wait(&bars->k_full[i % C::kPairs], (i / C::kPairs) & 1, nullptr);
    } else if (warp == C::kQWarp) {
        // ------------------------------------------------ Q and its rows' lse
        int qc = 0;                 // tiles asked for
        bool ok = true;
        auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
            const int got = lane != 0 || mbar_wait(bar, parity, abort_flag);
            return __shfl_sync(0xffffffffu, got, 0) != 0;
        };
        // the lane's four rows of a tile: token, and place in [token, head] lse
        int tok[4], at[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int row = 32 * e + (int)lane;
            tok[e] = row < tt * G ? row / G : 1 << 30;
            at[e] = row / G * a.H + row % G;
        }
        for (; ok && !w.done(); w.next(a)) {
            const int f = first_tile(w.sq, tt, w.i);
            for (int u = w.u0; ok && u < w.u1; ++u) {
                const int s = qc % C::kQStages;
                const int tok0 = (f + u) * tt;
                const float* rows = a.lse + (size_t)(w.sq.q0 + tok0) * a.H + w.h * G;
                float ls[4];        // loaded while the stage drains
#pragma unroll
                for (int e = 0; e < 4; ++e) ls[e] = tok[e] < w.sq.n - tok0 ? rows[at[e]] * -kLog2e : 0.f;
                if (qc >= C::kQStages && !(ok = wait(&bars->q_empty[s], (qc / C::kQStages - 1) & 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&bars->q_full[s], (unsigned)(G * tt * D * 2));
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_3d(sQ + s * C::kQBytes + x * C::kQBox, &tm_q, &bars->q_full[s], x * 64, w.h * G,
                                    w.sq.q0 + tok0);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) sLse[s * kTile + 32 * e + (int)lane] = ls[e];
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->q_full[s]);
                ++qc;
            }
        }
        for (int c = qc > C::kQStages ? qc - C::kQStages : 0; c < qc; ++c)
            mbar_wait(&bars->q_full[c % C::kQStages], (c / C::kQStages) & 1, nullptr);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            const unsigned idesc = make_idesc_bf16(128, (unsigned)((tt * G + 15) / 16 * 16), 0, 0);
            const uint32_t k_lo = desc_lo_kmajor(smem_u32(sK));
            const uint32_t q_lo = desc_lo_kmajor(smem_u32(sQ));
            constexpr uint32_t kStep = C::kTileBytes >> 4;
            bool ok = true;
            int li = 0, qc = 0;
            int cnt0 = 0, cnt1 = 0;   // units of each key tile: buffer and phase of s_full / s_free
            for (; ok && !w.done(); w.next(a), ++li) {
                const int ks = li % C::kPairs;
                const bool two = w.two();
                if (!(ok = mbar_wait(&bars->k_full[ks], (li / C::kPairs) & 1, abort_flag))) break;
                for (int u = w.u0; ok && u < w.u1; ++u, ++qc) {
                    const int s = qc % C::kQStages;
                    if (!(ok = mbar_wait(&bars->q_full[s], (qc / C::kQStages) & 1, abort_flag))) break;
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t == 1 && !two) break;
                        const int cnt = t ? cnt1 : cnt0;
                        const int buf = cnt & 1;
                        if (cnt >= 2 && !(ok = mbar_wait(&bars->s_free[t][buf], ((cnt >> 1) - 1) & 1, abort_flag))) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_ss_desc(tmem + (unsigned)(t * 256 + buf * 128),
                                        k_lo + (2 * ks + t) * kStep + PageTile<D>::kmajor(kk), PageTile<D>::kHi,
                                        q_lo + s * (C::kQBytes >> 4) + (kk >> 2) * (C::kQBox >> 4) + (kk & 3) * 2, kDescHiSw128, idesc, kk > 0);
                        mma_commit(&bars->s_full[t][buf]);
                        if (t) ++cnt1; else ++cnt0;
                    }
                    if (!ok) break;
                    mma_commit(&bars->q_empty[s]);
                }
                if (ok) mma_commit(&bars->k_empty[ks]);
            }
            mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, nullptr);
        }
    } else {
        // ------------------------------------------------ one or two threads per key
        const int t = ((warp - 2) >> 2) & 1;               // key tile
        const int half = (int)(warp - 2) >> 3;             // columns [64 half, 64 half + 64) of every unit
        const unsigned sub = warp & 3;
        const int r = (int)sub * 32 + (int)lane;
        const unsigned tS = tmem + ((sub * 32u) << 16) + (unsigned)(t * 256 + half * 64);
        const float c_log2 = a.scale * kLog2e;
        // a wait that gives up does so for the whole warp: the code behind it is collective
        auto wait_all = [&](uint64_t* bar, unsigned parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        };
        bool ok = true;
        int cnt = 0, qc = 0;
        for (int li = 0; ok && !w.done(); w.next(a), ++li) {
            const int key = (2 * w.i + t) * kTile + r;
            const bool work = t == 0 || w.two();
            const bool whole = w.whole();
            // the key's page, looked up while the tiles arrive and not used before the end
            const bool mine = half == 0 && key < w.sq.L;
            const int page = mine && whole ? page_to_write(a.s, w.b, key >> a.s.page_shift) : -1;
            [[maybe_unused]] float old = 0.f;
            const int f = first_tile(w.sq, tt, w.i);
            const int seen = w.sq.L - w.sq.n;
            float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
            for (int u = w.u0; u < w.u1; ++u, ++qc) {
                const int s = qc % C::kQStages;
                if (!(ok = wait_all(&bars->q_full[s], (qc / C::kQStages) & 1))) break;
                // decode, an item a unit: the weight before, asked for ahead of the wait for the scores
                if constexpr (FEW)
                    if (u == w.u0 && page >= 0) old = a.weights[weight_at(a.s, a.Hkv, page, w.h, key)];
                if (!work) {
                    mbar_arrive(&bars->q_empty[s]);
                    continue;
                }
                const int buf = cnt & 1;
                if (!(ok = wait_all(&bars->s_full[t][buf], (cnt >> 1) & 1))) break;
                ++cnt;
                tc_fence_after();
                const int tok0 = (f + u) * tt;
                // this half's rows, the first one that sees this key, and whether
                // some lane of the warp masks any
                const int rows = min(tt, w.sq.n - tok0) * G - half * 64;
                const int first = max(0, key - seen - tok0) * G - half * 64;
                const bool masked = key - (int)lane + 31 - seen - tok0 > 0;
                const float* ls = sLse + s * kTile + half * 64;
                if constexpr (FEW) {
                    uint32_t x[16];
                    tmem_ld16(tS + buf * 128, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < kFewRows; ++i) {
                        if (i >= rows) break;
                        const float p = ex2_approx(fmaf(__uint_as_float(x[i]), c_log2, ls[i]));
                        if (i >= first) sum[i & 7] += p;
                    }
                } else {
#pragma unroll 1
                for (int c0 = 0; c0 < min(rows, 64); c0 += 32) {
                    uint32_t x[32];
                    tmem_ld32(tS + buf * 128 + c0, x);
                    tmem_wait_ld();
                    if (!masked && c0 + 32 <= rows) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            const float4 l4 = *reinterpret_cast<const float4*>(ls + c0 + i);
                            float p0, p1, p2, p3;
                            scale_pair(p0, p1, __uint_as_float(x[i]), __uint_as_float(x[i + 1]), c_log2, l4.x, l4.y);
                            scale_pair(p2, p3, __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]), c_log2, l4.z, l4.w);
                            add_pair(sum[i & 4], sum[(i & 4) + 1], ex2_approx(p0), ex2_approx(p1));
                            add_pair(sum[(i & 4) + 2], sum[(i & 4) + 3], ex2_approx(p2), ex2_approx(p3));
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float p = ex2_approx(fmaf(__uint_as_float(x[i]), c_log2, ls[c0 + i]));
                            if (c0 + i >= first && c0 + i < rows) sum[i & 7] += p;
                        }
                    }
                }
                }
                tc_fence_before();
                mbar_arrive(&bars->s_free[t][buf]);
                mbar_arrive(&bars->q_empty[s]);
            }
            if (!ok) break;
            float total = ((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7]));
            if constexpr (C::kHalves == 2) {
                // the two warps of the same keys: the second half's sum comes through shared memory
                const int pair = t * 4 + (int)sub;
                if (half == 1) {
                    if (li > 0 && !(ok = wait_all(&bars->sum_free[pair], (li - 1) & 1))) break;
                    sSum[t * kTile + r] = total;
                    mbar_arrive(&bars->sum_full[pair]);
                    continue;
                }
                if (!(ok = wait_all(&bars->sum_full[pair], li & 1))) break;
                total += sSum[t * kTile + r];
                mbar_arrive(&bars->sum_free[pair]);
            }
            if (!whole) {
                a.part_sum[(size_t)(2 * blockIdx.x + (w.first ? 0 : 1)) * 2 * kTile + t * kTile + r] = total;
            } else if (page >= 0) {
                // One addition per slot and call, by this thread alone.  (A global fp32
                // atomic would flush subnormal sums, which the merge of parts keeps.)
                float& slot = a.weights[weight_at(a.s, a.Hkv, page, w.h, key)];
                slot = (FEW ? old : slot) + total;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Adds the parts of the item that CTA blockIdx.x began and did not finish, in
// the order of their rows; a thread per key.  The share behind is looked up with the own,
// most often it is the last; a warp looks up 32 of the others at once and
// loads four sums at a time: one after the other they cost 6 us of 20 (1024 tokens
// over 4096 keys, 4 heads), now 3.5 of 17.4.
__global__ void __launch_bounds__(2 * kTile) weights_merge_kernel(const PagedWeightsTcArgs a, int ctas) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c0 = (int)blockIdx.x, lane = (int)lane_id();
    const PagedPart p0 = a.parts[2 * c0], p1 = a.parts[2 * c0 + 1];
    PagedPart n = {};   // the share behind: most often it ends the item
    if (c0 + 1 < ctas) n = a.parts[2 * (c0 + 1)];
    const int slot = 2 * c0 + (p0.n_kv != 0 && p0.t0 == 0 ? 0 : 1);
    const PagedPart p = slot == 2 * c0 ? p0 : p1;
    if (p.n_kv == 0 || p.t0 != 0) return;
    const Seq sq = load_seq(a.s, p.b);
    const int key = p.i * 2 * kTile + (int)threadIdx.x;
    const float* part_sum = a.part_sum + threadIdx.x;
    float sum = part_sum[(size_t)slot * 2 * kTile];
    bool ended = p.t1 == p.n_kv;
    int c = c0 + 1;
    if (!ended && c < ctas && n.n_kv != 0) {
        sum += part_sum[(size_t)2 * c * 2 * kTile];
        ended = n.t1 == n.n_kv;
    }
    for (++c; !ended && c < ctas; c += 32) {
        // the shares with a part, up to the first that ends the item (with fewer units than CTAs some have none)
        int n_kv = 0, t1 = 0;
        if (c + lane < ctas) {
            n_kv = a.parts[2 * (c + lane)].n_kv;
            t1 = a.parts[2 * (c + lane)].t1;
        }
        unsigned part = __ballot_sync(0xffffffffu, n_kv != 0);
        const unsigned end = __ballot_sync(0xffffffffu, n_kv != 0 && t1 == n_kv);
        if (end) part &= (end & (0u - end)) * 2u - 1u;
        ended = end != 0;
        while (part) {
            float x[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                x[u] = part ? part_sum[(size_t)2 * (c + __ffs((int)part) - 1) * 2 * kTile] : 0.f;
                part &= part - 1u;
            }
            sum += x[0];
            sum += x[1];
            sum += x[2];
            sum += x[3];
        }
    }
    const int page = key < sq.L ? page_to_write(a.s, p.b, key >> a.s.page_shift) : -1;
    if (page >= 0) a.weights[weight_at(a.s, a.Hkv, page, p.h, key)] += sum;
}

template <int D, bool FEW>
cudaError_t launch_d(const PagedWeightsTcArgs& a, int sm_count, cudaStream_t stream) {
    using C = Cfg<D, FEW>;
    auto kern = paged_weights_tc_kernel<D, FEW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kern, a.tm_q, a.tm_k, a)) != cudaSuccess) return e;
    if ((e = cudaGetLastError()) != cudaSuccess || !a.split) return e;
    cfg.blockDim = dim3(2 * kTile);
    cfg.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&cfg, weights_merge_kernel, a, sm_count)) != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weights_tc(const PagedWeightsTcArgs& a, int sm_count, cudaStream_t stream) {
    const bool few = a.tt * (a.H / a.Hkv) <= kFewRows;
    if (a.D == 64) return few ? launch_d<64, true>(a, sm_count, stream) : launch_d<64, false>(a, sm_count, stream);
    return few ? launch_d<128, true>(a, sm_count, stream) : launch_d<128, false>(a, sm_count, stream);
}

}  // namespace mea
