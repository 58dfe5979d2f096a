// paged_tc.cu -- bf16 attention of ragged chunks of new tokens over a paged
// cache on the 5th-generation tensor cores (sm_100a).
//
// Same definition as paged_attn.cu; per key block j the recurrence of
// fwd_bf16.cu: m' = max(m, rowmax S_j), l' = l e^(m-m') + sum e^(S_j-m'),
// O' = O e^(m-m') + e^(S_j-m') V_j, normalised once at the end.
//
// Work.  The rows of a key/value head are its (token, head of the group) pairs,
// token by token; tt tokens (tt * G <= 128 rows) make a query tile and two
// tiles an item, which needs the key tiles (128 keys) up to what its last
// token sees.  Lengths are ragged and only known on the device, so the launch
// has one CTA per SM, and each CTA takes an equal share of all key tiles of all
// items (sequence by sequence, head by head, item by item): it begins and ends
// inside an item where the share does.  A whole item goes straight to o and
// lse; a part of one leaves its rows' summary (reference maximum, exp-sum,
// unnormalised accumulator) in the CTA's first or second workspace slot, and
// paged_tc_merge_kernel joins the parts of every item in the order of their
// keys.  Every CTA finds its share by summing the key tiles of all sequences
// itself; nothing is planned on the host, and a captured launch follows the
// lengths that it finds.
// (Cutting the list into several rounds of shares, so that the CTAs work on the
// same heads at a time and their keys stay in L2, cost more in split items than it
// gained: 4 prompts of 4096 tokens, 16 heads: 375 us in one round, 390 in two, 447
// in four.)
//
// Roles and TMEM are those of fwd_persist.cu (320 threads):
//   warp 0       TMEM allocator, then TMA producer: Q tiles per item, then K_0,
//                V_0, K_1, V_1, ... of the item through the ring, one lane and box per
//                page; no multicast.  Pages behind the
//                sequence's last key are not looked up: their boxes lie outside
//                the tensor and read as zero.
//   warp 1       MMA issuer (one thread)
//   warps 2-5    softmax / epilogue of slot 0, warps 6-9 of slot 1
// Slot t holds query tile t of an item and the key tiles that tile sees; when
// the item has one query tile both slots run it over alternate key tiles and
// fold their summaries at the end.
// Bound: with many rows each slot's chain softmax (2,000 cycles: 128 exponentials
// per row at 16 per clock and SM, and their issue) -> P V -> next S, about 3,550
// cycles per key tile of an item against 2,048 of MMAs, at the clock that the 1 kW
// power limit leaves (1.5-1.8 GHz): 2048 tokens over 16384 keys of 16 heads
// (D = 128) take 260 us, 990 TFLOP/s.  A slot that waits for the other's softmax
// before its first S, or before every S, is not faster (264 and 298 us when this
// took 263); exponentials on the FMA pipe are slower with every share tried (one
// pair in eight: 11% for 4 prompts): issue, not the exponential unit, binds.  With
// few rows HBM: 37 sequences of 4096 keys, 16 over 4 heads, 57 us, 5.4 TB/s.
//
// S is masked per row (keys past the row's token).  The values behind a
// sequence's last key in its last page may be anything, and 0 x NaN is NaN, so
// the first slot that uses such a V tile overwrites those rows with zeros.
// TMEM: S_0 [0,128) S_1 [128,256) O_0 [256,256+D) O_1 [384,384+D).
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace mea {
namespace {

constexpr int kTile = 128;        // query rows per tile, keys per tile
constexpr int kThreads = 320;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kNoKey = -1e30f;  // reference maximum of a row that has seen no key (finite: no inf - inf)
constexpr unsigned kIdescNegateA = 1u << 13;

// FEW: at most kFewRows rows per query tile (decode).  Their Q takes 4 KB per 64
// head dims instead of 16 KB (the MMA's other rows read whatever follows, and a
// row of S depends on its own row of Q alone), and the space goes to the ring:
// six tiles in flight instead of four.
//
// Rounding of P.  P V takes bf16 operands.  With few rows a probability is the sum
// of two bf16 terms, p and what rounding p leaves: at most 2^-16 p is lost, as little
// as the fp32 decode of contiguous keys (decode.cu) would notice in a bf16 result.
// The terms are two rows of the same MMA: Q is loaded twice, 16 rows apart, the
// lanes of a row and of its copy have the same S, form 32 of every 64 probabilities
// each and exchange the terms; the two rows of O are added at the item's end (ragged
// decode of 16 over 500 to 8191 keys, 32 over 8 heads: 65.9 us with one term, 64.2
// so; 64 over 300 to 2000 keys, 3.5 item ends a CTA: 82.0 and 83.6.  With every lane
// on all of its row's columns the first takes 74.5, as a second MMA 82).
// Larger tiles have no rows to spare: there P is rounded to bf16 once, at most 2^-8 p
// of each value with either sign, as in the forward kernels; a second MMA for the
// rest takes 3 chunks of 97 to 250 tokens over 16384 keys from 158 to 218 us, 4
// prompts of 4096 from 326 to 454.  The sums take p in fp32 in both.
constexpr int kFewRows = 16;

template <int D, bool FEW>
struct Cfg {
    static constexpr int kCopies = FEW ? 2 : 1;                      // of every query row
    static constexpr int kQBox = FEW ? kCopies * kFewRows * 128 : 128 * 128;   // 64 head dims of a query tile
    static constexpr int kQBytes = D / 64 * kQBox;
    static constexpr int kTileBytes = kTile * D * 2;     // K or V tile
    static constexpr int kStages = D == 64 ? (FEW ? 8 : 6) : (FEW ? 6 : 4);
    static constexpr int kSmemData = (2 * kQBytes + kStages * kTileBytes + 1023) / 1024 * 1024;
    static constexpr int kMergeBytes = 2 * kTile * 2 * 4;   // both slots' (m, l) per row
    static constexpr int kStageBytes = FEW ? 2 * 4096 : 8 * 2048;   // epilogue: 32 rows x 128 or 64 bytes per warp
    static constexpr int kSmemBytes = kSmemData + kMergeBytes + kStageBytes + 1024 /*barriers*/ + 1024 /*alignment*/;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// An item as the softmax warps need it, written by the MMA issuer when it begins
// the item.  Four of them: the issuer is at most two items ahead of a slot.
struct Item {
    int cnt;          // key tiles of the CTA's part; 0: no more items
    int n0;           // of those, the ones that query tile 0 of a two-tile item sees
    int single;       // one query tile: both slots on its rows
    int tok0;         // first token
    int n, q0;        // new tokens of the sequence, its first packed row
    int seen;         // keys in front of the new tokens' own
    int L;            // cached keys
    int base;         // first key of the part
    int h;
    int part;         // the CTA's workspace slot for it, or -1: the item is whole
    int pad;
};

struct Barriers {
    uint64_t q_full, q_empty;
    uint64_t full[8], empty[8];
    uint64_t s_full[2], p_half[2], p_ready[2], o_free[2], o_final[2];
    uint64_t item[4];
    uint64_t merge_ready, drain;
    Item items[4];
    unsigned tmem_base;
    int abort_flag;
    // this CTA's share: where it begins, and what it costs
    struct Share {
        Seq sq;
        int b, h, i, t0;
        long long cost;
    } share;
    long long warp_sum[kThreads / 32];
};

// Items of a sequence, and the key tiles of item i (an item whose rows see no
// key has one tile, fully masked, so that its rows are written).
__device__ __forceinline__ int items_of(const Seq& sq, int tt) { return (sq.n + 2 * tt - 1) / (2 * tt); }
__device__ __forceinline__ int keys_seen(const Seq& sq, int tokens) {   // by the last of the first `tokens`
    return max(0, sq.L - sq.n + min(tokens, sq.n));
}
__device__ __forceinline__ int tiles_of(const Seq& sq, int tt, int i) {
    return max(1, (keys_seen(sq, (i + 1) * 2 * tt) + kTile - 1) / kTile);
}

// Position in the list of items; walks on item by item.  A key tile costs 1, an
// item's end kEndCost: an epilogue takes about 4 us, a key tile 1.9 (1 to 4 measure
// within 2% of one another; 6 is slower for a ragged decode).
constexpr int kEndCost = 2;

struct Walk {
    Seq sq;
    int b, h, i, items;
    int t0, t1, n_kv;       // key tiles [t0, t1) of the item's n_kv
    long long left;         // of the share, from t0 on
    bool first;

    __device__ __forceinline__ void begin(const PagedBatch& s, const Barriers::Share& at, int Hkv, int tt) {
        sq = at.sq;
        b = at.b;
        h = at.h;
        i = at.i;
        t0 = at.t0;
        left = at.cost;
        first = true;
        if (left <= 0) return;
        items = items_of(sq, tt);
        n_kv = tiles_of(sq, tt, i);
        t1 = (int)min((long long)n_kv, t0 + left);
        if (t0 >= n_kv) {   // nothing but the end of an item, which the CTA in front has taken
            next(s, Hkv, tt);
            first = true;
        }
    }
    __device__ __forceinline__ bool done() const { return left <= 0; }
    __device__ __forceinline__ void next(const PagedBatch& s, int Hkv, int tt) {
        left -= n_kv + kEndCost - t0;
        first = false;
        if (left <= 0) return;
        if (++i == items) {
            i = 0;
            if (++h == Hkv) {
                h = 0;
                do {   // sequences without new tokens have no item
                    ++b;
                    if (b >= s.B) {
                        left = 0;
                        return;
                    }
                    sq = load_seq(s, b);
                } while (sq.n == 0);
                items = items_of(sq, tt);
            }
        }
        n_kv = tiles_of(sq, tt, i);
        t0 = 0;
        t1 = (int)min((long long)n_kv, left);
    }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == n_kv; }
    __device__ __forceinline__ bool two(int tt) const { return i * 2 * tt + tt < sq.n; }   // both query tiles live
    // key tiles of [t0, t1) that query tile 0 of a two-tile item sees
    __device__ __forceinline__ int tiles_slot0(int tt) const {
        const int seen = (keys_seen(sq, i * 2 * tt + tt) + kTile - 1) / kTile;
        return max(0, min(t1, seen) - t0);
    }
};

// Every thread of the CTA: finds its share [W c / C, W (c + 1) / C) of the cost W of all items.
__device__ __forceinline__ void find_share(const PagedTcArgs& a, Barriers* bars) {
    if (threadIdx.x == 0) bars->share.cost = 0;
    __syncthreads();
    Seq sq;
    auto cost = [&](int b) {
        sq = load_seq(a.s, b);
        const int items = items_of(sq, a.tt);
        long long sum = 0;
        for (int i = 0; i < items; ++i) sum += tiles_of(sq, a.tt, i) + kEndCost;
        return sum * a.Hkv;
    };
    auto locate = [&](int b, long long before, long long sum, long long W) {
        const long long w0 = share_begin(W, blockIdx.x, gridDim.x), w1 = share_begin(W, blockIdx.x + 1, gridDim.x);
        if (w0 < before || w0 >= before + sum || w1 <= w0) return;
        const int items = items_of(sq, a.tt);   // sq is b's since cost(b)
        const long long per_head = divide(sum, a.Hkv);
        long long x = w0 - before;
        Barriers::Share& at = bars->share;
        at.cost = w1 - w0;
        at.sq = sq;
        at.b = b;
        at.h = (int)divide(x, per_head);
        x -= at.h * per_head;
        int i = 0;
        for (; i + 1 < items; ++i) {
            const int n = tiles_of(sq, a.tt, i) + kEndCost;
            if (x < n) break;
            x -= n;
        }
        at.i = i;
        at.t0 = (int)x;
    };
    lay_out_costs<kThreads>(a.s.B, bars->warp_sum, cost, locate);
    __syncthreads();
}

template <int D, bool FEW>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const PagedTcArgs a) {
    using C = Cfg<D, FEW>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* sQ = smem;
    uint8_t* sRing = smem + 2 * C::kQBytes;
    float* sMerge = reinterpret_cast<float*>(smem + C::kSmemData);
    uint8_t* sStage = smem + C::kSmemData + C::kMergeBytes;
    Barriers* bars = reinterpret_cast<Barriers*>(smem + C::kSmemData + C::kMergeBytes + C::kStageBytes);
    static_assert(sizeof(Barriers) <= 1024, "shared memory");

    const unsigned warp = warp_id();
    const unsigned lane = lane_id();
    const int tt = a.tt;
    const int G = a.H / a.Hkv;

    if (threadIdx.x == 0) {
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->q_empty, 1);
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&bars->full[s], 1);
            mbar_init(&bars->empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->p_half[t], 128);
            mbar_init(&bars->p_ready[t], 128);
            mbar_init(&bars->o_free[t], 128);
            mbar_init(&bars->o_final[t], 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&bars->item[i], 1);
        mbar_init(&bars->merge_ready, 256);
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
            prefetch_tmap(&tm_v);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const unsigned tmem = bars->tmem_base;
    volatile int* abort_flag = &bars->abort_flag;
    // programmatic stream serialisation: nothing global is touched before the
    // previous kernel's results are complete and visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    find_share(a, bars);

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        Walk w;
        const int shift = a.s.page_shift;
        const int box_rows = min(kTile, 1 << shift);
        const int my_row = (int)lane * box_rows;         // first key of the lane's box in the tile
        const bool mine = my_row < kTile;
        const int outside = a.s.num_pages * a.Hkv;       // a page behind the tensor: reads as zero
        int c_glob = 0;
        int li = 0, q_asked = 0;    // items; those whose Q has been asked for
        bool ok = true;
        // lane 0 waits, the warp follows its verdict
        auto wait = [&](uint64_t* bar, unsigned parity) -> bool {
            const int got = lane != 0 || mbar_wait(bar, parity, abort_flag);
            return __shfl_sync(0xffffffffu, got, 0) != 0;
        };
        const int slot = 2 * (int)blockIdx.x;           // the CTA's workspace slots
        if (lane == 0) a.parts[slot].n_kv = a.parts[slot + 1].n_kv = 0;     // no part yet
        // the lane's entry of the page table for key tile j, asked for a tile ahead
        auto look_up = [&](int j) {
            const int key = j * kTile + my_row;
            return mine && key < w.sq.L ? page_entry(a.s, w.b, key >> shift) : 0;
        };
        for (w.begin(a.s, bars->share, a.Hkv, tt); ok && !w.done(); w.next(a.s, a.Hkv, tt), ++li) {
            const int n_qt = w.two(tt) ? 2 : 1;
            int entry = look_up(w.t0);
            if (li > 0 && !(ok = wait(&bars->q_empty, (li - 1) & 1))) break;
            if (lane == 0) {
                if (!w.whole()) {
                    PagedPart& p = a.parts[slot + (w.first ? 0 : 1)];
                    p.b = w.b;
                    p.h = w.h;
                    p.i = w.i;
                    p.t0 = w.t0;
                    p.t1 = w.t1;
                    p.n_kv = w.n_kv;
                    p.q0 = w.sq.q0;
                    p.n = w.sq.n;
                }
                mbar_arrive_expect_tx(&bars->q_full, (unsigned)(n_qt * C::kCopies * G * tt * D * 2));
                for (int t = 0; t < n_qt; ++t)
                    for (int x = 0; x < D / 64 * C::kCopies; ++x)
                        tma_load_3d(sQ + t * C::kQBytes + x * (C::kQBox / C::kCopies), &tm_q, &bars->q_full,
                                    x / C::kCopies * 64, w.h * G, w.sq.q0 + (2 * w.i + t) * tt);
            }
            q_asked = li + 1;
            for (int j = w.t0; ok && j < w.t1; ++j) {
                const int key = j * kTile + my_row;
                int z = outside;
                if (mine && key < w.sq.L) z = page_of(a.s, entry) * a.Hkv + w.h;
                if (j + 1 < w.t1) entry = look_up(j + 1);
                const int group = (key & ((1 << shift) - 1)) >> 3;
#pragma unroll
                for (int v = 0; v < 2; ++v, ++c_glob) {
                    const int s = c_glob % C::kStages;
                    if (c_glob >= C::kStages && !(ok = wait(&bars->empty[s], ((c_glob / C::kStages) - 1) & 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars->full[s], C::kTileBytes);
                    __syncwarp();
                    if (mine)
                        tma_load_5d(sRing + s * C::kTileBytes + PageTile<D>::row(my_row, 0), v ? &tm_v : &tm_k,
                                    &bars->full[s], 0, 0, 0, group, z);
                    __syncwarp();
                }
            }
        }
        // never leave with copies in flight
        for (int c = (c_glob > C::kStages ? c_glob - C::kStages : 0); c < c_glob; ++c)
            mbar_wait(&bars->full[c % C::kStages], (c / C::kStages) & 1, nullptr);
        if (q_asked > 0) mbar_wait(&bars->q_full, (q_asked - 1) & 1, nullptr);
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issuer
        if (lane == 0) {
            // scale < 0: S is formed as (-Q) K^T and the softmax uses |scale|
            const unsigned idesc_s = make_idesc_bf16(128, kTile, 0, 0) | (a.scale < 0.f ? kIdescNegateA : 0u);
            constexpr unsigned idesc_o = make_idesc_bf16(128, D, 0, 1);
            const uint32_t q_lo0 = desc_lo_kmajor(smem_u32(sQ));
            const uint32_t q_lo1 = desc_lo_kmajor(smem_u32(sQ + C::kQBytes));
            const uint32_t ring_k_lo = desc_lo_kmajor(smem_u32(sRing));
            const uint32_t ring_v_lo = PageTile<D>::mn_lo(smem_u32(sRing));
            constexpr uint32_t kStageStep = C::kTileBytes >> 4;
            const unsigned tS0 = tmem, tS1 = tmem + 128u, tO0 = tmem + 256u, tO1 = tmem + 384u;
            int stage = 0;
            unsigned phase = 0;
            auto next_tile = [&](uint32_t& off, int& st_used) -> bool {
                if (!mbar_wait(&bars->full[stage], phase, abort_flag)) return false;
                off = (uint32_t)stage * kStageStep;
                st_used = stage;
                if (++stage == C::kStages) { stage = 0; phase ^= 1u; }
                return true;
            };
            auto issue_s = [&](unsigned tS, uint32_t q_lo, uint32_t k_off) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ss_desc(tS, q_lo + (kk >> 2) * (C::kQBox >> 4) + (kk & 3) * 2, kDescHiSw128,
                                ring_k_lo + k_off + PageTile<D>::kmajor(kk), PageTile<D>::kHi, idesc_s, kk > 0);
            };
            auto pv_halves = [&](int t, unsigned parity, uint32_t v_off, unsigned acc0) -> bool {
                const unsigned tO = t ? tO1 : tO0, tS = t ? tS1 : tS0;
                if (!mbar_wait(&bars->p_half[t], parity, abort_flag)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kTile / 32; ++kk)
                    mma_ts_desc(tO, tS + kk * 8, ring_v_lo + v_off + PageTile<D>::mnmajor(kk), PageTile<D>::kHi, idesc_o,
                                (acc0 | kk) ? 1u : 0u);
                if (!mbar_wait(&bars->p_ready[t], parity, abort_flag)) return false;
                tc_fence_after();
#pragma unroll
                for (int kk = kTile / 32; kk < kTile / 16; ++kk)
                    mma_ts_desc(tO, tS + kk * 8, ring_v_lo + v_off + PageTile<D>::mnmajor(kk), PageTile<D>::kHi, idesc_o, 1u);
                return true;
            };
            Walk w;
            bool ok = true, prev_single = false;
            int cnt0 = 0, cnt1 = 0;   // key tiles completed by each slot: phase of s_full / p_half / p_ready
            int li = 0;
            for (w.begin(a.s, bars->share, a.Hkv, tt); ok && !w.done(); w.next(a.s, a.Hkv, tt), ++li) {
                const bool single = !w.two(tt);
                const int n1 = w.t1 - w.t0;
                const int n0 = single ? 0 : w.tiles_slot0(tt);   // <= n1
                {
                    Item& it = bars->items[li & 3];
                    it.cnt = n1;
                    it.n0 = n0;
                    it.single = single;
                    it.tok0 = 2 * w.i * tt;
                    it.n = w.sq.n;
                    it.q0 = w.sq.q0;
                    it.seen = w.sq.L - w.sq.n;
                    it.L = w.sq.L;
                    it.base = w.t0 * kTile;
                    it.h = w.h;
                    it.part = w.whole() ? -1 : 2 * (int)blockIdx.x + (w.first ? 0 : 1);
                    mbar_arrive(&bars->item[li & 3]);
                }
                // A slot's first P V overwrites its O.  Its own epilogue of the
                // item before is over when its softmax hands over P; after a
                // single item the other slot's epilogue has read it as well.
                // The parity names the item before: the wait must come ahead of
                // the o_final that lets slot t ^ 1 finish this item, or that slot
                // may arrive once more and the parity is that of the item after.
                auto o_is_free = [&](int t) -> bool {
                    return !prev_single || mbar_wait(&bars->o_free[t ^ 1], (li - 1) & 1, abort_flag);
                };
                if (!(ok = mbar_wait(&bars->q_full, li & 1, abort_flag))) break;
                uint32_t k_off = 0;
                int k_stage = 0;
                if (single) {
                    uint32_t v_off0 = 0, v_off1 = 0;
                    int v_stage0 = 0, v_stage1 = 0;
                    for (int t = 0; ok && t < 2 && t < n1; ++t) {
                        if (!(ok = next_tile(k_off, k_stage))) break;
                        tc_fence_after();
                        issue_s(t ? tS1 : tS0, q_lo0, k_off);
                        mma_commit(&bars->s_full[t]);
                        mma_commit(&bars->empty[k_stage]);
                        if (t + 1 == n1) mma_commit(&bars->q_empty);   // Q read by its last S
                        ok = t ? next_tile(v_off1, v_stage1) : next_tile(v_off0, v_stage0);
                    }
                    for (int j = 0; ok && j < n1; ++j) {
                        const int t = j & 1;
                        if (j < 2 && !(ok = o_is_free(t))) break;
                        if (!(ok = pv_halves(t, (t ? cnt1 : cnt0) & 1, t ? v_off1 : v_off0, j >= 2 ? 1u : 0u))) break;
                        if (t) ++cnt1; else ++cnt0;
                        mma_commit(&bars->empty[t ? v_stage1 : v_stage0]);
                        if (j + 2 < n1) {
                            if (!(ok = next_tile(k_off, k_stage))) break;
                            tc_fence_after();
                            issue_s(t ? tS1 : tS0, q_lo0, k_off);
                            mma_commit(&bars->s_full[t]);
                            mma_commit(&bars->empty[k_stage]);
                            if (j + 3 == n1) mma_commit(&bars->q_empty);
                            ok = t ? next_tile(v_off1, v_stage1) : next_tile(v_off0, v_stage0);
                        }
                    }
                } else {
                    if (!(ok = next_tile(k_off, k_stage))) break;
                    tc_fence_after();
                    if (n0 > 0) {
                        issue_s(tS0, q_lo0, k_off);
                        mma_commit(&bars->s_full[0]);
                    }
                    issue_s(tS1, q_lo1, k_off);
                    mma_commit(&bars->s_full[1]);
                    mma_commit(&bars->empty[k_stage]);
                    if (n1 == 1) mma_commit(&bars->q_empty);
                    for (int j = 0; ok && j < n1; ++j) {
                        const bool more = j + 1 < n1;
                        const unsigned acc0 = j > 0 ? 1u : 0u;
                        uint32_t v_off = 0;
                        int v_stage = 0;
                        if (!(ok = next_tile(v_off, v_stage))) break;
                        if (j < n0) {
                            if (j == 0 && !(ok = o_is_free(0))) break;
                            if (!(ok = pv_halves(0, cnt0 & 1, v_off, acc0))) break;
                            ++cnt0;
                            if (j == n0 - 1 && j > 0) mma_commit(&bars->o_final[0]);
                        }
                        if (more) {
                            if (!(ok = next_tile(k_off, k_stage))) break;
                            tc_fence_after();
                            if (j + 1 < n0) {
                                issue_s(tS0, q_lo0, k_off);
                                mma_commit(&bars->s_full[0]);
                            }
                        }
                        if (j == 0) {
                            // Behind the next S, where it delays nothing (ahead of it 4 prompts
                            // take 323 us, here 313); a slot 0 of one key tile is let go after it.
                            if (!(ok = o_is_free(1))) break;
                            if (n0 == 1) mma_commit(&bars->o_final[0]);
                        }
                        if (!(ok = pv_halves(1, cnt1 & 1, v_off, acc0))) break;
                        ++cnt1;
                        mma_commit(&bars->empty[v_stage]);
                        if (more) {
                            issue_s(tS1, q_lo1, k_off);
                            mma_commit(&bars->s_full[1]);
                            mma_commit(&bars->empty[k_stage]);
                            if (j + 2 == n1) mma_commit(&bars->q_empty);
                        }
                    }
                }
                // A slot that handed over a P in this item has finished the item
                // before.  One that had no key tile must not fall a whole phase
                // of o_final behind: both slots have finished the item before.
                const bool idle = single ? n1 == 1 : n0 == 0;
                if (ok && idle && li > 0)
                    ok = mbar_wait(&bars->o_free[0], (li - 1) & 1, abort_flag) &&
                         mbar_wait(&bars->o_free[1], (li - 1) & 1, abort_flag);
                if (ok) {
                    if (single || idle) mma_commit(&bars->o_final[0]);
                    mma_commit(&bars->o_final[1]);
                }
                prev_single = single;
            }
            if (ok) {
                bars->items[li & 3].cnt = 0;
                mbar_arrive(&bars->item[li & 3]);
            }
            mma_commit(&bars->drain);
            mbar_wait(&bars->drain, 0, nullptr);
        }
    } else {
        // ------------------------------------------------ softmax / epilogue
        const int t = (warp - 2) >> 2;
        const unsigned sub = warp & 3;
        const int r = (int)sub * 32 + (int)lane;
        const unsigned lane_off = (sub * 32u) << 16;
        const unsigned tS = tmem + lane_off + (t ? 128u : 0u);
        const unsigned tO = tmem + lane_off + (t ? 384u : 256u);
        // S carries the sign; a scale of 0 must not meet the mask's infinity
        const float c_log2 = fmaxf(fabsf(a.scale) * kLog2e, 1e-37f);
        // row of the query tile; with few rows lanes 16-31 hold the copies of rows 0-15
        const int q_r = FEW && sub == 0 ? r % kFewRows : r;
        const bool copy = FEW && r >= kFewRows;
        const int tok_r = q_r / G;             // its token in the query tile
        const int g_r = q_r - tok_r * G;
        const int page = 1 << a.s.page_shift;
        // a wait that gives up does so for the whole warp: the code behind it is collective
        auto wait_all = [&](uint64_t* bar, unsigned parity) -> bool {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag));
        };
        bool ok = true;
        int kt = 0;         // key tiles completed by this slot (all items)
        int ring = 0;       // ring tiles in front of the current item
        int n_single = 0;   // single items completed by this CTA
        int li = 0;
        for (;; ++li) {
            if (!(ok = wait_all(&bars->item[li & 3], (li >> 2) & 1))) break;
            const Item& w = bars->items[li & 3];
            const int cnt = w.cnt;
            if (cnt == 0) break;
            const bool single = w.single != 0;
            const int n0 = w.n0;
            // a two-tile item's slot t owns query tile t; a single item's slots
            // own its one tile and key tiles t, t+2, ...
            const int n_mine = single ? (cnt + 1 - t) / 2 : (t ? cnt : n0);
            const int tok = w.tok0 + (single ? 0 : t * tt) + tok_r;
            const bool valid = !copy && tok_r < tt && tok < w.n;
            const bool live = __any_sync(0xffffffffu, valid);   // rows of other lanes never meet this warp's
            // keys the row sees, from the part's first key on
            const int lim = max(0, w.seen + min(tok, w.n - 1) + 1) - w.base;
            // from this key tile on some row of the warp is masked (uniform, so that
            // the other tiles skip the selects by a branch)
            const int mask_j = max(0, __reduce_min_sync(0xffffffffu, lim)) / kTile;
            // The key tile (of this slot, else -1) whose values behind the
            // sequence's last key are to be overwritten, and their first row.
            const int last = (w.L - 1 - w.base) >> 7;
            const int nv = w.L - w.base - last * kTile;
            const int fix = w.L > 0 && last < cnt && nv % page != 0 &&
                            (single ? (last & 1) == t : t == (last < n0 ? 0 : 1)) ? last : -1;
            float m_ref = kNoKey;
            float l = 0.f;
            for (int it = 0; it < n_mine; ++it, ++kt) {
                const int j = single ? 2 * it + t : it;          // key tile of this share of the item
                if (!(ok = wait_all(&bars->s_full[t], kt & 1))) break;
                tc_fence_after();
                if (j == fix) {   // zeros, before any P V reads the tile
                    const int c = ring + 2 * j + 1;
                    const int s = c % C::kStages;
                    if (!(ok = wait_all(&bars->full[s], (c / C::kStages) & 1))) break;
                    const int stop = min(kTile, (nv + page - 1) / page * page);
                    uint8_t* tile = sRing + s * C::kTileBytes;
                    constexpr int kPieces = D / 8;                // 16-byte pieces of one key's values
                    for (int e = r; e < (stop - nv) * kPieces; e += 128) {
                        const int q = e % kPieces;
                        *reinterpret_cast<uint4*>(tile + PageTile<D>::row(nv + e / kPieces, q >> 3) + (q & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                if (!live) {
                    mbar_arrive(&bars->p_half[t]);
                    mbar_arrive(&bars->p_ready[t]);
                    continue;
                }
                // the lane's scores: with few rows 32 of every 64, the copy's lane has the others
                constexpr int kOwn = FEW ? kTile / 2 : kTile;
                uint32_t sr[kOwn];
                if constexpr (FEW) {
                    uint32_t all[kTile];
#pragma unroll
                    for (int c0 = 0; c0 < kTile; c0 += 32) tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(&all[c0]));
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < kOwn; ++c) sr[c] = copy ? all[c + (c & 32) + 32] : all[c + (c & 32)];
                } else {
#pragma unroll
                    for (int c0 = 0; c0 < kTile; c0 += 32) tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(&sr[c0]));
                    tmem_wait_ld();
                }
                if (j >= mask_j) {
                    const int nvalid = lim - j * kTile - (copy ? 32 : 0);
#pragma unroll
                    for (int c = 0; c < kOwn; ++c)
                        if ((FEW ? c + (c & 32) : c) >= nvalid) sr[c] = __float_as_uint(-INFINITY);
                }
                float mxa[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) mxa[i] = fmaxf(__uint_as_float(sr[i]), __uint_as_float(sr[8 + i]));
#pragma unroll
                for (int c = 16; c < kOwn; c += 16)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        mxa[i] = fmax3(mxa[i], __uint_as_float(sr[c + i]), __uint_as_float(sr[c + 8 + i]));
                float mx = fmaxf(fmax3(mxa[0], mxa[1], mxa[2]), fmax3(fmax3(mxa[3], mxa[4], mxa[5]), mxa[6], mxa[7]));
                if constexpr (FEW) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, kFewRows));
                const float m_blk = fmaxf(mx * c_log2, kNoKey);
                // Only the sequence's rows say when the warp's references move: the others
                // hold other sequences' tokens or what ran before, and a move out of turn
                // rounds the rows' probabilities to other bits.  A row and its copy agree.
                float alpha = 1.f;
                bool rescale = false;
                if (it == 0) {
                    m_ref = m_blk;
                } else if (__any_sync(0xffffffffu, valid && m_blk - m_ref > kRescaleThreshold)) {
                    const float m_new = fmaxf(m_ref, m_blk);
                    alpha = ex2_approx(m_ref - m_new);
                    m_ref = m_new;
                    rescale = true;
                }
                l *= alpha;
                float rsa[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) rsa[i] = 0.f;
#pragma unroll
                for (int c0 = 0; c0 < kOwn; c0 += 32) {
                    uint32_t pk[16];
                    [[maybe_unused]] uint32_t rest[16];
#pragma unroll
                    for (int c = 0; c < 32; c += 2) {
                        float p0 = -m_ref, p1 = -m_ref;
                        fma2(p0, p1, __uint_as_float(sr[c0 + c]), __uint_as_float(sr[c0 + c + 1]), c_log2, c_log2);
                        p0 = ex2_approx(p0);
                        p1 = ex2_approx(p1);
                        rsa[(c / 2) & 7] += p0 + p1;
                        pk[c / 2] = pack_bf16x2(p0, p1);
                        if constexpr (FEW)
                            rest[c / 2] = pack_bf16x2(p0 - __uint_as_float(pk[c / 2] << 16),
                                                      p1 - __uint_as_float(pk[c / 2] & 0xffff0000u));
                    }
                    if constexpr (FEW) {
                        // the row's lane stores the first terms, the copy's lane the second ones
#pragma unroll
                        for (int c = 0; c < 16; ++c) {
                            const uint32_t below = __shfl_up_sync(0xffffffffu, rest[c], kFewRows);
                            const uint32_t above = __shfl_down_sync(0xffffffffu, pk[c], kFewRows);
                            pk[c] = copy ? below : pk[c];
                            rest[c] = copy ? rest[c] : above;
                        }
                        tmem_st16(tS + c0, pk);
                        tmem_st16(tS + c0 + 16, rest);
                    } else {
                        tmem_st16(tS + c0 / 2, pk);
                    }
                    if (c0 == kOwn / 2 - 32 && !rescale) {
                        tmem_wait_st();
                        tc_fence_before();
                        mbar_arrive(&bars->p_half[t]);
                    }
                }
                l += ((rsa[0] + rsa[1]) + (rsa[2] + rsa[3])) + ((rsa[4] + rsa[5]) + (rsa[6] + rsa[7]));
                if (rescale) {
                    // P V of this slot's previous key tile has completed (it was
                    // issued before S of this one, whose commit was waited on)
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t ov[32];
                        tmem_ld32(tO + c0, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                        tmem_st32(tO + c0, ov);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                if (rescale) mbar_arrive(&bars->p_half[t]);
                mbar_arrive(&bars->p_ready[t]);
            }
            if (!ok) break;
            ring += 2 * cnt;
            if constexpr (FEW) l += __shfl_xor_sync(0xffffffffu, l, kFewRows);
            // A single item's slots fold their summaries of the same rows and
            // each writes half of the head dims, reading both slots' O (slot 1
            // has none when the share has one key tile).
            const bool with1 = single && cnt >= 2;
            float w0 = 1.f, w1 = 0.f, M = m_ref, L = l;
            if (single) {
                // the other slot has read the previous item's summaries
                if (li > 0 && !(ok = wait_all(&bars->o_free[t ^ 1], (li - 1) & 1))) break;
                sMerge[2 * (t * kTile + r)] = m_ref;
                sMerge[2 * (t * kTile + r) + 1] = l;
                mbar_arrive(&bars->merge_ready);
                if (!(ok = wait_all(&bars->merge_ready, n_single & 1))) break;
                ++n_single;
                const float m_o = sMerge[2 * ((t ^ 1) * kTile + r)];
                const float l_o = sMerge[2 * ((t ^ 1) * kTile + r) + 1];
                M = fmaxf(m_ref, m_o);
                const float w_self = ex2_approx(m_ref - M), w_oth = ex2_approx(m_o - M);
                L = w_self * l + w_oth * l_o;
                w0 = t ? w_oth : w_self;
                w1 = t ? w_self : w_oth;
            }
            if (!(ok = wait_all(&bars->o_final[t], li & 1))) break;
            if (single && !(ok = wait_all(&bars->o_final[t ^ 1], li & 1))) break;
            tc_fence_after();
            const bool whole = w.part < 0;
            const bool none = L == 0.f;     // no key in sight: O may never have been written
            const float inv = none ? 0.f : whole ? 1.f / L : 1.f;
            const float s0 = w0 * inv, s1 = w1 * inv;
            const int row = whole ? (w.q0 + tok) * a.H + w.h * G + g_r
                                  : (2 * w.part + (single ? 0 : t)) * tt * G + r;
            // Rows go out through the warp's part of shared memory, 64 bytes of
            // each of the 32 rows a round: a store instruction then covers 8 rows
            // of 64 contiguous bytes, not 32 rows of 16.  16-byte pieces are
            // permuted by row against bank conflicts.  With few rows a round is 32
            // fp32 columns, and a row and its copy, the two terms' P V, are added on
            // the way (64 x 2000 keys, 32 over 8 heads: 83.6 us; with a shuffle per column
            // in the registers 85.7).
            uint8_t* stage = sStage + (FEW ? t * 4096 : ((int)warp - 2) * 2048);
            const int dst = valid ? row : -1;
            const int c_begin = single ? t * (D / 2) : 0;
            auto put = [&](int q, const uint4& v) {   // piece q of this lane's row
                *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) * 16)) = v;
            };
            auto store = [&](void* base, size_t row_bytes, int byte0) {
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int rr = 8 * i + (int)lane / 4, q = (int)lane % 4;
                    const int d = __shfl_sync(0xffffffffu, dst, rr);
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((q ^ ((rr >> 1) & 3)) * 16));
                    if (d >= 0) *reinterpret_cast<uint4*>(static_cast<uint8_t*>(base) + d * row_bytes + byte0 + q * 16) = v;
                }
                __syncwarp();
            };
            auto emit = [&](const uint32_t (&x)[32], int col) {   // 32 columns of the warp's rows
                if constexpr (FEW) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        *reinterpret_cast<uint4*>(stage + lane * 128 + ((q ^ (lane & 7)) * 16)) =
                            make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < kFewRows / 4; ++i) {
                        const int rr = 4 * i + (int)lane / 8, q = (int)lane % 8;
                        const int d = __shfl_sync(0xffffffffu, dst, rr);
                        const uint8_t* piece = stage + rr * 128 + ((q ^ (rr & 7)) * 16);
                        float4 v = *reinterpret_cast<const float4*>(piece);
                        const float4 w2 = *reinterpret_cast<const float4*>(piece + kFewRows * 128);
                        v = make_float4(v.x + w2.x, v.y + w2.y, v.z + w2.z, v.w + w2.w);
                        if (d < 0) continue;
                        if (whole)
                            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + (size_t)d * D + col + 4 * q) =
                                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                        else
                            *reinterpret_cast<float4*>(a.part_acc + (size_t)d * D + col + 4 * q) = v;
                    }
                    __syncwarp();
                } else if (whole) {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        put(q, make_uint4(pack_bf16x2(__uint_as_float(x[8 * q]), __uint_as_float(x[8 * q + 1])),
                                          pack_bf16x2(__uint_as_float(x[8 * q + 2]), __uint_as_float(x[8 * q + 3])),
                                          pack_bf16x2(__uint_as_float(x[8 * q + 4]), __uint_as_float(x[8 * q + 5])),
                                          pack_bf16x2(__uint_as_float(x[8 * q + 6]), __uint_as_float(x[8 * q + 7]))));
                    store(a.o, D * 2, col * 2);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; c += 16) {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            put(q, make_uint4(x[c + 4 * q], x[c + 4 * q + 1], x[c + 4 * q + 2], x[c + 4 * q + 3]));
                        store(a.part_acc, D * 4, (col + c) * 4);
                    }
                }
            };
            // 64 accumulators at a time: of a two-tile item 64 columns of its own O,
            // of a single item 32 columns of both O
#pragma unroll 1
            for (int pass = 0; live && pass < D / 64; ++pass) {
                uint32_t x0[32], x1[32];
                tmem_ld32(single ? tmem + lane_off + 256u + c_begin + 32 * pass : tO + 64 * pass, x0);
                tmem_ld32(single ? tmem + lane_off + 384u + c_begin + 32 * pass : tO + 64 * pass + 32, x1);
                tmem_wait_ld();
                if (pass == D / 64 - 1) {   // the accumulators are free before the last rows are stored
                    tc_fence_before();
                    mbar_arrive(&bars->o_free[t]);
                }
                if (single) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        float f = __uint_as_float(x0[c]) * s0;
                        if (with1) f = fmaf(__uint_as_float(x1[c]), s1, f);
                        x0[c] = __float_as_uint(none ? 0.f : f);
                    }
                    emit(x0, c_begin + 32 * pass);
                } else {
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        x0[c] = __float_as_uint(none ? 0.f : __uint_as_float(x0[c]) * s0);
                        x1[c] = __float_as_uint(none ? 0.f : __uint_as_float(x1[c]) * s0);
                    }
                    emit(x0, 64 * pass);
                    emit(x1, 64 * pass + 32);
                }
            }
            if (valid && (!single || t == 0)) {
                if (whole)
                    a.lse[row] = none ? -INFINITY : (M + __log2f(L)) * kLn2;
                else
                    *reinterpret_cast<float2*>(a.part_ml + 2 * (size_t)row) = make_float2(none ? -INFINITY : M, L);
            }
            if (!live) {
                tc_fence_before();
                mbar_arrive(&bars->o_free[t]);
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

// Joins the parts of the items that shares of the main kernel began and did not
// finish.  A share has a part in its first slot, its second, both or none; taken
// share by share they are in the order of the work, so an item's parts follow one
// another, the first with t0 = 0.  Every CTA lists them (a share per thread) and
// takes slices of kRows rows of the items: W warps take R rows, each every W-th
// part, a lane D / 32 head dims; the warps' results are joined through shared memory
// (W = 8, R = 1 where an item has few rows: decode cuts a long cache into many parts).
// The slices' first rows come first: an item that is not full leaves the last idle.
// Bound: launch, the look-up (2 us) and a round of loads; from 20 MB of parts on L2.
// With a CTA per share and slice, most of them idle, and every part's loads behind a
// look-up and the exponential of the part in front, 60 tokens over 1000 keys (8 parts
// an item) took 28.9 us, now 17.4 (12.5 without this kernel); 8 prompts of 97 to 500
// tokens 33.5, now 29.4.  More CTAs per SM spill or wait for one another's registers.
constexpr int kMergeThreads = 256;
constexpr int kMergeBatch = 4;
constexpr int kMergeBlocks = 2, kMergeBlocksFew = 3;   // per SM

// Loads that the compiler leaves where they are (it sinks plain ones to their uses,
// each behind the exponential of the part in front).
__device__ __forceinline__ void load_now(const float* p, float2& x) {
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(p));
}
__device__ __forceinline__ void load_now(const float* p, float (&x)[2]) {
    asm volatile("ld.global.v2.f32 {%0, %1}, [%2];" : "=f"(x[0]), "=f"(x[1]) : "l"(p));
}
__device__ __forceinline__ void load_now(const float* p, float (&x)[4]) {
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]) : "l"(p));
}

template <int DPL, int W, int R>
__global__ void __launch_bounds__(kMergeThreads, W > 1 ? kMergeBlocksFew : kMergeBlocks) paged_tc_merge_kernel(const PagedTcArgs a, int shares) {
    constexpr int D = 32 * DPL;
    constexpr int kWarps = kMergeThreads / 32;
    constexpr int kRows = kWarps / W * R;
    struct Split {
        int at;               // its first part in s_slot
        int n, q0, h, tok0;   // new tokens of the sequence, its first packed row; head; first token
    };
    __shared__ int s_parts[kWarps], s_items[kWarps];
    __shared__ int s_slot[2 * kMergeThreads];
    __shared__ Split s_item[kMergeThreads + 1];
    __shared__ float s_acc[W > 1 ? kWarps : 1][D];
    __shared__ float2 s_ml[W > 1 ? kWarps : 1];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = (int)warp_id(), lane = (int)lane_id();
    PagedPart p0 = {}, p1 = {};
    if ((int)threadIdx.x < shares) {
        p0 = a.parts[2 * threadIdx.x];
        p1 = a.parts[2 * threadIdx.x + 1];
    }
    const bool has0 = p0.n_kv != 0, has1 = p1.n_kv != 0;
    const bool first0 = has0 && p0.t0 == 0, first1 = has1 && p1.t0 == 0;   // at most one of them
    const unsigned below = (1u << lane) - 1u;
    const unsigned b0 = __ballot_sync(0xffffffffu, has0), b1 = __ballot_sync(0xffffffffu, has1);
    const unsigned bf = __ballot_sync(0xffffffffu, first0 || first1);
    if (lane == 0) {
        s_parts[warp] = __popc(b0) + __popc(b1);
        s_items[warp] = __popc(bf);
    }
    __syncthreads();
    int at = __popc(b0 & below) + __popc(b1 & below), item = __popc(bf & below), parts = 0, items = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
        at += k < warp ? s_parts[k] : 0;
        item += k < warp ? s_items[k] : 0;
        parts += s_parts[k];
        items += s_items[k];
    }
    if (has0) s_slot[at] = 2 * (int)threadIdx.x;
    if (has1) s_slot[at + has0] = 2 * (int)threadIdx.x + 1;
    if (first0 || first1) {
        const PagedPart& p = first0 ? p0 : p1;
        s_item[item] = {at + (first0 ? 0 : (int)has0), p.n, p.q0, p.h, p.i * 2 * a.tt};
    }
    if (threadIdx.x == 0) s_item[items].at = parts;
    __syncthreads();
    const int G = a.H / a.Hkv;
    const int rows = 2 * a.tt * G;
    const int slices = (rows + kRows - 1) / kRows;
    // r / G of a row (exact for r < 600, G <= 128): the divisions were half of the kernel's instructions
    const unsigned over_g = (1u << 20) / (unsigned)G + 1u;
    auto token_of = [&](int r) { return (int)(((unsigned)r * over_g) >> 20); };
    // unit: slice u of item k, the items' first slices first
    int u0 = items > 0 ? (int)blockIdx.x / items : slices, k0 = (int)blockIdx.x - u0 * items;
    auto advance = [&] {
        for (k0 += (int)gridDim.x; k0 >= items && u0 < slices; k0 -= items) ++u0;
    };
    for (; u0 < slices; advance()) {
        const Split p = s_item[k0];
        const int* slot = s_slot + p.at;
        const int count = s_item[k0 + 1].at - p.at;
        const int row0 = u0 * kRows;
        if (p.tok0 + token_of(row0) >= p.n) continue;
        const int wi = warp % W;
        float M[R], L[R], A[R][DPL];
        int r[R];
#pragma unroll
        for (int k = 0; k < R; ++k) {
            r[k] = row0 + warp / W * R + k;
            M[k] = -INFINITY;
            L[k] = 0.f;
#pragma unroll
            for (int i = 0; i < DPL; ++i) A[k][i] = 0.f;
        }
        for (int n0 = wi; n0 < count; n0 += W * kMergeBatch) {
            float2 ml[kMergeBatch][R];
            float x[kMergeBatch][R][DPL];
#pragma unroll
            for (int u = 0; u < kMergeBatch; ++u) {
                const size_t base = (size_t)slot[min(n0 + u * W, count - 1)] * rows;
#pragma unroll
                for (int k = 0; k < R; ++k) {
                    const size_t row = base + min(r[k], rows - 1);
                    load_now(a.part_ml + 2 * row, ml[u][k]);
                    load_now(a.part_acc + row * D + lane * DPL, x[u][k]);
                }
            }
#pragma unroll
            for (int k = 0; k < R; ++k) {
                float mn = M[k];
#pragma unroll
                for (int u = 0; u < kMergeBatch; ++u)
                    if (n0 + u * W < count) mn = fmaxf(mn, ml[u][k].x);
                const float ref = mn == -INFINITY ? 0.f : mn;
                const float al = ex2_approx(M[k] - ref);   // 0 while M = -inf
                M[k] = mn;
                L[k] *= al;
#pragma unroll
                for (int i = 0; i < DPL; ++i) A[k][i] *= al;
#pragma unroll
                for (int u = 0; u < kMergeBatch; ++u) {
                    if (n0 + u * W < count) {
                        const float w = ex2_approx(ml[u][k].x - ref);
                        L[k] = fmaf(w, ml[u][k].y, L[k]);
#pragma unroll
                        for (int i = 0; i < DPL; ++i) A[k][i] = fmaf(w, x[u][k][i], A[k][i]);
                    }
                }
            }
        }
        if constexpr (W > 1) {
            static_assert(R == 1, "a row a warp");
            __syncthreads();   // the unit's before has been read
#pragma unroll
            for (int i = 0; i < DPL; ++i) s_acc[warp][lane * DPL + i] = A[0][i];
            if (lane == 0) s_ml[warp] = make_float2(M[0], L[0]);
            __syncthreads();
            if (wi != 0) continue;
            M[0] = -INFINITY;
#pragma unroll
            for (int k = 0; k < W; ++k) M[0] = fmaxf(M[0], s_ml[warp + k].x);
            L[0] = 0.f;
#pragma unroll
            for (int i = 0; i < DPL; ++i) A[0][i] = 0.f;
#pragma unroll
            for (int k = 0; k < W; ++k) {
                const float2 ml = s_ml[warp + k];
                const float wk = ml.x == -INFINITY ? 0.f : ex2_approx(ml.x - M[0]);
                L[0] = fmaf(wk, ml.y, L[0]);
#pragma unroll
                for (int i = 0; i < DPL; ++i) A[0][i] = fmaf(wk, s_acc[warp + k][lane * DPL + i], A[0][i]);
            }
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            const int t = token_of(r[k]);
            const int tok = p.tok0 + t;
            if (r[k] >= rows || tok >= p.n) continue;
            const float inv = L[k] == 0.f ? 0.f : 1.f / L[k];
            const size_t row = (size_t)(p.q0 + tok) * a.H + p.h * G + r[k] - t * G;
            uint16_t* out = static_cast<uint16_t*>(a.o) + row * D + lane * DPL;
#pragma unroll
            for (int i = 0; i < DPL; i += 2)
                *reinterpret_cast<uint32_t*>(out + i) = pack_bf16x2(A[k][i] * inv, A[k][i + 1] * inv);
            if (lane == 0) a.lse[row] = L[k] == 0.f ? -INFINITY : (M[k] + __log2f(L[k])) * kLn2;
        }
    }
}

template <int D, bool FEW>
cudaError_t launch_d(const PagedTcArgs& a, int sm_count, cudaStream_t stream) {
    using C = Cfg<D, FEW>;
    auto kern = paged_tc_kernel<D, FEW>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)sm_count);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::kSmemBytes;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, kern, a.tm_q, a.tm_k, a.tm_v, a)) != cudaSuccess) return e;
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    constexpr int kW = FEW ? 8 : 1, kR = FEW ? 1 : 2;
    cfg.gridDim = dim3((unsigned)((FEW ? kMergeBlocksFew : kMergeBlocks) * sm_count));
    cfg.blockDim = dim3(kMergeThreads);
    cfg.dynamicSmemBytes = 0;
    e = cudaLaunchKernelEx(&cfg, paged_tc_merge_kernel<D / 32, kW, kR>, a, sm_count);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

int paged_tc_tokens(int G, int max_q) {
    if (G > kTile) return 0;
    const int most = kTile / G;
    return max_q >= 1 && max_q < most ? max_q : most;
}

cudaError_t launch_paged_tc(const PagedTcArgs& a, int sm_count, cudaStream_t stream) {
    const bool few = a.tt * (a.H / a.Hkv) <= kFewRows;
    sm_count = sm_count < kMergeThreads ? sm_count : kMergeThreads;   // the merge looks at a share per thread
    if (a.D == 64) return few ? launch_d<64, true>(a, sm_count, stream) : launch_d<64, false>(a, sm_count, stream);
    return few ? launch_d<128, true>(a, sm_count, stream) : launch_d<128, false>(a, sm_count, stream);
}

}  // namespace mea
