// paged_attn.cu -- attention of ragged chunks of new tokens over a paged cache
// on the CUDA cores (any supported type and head dim, any number of rows), and
// the merge of the chunk summaries that the paged kernels leave.
//
// For new token i of a sequence's n, with L cached keys (the n new ones last):
//     o_i = sum_j p_ij v_j,  p_ij = exp(scale q_i . k_j - lse_i),  j < L - n + i + 1,
// with the running maximum, exp-sum and rescaled accumulator of "Self-attention
// Does Not Need O(n^2) Memory" (English summary, method bullets 1-4).  A row
// that sees no key gets o = 0 and lse = -inf.
//
// The rows of one key/value head are its n * G (token, head of the group)
// pairs, token by token; a CTA takes 1, 2, 4 or 8 of them over one chunk of
// their keys.  The arithmetic is that of decode.cu (its header explains the
// lane layout and the reduce-scatter): K and V stream through a ring of
// 64-key stages, here filled page by page, one bulk copy per page and tensor,
// and each (key, row) score has a mask of its own.  Keys behind a sequence's
// last are never copied; shared memory they would occupy is never used.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace mea {
namespace {

constexpr int kTK = kDecodeTileKeys;             // keys per tile
constexpr int kCompWarps = 8;                    // compute warps
constexpr int kKeysPerWarp = kTK / kCompWarps;   // keys of a tile per compute warp
constexpr int kThreads = 32 * (kCompWarps + 1);  // + producer warp
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleThreshold = 8.0f;        // log2 of the largest weight left unrescaled

template <typename T, int DPL, int RMAX>
struct Cfg {
    static constexpr int D = 32 * DPL;
    static constexpr int LPK = (RMAX == 2 || RMAX == 4) ? 16 : 32;   // lanes per key
    static constexpr int kGroups = 32 / LPK;              // key groups per warp (1 or 2)
    static constexpr int kKPG = kKeysPerWarp / kGroups;   // keys per group in a tile
    static constexpr int DL = D / LPK;                    // head dims per lane
    static constexpr int kRowBytes = D * (int)sizeof(T);
    static constexpr int kTileBytes = kTK * kRowBytes;   // K or V part of a stage
    static constexpr int kStageBytes = 2 * kTileBytes;
    static constexpr int kMinBlocks = (RMAX <= 4 && kStageBytes <= 32768) ? (RMAX == 1 ? 3 : 2) : 1;
    static constexpr int kRingBudget = (kMinBlocks == 3 ? 64 : kMinBlocks == 2 ? 96 : 192) * 1024;
    static constexpr int kStages = kRingBudget / kStageBytes < 2 ? 2 : kRingBudget / kStageBytes;
    static constexpr int RR = RMAX < 4 ? RMAX : 4;        // rows per pass
    static constexpr int kPasses = RMAX / RR;
    static constexpr int kN = kKPG * RR;                  // values per reduce-scatter: 8, 16 or 32
    static constexpr int kSh = ilog2(LPK) - ilog2(kN);    // lane in group -> value: v = li >> kSh
    static constexpr int kScratchBytes = kCompWarps * RMAX * (D + 2) * 4;
    static constexpr int kRingBytes = kStages * kStageBytes;
    static constexpr int kSmemData = kRingBytes > kScratchBytes ? kRingBytes : kScratchBytes;
    static constexpr int kSmemBytes = kSmemData + 2 * 8 * kStages + 16;
    static_assert(kSmemBytes <= 227 * 1024, "shared memory");
};

// One tile of rows of one key/value head, and the part of its keys that a CTA takes.
struct Item {
    Seq sq;
    int b, r0, rows;           // first row in the sequence's n * G, rows that exist (0: nothing to do)
    int begin, end;            // keys
};

__device__ __forceinline__ Item load_item(const PagedAttnArgs& a, int x, int split) {
    Item it;
    it.rows = 0;
    int tile;
    const int G = a.H / a.Hkv;
    it.b = find_tile(a.s, x, G, a.rows, &tile);
    if (it.b < 0) return it;
    it.sq = load_seq(a.s, it.b);
    const long long total = (long long)it.sq.n * G;
    const long long r0 = (long long)tile * a.rows;
    if (r0 >= total) return it;
    it.r0 = (int)r0;
    it.rows = (int)min((long long)a.rows, total - r0);
    // what the tile's last row sees
    const int last = (it.r0 + it.rows - 1) / G;
    const int kmax = max(0, it.sq.L - it.sq.n + last + 1);
    if (a.nsplit == 1) {
        it.begin = 0;
        it.end = kmax;
    } else {
        const int tiles = (kmax + kTK - 1) / kTK;
        const int per = (tiles + a.nsplit - 1) / a.nsplit * kTK;
        it.begin = (int)min((long long)kmax, (long long)split * per);
        it.end = (int)min((long long)kmax, (long long)it.begin + per);
    }
    return it;
}

template <typename T, int DPL, int RMAX>
__global__ void __launch_bounds__(kThreads, Cfg<T, DPL, RMAX>::kMinBlocks)
paged_simt_kernel(const PagedAttnArgs a) {
    using C = Cfg<T, DPL, RMAX>;
    constexpr int D = C::D;
    constexpr int RR = C::RR;
    constexpr int kSh = C::kSh;
    extern __shared__ __align__(16) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kSmemData);
    uint64_t* empty = full + C::kStages;
    int* abort_flag = reinterpret_cast<int*>(empty + C::kStages);
    int* issued_s = abort_flag + 1;
    const unsigned warp = warp_id();
    const unsigned lane = lane_id();

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kCompWarps);
        }
        *abort_flag = 0;
        *issued_s = 0;
        fence_mbar_init();
    }
    __syncthreads();
    // programmatic stream serialisation: nothing global is touched before the
    // previous kernel's results are complete and visible
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const int kvh = (int)blockIdx.y;
    const int split = (int)blockIdx.z;
    const Item it = load_item(a, (int)blockIdx.x, split);
    if (it.rows == 0) return;
    const int G = a.H / a.Hkv;
    const int n_keys = it.end - it.begin;
    const int n_tiles = (n_keys + kTK - 1) / kTK;

    if (warp == kCompWarps) {
        if (lane == 0) {
            const int shift = a.s.page_shift;
            const int per = min(kTK, 1 << shift);          // keys per copy
            const T* kg = static_cast<const T*>(a.k);
            const T* vg = static_cast<const T*>(a.v);
            int page[kTK / 16];                             // pages of the next tile, loaded ahead
            auto pages_of = [&](int t) {
                const int key0 = it.begin + t * kTK;
#pragma unroll
                for (int i = 0; i < kTK / 16; ++i)
                    if (i * per < kTK && key0 + i * per < it.end) page[i] = load_page(a.s, it.b, (key0 + i * per) >> shift);
            };
            if (n_tiles > 0) pages_of(0);
            int t = 0;
            for (; t < n_tiles; ++t) {
                const int s = t % C::kStages;
                if (t >= C::kStages && !mbar_wait(&empty[s], ((t / C::kStages) - 1) & 1, abort_flag)) break;
                const int key0 = it.begin + t * kTK;
                const int keys = min(kTK, it.end - key0);
                uint8_t* st = smem + (size_t)s * C::kStageBytes;
                mbar_arrive_expect_tx(&full[s], 2u * (unsigned)(keys * C::kRowBytes));
#pragma unroll
                for (int i = 0; i < kTK / 16; ++i) {
                    const int k0 = i * per;
                    if (k0 >= keys) break;
                    const unsigned bytes = (unsigned)(min(per, keys - k0) * C::kRowBytes);
                    const size_t at = ((((size_t)page[i] * a.Hkv + kvh) << shift) + ((key0 + k0) & ((1 << shift) - 1))) * D;
                    bulk_load(st + k0 * C::kRowBytes, kg + at, bytes, &full[s]);
                    bulk_load(st + C::kTileBytes + k0 * C::kRowBytes, vg + at, bytes, &full[s]);
                }
                if (t + 1 < n_tiles) pages_of(t + 1);
            }
            *issued_s = t;
        }
    } else {
        // ---------------------------------------------------------- compute
        // Lane = (group g, lane-in-group li): group g takes keys
        // [8w + g*kKPG, 8w + (g+1)*kKPG) of every tile, and li owns head dims
        // [li*DL, (li+1)*DL) of q, of those keys' K/V rows and of acc.
        constexpr int LPK = C::LPK;
        constexpr int DL = C::DL;
        constexpr int kKPG = C::kKPG;
        const int w = (int)warp;
        const int g = (int)(lane / LPK);
        const int li = (int)(lane % LPK);
        float qr[RMAX][DL];
        {
            const float qs = a.scale * kLog2e;
            const T* qg = static_cast<const T*>(a.q) + (size_t)kvh * G * D + li * DL;
#pragma unroll
            for (int r = 0; r < RMAX; ++r) {
                if (r < it.rows) {
                    const int row = it.r0 + r;
                    const int tok = row / G;
                    load_row(qg + (long long)(it.sq.q0 + tok) * a.q_stride + (size_t)(row - tok * G) * D, qr[r]);
#pragma unroll
                    for (int i = 0; i < DL; ++i) qr[r][i] *= qs;
                } else {
#pragma unroll
                    for (int i = 0; i < DL; ++i) qr[r][i] = 0.f;
                }
            }
        }
        float acc[RMAX][DL];
#pragma unroll
        for (int r = 0; r < RMAX; ++r)
#pragma unroll
            for (int i = 0; i < DL; ++i) acc[r][i] = 0.f;
        // this lane's (key, row) value of the reduce-scatter, per pass
        const int v_mine = li >> kSh;
        const int j_mine = v_mine / RR;
        const int rr_mine = v_mine % RR;
        float m_mine[C::kPasses], l_mine[C::kPasses];
        int lim_mine[C::kPasses];                   // keys from it.begin that the lane's row sees
#pragma unroll
        for (int p = 0; p < C::kPasses; ++p) {
            m_mine[p] = -INFINITY;
            l_mine[p] = 0.f;
            const int row = it.r0 + min(p * RR + rr_mine, it.rows - 1);
            lim_mine[p] = min(it.end, it.sq.L - it.sq.n + row / G + 1) - it.begin;
        }

        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % C::kStages;
            if (!mbar_wait(&full[s], (t / C::kStages) & 1, abort_flag)) break;
            const int key0 = w * kKeysPerWarp + g * kKPG;            // first key of this group in the tile
            const T* ks = reinterpret_cast<const T*>(smem + (size_t)s * C::kStageBytes) + (size_t)key0 * D + li * DL;
            const T* vs = ks + C::kTileBytes / (int)sizeof(T);
            // keys of this group in this tile that exist; rows past them hold
            // stale or unwritten shared memory and are never used
            const int valid = min(kKPG, max(0, n_keys - t * kTK - key0));
#pragma unroll
            for (int p = 0; p < C::kPasses; ++p) {
                float part[C::kN];
#pragma unroll
                for (int j = 0; j < kKPG; ++j) {
                    float kf[DL];
                    load_row(ks + j * D, kf);
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) part[j * RR + rr] = dot_slice<DL>(qr[p * RR + rr], kf);
                }
                float sv = reduce_scatter<C::kN, LPK>(part, lane);
                sv = (t * kTK + key0 + j_mine < lim_mine[p]) ? sv : -INFINITY;
                float& m = m_mine[p];
                if (__any_sync(0xffffffffu, sv > m + kRescaleThreshold)) {
                    // exact maximum of this tile per row: over the lanes of the same row
                    float tmax = sv;
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) tmax = fmaxf(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
                    const float mn = fmaxf(m, tmax);
                    const float alpha = (mn == -INFINITY) ? 1.f : ex2_approx(m - mn);
                    m = mn;
                    l_mine[p] *= alpha;
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) {
                        const float ar = __shfl_sync(0xffffffffu, alpha, rr << kSh);
#pragma unroll
                        for (int i = 0; i < DL; ++i) acc[p * RR + rr][i] *= ar;
                    }
                }
                const float pw = (m == -INFINITY) ? 0.f : ex2_approx(sv - m);
                l_mine[p] += pw;
#pragma unroll
                for (int j = 0; j < kKPG; ++j) {
                    float vf[DL];
                    if (j < valid) {
                        load_row(vs + j * D, vf);
                    } else {
#pragma unroll
                        for (int i = 0; i < DL; ++i) vf[i] = 0.f;
                    }
#pragma unroll
                    for (int rr = 0; rr < RR; ++rr) {
                        const float pj = __shfl_sync(0xffffffffu, pw, g * LPK + ((j * RR + rr) << kSh));
                        axpy_slice<DL>(acc[p * RR + rr], pj, vf);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        // exp-sum of this warp's keys per row: over the key lanes and groups of each row
#pragma unroll
        for (int p = 0; p < C::kPasses; ++p)
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l_mine[p] += __shfl_xor_sync(0xffffffffu, l_mine[p], o);
        // the groups of a warp accumulate the same dims over different keys
        if constexpr (C::kGroups == 2) {
#pragma unroll
            for (int r = 0; r < RMAX; ++r)
#pragma unroll
                for (int i = 0; i < DL; ++i) acc[r][i] += __shfl_xor_sync(0xffffffffu, acc[r][i], 16);
        }

        // all compute warps are past the ring before it is reused as scratch
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kCompWarps) : "memory");
        float* sc_acc = reinterpret_cast<float*>(smem);                 // [warp][RMAX][D]
        float* sc_ml = sc_acc + kCompWarps * RMAX * D;                  // [warp][RMAX][2]
        if (g == 0) {
#pragma unroll
            for (int r = 0; r < RMAX; ++r)
#pragma unroll
                for (int i = 0; i < DL; ++i) sc_acc[(w * RMAX + r) * D + li * DL + i] = acc[r][i];
        }
#pragma unroll
        for (int p = 0; p < C::kPasses; ++p) {
            // lane (rr << kSh) holds row p*RR + rr (key 0 of the value index)
            if (g == 0 && (li & ((1 << kSh) - 1)) == 0 && j_mine == 0) {
                const int r = p * RR + v_mine;
                sc_ml[(w * RMAX + r) * 2] = m_mine[p];
                sc_ml[(w * RMAX + r) * 2 + 1] = l_mine[p];
            }
        }
        asm volatile("bar.sync 1, %0;" ::"n"(32 * kCompWarps) : "memory");
        if (!*abort_flag) {
            for (int e = (int)threadIdx.x; e < it.rows * D; e += 32 * kCompWarps) {
                const int r = e / D;
                const int d = e - r * D;
                float M = -INFINITY;
#pragma unroll
                for (int ww = 0; ww < kCompWarps; ++ww) M = fmaxf(M, sc_ml[(ww * RMAX + r) * 2]);
                float L = 0.f, A = 0.f;
#pragma unroll
                for (int ww = 0; ww < kCompWarps; ++ww) {
                    const float mw = sc_ml[(ww * RMAX + r) * 2];
                    const float wt = (mw == -INFINITY) ? 0.f : ex2_approx(mw - M);
                    L = fmaf(wt, sc_ml[(ww * RMAX + r) * 2 + 1], L);
                    A = fmaf(wt, sc_acc[(ww * RMAX + r) * D + d], A);
                }
                const int row = it.r0 + r;
                const int tok = row / G;
                const size_t orow = (size_t)(it.sq.q0 + tok) * a.H + (size_t)kvh * G + (row - tok * G);
                if (a.nsplit == 1) {
                    // no key in sight: o = 0, lse = -inf
                    store_out(static_cast<T*>(a.o) + orow * D + d, L == 0.f ? 0.f : A / L);
                    if (d == 0) a.lse[orow] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
                } else {
                    const size_t prow = (size_t)split * a.s.T * a.H + orow;
                    a.part_acc[prow * D + d] = A;
                    if (d == 0) {
                        a.part_ml[prow * 2] = M;
                        a.part_ml[prow * 2 + 1] = L;
                    }
                }
            }
        }
    }
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) {
        // a wait gave up: let every copy still in flight land before the CTA
        // (and its shared memory) goes away
        const int issued = *issued_s;
        for (int t = issued - C::kStages < 0 ? 0 : issued - C::kStages; t < issued; ++t)
            mbar_wait(&full[t % C::kStages], (t / C::kStages) & 1, nullptr);
    }
}

// Merge of the chunk summaries: W warps per packed (token, head) row, each lane
// owning D / 32 head dims; chunk c goes to warp c mod W of the row.  A summary
// of no keys has m = -inf and its accumulator is not read.
constexpr int kMergeThreads = 256;
constexpr int kMergeBatch = 4;

template <typename T, int DPL, int W>
__global__ void __launch_bounds__(kMergeThreads) paged_merge_kernel(const PagedAttnArgs a) {
    constexpr int D = 32 * DPL;
    constexpr int kRows = kMergeThreads / 32 / W;   // rows per CTA
    __shared__ float s_acc[W > 1 ? W : 1][D];
    __shared__ float s_ml[W > 1 ? W : 1][2];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = (int)warp_id();
    const int lane = (int)lane_id();
    const long long rows = (long long)a.s.T * a.H;
    const long long row = (long long)blockIdx.x * kRows + warp / W;
    const int wi = warp % W;
    // rows outside every sequence stay as they were
    if (row >= rows || find_row(a.s, (int)(row / a.H)) < 0) return;   // W > 1: one row per CTA, uniform
    float M = -INFINITY, L = 0.f, A[DPL];
#pragma unroll
    for (int i = 0; i < DPL; ++i) A[i] = 0.f;
    for (int c0 = wi; c0 < a.nsplit; c0 += W * kMergeBatch) {
        float mc[kMergeBatch], lc[kMergeBatch], x[kMergeBatch][DPL];
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            const int c = c0 + u * W;
            mc[u] = -INFINITY;
            if (c < a.nsplit) {
                const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + (c * rows + row) * 2);
                mc[u] = ml.x;
                lc[u] = ml.y;
                load_row(a.part_acc + (c * rows + row) * D + lane * DPL, x[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kMergeBatch; ++u) {
            if (mc[u] == -INFINITY) continue;
            const float mn = fmaxf(M, mc[u]);
            const float al = ex2_approx(M - mn);   // 0 while M = -inf
            const float wc = ex2_approx(mc[u] - mn);
            M = mn;
            L = fmaf(wc, lc[u], L * al);
#pragma unroll
            for (int i = 0; i < DPL; ++i) A[i] = fmaf(wc, x[u][i], A[i] * al);
        }
    }
    if constexpr (W > 1) {
#pragma unroll
        for (int i = 0; i < DPL; ++i) s_acc[wi][lane * DPL + i] = A[i];
        if (lane == 0) {
            s_ml[wi][0] = M;
            s_ml[wi][1] = L;
        }
        __syncthreads();
        if (wi != 0) return;
        M = -INFINITY;
#pragma unroll
        for (int k = 0; k < W; ++k) M = fmaxf(M, s_ml[k][0]);
        L = 0.f;
#pragma unroll
        for (int i = 0; i < DPL; ++i) A[i] = 0.f;
        for (int k = 0; k < W; ++k) {
            if (s_ml[k][0] == -INFINITY) continue;
            const float wk = ex2_approx(s_ml[k][0] - M);
            L = fmaf(wk, s_ml[k][1], L);
#pragma unroll
            for (int i = 0; i < DPL; ++i) A[i] = fmaf(wk, s_acc[k][lane * DPL + i], A[i]);
        }
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
    T* out = static_cast<T*>(a.o) + row * D + lane * DPL;
    if constexpr (sizeof(T) == 2 && DPL % 2 == 0) {
#pragma unroll
        for (int i = 0; i < DPL; i += 2)
            *reinterpret_cast<uint32_t*>(out + i) = pack_bf16x2(A[i] * inv, A[i + 1] * inv);
    } else {
#pragma unroll
        for (int i = 0; i < DPL; ++i) store_out(out + i, A[i] * inv);
    }
    if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
}

template <typename K>
cudaError_t launch_chained(K kern, dim3 grid, unsigned threads, size_t smem, const PagedAttnArgs& a,
                           cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int DPL, int RMAX>
cudaError_t launch_rows(const PagedAttnArgs& a, cudaStream_t stream) {
    using C = Cfg<T, DPL, RMAX>;
    auto kern = paged_simt_kernel<T, DPL, RMAX>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
    if (e != cudaSuccess) return e;
    const long long tiles = (long long)a.s.T * (a.H / a.Hkv) / RMAX + a.s.B;
    if (tiles > 0x7fffffffLL || a.Hkv > 65535 || a.nsplit < 1 || a.nsplit > 65535) return cudaErrorInvalidValue;
    return launch_chained(kern, dim3((unsigned)tiles, (unsigned)a.Hkv, (unsigned)a.nsplit), kThreads, C::kSmemBytes,
                          a, stream);
}

template <typename T, int DPL>
cudaError_t dispatch_rows(const PagedAttnArgs& a, cudaStream_t stream) {
    // bf16 comes here with groups above 128 heads alone: always eight rows
    if constexpr (sizeof(T) == 2) return launch_rows<T, DPL, 8>(a, stream);
    else switch (a.rows) {
        case 1: return launch_rows<T, DPL, 1>(a, stream);
        case 2: return launch_rows<T, DPL, 2>(a, stream);
        case 4: return launch_rows<T, DPL, 4>(a, stream);
        default: return launch_rows<T, DPL, 8>(a, stream);
    }
}

template <typename T, int DPL>
int blocks_rows(int rows) {
    if constexpr (sizeof(T) == 2) return Cfg<T, DPL, 8>::kMinBlocks;
    return rows <= 1 ? Cfg<T, DPL, 1>::kMinBlocks : rows <= 2 ? Cfg<T, DPL, 2>::kMinBlocks
         : rows <= 4 ? Cfg<T, DPL, 4>::kMinBlocks : Cfg<T, DPL, 8>::kMinBlocks;
}

template <typename T, int DPL>
cudaError_t merge_rows(const PagedAttnArgs& a, cudaStream_t stream) {
    const long long rows = (long long)a.s.T * a.H;
    // many chunks of few rows: a CTA per row, or the chunks are read one after the other
    const bool wide = a.nsplit > 8;
    const long long blocks = wide ? rows : (rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    return wide ? launch_chained(paged_merge_kernel<T, DPL, 8>, dim3((unsigned)blocks), kMergeThreads, 0, a, stream)
                : launch_chained(paged_merge_kernel<T, DPL, 1>, dim3((unsigned)blocks), kMergeThreads, 0, a, stream);
}

}  // namespace

int paged_simt_blocks_per_sm(bool bf16, int D, int rows) {
    if (bf16) return D == 64 ? blocks_rows<uint16_t, 2>(rows) : blocks_rows<uint16_t, 4>(rows);
    switch (D) {
        case 32: return blocks_rows<float, 1>(rows);
        case 64: return blocks_rows<float, 2>(rows);
        case 96: return blocks_rows<float, 3>(rows);
        default: return blocks_rows<float, 4>(rows);
    }
}

cudaError_t launch_paged_simt(const PagedAttnArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.D == 64 ? dispatch_rows<uint16_t, 2>(a, stream) : dispatch_rows<uint16_t, 4>(a, stream);
    switch (a.D) {
        case 32: return dispatch_rows<float, 1>(a, stream);
        case 64: return dispatch_rows<float, 2>(a, stream);
        case 96: return dispatch_rows<float, 3>(a, stream);
        default: return dispatch_rows<float, 4>(a, stream);
    }
}

cudaError_t launch_paged_merge(const PagedAttnArgs& a, bool bf16, cudaStream_t stream) {
    if (bf16) return a.D == 64 ? merge_rows<uint16_t, 2>(a, stream) : merge_rows<uint16_t, 4>(a, stream);
    switch (a.D) {
        case 32: return merge_rows<float, 1>(a, stream);
        case 64: return merge_rows<float, 2>(a, stream);
        case 96: return merge_rows<float, 3>(a, stream);
        default: return merge_rows<float, 4>(a, stream);
    }
}

}  // namespace mea
