// rope.cu -- rotary positions: the rotation of q and k by their tokens'
// positions, on its own (mea_rope, forward and gradient) and on the way into
// the paged cache (mea_paged_append).
//
// Pair i of a head's first `rot` values is turned by the angle pos * freq_i
// and scaled by mscale:
//     (a, b) -> mscale (a cos - b sin, b cos + a sin);
// the pairs are (x_2i, x_2i+1) (interleaved) or (x_i, x_i+rot/2).  The map is
// linear, so its gradient is the transposed map: the same with -sin.
//
// An angle of 1e6 radians has a spacing of 0.06 in fp32, so angles are formed
// in fp64 as revolutions, pos * freq / 2pi, brought into [-1/2, 1/2] by taking
// off the nearest whole number (exact), and only then rounded to fp32 for
// sincospif: the error left is 2^-24 of half a turn plus 2^-52 of the
// revolutions.  Sine and cosine, their products with mscale and those with x are
// fp32, a rounding of 2^-24 each; each result is rounded once to its type.
//
// A thread owns one 16-byte vector of a head (two at the distance rot / 2 for
// the half layout) of one token, forms its 2 to 8 sines and cosines once, and
// walks over a slice of the heads with them.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace mea {
namespace {

constexpr int kThreads = 128;
constexpr double kInvTwoPi = 0.15915494309189533577;

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);   // values per 16-byte vector

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&x)[kVec<T>]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[i]);
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&x)[kVec<T>]) {
    if constexpr (sizeof(T) == 2)
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    else
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
}

__device__ __forceinline__ uint4 load16(const void* p) { return *static_cast<const uint4*>(p); }
__device__ __forceinline__ void store16(void* p, const uint4& u) { *static_cast<uint4*>(p) = u; }

// Units of one head: the vectors (or vector pairs) that a thread owns.
template <typename T, bool INTER>
__host__ __device__ __forceinline__ int turned_units(int rot) {
    return INTER ? rot / kVec<T> : rot / (2 * kVec<T>);
}
template <typename T, bool INTER>
__host__ __device__ __forceinline__ int head_units(int D, int rot) {
    return turned_units<T, INTER>(rot) + (D - rot) / kVec<T>;
}

// Sines and cosines of a unit's pairs (VEC / 2 of them interleaved, VEC in the half layout).
template <typename T, bool INTER>
struct Turn {
    static constexpr int kPairs = INTER ? kVec<T> / 2 : kVec<T>;
    float c[kPairs], s[kPairs];
    __device__ __forceinline__ void load(const double* freq, int unit, int pos, float mscale, bool inverse) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const double rev = (double)pos * (freq[unit * kPairs + i] * kInvTwoPi);
            const float half_turns = 2.f * (float)(rev - rint(rev));
            float sn, cs;
            sincospif(half_turns, &sn, &cs);
            c[i] = cs * mscale;
            s[i] = (inverse ? -sn : sn) * mscale;
        }
    }
};

// Heads [0, heads) of one token: x points at the first head's first value, y()
// gives the same of the output, turn() the sines and cosines.  `unit` <
// turned_units turns, the others copy one vector.  The bound is HBM: loads run a
// batch of heads ahead, the first one before the addresses and angles are worked
// out (1 x 16 x 16384 x 128 bf16: 35.3 us with the loads behind them, 22.4 so;
// batches of two heads 23.8).
constexpr int kBatch = 4;

template <typename T, bool INTER, typename Y, typename A>
__device__ __forceinline__ void turn_heads(const T* x, long long x_head, long long y_head, int heads, int unit,
                                           int rot, Y&& dst, A&& turn) {
    constexpr int V = kVec<T>;
    const int turned = turned_units<T, INTER>(rot);
    const bool copies = unit >= turned;
    const int d = copies ? rot + (unit - turned) * V : unit * V;
    uint4 a[kBatch], b[kBatch];
    auto fetch = [&](int h0) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u >= heads) break;
            const T* xp = x + (h0 + u) * x_head + d;
            a[u] = load16(xp);
            if (!INTER && !copies) b[u] = load16(xp + rot / 2);
        }
    };
    fetch(0);
    T* y = dst();
    if (y == nullptr) return;
    Turn<T, INTER> t;
    if (!copies) turn(t);
    for (int h0 = 0; h0 < heads; h0 += kBatch) {
        uint4 ca[kBatch], cb[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            ca[u] = a[u];
            cb[u] = b[u];
        }
        fetch(h0 + kBatch);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            if (h0 + u >= heads) break;
            T* yp = y + (h0 + u) * y_head + d;
            if (copies) {
                store16(yp, ca[u]);
                continue;
            }
            float p[V], q[V], r[V];
            unpack<T>(ca[u], p);
            if constexpr (INTER) {
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    r[2 * i] = p[2 * i] * t.c[i] - p[2 * i + 1] * t.s[i];
                    r[2 * i + 1] = p[2 * i + 1] * t.c[i] + p[2 * i] * t.s[i];
                }
                store16(yp, pack<T>(r));
            } else {
                float w[V];
                unpack<T>(cb[u], q);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    r[i] = p[i] * t.c[i] - q[i] * t.s[i];
                    w[i] = q[i] * t.c[i] + p[i] * t.s[i];
                }
                store16(yp, pack<T>(r));
                store16(yp + rot / 2, pack<T>(w));
            }
        }
    }
}

// grid.x: B * N * units threads, grid.y: slices of per_slice heads.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeArgs a, int units, int per_slice) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)a.B * a.N * units) return;
    const long long row = id / units;
    const int unit = (int)(id - row * units);
    const long long b = row / a.N;
    const long long n = row - b * a.N;
    const int h0 = (int)blockIdx.y * per_slice;
    const T* x = static_cast<const T*>(a.x) + b * a.x_batch + n * a.x_token + h0 * a.x_head;
    T* y = static_cast<T*>(a.y) + b * a.y_batch + n * a.y_token + h0 * a.y_head;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    turn_heads<T, INTER>(
        x, a.x_head, a.y_head, min(per_slice, a.H - h0), unit, a.rot, [&] { return y; },
        [&](Turn<T, INTER>& t) { t.load(a.freq, unit, a.positions[b * a.pos_batch + n], a.mscale, a.inverse); });
}

// grid.x: T * units threads; grid.y: slices of q's heads, then of k's, then of v's.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendArgs a, int units, int copy_units, int per_slice,
                                                          int q_slices, int kv_slices) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const bool is_v = (int)blockIdx.y >= q_slices + kv_slices;
    const int u = is_v ? copy_units : units;
    if (id >= (long long)a.s.T * u) return;
    const int tok = (int)(id / u);
    const int unit = (int)(id - (long long)tok * u);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int slice = (int)blockIdx.y;
    const long long page_heads = 1LL << a.s.page_shift;   // keys of one head in a page
    int slot = 0;
    // the token's sequence and, for a key or value, its slot: the offset of head 0
    // in the cache, or -1 (rows outside every sequence stay as they were; with
    // more new tokens than keys the first ones have no slot; a page table entry
    // out of range names none)
    auto locate = [&](bool cached) -> long long {
        const int b = find_row(a.s, tok);
        if (b < 0) return -1;
        if (!cached && a.positions != nullptr) return 0;
        const Seq sq = load_seq(a.s, b);
        if (tok < sq.q0 || tok >= sq.q0 + sq.n) return -1;   // offsets that run backwards
        slot = sq.L - sq.n + (tok - sq.q0);
        if (!cached) return 0;
        if (slot < 0) return -1;
        const int page = page_to_write(a.s, b, slot >> a.s.page_shift);
        if (page < 0) return -1;
        return (long long)page * a.Hkv * page_heads + (slot & ((1 << a.s.page_shift) - 1));
    };
    auto turn = [&](Turn<T, INTER>& t) {
        t.load(a.freq, unit, a.positions ? a.positions[tok] : slot, a.mscale, false);
    };
    if (slice < q_slices) {
        const int h0 = slice * per_slice;
        turn_heads<T, INTER>(
            static_cast<const T*>(a.q) + tok * a.q_stride + (long long)h0 * a.D, a.D, a.D, min(per_slice, a.H - h0),
            unit, a.rot,
            [&]() -> T* {
                return locate(false) < 0 ? nullptr : static_cast<T*>(a.q_out) + ((long long)tok * a.H + h0) * a.D;
            },
            turn);
        return;
    }
    const int h0 = (slice - q_slices - (is_v ? kv_slices : 0)) * per_slice;
    const int heads = min(per_slice, a.Hkv - h0);
    const T* x = is_v ? static_cast<const T*>(a.v) + tok * a.v_stride : static_cast<const T*>(a.k) + tok * a.k_stride;
    // values are copied whole: every unit is behind a rotation of nothing
    turn_heads<T, INTER>(
        x + (long long)h0 * a.D, a.D, page_heads * a.D, heads, unit, is_v ? 0 : a.rot,
        [&]() -> T* {
            const long long at = locate(true);
            if (at < 0) return nullptr;
            const long long key = at + h0 * page_heads;
            if (is_v && a.weights != nullptr && unit == 0)
                for (int h = 0; h < heads; ++h) a.weights[key + h * page_heads] = 0.f;
            return static_cast<T*>(is_v ? a.v_cache : a.k_cache) + key * a.D;
        },
        turn);
}

// Heads per thread: as many as leave every SM some 768 threads (the sines are
// formed once per slice), at most 16: rope of 1 x 16 x 16384 x 128 bf16 takes
// 21.5 us, with 1,024 threads and at most 8 heads 22.4, with at most 4
// heads 25.4.
int heads_per_slice(long long threads_per_head, int H, int sm_count) {
    const long long per = threads_per_head * H / ((long long)sm_count * 768);
    const long long least = H / 32768 + 1;   // slices are a grid dimension of at most 65535
    return (int)(per < least ? least : per > 16 ? (least > 16 ? least : 16) : per);
}

// Programmatic stream serialisation: the blocks are brought up while the kernel in
// front drains, and touch nothing before its results are visible (calls back to back:
// rope of 1 x 16 x 16384 x 128 bf16 22.7 -> 20.8 us, append of 16 tokens 5.2 -> 3.4).
template <typename... P, typename... Q>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, cudaStream_t stream, const Q&... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, bool INTER>
cudaError_t launch_rope_t(const RopeArgs& a, int sm_count, cudaStream_t stream) {
    const int units = head_units<T, INTER>(a.D, a.rot);
    const long long threads = (long long)a.B * a.N * units;
    const int per = heads_per_slice(threads, a.H, sm_count);
    const long long blocks = (threads + kThreads - 1) / kThreads;
    const int slices = (a.H + per - 1) / per;
    if (blocks > 0x7fffffffLL || slices > 65535) return cudaErrorInvalidValue;
    return launch_chained(rope_kernel<T, INTER>, dim3((unsigned)blocks, (unsigned)slices), stream, a, units, per);
}

template <typename T, bool INTER>
cudaError_t launch_append_t(const AppendArgs& a, int sm_count, cudaStream_t stream) {
    const int units = head_units<T, INTER>(a.D, a.rot);
    const int copy_units = a.D / kVec<T>;
    const int heads = a.H + 2 * a.Hkv;
    const int per = heads_per_slice((long long)a.s.T * units, heads, sm_count);
    const int q_slices = (a.H + per - 1) / per;
    const int kv_slices = (a.Hkv + per - 1) / per;
    const long long blocks = ((long long)a.s.T * copy_units + kThreads - 1) / kThreads;   // copy_units >= units
    if (blocks > 0x7fffffffLL || q_slices + 2 * kv_slices > 65535) return cudaErrorInvalidValue;
    return launch_chained(append_kernel<T, INTER>, dim3((unsigned)blocks, (unsigned)(q_slices + 2 * kv_slices)), stream,
                          a, units, copy_units, per, q_slices, kv_slices);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool bf16, int sm_count, cudaStream_t stream) {
    if (bf16)
        return a.interleaved ? launch_rope_t<uint16_t, true>(a, sm_count, stream)
                             : launch_rope_t<uint16_t, false>(a, sm_count, stream);
    return a.interleaved ? launch_rope_t<float, true>(a, sm_count, stream)
                         : launch_rope_t<float, false>(a, sm_count, stream);
}

cudaError_t launch_append(const AppendArgs& a, bool bf16, int sm_count, cudaStream_t stream) {
    if (bf16)
        return a.interleaved ? launch_append_t<uint16_t, true>(a, sm_count, stream)
                             : launch_append_t<uint16_t, false>(a, sm_count, stream);
    return a.interleaved ? launch_append_t<float, true>(a, sm_count, stream)
                         : launch_append_t<float, false>(a, sm_count, stream);
}

}  // namespace mea
