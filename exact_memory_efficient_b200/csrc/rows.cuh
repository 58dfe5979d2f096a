// rows.cuh -- fp32 arithmetic on slices of bf16 or fp32 rows, shared by the
// CUDA-core decode kernels (decode.cu, paged_attn.cu).
#pragma once

#include <cstdint>

#include "ptx.cuh"

namespace mea {

constexpr int ilog2(int x) { return x <= 1 ? 0 : 1 + ilog2(x / 2); }

// DPL consecutive elements of one row, as fp32.
__device__ __forceinline__ void load_row(const uint16_t* p, float (&x)[2]) {
    const uint32_t u = *reinterpret_cast<const uint32_t*>(p);
    x[0] = __uint_as_float(u << 16);
    x[1] = __uint_as_float(u & 0xffff0000u);
}
__device__ __forceinline__ void load_row(const uint16_t* p, float (&x)[4]) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xffff0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xffff0000u);
}
__device__ __forceinline__ void load_row(const uint16_t* p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[1]) { x[0] = *p; }
__device__ __forceinline__ void load_row(const float* p, float (&x)[2]) {
    const float2 u = *reinterpret_cast<const float2*>(p);
    x[0] = u.x;
    x[1] = u.y;
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[3]) {
    x[0] = p[0];
    x[1] = p[1];
    x[2] = p[2];
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    x[0] = u.x;
    x[1] = u.y;
    x[2] = u.z;
    x[3] = u.w;
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[6]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const float2 u = reinterpret_cast<const float2*>(p)[i];
        x[2 * i] = u.x;
        x[2 * i + 1] = u.y;
    }
}
__device__ __forceinline__ void load_row(const float* p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 u = reinterpret_cast<const float4*>(p)[i];
        x[4 * i] = u.x;
        x[4 * i + 1] = u.y;
        x[4 * i + 2] = u.z;
        x[4 * i + 3] = u.w;
    }
}

__device__ __forceinline__ void store_out(uint16_t* p, float x) {
    *p = (uint16_t)(pack_bf16x2(x, 0.f) & 0xffffu);
}
__device__ __forceinline__ void store_out(float* p, float x) { *p = x; }

// (d0, d1) += (a0, a1) * (b0, b1) as one packed fp32 FMA (each lane rounded as fmaf)
__device__ __forceinline__ void fma2(float& d0, float& d1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 pa, pb, pd;\n\t"
        "mov.b64 pa, {%2, %3};\n\t"
        "mov.b64 pb, {%4, %5};\n\t"
        "mov.b64 pd, {%0, %1};\n\t"
        "fma.rn.f32x2 pd, pa, pb, pd;\n\t"
        "mov.b64 {%0, %1}, pd;\n\t}"
        : "+f"(d0), "+f"(d1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// Dot product of DPL-element slices: pairs through the packed FMA.
template <int DPL>
__device__ __forceinline__ float dot_slice(const float (&a)[DPL], const float (&b)[DPL]) {
    float d0 = 0.f, d1 = 0.f;
#pragma unroll
    for (int i = 0; i + 1 < DPL; i += 2) fma2(d0, d1, a[i], a[i + 1], b[i], b[i + 1]);
    if constexpr (DPL % 2 == 1) d0 = fmaf(a[DPL - 1], b[DPL - 1], d0);
    return d0 + d1;
}

// acc += p * v over a DPL-element slice, pairs through the packed FMA.
template <int DPL>
__device__ __forceinline__ void axpy_slice(float (&acc)[DPL], float p, const float (&v)[DPL]) {
#pragma unroll
    for (int i = 0; i + 1 < DPL; i += 2) fma2(acc[i], acc[i + 1], p, p, v[i], v[i + 1]);
    if constexpr (DPL % 2 == 1) acc[DPL - 1] = fmaf(p, v[DPL - 1], acc[DPL - 1]);
}

// Butterfly reduce-scatter of N values (N = 8, 16 or 32) over groups of L
// lanes (L = 16 or 32, aligned): on return the lane holds the group-wide sum of
// value v = (lane mod L) >> (log2 L - log2 N).  Each halving step exchanges
// half of the remaining values with the partner lane (lane ^ o); the lanes
// left holding the same value after the halving steps are summed by plain
// butterfly steps.
template <int N, int L>
__device__ __forceinline__ float reduce_scatter(float (&x)[N], unsigned lane) {
    static_assert(N <= L, "one value per lane at least");
#pragma unroll
    for (int st = 0; (N >> st) > 1; ++st) {
        const int o = (L / 2) >> st;
        const int h = (N >> st) / 2;
        const bool upper = (lane & (unsigned)o) != 0;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            const float send = upper ? x[i] : x[i + h];
            const float keep = upper ? x[i + h] : x[i];
            x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
    float s = x[0];
#pragma unroll
    for (int o = L / (2 * N); o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

}  // namespace mea
