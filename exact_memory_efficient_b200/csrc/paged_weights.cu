// paged_weights.cu -- the attention weight that every cached key receives from
// the rows of one call, added to the cache's running sums:
//     weight_j += sum over rows i of the key's group of exp(scale q_i . k_j - lse_i),
// over the rows that see key j, with lse from the attention of the same call.
// Only Q K^T is formed: with lse known no maximum and no normalisation remain.
//
// CUDA-core kernel: a CTA owns 64 keys of one key/value head and walks over the
// rows that see them, 64 at a time, so every sum has one owner and one order
// (no atomics).  256 threads form the 64 x 64 scores, 4 x 4 each, in fp32 from
// transposed tiles in shared memory.
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "rows.cuh"

namespace mea {
namespace {

constexpr int kKeys = 64, kRows = 64, kThreads = 256;
constexpr int kPad = 4;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float as_float(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ float as_float(float x) { return x; }

template <typename T>
__global__ void __launch_bounds__(kThreads) paged_weights_kernel(const PagedWeightsArgs a) {
    extern __shared__ __align__(16) float sm[];
    float* kt = sm;                                  // [D][kKeys + kPad]
    float* qt = kt + a.D * (kKeys + kPad);           // [D][kRows + kPad]
    __shared__ float s_lse[kRows];
    __shared__ int s_lim[kRows];
    const int b = (int)blockIdx.z;
    const int kvh = (int)blockIdx.y;
    const Seq sq = load_seq(a.s, b);
    const int G = a.H / a.Hkv;
    const int total = sq.n * G;
    const int tx = (int)threadIdx.x % 16, ty = (int)threadIdx.x / 16;
    const int mask = (1 << a.s.page_shift) - 1;
    const float c = a.scale * kLog2e;
    for (long long k00 = (long long)blockIdx.x * kKeys; k00 < sq.L; k00 += (long long)gridDim.x * kKeys) {
        const int k0 = (int)k00;
        const int keys = min(kKeys, sq.L - k0);
        __syncthreads();   // the tiles of the last turn have been read
        for (int e = (int)threadIdx.x; e < kKeys * a.D; e += kThreads) {
            const int j = e / a.D, d = e - j * a.D;
            float x = 0.f;
            if (j < keys) {
                const int key = k0 + j;
                const size_t row = (((size_t)load_page(a.s, b, key >> a.s.page_shift) * a.Hkv + kvh) << a.s.page_shift) + (key & mask);
                x = as_float(static_cast<const T*>(a.k)[row * a.D + d]);
            }
            kt[d * (kKeys + kPad) + j] = x;
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        // the first row that sees key k0: token k0 - (L - n)
        const long long first = max(0LL, (long long)k0 - (sq.L - sq.n)) * G;
        for (int r0 = (int)min((long long)total, first / kRows * kRows); r0 < total; r0 += kRows) {
            __syncthreads();
            for (int e = (int)threadIdx.x; e < kRows * a.D; e += kThreads) {
                const int r = e / a.D, d = e - r * a.D;
                const int row = r0 + r;
                float x = 0.f;
                if (row < total) {
                    const int tok = row / G;
                    x = as_float(static_cast<const T*>(a.q)[(long long)(sq.q0 + tok) * a.q_stride + (size_t)(kvh * G + row - tok * G) * a.D + d]);
                }
                qt[d * (kRows + kPad) + r] = x;
            }
            if (threadIdx.x < kRows) {
                const int row = r0 + (int)threadIdx.x;
                const int tok = min(row, total - 1) / G;
                s_lim[threadIdx.x] = row < total ? min(keys, sq.L - sq.n + tok + 1 - k0) : 0;
                s_lse[threadIdx.x] = row < total ? a.lse[(size_t)(sq.q0 + tok) * a.H + kvh * G + row - tok * G] * kLog2e : 0.f;
            }
            __syncthreads();
            float acc[4][4];   // [key][row]
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
            for (int d = 0; d < a.D; ++d) {
                const float4 kv = *reinterpret_cast<const float4*>(kt + d * (kKeys + kPad) + 4 * ty);
                const float4 qv = *reinterpret_cast<const float4*>(qt + d * (kRows + kPad) + 4 * tx);
                const float kf[4] = {kv.x, kv.y, kv.z, kv.w}, qf[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(kf[i], qf[j], acc[i][j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int lim = s_lim[4 * tx + j];
                const float ls = s_lse[4 * tx + j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (4 * ty + i < lim) sum[i] += ex2_approx(fmaf(acc[i][j], c, -ls));
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int o = 1; o < 16; o <<= 1) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
            const int j = 4 * ty + i;
            if (tx == 0 && j < keys) {
                const int key = k0 + j;
                const int page = page_to_write(a.s, b, key >> a.s.page_shift);
                if (page >= 0) a.weights[(((size_t)page * a.Hkv + kvh) << a.s.page_shift) + (key & mask)] += sum[i];
            }
        }
    }
}

template <typename T>
cudaError_t launch_t(const PagedWeightsArgs& a, cudaStream_t stream) {
    auto kern = paged_weights_kernel<T>;
    const size_t smem = (size_t)a.D * (kKeys + kPad + kRows + kPad) * sizeof(float);
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    // max_kv is only a bound on what is usual: a CTA walks on from tile to tile
    const long long cap = (long long)a.s.max_pages << a.s.page_shift;
    const long long tiles = ((a.max_kv < cap ? a.max_kv : cap) + kKeys - 1) / kKeys;
    const dim3 grid((unsigned)(tiles < 1 ? 1 : tiles), (unsigned)a.Hkv, (unsigned)a.s.B);
    kern<<<grid, kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_weights_simt(const PagedWeightsArgs& a, bool bf16, cudaStream_t stream) {
    return bf16 ? launch_t<uint16_t>(a, stream) : launch_t<float>(a, stream);
}

}  // namespace mea
