// api_paged.cu -- the C entry points of rotary positions and the paged
// key/value cache (include/mea_attn.h): argument validation, launch plans and
// launches on the caller's stream.  Nothing here allocates or synchronises.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_internal.h"
#include "kernels.h"

namespace {

using mea::api_fail;

bool aligned(const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }

mea_status_t invalid(const char* where, const char* what) { return api_fail(MEA_ERR_INVALID_ARG, where, what); }

mea_status_t check_dtype(const char* where, int D, mea_dtype_t dtype) {
    if (dtype != MEA_DTYPE_F32 && dtype != MEA_DTYPE_BF16) return invalid(where, "unknown dtype");
    if (D <= 0) return invalid(where, "head dim not positive");
    if (dtype == MEA_DTYPE_BF16 && D != 64 && D != 128)
        return api_fail(MEA_ERR_UNSUPPORTED, where, "bf16 head dims are 64 and 128");
    if (dtype == MEA_DTYPE_F32 && (D % 32 != 0 || D > 128))
        return api_fail(MEA_ERR_UNSUPPORTED, where, "fp32 head dims are 32, 64, 96 and 128");
    return MEA_OK;
}

mea_status_t check_rope(const char* where, int rot_dim, int D, mea_rope_layout_t layout, float mscale) {
    if (layout != MEA_ROPE_HALF && layout != MEA_ROPE_INTERLEAVED) return invalid(where, "unknown rotary layout");
    if (rot_dim <= 0 || rot_dim > D) return invalid(where, "rot_dim must be in 1..D");
    if (rot_dim % 16 != 0) return api_fail(MEA_ERR_UNSUPPORTED, where, "rot_dim must be a multiple of 16");
    if (!std::isfinite(mscale)) return invalid(where, "mscale not finite");
    return MEA_OK;
}

// Sizes of a ragged batch over a paged cache.
mea_status_t check_batch(const char* where, int T, int B, int H_kv, int D, int num_pages, int page_size,
                         int max_pages, mea_dtype_t dtype) {
    mea_status_t st = check_dtype(where, D, dtype);
    if (st != MEA_OK) return st;
    if (T < 0 || B < 0 || num_pages < 0 || max_pages < 0) return invalid(where, "negative size");
    if (H_kv < 1) return invalid(where, "H_kv below 1");
    if (page_size <= 0) return invalid(where, "page_size not positive");
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
        return api_fail(MEA_ERR_UNSUPPORTED, where, "page_size must be 16, 32, 64, 128 or 256");
    if ((long long)max_pages * page_size > 0x7fffffffLL - 65536) return invalid(where, "max_pages * page_size too large");
    if ((long long)num_pages * H_kv > 0x7fffffffLL) return invalid(where, "num_pages * H_kv too large");
    if (B > 65535 || H_kv > 65535)
        return api_fail(MEA_ERR_UNSUPPORTED, where, "at most 65535 sequences and key/value heads");
    return MEA_OK;
}

mea_status_t check_heads(const char* where, int T, int H, int H_kv, int D, long long q_stride) {
    if (H < 1 || H % H_kv != 0) return invalid(where, "H must be a multiple of H_kv");
    if ((long long)T * H > 0x7fffffffLL - 65536) return invalid(where, "T * H too large");
    if (q_stride < (long long)H * D) return invalid(where, "token stride of q below H * D");
    if (q_stride % 8 != 0) return api_fail(MEA_ERR_MISALIGNED, where, "token stride of q not a multiple of 8");
    return MEA_OK;
}

mea::PagedBatch batch_of(const int* cu_q, const int* kv_len, const int* page_table, int T, int B, int num_pages,
                         int page_size, int max_pages) {
    mea::PagedBatch s;
    s.cu_q = cu_q;
    s.kv_len = kv_len;
    s.page_table = page_table;
    s.B = B;
    s.T = T;
    s.max_pages = max_pages;
    s.num_pages = num_pages;
    s.page_shift = 0;
    while ((1 << s.page_shift) < page_size) ++s.page_shift;
    return s;
}

// Rows per tile of the CUDA-core kernel: what one sequence brings to a key/value head, up to 8.
int simt_rows(int G, int max_q) {
    const long long rows = (long long)G * (max_q < 1 ? 1 : max_q);
    return rows <= 1 ? 1 : rows <= 2 ? 2 : rows <= 4 ? 4 : 8;
}

struct AttnPlan {
    int tt = 0;                // tokens per query tile of the tensor-core kernel; 0: the CUDA-core kernel
    int rows = 1;
    int nsplit = 1;
    size_t ws_bytes = 0;
};

// Chunks of the keys so that the launch fills the device's slots about once.
AttnPlan attn_plan(int sm_count, int T, int B, int H, int H_kv, int D, int max_q, int max_kv, bool bf16) {
    AttnPlan p;
    if (bf16 && (p.tt = mea::paged_tc_tokens(H / H_kv, max_q)) > 0) {
        p.rows = 2 * p.tt * (H / H_kv);
        p.ws_bytes = (size_t)2 * sm_count * (p.rows * (D + 2) * sizeof(float) + sizeof(mea::PagedPart));
        return p;
    }
    p.rows = simt_rows(H / H_kv, max_q);
    const long long tiles = std::max(1LL, (long long)T * (H / H_kv) / p.rows) * H_kv;
    const long long slots = (long long)sm_count * mea::paged_simt_blocks_per_sm(bf16, D, p.rows);
    const long long key_tiles = std::max(1LL, ((long long)max_kv + mea::kDecodeTileKeys - 1) / mea::kDecodeTileKeys);
    p.nsplit = (int)std::max(1LL, std::min(slots / tiles, key_tiles));
    if (p.nsplit > 1) p.ws_bytes = (size_t)p.nsplit * T * H * (D + 2) * sizeof(float);
    return p;
}

// Maps of packed q (boxes of tt tokens of one group) and of a cache's pages.
mea_status_t map_q(CUtensorMap* m, const void* q, int T, int H, int G, int D, long long q_stride, int tt) {
    const cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)tt};
    return mea::api_map_bf16(m, q, 3, dims, strides, box, "q");
}
mea_status_t map_pages(CUtensorMap* m, const void* cache, int num_pages, int H_kv, int page_size, int D) {
    // {64 head dims, 8 keys, blocks of head dims, groups of 8 keys, (page, head)}: PageTile's layout
    const cuuint64_t dims[5] = {64, 8, (cuuint64_t)D / 64, (cuuint64_t)page_size / 8, (cuuint64_t)num_pages * H_kv};
    const cuuint64_t strides[4] = {(cuuint64_t)D * 2, 128, (cuuint64_t)D * 16, (cuuint64_t)page_size * D * 2};
    const cuuint32_t box[5] = {64, 8, (cuuint32_t)D / 64, (cuuint32_t)std::min(page_size, 128) / 8, 1};
    return mea::api_map_bf16(m, cache, 5, dims, strides, box, "cache");
}

struct WeightsPlan {
    int tt = 0;                // 0: the CUDA-core kernel
    bool split = false;
    size_t ws_bytes = 0;
};
// Where one query tile holds all new tokens of a sequence an item has one unit
// and nothing to split.
WeightsPlan weights_plan(int sm_count, int G, int max_q, bool bf16) {
    WeightsPlan p;
    if (!bf16 || (p.tt = mea::paged_tc_tokens(G, max_q)) == 0) return p;
    p.split = max_q > p.tt;
    if (p.split) p.ws_bytes = (size_t)2 * sm_count * (mea::kWeightsPartKeys * sizeof(float) + sizeof(mea::PagedPart));
    return p;
}

}  // namespace

extern "C" {

mea_status_t mea_rope_frequencies(double* freq, int rot_dim, double base, mea_rope_scaling_t scaling, double factor,
                                  double original_len, double slow, double fast) {
    const char* where = "mea_rope_frequencies";
    if (freq == nullptr || rot_dim <= 0 || rot_dim % 2 != 0) return invalid(where, "freq or rot_dim");
    if (!std::isfinite(base) || !(base > 1.0)) return invalid(where, "base must be above 1");
    if (!std::isfinite(factor) || !(factor >= 1.0)) return invalid(where, "factor must be at least 1");
    const double pi = std::acos(-1.0);
    switch (scaling) {
        case MEA_ROPE_SCALE_NONE:
        case MEA_ROPE_SCALE_LINEAR:
            break;
        case MEA_ROPE_SCALE_BASE:
            if (rot_dim <= 2) return invalid(where, "rot_dim must be above 2 for a scaled base");
            base *= std::pow(factor, (double)rot_dim / (rot_dim - 2));
            break;
        case MEA_ROPE_SCALE_BY_PARTS:
            if (!std::isfinite(original_len) || !(original_len > 0.0)) return invalid(where, "original_len must be positive");
            if (!std::isfinite(slow) || !std::isfinite(fast) || !(slow < fast)) return invalid(where, "slow must be below fast");
            break;
        default:
            return invalid(where, "unknown scaling");
    }
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (scaling == MEA_ROPE_SCALE_LINEAR) f /= factor;
        if (scaling == MEA_ROPE_SCALE_BY_PARTS) {
            const double turns = original_len * f / (2.0 * pi);   // over the original context
            const double keep = std::min(1.0, std::max(0.0, (turns - slow) / (fast - slow)));
            f = (1.0 - keep) * f / factor + keep * f;
        }
        freq[i] = f;
    }
    return MEA_OK;
}

mea_status_t mea_rope(const void* x, void* y, const int* positions, const double* freq, int B, int H, int N, int D,
                      int rot_dim, int positions_per_batch, mea_rope_layout_t layout, float mscale, int inverse,
                      mea_dtype_t dtype, void* stream) {
    const char* where = "mea_rope";
    mea_status_t st = check_dtype(where, D, dtype);
    if (st != MEA_OK) return st;
    if (B < 0 || H < 0 || N < 0) return invalid(where, "negative size");
    if ((st = check_rope(where, rot_dim, D, layout, mscale)) != MEA_OK) return st;
    if ((long long)B * H > 0x7fffffffLL || (long long)B * H * N >= (1LL << 40) / D) return invalid(where, "too many elements");
    if ((long long)B * N > (1LL << 31) - 1) return api_fail(MEA_ERR_UNSUPPORTED, where, "B * N too large");
    if (B == 0 || H == 0 || N == 0) return MEA_OK;
    if (!x || !y || !positions || !freq) return invalid(where, "null pointer");
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(positions, 4) || !aligned(freq, 8)) return MEA_ERR_MISALIGNED;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    mea::RopeArgs a;
    a.x = x;
    a.y = y;
    a.positions = positions;
    a.freq = freq;
    a.x_token = a.y_token = D;
    a.x_head = a.y_head = (long long)N * D;
    a.x_batch = a.y_batch = (long long)H * N * D;
    a.pos_batch = positions_per_batch ? N : 0;
    a.B = B;
    a.H = H;
    a.N = N;
    a.D = D;
    a.rot = rot_dim;
    a.interleaved = layout == MEA_ROPE_INTERLEAVED;
    a.inverse = inverse != 0;
    a.mscale = mscale;
    return mea::api_cuda(mea::launch_rope(a, dtype == MEA_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)), where);
}

mea_status_t mea_paged_append(const void* q, void* q_out, const void* k, const void* v, void* k_cache, void* v_cache,
                              float* weights, const int* cu_q, const int* kv_len, const int* page_table,
                              const int* positions, const double* freq, int T, int B, int H, int H_kv, int D,
                              long long q_stride, long long k_stride, long long v_stride, int num_pages,
                              int page_size, int max_pages, int rot_dim, mea_rope_layout_t layout, float mscale,
                              mea_dtype_t dtype, void* stream) {
    const char* where = "mea_paged_append";
    mea_status_t st = check_batch(where, T, B, H_kv, D, num_pages, page_size, max_pages, dtype);
    if (st != MEA_OK) return st;
    if ((q == nullptr) != (q_out == nullptr)) return invalid(where, "q and q_out go together");
    if (q != nullptr && (st = check_heads(where, T, H, H_kv, D, q_stride)) != MEA_OK) return st;
    if (k_stride < (long long)H_kv * D || v_stride < (long long)H_kv * D)
        return invalid(where, "token stride of k or v below H_kv * D");
    if (k_stride % 8 != 0 || v_stride % 8 != 0)
        return api_fail(MEA_ERR_MISALIGNED, where, "token stride of k or v not a multiple of 8");
    if (freq != nullptr && (st = check_rope(where, rot_dim, D, layout, mscale)) != MEA_OK) return st;
    if (q != nullptr && q == q_out && q_stride != (long long)H * D)
        return invalid(where, "q_out is dense: it can be q only where q is");
    if (T == 0 || B == 0) return MEA_OK;
    if (!k || !v || !k_cache || !v_cache || !cu_q || !kv_len || !page_table) return invalid(where, "null pointer");
    if (num_pages == 0 || max_pages == 0) return invalid(where, "no pages");
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(weights, 4) || !aligned(cu_q, 4) || !aligned(kv_len, 4) ||
        !aligned(page_table, 4) || !aligned(positions, 4) || !aligned(freq, 8))
        return MEA_ERR_MISALIGNED;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    mea::AppendArgs a;
    a.s = batch_of(cu_q, kv_len, page_table, T, B, num_pages, page_size, max_pages);
    a.q = q;
    a.q_out = q_out;
    a.k = k;
    a.v = v;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.weights = weights;
    a.positions = positions;
    a.freq = freq;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.H = q != nullptr ? H : 0;
    a.Hkv = H_kv;
    a.D = D;
    a.rot = freq != nullptr ? rot_dim : 0;
    a.interleaved = layout == MEA_ROPE_INTERLEAVED;
    a.mscale = mscale;
    return mea::api_cuda(mea::launch_append(a, dtype == MEA_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)), where);
}

mea_status_t mea_attn_paged_workspace_size(int T, int B, int H, int H_kv, int D, int max_q, int max_kv,
                                           mea_dtype_t dtype, size_t* bytes) {
    const char* where = "mea_attn_paged_workspace_size";
    if (bytes == nullptr) return invalid(where, "null pointer");
    mea_status_t st = check_batch(where, T, B, H_kv, D, 1, 16, 1, dtype);
    if (st != MEA_OK) return st;
    if ((st = check_heads(where, T, H, H_kv, D, (long long)H * D)) != MEA_OK) return st;
    if (max_q < 0 || max_kv < 0) return invalid(where, "negative bound");
    *bytes = 0;
    if (T == 0 || B == 0) return MEA_OK;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    *bytes = attn_plan(sms, T, B, H, H_kv, D, max_q, max_kv, dtype == MEA_DTYPE_BF16).ws_bytes;
    return MEA_OK;
}

mea_status_t mea_attn_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                            const int* cu_q, const int* kv_len, const int* page_table, int T, int B, int H, int H_kv,
                            int D, long long q_stride, int num_pages, int page_size, int max_pages, int max_q,
                            int max_kv, float scale, mea_dtype_t dtype, void* workspace, size_t workspace_bytes,
                            void* stream) {
    const char* where = "mea_attn_paged";
    mea_status_t st = check_batch(where, T, B, H_kv, D, num_pages, page_size, max_pages, dtype);
    if (st != MEA_OK) return st;
    if ((st = check_heads(where, T, H, H_kv, D, q_stride)) != MEA_OK) return st;
    if (max_q < 0 || max_kv < 0) return invalid(where, "negative bound");
    if (!std::isfinite(scale)) return invalid(where, "scale not finite");
    if (T == 0 || B == 0) return MEA_OK;
    if (!q || !k_cache || !v_cache || !o || !lse || !cu_q || !kv_len || !page_table) return invalid(where, "null pointer");
    if (num_pages == 0 || max_pages == 0) return invalid(where, "no pages");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(o, 16) || !aligned(lse, 4) ||
        !aligned(cu_q, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4))
        return MEA_ERR_MISALIGNED;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    const bool bf16 = dtype == MEA_DTYPE_BF16;
    const AttnPlan p = attn_plan(sms, T, B, H, H_kv, D, max_q, max_kv, bf16);
    if (p.ws_bytes > 0) {
        if (workspace == nullptr || workspace_bytes < p.ws_bytes)
            return api_fail(MEA_ERR_WORKSPACE, where, "workspace missing or below mea_attn_paged_workspace_size");
        if (!aligned(workspace, 16)) return MEA_ERR_MISALIGNED;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.tt > 0) {
        mea::PagedTcArgs t;
        if ((st = map_q(&t.tm_q, q, T, H, H / H_kv, D, q_stride, p.tt)) != MEA_OK) return st;
        if ((st = map_pages(&t.tm_k, k_cache, num_pages, H_kv, page_size, D)) != MEA_OK) return st;
        if ((st = map_pages(&t.tm_v, v_cache, num_pages, H_kv, page_size, D)) != MEA_OK) return st;
        t.s = batch_of(cu_q, kv_len, page_table, T, B, num_pages, page_size, max_pages);
        t.o = o;
        t.lse = lse;
        t.part_acc = static_cast<float*>(workspace);
        t.part_ml = t.part_acc + (size_t)2 * sms * p.rows * D;
        t.parts = reinterpret_cast<mea::PagedPart*>(t.part_ml + (size_t)2 * sms * p.rows * 2);
        t.H = H;
        t.Hkv = H_kv;
        t.D = D;
        t.tt = p.tt;
        t.scale = scale;
        return mea::api_cuda(mea::launch_paged_tc(t, sms, s), where);
    }
    mea::PagedAttnArgs a;
    a.s = batch_of(cu_q, kv_len, page_table, T, B, num_pages, page_size, max_pages);
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.o = o;
    a.lse = lse;
    a.part_acc = static_cast<float*>(workspace);
    a.part_ml = p.nsplit > 1 ? a.part_acc + (size_t)p.nsplit * T * H * D : nullptr;
    a.q_stride = q_stride;
    a.H = H;
    a.Hkv = H_kv;
    a.D = D;
    a.rows = p.rows;
    a.nsplit = p.nsplit;
    a.scale = scale;
    if ((st = mea::api_cuda(mea::launch_paged_simt(a, bf16, s), where)) != MEA_OK || p.nsplit == 1) return st;
    return mea::api_cuda(mea::launch_paged_merge(a, bf16, s), where);
}

mea_status_t mea_attn_paged_weights_workspace_size(int T, int B, int H, int H_kv, int D, int max_q, int max_kv,
                                                   mea_dtype_t dtype, size_t* bytes) {
    const char* where = "mea_attn_paged_weights_workspace_size";
    if (bytes == nullptr) return invalid(where, "null pointer");
    mea_status_t st = check_batch(where, T, B, H_kv, D, 1, 16, 1, dtype);
    if (st != MEA_OK) return st;
    if ((st = check_heads(where, T, H, H_kv, D, (long long)H * D)) != MEA_OK) return st;
    if (max_q < 0 || max_kv < 0) return invalid(where, "negative bound");
    *bytes = 0;
    if (T == 0 || B == 0) return MEA_OK;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    *bytes = weights_plan(sms, H / H_kv, max_q, dtype == MEA_DTYPE_BF16).ws_bytes;
    return MEA_OK;
}

mea_status_t mea_attn_paged_weights(const void* q, const float* lse, const void* k_cache, float* weights,
                                    const int* cu_q, const int* kv_len, const int* page_table, int T, int B, int H,
                                    int H_kv, int D, long long q_stride, int num_pages, int page_size, int max_pages,
                                    int max_q, int max_kv, float scale, mea_dtype_t dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    const char* where = "mea_attn_paged_weights";
    mea_status_t st = check_batch(where, T, B, H_kv, D, num_pages, page_size, max_pages, dtype);
    if (st != MEA_OK) return st;
    if ((st = check_heads(where, T, H, H_kv, D, q_stride)) != MEA_OK) return st;
    if (max_q < 0 || max_kv < 0) return invalid(where, "negative bound");
    if (!std::isfinite(scale)) return invalid(where, "scale not finite");
    if (T == 0 || B == 0) return MEA_OK;
    if (!q || !lse || !k_cache || !weights || !cu_q || !kv_len || !page_table) return invalid(where, "null pointer");
    if (num_pages == 0 || max_pages == 0) return invalid(where, "no pages");
    if (!aligned(q, 16) || !aligned(k_cache, 16) || !aligned(lse, 4) || !aligned(weights, 4) || !aligned(cu_q, 4) ||
        !aligned(kv_len, 4) || !aligned(page_table, 4))
        return MEA_ERR_MISALIGNED;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    const WeightsPlan p = weights_plan(sms, H / H_kv, max_q, dtype == MEA_DTYPE_BF16);
    if (p.ws_bytes > 0) {
        if (workspace == nullptr || workspace_bytes < p.ws_bytes)
            return api_fail(MEA_ERR_WORKSPACE, where, "workspace missing or below mea_attn_paged_weights_workspace_size");
        if (!aligned(workspace, 16)) return MEA_ERR_MISALIGNED;
    }
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p.tt > 0) {
        mea::PagedWeightsTcArgs t;
        if ((st = map_q(&t.tm_q, q, T, H, H / H_kv, D, q_stride, p.tt)) != MEA_OK) return st;
        if ((st = map_pages(&t.tm_k, k_cache, num_pages, H_kv, page_size, D)) != MEA_OK) return st;
        t.s = batch_of(cu_q, kv_len, page_table, T, B, num_pages, page_size, max_pages);
        t.lse = lse;
        t.weights = weights;
        t.part_sum = static_cast<float*>(workspace);
        t.parts = p.split ? reinterpret_cast<mea::PagedPart*>(t.part_sum + (size_t)2 * sms * mea::kWeightsPartKeys) : nullptr;
        t.H = H;
        t.Hkv = H_kv;
        t.D = D;
        t.tt = p.tt;
        t.scale = scale;
        t.split = p.split;
        return mea::api_cuda(mea::launch_paged_weights_tc(t, sms, s), where);
    }
    mea::PagedWeightsArgs a;
    a.s = batch_of(cu_q, kv_len, page_table, T, B, num_pages, page_size, max_pages);
    a.q = q;
    a.lse = lse;
    a.k = k_cache;
    a.weights = weights;
    a.q_stride = q_stride;
    a.H = H;
    a.Hkv = H_kv;
    a.D = D;
    a.max_kv = max_kv;
    a.scale = scale;
    return mea::api_cuda(mea::launch_paged_weights_simt(a, dtype == MEA_DTYPE_BF16, s), where);
}

mea_status_t mea_paged_evict(void* k_cache, void* v_cache, float* weights, const int* page_table, const int* kv_len,
                             const int* dst_table, int* kv_len_out, int* keep_idx, int B, int H_kv, int D,
                             int num_pages, int page_size, int max_pages, int dst_max_pages, int n_keep, int n_recent,
                             mea_dtype_t dtype, void* stream) {
    const char* where = "mea_paged_evict";
    mea_status_t st = check_batch(where, 0, B, H_kv, D, num_pages, page_size, max_pages, dtype);
    if (st != MEA_OK) return st;
    if (n_keep < 1 || n_recent < 0 || n_recent > n_keep) return invalid(where, "0 <= n_recent <= n_keep, 1 <= n_keep");
    if (dst_max_pages < 0) return invalid(where, "negative size");
    if ((long long)B * H_kv > 65535) return api_fail(MEA_ERR_UNSUPPORTED, where, "B * H_kv above 65535");
    // slots are counted in ints, up to one batch of the kernels (a few thousand) beyond the last
    if ((long long)B * H_kv * n_keep > 0x7fffffffLL - 65536) return invalid(where, "B * H_kv * n_keep too large");
    if (B == 0) return MEA_OK;
    if (!k_cache || !v_cache || !weights || !page_table || !kv_len || !dst_table || !keep_idx)
        return invalid(where, "null pointer");
    if (num_pages == 0 || max_pages == 0) return invalid(where, "no pages");
    // a sequence may hold fewer keys than n_keep: the destination then needs no more pages than it has
    const long long most = std::min<long long>(n_keep, (long long)max_pages * page_size);
    if ((long long)dst_max_pages * page_size < most) return invalid(where, "dst_table too short for n_keep keys");
    const bool in_place = dst_table == page_table;
    if (in_place && dst_max_pages != max_pages) return invalid(where, "in place: dst_max_pages must be max_pages");
    if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(weights, 4) || !aligned(page_table, 4) ||
        !aligned(kv_len, 4) || !aligned(dst_table, 4) || !aligned(kv_len_out, 4) || !aligned(keep_idx, 4))
        return MEA_ERR_MISALIGNED;
    int sms = 0;
    if ((st = mea::api_device(&sms)) != MEA_OK) return st;
    mea::EvictArgs a;
    a.s = batch_of(nullptr, kv_len, page_table, 0, B, num_pages, page_size, max_pages);
    a.k = k_cache;
    a.v = v_cache;
    a.weights = weights;
    a.dst_table = dst_table;
    a.kv_len_out = kv_len_out;
    a.keep_idx = keep_idx;
    a.Hkv = H_kv;
    a.D = D;
    a.dst_max_pages = dst_max_pages;
    a.n_keep = n_keep;
    a.n_recent = n_recent;
    a.in_place = in_place;
    return mea::api_cuda(mea::launch_evict(a, dtype == MEA_DTYPE_BF16, sms, static_cast<cudaStream_t>(stream)), where);
}

}  // extern "C"
