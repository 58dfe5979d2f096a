// api_internal.h -- what the C entry points of api.cu share with those of
// api_paged.cu: the per-thread error text, the device check and the TMA
// tensor-map encoder.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "mea_attn.h"

namespace mea {

// Records "where: detail" for mea_last_error_message() and returns st.
mea_status_t api_fail(mea_status_t st, const char* where, const char* detail);
// MEA_OK, or MEA_ERR_CUDA with the error's text.
mea_status_t api_cuda(cudaError_t e, const char* where);
// The current device's SM count; MEA_ERR_UNSUPPORTED unless it is an sm_100.
mea_status_t api_device(int* sm_count);
// bf16 map of `rank` dims, 128-byte swizzle, elements outside the tensor read as zero.
mea_status_t api_map_bf16(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                          const cuuint64_t* strides, const cuuint32_t* box, const char* what);

}  // namespace mea
