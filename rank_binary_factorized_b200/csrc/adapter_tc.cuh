// adapter_tc.cuh -- what the tensor-core kernels of the adapters share.
#pragma once

#include "adapter.cuh"
#include "tc_common.cuh"

namespace nq_host {

// bf16 tensor of `dims` dimensions, innermost first, 128-byte swizzle.
inline bool tmap_bf16(CUtensorMap* map, const void* base, int dims, const int64_t* extent, const int64_t* stride_elems,
               const int* box) {
    auto enc = nq_host::tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t d[3], st[2];
    cuuint32_t bx[3], es[3] = {1, 1, 1};
    for (int i = 0; i < dims; ++i) {
        d[i] = static_cast<cuuint64_t>(extent[i]);
        bx[i] = static_cast<cuuint32_t>(box[i]);
        if (i > 0) st[i - 1] = static_cast<cuuint64_t>(stride_elems[i - 1]) * 2;
    }
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(dims), const_cast<void*>(base), d, st, bx, es,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace nq_host
