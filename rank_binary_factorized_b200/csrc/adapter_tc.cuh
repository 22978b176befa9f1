// adapter_tc.cuh -- what the tensor-core kernels of the adapters share.
#pragma once

#include "adapter.cuh"
#include "tc_common.cuh"

namespace nq {

// What v's bf16 part leaves of it (nothing of an infinity).
__device__ __forceinline__ float rest_of(float v, uint32_t part) {
    const float p = __uint_as_float(part);
    return isinf(p) ? 0.f : v - p;
}

// A sum over first parts and the same over second parts, which have accumulators of their own.  Against an
// infinity the second parts, which may be 0 or of the other sign, add up to an infinity or NaN that
// the value itself does not have; the first parts alone then give its infinity or NaN.
__device__ __forceinline__ float join_parts(uint32_t hi, uint32_t lo) {
    const float l = __uint_as_float(lo);
    return __uint_as_float(hi) + (isfinite(l) ? l : 0.f);
}

// Two fp32 values as the sum of two bf16 values each.
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = pack_bf16(a, b);
    lo = pack_bf16(rest_of(a, hi << 16), rest_of(b, hi & 0xFFFF0000u));
}

// The same for products that share an accumulator: the second part has the value's sign and is 0 only of a
// 0, so that against an infinity the parts agree.  The first is cut instead of rounded, and the smallest
// number, 2^-133, stands in for a second part of nothing: off by 2^-16 of the value or 2^-133 at most.
__device__ __forceinline__ uint32_t second_part(float v) {
    const uint32_t bits = __float_as_uint(v);
    const float first = __uint_as_float(bits & 0xFFFF0000u);
    const uint32_t rest = float_to_bf16_bits(v == first ? 0.f : v - first);
    return (rest & 0x7FFFu) != 0u || v == 0.f ? rest : (bits >> 16 & 0x8000u) | 1u;
}
__device__ __forceinline__ void split_bf16_same_sign(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    lo = second_part(a) | second_part(b) << 16;
}

}  // namespace nq

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
