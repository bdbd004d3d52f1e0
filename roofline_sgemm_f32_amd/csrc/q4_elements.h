// Elements of the 4-bit products' operands and results, by type.
#pragma once
#include "kernels.h"

namespace sgemm {
namespace {

// An element as its bits, and these as a float.
__device__ __forceinline__ uint32_t load_raw(int type, const void* p, int64_t i) {
    if (type == T_F32) return static_cast<const uint32_t*>(p)[i];
    return static_cast<const uint16_t*>(p)[i];
}
__device__ __forceinline__ float raw_to_float(int type, uint32_t v) {
    const float half = float(__builtin_bit_cast(_Float16, uint16_t(v)));
    return type == T_F32 ? __uint_as_float(v) : type == T_BF16 ? __uint_as_float(v << 16) : half;
}

template <int XT>
__device__ __forceinline__ void store_as(void* p, int64_t i, float v) {
    if constexpr (XT == T_F32) static_cast<float*>(p)[i] = v;
    else if constexpr (XT == T_F16) static_cast<_Float16*>(p)[i] = _Float16(v);
    else static_cast<__bf16*>(p)[i] = __bf16(v);
}

}  // namespace
}  // namespace sgemm
