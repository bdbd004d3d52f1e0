// Which rows a workgroup of the adapter kernels takes, and element types.
#pragma once
#include <type_traits>

#include "kernels.h"

namespace sgemm {

// How rows are dealt out in tiles.
struct RowPlan {
    enum Mode { SORTED, SINGLE, UNIFORM } mode;
    const void* ids;   // SINGLE: a tile is one row, with the adapter of its id
    bool id64;
    int M, L;
    const int* order;  // SORTED: row of each position, rows of one adapter together
    const int* head;   // SORTED: number of tiles, 3 unused, then RowTile's fields of each
};

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

template <int T> struct Elem;
template <> struct Elem<T_F32> { using type = float; };
template <> struct Elem<T_F16> { using type = _Float16; };
template <> struct Elem<T_BF16> { using type = __bf16; };
// Elements in 16 bytes.
template <int T> constexpr int kVec = T == T_F32 ? 4 : 8;

// A run of rows with one adapter (-1: none): positions [start, start + count)
// of the order; the place-th such run of its adapter.
struct RowTile {
    int adapter, start, count, place;
};

__device__ __forceinline__ int adapter_of(const void* ids, bool id64, int L, int64_t m) {
    // An int64 as its two halves, so that both types are loads without a branch.
    const uint32_t* const p = static_cast<const uint32_t*>(ids) + (id64 ? 2 * m : m);
    const uint32_t lo = p[0], hi = p[id64 ? 1 : 0];
    return (lo < uint32_t(L)) & (!id64 | (hi == 0)) ? int(lo) : -1;
}

// Tile t of `size` rows; count 0 past the last.
__device__ __forceinline__ RowTile row_tile(const RowPlan& p, int64_t t, int size) {
    if (p.mode == RowPlan::SORTED) {
        const int n = p.head[0];
        const int4 at = reinterpret_cast<const int4*>(p.head)[1 + t];  // in bounds, of no meaning past the last
        return {__builtin_amdgcn_readfirstlane(at.x), __builtin_amdgcn_readfirstlane(at.y),
                t < n ? __builtin_amdgcn_readfirstlane(at.z) : 0, __builtin_amdgcn_readfirstlane(at.w)};
    }
    if (p.mode == RowPlan::SINGLE) return {adapter_of(p.ids, p.id64, p.L, t), int(t), 1, 0};
    const int64_t start = t * size;
    if (start >= p.M) return {0, 0, 0, 0};
    return {0, int(start), int(p.M - start < size ? p.M - start : size), int(t)};
}

__device__ __forceinline__ int row_at(const RowPlan& p, int position) {
    return p.mode == RowPlan::SORTED ? p.order[position] : position;
}

// A workgroup's (x, y) of the grid, such that neighbours in x are on one XCD: they go
// to the eight in turn, and what workgroups of one y share then stays in one L2.
__device__ __forceinline__ uint2 block_of_run() {
    const uint32_t n = gridDim.x * gridDim.y, id = blockIdx.x + blockIdx.y * gridDim.x;
    const uint32_t q = n / 8, rem = n % 8, x = id % 8, t = x * q + (x < rem ? x : rem) + id / 8;
    return {t % gridDim.x, t / gridDim.x};
}

// 16 bytes from any address, and to any.
__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void store16(void* p, u32x4 v) { __builtin_memcpy(p, &v, 16); }

// The 16 bytes of elements [i, i + kVec) of a row of n elements, zero past its end.
template <int T>
__device__ __forceinline__ u32x4 load_chunk(const typename Elem<T>::type* row, int64_t i, int64_t n) {
    if (i + kVec<T> <= n) return load16(row + i);
    u32x4 r = {0, 0, 0, 0};
#pragma unroll 1
    for (int e = 0; i + e < n; e++) {
        if constexpr (T == T_F32) {
            const uint32_t w = __float_as_uint(row[i + e]);
#pragma unroll
            for (int q = 0; q < 4; q++) r[q] = q == e ? w : r[q];
        } else {
            const uint32_t w = uint32_t(__builtin_bit_cast(uint16_t, row[i + e])) << (16 * (e & 1));
#pragma unroll
            for (int q = 0; q < 4; q++) r[q] = q == e / 2 ? r[q] | w : r[q];
        }
    }
    return r;
}

template <int T>
__device__ __forceinline__ void unpack(u32x4 v, float (&f)[kVec<T>]) {
    typename Elem<T>::type e[kVec<T>];
    __builtin_memcpy(e, &v, 16);
#pragma unroll
    for (int i = 0; i < kVec<T>; i++) f[i] = float(e[i]);
}
template <int T>
__device__ __forceinline__ u32x4 pack(const float (&f)[kVec<T>]) {
    typename Elem<T>::type e[kVec<T>];
#pragma unroll
    for (int i = 0; i < kVec<T>; i++) e[i] = typename Elem<T>::type(f[i]);
    u32x4 v;
    __builtin_memcpy(&v, e, 16);
    return v;
}

// One 16 x 16 block plus the products of two operands of 16 bytes a lane: lane
// l has elements (l / 16) kVec .. of row l % 16 of either.
template <int T>
__device__ __forceinline__ v4f mma16(u32x4 a, u32x4 b, v4f c) {
    if constexpr (T == T_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else if constexpr (T == T_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else {
#pragma unroll
        for (int e = 0; e < 4; e++)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
        return c;
    }
}

// Float factors for the 16-bit instructions: the sum of three parts of the type (four
// where an instruction has room for them), which is all of a float's 24 bits.  Of
// float16 they come after a power of two that brings the largest of those that share it
// into [2^14, 2^15); what float16 cannot hold is below 2^-36 of that largest.
__device__ __forceinline__ float largest(float top, float v) {  // of the finite
    return fabsf(v) < __builtin_inff() ? fmaxf(top, fabsf(v)) : top;
}
// That power, 2^(14 - exponent of top); 1 for zero.
__device__ __forceinline__ float half_factor(float top) {
    if (!(top > 0.0f)) return 1.0f;
    int ex = int(__float_as_uint(top) >> 23) - 127;
    ex = ex < -100 ? -100 : ex;
    return __uint_as_float(uint32_t(14 - ex + 127) << 23);
}
// The scale with that power undone.  A finite scale's stays finite: a sum of zero is
// then zero, and any other (2^-48 at least) past float16's range as it should be.
__device__ __forceinline__ float undone(float s, float up) {
    const float f = s / up;
    return fabsf(s) < __builtin_inff() ? fminf(fmaxf(f, -__FLT_MAX__), __FLT_MAX__) : f;
}
// Two numbers' parts, the first's in the low half of each.  An infinity in the other
// operand meets every part, so all have the number's sign, and of a number that is not
// zero none is zero: each part is cut off the float just below the rest in magnitude,
// which leaves a rest, and the type's smallest takes the place of a zero.  Of an
// infinity the last part is one (the others are the largest finite), and of a NaN.
template <int T, int PARTS>
__device__ __forceinline__ void split_pair(float a, float b, float up_a, float up_b, uint32_t (&part)[PARTS]) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const float v[2] = {a, b}, up[2] = {up_a, up_b};
    uint32_t one[2];   // 0 for a zero
    float rest[2];
#pragma unroll
    for (int e = 0; e < 2; e++) {
        const uint32_t bits = __float_as_uint(v[e]) & 0x7FFFFFFFu;
        one[e] = min(bits, 1u);
        rest[e] = __uint_as_float(T == T_F16 ? max(__float_as_uint(__uint_as_float(bits) * up[e]), one[e]) : bits);
    }
    const uint32_t least = one[0] | one[1] << 16;
    const uint32_t sign = (__float_as_uint(a) >> 16 & 0x8000u) | (__float_as_uint(b) & 0x80000000u);
#pragma unroll
    for (int i = 0; i < PARTS; i++) {
        const bool last = i + 1 == PARTS;
        uint32_t c[2];
#pragma unroll
        for (int e = 0; e < 2; e++) c[e] = __float_as_uint(rest[e]) - (last ? 0 : one[e]);
        uint32_t cut;
        if constexpr (T == T_F16) cut = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(__uint_as_float(c[0]), __uint_as_float(c[1])));
        else cut = c[0] >> 16 | (c[1] & 0xFFFF0000u);
        if (!last) {
            rest[0] -= T == T_F16 ? float(__builtin_bit_cast(_Float16, uint16_t(cut))) : __uint_as_float(cut << 16);
            rest[1] -= T == T_F16 ? float(__builtin_bit_cast(_Float16, uint16_t(cut >> 16))) : __uint_as_float(cut & 0xFFFF0000u);
        }
        part[i] = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, cut), __builtin_bit_cast(u16x2, least))) | sign;
    }
}

}  // namespace
}  // namespace sgemm
