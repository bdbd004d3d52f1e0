// Products with 4-bit weights:
//   Y[m, n] = sum_g s[n, g] sum_{k in group g} X[m, k] (q[n, k] - z[n, g]),
// q two to a byte along K (low half first), groups of 2^shift along K, and
// the gated form H = act(G) * U of two such products (q4_glu).
//
// Arithmetic.  q - z is an integer of at most 4 bits and a sign, exact in
// bfloat16 and float16, so the products run on the matrix cores of the 16-bit
// types without rounding a weight: float16 X on float16, bfloat16 X on
// bfloat16, and float X as the sum of three bfloat16 parts of 8 bits each
// (24 bits: the float exactly, down to 2^-110), one matrix instruction per
// part.  That is 16 / 3 times the rate of the float matrix instructions, with
// products that are exact.  Each group's sum is formed from zero in float
// and joins the output's float sum through one multiply-add by its scale, so
// a scale is never rounded either.
#include <type_traits>

#include "activation.h"
#include "kernels.h"

namespace sgemm {

namespace {
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 128;      // K per step of a wave: 4 lane groups of 32 weights
constexpr int kRowsMax = 16;    // rows of X of one q4_rows workgroup

// bfloat16 parts of X for the matrix cores: 3 for float, 1 for 16-bit types.
template <int XT> constexpr int parts() { return XT == T_F32 ? 3 : 1; }

__device__ __forceinline__ float to_float(int type, const void* p, int64_t i) {
    if (type == T_F32) return static_cast<const float*>(p)[i];
    if (type == T_F16) return float(static_cast<const _Float16*>(p)[i]);
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
}

template <int XT>
__device__ __forceinline__ void store_as(void* p, int64_t i, float v) {
    if constexpr (XT == T_F32) static_cast<float*>(p)[i] = v;
    else if constexpr (XT == T_F16) static_cast<_Float16*>(p)[i] = _Float16(v);
    else static_cast<__bf16*>(p)[i] = __bf16(v);
}

// 16 bytes from any address.
__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// The 16 packed bytes at byte `off` of a row of `bytes`: zero past its end.
__device__ __forceinline__ u32x4 load_w(const uint8_t* row, int64_t off, int64_t bytes) {
    if (off + 16 <= bytes) return load16(row + off);
    u32x4 v = {0, 0, 0, 0};
    for (int i = 0; i < 16; i++)
        if (off + i < bytes) v[i / 4] |= uint32_t(row[off + i]) << (8 * (i % 4));
    return v;
}

// Zero point z as the constant that dequant<XT> takes.
template <int XT>
__device__ __forceinline__ uint32_t zero_const(int z) {
    if constexpr (XT == T_F16) return uint32_t(z);
    else return 0x80808080u - uint32_t(z) * 0x01010101u;
}

// The eight weights q - z of one packed word as the matrix instruction's
// operand.  bfloat16: the bytes 0x80 + q - z flip their top bit into signed
// bytes, which convert to float and keep their upper halves (2.4 operations a
// weight), in order k, k + 1, ...  float16: 0x6400 | q is 1024 + q and 0x6400
// | 16 q is 1024 + 16 q, so one packed add or multiply-add leaves q - z (1.1
// operations a weight), in order 0 4 1 5 2 6 3 7, which order_x gives X too.
template <int XT>
__device__ __forceinline__ u32x4 dequant(uint32_t w, uint32_t zc) {
    u32x4 r;
    if constexpr (XT == T_F16) {
        const _Float16 z = _Float16(int(zc));
        const f16x2 off = {_Float16(-1024.0f) - z, _Float16(-1024.0f) - z};
        const f16x2 off16 = {_Float16(-64.0f) - z, _Float16(-64.0f) - z};
        const f16x2 six = {_Float16(0.0625f), _Float16(0.0625f)};
#pragma unroll
        for (int h = 0; h < 2; h++) {
            const uint32_t v = w >> (8 * h);
            const f16x2 a = __builtin_bit_cast(f16x2, (v & 0x000F000Fu) | 0x64006400u);
            const f16x2 b = __builtin_bit_cast(f16x2, (v & 0x00F000F0u) | 0x64006400u);
            r[2 * h] = __builtin_bit_cast(uint32_t, a + off);
            r[2 * h + 1] = __builtin_bit_cast(uint32_t, __builtin_elementwise_fma(b, six, off16));
        }
    } else {
        const uint32_t lo = ((w & 0x0F0F0F0Fu) + zc) ^ 0x80808080u;
        const uint32_t hi = (((w >> 4) & 0x0F0F0F0Fu) + zc) ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const float a = float(int8_t(lo >> (8 * i))), b = float(int8_t(hi >> (8 * i)));
            r[i] = __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
        }
    }
    return r;
}

// Eight consecutive 16-bit X values in dequant's order.
template <int XT>
__device__ __forceinline__ u32x4 order_x(u32x4 x) {
    if constexpr (XT != T_F16) return x;
    // (0 1)(2 3)(4 5)(6 7) -> (0 4)(1 5)(2 6)(3 7)
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(x[2], x[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(x[2], x[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(x[3], x[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(x[3], x[1], 0x07060302u);
    return r;
}

// A float as three bfloat16 parts (each a float whose lower half is zero):
// the upper 8 bits of its mantissa, of the rest, and of what is left, which
// has no more than 8.  An infinity is its own first part (the differences
// would be NaN); a NaN becomes a quiet one, whose mark is in the upper half.
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    x = __builtin_canonicalizef(x);
    p[0] = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r = __builtin_isinf(x) ? 0.0f : x - p[0];
    p[1] = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
    p[2] = r - p[1];
}

template <int XT>
__device__ __forceinline__ v4f mfma16(u32x4 x, u32x4 w, v4f c) {
    if constexpr (XT == T_F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                       __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
}

// Lane group l (lanes 16 l ..) holds words 4 l .. 4 l + 3 of its row's 16; after
// this, v[j] of group l is word 4 j + l: step j's 32 weights, 8 per group.
__device__ __forceinline__ void transpose_groups(u32x4& v) {
    auto a = __builtin_amdgcn_permlane32_swap(v[0], v[2], false, false);
    auto b = __builtin_amdgcn_permlane32_swap(v[1], v[3], false, false);
    auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
    auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
    v[0] = c[0];
    v[1] = c[1];
    v[2] = d[0];
    v[3] = d[1];
}
}  // namespace

// Up to 16 rows of X.  A workgroup owns 16 columns n of Y for rows m0 ..
// m0 + 15; its waves deal the K units out among themselves and add their sums
// through LDS in wave order.  The weights are the B operand of the 16 x 16 x 32
// instruction (lane: column n = lane % 16, eight k of step j from lane group
// lane / 16) and go from memory to registers in 16-byte loads, one pass; X is
// the A operand, rows past M repeating the last one.  16-bit X comes straight
// from memory (each wave reads only its own K range); float X is split once
// per workgroup into LDS, chunk by chunk.
// GS: steps of 32 that share a scale (4 for groups of 128 or more).
template <int XT, int GS, int NWT>
__global__ void __launch_bounds__(1024)
q4_rows(Q4Args g, int64_t units, int64_t units_chunk, int64_t tiles_m, int64_t tiles) {
    constexpr int P = parts<XT>(), NS = 4 / GS;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nw = blockDim.x >> 6;
    const int r = lane & 15, lg = lane >> 4;
    const int64_t bytes = (g.K + 1) / 2, groups = (g.K + (int64_t(1) << g.shift) - 1) >> g.shift;
  for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int64_t n0 = tile / tiles_m * 16, m0 = tile % tiles_m * kRowsMax;
    const int rows = int(g.M - m0 < kRowsMax ? g.M - m0 : kRowsMax);
    const int64_t n = n0 + r < g.N ? n0 + r : g.N - 1;
    const int mr = r < rows ? r : rows - 1;

    struct Unit {
        u32x4 w[NWT];
        float s[NWT][NS];
        uint32_t z[NWT][NS];
    };
    auto load_unit = [&](Unit& u, int64_t idx) {
#pragma unroll
        for (int t = 0; t < NWT; t++) {
            u.w[t] = load_w(g.W[t] + n * g.ldw, idx * (kUnit / 2) + lg * 16, bytes);
#pragma unroll
            for (int q = 0; q < NS; q++) {
                int64_t gi = (idx * kUnit + q * (kUnit / NS)) >> g.shift;
                gi = gi < groups ? gi : groups - 1;
                u.s[t][q] = to_float(g.stype, g.S[t], n * g.lds + gi);
                u.z[t][q] = g.Z[t] ? g.Z[t][n * g.ldz + gi] : 8;
            }
        }
    };
    v4f acc[NWT];
#pragma unroll
    for (int t = 0; t < NWT; t++) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    // xs: this unit's staged X (float only).
    auto do_unit = [&](Unit& u, int64_t idx, const char* xs) {
#pragma unroll
        for (int t = 0; t < NWT; t++) transpose_groups(u.w[t]);
        v4f d[NWT];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            u32x4 x[P];
            if constexpr (P == 3) {
#pragma unroll
                for (int p = 0; p < P; p++)
                    x[p] = *reinterpret_cast<const u32x4*>(xs + (((j * P + p) * 4 + lg) * rows + mr) * 16);
            } else {
                const int64_t k = idx * kUnit + j * 32 + lg * 8;
                const uint16_t* xp = static_cast<const uint16_t*>(g.X) + (m0 + mr) * g.ldx + k;
                u32x4 v = {0, 0, 0, 0};
                if (k + 8 <= g.K) {
                    v = load16(xp);
                } else {
                    for (int i = 0; i < 8; i++)
                        if (k + i < g.K) v[i / 2] |= uint32_t(xp[i]) << (16 * (i % 2));
                }
                x[0] = order_x<XT>(v);
            }
#pragma unroll
            for (int t = 0; t < NWT; t++) {
                const u32x4 w = dequant<XT>(u.w[t][j], zero_const<XT>(u.z[t][j / GS]));
                // Largest part first.  The instruction rounds to nearest when
                // what it adds is smaller than the accumulator, and truncates
                // the accumulator downwards when that is the smaller one
                // (measured: with the smallest part first, products of one
                // float and one weight came out up to a unit too low).
#pragma unroll
                for (int p = 0; p < P; p++)
                    d[t] = mfma16<XT>(x[p], w, p == 0 && j % GS == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : d[t]);
                if (j % GS == GS - 1) {
#pragma unroll
                    for (int e = 0; e < 4; e++) acc[t][e] = fmaf(u.s[t][j / GS], d[t][e], acc[t][e]);
                }
            }
        }
    };

    if constexpr (P == 3) {
        // Chunks of units_chunk units: split X into LDS, then each wave its
        // own units of the chunk.
        const size_t unit_bytes = size_t(4) * P * 4 * rows * 16;
        for (int64_t c0 = 0; c0 < units; c0 += units_chunk) {
            const int cn = int(units - c0 < units_chunk ? units - c0 : units_chunk);
            Unit u;
            if (wave < cn) load_unit(u, c0 + wave);
            if (c0 > 0) __syncthreads();
            // One 8-element piece of a row per lane and trip: 16 of them per
            // unit and row.
            const int pieces = cn * 16 * rows;
            for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
                const int kk = i % (cn * 16), m = i / (cn * 16);
                const int64_t k = (c0 * 16 + kk) * 8;
                const float* xp = static_cast<const float*>(g.X) + (m0 + m) * g.ldx + k;
                float x[8];
                if (k + 8 <= g.K) {
                    *reinterpret_cast<u32x4*>(x) = load16(xp);
                    *reinterpret_cast<u32x4*>(x + 4) = load16(xp + 4);
                } else {
                    for (int e = 0; e < 8; e++) x[e] = k + e < g.K ? xp[e] : 0.0f;
                }
                u32x4 out[3];
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    float a[3], b[3];
                    split3(x[2 * e], a);
                    split3(x[2 * e + 1], b);
#pragma unroll
                    for (int p = 0; p < 3; p++)
                        out[p][e] = __builtin_amdgcn_perm(__float_as_uint(b[p]), __float_as_uint(a[p]), 0x07060302u);
                }
                char* dst = smem + (kk / 16) * unit_bytes;
                const int j = kk % 16 / 4, l = kk % 4;
#pragma unroll
                for (int p = 0; p < 3; p++)
                    *reinterpret_cast<u32x4*>(dst + (((j * 3 + p) * 4 + l) * rows + m) * 16) = out[p];
            }
            __syncthreads();
            for (int i = wave; i < cn; i += nw) {
                Unit v;
                if (i + nw < cn) load_unit(v, c0 + i + nw);
                do_unit(u, c0 + i, smem + i * unit_bytes);
                u = v;
            }
        }
    } else {
        Unit u;
        if (wave < units) load_unit(u, wave);
        for (int64_t i = wave; i < units; i += nw) {
            Unit v;
            if (i + nw < units) load_unit(v, i + nw);
            do_unit(u, i, nullptr);
            u = v;
        }
    }

    // Accumulator register e of lane (lg, r) is row 4 lg + e, column r.
    if constexpr (P == 3) __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < NWT; t++)
#pragma unroll
        for (int e = 0; e < 4; e++) red[(wave * NWT + t) * 256 + (4 * lg + e) * 16 + r] = acc[t][e];
    __syncthreads();
    for (int o = threadIdx.x; o < rows * 16; o += blockDim.x) {
        float sum[NWT];
#pragma unroll
        for (int t = 0; t < NWT; t++) {
            sum[t] = red[t * 256 + o];
            for (int w = 1; w < nw; w++) sum[t] += red[(w * NWT + t) * 256 + o];
        }
        const int64_t m = m0 + o / 16, nn = n0 + o % 16;
        if (nn < g.N)
            store_as<XT>(g.Y, m * g.ldy + nn, NWT == 2 ? act_value(g.act, sum[0]) * sum[NWT - 1] : sum[0]);
    }
    if (tile + gridDim.x < tiles) __syncthreads();
  }
}

template <int XT, int GS, int NWT>
static hipError_t launch_rows(const Q4Args& g, hipStream_t s) {
    const int64_t units = ceil_div(g.K, kUnit);
    const int nw = 8;
    const int rows = int(g.M < kRowsMax ? g.M : kRowsMax);
    // Float X: as many units a chunk as keep the split parts within 48 KiB,
    // in whole rounds of the waves where that allows.
    const int unit_bytes = 4 * 3 * 4 * rows * 16;
    int64_t chunk = units;
    size_t lds = size_t(nw) * NWT * 1024;
    if (XT == T_F32) {
        chunk = 49152 / unit_bytes;
        if (chunk < nw) chunk = nw;
        chunk = chunk / nw * nw;
        if (chunk > units) chunk = units;
        const size_t x = size_t(chunk) * unit_bytes;
        if (x > lds) lds = x;
    }
    const int64_t tm = ceil_div(g.M, kRowsMax), tiles = ceil_div(g.N, 16) * tm;
    hipLaunchKernelGGL((q4_rows<XT, GS, NWT>), dim3(grid_for(tiles)), dim3(64 * nw), lds, s, g, units,
                       chunk, tm, tiles);
    return hipGetLastError();
}

template <int XT, int NWT>
static hipError_t launch_xt(const Q4Args& g, hipStream_t s) {
    if (g.shift >= 7) return launch_rows<XT, 4, NWT>(g, s);
    if (g.shift == 6) return launch_rows<XT, 2, NWT>(g, s);
    return launch_rows<XT, 1, NWT>(g, s);
}

template <int NWT>
static hipError_t launch_nwt(const Q4Args& g, hipStream_t s) {
    switch (g.xtype) {
        case T_F32: return launch_xt<T_F32, NWT>(g, s);
        case T_F16: return launch_xt<T_F16, NWT>(g, s);
        default: return launch_xt<T_BF16, NWT>(g, s);
    }
}

hipError_t launch_q4(const Q4Args& g, hipStream_t s) {
    return g.act >= 0 ? launch_nwt<2>(g, s) : launch_nwt<1>(g, s);
}

}  // namespace sgemm
