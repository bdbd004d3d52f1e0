// Products with 4-bit weights:
//   Y[m, n] = sum_g s[n, g] sum_{k in group g} X[m, k] (q[n, k] - z[n, g]),
// q two to a byte along K (low half first), groups of 2^shift along K, and
// the gated form H = act(G) * U of two such products (q4_glu).
//
// Arithmetic.  q - z is an integer of at most 4 bits and a sign, exact in
// bfloat16 and float16, so the products run on the matrix cores of the 16-bit
// types without rounding a weight: float16 X on float16, bfloat16 X on
// bfloat16, and float X as the sum of three bfloat16 parts of 8 bits each
// (24 bits: the float exactly, down to 2^-110; smaller ones in steps of
// 2^-133), one matrix instruction per part.  That is 16 / 3 times the rate of
// the float matrix instructions, with products that are exact.  The sum of a
// group, or of 128 k of a longer one, is formed from zero in float and joins the
// output's float sum through one multiply-add by its scale, so a scale is never
// rounded either.
#pragma once
#include <type_traits>

#include "activation.h"
#include "kernels.h"
#include "q4_elements.h"

namespace sgemm {

namespace {
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kUnit = 128;      // K per step of a wave: 4 lane groups of 32 weights
// LDS of a q4_rows workgroup: half a CU's, unless one round of the waves takes
// more (float X of 8 rows, groups of 32, gated: 112 KiB).
constexpr int64_t kRowsLds = 80 * 1024;
// Rows of X that q4_rows takes.  Up to 16 fit the instruction; sixteen of float X
// do not fit the LDS (a round of the waves is 194 KiB), and of bfloat16 X they
// take more LDS than two workgroups a CU have, which costs where there are two
// (K = 4096, us, here and on tiles: 12 x 8192 25, 14; 16 x 8192 30, 14; gated 36,
// 23) and gains where there are fewer (9 x 4096 9.4, 13.6; 16 x 4096 14.9, 13.6;
// gated 15, 22 and 20, 22; 16 x 1024 x 2048 9.6, 10.4; gated 11, 16).
constexpr int kRowsMax = 8;

// bfloat16 parts of X for the matrix cores: 3 for float, 1 for 16-bit types.
template <int XT> constexpr int parts() { return XT == T_F32 ? 3 : 1; }

// 16 bytes from any address.
__device__ __forceinline__ u32x4 load16(const void* p) {
    u32x4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// The 16 packed bytes at byte `off` of a row of `bytes` that ends inside
// them (or before them): bytes past the end repeat the last one; X is zero
// there.
__device__ __forceinline__ u32x4 load_w_tail(const uint8_t* row, int off, int bytes) {
    u32x4 v;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        uint32_t w = 0;
#pragma unroll 1
        for (int i = 0; i < 4; i++) {
            const int at = off + 4 * j + i;
            w |= uint32_t(row[at < bytes ? at : bytes - 1]) << (8 * i);
        }
        v[j] = w;
    }
    return v;
}

// Zero point z as the constant that dequant<XT> takes.
template <int XT>
__device__ __forceinline__ uint32_t zero_const(int z) {
    if constexpr (XT == T_F16) return uint32_t(z);
    else return 0x80808080u - uint32_t(z) * 0x01010101u;
}

// (v & mask) | bits in one operation: the constants in registers, as the
// instruction takes no literal.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
    uint32_t r;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(r) : "v"(v), "s"(mask), "v"(bits));
    return r;
}

// The eight weights q - z of one packed word as the matrix instruction's
// operand.  bfloat16: the bytes 0x80 + q - z flip their top bit into signed
// bytes, which convert to float and keep their upper halves (2.4 operations a
// weight), in order k, k + 1, ...  float16: 0x6400 | q is 1024 + q and 0x6400
// | 16 q is 1024 + 16 q, so one packed add or multiply-add leaves q - z (1.1
// operations a weight), in order 0 4 1 5 2 6 3 7, which order_x gives X too.
// dequant_word is word i of the operand (two weights), from dequant_prepare's
// two words.
struct Halves { uint32_t a, b; };

template <int XT>
__device__ __forceinline__ Halves dequant_prepare(uint32_t w, uint32_t zc) {
    if constexpr (XT == T_F16) return {w, w >> 8};
    else return {((w & 0x0F0F0F0Fu) + zc) ^ 0x80808080u, (((w >> 4) & 0x0F0F0F0Fu) + zc) ^ 0x80808080u};
}

template <int XT>
__device__ __forceinline__ uint32_t dequant_word(Halves h, uint32_t zc, int i) {
    if constexpr (XT == T_F16) {
        const _Float16 z = _Float16(int(zc));
        const f16x2 off = {_Float16(-1024.0f) - z, _Float16(-1024.0f) - z};
        const f16x2 off16 = {_Float16(-64.0f) - z, _Float16(-64.0f) - z};
        const f16x2 six = {_Float16(0.0625f), _Float16(0.0625f)};
        const uint32_t v = i < 2 ? h.a : h.b;
        const f16x2 q = __builtin_bit_cast(f16x2, and_or(v, i % 2 ? 0x00F000F0u : 0x000F000Fu, 0x64006400u));
        return __builtin_bit_cast(uint32_t, i % 2 ? __builtin_elementwise_fma(q, six, off16) : q + off);
    } else {
        const float a = float(int8_t(h.a >> (8 * i))), b = float(int8_t(h.b >> (8 * i)));
        return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
    }
}

template <int XT>
__device__ __forceinline__ u32x4 dequant(uint32_t w, uint32_t zc) {
    const Halves h = dequant_prepare<XT>(w, zc);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = dequant_word<XT>(h, zc, i);
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
// has no more than 8.  Where a value may not be finite (FINITE false) an
// infinity is its own first part (the differences would be NaN), and a NaN
// becomes a quiet one, whose mark is in the upper half.
template <bool FINITE>
__device__ __forceinline__ void split3(float x, float (&p)[3]) {
    if (!FINITE) x = __builtin_canonicalizef(x);
    p[0] = __uint_as_float(__float_as_uint(x) & 0xFFFF0000u);
    const float r = !FINITE && __builtin_isinf(x) ? 0.0f : x - p[0];
    p[1] = __uint_as_float(__float_as_uint(r) & 0xFFFF0000u);
    p[2] = r - p[1];
}

// Eight consecutive elements of row m of X from column k, zero past K, as
// loaded, and as the matrix instruction's operand: the three parts of a
// float, or the elements.
template <int XT> struct RawX { u32x4 v[XT == T_F32 ? 2 : 1]; };

// left: how many elements of the row there are from p on.
template <int XT>
__device__ __forceinline__ void load_x_checked(const void* p, int left, RawX<XT>& raw) {
    if constexpr (XT == T_F32) {
        const uint32_t* xp = static_cast<const uint32_t*>(p);
        if (left >= 8) {
            raw.v[0] = load16(xp);
            raw.v[1] = load16(xp + 4);
        } else {
#pragma unroll
            for (int e = 0; e < 8; e++) raw.v[e / 4][e % 4] = e < left ? xp[e] : 0u;
        }
    } else {
        const uint16_t* xp = static_cast<const uint16_t*>(p);
        if (left >= 8) {
            raw.v[0] = load16(xp);
        } else {
            raw.v[0] = u32x4{0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (i < left) raw.v[0][i / 2] |= uint32_t(xp[i]) << (16 * (i % 2));
        }
    }
}

template <int XT>
__device__ __forceinline__ void operand_x(const RawX<XT>& raw, u32x4 (&out)[parts<XT>()]) {
    if constexpr (XT == T_F32) {
        auto split = [&](auto finite) {
#pragma unroll
            for (int e = 0; e < 4; e++) {
                float a[3], b[3];
                split3<decltype(finite)::value>(__uint_as_float(raw.v[e / 2][2 * (e % 2)]), a);
                split3<decltype(finite)::value>(__uint_as_float(raw.v[e / 2][2 * (e % 2) + 1]), b);
#pragma unroll
                for (int p = 0; p < 3; p++)
                    out[p][e] = __builtin_amdgcn_perm(__float_as_uint(b[p]), __float_as_uint(a[p]), 0x07060302u);
            }
        };
        // 0 times each value, added up, is 0 unless one is not finite: a third
        // fewer operations than treating every value as if it might be.
        float zero = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; e++) zero = fmaf(__uint_as_float(raw.v[e / 4][e % 4]), 0.0f, zero);
        if (__any(zero != 0.0f)) split(std::false_type{});
        else split(std::true_type{});
    } else {
        out[0] = order_x<XT>(raw.v[0]);
    }
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

template <int XT>
__device__ __forceinline__ v16f mfma32(u32x4 x, u32x4 w, v16f c) {
    if constexpr (XT == T_F16)
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, x),
                                                      __builtin_bit_cast(f16x8, w), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, x),
                                                       __builtin_bit_cast(bf16x8, w), c, 0, 0, 0);
}

// Half h of the wave (lanes 32 h ..) holds words 8 h .. 8 h + 7 of its row's
// 16; after this, step j's word (2 j in half 0, 2 j + 1 in half 1: 16 weights)
// is v[j & 1][j / 2 % 2 + 2 * (j / 4)].
__device__ __forceinline__ void transpose_halves(u32x4 (&v)[2]) {
    const u32x4 a = v[0], b = v[1];
    auto p0 = __builtin_amdgcn_permlane32_swap(a[0], a[1], false, false);  // steps 0, 4
    auto p1 = __builtin_amdgcn_permlane32_swap(a[2], a[3], false, false);  // steps 1, 5
    auto p2 = __builtin_amdgcn_permlane32_swap(b[0], b[1], false, false);  // steps 2, 6
    auto p3 = __builtin_amdgcn_permlane32_swap(b[2], b[3], false, false);  // steps 3, 7
    v[0] = u32x4{p0[0], p2[0], p0[1], p2[1]};
    v[1] = u32x4{p1[0], p3[0], p1[1], p3[1]};
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

// Up to 8 rows of X.  A workgroup owns 16 columns n of Y; its waves deal the K
// units out among themselves and add their sums through LDS in wave order.  The
// weights are the B operand of the 16 x 16 x 32 instruction (lane: column n =
// lane % 16, eight k of step j from lane group lane / 16) and go from memory to
// registers in 16-byte loads, one pass, PF units ahead.  X is the A operand,
// rows past M repeating the last one.  X, the scales (as floats) and the zero
// points (as dequant's constants) are staged in LDS chunk by chunk: a wave's X
// loads would otherwise take four times the load instructions of its weights,
// float X would be split by every wave, and loads as small as a scale's would
// hold up the weights' behind them, since loads complete in order.
// GS: steps of 32 that share a scale (4 for groups of 128 or more).
struct ScaleZero {
    float s;
    uint32_t z;
};

template <int XT, int GS, int NWT, int PF, int NW>
__global__ void __launch_bounds__(64 * NW, 4)
q4_rows(Q4Args g, int chunk, int tiles) {
    // 32-bit offsets within a tile: the host sends larger strides elsewhere.
    constexpr int P = parts<XT>(), NS = 4 / GS, XS = XT == T_F32 ? 4 : 2;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int nw = NW, nt = 64 * NW;
    const int r = lane & 15, lg = lane >> 4;
    const int K = int(g.K), bytes = (K + 1) / 2, last = (K - 1) >> g.shift;
    // All units, and those wholly inside a row.
    const int units = (K + kUnit - 1) / kUnit, full = bytes / (kUnit / 2);
    for (int tile = blockIdx.x; tile < tiles; tile += int(gridDim.x)) {
        const int64_t n0 = int64_t(tile) * 16;
        const int rows = int(g.M);
        const int cols = int(g.N - n0 < 16 ? g.N - n0 : 16);
        const int mr = r < rows ? r : rows - 1;
        const uint32_t woff = uint32_t(r < cols ? r : cols - 1) * uint32_t(g.ldw) + uint32_t(lg) * 16u;

        u32x4 ring[PF][NWT];
        auto load_unit = [&](u32x4 (&w)[NWT], int idx) {
#pragma unroll
            for (int t = 0; t < NWT; t++) w[t] = load16(g.W[t] + n0 * g.ldw + idx * (kUnit / 2) + woff);
        };
        v4f acc[NWT];
#pragma unroll
        for (int t = 0; t < NWT; t++) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        // LDS of a chunk: a run per lane group and row of X, of units x 4 steps
        // x P parts of 16 bytes and 16 more (runs an odd number of 16 bytes
        // apart fall on different banks), then per unit NWT x NS x 16 scales
        // and zeros.
        const int run = chunk * (4 * P * 16) + 16;
        ScaleZero* const sz = reinterpret_cast<ScaleZero*>(smem + 4 * rows * run);
        const char* const xlane = smem + (lg * rows + mr) * run;
        const ScaleZero* const szlane = sz + r;
        auto do_unit = [&](u32x4 (&w)[NWT], int local) {
            const char* xs = xlane + local * (4 * P * 16);
            const ScaleZero* su = szlane + local * (NWT * NS * 16);
#pragma unroll
            for (int t = 0; t < NWT; t++) transpose_groups(w[t]);
            v4f d[NWT];
            ScaleZero c[NWT];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                u32x4 x[P];
#pragma unroll
                for (int p = 0; p < P; p++)
                    x[p] = *reinterpret_cast<const u32x4*>(xs + (j * P + p) * 16);
#pragma unroll
                for (int t = 0; t < NWT; t++) {
                    if (j % GS == 0) c[t] = su[(t * NS + j / GS) * 16];
                    const u32x4 q = dequant<XT>(w[t][j], c[t].z);
                    // Largest part first.  The instruction rounds to nearest
                    // when what it adds is smaller than the accumulator, and
                    // truncates the accumulator downwards when that is the
                    // smaller one (measured: with the smallest part first,
                    // products of one float and one weight came out up to a
                    // unit too low).
#pragma unroll
                    for (int p = 0; p < P; p++)
                        d[t] = mfma16<XT>(x[p], q, p == 0 && j % GS == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : d[t]);
                    if (j % GS == GS - 1) {
#pragma unroll
                        for (int e = 0; e < 4; e++) acc[t][e] = fmaf(c[t].s, d[t][e], acc[t][e]);
                    }
                }
            }
        };

        // The wave's units in order: of each chunk, the wave-th of nw runs (64
        // bytes of a row per unit, so a wave reads whole stretches of its rows:
        // 33 MB in 7.5 us, against 9.7 with the units dealt out one by one).
        int next_c = 0, next_i = -1;
        auto load_next = [&](u32x4 (&w)[NWT]) {
            for (; next_c < full; next_c += chunk, next_i = -1) {
                const int cf = full - next_c < chunk ? full - next_c : chunk, per = (cf + nw - 1) / nw;
                if (next_i < 0) next_i = wave * per;
                const int i1 = (wave + 1) * per < cf ? (wave + 1) * per : cf;
                if (next_i < i1) {
                    load_unit(w, next_c + next_i++);
                    return;
                }
            }
        };
        // Staging of a chunk, BX pieces of 8 elements of X and BS scales a lane
        // at a time.  The first chunk's first loads go out before the first
        // weights': loads complete in order, so the staging then waits for
        // them alone while the weights are on their way.
        constexpr int BX = 2, BS = 2;
        const int tid = threadIdx.x;
        for (int c0 = 0; c0 < units; c0 += chunk) {
            const int cn = units - c0 < chunk ? units - c0 : chunk;
            // Pieces of X: (row xm, piece kk) by consecutive lanes along K;
            // scales: 16 rows by nt / 16 groups of a matrix a trip.
            const int nk = cn * 16, nq = cn * NS, row = tid % 16;
            const int64_t n = n0 + (row < cols ? row : cols - 1);
            int xm = 0, xk = 0, st = 0, sq = 0;
            if (c0 > 0) __syncthreads();
            while (xm < rows || st < NWT) {
                RawX<XT> x[BX];
                uint32_t s[BS], z[BS];
                const int xm0 = xm, xk0 = xk, st0 = st, sq0 = sq;
#pragma unroll
                for (int b = 0; b < BX; b++) {
                    // 32 bits: 64-bit products took 8 x 4096 x 4096 of floats 14.9 us, not 13.1.
                    const uint32_t off = (uint32_t(xm) * uint32_t(g.ldx) + uint32_t(c0 * 16 + xk + tid) * 8u) * XS;
                    if (xm < rows && xk + tid < nk)
                        load_x_checked<XT>(static_cast<const char*>(g.X) + off, K - (c0 * 16 + xk + tid) * 8, x[b]);
                    xk += nt;
                    if (xk >= nk) xk = 0, xm++;
                }
#pragma unroll
                for (int b = 0; b < BS; b++) {
                    const int q = sq + tid / 16;
                    if (st < NWT && q < nq) {
                        // Past the last group (X is zero there) the scale is 0.
                        const int at = ((c0 + q / NS) * kUnit + q % NS * (kUnit / NS)) >> g.shift;
                        const int gi = at < last ? at : last;
                        const void* sp = st ? g.S[NWT - 1] : g.S[0];
                        const uint8_t* zp = st ? g.Z[NWT - 1] : g.Z[0];
                        s[b] = load_raw(g.stype, sp, n * g.lds + gi);
                        if (at > last) s[b] = 0;
                        z[b] = zp ? zp[n * g.ldz + gi] : 8;
                    }
                    sq += nt / 16;
                    if (sq >= nq) sq = 0, st++;
                }
                if (c0 == 0 && xm0 == 0 && xk0 == 0) {
#pragma unroll
                    for (int p = 0; p < PF; p++) load_next(ring[p]);
                }
                xm = xm0, xk = xk0, st = st0, sq = sq0;
#pragma unroll
                for (int b = 0; b < BX; b++) {
                    const int kk = xk + tid;
                    if (xm < rows && kk < nk) {
                        u32x4 out[P];
                        operand_x<XT>(x[b], out);
                        char* dst = smem + (kk % 4 * rows + xm) * run + kk / 4 * (P * 16);
#pragma unroll
                        for (int p = 0; p < P; p++) *reinterpret_cast<u32x4*>(dst + p * 16) = out[p];
                    }
                    xk += nt;
                    if (xk >= nk) xk = 0, xm++;
                }
#pragma unroll
                for (int b = 0; b < BS; b++) {
                    const int q = sq + tid / 16;
                    if (st < NWT && q < nq) {
                        ScaleZero v;
                        v.s = raw_to_float(g.stype, s[b]);
                        v.z = zero_const<XT>(z[b]);
                        sz[(q / NS * NWT + st) * (NS * 16) + q % NS * 16 + row] = v;
                    }
                    sq += nt / 16;
                    if (sq >= nq) sq = 0, st++;
                }
            }
            __syncthreads();
            const int cf = full - c0 < cn ? full - c0 : cn, per = (cf + nw - 1) / nw;
            const int i0 = wave * per, i1 = i0 + per < cf ? i0 + per : cf;
            for (int i = i0; i < i1; i += PF)
#pragma unroll
                for (int p = 0; p < PF; p++)
                    if (i + p < i1) {
                        do_unit(ring[p], i + p);
                        load_next(ring[p]);
                    }
            // The unit that rows end in goes to the last wave.
            if (cf < cn && wave == nw - 1) {
                u32x4 w[NWT];
#pragma unroll
                for (int t = 0; t < NWT; t++)
                    w[t] = load_w_tail(g.W[t] + (n0 + (r < cols ? r : cols - 1)) * g.ldw,
                                       full * (kUnit / 2) + lg * 16, bytes);
                do_unit(w, full - c0);
            }
        }

        // Accumulator register e of lane (lg, r) is row 4 lg + e, column r.
        __syncthreads();
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int t = 0; t < NWT; t++)
#pragma unroll
            for (int e = 0; e < 4; e++) red[(wave * NWT + t) * 256 + (4 * lg + e) * 16 + r] = acc[t][e];
        __syncthreads();
        for (int o = threadIdx.x; o < rows * 16; o += nt) {
            float sum[NWT];
#pragma unroll
            for (int t = 0; t < NWT; t++) {
                sum[t] = red[t * 256 + o];
                for (int w = 1; w < nw; w++) sum[t] += red[(w * NWT + t) * 256 + o];
            }
            const int64_t m = o / 16, nn = n0 + o % 16;
            if (nn < g.N)
                store_as<XT>(g.Y, m * g.ldy + nn, NWT == 2 ? act_value(g.act, sum[0]) * sum[NWT - 1] : sum[0]);
        }
        if (tile + int(gridDim.x) < tiles) __syncthreads();
    }
}

// X and the scales are staged whole, or in chunks of whole rounds of the waves,
// PF units each.
template <int XT, int GS, int NWT, int PF, int NW>
static hipError_t launch_rows_cfg(const Q4Args& g, int64_t unit_bytes, hipStream_t s) {
    const int64_t units = ceil_div(g.K, kUnit), fixed = 64 * g.M, round = NW * PF;
    int64_t chunk = (kRowsLds - fixed) / unit_bytes / round * round;
    if (chunk < round) chunk = round;
    if (chunk > units) chunk = units;
    size_t lds = size_t(NW) * NWT * 1024;
    if (size_t(chunk * unit_bytes + fixed) > lds) lds = size_t(chunk * unit_bytes + fixed);
    const int64_t tiles = ceil_div(g.N, 16);
    hipLaunchKernelGGL((q4_rows<XT, GS, NWT, PF, NW>), dim3(grid_for(tiles)), dim3(64 * NW), lds, s, g,
                       int(chunk), int(tiles));
    return hipGetLastError();
}

template <int XT, int GS, int NWT>
static hipError_t launch_rows(const Q4Args& g, hipStream_t s) {
    const int64_t units = ceil_div(g.K, kUnit), rows = g.M;
    const int64_t unit_bytes = 4 * parts<XT>() * 4 * rows * 16 + NWT * (4 / GS) * 16 * int64_t(sizeof(ScaleZero));
    // Four units ahead in eight waves where that much of X leaves room for two
    // workgroups in a CU's LDS; more of it (float X of several rows) takes one
    // workgroup, of sixteen waves that load one unit ahead.
    if ((units < 32 ? units : 32) * unit_bytes + 64 * rows <= kRowsLds)
        return launch_rows_cfg<XT, GS, NWT, NWT == 1 ? 4 : 2, 8>(g, unit_bytes, s);
    return launch_rows_cfg<XT, GS, NWT, 1, 16>(g, unit_bytes, s);
}

// More rows of X: tiles on the 32 x 32 x 16 instruction.  A workgroup is WK
// groups of WN waves over one tile of BM = 32 TM rows and BN = 32 WN columns;
// K group kg takes units kg, kg + WK, ... of 128 k, and the groups' sums are
// added through LDS in group order.  Within a group every wave owns 32 columns
// (of each weight matrix) and all BM rows: its weights go from memory to its
// registers and are converted there, once in the workgroup, while X, which
// all waves of the group read, is staged in LDS in slabs of 64 k as the
// instruction takes it (float X split on the way), two slabs in turn with one
// barrier each.
// LDS of a slab: TM x 4 steps x P parts of two halves of 512 bytes (row L % 32
// of half L / 32 at 16 (L % 32): eight k each).  Halves are 128 bytes further
// apart than that and parts 32 (modulo the banks' 256), so that the 8 pieces
// each of two rows that 16 lanes write at once fall on different banks.
template <int XT, int GS, int NWT, int TM, int WN, int WK, bool S32>
__global__ void __launch_bounds__(64 * WN * WK)
q4_tile(Q4Args g, int tiles_m, int tiles_n) {
    constexpr int P = parts<XT>(), NS = 4 / GS, BM = 32 * TM, BN = 32 * WN;
    constexpr int HALF = 512 + 128, FRAG = 5 * 256 + 32, SLAB = TM * 4 * P * FRAG;
    constexpr int RED = WK > 1 ? (WK - 1) * WN * NWT * TM * 4096 : 0;
    constexpr int LDS = 2 * WK * SLAB > RED ? 2 * WK * SLAB : RED;
    constexpr int PIECES = BM * 8 / (64 * WN);  // of 8 elements, per lane and slab
    static_assert(PIECES * 64 * WN == BM * 8, "whole pieces");
    __shared__ __attribute__((aligned(16))) char smem[LDS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / WN, wn = wave % WN, gtid = threadIdx.x - kg * (64 * WN);
    const int r = lane & 31, half = lane >> 5;
    const int K = int(g.K), bytes = (K + 1) / 2, last = (K - 1) >> g.shift;
    const int units = (K + kUnit - 1) / kUnit, full = bytes / (kUnit / 2);
    const int iters = (units + WK - 1) / WK;
    constexpr int XS = XT == T_F32 ? 4 : 2, SB = S32 ? 4 : 2, SW = (NS * SB + 3) / 4;

    // Each XCD a contiguous range of tiles, four rows of tiles at a time: the
    // 32 tiles it runs together are about as wide as they are high in bytes,
    // which is the least to bring into its L2.
    const int tiles = tiles_m * tiles_n;
    for (int t0 = blockIdx.x; t0 < tiles; t0 += gridDim.x) {
        int lin = t0;
        if (int(gridDim.x) == tiles) {
            const int q = tiles / 8, rem = tiles % 8, x = t0 % 8;
            lin = x * q + (x < rem ? x : rem) + t0 / 8;
        }
        const int64_t per_group = 4 * int64_t(tiles_n);
        const int first = int(lin / per_group) * 4, in = int(lin % per_group);
        const int high = tiles_m - first < 4 ? tiles_m - first : 4;
        const int64_t m0 = int64_t(first + in % high) * BM, n0 = int64_t(in / high) * BN + wn * 32;
        // The lane's row of the weights, from the wave's first (or the last row
        // there is), and its pieces of X, from the tile's first row.
        const int64_t nb = n0 < g.N ? n0 : g.N - 1;
        const uint32_t rn = nb + r < g.N ? r : uint32_t(g.N - 1 - nb);
        const uint32_t woff = rn * uint32_t(g.ldw) + half * 32, soff = rn * uint32_t(g.lds) * SB,
                       zoff = rn * uint32_t(g.ldz);
        uint32_t xoff[PIECES];
#pragma unroll
        for (int p = 0; p < PIECES; p++) {
            const int i = gtid + p * (64 * WN), row = i / 8;
            xoff[p] = (uint32_t(m0 + row < g.M ? row : g.M - 1 - m0) * uint32_t(g.ldx) + i % 8 * 8) * XS;
        }

        // Loads of a unit's weights, scales and zero points and of a slab's X
        // into registers; CHECK: the unit is the one K ends in.  Without it
        // there are no branches, so that the waits for earlier loads can be
        // counted and later ones stay in flight.
        struct Unit {
            u32x4 w[NWT][2];
            uint32_t s[NWT][SW], z[NWT];  // NS scales as loaded, NS bytes
        };
        auto load_unit = [&](auto check, Unit& u, int idx) {
            constexpr bool CHECK = decltype(check)::value;
            const uint32_t gi = uint32_t(idx * kUnit) >> g.shift;
#pragma unroll
            for (int t = 0; t < NWT; t++) {
                const uint8_t* wp = g.W[t] + nb * g.ldw + idx * (kUnit / 2);
                const char* sp = static_cast<const char*>(g.S[t]) + nb * g.lds * SB;
                const uint8_t* zp = g.Z[t] ? g.Z[t] + nb * g.ldz : nullptr;
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    if (!CHECK || idx < full) u.w[t][h] = load16(wp + woff + h * 16);
                    else u.w[t][h] = load_w_tail(wp + woff, h * 16, bytes - idx * (kUnit / 2) - half * 32);
                }
                if constexpr (!CHECK) {
                    __builtin_memcpy(u.s[t], sp + (soff + gi * SB), NS * SB);
                    // Without zero points a load all the same, of the weights:
                    // one path, and its value is not used.
                    const uint8_t* any = zp ? zp + (zoff + gi) : wp + woff;
                    u.z[t] = 0;
                    __builtin_memcpy(&u.z[t], any, NS);
                } else {
                    u.z[t] = 0;
#pragma unroll
                    for (int q = 0; q < SW; q++) u.s[t][q] = 0;
#pragma unroll
                    for (int q = 0; q < NS; q++) {
                        // Past the last group (X is zero there) the scale is 0.
                        const int at = (idx * kUnit + q * (kUnit / NS)) >> g.shift, gq = at < last ? at : last;
                        const uint32_t raw = at > last ? 0u : load_raw(g.stype, sp, (soff / SB) + uint32_t(gq));
                        u.s[t][q * SB / 4] |= raw << (S32 ? 0 : q % 2 * 16);
                        u.z[t] |= uint32_t(zp ? zp[zoff + uint32_t(gq)] : 0) << (8 * q);
                    }
                }
            }
        };
        auto load_slab = [&](auto check, RawX<XT> (&x)[PIECES], int slab) {
            constexpr bool CHECK = decltype(check)::value;
            const char* xb = static_cast<const char*>(g.X) + (m0 * g.ldx + int64_t(slab) * 64) * XS;
#pragma unroll
            for (int p = 0; p < PIECES; p++) {
                if constexpr (CHECK) {
                    load_x_checked<XT>(xb + xoff[p], K - slab * 64 - (gtid + p * (64 * WN)) % 8 * 8, x[p]);
                } else {
                    x[p].v[0] = load16(xb + xoff[p]);
                    if constexpr (XT == T_F32) x[p].v[1] = load16(xb + xoff[p] + 16);
                }
            }
        };
        auto store_slab = [&](const RawX<XT> (&x)[PIECES], int buf) {
            char* base = smem + (buf * WK + kg) * SLAB;
#pragma unroll
            for (int p = 0; p < PIECES; p++) {
                const int i = gtid + p * (64 * WN), m = i / 8, kk = i % 8;
                u32x4 out[P];
                operand_x<XT>(x[p], out);
#pragma unroll
                for (int q = 0; q < P; q++)
                    *reinterpret_cast<u32x4*>(base + ((m / 32 * 4 + kk / 2) * P + q) * FRAG + kk % 2 * HALF + m % 32 * 16) = out[q];
            }
        };

        v16f acc[NWT][TM], d[NWT][TM];
#pragma unroll
        for (int t = 0; t < NWT; t++)
#pragma unroll
            for (int b = 0; b < TM; b++) acc[t][b] = v16f{};
        // Selected by masks, not branches: control flow between the matrix
        // instructions would keep them from being ordered together.
        const uint32_t bf_mask = g.stype == T_BF16 ? 0xFFFFFFFFu : 0u;
        const uint32_t z_mask = g.Z[0] ? 0xFFFFFFFFu : 0u, z_none = g.Z[0] ? 0u : 0x08080808u;
        auto scale_of = [&](const Unit& u, int t, int q) {
            if constexpr (S32) return __uint_as_float(u.s[t][q]);
            const uint32_t v = u.s[t][S32 ? 0 : q / 2] >> (q % 2 * 16) & 0xFFFFu;
            const uint32_t half = __float_as_uint(float(__builtin_bit_cast(_Float16, uint16_t(v))));
            return __uint_as_float((v << 16 & bf_mask) | (half & ~bf_mask));
        };
        auto zero_of = [&](const Unit& u, int t, int q) {
            return zero_const<XT>(((u.z[t] & z_mask) | z_none) >> (8 * q) & 255u);
        };
        // The four steps of one slab; h: which half of its unit it is.  In
        // TM pieces each, held in this order: the LDS read of the X that a
        // later piece needs (AHEAD pieces, about 128 cycles of matrix
        // instructions, cover its latency), the piece's matrix instructions,
        // and vector work beside them: part of the next step's weights, and
        // the scaling of the block before this one where a group ends.  The
        // empty asm statements tie that work to its place: free to move, it
        // all goes to the slab's end and every group's sums stay in registers
        // (2048 x 8192 x 4096 with groups of 32 spilled and took 1.4 ms).
        constexpr int AHEAD = P * NWT >= 6 ? 1 : P * NWT >= 2 ? 2 : 4, RING = AHEAD + 1, PIECE = 4 / TM;
        static_assert(TM * PIECE == 4, "four words of a step's weights over TM pieces");
        auto do_slab = [&](const Unit& u, int buf, auto hc) {
            constexpr int h = decltype(hc)::value, PER = 2 * GS;  // PER: steps that share a scale
            const char* base = smem + (buf * WK + kg) * SLAB + half * HALF + r * 16;
            u32x4 x[RING][P], q[2][NWT];
            auto read = [&](int c) {
                const int j = c / TM, b = c % TM;
#pragma unroll
                for (int p = 0; p < P; p++)
                    x[c % RING][p] = *reinterpret_cast<const u32x4*>(base + ((b * 4 + j) * P + p) * FRAG);
            };
            auto scale = [&](int t, int step, int b) {
                const float s = scale_of(u, t, step / PER);
#pragma unroll
                for (int e = 0; e < 16; e++) acc[t][b][e] = fmaf(s, d[t][b][e], acc[t][b][e]);
                asm volatile("" : "+v"(acc[t][b]));
            };
            auto word = [&](int t, int step) { return u.w[t][step & 1][(step & 3) / 2 + (step >> 2) * 2]; };
#pragma unroll
            for (int c = 0; c < AHEAD; c++) read(c);
#pragma unroll
            for (int t = 0; t < NWT; t++) q[0][t] = dequant<XT>(word(t, h * 4), zero_of(u, t, h * 4 / PER));
            Halves next[NWT];
#pragma unroll
            for (int c = 0; c < 4 * TM; c++) {
                const int j = c / TM, b = c % TM, step = h * 4 + j;
                __builtin_amdgcn_sched_barrier(0);
                if (c + AHEAD < 4 * TM) read(c + AHEAD);
                // With one block its sums go before they are overwritten.
                if (TM == 1 && c > 0 && (step - 1) % PER == PER - 1) {
#pragma unroll
                    for (int t = 0; t < NWT; t++) scale(t, step - 1, 0);
                }
#pragma unroll
                for (int t = 0; t < NWT; t++)
#pragma unroll
                    for (int p = 0; p < P; p++)
                        d[t][b] = mfma32<XT>(x[c % RING][p], q[j & 1][t], p == 0 && step % PER == 0 ? v16f{} : d[t][b]);
#pragma unroll
                for (int t = 0; t < NWT; t++) {
                    if (j < 3) {
                        const uint32_t z = zero_of(u, t, (step + 1) / PER);
                        if (b == 0) next[t] = dequant_prepare<XT>(word(t, step + 1), z);
#pragma unroll
                        for (int i = 0; i < PIECE; i++) {
                            uint32_t w = dequant_word<XT>(next[t], z, b * PIECE + i);
                            asm volatile("" : "+v"(w));
                            q[(j + 1) & 1][t][b * PIECE + i] = w;
                        }
                    }
                    const int cb = c - 1, sb = h * 4 + cb / TM;  // the block before
                    if (TM > 1 && c > 0 && sb % PER == PER - 1) scale(t, sb, cb % TM);
                    if (c == 4 * TM - 1 && step % PER == PER - 1) scale(t, step, b);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        };

        // The group's units kg, kg + WK, ...: X slabs are loaded two slabs
        // ahead of their use, weights one unit (two slabs) ahead.
        Unit u;
        RawX<XT> xa[PIECES], xb[PIECES];
        if (kg < units) {
            load_slab(std::true_type{}, xa, 2 * kg);
            load_unit(std::true_type{}, u, kg);
            load_slab(std::true_type{}, xb, 2 * kg + 1);
            store_slab(xa, 0);
        }
        __syncthreads();
        auto unit_step = [&](auto check, int idx, bool on, bool more) {
            Unit v;
            if (on) {
                v = u;
#pragma unroll
                for (int t = 0; t < NWT; t++) transpose_halves(v.w[t]);
                if (more) {
                    load_slab(check, xa, 2 * (idx + WK));
                    load_unit(check, u, idx + WK);
                }
                do_slab(v, 0, std::integral_constant<int, 0>{});
                store_slab(xb, 1);
            }
            __syncthreads();
            if (on) {
                if (more) load_slab(check, xb, 2 * (idx + WK) + 1);
                do_slab(v, 1, std::integral_constant<int, 1>{});
                if (more) store_slab(xa, 0);
            }
            __syncthreads();
        };
        // Unchecked while the next unit is whole in K.
        int i = 0;
        for (; i < iters && (i * WK + kg + WK + 1) * kUnit <= K; i++) unit_step(std::false_type{}, i * WK + kg, true, true);
        for (; i < iters; i++) {
            const int idx = i * WK + kg;
            unit_step(std::true_type{}, idx, idx < units, idx + WK < units);
        }

        if constexpr (WK > 1) {
            float* red = reinterpret_cast<float*>(smem);
            constexpr int PER_WAVE = NWT * TM * 1024;
            if (kg > 0) {
                float* o = red + ((kg - 1) * WN + wn) * PER_WAVE + lane;
#pragma unroll
                for (int t = 0; t < NWT; t++)
#pragma unroll
                    for (int b = 0; b < TM; b++)
#pragma unroll
                        for (int e = 0; e < 16; e++) o[((t * TM + b) * 16 + e) * 64] = acc[t][b][e];
            }
            __syncthreads();
            if (kg == 0) {
#pragma unroll 1
                for (int k = 0; k < WK - 1; k++) {
                    const float* o = red + (k * WN + wn) * PER_WAVE + lane;
#pragma unroll
                    for (int t = 0; t < NWT; t++)
#pragma unroll
                        for (int b = 0; b < TM; b++)
#pragma unroll
                            for (int e = 0; e < 16; e++) acc[t][b][e] += o[((t * TM + b) * 16 + e) * 64];
                }
            }
        }
        // Accumulator register e of a lane is row 8 (e / 4) + 4 half + e % 4 of
        // its block, column r.
        if (kg == 0 && n0 < g.N) {
            const int rows = int(g.M - m0 < BM ? g.M - m0 : BM);
            if constexpr (NWT == 2) {
#pragma unroll
                for (int b = 0; b < TM; b++) {
                    float gate[16];
#pragma unroll
                    for (int e = 0; e < 16; e++) gate[e] = acc[0][b][e];
                    act_values<16>(g.act, gate, gate);
#pragma unroll
                    for (int e = 0; e < 16; e++) acc[0][b][e] = gate[e] * acc[NWT - 1][b][e];
                }
            }
            constexpr int kRow[4] = {0, 8, 16, 24};
            if constexpr (WK == 1 && XS == 2) {
                // Through LDS (its stages are free), a block at a time, for
                // 16-byte stores: 2 bytes a lane took 9 % of a prompt's time
                // (floats, whose 32 lanes fill cache lines, lose by it).
                constexpr int PITCH = 32 * XS + 16, EL = 16 / XS, LPR = 32 / EL;
                static_assert(WN * 32 * PITCH <= LDS, "blocks fit the stages");
                char* const st = smem + wn * (32 * PITCH);
                const int cols = int(g.N - n0 < 32 ? g.N - n0 : 32);
#pragma unroll
                for (int b = 0; b < TM; b++) {
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int e = 0; e < 16; e++)
                        store_as<XT>(st + (kRow[e / 4] + e % 4 + 4 * half) * PITCH, r, acc[0][b][e]);
                    // Exchanged within the wave, whose LDS operations complete
                    // in order.
                    asm volatile("" ::: "memory");
                    __builtin_amdgcn_wave_barrier();
#pragma unroll
                    for (int q = 0; q < 32 * LPR; q += 64) {
                        const int row = (q + lane) / LPR, c = lane % LPR * EL;
                        if (b * 32 + row >= rows) continue;
                        const u32x4 v = *reinterpret_cast<const u32x4*>(st + row * PITCH + c * XS);
                        char* yp = static_cast<char*>(g.Y) + ((m0 + b * 32 + row) * g.ldy + n0 + c) * XS;
                        if (c + EL <= cols) {
                            __builtin_memcpy(yp, &v, 16);
                        } else {
                            for (int i = 0; i < EL; i++)
                                if (c + i < cols) __builtin_memcpy(yp + i * XS, st + row * PITCH + (c + i) * XS, XS);
                        }
                    }
                    asm volatile("" ::: "memory");
                }
            } else if (n0 + r < g.N) {
                char* yp = static_cast<char*>(g.Y) + (m0 * g.ldy + n0) * XS;
                const uint32_t yoff = (4 * half * uint32_t(g.ldy) + r) * XS;
#pragma unroll
                for (int b = 0; b < TM; b++)
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        const int row = b * 32 + kRow[e / 4] + e % 4;
                        if (row < rows - 4 * half) store_as<XT>(yp + int64_t(row) * g.ldy * XS + yoff, 0, acc[0][b][e]);
                    }
            }
        }
        if (t0 + int(gridDim.x) < tiles) __syncthreads();
    }
}

template <int XT, int GS, int NWT, int TM, int WN, int WK>
static hipError_t launch_tile(const Q4Args& g, hipStream_t s) {
    const int64_t tm = ceil_div(g.M, 32 * TM), tn = ceil_div(g.N, 32 * WN);
    const dim3 grid(grid_for(tm * tn)), block(64 * WN * WK);
    if (g.stype == T_F32)
        hipLaunchKernelGGL((q4_tile<XT, GS, NWT, TM, WN, WK, true>), grid, block, 0, s, g, int(tm), int(tn));
    else
        hipLaunchKernelGGL((q4_tile<XT, GS, NWT, TM, WN, WK, false>), grid, block, 0, s, g, int(tm), int(tn));
    return hipGetLastError();
}

// Tile by shape.  One round of workgroups, one per CU, takes about the same time
// whatever its number, and that time grows much more slowly than the tile (a
// small tile shares out K instead), so the choice is the configuration with the
// least rounds x time of a round.  Times measured on MI355X at K = 4096 (us; the
// ratios at K = 2048 are alike): bfloat16 and float16 / float, of one product and
// of the gated pair, on rounds that leave some CUs idle (a full one of the 128 x
// 256 tile takes 78 / 191, as the CUs then share the L2s and memory), and in
// groups of 128 / 64.  Over 9 to 1024 rows by 1024 to 8192 columns the choice is
// the fastest of these five, or within 15 % of it; always the 128 x 256 tile
// would take 70 us for 9 rows where 14 do, always the 32 x 32 one 383 for 1024
// rows where 78 do.  A sixth tile of the plain product, 64 x 256, would be faster
// where it fills one round (512 x 8192 x 4096 52 us where the choice takes 60,
// float 108 and 127; 1024 x 4096 x 4096 53 and 62).
template <int XT, int GS, int NWT>
static hipError_t launch_tiles(const Q4Args& g, hipStream_t s) {
    constexpr bool f = XT == T_F32, two = NWT == 2;
    constexpr int kTiles[5][2] = {{32, 32}, {32, 64}, {32, 128}, {64, 128}, {two ? 64 : 128, 256}};
    constexpr int kTime[5] = {two ? (f ? 37 : 23) : (f ? 28 : 14), two ? (f ? 44 : 29) : (f ? 29 : 16),
                              two ? (f ? 68 : 49) : (f ? 41 : 23), two ? (f ? 117 : 61) : (f ? 62 : 31),
                              two ? (f ? 162 : 101) : (f ? 160 : 70)};
    constexpr int64_t kCUs = 256;
    int best = 0;
    int64_t best_time = 0;
    for (int c = 0; c < 5; c++) {
        const int64_t tiles = ceil_div(g.M, kTiles[c][0]) * ceil_div(g.N, kTiles[c][1]);
        const int64_t time = ceil_div(tiles, kCUs) * kTime[c];
        if (c == 0 || time < best_time) {
            best = c;
            best_time = time;
        }
    }
    switch (best) {
        case 0: return launch_tile<XT, GS, NWT, 1, 1, f ? 4 : 8>(g, s);
        case 1: return launch_tile<XT, GS, NWT, 1, 2, 4>(g, s);
        case 2: return launch_tile<XT, GS, NWT, 1, 4, 2>(g, s);
        case 3: return launch_tile<XT, GS, NWT, 2, 4, two ? 1 : 2>(g, s);
        default: return launch_tile<XT, GS, NWT, two ? 2 : 4, 8, 1>(g, s);
    }
}

template <int XT, int GS, int NWT>
static hipError_t launch_gs(const Q4Args& g, hipStream_t s) {
    return g.M <= kRowsMax ? launch_rows<XT, GS, NWT>(g, s) : launch_tiles<XT, GS, NWT>(g, s);
}

// The kernels of one type of X and one form (NWT 1: the product, 2: gated).
template <int XT, int NWT>
hipError_t launch_q4_kernels(const Q4Args& g, hipStream_t s) {
    if (g.shift >= 7) return launch_gs<XT, 4, NWT>(g, s);
    if (g.shift == 6) return launch_gs<XT, 2, NWT>(g, s);
    return launch_gs<XT, 1, NWT>(g, s);
}

}  // namespace sgemm
