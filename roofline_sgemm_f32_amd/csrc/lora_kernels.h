// Low-rank adapters: Y[m] = base[m] + s_l (X[m] A_l^T) B_l^T, l = ids[m].
//
// Two products, both bound by memory.  lora_shrink forms H = X A^T (long sums,
// R results a row) in float partial sums, one plane for each share of K;
// lora_expand adds the planes up and forms Y (short sums, N results a row).
// Rows come in tiles of one adapter each (RowPlan), so an adapter is read once
// for up to 64 rows.  Nothing is staged: the matrix instructions' operands are
// 16 bytes along K (or R) of one row, which is how memory holds them.
#pragma once
#include "lora_rows.h"

namespace sgemm {
namespace {

// ---- H = X A^T ----------------------------------------------------------------

struct ShrinkArgs {
    const void* X;      // rows of K elements
    int64_t ldx;
    const void* W;      // L x R x K
    int64_t ldw, sw;
    int64_t K;
    int R;
    const float* scales;  // with scaled: the sums times alpha scales[l]
    float alpha;
    bool scaled;
    float* P;           // planes of M x R, one for each K share
    int64_t plane;
    int64_t kshare;     // K per grid.y
    RowPlan rows;
    int64_t tiles;
};

constexpr int kShrinkWaves = 4;

// A workgroup: a tile of 16 TMB rows, 16 RB of the R columns, a share of K split
// again over its waves, whose sums are added through LDS.
template <int T, int RB, int TMB>
__global__ void __launch_bounds__(64 * kShrinkWaves) lora_shrink(ShrinkArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, STEP = 4 * V;  // K of one mma16
    __shared__ float red[2][TMB * RB * 256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int r0 = blockIdx.z * 16 * RB;
    const int64_t kb = blockIdx.y * a.kshare, ke = kb + a.kshare < a.K ? kb + a.kshare : a.K;
    // The wave's part: whole double steps, the last wave's shorter.
    const int64_t part = ((ke - kb + kShrinkWaves - 1) / kShrinkWaves + 2 * STEP - 1) / (2 * STEP) * (2 * STEP);
    for (int64_t t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const RowTile tile = row_tile(a.rows, t, 16 * TMB);
        if (tile.count == 0) break;       // past the last tile
        if (tile.adapter < 0) continue;
        const E* x[TMB];
#pragma unroll
        for (int b = 0; b < TMB; b++) {
            const int p = 16 * b + i;
            x[b] = static_cast<const E*>(a.X) + int64_t(row_at(a.rows, tile.start + (p < tile.count ? p : 0))) * a.ldx;
        }
        const E* w[RB];
#pragma unroll
        for (int b = 0; b < RB; b++) {
            const int r = r0 + 16 * b + i;
            w[b] = static_cast<const E*>(a.W) + tile.adapter * a.sw + int64_t(r < a.R ? r : a.R - 1) * a.ldw;
        }
        v4f acc[TMB][RB];
#pragma unroll
        for (int m = 0; m < TMB; m++)
#pragma unroll
            for (int n = 0; n < RB; n++) acc[m][n] = v4f{0, 0, 0, 0};
        int64_t k = kb + wave * part;
        const int64_t end = k + part < ke ? k + part : ke;
        auto step = [&](const u32x4 (&xf)[TMB], const u32x4 (&wf)[RB]) {
#pragma unroll
            for (int m = 0; m < TMB; m++)
#pragma unroll
                for (int n = 0; n < RB; n++) acc[m][n] = mma16<T>(xf[m], wf[n], acc[m][n]);
        };
        for (; k + 2 * STEP <= end; k += 2 * STEP) {
            u32x4 xf[2][TMB], wf[2][RB];
#pragma unroll
            for (int u = 0; u < 2; u++) {
#pragma unroll
                for (int n = 0; n < RB; n++) wf[u][n] = load16(w[n] + k + u * STEP + g * V);
#pragma unroll
                for (int m = 0; m < TMB; m++) xf[u][m] = load16(x[m] + k + u * STEP + g * V);
            }
            step(xf[0], wf[0]);
            step(xf[1], wf[1]);
        }
        for (; k < end; k += STEP) {
            u32x4 xf[TMB], wf[RB];
#pragma unroll
            for (int n = 0; n < RB; n++) wf[n] = load_chunk<T>(w[n], k + g * V, end);
#pragma unroll
            for (int m = 0; m < TMB; m++) xf[m] = load_chunk<T>(x[m], k + g * V, end);
            step(xf, wf);
        }
        // Waves 2, 3 to 0, 1, then wave 1 to 0.
#pragma unroll
        for (int half = kShrinkWaves / 2; half; half /= 2) {
            __syncthreads();
            if (wave >= half && wave < 2 * half) {
#pragma unroll
                for (int m = 0; m < TMB; m++)
#pragma unroll
                    for (int n = 0; n < RB; n++)
                        *reinterpret_cast<v4f*>(&red[wave - half][(m * RB + n) * 256 + 4 * lane]) = acc[m][n];
            }
            __syncthreads();
            if (wave < half) {
#pragma unroll
                for (int m = 0; m < TMB; m++)
#pragma unroll
                    for (int n = 0; n < RB; n++)
                        acc[m][n] += *reinterpret_cast<v4f*>(&red[wave][(m * RB + n) * 256 + 4 * lane]);
            }
        }
        if (wave == 0) {
            const float f = a.scaled ? a.alpha * (a.scales ? a.scales[tile.adapter] : 1.0f) : 1.0f;
            float* P = a.P + blockIdx.y * a.plane;
#pragma unroll
            for (int m = 0; m < TMB; m++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int p = 16 * m + 4 * g + e;
                    if (p >= tile.count) continue;
                    float* row = P + int64_t(row_at(a.rows, tile.start + p)) * a.R;
#pragma unroll
                    for (int n = 0; n < RB; n++) {
                        const int r = r0 + 16 * n + i;
                        if (r < a.R) row[r] = a.scaled ? acc[m][n][e] * f : acc[m][n][e];
                    }
                }
        }
    }
}

// ---- Y = base + s H B^T -------------------------------------------------------

struct ExpandArgs {
    const float* P;     // H: the sum of `planes` planes of rows of R floats
    int64_t plane;
    int planes, R;
    const void* W;      // L x N x R
    int64_t ldw, sw;
    int64_t N;
    const float* scales;
    float alpha;
    bool scaled;
    const void* base;
    int64_t ldbase;
    void* Y;
    int64_t ldy;
    float* H;           // also store H here
    int64_t ldh;
    int64_t nshare;     // N per grid.y, a multiple of 256
    RowPlan rows;
    int64_t tiles;
};

// LDS of a workgroup: H in the operands' form (two 16-bit parts, or floats) with
// rows padded by 16 bytes, and a factor for each row.
template <int T> inline size_t expand_lds(int R, int rows) {
    const int rp = (R + 31) / 32 * 32;
    return size_t(rows) * (T == T_F32 ? (rp + 4) * 4 : 2 * (rp + 8) * 2) + size_t(rows) * 4;
}

// A workgroup: a tile of 16 TMB rows and a share of N, 64 columns a wave at a
// time.  H is rounded to no fewer than 16 bits: for 16-bit types it is the sum
// of two parts, of bfloat16 cut off and rounded (2^-16 of an element), or of
// float16 after a power of two for the row that brings its largest element
// below 2^15 (2^-22, and 2^-39 of that element).  One matrix instruction sums
// over 32: both parts of up to 16 columns (PACKED), or one part of 32.
template <int T, int TMB, bool PACKED>
__global__ void __launch_bounds__(256) lora_expand(ExpandArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, TM = 16 * TMB, STEP = 4 * V;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int rp = (a.R + 31) / 32 * 32;
    const int pitch = T == T_F32 ? (rp + 4) * 4 : (rp + 8) * 2;  // bytes
    char* const hi = smem;
    char* const lo = smem + TM * pitch;  // 16-bit types
    float* const factor = reinterpret_cast<float*>(smem + TM * pitch * (T == T_F32 ? 1 : 2));
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    for (int64_t t = blockIdx.x; t < a.tiles; t += gridDim.x) {
        const RowTile tile = row_tile(a.rows, t, TM);
        if (tile.count == 0) break;
        const bool has = tile.adapter >= 0;
        const bool in_place = a.base == a.Y;
        if (!has && in_place && !a.H) continue;
        const float s = !has || !a.scaled ? 1.0f : a.alpha * (a.scales ? a.scales[tile.adapter] : 1.0f);
        __syncthreads();
        // Sixteen lanes a row.
        for (int p = threadIdx.x >> 4; p < TM; p += 16) {
            const bool in = p < tile.count;
            const int64_t row = in ? row_at(a.rows, tile.start + p) : 0;
            const int c = threadIdx.x & 15;
            float v[16], top = 0.0f;
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const int r = c + 16 * q;
                v[q] = 0.0f;
                if (16 * q < rp) {
                    if (in && has && r < a.R)
                        for (int z = 0; z < a.planes; z++) v[q] += a.P[z * a.plane + row * a.R + r];
                    if (in && r < a.R && a.H && blockIdx.y == 0) a.H[row * a.ldh + r] = v[q];
                    if (fabsf(v[q]) <= 3.4e38f) top = fmaxf(top, fabsf(v[q]));
                }
            }
            float f = s, up = 1.0f;
            if constexpr (T == T_F16) {
#pragma unroll
                for (int d = 1; d < 16; d *= 2) top = fmaxf(top, __shfl_xor(top, d, 16));
                // The power that brings the largest finite one into [2^14, 2^15).
                if (top > 0.0f) {
                    int ex = int(__float_as_uint(top) >> 23) - 127;
                    ex = ex < -100 ? -100 : ex;
                    up = __uint_as_float(uint32_t(14 - ex + 127) << 23);
                    f = s * __uint_as_float(uint32_t(ex - 14 + 127) << 23);
                }
            }
            if (c == 0) factor[p] = f;
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const int r = c + 16 * q;
                if (16 * q >= rp) continue;
                if constexpr (T == T_F32) {
                    *reinterpret_cast<float*>(hi + p * pitch + r * 4) = v[q];
                } else if constexpr (T == T_F16) {
                    const float x = v[q] * up;
                    const _Float16 h = _Float16(x);
                    const float d = x - float(h);
                    *reinterpret_cast<_Float16*>(hi + p * pitch + r * 2) = h;
                    *reinterpret_cast<_Float16*>(lo + p * pitch + r * 2) = _Float16(fabsf(x) <= 65504.0f ? d : 0.0f);
                } else {
                    const uint32_t cut = __float_as_uint(v[q]) & 0xFFFF0000u;
                    const bool finite = (cut & 0x7F800000u) != 0x7F800000u;
                    // A NaN whose payload is in the cut bits stays one.
                    const uint32_t top16 = !finite && v[q] != v[q] ? 0x7FC0u : cut >> 16;
                    *reinterpret_cast<uint16_t*>(hi + p * pitch + r * 2) = uint16_t(top16);
                    *reinterpret_cast<__bf16*>(lo + p * pitch + r * 2) = __bf16(finite ? v[q] - __uint_as_float(cut) : 0.0f);
                }
            }
        }
        __syncthreads();
        const E* const w = static_cast<const E*>(a.W) + (has ? tile.adapter : 0) * a.sw;
        const int64_t nb = blockIdx.y * a.nshare, ne = nb + a.nshare < a.N ? nb + a.nshare : a.N;
        const E* base[TMB];
        E* out[TMB];
        float f[TMB];
        bool in[TMB];
#pragma unroll
        for (int m = 0; m < TMB; m++) {
            in[m] = 16 * m + i < tile.count;
            const int64_t row = row_at(a.rows, tile.start + (in[m] ? 16 * m + i : 0));
            base[m] = a.base ? static_cast<const E*>(a.base) + row * a.ldbase : nullptr;
            out[m] = static_cast<E*>(a.Y) + row * a.ldy;
            f[m] = factor[16 * m + i];
        }
        // Columns of a lane's results: group j of V neighbours starts at column
        // n0 + col(j), so that four lanes' pieces adjoin.
        constexpr int NG = 16 / V;  // groups: 4 of 4, or 2 of 8
        auto col = [&](int j) { return T == T_F32 ? 16 * j + 4 * g : 32 * j + 8 * g; };
        for (int64_t n0 = nb + wave * 64; n0 < ne; n0 += 256) {
            u32x4 bq[TMB][NG];
            const bool whole = n0 + 64 <= a.N;
            if (whole && a.base) {
#pragma unroll
                for (int m = 0; m < TMB; m++)
#pragma unroll
                    for (int j = 0; j < NG; j++)
                        if (in[m]) bq[m][j] = load16(base[m] + n0 + col(j));
            }
            v4f acc[4][TMB];
#pragma unroll
            for (int q = 0; q < 4; q++)
#pragma unroll
                for (int m = 0; m < TMB; m++) acc[q][m] = v4f{0, 0, 0, 0};
            if (has) {
                const E* wr[4];
#pragma unroll
                for (int q = 0; q < 4; q++) {
                    // Row of block q that becomes the lane's columns above.
                    const int at = T == T_F32 ? 16 * q + i : 32 * (q >> 1) + 8 * (i >> 2) + 4 * (q & 1) + (i & 3);
                    const int64_t n = n0 + at < a.N ? n0 + at : a.N - 1;
                    wr[q] = w + n * a.ldw;
                }
                const int steps = (a.R + STEP - 1) / STEP;
                for (int u = 0; u < (PACKED ? 1 : steps); u++) {
                    u32x4 wf[4];
                    const int r = PACKED ? 8 * (g & 1) : u * STEP + g * V;
#pragma unroll
                    for (int q = 0; q < 4; q++) wf[q] = load_chunk<T>(wr[q], r, a.R);
#pragma unroll
                    for (int m = 0; m < TMB; m++) {
                        const int at = (16 * m + i) * pitch;
                        if constexpr (PACKED) {
                            const u32x4 h = *reinterpret_cast<const u32x4*>((g < 2 ? hi : lo) + at + r * 2);
#pragma unroll
                            for (int q = 0; q < 4; q++) acc[q][m] = mma16<T>(wf[q], h, acc[q][m]);
                        } else {
                            const u32x4 h = *reinterpret_cast<const u32x4*>(hi + at + r * int(sizeof(E)));
#pragma unroll
                            for (int q = 0; q < 4; q++) acc[q][m] = mma16<T>(wf[q], h, acc[q][m]);
                            if constexpr (T != T_F32) {
                                const u32x4 l = *reinterpret_cast<const u32x4*>(lo + at + r * 2);
#pragma unroll
                                for (int q = 0; q < 4; q++) acc[q][m] = mma16<T>(wf[q], l, acc[q][m]);
                            }
                        }
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < TMB; m++) {
                if (!in[m]) continue;
#pragma unroll
                for (int j = 0; j < NG; j++) {
                    float d[V], b[V];
#pragma unroll
                    for (int e = 0; e < V; e++) d[e] = f[m] * acc[j * V / 4 + e / 4][m][e % 4];
                    const int64_t c = n0 + col(j);
                    if (whole) {
                        if (a.base) {
                            unpack<T>(bq[m][j], b);
#pragma unroll
                            for (int e = 0; e < V; e++) d[e] = has ? b[e] + d[e] : b[e];
                        }
                        store16(out[m] + c, pack<T>(d));
                    } else {
#pragma unroll
                        for (int e = 0; e < V; e++)
                            if (c + e < a.N) {
                                const float b1 = a.base ? float(base[m][c + e]) : 0.0f;
                                out[m][c + e] = E(!a.base ? d[e] : has ? b1 + d[e] : b1);
                            }
                    }
                }
            }
        }
    }
}

}  // namespace
}  // namespace sgemm
