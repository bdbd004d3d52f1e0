// Low-rank adapters: Y[m] = base[m] + s_l (X[m] A_l^T) B_l^T, l = ids[m].
//
// Two products, both bound by memory.  lora_shrink forms H = X A^T (long sums,
// R results a row) in float partial sums, one plane for each share of K;
// lora_expand adds the planes up and forms Y (short sums, N results a row).
// Rows come in tiles of one adapter each (RowPlan), so an adapter is read once
// for up to 64 rows.  The matrix instructions' operands are 16 bytes along K (or
// R) of one row, which is how memory holds them: they are loaded as they are, but
// for what four waves share (lora_expand_tiles' adapter, through LDS).
#pragma once
#include "lora.h"

namespace sgemm {
namespace {

// ---- H = X A^T ----------------------------------------------------------------

constexpr int kShrinkWaves = 4;

// A workgroup: a tile of 16 TMB rows, 16 RB of the R columns, a share of K split
// again over its waves, whose sums are added through LDS.  R gives few
// workgroups, so K is shared until there are about 512; the planes of sums cost
// less than idle CUs.  Bound by memory: 8192 x 4096 bfloat16 of rank 64 26 us (67 MB
// of X, 2.6 TB/s, the adapters from the caches); of rank 16 20 us (3.4 TB/s).
template <int T, int RB, int TMB>
__global__ void __launch_bounds__(64 * kShrinkWaves) __attribute__((amdgpu_waves_per_eu(TMB * RB > 8 ? 2 : 3)))
lora_shrink(ShrinkArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, STEP = 4 * V;  // K of one mma16
    __shared__ float red[2][TMB * RB * 256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int r0 = blockIdx.z * 16 * RB;
    const int64_t kb = blockIdx.y * a.kshare, ke = kb + a.kshare < a.K ? kb + a.kshare : a.K;
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
        auto step = [&](const u32x4 (&xf)[TMB], const u32x4 (&wf)[RB]) {
#pragma unroll
            for (int m = 0; m < TMB; m++)
#pragma unroll
                for (int n = 0; n < RB; n++) acc[m][n] = mma16<T>(xf[m], wf[n], acc[m][n]);
        };
        // Double steps are dealt to the waves in turn: together they read 8 STEP
        // neighbouring elements of each row.
        int64_t k = kb + wave * 2 * STEP;
        for (; k + 2 * STEP <= ke; k += kShrinkWaves * 2 * STEP) {
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
        // The wave that the last, shorter double step falls to.
        for (; k < ke; k += STEP) {
            u32x4 xf[TMB], wf[RB];
#pragma unroll
            for (int n = 0; n < RB; n++) wf[n] = load_chunk<T>(w[n], k + g * V, ke);
#pragma unroll
            for (int m = 0; m < TMB; m++) xf[m] = load_chunk<T>(x[m], k + g * V, ke);
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
            const int pitch = lora_pitch(a.R);
            float* P = a.P + blockIdx.y * a.plane + int64_t(tile.start) * pitch;
#pragma unroll
            for (int m = 0; m < TMB; m++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const int p = 16 * m + 4 * g + e;
                    if (p >= tile.count) continue;
                    float* row = P + p * pitch;
#pragma unroll
                    for (int n = 0; n < RB; n++) {
                        const int r = r0 + 16 * n + i;
                        if (r < pitch) row[r] = r >= a.R ? 0.0f : a.scaled ? acc[m][n][e] * f : acc[m][n][e];
                    }
                }
        }
    }
}

enum ExpandKind { EXPAND_PACKED, EXPAND_HELD, EXPAND_LONG };

// ---- Y = base + s H B^T -------------------------------------------------------

// LDS of a workgroup: H in the operands' form (16-bit parts, or floats) with rows
// padded by 16 bytes, and a factor for each row.
__host__ __device__ constexpr int expand_ranks(int R) { return R <= 16 ? 32 : (R + 63) / 64 * 64; }
// Parts of an element of H: of ranks up to 16 two share an instruction.
template <int T> __host__ __device__ constexpr int h_parts(bool packed) { return T == T_F32 ? 1 : packed ? 4 : 3; }
template <int T> inline size_t expand_lds(int R) {
    const int rp = expand_ranks(R);
    return 16 * size_t((T == T_F32 ? (rp + 4) * 4 : h_parts<T>(R <= 16) * (rp + 8) * 2) + 4);
}

// The largest of sixteen lanes' values.
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int d = 1; d < 16; d *= 2) v = fmaxf(v, __shfl_xor(v, d, 16));
    return v;
}
// Elements r .. r + 3 of a row of H in the operands' form, `plane` bytes between parts.
template <int T, int PARTS>
__device__ __forceinline__ void store_h(char* to, int plane, int r, v4f v, float up) {
    if constexpr (T == T_F32) {
        *reinterpret_cast<v4f*>(to + r * 4) = v;
    } else {
        uint32_t a[PARTS], b[PARTS];
        split_pair<T, PARTS>(v[0], v[1], up, up, a);
        split_pair<T, PARTS>(v[2], v[3], up, up, b);
#pragma unroll
        for (int i = 0; i < PARTS; i++) *reinterpret_cast<uint2*>(to + i * plane + r * 2) = uint2{a[i], b[i]};
    }
}

// A lane's V sums d at columns c .. of a row of N, past whose end nothing is
// stored; the loop is not unrolled, to keep this rare path small.
template <int T>
__device__ __forceinline__ void store_edge(const typename Elem<T>::type* base, typename Elem<T>::type* out, int64_t c,
                                           int64_t N, bool has, bool add, const float (&d)[kVec<T>]) {
#pragma unroll 1
    for (int e = 0; e < kVec<T> && c + e < N; e++) {
        float x = d[0];
#pragma unroll
        for (int z = 1; z < kVec<T>; z++) x = e == z ? d[z] : x;
        const float b = add ? float(base[c + e]) : 0.0f;
        out[c + e] = typename Elem<T>::type(!add ? x : has ? b + x : b);
    }
}

// Elements r .. of a row of R, zero past its end, without a branch.  ODD: R is
// no multiple of the 16 bytes' elements, which are then loaded one by one.
template <int T, bool ODD>
__device__ __forceinline__ u32x4 load_ranks(const typename Elem<T>::type* row, int r, int R) {
    u32x4 v;
    if constexpr (ODD) {
        typename Elem<T>::type e[kVec<T>];
#pragma unroll
        for (int z = 0; z < kVec<T>; z++) e[z] = row[r + z < R ? r + z : 0];
#pragma unroll
        for (int z = 0; z < kVec<T>; z++) e[z] = r + z < R ? e[z] : typename Elem<T>::type(0.0f);
        __builtin_memcpy(&v, e, 16);
    } else {
        v = load16(row + (r < R ? r : 0));
#pragma unroll
        for (int z = 0; z < 4; z++) v[z] = r < R ? v[z] : 0;
    }
    return v;
}

// A workgroup: a tile of 16 rows and a share of N, 64 columns a wave at a time.  H
// keeps its float precision on the 16-bit instructions as the sum of three parts.  One
// such instruction sums over 32: two of four parts of a rank of up to 16 (PACKED), else
// one part of 32.  Of ranks up to 64 (float: 32) the next columns' operands are fetched
// while these are multiplied (HELD); of more ranks there are too many for that (LONG).
// For tiles of few rows, bound by reading the adapters (257 rows x 8192, 32 adapters of
// rank 32, bfloat16: 15 us).  At three waves a SIMD the 16-bit HELD forms keep 4 to 6
// registers in memory (ranks that are no multiple of 8: 22), all but two of them
// outside the loop over columns.
template <int T, int KIND, bool ODD>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(T == T_F32 ? 2 : 3))) lora_expand(ExpandArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, TM = 16, STEP = 4 * V;
    // Operands of the adapter at a time.
    constexpr int HELD = KIND == EXPAND_PACKED ? 1 : 2;
    constexpr int NG = 16 / V;  // groups of V results a lane
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int rp = expand_ranks(a.R), steps = rp / STEP;
    const int pitch = T == T_F32 ? (rp + 4) * 4 : (rp + 8) * 2;  // bytes
    constexpr int PARTS = h_parts<T>(KIND == EXPAND_PACKED);
    const int plane = TM * pitch;
    float* const factor = reinterpret_cast<float*>(smem + PARTS * plane);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const uint2 block = block_of_run();
    const int64_t nb = block.y * a.nshare, ne = nb + a.nshare < a.N ? nb + a.nshare : a.N;
    // Columns of a lane's results: group j starts at column n0 + col(j), so that
    // four lanes' pieces adjoin; and the row of block q that becomes them.
    auto col = [&](int j) { return T == T_F32 ? 16 * j + 4 * g : 32 * j + 8 * g; };
    auto w_row = [&](int q) {
        return T == T_F32 ? 16 * q + i : 32 * (q >> 1) + 8 * (i >> 2) + 4 * (q & 1) + (i & 3);
    };
    for (int64_t t = block.x; t < a.tiles; t += gridDim.x) {
        const RowTile tile = row_tile(a.rows, t, TM);
        if (tile.count == 0) break;
        const bool has = tile.adapter >= 0;
        const bool in_place = a.base == a.Y;
        if (!has && in_place && !a.H) continue;
        const float s = !has || !a.scaled ? 1.0f : a.alpha * (a.scales ? a.scales[tile.adapter] : 1.0f);
        const E* const w = static_cast<const E*>(a.W) + (has ? tile.adapter : 0) * a.sw;
        const bool own = i < tile.count;
        const int64_t row = row_at(a.rows, tile.start + (own ? i : 0));
        const E* const base = static_cast<const E*>(a.base) + row * a.ldbase;
        E* const out = static_cast<E*>(a.Y) + row * a.ldy;
        // What 64 columns take from memory, fetched one turn ahead.
        struct Turn {
            u32x4 b[NG], w[HELD][4];
        };
        auto load_w = [&](int64_t n0, int u, Turn& v) {
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int64_t n = n0 + w_row(q) < a.N ? n0 + w_row(q) : a.N - 1;
#pragma unroll
                for (int h = 0; h < HELD; h++) {
                    const int r = KIND == EXPAND_PACKED ? 8 * (g & 1) : (u + h) * STEP + g * V;
                    v.w[h][q] = load_ranks<T, ODD>(w + n * a.ldw, r, a.R);
                }
            }
        };
        auto fetch = [&](int64_t n0, Turn& v) {
            if (n0 >= ne) return;
            if (n0 + 64 <= a.N && a.base) {
#pragma unroll
                for (int j = 0; j < NG; j++) v.b[j] = load16(base + n0 + col(j));
            }
            if (has && KIND != EXPAND_LONG) load_w(n0, 0, v);
        };
        Turn cur;
        fetch(nb + wave * 64, cur);
        __syncthreads();
        // Sixteen lanes a row, four neighbours of each 64 columns a lane; the loads
        // of the planes in flight together.
        const int c = threadIdx.x & 15, p = threadIdx.x >> 4, hp = lora_pitch(a.R);
        const bool in = p < tile.count;
        // Rows past the tile's repeat its first.
        const float* const P = a.P + (int64_t(tile.start) + (in ? p : 0)) * hp;
        float top = 0.0f;
        for (int pass = 0; pass < (T == T_F16 && rp > 64 ? 2 : 1); pass++) {
            for (int q0 = 0; q0 < rp; q0 += 64) {
                const int rq = q0 + 4 * c;
                v4f v = {0, 0, 0, 0};
                if (has && rq < hp) {
                    constexpr int AT_ONCE = 8;
                    int z = 0;
                    for (; z + AT_ONCE <= a.planes; z += AT_ONCE) {
                        v4f q[AT_ONCE];
#pragma unroll
                        for (int y = 0; y < AT_ONCE; y++) q[y] = *reinterpret_cast<const v4f*>(P + (z + y) * a.plane + rq);
#pragma unroll
                        for (int y = 0; y < AT_ONCE; y++) v += q[y];
                    }
                    for (; z < a.planes; z++) v += *reinterpret_cast<const v4f*>(P + z * a.plane + rq);
                }
                if (!in) v = v4f{0, 0, 0, 0};
                float up = 1.0f;
                if constexpr (T == T_F16) {
                    // The power that brings the row's largest finite element into [2^14, 2^15).
                    if (pass == 0) {
#pragma unroll
                        for (int e = 0; e < 4; e++) top = largest(top, v[e]);
                        if (rp > 64) continue;
                    }
                    // Every lane of the row's sixteen is here.
                    up = half_factor(group_max(top));
                }
                if (rq < rp) store_h<T, PARTS>(smem + p * pitch, plane, rq, v, up);
                if (a.H && block.y == 0 && in) {
                    float* const h = a.H + row_at(a.rows, tile.start + p) * a.ldh;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        if (rq + e < a.R) h[rq + e] = v[e];
                }
            }
        }
        if constexpr (T == T_F16) {
            const float up = half_factor(group_max(top));
            if (c == 0) factor[p] = undone(s, up);
        } else {
            if (c == 0) factor[p] = s;
        }
        __syncthreads();
        const float f = factor[i];
        for (int64_t n0 = nb + wave * 64; n0 < ne; n0 += 256) {
            Turn next;
            fetch(n0 + 256, next);
            const bool whole = n0 + 64 <= a.N;
            v4f acc[4];
#pragma unroll
            for (int q = 0; q < 4; q++) acc[q] = v4f{0, 0, 0, 0};
            if (has) {
                const int at = i * pitch;
                for (int u = 0; u < (KIND == EXPAND_LONG ? steps : 1); u += HELD) {
                    if constexpr (KIND == EXPAND_LONG) load_w(n0, u, cur);
#pragma unroll
                    for (int h = 0; h < HELD; h++) {
                        const int r = KIND == EXPAND_PACKED ? 8 * (g & 1) : (u + h) * STEP + g * V;
                        // PACKED: lanes of the sum's second half have the next part.
                        constexpr int STRIDE = KIND == EXPAND_PACKED ? 2 : 1;
                        const char* const from = smem + at + r * int(sizeof(E)) + (KIND == EXPAND_PACKED && g >= 2 ? plane : 0);
#pragma unroll
                        for (int i = 0; i < PARTS; i += STRIDE) {
                            const u32x4 x = *reinterpret_cast<const u32x4*>(from + i * plane);
#pragma unroll
                            for (int q = 0; q < 4; q++) acc[q] = mma16<T>(cur.w[h][q], x, acc[q]);
                        }
                    }
                }
            }
            if (own)
#pragma unroll
                for (int j = 0; j < NG; j++) {
                    float d[V], b[V];
#pragma unroll
                    for (int e = 0; e < V; e++) d[e] = f * acc[j * V / 4 + e / 4][e % 4];
                    const int64_t c = n0 + col(j);
                    if (whole) {
                        if (a.base) {
                            unpack<T>(cur.b[j], b);
#pragma unroll
                            for (int e = 0; e < V; e++) d[e] = has ? b[e] + d[e] : b[e];
                        }
                        store16(out + c, pack<T>(d));
                    } else {
                        store_edge<T>(base, out, c, a.N, has, a.base != nullptr, d);
                    }
                }
            cur = next;
        }
    }
}

// The same for tiles of many rows: a workgroup takes 64 rows and a share of N,
// each wave 16 of the rows, with their H in registers (in parts, as above)
// for the whole of it.  64 columns of the adapter are staged in LDS for the four
// waves, up to 64 ranks at a time, while the ones before are multiplied: read
// from memory by each wave for itself (into registers), they passed through the L1
// four times and took as long as base and Y (8192 x 8192 bfloat16 of rank 64: 97 us,
// staged 80).  A share's workgroups are on as few XCDs as can be, whose L2s then keep
// that share of the adapters (77 to 82 us, 3.3 to 3.5 TB/s of base and Y; of rank 16 8192 x 4096
// 38 -> 35).  Waves wait for base most of the time; two turns of it are in flight
// (four, or the adapter's two turns ahead, are slower).
// NS: matrix instructions' sums of one part that R takes.  Ranks up to 64 of 16-bit
// types have three waves a SIMD: for four, 20 registers go to memory (4096 x 4096 of
// rank 64 27 us, 24 with three; 8192 x 8192 the same).
template <int T, int KIND, int NS, bool ODD>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(T == T_F32 ? (NS <= 2 ? 3 : NS <= 8 ? 2 : 1) : (NS <= 1 ? 4 : NS <= 2 ? 3 : NS <= 4 ? 2 : 1))))
lora_expand_tiles(ExpandArgs a) {
    using E = typename Elem<T>::type;
    constexpr bool PACKED = KIND == EXPAND_PACKED;
    constexpr int V = kVec<T>, STEP = 4 * V, NG = 16 / V;
    constexpr int CHUNK = PACKED ? 1 : NS < 64 / STEP ? NS : 64 / STEP;  // sums staged at a time
    constexpr int ROW = PACKED ? 16 : CHUNK * STEP;                      // ranks of those
    constexpr int PITCH = ROW * int(sizeof(E)) + 16;                     // bytes of a staged row
    constexpr int PIECES = ROW / V * 64 / 256 > 0 ? ROW / V * 64 / 256 : 1;
    constexpr int CHUNKS = PACKED ? 1 : NS / CHUNK;
    constexpr int AHEAD = 2;
    __shared__ __attribute__((aligned(16))) char stage[2][64 * PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const uint2 block = block_of_run();
    const int64_t nb = block.y * a.nshare, ne = nb + a.nshare < a.N ? nb + a.nshare : a.N;
    auto col = [&](int j) { return T == T_F32 ? 16 * j + 4 * g : 32 * j + 8 * g; };
    auto w_row = [&](int q) {
        return T == T_F32 ? 16 * q + i : 32 * (q >> 1) + 8 * (i >> 2) + 4 * (q & 1) + (i & 3);
    };
    for (int64_t t = block.x; t < a.tiles; t += gridDim.x) {
        const RowTile tile = row_tile(a.rows, t, 64);
        if (tile.count == 0) break;
        const bool has = tile.adapter >= 0;
        if (!has && a.base == a.Y && !a.H) continue;
        const float s = !has || !a.scaled ? 1.0f : a.alpha * (a.scales ? a.scales[tile.adapter] : 1.0f);
        const E* const w = static_cast<const E*>(a.W) + (has ? tile.adapter : 0) * a.sw;
        const int p = 16 * wave + i;
        const bool own = p < tile.count;
        const int64_t row = row_at(a.rows, tile.start + (own ? p : 0));
        const E* const base = static_cast<const E*>(a.base) + row * a.ldbase;
        E* const out = static_cast<E*>(a.Y) + row * a.ldy;
        const int turns = int((ne - nb + 63) / 64);
        // Sixteen bytes of the adapter's columns n0 .., chunk ch, for LDS; past R they
        // are zeroed only when they are put there, as that waits for them.
        u32x4 piece[PIECES];
        auto fetch_w = [&](int64_t n0, int ch) {
#pragma unroll
            for (int q = 0; q < PIECES; q++) {
                const int e = threadIdx.x + 256 * q, n = e / (ROW / V) & 63, r = ch * ROW + e % (ROW / V) * V;
                const int64_t at = n0 + n < a.N ? n0 + n : a.N - 1;
                if constexpr (ODD) piece[q] = load_ranks<T, true>(w + at * a.ldw, r, a.R);
                else piece[q] = load16(w + at * a.ldw + (r < a.R ? r : 0));
            }
        };
        auto put_w = [&](char* to, int ch) {
#pragma unroll
            for (int q = 0; q < PIECES; q++) {
                const int e = threadIdx.x + 256 * q, n = e / (ROW / V), c = e % (ROW / V);
                u32x4 v = piece[q];
#pragma unroll
                for (int z = 0; z < 4; z++) v[z] = ODD || ch * ROW + c * V < a.R ? v[z] : 0;
                if (64 * (ROW / V) >= 256 || n < 64) *reinterpret_cast<u32x4*>(to + n * PITCH + 16 * c) = v;
            }
        };
        // base, AHEAD turns of 64 columns in flight.  Where there is less to fetch the
        // last columns are fetched again: a wait can then be for all but so many loads.
        const bool wide = a.base != nullptr && a.N >= 64;
        u32x4 b[AHEAD][NG];
        auto fetch_base = [&](int turn, int slot) {
            const int64_t n0 = nb + 64 * int64_t(turn);
            const E* const from = base + (n0 + 64 <= a.N ? n0 : a.N - 64);
#pragma unroll
            for (int j = 0; j < NG; j++) b[slot][j] = load16(from + col(j));
        };
        if (has && turns > 0) fetch_w(nb, 0);
        if (wide && turns > 0)
#pragma unroll
            for (int slot = 0; slot < AHEAD; slot++) fetch_base(slot, slot);
        // H: the lane's V ranks of each sum, all planes.
        const int hp = lora_pitch(a.R);
        constexpr int PARTS = h_parts<T>(PACKED), HELD = PACKED ? 2 : PARTS;
        u32x4 held[NS][HELD];
        float f = s;
        {
            const float* const P = a.P + int64_t(tile.start + (own ? p : 0)) * hp;
            float v[NS][V];
#pragma unroll
            for (int u = 0; u < NS; u++) {
#pragma unroll
                for (int e = 0; e < V; e++) v[u][e] = 0.0f;
            }
            if (has)
                for (int z = 0; z < a.planes; z++) {
                    v4f x[NS][V / 4];
#pragma unroll
                    for (int u = 0; u < NS; u++) {
                        const int r = PACKED ? 8 * (g & 1) : u * STEP + g * V;
#pragma unroll
                        for (int e = 0; e < V; e += 4)
                            x[u][e / 4] = *reinterpret_cast<const v4f*>(P + z * a.plane + (r + e < hp ? r + e : 0));
                    }
#pragma unroll
                    for (int u = 0; u < NS; u++)
#pragma unroll
                        for (int e = 0; e < V; e++) v[u][e] += x[u][e / 4][e % 4];
                }
#pragma unroll
            for (int u = 0; u < NS; u++) {
                const int r = PACKED ? 8 * (g & 1) : u * STEP + g * V;
#pragma unroll
                for (int e = 0; e < V; e++)
                    if (!own || r + e >= a.R) v[u][e] = 0.0f;
                if (a.H && block.y == 0 && own && (!PACKED || g < 2))
#pragma unroll
                    for (int e = 0; e < V; e++)
                        if (r + e < a.R) a.H[row * a.ldh + r + e] = v[u][e];
            }
            float up = 1.0f;
            if constexpr (T == T_F16) {
                float top = 0.0f;
#pragma unroll
                for (int u = 0; u < NS; u++)
#pragma unroll
                    for (int e = 0; e < V; e++)
                        top = largest(top, v[u][e]);
                top = fmaxf(top, __shfl_xor(top, 16));
                up = half_factor(fmaxf(top, __shfl_xor(top, 32)));
                f = undone(s, up);
            }
#pragma unroll
            for (int u = 0; u < NS; u++) {
                if constexpr (T == T_F32) {
                    held[u][0] = pack<T>(v[u]);
                } else {
#pragma unroll
                    for (int y = 0; y < 4; y++) {
                        uint32_t p[PARTS];
                        split_pair<T, PARTS>(v[u][2 * y], v[u][2 * y + 1], up, up, p);
#pragma unroll
                        for (int i = 0; i < HELD; i++) {
                            const uint32_t one = p[PACKED ? 2 * i : i], two = p[PACKED ? 2 * i + 1 : i];
                            held[u][i][y] = g < 2 ? one : two;
                        }
                    }
                }
            }
        }
        int half = 0;
        __syncthreads();  // the tile before is done with LDS
        // One turn's sums, for the lane's row.
        auto multiply = [&](int64_t n0, v4f (&acc)[4]) {
#pragma unroll
            for (int q = 0; q < 4; q++) acc[q] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int ch = 0; ch < CHUNKS; ch++) {
                char* const st = stage[half];
                half ^= 1;
                put_w(st, ch);
                __syncthreads();
                if (ch + 1 < CHUNKS) fetch_w(n0, ch + 1);
                else fetch_w(n0 + 64, 0);
#pragma unroll
                for (int u = 0; u < CHUNK; u++) {
                    const int c = PACKED ? 16 * (g & 1) : (u * 4 + g) * 16;
#pragma unroll
                    for (int q = 0; q < 4; q++) {
                        const u32x4 x = *reinterpret_cast<const u32x4*>(st + w_row(q) * PITCH + c);
#pragma unroll
                        for (int i = 0; i < HELD; i++) acc[q] = mma16<T>(x, held[ch * CHUNK + u][i], acc[q]);
                    }
                }
            }
        };
        const int full = int(((ne < a.N ? ne : a.N) - nb) / 64);  // turns of whole 64 columns
        auto columns = [&](auto with_h, auto with_base) {
            constexpr bool HAS = decltype(with_h)::value, WIDE = decltype(with_base)::value;
            for (int turn4 = 0; turn4 < full; turn4 += AHEAD)
#pragma unroll
                for (int slot = 0; slot < AHEAD; slot++) {
                    const int turn = turn4 + slot;
                    if (turn >= full) break;
                    const int64_t n0 = nb + 64 * int64_t(turn);
                    v4f acc[4];
                    if constexpr (HAS) multiply(n0, acc);
                    u32x4 y[NG];
#pragma unroll
                    for (int j = 0; j < NG; j++) {
                        float d[V], x[V];
#pragma unroll
                        for (int e = 0; e < V; e++) d[e] = HAS ? f * acc[j * V / 4 + e / 4][e % 4] : 0.0f;
                        if constexpr (WIDE) {
                            unpack<T>(b[slot][j], x);
#pragma unroll
                            for (int e = 0; e < V; e++) d[e] = HAS ? x[e] + d[e] : x[e];
                        }
                        y[j] = pack<T>(d);
                    }
                    // Before the stores: the wait for these then does not wait for those.
                    if constexpr (WIDE) fetch_base(turn + AHEAD, slot);
                    asm volatile("" ::: "memory");
                    if (own)
#pragma unroll
                        for (int j = 0; j < NG; j++) store16(out + n0 + col(j), y[j]);
                }
        };
        if (has && wide) columns(std::true_type{}, std::true_type{});
        else if (has) columns(std::true_type{}, std::false_type{});
        else if (wide) columns(std::false_type{}, std::true_type{});
        else columns(std::false_type{}, std::false_type{});
        if (full < turns) {  // columns up to N
            const int64_t n0 = nb + 64 * int64_t(full);
            v4f acc[4] = {};
            if (has) multiply(n0, acc);
            if (own)
#pragma unroll
                for (int j = 0; j < NG; j++)
#pragma unroll
                    for (int e = 0; e < V; e++) {
                        const int64_t c = n0 + col(j) + e;
                        if (c >= a.N) continue;
                        const float d = f * acc[j * V / 4 + e / 4][e % 4];
                        out[c] = E(!a.base ? (has ? d : 0.0f) : has ? float(base[c]) + d : float(base[c]));
                    }
        }
    }
}

// Y of single rows, each with an adapter of its own: G neighbouring lanes share a
// column's sum, so that a wave reads the adapter in one piece, and H is in LDS in
// float.  On the vector units: with one row the matrix instructions' other fifteen
// would be empty, and what counts is how soon the loads are out (64 rows x 8192 of
// rank 16: 5.9 us, lora_expand 9.1).
constexpr int kOneCols = 4;  // columns of a lane group in flight

template <int T, int G, bool ODD>
__global__ void __launch_bounds__(256) lora_expand_one(ExpandArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, COLS = 256 / G;  // columns of a workgroup at a time
    __shared__ __attribute__((aligned(16))) float h[256 + 16];
    const int lane = threadIdx.x % G, at = threadIdx.x / G;
    const int64_t m = blockIdx.x;
    const int64_t nb = blockIdx.y * a.nshare, ne = nb + a.nshare < a.N ? nb + a.nshare : a.N;
    const int l = __builtin_amdgcn_readfirstlane(adapter_of(a.rows.ids, a.rows.id64, a.rows.L, m));
    const bool has = l >= 0;
    if (!has && a.base == a.Y && !a.H) return;
    const float s = has ? a.alpha * (a.scales ? a.scales[l] : 1.0f) : 0.0f;
    const E* const w = static_cast<const E*>(a.W) + (has ? l : 0) * a.sw;
    const E* const base = static_cast<const E*>(a.base) + m * a.ldbase;
    E* const out = static_cast<E*>(a.Y) + m * a.ldy;
    // The first columns' pieces, before H is known.
    u32x4 first[kOneCols];
    float b[kOneCols];
    auto fetch = [&](int64_t n0) {
#pragma unroll
        for (int q = 0; q < kOneCols; q++) {
            const int64_t n = n0 + q * COLS + at < a.N ? n0 + q * COLS + at : a.N - 1;
            if (has) first[q] = load_ranks<T, ODD>(w + n * a.ldw, lane * V, a.R);
            b[q] = a.base ? float(base[n]) : 0.0f;
        }
    };
    if (nb < ne) fetch(nb);
    const int hp = lora_pitch(a.R);
    for (int r = threadIdx.x; r < hp; r += 256) {
        float v = 0.0f;
        if (has) {
            const float* const p = a.P + m * hp + r;
            float q[8];
#pragma unroll
            for (int z = 0; z < 8; z++) q[z] = p[(z < a.planes ? z : 0) * a.plane];
#pragma unroll
            for (int z = 0; z < 8; z++) v += z < a.planes ? q[z] : 0.0f;
        }
        h[r] = r < a.R ? v : 0.0f;
        if (a.H && blockIdx.y == 0 && r < a.R) a.H[m * a.ldh + r] = v;
    }
    __syncthreads();
    for (int64_t n0 = nb; n0 < ne; n0 += kOneCols * COLS) {
        float v[kOneCols] = {};
        if (has)
            for (int r = lane * V; r < a.R; r += G * V) {
                float x[V];
#pragma unroll
                for (int e = 0; e < V; e += 4) {
                    const v4f y = *reinterpret_cast<const v4f*>(&h[r + e]);
                    x[e] = y[0], x[e + 1] = y[1], x[e + 2] = y[2], x[e + 3] = y[3];
                }
#pragma unroll
                for (int q = 0; q < kOneCols; q++) {
                    const int64_t n = n0 + q * COLS + at < a.N ? n0 + q * COLS + at : a.N - 1;
                    float f[V];
                    unpack<T>(r == lane * V ? first[q] : load_ranks<T, ODD>(w + n * a.ldw, r, a.R), f);
                    // A zero of H past R may meet no more than a zero.
#pragma unroll
                    for (int e = 0; e < V; e++) v[q] = fmaf(x[e], f[e], v[q]);
                }
            }
#pragma unroll
        for (int q = 0; q < kOneCols; q++) {
#pragma unroll
            for (int d = 1; d < G; d *= 2) v[q] += __shfl_xor(v[q], d);
            const int64_t n = n0 + q * COLS + at;
            if (lane == 0 && n < ne) out[n] = E(!has ? b[q] : a.base ? b[q] + s * v[q] : s * v[q]);
        }
        if (n0 + kOneCols * COLS < ne) fetch(n0 + kOneCols * COLS);
    }
}

// ---- few rows ------------------------------------------------------------------

// A row's Y, 512 columns a workgroup, in one launch: every workgroup forms the row's
// H for itself (its eight waves share K), then a lane a column its sum of R terms, in
// float.  The adapter's A is so read once for each 512 columns, by one CU at about
// 25 GB/s: worth it where both are small (see few_rows).
constexpr int kFewCols = 512;

template <int T, bool ODD>
__global__ void __launch_bounds__(512) lora_few(LoraArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, STEP = 4 * V, KEPT = T == T_F32 ? 16 : 32;  // ranks fetched ahead
    __shared__ float part[8][64], h[256];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int64_t m = blockIdx.y, n = int64_t(blockIdx.x) * kFewCols + threadIdx.x;
    const int l = __builtin_amdgcn_readfirstlane(a.ids ? adapter_of(a.ids, a.id64, a.L, m) : 0);
    const bool has = l >= 0, in = n < a.N;
    const float b = in && a.base ? float(static_cast<const E*>(a.base)[m * a.ldbase + n]) : 0.0f;
    if (has) {
        const E* const w = static_cast<const E*>(a.B) + l * a.sb + (in ? n : a.N - 1) * a.ldb;
        u32x4 kept[KEPT / V];
        if (a.N > 0)
#pragma unroll
            for (int q = 0; q < KEPT / V; q++) kept[q] = load_ranks<T, ODD>(w, q * V, a.R);
        const E* const x = static_cast<const E*>(a.X) + m * a.ldx;
        for (int r0 = 0; r0 < a.R; r0 += 64) {
            const E* wr[4];
            v4f acc[4];
#pragma unroll
            for (int q = 0; q < 4; q++) {
                const int r = r0 + 16 * q + i;
                wr[q] = static_cast<const E*>(a.A) + l * a.sa + int64_t(r < a.R ? r : a.R - 1) * a.lda;
                acc[q] = v4f{0, 0, 0, 0};
            }
            const int blocks = (a.R - r0 + 15) / 16;
            // Rows 1 .. 15 of the products' left operand repeat row 0; its results count.
            int64_t k = wave * STEP;
            for (; k + STEP <= a.K; k += 8 * STEP) {
                const u32x4 xf = load16(x + k + g * V);
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (q < blocks) acc[q] = mma16<T>(xf, load16(wr[q] + k + g * V), acc[q]);
            }
            if (k < a.K) {
                const u32x4 xf = load_chunk<T>(x, k + g * V, a.K);
#pragma unroll
                for (int q = 0; q < 4; q++)
                    if (q < blocks) acc[q] = mma16<T>(xf, load_chunk<T>(wr[q], k + g * V, a.K), acc[q]);
            }
            if (g == 0)
#pragma unroll
                for (int q = 0; q < 4; q++) part[wave][16 * q + i] = acc[q][0];
            __syncthreads();
            if (threadIdx.x < 64) {
                float v = 0.0f;
#pragma unroll
                for (int q = 0; q < 8; q++) v += part[q][threadIdx.x];
                if (r0 + int(threadIdx.x) < 256) h[r0 + threadIdx.x] = r0 + int(threadIdx.x) < a.R ? v : 0.0f;
            }
            __syncthreads();
        }
        float v = 0.0f;
        auto add = [&](u32x4 q, int r) {
            float f[V];
            unpack<T>(q, f);
#pragma unroll
            for (int e = 0; e < V; e++) v = r + e < a.R ? fmaf(h[r + e], f[e], v) : v;
        };
        if (a.N > 0) {
#pragma unroll
            for (int q = 0; q < KEPT / V; q++) add(kept[q], q * V);
            for (int r = KEPT; r < a.R; r += V) add(load_ranks<T, ODD>(w, r, a.R), r);
        }
        const float s = a.alpha * (a.scales ? a.scales[l] : 1.0f);
        if (in) static_cast<E*>(a.Y)[m * a.ldy + n] = E(a.base ? b + s * v : s * v);
    } else if (in) {
        static_cast<E*>(a.Y)[m * a.ldy + n] = E(b);
    }
    if (a.H && blockIdx.x == 0)
        for (int r = threadIdx.x; r < a.R; r += 512) a.H[m * a.ldh + r] = has ? h[r] : 0.0f;
}

}  // namespace
}  // namespace sgemm
