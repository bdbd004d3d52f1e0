// Orthogonalised updates by Newton-Schulz products: X = G / (|G| + eps), then
// X <- P X with P = a I + b S + c S^2, S = X X^T, for each step.
//
// Arithmetic.  The values between the products are bounded by numbers that the
// coefficients alone give, so each is kept as two float16 parts of 11 bits
// times a power of two: v = hi + lo to 2^-22 of itself (2^-39 of the bound where
// it is small against that).  A product is then three matrix instructions of
// float16, hi hi + hi lo + lo hi with float sums, at 16 / 3 of the rate of the
// float instruction; what is left out, lo lo, is 2^-22 of a term.
//
// Layout.  m <= n is the smaller side; a tall G is taken as its transpose.  Both
// operands of a product are read along the sum, so S needs X by rows (m x n),
// P X needs X^T by rows (n x m), and the kernel that forms X stores both.  S and
// P are symmetric: only tiles on and below the diagonal are computed, and each is
// stored twice.  Rows are padded with zeros to whole steps of the sum, and there
// is room for a tile's overhang of rows, whose values reach no other row.  A row
// holds 32 high parts, their 32 low parts, the next 32 ...:
// 128 bytes are a row's share of one step of the sum.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "orthogonalize.h"

namespace sgemm {
namespace {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

constexpr int kStep = 32;  // of the sum, at a time

__device__ __forceinline__ float load_as(int type, const void* p, int64_t i) {
    if (type == T_F32) return static_cast<const float*>(p)[i];
    if (type == T_F16) return float(static_cast<const _Float16*>(p)[i]);
    return float(static_cast<const __bf16*>(p)[i]);
}
__device__ __forceinline__ void store_as(int type, void* p, int64_t i, float v) {
    if (type == T_F32) static_cast<float*>(p)[i] = v;
    else if (type == T_F16) static_cast<_Float16*>(p)[i] = _Float16(v);
    else static_cast<__bf16*>(p)[i] = __bf16(v);
}

// Where the high part of column k is in a row; its low part is 32 further.
__host__ __device__ constexpr int64_t part_at(int64_t k) { return k / 32 * 64 + k % 32; }

__device__ __forceinline__ void split(float v, _Float16& hi, _Float16& lo) {
    hi = _Float16(v);
    lo = _Float16(v - float(hi));
}

// ---- the norm and the first X ---------------------------------------------------

constexpr int kNormBlocks = 512;  // partial sums of a matrix

// Partial sums of squares in double, block x of matrix y; 16 bytes a lane at a
// time, four in flight, where the matrix has no gaps (4096 x 4096 float: 14 us,
// 4.8 TB/s, a copy's rate).
template <int TYPE>
__global__ void __launch_bounds__(256) ortho_squares(const void* G, int64_t M, int64_t N, int64_t ldg, int64_t sg,
                                                     double* out) {
    constexpr int V = TYPE == T_F32 ? 4 : 8, SIZE = TYPE == T_F32 ? 4 : 2;
    __shared__ double part[4];
    double v = 0;
    const char* const g = static_cast<const char*>(G) + int64_t(blockIdx.y) * sg * SIZE;
    if (ldg == N) {
        const int64_t n = M * N, whole = n / V, stride = int64_t(gridDim.x) * 256;
        auto add = [&](int64_t t) {
            float x[V];
            char raw[16];
            __builtin_memcpy(raw, g + t * 16, 16);
#pragma unroll
            for (int e = 0; e < V; e++) x[e] = load_as(TYPE, raw, e);
#pragma unroll
            for (int e = 0; e < V; e++) v += double(x[e]) * double(x[e]);
        };
        int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x;
        for (; t + 3 * stride < whole; t += 4 * stride) {
#pragma unroll
            for (int u = 0; u < 4; u++) add(t + u * stride);
        }
        for (; t < whole; t += stride) add(t);
        if (blockIdx.x == 0 && threadIdx.x < n - whole * V) {
            const double x = load_as(TYPE, g, whole * V + threadIdx.x);
            v += x * x;
        }
    } else {
        for (int64_t r = blockIdx.x; r < M; r += gridDim.x)
            for (int64_t c = threadIdx.x; c < N; c += 256) {
                const double x = load_as(TYPE, g, r * ldg + c);
                v += x * x;
            }
    }
    for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) out[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and X^T in parts, times `scale`, from G: a 64 x 64 tile of X (m x n) a
// workgroup, turned in LDS.  Rows have kn and km columns.  Bound by memory (4096 x
// 4096 float: 201 MB in 37 us, 5.4 TB/s).
template <int TYPE>
__global__ void __launch_bounds__(256) ortho_split(const void* G, bool tall, int64_t m, int64_t n, int64_t ldg,
                                                   int64_t sg, const double* squares, int parts, double eps,
                                                   float scale, _Float16* X, _Float16* Xt, int64_t km, int64_t kn,
                                                   int64_t sx, int64_t st) {
    __shared__ float tile[64][65];
    __shared__ double total;
    const int64_t b = blockIdx.z;
    if (threadIdx.x < 64) {
        double v = 0;
        for (int i = threadIdx.x; i < parts; i += 64) v += squares[b * parts + i];
        for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
        if (threadIdx.x == 0) total = v;
    }
    const int64_t r0 = int64_t(blockIdx.y) * 64, c0 = int64_t(blockIdx.x) * 64;  // of X
    __syncthreads();
    const double f = double(scale) / (sqrt(total) + eps);
    X += b * sx;
    Xt += b * st;
    // Rows of G as they lie: X's rows, or its columns; the loads first.
    float v[16];
#pragma unroll
    for (int u = 0; u < 16; u++) {
        const int y = u * 4 + int(threadIdx.x) / 64, x = threadIdx.x % 64;
        const int64_t r = tall ? r0 + x : r0 + y, c = tall ? c0 + y : c0 + x;
        const bool in = r < m && c < n;
        v[u] = load_as(TYPE, G, b * sg + (in ? (tall ? c * ldg + r : r * ldg + c) : 0));
        if (!in) v[u] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < 16; u++) {
        const int y = u * 4 + int(threadIdx.x) / 64, x = threadIdx.x % 64;
        const float w = v[u] == 0 ? 0.0f : float(double(v[u]) * f);  // zeros stay so whatever f
        if (tall) tile[x][y] = w;
        else tile[y][x] = w;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 512; e += 256) {
        const int y = e / 8, x = e % 8 * 8;
        f16x8 h, l;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            _Float16 a, c;
            split(tile[y][x + i], a, c);
            h[i] = a, l[i] = c;
        }
        if (c0 + x < kn) {
            _Float16* at = X + (r0 + y) * kn * 2 + part_at(c0 + x);
            *reinterpret_cast<f16x8*>(at) = h;
            *reinterpret_cast<f16x8*>(at + 32) = l;
        }
#pragma unroll
        for (int i = 0; i < 8; i++) {
            _Float16 a, c;
            split(tile[x + i][y], a, c);
            h[i] = a, l[i] = c;
        }
        if (r0 + x < km) {
            _Float16* at = Xt + (c0 + y) * km * 2 + part_at(r0 + x);
            *reinterpret_cast<f16x8*>(at) = h;
            *reinterpret_cast<f16x8*>(at + 32) = l;
        }
    }
}

// ---- the products -----------------------------------------------------------------

enum Epilogue { GRAM, POLY, APPLY, LAST };

struct ProductArgs {
    const _Float16 *A, *B;      // C = A B^T: rows of K sums in parts
    int64_t K;                  // a multiple of 32
    int64_t stride_a, stride_b; // between matrices, in float16
    int tiles_m, tiles_n;
    int share;                  // steps of a workgroup (grid.y of them)
    float* partial;             // their sums, where there is more than one
    float scale;                // of the sums
    // GRAM, POLY: S or P, twice.  APPLY: X and X^T.  Rows of ldn and ldt columns;
    // those from rows and cols on are zero.
    _Float16 *N, *T;
    int64_t ldn, ldt, stride_n, stride_t;  // in columns, and in float16
    int64_t rows, cols;
    // POLY: out = scale sum + b S + diagonal, S the operand.
    float b, diagonal;
    // LAST: out in `type`.
    int type;
    bool tall;
    void* out;
    int64_t ldo, stride_o;
};

// Tile t of those on and below the diagonal: bands of four rows, within a band
// column by column, so that tiles that run at a time share operands.
__device__ __forceinline__ void triangle(int t, int tiles, int& i, int& j) {
    int band = 0;
    for (;; band++) {
        const int r0 = 4 * band, h = tiles - r0 < 4 ? tiles - r0 : 4;
        const int count = h * r0 + h * (h + 1) / 2;
        if (t < count) {
            if (t < h * (r0 + 1)) {
                i = r0 + t % h, j = t / h;
                return;
            }
            t -= h * (r0 + 1);
            j = r0 + 1;
            for (int left = h - 1; t >= left; left--) t -= left, j++;
            i = j + t;
            return;
        }
        t -= count;
    }
}

template <int EPI>
__device__ __forceinline__ void tile_of(const ProductArgs& a, int t, int& ti, int& tj) {
    if constexpr (EPI == GRAM || EPI == POLY) {
        triangle(t, a.tiles_m, ti, tj);
    } else {
        // Groups of eight tile rows, column by column.
        const int per = 8 * a.tiles_n, first = t / per * 8, h = a.tiles_m - first < 8 ? a.tiles_m - first : 8;
        ti = first + t % per % h;
        tj = t % per / h;
    }
}

// Stored results.  Eight neighbours of row r (columns c ..), four of column c
// (rows r .., in the transposed copy's row c), and of LAST one.
__device__ __forceinline__ void store_row(const ProductArgs& a, int64_t z, int64_t r, int64_t c, const float (&v)[8]) {
    if (c >= a.ldn) return;
    f16x8 h, l;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        _Float16 p, o;
        split(c + i < a.cols ? v[i] : 0.0f, p, o);
        h[i] = p, l[i] = o;
    }
    _Float16* at = a.N + z * a.stride_n + r * a.ldn * 2 + part_at(c);
    *reinterpret_cast<f16x8*>(at) = h;
    *reinterpret_cast<f16x8*>(at + 32) = l;
}
__device__ __forceinline__ void store_column(const ProductArgs& a, int64_t z, int64_t r, int64_t c, const float (&v)[4]) {
    if (r >= a.ldt) return;
    f16x4 h, l;
#pragma unroll
    for (int i = 0; i < 4; i++) {
        _Float16 p, o;
        split(r + i < a.rows ? v[i] : 0.0f, p, o);
        h[i] = p, l[i] = o;
    }
    _Float16* at = a.T + z * a.stride_t + c * a.ldt * 2 + part_at(r);
    *reinterpret_cast<f16x4*>(at) = h;
    *reinterpret_cast<f16x4*>(at + 32) = l;
}
__device__ __forceinline__ void store_out(const ProductArgs& a, int64_t z, int64_t r, int64_t c, float v) {
    if (r < a.rows && c < a.cols) store_as(a.type, a.out, z * a.stride_o + (a.tall ? c * a.ldo + r : r * a.ldo + c), v);
}

// Tile configurations: WM x WN waves of MBM x MBN accumulators of 32 x 32, and LDS
// stages of 32 of the sum.
template <int WM_, int WN_, int MBM_, int MBN_, int STAGES_, int OCC_>
struct Tile {
    static constexpr int WM = WM_, WN = WN_, MBM = MBM_, MBN = MBN_, STAGES = STAGES_, OCC = OCC_;
    static constexpr int WAVES = WM * WN, SIDE = 32 * MBM * WM;
    static_assert(SIDE == 32 * MBN * WN, "square tiles");
    static constexpr int BYTES = SIDE * 128;  // of one operand's stage
};
using Tile64 = Tile<2, 2, 1, 1, 4, 2>;
using Tile128 = Tile<2, 4, 2, 1, 4, 2>;
using Tile192 = Tile<2, 2, 3, 3, 3, 1>;
using Tile256 = Tile<2, 4, 4, 2, 2, 2>;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const char* base) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), (short)0, int(0x80000000u), 0x00020000);
}

// One buffer load that writes LDS directly: lane L's bytes go to lds + BYTES L.  (A
// template, as the host pass does not know the builtin.)
template <int BYTES>
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t r, char* lds, unsigned off, int at) {
    static_assert(BYTES == 16, "the one width used");
    if constexpr (BYTES == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(lds), 16, off, at, 0, 0);
}

// Every load of this wave but the latest N has landed and its LDS reads are done,
// then the same of every wave.  (__syncthreads would wait for all loads.)
template <int N>
__device__ __forceinline__ void step_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// A workgroup: one tile.  Steps of 32 of the sum go through the LDS stages, written
// by loads that bypass the registers, STAGES - 1 ahead; a row's eight 16-byte
// pieces are turned by (row / 2) % 8 places, so that sixteen lanes that read the
// same piece of sixteen rows are on sixteen different bank groups.
//   Bound by the matrix instructions, whose clock falls under their load: P X of
// 4096 x 4096 takes 316 to 331 us, 1.25 to 1.3 PFLOP/s of float16 instructions (a
// library's plain float16 product: 1.17), the matrix units 68 % busy at 1.78 GHz; S
// and P there 193 to 207 us.  Halves of a step pipelined across the barrier were slower.
template <class CF, int EPI, bool SPLIT>
__global__ void __launch_bounds__(64 * CF::WAVES) __attribute__((amdgpu_waves_per_eu(CF::OCC)))
ortho_product(ProductArgs a) {
    constexpr int MBM = CF::MBM, MBN = CF::MBN, SIDE = CF::SIDE, STAGE = 2 * CF::BYTES, NS = CF::STAGES;
    __shared__ __attribute__((aligned(1024))) char smem[NS * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / CF::WN, wn = wave % CF::WN, li = lane & 31, lh = lane >> 5;
    const int64_t z = blockIdx.z;
    // Workgroups go to the eight XCDs in turn: give each a run of neighbouring tiles.
    const int tiles = gridDim.x, q = tiles / 8, rem = tiles % 8, x = blockIdx.x % 8;
    const int t = x * q + (x < rem ? x : rem) + blockIdx.x / 8;
    int ti, tj;
    tile_of<EPI>(a, t, ti, tj);
    const int first = blockIdx.y * a.share, all = int(a.K / kStep);
    const int steps = all - first < a.share ? all - first : a.share;
    const char* const ga = reinterpret_cast<const char*>(a.A + z * a.stride_a) + int64_t(ti) * SIDE * a.K * 4 + int64_t(first) * 128;
    const char* const gb = reinterpret_cast<const char*>(a.B + z * a.stride_b) + int64_t(tj) * SIDE * a.K * 4 + int64_t(first) * 128;
    // A wave's loads: each 8 rows, lane L the piece that lies at L.
    constexpr int LOADS = SIDE / 8 / CF::WAVES;
    static_assert(SIDE % (8 * CF::WAVES) == 0, "whole loads");
    unsigned off[LOADS];  // below 256 rows of 256 KiB
#pragma unroll
    for (int u = 0; u < LOADS; u++) {
        const int r = (wave * LOADS + u) * 8 + (lane >> 3);
        off[u] = unsigned(r) * unsigned(a.K) * 4u + (((lane & 7) ^ (r >> 1 & 7)) * 16);
    }
    auto issue = [&](int s) {
        const __amdgpu_buffer_rsrc_t ra = make_rsrc(ga), rb = make_rsrc(gb);
        char* const to = smem + s % NS * STAGE + wave * LOADS * 1024;
#pragma unroll
        for (int u = 0; u < LOADS; u++) {
            load_lds<16>(ra, to + u * 1024, off[u], s * 128);
            load_lds<16>(rb, to + CF::BYTES + u * 1024, off[u], s * 128);
        }
    };
    v16f acc[MBM][MBN];
#pragma unroll
    for (int m = 0; m < MBM; m++)
#pragma unroll
        for (int n = 0; n < MBN; n++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[m][n][r] = 0.0f;
#pragma unroll
    for (int s = 0; s < NS - 1; s++)
        if (s < steps) issue(s);
    auto step = [&](int s, auto load) {
        const char* const st = smem + s % NS * STAGE;
        f16x8 fa[2][2][MBM], fb[2][2][MBN];
        auto read = [&](int k) {
#pragma unroll
            for (int p = 0; p < 2; p++) {
                const int piece = 4 * p + 2 * k + lh;
#pragma unroll
                for (int i = 0; i < MBM; i++) {
                    const int r = wm * 32 * MBM + 32 * i + li;
                    fa[k][p][i] = *reinterpret_cast<const f16x8*>(st + r * 128 + (piece ^ (r >> 1 & 7)) * 16);
                }
#pragma unroll
                for (int i = 0; i < MBN; i++) {
                    const int r = wn * 32 * MBN + 32 * i + li;
                    fb[k][p][i] = *reinterpret_cast<const f16x8*>(st + CF::BYTES + r * 128 + (piece ^ (r >> 1 & 7)) * 16);
                }
            }
        };
        auto multiply = [&](int k) {
#pragma unroll
            for (int p = 0; p < 3; p++)  // hi hi, hi lo, lo hi
#pragma unroll
                for (int m = 0; m < MBM; m++)
#pragma unroll
                    for (int n = 0; n < MBN; n++)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[k][p == 2][m], fb[k][p == 1][n], acc[m][n], 0, 0, 0);
        };
        read(0);
        read(1);
        if constexpr (decltype(load)::value) issue(s + NS - 1);
        multiply(0);
        multiply(1);
        // Order: the first half's reads, an instruction on them, the second half's
        // reads, then the loads, one after each of the following instructions.
        constexpr int RD = 2 * (MBM + MBN), MF = 6 * MBM * MBN, LD = decltype(load)::value ? 2 * LOADS : 0;
        static_assert(LD < MF, "loads fit between the instructions");
        __builtin_amdgcn_sched_group_barrier(0x100, RD, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, RD, 0);
#pragma unroll
        for (int u = 0; u < LD; u++) {
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, MF - 1 - LD, 0);
    };
    // Before a step: this wave's loads for it have landed (those of the NS - 2 steps
    // after it may be in flight), then every wave's; and every wave is done with the
    // stage that is written next.
    int s = 0;
    for (; s + NS - 1 < steps; s++) {
        step_barrier<(NS - 2) * 2 * LOADS>();
        step(s, std::true_type{});
    }
    for (; s < steps; s++) {
        step_barrier<0>();
        step(s, std::false_type{});
    }
    __syncthreads();
    // Results by rows through LDS, 32 rows of the wave's columns at a time; the
    // transposed ones, four neighbours a lane, straight from the registers.
    constexpr int COLS = 32 * MBN, PITCH = COLS + 4;
    static_assert(CF::WAVES * 32 * PITCH * 4 <= NS * STAGE, "epilogue fits the stages");
    float* const mine = reinterpret_cast<float*>(smem) + wave * 32 * PITCH;
    const bool diagonal = (EPI == GRAM || EPI == POLY) && ti == tj;
    float* const partial = SPLIT ? a.partial + ((z * gridDim.y + blockIdx.y) * tiles + t) * SIDE * SIDE : nullptr;
#pragma unroll
    for (int m = 0; m < MBM; m++) {
        const int y0 = wm * 32 * MBM + 32 * m, x0 = wn * 32 * MBN;
        const int64_t r0 = int64_t(ti) * SIDE + y0, c0 = int64_t(tj) * SIDE + x0;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int n = 0; n < MBN; n++) {
            const int64_t c = c0 + 32 * n + li;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int64_t r = r0 + 8 * g + 4 * lh;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = SPLIT ? acc[m][n][4 * g + e] : acc[m][n][4 * g + e] * a.scale;
                if constexpr (EPI == POLY) {
                    // S[r + e][c] as S[c][r + e].
                    if (r < a.K) {
                        const _Float16* at = a.A + z * a.stride_a + c * a.K * 2 + part_at(r);
                        const f16x4 h = *reinterpret_cast<const f16x4*>(at), l = *reinterpret_cast<const f16x4*>(at + 32);
#pragma unroll
                        for (int e = 0; e < 4; e++) {
                            v[e] = fmaf(a.b, float(h[e]) + float(l[e]), v[e]);
                            if (r + e == c) v[e] += a.diagonal;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e++) mine[(8 * g + 4 * lh + e) * PITCH + 32 * n + li] = v[e];
                if constexpr (!SPLIT && EPI == LAST) {
                    if (a.tall)
#pragma unroll
                        for (int e = 0; e < 4; e++) store_out(a, z, r + e, c, v[e]);
                } else if constexpr (!SPLIT) {
                    if (!diagonal) store_column(a, z, r, c, v);
                }
            }
        }
        // The wave's own lanes exchange these; its LDS operations complete in order.
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        if constexpr (SPLIT) {
            for (int e = lane; e < 32 * COLS / 4; e += 64) {
                const int y = e / (COLS / 4), cx = e % (COLS / 4) * 4;
                *reinterpret_cast<v4f*>(partial + (y0 + y) * SIDE + x0 + cx) = *reinterpret_cast<const v4f*>(mine + y * PITCH + cx);
            }
        } else if constexpr (EPI == LAST) {
            if (!a.tall)
                for (int e = lane; e < 32 * COLS; e += 64) store_out(a, z, r0 + e / COLS, c0 + e % COLS, mine[e / COLS * PITCH + e % COLS]);
        } else {
            for (int e = lane; e < 32 * COLS / 8; e += 64) {
                const int y = e / (COLS / 8), cx = e % (COLS / 8) * 8;
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; i++) v[i] = mine[y * PITCH + cx + i];
                store_row(a, z, r0 + y, c0 + cx, v);
            }
        }
        asm volatile("" ::: "memory");
    }
}

// S from the shares' sums, added in order: 64 x 64 of a tile a workgroup (1024 x 1024
// in four shares: 8 us).
template <int SIDE>
__global__ void __launch_bounds__(256) ortho_finish(ProductArgs a, int tiles, int shares) {
    __shared__ float tile[64][68];
    constexpr int B = SIDE / 64;
    const int64_t z = blockIdx.z;
    const int t = blockIdx.x / (B * B), by = blockIdx.x % (B * B) / B, bx = blockIdx.x % B;
    int ti, tj;
    tile_of<GRAM>(a, t, ti, tj);
    const int64_t r0 = int64_t(ti) * SIDE + 64 * by, c0 = int64_t(tj) * SIDE + 64 * bx;
    const float* const from = a.partial + (z * shares * tiles + t) * SIDE * SIDE + int64_t(64 * by) * SIDE + 64 * bx;
    const int64_t plane = int64_t(tiles) * SIDE * SIDE;
#pragma unroll
    for (int e = threadIdx.x; e < 1024; e += 256) {
        const int y = e / 16, cx = e % 16 * 4;
        v4f v = {0, 0, 0, 0};
        const float* at = from + y * SIDE + cx;
#pragma unroll 4
        for (int s = 0; s < shares; s++) v += *reinterpret_cast<const v4f*>(at + s * plane);
        *reinterpret_cast<v4f*>(&tile[y][cx]) = v * a.scale;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 512; e += 256) {
        const int y = e / 8, cx = e % 8 * 8;
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; i++) v[i] = tile[y][cx + i];
        store_row(a, z, r0 + y, c0 + cx, v);
    }
    if (ti != tj)
        for (int e = threadIdx.x; e < 1024; e += 256) {
            const int y = e % 16 * 4, cx = e / 16;
            const float v[4] = {tile[y][cx], tile[y + 1][cx], tile[y + 2][cx], tile[y + 3][cx]};
            store_column(a, z, r0 + y, c0 + cx, v);
        }
}

// ---- host ---------------------------------------------------------------------------

// How one product is run: tile side and shares of the sum.
struct ProductPlan {
    int side, shares, share;  // share: steps
    int64_t tiles;            // of a matrix
};

// The cheapest by a model of rounds of workgroups over the 256 CUs, fitted (us) to
// every configuration and 1 to 8 shares on ten shapes of 256 x 256 to 4096 x 4096.  For
// example S of 4096 x 4096: tiles of 64 242, 128 250, 192 199, 256 250; P X there 471,
// 375, 383, 317; S of 1024 x 4096: 29, 68, 149, 217, and 29 and 30 in three and four
// shares of tiles of 64 and 128; P X of 2048 x 2048: 61, 55, 94, 131.
ProductPlan product_plan(bool half, bool long_sum, int64_t rows, int64_t cols, int64_t K, int64_t batch) {
    struct Option {
        int side;
        double step, tile;  // of a workgroup, with every CU busy
    };
    static const Option options[] = {{64, 0.23, 0.8}, {128, 0.72, 5.0}, {192, 1.48, 8.0}, {256, 2.42, 8.0}};
    ProductPlan best{};
    double least = 0;
    const int64_t steps = ceil_div(K, kStep);
    for (const Option& o : options) {
        const int64_t tm = ceil_div(rows, o.side), tn = ceil_div(cols, o.side);
        const int64_t tiles = half ? tm * (tm + 1) / 2 : tm * tn;
        for (int shares : {1, 2, 3, 4, 6, 8, 12, 16}) {
            // Only S has sums long enough against its tiles.
            if (shares > 1 && (!long_sum || steps / shares < 4)) break;
            const int64_t share = ceil_div(steps, shares), n = ceil_div(steps, share);
            const double u = double(tiles * n * batch) / 256, whole = std::floor(u), part = u - whole;
            // Two workgroups of tiles of 64 run on a CU at a time, which evens the rounds
            // out; one of larger tiles, faster where fewer CUs are busy.
            const double rounds = o.side == 64 ? std::max(1.0, std::min(u + 0.5, std::ceil(u)))
                                               : whole + (part > 0 ? 0.65 + 0.35 * part : 0.0);
            double us = 4.0 + rounds * (double(share) * o.step + o.tile);
            if (n > 1) us += 6.0 + double(tiles * batch * o.side * o.side) * double(n) * 4 / 4e6;
            if (best.side == 0 || us < least) {
                least = us;
                best = {o.side, int(n), int(share), tiles};
            }
        }
    }
    return best;
}

struct OrthoPlan {
    bool tall;
    int64_t m, n, km, kn, am, an;  // sides; columns of rows; rows with a tile's overhang
    ProductPlan gram, poly, apply;
    size_t squares_at, x_at, xt_at[2], s_at, p_at, partial_at, bytes;
};

OrthoPlan ortho_plan(int64_t batch, int64_t M, int64_t N) {
    OrthoPlan p{};
    p.tall = M > N;
    p.m = std::min(M, N);
    p.n = std::max(M, N);
    p.km = ceil_div(p.m, 32) * 32;
    p.kn = ceil_div(p.n, 32) * 32;
    p.am = p.km + 256;
    p.an = p.kn + 256;
    p.gram = product_plan(true, true, p.m, p.m, p.n, batch);
    p.poly = product_plan(true, false, p.m, p.m, p.m, batch);
    p.apply = product_plan(false, false, p.m, p.n, p.m, batch);
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    p.squares_at = take(size_t(batch) * kNormBlocks * sizeof(double));
    p.x_at = take(size_t(batch) * p.am * p.kn * 4);
    p.xt_at[0] = take(size_t(batch) * p.an * p.km * 4);
    p.xt_at[1] = take(size_t(batch) * p.an * p.km * 4);
    p.s_at = take(size_t(batch) * p.am * p.km * 4);
    p.p_at = take(size_t(batch) * p.am * p.km * 4);
    p.partial_at = take(p.gram.shares > 1 ? size_t(batch) * p.gram.shares * p.gram.tiles * p.gram.side * p.gram.side * 4 : 0);
    p.bytes = at;
    return p;
}

// The power of two that brings numbers of up to `bound` to at most 2^14.
int power_for(double bound) {
    int e = 0;
    (void)std::frexp(bound, &e);  // bound < 2^e
    return 14 - e;
}

template <class CF, int EPI>
void launch_tiles(const ProductArgs& a, const ProductPlan& p, unsigned batch, hipStream_t s) {
    const dim3 grid(unsigned(p.tiles), p.shares, batch), block(64 * CF::WAVES);
    if constexpr (EPI == GRAM) {
        if (p.shares > 1) {
            hipLaunchKernelGGL((ortho_product<CF, EPI, true>), grid, block, 0, s, a);
            constexpr int B = CF::SIDE / 64;
            hipLaunchKernelGGL(ortho_finish<CF::SIDE>, dim3(unsigned(p.tiles * B * B), 1, batch), dim3(256), 0, s, a,
                               int(p.tiles), p.shares);
            return;
        }
    }
    hipLaunchKernelGGL((ortho_product<CF, EPI, false>), grid, block, 0, s, a);
}

template <int EPI>
void launch_product(ProductArgs a, const ProductPlan& p, unsigned batch, hipStream_t s) {
    a.tiles_m = int(ceil_div(a.rows, p.side));
    a.tiles_n = int(ceil_div(a.cols, p.side));
    a.share = p.share;
    if (p.side == 64) launch_tiles<Tile64, EPI>(a, p, batch, s);
    else if (p.side == 128) launch_tiles<Tile128, EPI>(a, p, batch, s);
    else if (p.side == 192) launch_tiles<Tile192, EPI>(a, p, batch, s);
    else launch_tiles<Tile256, EPI>(a, p, batch, s);
}

hipError_t run_steps(const OrthoArgs& g, const OrthoPlan& p, hipStream_t s) {
    char* const ws = static_cast<char*>(g.ws);
    _Float16* const X = reinterpret_cast<_Float16*>(ws + p.x_at);
    _Float16* const S = reinterpret_cast<_Float16*>(ws + p.s_at);
    _Float16* const P = reinterpret_cast<_Float16*>(ws + p.p_at);
    const int64_t sx = p.am * p.kn * 2, st = p.an * p.km * 2, ss = p.am * p.km * 2;
    const unsigned batch = unsigned(g.batch);
    for (int i = 0; i < g.steps; i++) {
        const double a = g.coef[3 * i], b = g.coef[3 * i + 1], c = g.coef[3 * i + 2], r = g.bounds[i];
        const int ex = power_for(r), es = power_for(r * r);
        const int ep = power_for(std::fabs(a) + std::fabs(b) * r * r + std::fabs(c) * r * r * r * r);
        const int en = power_for(g.bounds[i + 1]);
        const bool last = i + 1 == g.steps;
        ProductArgs q{};
        q.partial = reinterpret_cast<float*>(ws + p.partial_at);
        q.A = q.B = X;
        q.K = p.kn;
        q.stride_a = q.stride_b = sx;
        q.rows = q.cols = p.m;
        q.scale = float(std::ldexp(1.0, es - 2 * ex));
        q.N = q.T = S;
        q.ldn = q.ldt = p.km;
        q.stride_n = q.stride_t = ss;
        launch_product<GRAM>(q, p.gram, batch, s);
        q.A = q.B = S;
        q.K = p.km;
        q.stride_a = q.stride_b = ss;
        q.scale = float(std::ldexp(c, ep - 2 * es));
        q.N = q.T = P;
        q.b = float(std::ldexp(b, ep - es));
        q.diagonal = float(std::ldexp(a, ep));
        launch_product<POLY>(q, p.poly, batch, s);
        q.A = P;
        q.B = reinterpret_cast<const _Float16*>(ws + p.xt_at[i & 1]);
        q.stride_b = st;
        q.rows = p.m;
        q.cols = p.n;
        q.scale = float(std::ldexp(1.0, (last ? 0 : en) - ep - ex));
        q.N = X;
        q.ldn = p.kn;
        q.stride_n = sx;
        q.T = reinterpret_cast<_Float16*>(ws + p.xt_at[~i & 1]);
        q.ldt = p.km;
        q.stride_t = st;
        q.type = g.type;
        q.tall = p.tall;
        q.out = g.O;
        q.ldo = g.ldo;
        q.stride_o = g.so;
        if (last) launch_product<LAST>(q, p.apply, batch, s);
        else launch_product<APPLY>(q, p.apply, batch, s);
    }
    return hipGetLastError();
}

}  // namespace

size_t ortho_workspace_bytes(int64_t batch, int64_t M, int64_t N) {
    if (!batch || !M || !N) return 0;
    if (std::min(M, N) <= kOrthoSmall) return ortho_small_bytes(batch, M, N);
    return ortho_plan(batch, M, N).bytes;
}

hipError_t launch_orthogonalize(const OrthoArgs& g, hipStream_t s) {
    if (std::min(g.M, g.N) <= kOrthoSmall) return launch_ortho_small(g, s);
    const OrthoPlan p = ortho_plan(g.batch, g.M, g.N);
    char* const ws = static_cast<char*>(g.ws);
    double* const squares = reinterpret_cast<double*>(ws + p.squares_at);
    const int blocks = int(std::min<int64_t>(kNormBlocks, ceil_div(g.M * g.N, 4096)));
    const dim3 grid(blocks, unsigned(g.batch));
    if (g.type == T_F32) hipLaunchKernelGGL(ortho_squares<T_F32>, grid, dim3(256), 0, s, g.G, g.M, g.N, g.ldg, g.sg, squares);
    else if (g.type == T_F16) hipLaunchKernelGGL(ortho_squares<T_F16>, grid, dim3(256), 0, s, g.G, g.M, g.N, g.ldg, g.sg, squares);
    else hipLaunchKernelGGL(ortho_squares<T_BF16>, grid, dim3(256), 0, s, g.G, g.M, g.N, g.ldg, g.sg, squares);
    const dim3 tiles(unsigned(ceil_div(p.kn, 64)), unsigned(ceil_div(p.km, 64)), unsigned(g.batch));
    auto start = [&](auto type) {
        hipLaunchKernelGGL(ortho_split<decltype(type)::value>, tiles, dim3(256), 0, s, g.G, p.tall, p.m, p.n, g.ldg, g.sg,
                           squares, blocks, g.eps, float(std::ldexp(1.0, power_for(g.bounds[0]))),
                           reinterpret_cast<_Float16*>(ws + p.x_at), reinterpret_cast<_Float16*>(ws + p.xt_at[0]), p.km,
                           p.kn, p.am * p.kn * 2, p.an * p.km * 2);
    };
    if (g.type == T_F32) start(std::integral_constant<int, T_F32>{});
    else if (g.type == T_F16) start(std::integral_constant<int, T_F16>{});
    else start(std::integral_constant<int, T_BF16>{});
    return run_steps(g, p, s);
}

}  // namespace sgemm
