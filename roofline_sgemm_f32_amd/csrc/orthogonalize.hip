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
// stored twice.  Rows are padded with zeros to whole tiles, so that no product
// has an edge.  A row holds 32 high parts, their 32 low parts, the next 32 ...:
// 128 bytes are a row's share of one step of the sum.
#include <algorithm>
#include <cmath>

#include "kernels.h"

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

constexpr int kNormBlocks = 256;  // partial sums of a matrix

// Partial sums of squares in double, block x of matrix y.
__global__ void __launch_bounds__(256) ortho_squares(int type, const void* G, int64_t M, int64_t N, int64_t ldg,
                                                     int64_t sg, double* out) {
    __shared__ double part[4];
    double v = 0;
    const int64_t at = int64_t(blockIdx.y) * sg;
    if (ldg == N) {
        const int64_t n = M * N;
        for (int64_t t = int64_t(blockIdx.x) * 256 + threadIdx.x; t < n; t += int64_t(gridDim.x) * 256) {
            const double x = load_as(type, G, at + t);
            v += x * x;
        }
    } else {
        for (int64_t r = blockIdx.x; r < M; r += gridDim.x)
            for (int64_t c = threadIdx.x; c < N; c += 256) {
                const double x = load_as(type, G, at + r * ldg + c);
                v += x * x;
            }
    }
    for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    if (threadIdx.x == 0) out[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = part[0] + part[1] + part[2] + part[3];
}

// X and X^T in parts, times `scale`, from G: a 64 x 64 tile of X (m x n, padded
// to mp x np) a workgroup, turned in LDS.
__global__ void __launch_bounds__(256) ortho_split(int type, const void* G, bool tall, int64_t m, int64_t n, int64_t ldg,
                                                   int64_t sg, const double* squares, int parts, double eps,
                                                   float scale, _Float16* X, _Float16* Xt, int64_t mp, int64_t np) {
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
    X += b * mp * np * 2;
    Xt += b * mp * np * 2;
    // Rows of G as they lie: X's rows, or its columns.
    for (int e = threadIdx.x; e < 4096; e += 256) {
        const int y = e / 64, x = e % 64;
        const int64_t r = tall ? r0 + x : r0 + y, c = tall ? c0 + y : c0 + x;
        float v = 0.0f;
        if (r < m && c < n) {
            const double g = load_as(type, G, b * sg + (tall ? c * ldg + r : r * ldg + c));
            v = g == 0 ? 0.0f : float(g * f);  // zeros stay so whatever f
        }
        if (tall) tile[x][y] = v;
        else tile[y][x] = v;
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
        _Float16* at = X + (r0 + y) * np * 2 + part_at(c0 + x);
        *reinterpret_cast<f16x8*>(at) = h;
        *reinterpret_cast<f16x8*>(at + 32) = l;
#pragma unroll
        for (int i = 0; i < 8; i++) {
            _Float16 a, c;
            split(tile[x + i][y], a, c);
            h[i] = a, l[i] = c;
        }
        at = Xt + (c0 + y) * mp * 2 + part_at(r0 + x);
        *reinterpret_cast<f16x8*>(at) = h;
        *reinterpret_cast<f16x8*>(at + 32) = l;
    }
}

// ---- the products -----------------------------------------------------------------

enum Epilogue { GRAM, POLY, APPLY, LAST };

struct ProductArgs {
    const _Float16 *A, *B;      // C = A B^T: rows of K sums in parts
    int64_t K;                  // padded
    int64_t stride_a, stride_b; // between matrices, in float16
    int tiles_m, tiles_n;
    float scale;                // of the sums
    // GRAM, POLY: S or P, ld its padded side.  APPLY: X and X^T.
    _Float16 *N, *T;
    int64_t ldn, ldt, stride_n, stride_t;  // in columns, and in float16
    // POLY: out = scale sum + b S + diagonal, S the operand.
    float b, diagonal;
    int m;
    // LAST: out in `type`, rows and columns that exist.
    int type;
    bool tall;
    void* out;
    int64_t ldo, stride_o;
    int64_t rows, cols;
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

// A workgroup: one 64 MB x 64 MB tile, four waves of 32 MB x 32 MB.  Steps of 32
// of the sum go through two LDS stages, written by loads that bypass the
// registers; a row's eight 16-byte pieces are turned by (row / 2) % 8 places,
// so that sixteen lanes that read the same piece of sixteen rows are on sixteen
// different bank groups.
template <int MB, int EPI>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) ortho_product(ProductArgs a) {
    constexpr int TILE = 64 * MB, SIDE = TILE * 128, STAGE = 2 * SIDE;  // bytes
    __shared__ __attribute__((aligned(1024))) char smem[2 * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1, li = lane & 31, lh = lane >> 5;
    const int64_t z = blockIdx.z;
    // Workgroups go to the eight XCDs in turn: give each a run of neighbouring tiles.
    const int tiles = gridDim.x, q = tiles / 8, rem = tiles % 8, x = blockIdx.x % 8;
    const int t = x * q + (x < rem ? x : rem) + blockIdx.x / 8;
    int ti, tj;
    if constexpr (EPI == GRAM || EPI == POLY) {
        triangle(t, a.tiles_m, ti, tj);
    } else {
        // Groups of eight tile rows, column by column.
        const int per = 8 * a.tiles_n, first = t / per * 8, h = a.tiles_m - first < 8 ? a.tiles_m - first : 8;
        ti = first + t % per % h;
        tj = t % per / h;
    }
    const char* const ga = reinterpret_cast<const char*>(a.A + z * a.stride_a) + int64_t(ti) * TILE * a.K * 4;
    const char* const gb = reinterpret_cast<const char*>(a.B + z * a.stride_b) + int64_t(tj) * TILE * a.K * 4;
    // A wave's loads: each 8 rows, lane L the piece that lies at L.
    constexpr int LOADS = TILE / 8 / 4;
    const int row8 = lane >> 3;
    auto issue = [&](int64_t s, int stage) {
        char* const to = smem + stage * STAGE;
#pragma unroll
        for (int u = 0; u < LOADS; u++) {
            const int r = (wave * LOADS + u) * 8 + row8;
            const int64_t off = int64_t(r) * a.K * 4 + s * 128 + (((lane & 7) ^ (r >> 1 & 7)) * 16);
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<const __attribute__((address_space(1))) void*>(reinterpret_cast<uintptr_t>(ga + off)),
                LDS_PTR(to + (wave * LOADS + u) * 1024), 16, 0, 0);
            __builtin_amdgcn_global_load_lds(
                reinterpret_cast<const __attribute__((address_space(1))) void*>(reinterpret_cast<uintptr_t>(gb + off)),
                LDS_PTR(to + SIDE + (wave * LOADS + u) * 1024), 16, 0, 0);
        }
    };
    v16f acc[MB][MB];
#pragma unroll
    for (int m = 0; m < MB; m++)
#pragma unroll
        for (int n = 0; n < MB; n++)
#pragma unroll
            for (int r = 0; r < 16; r++) acc[m][n][r] = 0.0f;
    const int steps = int(a.K / kStep);
    issue(0, 0);
    for (int s = 0; s < steps; s++) {
        // This wave's loads of step s have landed, then every wave's; and every wave
        // is done with the other stage.
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (s + 1 < steps) issue(s + 1, (s + 1) & 1);
        const char* const st = smem + (s & 1) * STAGE;
#pragma unroll
        for (int k = 0; k < 2; k++) {
            f16x8 fa[2][MB], fb[2][MB];
#pragma unroll
            for (int p = 0; p < 2; p++)
#pragma unroll
                for (int i = 0; i < MB; i++) {
                    const int ra = wm * 32 * MB + 32 * i + li, rb = wn * 32 * MB + 32 * i + li;
                    const int piece = 4 * p + 2 * k + lh;
                    fa[p][i] = *reinterpret_cast<const f16x8*>(st + ra * 128 + (piece ^ (ra >> 1 & 7)) * 16);
                    fb[p][i] = *reinterpret_cast<const f16x8*>(st + SIDE + rb * 128 + (piece ^ (rb >> 1 & 7)) * 16);
                }
#pragma unroll
            for (int p = 0; p < 3; p++)  // hi hi, hi lo, lo hi
#pragma unroll
                for (int m = 0; m < MB; m++)
#pragma unroll
                    for (int n = 0; n < MB; n++)
                        acc[m][n] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[p == 2][m], fb[p == 1][n], acc[m][n], 0, 0, 0);
        }
    }
    __syncthreads();
    // Results by rows through LDS, 32 rows of the wave's columns at a time; the
    // transposed ones, four neighbours a lane, straight from the registers.
    constexpr int COLS = 32 * MB, PITCH = COLS + 4;
    static_assert(4 * 32 * PITCH * 4 <= 2 * STAGE, "epilogue fits the stages");
    float* const mine = reinterpret_cast<float*>(smem) + wave * 32 * PITCH;
    const bool diagonal = (EPI == GRAM || EPI == POLY) && ti == tj;
#pragma unroll
    for (int m = 0; m < MB; m++) {
        const int64_t r0 = int64_t(ti) * TILE + wm * 32 * MB + 32 * m;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int n = 0; n < MB; n++) {
            const int64_t c = int64_t(tj) * TILE + wn * 32 * MB + 32 * n + li;
#pragma unroll
            for (int g = 0; g < 4; g++) {
                const int64_t r = r0 + 8 * g + 4 * lh;
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; e++) v[e] = acc[m][n][4 * g + e] * a.scale;
                if constexpr (EPI == POLY) {
                    // S[r + e][c] as S[c][r + e].
                    const _Float16* at = a.A + z * a.stride_a + c * a.K * 2 + part_at(r);
                    const f16x4 h = *reinterpret_cast<const f16x4*>(at), l = *reinterpret_cast<const f16x4*>(at + 32);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        v[e] = fmaf(a.b, float(h[e]) + float(l[e]), v[e]);
                        if (r + e == c && r + e < a.m) v[e] += a.diagonal;
                    }
                }
#pragma unroll
                for (int e = 0; e < 4; e++) mine[(8 * g + 4 * lh + e) * PITCH + 32 * n + li] = v[e];
                if constexpr (EPI == LAST) {
                    if (a.tall && c < a.cols)
#pragma unroll
                        for (int e = 0; e < 4; e++)
                            if (r + e < a.rows) store_as(a.type, a.out, z * a.stride_o + c * a.ldo + r + e, v[e]);
                } else if (!diagonal) {
                    f16x4 h, l;
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        _Float16 p, o;
                        split(v[e], p, o);
                        h[e] = p, l[e] = o;
                    }
                    _Float16* at = a.T + z * a.stride_t + c * a.ldt * 2 + part_at(r);
                    *reinterpret_cast<f16x4*>(at) = h;
                    *reinterpret_cast<f16x4*>(at + 32) = l;
                }
            }
        }
        // The wave's own lanes exchange these; its LDS operations complete in order.
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        if constexpr (EPI == LAST) {
            if (!a.tall)
                for (int e = lane; e < 32 * COLS; e += 64) {
                    const int64_t r = r0 + e / COLS, c = int64_t(tj) * TILE + wn * 32 * MB + e % COLS;
                    if (r < a.rows && c < a.cols)
                        store_as(a.type, a.out, z * a.stride_o + r * a.ldo + c, mine[e / COLS * PITCH + e % COLS]);
                }
        } else {
            for (int e = lane; e < 32 * COLS / 8; e += 64) {
                const int y = e / (COLS / 8), cx = e % (COLS / 8) * 8;
                f16x8 h, l;
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    _Float16 p, o;
                    split(mine[y * PITCH + cx + i], p, o);
                    h[i] = p, l[i] = o;
                }
                const int64_t c = int64_t(tj) * TILE + wn * 32 * MB + cx;
                _Float16* at = a.N + z * a.stride_n + (r0 + y) * a.ldn * 2 + part_at(c);
                *reinterpret_cast<f16x8*>(at) = h;
                *reinterpret_cast<f16x8*>(at + 32) = l;
            }
        }
        asm volatile("" ::: "memory");
    }
}

// ---- host ---------------------------------------------------------------------------

struct OrthoPlan {
    bool tall;
    int64_t m, n, mp, np;
    int mb;  // 64 mb: a tile's side
    size_t squares_at, x_at, xt_at[2], s_at, p_at, bytes;
};

OrthoPlan ortho_plan(int64_t batch, int64_t M, int64_t N) {
    OrthoPlan p{};
    p.tall = M > N;
    p.m = std::min(M, N);
    p.n = std::max(M, N);
    p.mb = p.m > 512 ? 2 : 1;
    const int64_t side = 64 * p.mb;
    p.mp = ceil_div(p.m, side) * side;
    p.np = ceil_div(p.n, side) * side;
    const size_t x = size_t(batch) * p.mp * p.np * 4, s = size_t(batch) * p.mp * p.mp * 4;
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t here = at;
        at += (n + 255) / 256 * 256;
        return here;
    };
    p.squares_at = take(size_t(batch) * kNormBlocks * sizeof(double));
    p.x_at = take(x);
    p.xt_at[0] = take(x);
    p.xt_at[1] = take(x);
    p.s_at = take(s);
    p.p_at = take(s);
    p.bytes = at;
    return p;
}

// The power of two that brings numbers of up to `bound` to at most 2^14.
int power_for(double bound) {
    int e = 0;
    (void)std::frexp(bound, &e);  // bound < 2^e
    return 14 - e;
}

template <int MB>
hipError_t run_steps(const OrthoArgs& g, const OrthoPlan& p, hipStream_t s) {
    char* const ws = static_cast<char*>(g.ws);
    _Float16* const X = reinterpret_cast<_Float16*>(ws + p.x_at);
    _Float16* const S = reinterpret_cast<_Float16*>(ws + p.s_at);
    _Float16* const P = reinterpret_cast<_Float16*>(ws + p.p_at);
    const int tm = int(p.mp / (64 * MB)), tn = int(p.np / (64 * MB)), half = tm * (tm + 1) / 2;
    const int64_t sx = p.mp * p.np * 2, ss = p.mp * p.mp * 2;
    const unsigned batch = unsigned(g.batch);
    for (int i = 0; i < g.steps; i++) {
        const double a = g.coef[3 * i], b = g.coef[3 * i + 1], c = g.coef[3 * i + 2], r = g.bounds[i];
        const _Float16* Xt = reinterpret_cast<const _Float16*>(ws + p.xt_at[i & 1]);
        _Float16* Xt2 = reinterpret_cast<_Float16*>(ws + p.xt_at[~i & 1]);
        const int ex = power_for(r), es = power_for(r * r);
        const int ep = power_for(std::fabs(a) + std::fabs(b) * r * r + std::fabs(c) * r * r * r * r);
        const int en = power_for(g.bounds[i + 1]);
        ProductArgs q{};
        q.A = q.B = X;
        q.K = p.np;
        q.stride_a = q.stride_b = sx;
        q.tiles_m = q.tiles_n = tm;
        q.scale = float(std::ldexp(1.0, es - 2 * ex));
        q.N = q.T = S;
        q.ldn = q.ldt = p.mp;
        q.stride_n = q.stride_t = ss;
        hipLaunchKernelGGL((ortho_product<MB, GRAM>), dim3(half, 1, batch), dim3(256), 0, s, q);
        q.A = q.B = S;
        q.K = p.mp;
        q.stride_a = q.stride_b = ss;
        q.scale = float(std::ldexp(c, ep - 2 * es));
        q.N = q.T = P;
        q.b = float(std::ldexp(b, ep - es));
        q.diagonal = float(std::ldexp(a, ep));
        q.m = int(p.m);
        hipLaunchKernelGGL((ortho_product<MB, POLY>), dim3(half, 1, batch), dim3(256), 0, s, q);
        q.A = P;
        q.B = Xt;
        q.stride_b = sx;
        q.tiles_n = tn;
        const bool last = i + 1 == g.steps;
        q.scale = float(std::ldexp(1.0, (last ? 0 : en) - ep - ex));
        q.N = X;
        q.ldn = p.np;
        q.stride_n = sx;
        q.T = Xt2;
        q.ldt = p.mp;
        q.stride_t = sx;
        q.type = g.type;
        q.tall = p.tall;
        q.out = g.O;
        q.ldo = g.ldo;
        q.stride_o = g.so;
        q.rows = p.m;
        q.cols = p.n;
        if (last) hipLaunchKernelGGL((ortho_product<MB, LAST>), dim3(tm * tn, 1, batch), dim3(256), 0, s, q);
        else hipLaunchKernelGGL((ortho_product<MB, APPLY>), dim3(tm * tn, 1, batch), dim3(256), 0, s, q);
    }
    return hipGetLastError();
}

}  // namespace

size_t ortho_workspace_bytes(int64_t batch, int64_t M, int64_t N) {
    return batch && M && N ? ortho_plan(batch, M, N).bytes : 0;
}

hipError_t launch_orthogonalize(const OrthoArgs& g, hipStream_t s) {
    const OrthoPlan p = ortho_plan(g.batch, g.M, g.N);
    char* const ws = static_cast<char*>(g.ws);
    double* const squares = reinterpret_cast<double*>(ws + p.squares_at);
    const int blocks = int(std::min<int64_t>(kNormBlocks, ceil_div(g.M * g.N, 2048)));
    hipLaunchKernelGGL(ortho_squares, dim3(blocks, unsigned(g.batch)), dim3(256), 0, s, g.type, g.G, g.M, g.N, g.ldg, g.sg, squares);
    hipLaunchKernelGGL(ortho_split, dim3(unsigned(p.np / 64), unsigned(p.mp / 64), unsigned(g.batch)), dim3(256), 0, s,
                       g.type, g.G, p.tall, p.m, p.n, g.ldg, g.sg, squares, blocks, g.eps,
                       float(std::ldexp(1.0, power_for(g.bounds[0]))), reinterpret_cast<_Float16*>(ws + p.x_at),
                       reinterpret_cast<_Float16*>(ws + p.xt_at[0]), p.mp, p.np);
    return p.mb == 2 ? run_steps<2>(g, p, s) : run_steps<1>(g, p, s);
}

}  // namespace sgemm
