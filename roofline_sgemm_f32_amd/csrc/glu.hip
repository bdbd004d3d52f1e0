// Gated feed-forward block, H = act(X Wg) * (X Wu), and the elementwise part
// of its backward pass.
//
// Forward: G = X Wg and U = X Wu share X, so one kernel forms both sums and
// applies the activation to the finished pair; G and U go to memory only when
// the caller keeps them for the backward pass.
//
// Backward, from dH: dG = dH U act'(G) and dU = dH act(G) elementwise (this
// file), then products on the library's own matrix kernels:
//   dX = dG Wg^T + dU Wu^T,   dWg = X^T dG,   dWu = X^T dU.
#include "activation.h"
#include "kernels.h"

namespace sgemm {

// One output per lane, the lanes of a wave along a row of H; 64-bit offsets.
__global__ void __launch_bounds__(256)
glu_general(GluArgs g, int64_t tiles_n, int64_t tiles) {
    const int lane = threadIdx.x % 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t row = (t / tiles_n) * 4 + wave;
        const int64_t col = (t % tiles_n) * 64 + lane;
        if (row >= g.M || col >= g.F) continue;
        const int64_t step = g.transw ? 1 : g.ldw, base = g.transw ? col * g.ldw : col;
        const float *x = g.X + row * g.ldx, *wg = g.Wg + base, *wu = g.Wu + base;
        float sg = 0.0f, su = 0.0f;
        for (int64_t k = 0; k < g.K; k++) {
            sg = fmaf(x[k], wg[k * step], sg);
            su = fmaf(x[k], wu[k * step], su);
        }
        g.H[row * g.ldh + col] = act_value(g.act, sg) * su;
        if (g.G) {
            g.G[row * g.ldgu + col] = sg;
            g.U[row * g.ldgu + col] = su;
        }
    }
}

hipError_t launch_glu_general(const GluArgs& g, hipStream_t s) {
    const int64_t tn = ceil_div(g.F, 64), tiles = tn * ceil_div(g.M, 4);
    hipLaunchKernelGGL(glu_general, dim3(grid_for(tiles)), dim3(256), 0, s, g, tn, tiles);
    return hipGetLastError();
}

namespace {
typedef float v4f __attribute__((ext_vector_type(4)));
constexpr int kThinWaves = 8;  // per workgroup

// Four floats from any 4-byte aligned address.
__device__ __forceinline__ v4f load4(const float* p) {
    v4f v;
    __builtin_memcpy(&v, p, 16);
    return v;
}

// Four floats of a row of n from element k, zero past its end.
__device__ __forceinline__ v4f load4_tail(const float* row, int64_t k, int64_t n) {
    v4f v;
#pragma unroll
    for (int e = 0; e < 4; e++) v[e] = k + e < n ? row[k + e] : 0.0f;
    return v;
}

// Sums of V values over the lanes that differ in lane bits OFF, OFF / 2, ...,
// LAST.  Each step hands half of the values to the partner lane and adds the
// partner's other half, so V - 1 exchanges do for up to log2 V steps; further
// steps add the one value left.  Lane l then holds, in v[0 ..], values
// first ... of the V, first returned.
template <int OFF, int LAST, int N, int V>
__device__ __forceinline__ int reduce_lanes(float (&v)[V], int lane) {
    if constexpr (OFF < LAST) {
        return 0;
    } else if constexpr (N > 1) {
        constexpr int H = N / 2;
        const bool up = (lane & OFF) != 0;
#pragma unroll
        for (int i = 0; i < H; i++) {
            const float keep = up ? v[i + H] : v[i], send = up ? v[i] : v[i + H];
            v[i] = keep + __shfl_xor(send, OFF);
        }
        return (up ? H : 0) + reduce_lanes<OFF / 2, LAST, H>(v, lane);
    } else {
        v[0] += __shfl_xor(v[0], OFF);
        return reduce_lanes<OFF / 2, LAST, 1>(v, lane);
    }
}

// The result at (m, f) from its two finished sums.
__device__ __forceinline__ void finish(const GluArgs& g, int64_t m, int64_t f, float sg, float su) {
    g.H[m * g.ldh + f] = act_value(g.act, sg) * su;
    if (g.G) {
        g.G[m * g.ldgu + f] = sg;
        g.U[m * g.ldgu + f] = su;
    }
}
}  // namespace

// One to sixteen rows of X (MR rounds M up to a power of two; rows past M repeat
// the last): the weights are read once and bound the time, at two operations
// per float and row; a matrix-core tile would stage them through LDS beside as
// much of X.  Measured at F = 8192, K = 4096 (268 MB, 41 us at the copy's rate):
// 46.8 us for one row and weights F x K, 54.9 for 8, 70.8 for 16 (83 on matrix
// tiles); K x F 55.7, 56.1 and 64.1 (79).
//
// Weights F x K: a wave owns RF rows of both weights and its lanes split K,
// four floats each, so its loads are 1 KiB contiguous; WKW waves share K.  X
// comes from the caches.
template <int MR, int RF, int WKW>
__global__ void __launch_bounds__(64 * kThinWaves)
glu_thin_fk(GluArgs g) {
    constexpr bool XPRE = MR <= 2;
    constexpr int MX = MR < 8 ? MR : 8;
    constexpr int V = 2 * MR * RF, GROUPS = kThinWaves / WKW;
    __shared__ float red[kThinWaves][V];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t f0 = (int64_t(blockIdx.x) * GROUPS + w / WKW) * RF;
    const float* wrow[2][RF];
#pragma unroll
    for (int r = 0; r < RF; r++) {
        const int64_t f = f0 + r < g.F ? f0 + r : g.F - 1;
        wrow[0][r] = g.Wg + f * g.ldw;
        wrow[1][r] = g.Wu + f * g.ldw;
    }
    const auto xrow = [&](int m) { return g.X + (m < g.M ? m : g.M - 1) * g.ldx; };
    float acc[V];  // [matrix][row of X][row of the weight]
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    // MX rows of X from row mg on.
    auto add = [&](const v4f (&wv)[2][RF], const v4f (&xv)[MX], int mg) {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int m = 0; m < MX; m++)
#pragma unroll
                for (int r = 0; r < RF; r++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        float& a = acc[(t * MR + mg + m) * RF + r];
                        a = fmaf(xv[m][e], wv[t][r][e], a);
                    }
    };
    auto loadw = [&](v4f (&wv)[2][RF], int64_t k) {
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int r = 0; r < RF; r++) wv[t][r] = load4(wrow[t][r] + k);
    };
    const int64_t step = 256 * WKW, k0 = (w % WKW) * 256 + lane * 4;
    int64_t k = k0;
    // A step ahead: its weights, and with one or two rows its X (from the
    // caches; of more rows it takes the registers of a resident wave).
    auto loadx = [&](v4f (&xv)[MX], int64_t at, int mg) {
#pragma unroll
        for (int m = 0; m < MX; m++) xv[m] = load4(xrow(mg + m) + at);
    };
    v4f wv[2][RF], xv[MX];
    if (k + 4 <= g.K) {
        loadw(wv, k);
        if (XPRE) loadx(xv, k, 0);
    }
    for (; k + 4 <= g.K; k += step) {
        v4f wn[2][RF], xn[MX];
        const bool more = k + step + 4 <= g.K;
        if (!XPRE) loadx(xv, k, 0);
        if (more) {
            loadw(wn, k + step);
            if (XPRE) loadx(xn, k + step, 0);
        }
        add(wv, xv, 0);
#pragma unroll
        for (int mg = MX; mg < MR; mg += MX) {
            loadx(xv, k, mg);
            add(wv, xv, mg);
        }
        if (more) {
#pragma unroll
            for (int r = 0; r < RF; r++) wv[0][r] = wn[0][r], wv[1][r] = wn[1][r];
#pragma unroll
            for (int m = 0; m < MX && XPRE; m++) xv[m] = xn[m];
        }
    }
    if (k < g.K) {  // one lane at most: the row's last, incomplete four
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int r = 0; r < RF; r++) wv[t][r] = load4_tail(wrow[t][r], k, g.K);
#pragma unroll
        for (int mg = 0; mg < MR; mg += MX) {
#pragma unroll
            for (int m = 0; m < MX; m++) xv[m] = load4_tail(xrow(mg + m), k, g.K);
            add(wv, xv, mg);
        }
    }
    constexpr int HELD = V > 64 ? V / 64 : 1;
    const int first = reduce_lanes<32, 1, V>(acc, lane);
#pragma unroll
    for (int i = 0; i < HELD; i++) red[w][first + i] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < GROUPS * MR * RF; o += blockDim.x) {
        const int grp = o / (MR * RF), m = o / RF % MR, r = o % RF;
        const int64_t f = (int64_t(blockIdx.x) * GROUPS + grp) * RF + r;
        if (m >= g.M || f >= g.F) continue;
        float s[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            s[t] = red[grp * WKW][(t * MR + m) * RF + r];
            for (int q = 1; q < WKW; q++) s[t] += red[grp * WKW + q][(t * MR + m) * RF + r];
        }
        finish(g, m, f, s[0], s[1]);
    }
}

// Weights K x F: a lane owns four columns of both weights, LC lanes a stretch
// of 4 LC columns, and the 64 / LC lane groups of the waves deal out K in blocks
// of four rows, whose X values are then one load per row of X.
template <int MR, int LC, int NW>
__global__ void __launch_bounds__(64 * NW)
glu_thin_kf(GluArgs g) {
    constexpr bool XPRE = MR <= 2;
    constexpr int MX = MR < 8 ? MR : 8;
    constexpr int KG = 64 / LC, V = 8 * MR, HELD = V / KG > 0 ? V / KG : 1;
    __shared__ float red[NW][LC][V];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int lc = lane % LC, kg = lane / LC;
    // Neighbouring stretches on one XCD: where they share a cache line its L2
    // then brings it in once.
    const int q8 = gridDim.x / 8, r8 = gridDim.x % 8, x8 = blockIdx.x % 8;
    const int64_t tile = x8 * q8 + (x8 < r8 ? x8 : r8) + blockIdx.x / 8;
    const int64_t c0 = tile * (4 * LC) + lc * 4;
    // Lanes at the end of a row take its last four columns again.
    const int64_t c = c0 + 4 <= g.F ? c0 : g.F - 4;
    const auto xrow = [&](int m) { return g.X + (m < g.M ? m : g.M - 1) * g.ldx; };
    float acc[V];  // [matrix][row of X][column]
#pragma unroll
    for (int i = 0; i < V; i++) acc[i] = 0.0f;
    // MX rows of X from row mg on.
    auto add = [&](const v4f (&wv)[2][4], const v4f (&xv)[MX], int mg) {
#pragma unroll
        for (int q = 0; q < 4; q++)
#pragma unroll
            for (int t = 0; t < 2; t++)
#pragma unroll
                for (int m = 0; m < MX; m++)
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        float& a = acc[(t * MR + mg + m) * 4 + e];
                        a = fmaf(xv[m][q], wv[t][q][e], a);
                    }
    };
    auto loadw = [&](v4f (&wv)[2][4], int64_t k) {
#pragma unroll
        for (int q = 0; q < 4; q++) {
            wv[0][q] = load4(g.Wg + (k + q) * g.ldw + c);
            wv[1][q] = load4(g.Wu + (k + q) * g.ldw + c);
        }
    };
    const int64_t step = 4 * KG * NW;
    int64_t k = (int64_t(w) * KG + kg) * 4;
    auto loadx = [&](v4f (&xv)[MX], int64_t at, int mg) {
#pragma unroll
        for (int m = 0; m < MX; m++) xv[m] = load4(xrow(mg + m) + at);
    };
    v4f wv[2][4], xv[MX];
    if (k + 4 <= g.K) {
        loadw(wv, k);
        if (XPRE) loadx(xv, k, 0);
    }
    for (; k + 4 <= g.K; k += step) {
        v4f wn[2][4], xn[MX];
        const bool more = k + step + 4 <= g.K;
        if (!XPRE) loadx(xv, k, 0);
        if (more) {
            loadw(wn, k + step);
            if (XPRE) loadx(xn, k + step, 0);
        }
        add(wv, xv, 0);
#pragma unroll
        for (int mg = MX; mg < MR; mg += MX) {
            loadx(xv, k, mg);
            add(wv, xv, mg);
        }
        if (more) {
#pragma unroll
            for (int q = 0; q < 4; q++) wv[0][q] = wn[0][q], wv[1][q] = wn[1][q];
#pragma unroll
            for (int m = 0; m < MX && XPRE; m++) xv[m] = xn[m];
        }
    }
    if (k < g.K) {  // the last, incomplete block of rows
#pragma unroll
        for (int q = 0; q < 4; q++) {
            const bool in = k + q < g.K;
            wv[0][q] = in ? load4(g.Wg + (k + q) * g.ldw + c) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
            wv[1][q] = in ? load4(g.Wu + (k + q) * g.ldw + c) : v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
#pragma unroll
        for (int mg = 0; mg < MR; mg += MX) {
#pragma unroll
            for (int m = 0; m < MX; m++) xv[m] = load4_tail(xrow(mg + m), k, g.K);
            add(wv, xv, mg);
        }
    }
    const int first = reduce_lanes<32, LC, V>(acc, lane);
#pragma unroll
    for (int i = 0; i < HELD; i++) red[w][lc][first + i] = acc[i];
    __syncthreads();
    for (int o = threadIdx.x; o < MR * LC * 4; o += blockDim.x) {
        const int m = o / (LC * 4), l = o / 4 % LC, e = o % 4;
        const int64_t l0 = tile * (4 * LC) + l * 4;
        if (m >= g.M || l0 >= g.F) continue;
        const int64_t f = (l0 + 4 <= g.F ? l0 : g.F - 4) + e;
        if (f < l0) continue;  // another lane's column
        float s[2];
#pragma unroll
        for (int t = 0; t < 2; t++) {
            s[t] = red[0][l][(t * MR + m) * 4 + e];
            for (int q = 1; q < NW; q++) s[t] += red[q][l][(t * MR + m) * 4 + e];
        }
        finish(g, m, f, s[0], s[1]);
    }
}

// Waves share K, in steps of 256, until there are two workgroups per CU.
template <int MR, int RF>
static hipError_t launch_thin_fk(const GluArgs& g, hipStream_t s) {
    int w = 1;
    while (w < kThinWaves && ceil_div(g.F, RF * kThinWaves / w) < 512 && g.K >= 512 * w) w *= 2;
    const dim3 grid(unsigned(ceil_div(g.F, RF * kThinWaves / w))), block(64 * kThinWaves);
    switch (w) {
        case 1: hipLaunchKernelGGL((glu_thin_fk<MR, RF, 1>), grid, block, 0, s, g); break;
        case 2: hipLaunchKernelGGL((glu_thin_fk<MR, RF, 2>), grid, block, 0, s, g); break;
        case 4: hipLaunchKernelGGL((glu_thin_fk<MR, RF, 4>), grid, block, 0, s, g); break;
        default: hipLaunchKernelGGL((glu_thin_fk<MR, RF, 8>), grid, block, 0, s, g); break;
    }
    return hipGetLastError();
}

template <int MR>
static hipError_t launch_thin_mr(const GluArgs& g, hipStream_t s) {
    if (g.transw) {
        // Four rows of the weights a wave reuse its X more, two leave more
        // waves resident: 8 x 8192 x 4096 54.9 us against 60.4, 5 x 4099 x 2047
        // 26.9 against 20.7, 8 x 1024 x 1024 6.1 against 5.0.
        if constexpr (MR >= 4) {
            if (g.F >= 6144) return launch_thin_fk<MR, 4>(g, s);
        }
        return launch_thin_fk<MR, 2>(g, s);
    } else {
        constexpr int NW = MR <= 2 ? 16 : 8;
        // Stretches of 16 columns (64 bytes) occupy the CUs of outputs up to
        // 6144 wide (8 x 4096 x 4096 44 -> 38 us), if they are aligned; those of
        // unaligned rows straddle two cache lines each (7 x 4099 x 2047 26 -> 29)
        // and keep 32.
        const bool lines = (reinterpret_cast<uintptr_t>(g.Wg) | reinterpret_cast<uintptr_t>(g.Wu)) % 64 == 0 && g.ldw % 16 == 0;
        if (g.F < 6144 && lines)
            hipLaunchKernelGGL((glu_thin_kf<MR, 4, NW>), dim3(unsigned(ceil_div(g.F, 16))), dim3(64 * NW), 0, s, g);
        else
            hipLaunchKernelGGL((glu_thin_kf<MR, 8, NW>), dim3(unsigned(ceil_div(g.F, 32))), dim3(64 * NW), 0, s, g);
    }
    return hipGetLastError();
}

bool glu_thin_ok(const GluArgs& g) {
    // The grids' work-items (at most 256 and 32 per row or column of weights)
    // stay below 2^32.
    if (g.F >= (int64_t(1) << 24)) return false;
    if (g.transw) return g.M <= 16;
    // Weights K x F, 9 to 16 rows: few columns occupy too few workgroups of that
    // many sums (9 x 1024 x 1024 11.2 us, 9.3 on matrix tiles).
    return g.F >= 4 && (g.M <= 8 || (g.M <= 16 && g.K * g.F >= (int64_t(1) << 22)));
}

hipError_t launch_glu_thin(const GluArgs& g, hipStream_t s) {
    if (g.M == 1) return launch_thin_mr<1>(g, s);
    if (g.M == 2) return launch_thin_mr<2>(g, s);
    if (g.M <= 4) return launch_thin_mr<4>(g, s);
    if (g.M <= 8) return launch_thin_mr<8>(g, s);
    return launch_thin_mr<16>(g, s);
}

// dG and dU; each may be stored over G, U or dH (every lane reads its three
// inputs before it stores, and no other lane reads them).  A lane takes four
// columns of a row at a time: five streams of one access each, bound by memory
// (20 bytes per element).
__global__ void __launch_bounds__(256)
glu_pregrad(int act, int64_t M, int64_t F, const float* G, const float* U, int64_t ldgu,
            const float* dH, int64_t lddh, float* dG, float* dU, int64_t lddgu, int64_t strips,
            int64_t tiles) {
    typedef float v4u __attribute__((ext_vector_type(4), aligned(4)));
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t r = t / strips, c = (t - r * strips) * 1024 + threadIdx.x * 4;
        const float *gp = G + r * ldgu + c, *up = U + r * ldgu + c, *hp = dH + r * lddh + c;
        float *gq = dG + r * lddgu + c, *uq = dU + r * lddgu + c;
        float a, da;
        if (c + 4 <= F) {
            const v4u g = *(const v4u*)gp, u = *(const v4u*)up, d = *(const v4u*)hp;
            v4u og, ou;
#pragma unroll
            for (int e = 0; e < 4; e++) {
                act_grad(act, g[e], &a, &da);
                og[e] = d[e] * u[e] * da;
                ou[e] = d[e] * a;
            }
            *(v4u*)gq = og;
            *(v4u*)uq = ou;
        } else {
            for (int64_t e = 0; c + e < F; e++) {
                const float d = hp[e], u = up[e];
                act_grad(act, gp[e], &a, &da);
                gq[e] = d * u * da;
                uq[e] = d * a;
            }
        }
    }
}

static hipError_t launch_glu_pregrad(const GluGradArgs& g, hipStream_t s) {
    const int64_t strips = ceil_div(g.F, 1024), tiles = g.M * strips;
    hipLaunchKernelGGL(glu_pregrad, dim3(grid_for(tiles)), dim3(256), 0, s, g.act, g.M, g.F, g.G, g.U,
                       g.ldgu, g.dH, g.lddh, g.dG, g.dU, g.lddgu, strips, tiles);
    return hipGetLastError();
}

// C = A B (+ beta C) by the shape-chosen matrix path, whatever the sizes.
static hipError_t product(bool ta, bool tb, int64_t M, int64_t N, int64_t K, const float* A,
                          int64_t lda, const float* B, int64_t ldb, float beta, float* C,
                          int64_t ldc, hipStream_t s) {
    if (M == 0 || N == 0) return hipSuccess;
    if (K == 0) return launch_scale(C, M, N, ldc, beta, s);
    GemmArgs g{M, N, K, A, lda, B, ldb, C, ldc};
    g.trans_a = ta;
    g.trans_b = tb;
    g.beta = beta;
    g.pack_long = true;
    return k4_supports(g) ? launch_k4_mfma(g, s) : launch_k1_general(g, s);
}

hipError_t launch_glu_backward(const GluGradArgs& g, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (g.M > 0 && g.F > 0 && (e = launch_glu_pregrad(g, s)) != hipSuccess) return e;
    // Halves of one buffer, [dG | dU], make the pair of products one product
    // with both halves along its K (dX) or its M or N (dW).
    const bool d_pair = g.dU == g.dG + g.F && g.lddgu >= 2 * g.F;
    if (g.dX) {
        // One sum over 2F for dX up to the length of sum the separate products
        // have at F = 8192: beyond it, the longer float sums cost accuracy
        // (4096 x 8192 x 4096: 2.3e-6 of dX's size in one sum, 1.6e-6 in two)
        // and the second product's pass over dX little time (20 us of 7.5 ms).
        const bool w_pair = g.transw ? g.Wu == g.Wg + g.F * g.ldw
                                     : g.Wu == g.Wg + g.F && g.ldw >= 2 * g.F;
        if (d_pair && w_pair && g.F <= 4096) {
            e = product(false, !g.transw, g.M, g.K, 2 * g.F, g.dG, g.lddgu, g.Wg, g.ldw, 0.0f, g.dX,
                        g.lddx, s);
        } else {
            e = product(false, !g.transw, g.M, g.K, g.F, g.dG, g.lddgu, g.Wg, g.ldw, 0.0f, g.dX,
                        g.lddx, s);
            if (e == hipSuccess)
                e = product(false, !g.transw, g.M, g.K, g.F, g.dU, g.lddgu, g.Wu, g.ldw, 1.0f, g.dX,
                            g.lddx, s);
        }
        if (e != hipSuccess) return e;
    }
    if (g.dWg) {
        if (g.transw) {  // dW (F x K) = dG^T X
            const bool pair = d_pair && g.dWu == g.dWg + g.F * g.lddw;
            e = product(true, false, pair ? 2 * g.F : g.F, g.K, g.M, g.dG, g.lddgu, g.X, g.ldx, g.beta,
                        g.dWg, g.lddw, s);
            if (e == hipSuccess && !pair)
                e = product(true, false, g.F, g.K, g.M, g.dU, g.lddgu, g.X, g.ldx, g.beta, g.dWu,
                            g.lddw, s);
        } else {  // dW (K x F) = X^T dG
            const bool pair = d_pair && g.dWu == g.dWg + g.F && g.lddw >= 2 * g.F;
            e = product(true, false, g.K, pair ? 2 * g.F : g.F, g.M, g.X, g.ldx, g.dG, g.lddgu, g.beta,
                        g.dWg, g.lddw, s);
            if (e == hipSuccess && !pair)
                e = product(true, false, g.K, g.F, g.M, g.X, g.ldx, g.dU, g.lddgu, g.beta, g.dWu,
                            g.lddw, s);
        }
    }
    return e;
}

}  // namespace sgemm
