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

// dG and dU; each may be stored over G, U or dH (every lane reads its three
// inputs before it stores).
__global__ void __launch_bounds__(256)
glu_pregrad(int act, int64_t M, int64_t F, const float* G, const float* U, int64_t ldgu,
            const float* dH, int64_t lddh, float* dG, float* dU, int64_t lddgu) {
    const int64_t total = M * F, stride = (int64_t)gridDim.x * blockDim.x;
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < total; i += stride) {
        const int64_t r = i / F, c = i % F;
        float a, da;
        act_grad(act, G[r * ldgu + c], &a, &da);
        const float d = dH[r * lddh + c], u = U[r * ldgu + c];
        dG[r * lddgu + c] = d * u * da;
        dU[r * lddgu + c] = d * a;
    }
}

hipError_t launch_glu_pregrad(const GluGradArgs& g, hipStream_t s) {
    hipLaunchKernelGGL(glu_pregrad, dim3(grid_for(ceil_div(g.M * g.F, 256))), dim3(256), 0, s,
                       g.act, g.M, g.F, g.G, g.U, g.ldgu, g.dH, g.lddh, g.dG, g.dU, g.lddgu);
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
    return k4_supports(g) ? launch_k4_mfma(g, s) : launch_k1_general(g, s);
}

hipError_t launch_glu_backward(const GluGradArgs& g, hipStream_t s) {
    hipError_t e = hipSuccess;
    if (g.M > 0 && g.F > 0 && (e = launch_glu_pregrad(g, s)) != hipSuccess) return e;
    // Halves of one buffer, [dG | dU], make the pair of products one product
    // with both halves along its K (dX) or its M or N (dW).
    const bool d_pair = g.dU == g.dG + g.F && g.lddgu >= 2 * g.F;
    if (g.dX) {
        const bool w_pair = g.transw ? g.Wu == g.Wg + g.F * g.ldw
                                     : g.Wu == g.Wg + g.F && g.ldw >= 2 * g.F;
        if (d_pair && w_pair) {
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
