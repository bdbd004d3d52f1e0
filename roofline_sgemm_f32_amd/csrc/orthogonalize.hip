// Orthogonalised updates by Newton-Schulz products, on the library's float32
// products.
#include <cmath>

#include "kernels.h"

namespace sgemm {
namespace {

__device__ __forceinline__ float load_as(int type, const void* p, int64_t i) {
    if (type == T_F32) return static_cast<const float*>(p)[i];
    if (type == T_F16) return float(static_cast<const _Float16*>(p)[i]);
    return float(static_cast<const __bf16*>(p)[i]);
}

// out = the sum of squares of G, one workgroup.
__global__ void __launch_bounds__(1024) ortho_norm(int type, const void* G, int64_t M, int64_t N, int64_t ldg, double* out) {
    __shared__ double part[1024];
    double v = 0;
    for (int64_t t = threadIdx.x; t < M * N; t += 1024) {
        const double x = load_as(type, G, t / N * ldg + t % N);
        v += x * x;
    }
    part[threadIdx.x] = v;
    __syncthreads();
    for (int d = 512; d; d /= 2) {
        if (threadIdx.x < d) part[threadIdx.x] += part[threadIdx.x + d];
        __syncthreads();
    }
    if (threadIdx.x == 0) *out = part[0];
}

__global__ void __launch_bounds__(256) ortho_scale(int type, const void* G, int64_t M, int64_t N, int64_t ldg, const double* sq, double eps, float* X) {
    const double f = 1.0 / (sqrt(*sq) + eps);
    for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < M * N; t += int64_t(gridDim.x) * 256) {
        const double x = load_as(type, G, t / N * ldg + t % N);
        X[t] = x == 0 ? 0.0f : float(x * f);
    }
}

__global__ void __launch_bounds__(256) ortho_copy(const float* src, float* dst, int64_t n) {
    for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < n; t += int64_t(gridDim.x) * 256) dst[t] = src[t];
}

__global__ void __launch_bounds__(256) ortho_out(int type, const float* X, int64_t M, int64_t N, void* O, int64_t ldo) {
    for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < M * N; t += int64_t(gridDim.x) * 256) {
        const int64_t i = t / N * ldo + t % N;
        if (type == T_F32) static_cast<float*>(O)[i] = X[t];
        else if (type == T_F16) static_cast<_Float16*>(O)[i] = _Float16(X[t]);
        else static_cast<__bf16*>(O)[i] = __bf16(X[t]);
    }
}

}  // namespace

size_t ortho_workspace_bytes(int64_t, int64_t M, int64_t N) {
    const int64_t m = M < N ? M : N;
    return 256 + sizeof(float) * size_t(2 * M * N + 2 * m * m);
}

hipError_t launch_orthogonalize(const OrthoArgs& g, hipStream_t s) {
    const int64_t M = g.M, N = g.N, m = M < N ? M : N, n = M * N;
    double* sq = static_cast<double*>(g.ws);
    float* X = reinterpret_cast<float*>(static_cast<char*>(g.ws) + 256);
    float *X2 = X + n, *S = X2 + n, *P = S + m * m;
    const bool left = M <= N;
    auto mm = [&](GemmArgs a) { return k4_supports(a) ? launch_k4_mfma(a, s, 1) : launch_k1_general(a, s); };
    const size_t es = g.type == T_F32 ? 4 : 2;
    for (int64_t b = 0; b < g.batch; b++) {
        const char* G = static_cast<const char*>(g.G) + b * g.sg * es;
        hipLaunchKernelGGL(ortho_norm, dim3(1), dim3(1024), 0, s, g.type, G, M, N, g.ldg, sq);
        hipLaunchKernelGGL(ortho_scale, dim3(grid_for(ceil_div(n, 256))), dim3(256), 0, s, g.type, G, M, N, g.ldg, sq, g.eps, X);
        for (int i = 0; i < g.steps; i++) {
            hipError_t e;
            GemmArgs q{m, m, left ? N : M, X, N, X, N, S, m};
            q.trans_a = !left;
            q.trans_b = left;
            if ((e = mm(q)) != hipSuccess) return e;
            hipLaunchKernelGGL(ortho_copy, dim3(grid_for(ceil_div(m * m, 256))), dim3(256), 0, s, S, P, m * m);
            GemmArgs p{m, m, m, S, m, S, m, P, m};
            p.alpha = float(g.coef[3 * i + 2]);
            p.beta = float(g.coef[3 * i + 1]);
            if ((e = mm(p)) != hipSuccess) return e;
            hipLaunchKernelGGL(ortho_copy, dim3(grid_for(ceil_div(n, 256))), dim3(256), 0, s, X, X2, n);
            GemmArgs x{M, N, m, left ? P : X, left ? m : N, left ? X : P, left ? N : m, X2, N};
            x.beta = float(g.coef[3 * i]);
            if ((e = mm(x)) != hipSuccess) return e;
            std::swap(X, X2);
        }
        char* O = static_cast<char*>(g.O) + b * g.so * es;
        hipLaunchKernelGGL(ortho_out, dim3(grid_for(ceil_div(n, 256))), dim3(256), 0, s, g.type, X, M, N, O, g.ldo);
    }
    return hipGetLastError();
}

}  // namespace sgemm
