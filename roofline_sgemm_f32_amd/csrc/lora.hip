// Low-rank adapters beside a projection, and their gradients: one output per
// lane (or wave, for the sums along K and N).
#include "kernels.h"

namespace sgemm {
namespace {

__device__ __forceinline__ float load_as(int type, const void* p, int64_t i) {
    if (type == T_F32) return static_cast<const float*>(p)[i];
    if (type == T_F16) return float(static_cast<const _Float16*>(p)[i]);
    return float(static_cast<const __bf16*>(p)[i]);
}
__device__ __forceinline__ void store_to(int type, void* p, int64_t i, float v) {
    if (type == T_F32) static_cast<float*>(p)[i] = v;
    else if (type == T_F16) static_cast<_Float16*>(p)[i] = _Float16(v);
    else static_cast<__bf16*>(p)[i] = __bf16(v);
}
// Row m's adapter, or -1.
__device__ __forceinline__ int adapter_of(const LoraArgs& g, int64_t m) {
    if (!g.ids) return 0;
    const int64_t id = g.id64 ? static_cast<const int64_t*>(g.ids)[m] : static_cast<const int32_t*>(g.ids)[m];
    return id >= 0 && id < g.L ? int(id) : -1;
}
__device__ __forceinline__ float scale_of(const LoraArgs& g, int l) { return g.alpha * (g.scales ? g.scales[l] : 1.0f); }
__device__ __forceinline__ float wave_sum(float v) {
    for (int d = 32; d; d /= 2) v += __shfl_xor(v, d);
    return v;
}

// H[m, r] = sum_k X[m, k] A[r, k], a wave each; dh: sum_n dY[m, n] B[n, r] scaled.
__global__ void __launch_bounds__(256) lora_reduce(LoraArgs g, float* out, int64_t ldo, bool dh) {
    const int lane = threadIdx.x % 64;
    for (int64_t t = blockIdx.x * 4 + threadIdx.x / 64; t < g.M * g.R; t += int64_t(gridDim.x) * 4) {
        const int64_t m = t / g.R;
        const int r = int(t % g.R), l = adapter_of(g, m);
        float v = 0.0f;
        if (l >= 0) {
            if (dh)
                for (int64_t n = lane; n < g.N; n += 64)
                    v = fmaf(load_as(g.type, g.Y, m * g.ldy + n), load_as(g.type, g.B, l * g.sb + n * g.ldb + r), v);
            else
                for (int64_t k = lane; k < g.K; k += 64)
                    v = fmaf(load_as(g.type, g.X, m * g.ldx + k), load_as(g.type, g.A, l * g.sa + r * g.lda + k), v);
            v = wave_sum(v);
            if (dh) v *= scale_of(g, l);
        }
        if (lane == 0) out[m * ldo + r] = v;
    }
}

// Y = base + scale H B^T (rows of H: ldh), or dX = base + dH A.
__global__ void __launch_bounds__(256) lora_expand(LoraArgs g, const float* H, int64_t ldh, void* out, int64_t ldo,
                                                   int64_t cols, bool dx) {
    for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < g.M * cols; t += int64_t(gridDim.x) * 256) {
        const int64_t m = t / cols, n = t % cols;
        const int l = adapter_of(g, m);
        float v = 0.0f;
        if (l >= 0) {
            for (int r = 0; r < g.R; r++)
                v = fmaf(H[m * ldh + r], dx ? load_as(g.type, g.A, l * g.sa + r * g.lda + n)
                                            : load_as(g.type, g.B, l * g.sb + n * g.ldb + r), v);
            if (!dx) v *= scale_of(g, l);
        }
        if (g.base) v = load_as(g.type, g.base, m * g.ldbase + n) + v;
        store_to(g.type, out, m * ldo + n, v);
    }
}

// dA[l, r, k] = sum dH[m, r] X[m, k], or dB[l, n, r] = scale sum dY[m, n] H[m, r].
__global__ void __launch_bounds__(256) lora_weights(LoraArgs g, const float* V, int64_t ldv, void* out, int64_t ldo,
                                                    int64_t so, int64_t cols, bool db) {
    const int64_t total = int64_t(g.L) * g.R * cols;
    for (int64_t t = blockIdx.x * 256 + threadIdx.x; t < total; t += int64_t(gridDim.x) * 256) {
        const int64_t c = t % cols;
        const int r = int(t / cols % g.R), l = int(t / cols / g.R);
        float v = 0.0f;
        for (int64_t m = 0; m < g.M; m++)
            if (adapter_of(g, m) == l)
                v = fmaf(V[m * ldv + r], db ? load_as(g.type, g.Y, m * g.ldy + c) : load_as(g.type, g.X, m * g.ldx + c), v);
        if (db) store_to(g.type, out, l * so + c * ldo + r, v * scale_of(g, l));
        else store_to(g.type, out, l * so + r * ldo + c, v);
    }
}

}  // namespace

size_t lora_workspace_bytes(bool, int, int64_t M, int64_t, int64_t, int R, int) { return size_t(M) * R * sizeof(float); }

hipError_t launch_lora(const LoraArgs& g, hipStream_t s) {
    float* H = g.H ? g.H : static_cast<float*>(g.ws);
    const int64_t ldh = g.H ? g.ldh : g.R;
    hipLaunchKernelGGL(lora_reduce, dim3(grid_for(ceil_div(g.M * g.R, 4))), dim3(256), 0, s, g, H, ldh, false);
    if (g.N > 0)
        hipLaunchKernelGGL(lora_expand, dim3(grid_for(ceil_div(g.M * g.N, 256))), dim3(256), 0, s, g, H, ldh, g.Y, g.ldy, g.N, false);
    return hipGetLastError();
}

hipError_t launch_lora_backward(const LoraGradArgs& b, hipStream_t s) {
    const LoraArgs& g = b.f;
    float* dH = static_cast<float*>(g.ws);
    if (g.M > 0 && (b.dX || b.dA))
        hipLaunchKernelGGL(lora_reduce, dim3(grid_for(ceil_div(g.M * g.R, 4))), dim3(256), 0, s, g, dH, int64_t(g.R), true);
    if (b.dX && g.M > 0 && g.K > 0)
        hipLaunchKernelGGL(lora_expand, dim3(grid_for(ceil_div(g.M * g.K, 256))), dim3(256), 0, s, g, dH, int64_t(g.R), b.dX, b.lddx, g.K, true);
    if (b.dA && g.K > 0)
        hipLaunchKernelGGL(lora_weights, dim3(grid_for(ceil_div(int64_t(g.L) * g.R * g.K, 256))), dim3(256), 0, s, g, dH, int64_t(g.R), b.dA, b.ldda, b.sda, g.K, false);
    if (b.dB && g.N > 0)
        hipLaunchKernelGGL(lora_weights, dim3(grid_for(ceil_div(int64_t(g.L) * g.R * g.N, 256))), dim3(256), 0, s, g, g.H, g.ldh, b.dB, b.lddb, b.sdb, g.N, true);
    return hipGetLastError();
}

}  // namespace sgemm
