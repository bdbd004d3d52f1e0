// Products with 4-bit weights:
//   Y[m, n] = sum_g s[n, g] sum_{k in group g} X[m, k] (q[n, k] - z[n, g]),
// q two to a byte along K (low half first), groups of 2^shift along K, and
// the gated form H = act(G) * U of two such products.
#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "activation.h"
#include "kernels.h"

namespace sgemm {

namespace {
__device__ __forceinline__ float load_as_float(const void* p, int type, int64_t i) {
    if (type == T_F32) return static_cast<const float*>(p)[i];
    if (type == T_F16) return __half2float(static_cast<const __half*>(p)[i]);
    return __uint_as_float(uint32_t(static_cast<const uint16_t*>(p)[i]) << 16);
}

__device__ __forceinline__ void store_from_float(void* p, int type, int64_t i, float v) {
    if (type == T_F32) static_cast<float*>(p)[i] = v;
    else if (type == T_F16) static_cast<__half*>(p)[i] = __float2half(v);
    else static_cast<__hip_bfloat16*>(p)[i] = __float2bfloat16(v);
}
}  // namespace

// One output per wave: its lanes take groups in turn, and their sums are
// added across the wave.
__global__ void __launch_bounds__(64)
q4_general(Q4Args g, int64_t tiles) {
    const int64_t group = int64_t(1) << g.shift, groups = (g.K + group - 1) >> g.shift;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m = t / g.N, n = t % g.N;
        float out[2] = {0.0f, 0.0f};
        for (int w = 0; w < (g.act >= 0 ? 2 : 1); w++) {
            float sum = 0.0f;
            for (int64_t q = 0; q < groups; q++) {
                const int64_t k0 = q << g.shift, k1 = k0 + group < g.K ? k0 + group : g.K;
                const int z = g.Z[w] ? g.Z[w][n * g.ldz + q] : 8;
                float part = 0.0f;
                for (int64_t k = k0 + threadIdx.x; k < k1; k += 64) {
                    const int b = g.W[w][n * g.ldw + k / 2];
                    const int v = (k & 1 ? b >> 4 : b & 15) - z;
                    part = fmaf(load_as_float(g.X, g.xtype, m * g.ldx + k), float(v), part);
                }
                sum = fmaf(load_as_float(g.S[w], g.stype, n * g.lds + q), part, sum);
            }
            for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
            out[w] = sum;
        }
        if (threadIdx.x == 0)
            store_from_float(g.Y, g.xtype, m * g.ldy + n,
                             g.act >= 0 ? act_value(g.act, out[0]) * out[1] : out[0]);
    }
}

hipError_t launch_q4(const Q4Args& g, hipStream_t s) {
    const int64_t tiles = g.M * g.N;
    hipLaunchKernelGGL(q4_general, dim3(grid_for(tiles)), dim3(64), 0, s, g, tiles);
    return hipGetLastError();
}

}  // namespace sgemm
