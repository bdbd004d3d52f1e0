// Products with 4-bit weights: the general kernel, and the choice between it
// and the kernels of q4_kernels.h.
#include "activation.h"
#include "kernels.h"
#include "q4_elements.h"

namespace sgemm {

static __device__ __forceinline__ float load_float(int type, const void* p, int64_t i) {
    return raw_to_float(type, load_raw(type, p, i));
}

// Any strides and sizes (64-bit offsets): one output per wave, four groups at a
// time, their K dealt to the lanes.  The fallback for operands whose rows are
// too long for the 32-bit offsets of the kernels above.  A group's whole sum
// meets its scale: lanes without a part of it (groups of 32) would make NaN of
// an infinite one.  The four sums meet by halving exchanges, seven in all, and
// lanes 16 i .. hold group i's (8 x 4096 x 4096, float16: groups of 32 321 us, of
// 128 122; with every lane scaling its part of each group 333 and 126; one
// group's exchanges at a time 443 and 150).
__global__ void __launch_bounds__(64)
q4_general(Q4Args g, int64_t tiles) {
    const int64_t group = int64_t(1) << g.shift, groups = (g.K + group - 1) >> g.shift;
    const int lane = threadIdx.x;
    for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
        const int64_t m = t / g.N, n = t % g.N;
        float out[2] = {0.0f, 0.0f};
        for (int w = 0; w < (g.act >= 0 ? 2 : 1); w++) {
            float sum = 0.0f;
            for (int64_t q0 = 0; q0 < groups; q0 += 4) {
                float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int64_t q = q0 + i;
                    if (q >= groups) break;
                    const int64_t k0 = q << g.shift, k1 = k0 + group < g.K ? k0 + group : g.K;
                    const int z = g.Z[w] ? g.Z[w][n * g.ldz + q] : 8;
                    for (int64_t k = k0 + lane; k < k1; k += 64) {
                        const int b = g.W[w][n * g.ldw + k / 2];
                        const int v = (k & 1 ? b >> 4 : b & 15) - z;
                        part[i] = fmaf(load_float(g.xtype, g.X, m * g.ldx + k), float(v), part[i]);
                    }
                }
                const bool hi = lane & 32, odd = lane & 16;
                const float a = (hi ? part[2] : part[0]) + __shfl_xor(hi ? part[0] : part[2], 32);
                const float b = (hi ? part[3] : part[1]) + __shfl_xor(hi ? part[1] : part[3], 32);
                float d = (odd ? b : a) + __shfl_xor(odd ? a : b, 16);
                for (int o = 8; o > 0; o >>= 1) d += __shfl_xor(d, o);
                const int64_t q = q0 + lane / 16;
                if (q < groups) sum = fmaf(load_float(g.stype, g.S[w], n * g.lds + q), d, sum);
            }
            sum += __shfl_xor(sum, 32);
            sum += __shfl_xor(sum, 16);
            out[w] = sum;
        }
        const float y = g.act >= 0 ? act_value(g.act, out[0]) * out[1] : out[0];
        const int64_t at = m * g.ldy + n;
        if (threadIdx.x == 0) {
            if (g.xtype == T_F32) store_as<T_F32>(g.Y, at, y);
            else if (g.xtype == T_F16) store_as<T_F16>(g.Y, at, y);
            else store_as<T_BF16>(g.Y, at, y);
        }
    }
}

// The kernels of q4_kernels.h, by type of X and form (q4_f32.hip, q4_glu_f32.hip,
// ...): NWT 1 the product, 2 the gated form.
template <int XT, int NWT> hipError_t launch_q4_kernels(const Q4Args& g, hipStream_t s);

// Whether a tile's 32-bit offsets reach every operand.
static bool offsets_fit(const Q4Args& g) {
    const int64_t lim = int64_t(1) << 31;
    return g.K < lim - 128 && 256 * g.ldw < lim && 256 * 4 * g.lds < lim && 256 * g.ldz < lim &&
           128 * 4 * g.ldx < lim && 32 * g.ldy < lim && ceil_div(g.M, 8) * ceil_div(g.N, 16) < lim / 2;
}

hipError_t launch_q4(const Q4Args& a, hipStream_t s) {
    Q4Args g = a;
    if (g.K == 0 || !offsets_fit(g)) {
        const int64_t tiles = g.M * g.N;
        hipLaunchKernelGGL(q4_general, dim3(grid_for(tiles)), dim3(64), 0, s, g, tiles);
        return hipGetLastError();
    }
    // The kernels shift 32-bit positions: a group longer than any row they take
    // is one group all the same.
    if (g.shift > 30) g.shift = 30;
    const bool two = g.act >= 0;
    switch (g.xtype) {
        case T_F32: return two ? launch_q4_kernels<T_F32, 2>(g, s) : launch_q4_kernels<T_F32, 1>(g, s);
        case T_F16: return two ? launch_q4_kernels<T_F16, 2>(g, s) : launch_q4_kernels<T_F16, 1>(g, s);
        default: return two ? launch_q4_kernels<T_BF16, 2>(g, s) : launch_q4_kernels<T_BF16, 1>(g, s);
    }
}

}  // namespace sgemm
