// Low-rank adapters beside a projection, and their gradients: one output per
// lane (or wave, for the sums along K and N).
#include "lora.h"
#include "lora_kernels.h"

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

namespace {

// Sizes of a forward pass's launches and of its workspace.
struct ForwardPlan {
    RowPlan::Mode mode;
    int tmb;                 // 16-row blocks of a tile
    int64_t tiles;           // at most this many
    int planes;
    int64_t kshare, nshare;
    size_t p_at, order_at, tiles_at, bytes;
};

size_t align_up(size_t n) { return (n + 255) / 256 * 256; }

ForwardPlan forward_plan(int type, bool ids, int64_t M, int64_t N, int64_t K, int R, int L) {
    ForwardPlan p{};
    const int64_t adapters = L < M ? L : M;
    p.mode = !ids ? RowPlan::UNIFORM : M <= 64 ? RowPlan::SINGLE : RowPlan::SORTED;
    p.tmb = p.mode == RowPlan::SINGLE || M / (ids ? adapters : 1) < 32 ? 1 : 4;
    const int tile = 16 * p.tmb;
    p.tiles = p.mode == RowPlan::SINGLE ? M : ceil_div(M, tile) + (ids ? adapters + 1 : 0);
    const int64_t busy = p.mode == RowPlan::SINGLE ? M : ceil_div(M, tile);
    const int64_t kunit = type == T_F32 ? 128 : 256;  // four waves' double steps
    int64_t planes = ceil_div(512, busy), most = ceil_div(K, kunit);
    planes = planes > most ? most : planes;
    planes = planes > 16 ? 16 : planes < 1 ? 1 : planes;
    p.kshare = K > 0 ? ceil_div(ceil_div(K, planes), kunit) * kunit : 1;
    p.planes = int(K > 0 ? ceil_div(K, p.kshare) : 1);
    const int64_t nunit = p.tmb == 1 ? 256 : 64;
    int64_t shares = ceil_div(1024, busy), top = ceil_div(N, nunit);
    shares = shares > top ? top : shares;
    shares = shares < 1 ? 1 : shares > 4096 ? 4096 : shares;
    p.nshare = N > 0 ? ceil_div(ceil_div(N, shares), nunit) * nunit : nunit;
    p.p_at = 0;
    p.order_at = align_up(size_t(p.planes) * M * lora_pitch(R) * sizeof(float));
    p.tiles_at = p.order_at + align_up(size_t(M) * sizeof(int));
    p.bytes = p.mode == RowPlan::SORTED ? p.tiles_at + align_up(size_t(4 + 4 * (p.tiles + 1)) * sizeof(int)) : p.order_at;
    return p;
}

template <int T, int TMB>
void shrink(const ShrinkArgs& a, int64_t tiles, int planes, hipStream_t s) {
    const dim3 block(64 * kShrinkWaves);
    const unsigned x = grid_for(tiles);
    if (a.R <= 16) hipLaunchKernelGGL((lora_shrink<T, 1, TMB>), dim3(x, planes, 1), block, 0, s, a);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_shrink<T, 2, TMB>), dim3(x, planes, 1), block, 0, s, a);
    else hipLaunchKernelGGL((lora_shrink<T, 4, TMB>), dim3(x, planes, (a.R + 63) / 64), block, 0, s, a);
}

template <int T, int TMB>
void expand(const ExpandArgs& a, int64_t tiles, hipStream_t s) {
    const dim3 grid(grid_for(tiles), unsigned(ceil_div(a.N > 0 ? a.N : 1, a.nshare)));
    const bool odd = a.R % kVec<T> != 0;
    if constexpr (TMB == 1) {
        const size_t lds = expand_lds<T>(a.R, 16 * TMB);
        auto run = [&](auto kind) {
            constexpr int KIND = decltype(kind)::value;
            if (odd) hipLaunchKernelGGL((lora_expand<T, TMB, KIND, true>), grid, dim3(256), lds, s, a);
            else hipLaunchKernelGGL((lora_expand<T, TMB, KIND, false>), grid, dim3(256), lds, s, a);
        };
        if (a.R > (T == T_F32 ? 32 : 64)) return run(std::integral_constant<int, EXPAND_LONG>{});
        if constexpr (T != T_F32)
            if (a.R <= 16) return run(std::integral_constant<int, EXPAND_PACKED>{});
        run(std::integral_constant<int, EXPAND_HELD>{});
    } else {
        auto run = [&](auto kind, auto sums) {
            constexpr int KIND = decltype(kind)::value, NS = decltype(sums)::value;
            if (odd) hipLaunchKernelGGL((lora_expand_tiles<T, KIND, NS, true>), grid, dim3(256), 0, s, a);
            else hipLaunchKernelGGL((lora_expand_tiles<T, KIND, NS, false>), grid, dim3(256), 0, s, a);
        };
        constexpr int PER = 4 * kVec<T>;  // ranks of a sum
        using H = std::integral_constant<int, EXPAND_HELD>;
        if constexpr (T != T_F32) {
            if (a.R <= 16) return run(std::integral_constant<int, EXPAND_PACKED>{}, std::integral_constant<int, 1>{});
        } else {
            if (a.R <= 16) return run(H{}, std::integral_constant<int, 1>{});
        }
        if (a.R <= 32) run(H{}, std::integral_constant<int, 32 / PER>{});
        else if (a.R <= 64) run(H{}, std::integral_constant<int, 64 / PER>{});
        else if (a.R <= 128) run(H{}, std::integral_constant<int, 128 / PER>{});
        else run(H{}, std::integral_constant<int, 256 / PER>{});
    }
}

template <int T>
hipError_t forward(const LoraArgs& g, const ForwardPlan& p, hipStream_t s) {
    char* const ws = static_cast<char*>(g.ws);
    RowPlan rows{p.mode, g.ids, g.id64, int(g.M), g.L, reinterpret_cast<int*>(ws + p.order_at),
                 reinterpret_cast<int*>(ws + p.tiles_at)};
    if (p.mode == RowPlan::SORTED) {
        GroupArgs a{g.ids, g.id64, int(g.M), g.L, 0, reinterpret_cast<int*>(ws + p.order_at), 16 * p.tmb,
                    reinterpret_cast<int*>(ws + p.tiles_at), 0, nullptr, nullptr};
        const hipError_t e = launch_lora_group(a, s);
        if (e != hipSuccess) return e;
    }
    float* P = reinterpret_cast<float*>(ws + p.p_at);
    const ShrinkArgs sh{g.X, g.ldx, g.A, g.lda, g.sa, g.K, g.R, nullptr, 1.0f, false, P, g.M * lora_pitch(g.R), p.kshare, rows, p.tiles};
    const ExpandArgs ex{P, g.M * lora_pitch(g.R), p.planes, g.R, g.B, g.ldb, g.sb, g.N, g.scales, g.alpha, true,
                        g.base, g.ldbase, g.Y, g.ldy, g.H, g.ldh, p.nshare, rows, p.tiles};
    if (p.tmb == 1) shrink<T, 1>(sh, p.tiles, p.planes, s), expand<T, 1>(ex, p.tiles, s);
    else shrink<T, 4>(sh, p.tiles, p.planes, s), expand<T, 4>(ex, p.tiles, s);
    return hipGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(bool backward, int type, int64_t M, int64_t N, int64_t K, int R, int L) {
    if (M == 0) return 0;
    if (backward) return size_t(M) * R * sizeof(float);
    const size_t a = forward_plan(type, false, M, N, K, R, L).bytes, b = forward_plan(type, true, M, N, K, R, L).bytes;
    return a > b ? a : b;
}

hipError_t launch_lora(const LoraArgs& g, hipStream_t s) {
    const ForwardPlan p = forward_plan(g.type, g.ids != nullptr, g.M, g.N, g.K, g.R, g.L);
    if (g.type == T_F32) return forward<T_F32>(g, p, s);
    if (g.type == T_F16) return forward<T_F16>(g, p, s);
    return forward<T_BF16>(g, p, s);
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
