// Low-rank adapters beside a projection: plan and launches.
#include "lora.h"
#include "lora_kernels.h"

namespace sgemm {
namespace {

template <int T, int TMB>
void shrink(const ShrinkArgs& a, const PassPlan& p, hipStream_t s) {
    const dim3 block(64 * kShrinkWaves);
    const unsigned x = grid_for(p.tiles);
    if (a.R <= 16) hipLaunchKernelGGL((lora_shrink<T, 1, TMB>), dim3(x, p.planes, 1), block, 0, s, a);
    else if (a.R <= 32) hipLaunchKernelGGL((lora_shrink<T, 2, TMB>), dim3(x, p.planes, 1), block, 0, s, a);
    else hipLaunchKernelGGL((lora_shrink<T, 4, TMB>), dim3(x, p.planes, (a.R + 63) / 64), block, 0, s, a);
}

// Tiles of 16 rows.
template <int T>
void expand_rows(const ExpandArgs& a, dim3 grid, hipStream_t s) {
    const size_t lds = expand_lds<T>(a.R);
    auto run = [&](auto kind) {
        constexpr int KIND = decltype(kind)::value;
        if (a.R % kVec<T> != 0) hipLaunchKernelGGL((lora_expand<T, KIND, true>), grid, dim3(256), lds, s, a);
        else hipLaunchKernelGGL((lora_expand<T, KIND, false>), grid, dim3(256), lds, s, a);
    };
    if (a.R > (T == T_F32 ? 32 : 64)) return run(std::integral_constant<int, EXPAND_LONG>{});
    if constexpr (T != T_F32)
        if (a.R <= 16) return run(std::integral_constant<int, EXPAND_PACKED>{});
    run(std::integral_constant<int, EXPAND_HELD>{});
}

// Single rows.
template <int T>
void expand_one(const ExpandArgs& a, dim3 grid, hipStream_t s) {
    constexpr int V = kVec<T>;
    auto run = [&](auto lanes) {
        constexpr int G = decltype(lanes)::value;
        if (a.R % V != 0) hipLaunchKernelGGL((lora_expand_one<T, G, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((lora_expand_one<T, G, false>), grid, dim3(256), 0, s, a);
    };
    if (a.R <= V) run(std::integral_constant<int, 1>{});
    else if (a.R <= 2 * V) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 4>{});
}

// Tiles of 64 rows.
template <int T>
void expand_tiles(const ExpandArgs& a, dim3 grid, hipStream_t s) {
    auto run = [&](auto kind, auto sums) {
        constexpr int KIND = decltype(kind)::value, NS = decltype(sums)::value;
        if (a.R % kVec<T> != 0) hipLaunchKernelGGL((lora_expand_tiles<T, KIND, NS, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((lora_expand_tiles<T, KIND, NS, false>), grid, dim3(256), 0, s, a);
    };
    constexpr int PER = 4 * kVec<T>;  // ranks of a sum
    using H = std::integral_constant<int, EXPAND_HELD>;
    if (a.R <= 16) {
        if constexpr (T == T_F32) run(H{}, std::integral_constant<int, 1>{});
        else run(std::integral_constant<int, EXPAND_PACKED>{}, std::integral_constant<int, 1>{});
    } else if (a.R <= 32) {
        run(H{}, std::integral_constant<int, 32 / PER>{});
    } else if (a.R <= 64) {
        run(H{}, std::integral_constant<int, 64 / PER>{});
    } else if (a.R <= 128) {
        run(H{}, std::integral_constant<int, 128 / PER>{});
    } else {
        run(H{}, std::integral_constant<int, 256 / PER>{});
    }
}

template <class F>
hipError_t by_type(int type, F f) {
    if (type == T_F32) f(std::integral_constant<int, T_F32>{});
    else if (type == T_F16) f(std::integral_constant<int, T_F16>{});
    else f(std::integral_constant<int, T_BF16>{});
    return hipGetLastError();
}

// Bound by its launch: 4 planes of 8192 x 64, 10 MB, 5 us, where every share of N would
// read them again.
__global__ void __launch_bounds__(256) lora_join(float* P, int64_t plane, int planes) {
    for (int64_t e = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4; e < plane; e += int64_t(gridDim.x) * 1024) {
        v4f v = *reinterpret_cast<const v4f*>(P + e);
#pragma unroll 4
        for (int z = 1; z < planes; z++) v += *reinterpret_cast<const v4f*>(P + z * plane + e);
        *reinterpret_cast<v4f*>(P + e) = v;
    }
}

}  // namespace

hipError_t launch_join(float* P, int64_t plane, int planes, hipStream_t s) {
    hipLaunchKernelGGL(lora_join, dim3(grid_for(ceil_div(plane, 1024))), dim3(256), 0, s, P, plane, planes);
    return hipGetLastError();
}

PassPlan pass_plan(int type, bool ids, bool single, int64_t M, int64_t N, int64_t K, int R, int L) {
    PassPlan p{};
    const int64_t adapters = L < M ? L : M;
    p.mode = !ids ? RowPlan::UNIFORM : single && M <= 64 ? RowPlan::SINGLE : RowPlan::SORTED;
    p.tmb = p.mode == RowPlan::SINGLE || M / (ids ? adapters : 1) < 32 ? 1 : 4;
    const int tile = 16 * p.tmb;
    p.tiles = p.mode == RowPlan::SINGLE ? M : ceil_div(M, tile) + (ids ? adapters + 1 : 0);
    const int64_t busy = p.mode == RowPlan::SINGLE ? M : ceil_div(M, tile);
    const int64_t kunit = type == T_F32 ? 128 : 256;  // four waves' double steps
    int64_t planes = ceil_div(512, busy), most = ceil_div(K, kunit);
    planes = planes > most ? most : planes;
    const int64_t cap = p.mode == RowPlan::SINGLE ? 8 : 16;
    planes = planes > cap ? cap : planes < 1 ? 1 : planes;
    p.kshare = K > 0 ? ceil_div(ceil_div(K, planes), kunit) * kunit : 1;
    p.planes = int(K > 0 ? ceil_div(K, p.kshare) : 1);
    const int64_t nunit = p.tmb == 1 ? 256 : 64;
    // About as many workgroups as are resident at a time (lora_expand_tiles by its
    // registers: 1024, 768 with the 16-bit types' ranks 33 to 64, 512; 8192 x 8192
    // bfloat16 of rank 64 77 us, with half as many 98; float 2048 x 4096 of rank 64
    // 24 us, with twice as many 30).
    const int64_t resident = p.tmb == 1 || R <= 32 || (type != T_F32 && R <= 64) ? 1024 : 512;
    int64_t shares = ceil_div(resident, busy), top = ceil_div(N, nunit);
    shares = shares > top ? top : shares;
    shares = shares < 1 ? 1 : shares > 4096 ? 4096 : shares;
    p.nshare = N > 0 ? ceil_div(ceil_div(N, shares), nunit) * nunit : nunit;
    p.p_at = 0;
    p.order_at = align_up(size_t(p.planes) * M * lora_pitch(R) * sizeof(float));
    p.tiles_at = p.order_at + align_up(size_t(M) * sizeof(int));
    p.bytes = p.mode == RowPlan::SORTED ? p.tiles_at + align_up(size_t(4 + 4 * (p.tiles + 1)) * sizeof(int)) : p.order_at;
    return p;
}

hipError_t launch_shrink(int type, const ShrinkArgs& a, const PassPlan& p, hipStream_t s) {
    return by_type(type, [&](auto t) {
        if (p.tmb == 1) shrink<decltype(t)::value, 1>(a, p, s);
        else shrink<decltype(t)::value, 4>(a, p, s);
    });
}

hipError_t launch_expand(int type, const ExpandArgs& a, const PassPlan& p, hipStream_t s) {
    const dim3 grid(grid_for(p.tiles), unsigned(ceil_div(a.N > 0 ? a.N : 1, a.nshare)));
    return by_type(type, [&](auto t) {
        if (p.mode == RowPlan::SINGLE) expand_one<decltype(t)::value>(a, grid, s);
        else if (p.tmb == 1) expand_rows<decltype(t)::value>(a, grid, s);
        else expand_tiles<decltype(t)::value>(a, grid, s);
    });
}

// Whether one launch (lora_few) is better than two: at most 16 workgroups, which each
// read an adapter's A of at most 128 KiB.  Calls in a replayed graph, us, one launch
// against two: A of 16 KiB 3.8 and 6.0, 64 KiB 5.2 and 6.3, 128 KiB 7.0 to 7.5 and 6.7
// to 6.9 (8192 x 4096 of rank 8 9.4 and 6.5), 256 KiB 10.9 and 7.3, 512 KiB 19.9 and
// 8.9.  At 128 KiB the one launch is for calls from a host that each pay for their
// launches (from Python 11 to 12 against 15); in a graph it loses up to 3 us there.
bool few_rows(int type, int64_t M, int64_t N, int64_t K, int64_t R) {
    return M * ceil_div(N > 0 ? N : 1, kFewCols) <= 16 && R * K * (type == T_F32 ? 4 : 2) <= 128 * 1024;
}

size_t lora_workspace_bytes(bool backward, int type, int64_t M, int64_t N, int64_t K, int R, int L) {
    if (M == 0 || (!backward && few_rows(type, M, N, K, R))) return 0;
    size_t most = 0;
    for (bool ids : {false, true}) {
        const size_t n = backward ? lora_backward_bytes(type, ids, M, N, K, R, L)
                                  : pass_plan(type, ids, true, M, N, K, R, L).bytes;
        most = n > most ? n : most;
    }
    return most;
}

hipError_t launch_lora(const LoraArgs& g, hipStream_t s) {
    if (few_rows(g.type, g.M, g.N, g.K, g.R)) {
        const dim3 grid(unsigned(ceil_div(g.N > 0 ? g.N : 1, kFewCols)), unsigned(g.M));
        return by_type(g.type, [&](auto t) {
            constexpr int T = decltype(t)::value;
            if (g.R % kVec<T> != 0) hipLaunchKernelGGL((lora_few<T, true>), grid, dim3(512), 0, s, g);
            else hipLaunchKernelGGL((lora_few<T, false>), grid, dim3(512), 0, s, g);
        });
    }
    const PassPlan p = pass_plan(g.type, g.ids != nullptr, true, g.M, g.N, g.K, g.R, g.L);
    char* const ws = static_cast<char*>(g.ws);
    int* const order = reinterpret_cast<int*>(ws + p.order_at);
    int* const head = reinterpret_cast<int*>(ws + p.tiles_at);
    const RowPlan rows{p.mode, g.ids, g.id64, int(g.M), g.L, order, head};
    hipError_t e = hipSuccess;
    if (p.mode == RowPlan::SORTED) {
        const GroupArgs a{g.ids, g.id64, int(g.M), g.L, 0, order, p.tmb == 1 ? 4 : 6, head, 0, nullptr, nullptr, nullptr};
        if ((e = launch_lora_group(a, s)) != hipSuccess) return e;
    }
    float* const P = reinterpret_cast<float*>(ws + p.p_at);
    const int64_t plane = g.M * lora_pitch(g.R);
    const ShrinkArgs sh{g.X, g.ldx, g.A, g.lda, g.sa, g.K, g.R, nullptr, 1.0f, false, P, plane, p.kshare, rows, p.tiles};
    if ((e = launch_shrink(g.type, sh, p, s)) != hipSuccess) return e;
    // Tiles of 64 rows read the planes once for each share of N: more than a few
    // planes are worth a launch that adds them first.
    const bool join = p.tmb == 4 && p.planes > 2;
    if (join && (e = launch_join(P, plane, p.planes, s)) != hipSuccess) return e;
    const ExpandArgs ex{P, plane, join ? 1 : p.planes, g.R, g.B, g.ldb, g.sb, g.N, g.scales, g.alpha, true,
                        g.base, g.ldbase, g.Y, g.ldy, g.H, g.ldh, p.nshare, rows, p.tiles};
    return launch_expand(g.type, ex, p, s);
}

}  // namespace sgemm
