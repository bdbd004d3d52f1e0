// Gradients of low-rank adapters:
//   dH[m] = s_l dY[m] B_l,  dX[m] = base[m] + dH[m] A_l      (l = ids[m])
//   dA_l = sum dH[m]^T X[m],  dB_l = s_l sum dY[m]^T H[m]     (over l's rows m)
// The first two are the forward pass's products with the adapters transposed: a copy
// of all of them, whichever have rows.  It is small beside many rows; with few rows of
// many adapters it is most of the work, as the zeros of the unused dA and dB are.  The
// others are sums over rows: each chunk of an adapter's rows gives a partial sum, and
// these are added in order.
#include "lora.h"

namespace sgemm {
namespace {

// ---- sums over rows ----------------------------------------------------------------

// One of the two gradients: W[r, c] = sum over rows m of V[m, r] Z[m, c].
struct SideArgs {
    const void* Z;        // M rows of C elements
    int64_t ldz, C;
    const float* V;       // by_position: in the order of positions, else by rows
    int64_t ldv;
    bool by_position;
    float* partial;       // slots of R x C
    void* out;            // an adapter's only chunk: R x C, or C x R (turned), times the scale
    int64_t ldo, so;
    bool turned;
    const float* scales;  // with scaled
    float alpha;
    bool scaled;
    int64_t groups;       // column groups
};

struct WeightArgs {
    SideArgs side[2];
    int R, chunk;
    RowPlan rows;         // of chunks
    int64_t chunks;       // at most
    const int* slot_start;  // SORTED; else: chunks, if more than one
    const int* chunk_start;
};

constexpr int kWeightRows = 64;  // of V in LDS at a time

template <int T> constexpr int kGroupCols = T == T_F32 ? 64 : 128;  // columns of a wave

// The slot of a chunk's partial sum, or -1: it is the adapter's only one.
__device__ __forceinline__ int64_t slot_of(const WeightArgs& a, const RowTile& t) {
    if (a.rows.mode != RowPlan::SORTED) return a.rows.M > a.chunk ? t.place : -1;
    const int first = a.slot_start[t.adapter];
    return a.slot_start[t.adapter + 1] > first ? first + t.place : -1;
}

// A workgroup: a chunk of an adapter's rows, four waves' column groups, 16 RB of
// the ranks.  The sum of a matrix instruction runs over rows, so its operands
// hold 8 rows of one column (16-bit types: a lane's 8 rows x 8 columns, 16 bytes a
// row, are turned in registers, two rows by one byte permutation), or one row
// (float).  V is in three 16-bit parts, as in the forward pass; for float16 after a
// power of two for each rank that brings the chunk's largest into [2^14, 2^15).
// NARROW: fewer columns than a lane's on either side.
//   Up to rank 16 it is bound by reading X and dY (8192 rows of 4096 + 4096 bfloat16:
// 134 MB in 31 us, 4.3 TB/s).  Above, the chunks, chosen from M alone, leave the card
// half empty: 4096 rows of 4096 + 4096 are 256 workgroups, one a CU, where registers
// allow two (67 MB in 47 us; float, 2048 rows of 4096 + 2048: 50 MB in 35 us).  Loads one
// batch ahead and other layouts of V in LDS changed nothing there.  With 64 ranks' sums
// the 16-bit forms keep 48 to 77 registers in memory, of what a chunk begins and ends
// with: one of them is read in the loop over rows.
template <int T, int RB, bool NARROW>
__global__ void __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2))) lora_weights(WeightArgs a) {
    using E = typename Elem<T>::type;
    constexpr int V = kVec<T>, COLS = kGroupCols<T>, RN = 16 * RB;
    constexpr int VP = kWeightRows + 8;  // 16-bit: rows of a rank, padded
    __shared__ __attribute__((aligned(16))) char vs[T == T_F32 ? kWeightRows * RN * 4 : 3 * RN * VP * 2];
    __shared__ int row_of[kWeightRows];
    __shared__ uint32_t top[RN];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int r0 = blockIdx.z * RN;
    const int64_t groups = a.side[0].groups + a.side[1].groups;
    for (int64_t t = blockIdx.x; t < a.chunks * groups; t += gridDim.x) {
        const RowTile tile = row_tile(a.rows, t / groups, a.chunk);
        if (tile.count == 0) break;
        const bool second = t % groups >= a.side[0].groups;
        const SideArgs& sd = a.side[second];
        const int64_t c0 = ((second ? t % groups - a.side[0].groups : t % groups) * 4 + wave) * COLS;
        // The lane's columns.  Past the last they are the last ones again, so that the
        // loads need no check: two lanes then find, and store, the same sums.
        const int64_t c = NARROW || c0 + i * V + V <= sd.C ? c0 + i * V : sd.C - V;
        const float s = sd.scaled ? sd.alpha * (sd.scales ? sd.scales[tile.adapter] : 1.0f) : 1.0f;
        // Ranks r0 + r .. + 3 of V at position p.
        auto v_at = [&](int p, int r) {
            v4f v = {0, 0, 0, 0};
            if (p >= tile.count || r0 + r >= a.R) return v;
            const float* const at = sd.by_position ? sd.V + int64_t(tile.start + p) * sd.ldv + r0 + r
                                                   : sd.V + int64_t(row_at(a.rows, tile.start + p)) * sd.ldv + r0 + r;
            if (r0 + r + 4 <= a.R) {
                __builtin_memcpy(&v, at, 16);
            } else {
#pragma unroll
                for (int e = 0; e < 3; e++)
                    if (r0 + r + e < a.R) v[e] = at[e];
            }
            return v;
        };
        if constexpr (T == T_F16) {
            __syncthreads();
            if (threadIdx.x < RN) top[threadIdx.x] = 0;
            __syncthreads();
#pragma unroll 2
            for (int e = threadIdx.x; e < tile.count * (RN / 4); e += 256) {
                const int r = e % (RN / 4) * 4;
                const v4f v = v_at(e / (RN / 4), r);
#pragma unroll
                for (int y = 0; y < 4; y++)  // a maximum has no order
                    if (fabsf(v[y]) < __builtin_inff()) atomicMax(&top[r + y], __float_as_uint(fabsf(v[y])));
            }
        }
        v4f acc[V][RB];
#pragma unroll
        for (int e = 0; e < V; e++)
#pragma unroll
            for (int n = 0; n < RB; n++) acc[e][n] = v4f{0, 0, 0, 0};
        // The next rows' V and numbers, fetched while the ones before are multiplied.
        v4f next[RB];
        int next_row = 0;
        auto fetch = [&](int p0) {
#pragma unroll
            for (int u = 0; u < RB; u++) {
                const int e = threadIdx.x + 256 * u;
                next[u] = v_at(p0 + e / (RN / 4), e % (RN / 4) * 4);
            }
            const int p = p0 + int(threadIdx.x);
            if (threadIdx.x < kWeightRows) next_row = row_at(a.rows, tile.start + (p < tile.count ? p : 0));
        };
        fetch(0);
        for (int p0 = 0; p0 < tile.count; p0 += kWeightRows) {
            __syncthreads();
#pragma unroll
            for (int u = 0; u < RB; u++) {
                const int e = threadIdx.x + 256 * u, p = e / (RN / 4), r = e % (RN / 4) * 4;
                const v4f v = next[u];
                if constexpr (T == T_F32) {
                    *reinterpret_cast<v4f*>(vs + (p * RN + r) * 4) = v;
                } else {
#pragma unroll
                    for (int y = 0; y < 4; y += 2) {
                        uint16_t* const at = reinterpret_cast<uint16_t*>(vs) + (r + y) * VP + p;
                        uint32_t part[3];
                        float up[2] = {1.0f, 1.0f};
                        if constexpr (T == T_F16)
#pragma unroll
                            for (int z = 0; z < 2; z++) up[z] = half_factor(__uint_as_float(top[r + y + z]));
                        split_pair<T, 3>(v[y], v[y + 1], up[0], up[1], part);
#pragma unroll
                        for (int i = 0; i < 3; i++) {
                            at[i * RN * VP] = uint16_t(part[i]);
                            at[i * RN * VP + VP] = uint16_t(part[i] >> 16);
                        }
                    }
                }
            }
            if (threadIdx.x < kWeightRows) row_of[threadIdx.x] = next_row;
            __syncthreads();
            if (p0 + kWeightRows < tile.count) fetch(p0 + kWeightRows);
            if (c0 >= sd.C) continue;
            const int left = tile.count - p0 < kWeightRows ? tile.count - p0 : kWeightRows;
            // Rows past the chunk repeat its first, and are zeroed: what other adapters'
            // rows hold must not meet a zero of V.
            auto load_z = [&](int p) {
                const E* const row = static_cast<const E*>(sd.Z) + int64_t(row_of[p]) * sd.ldz;
                u32x4 z;
                if constexpr (NARROW) z = load_chunk<T>(row, c, sd.C);
                else z = load16(row + c);
                if (p >= left) z = u32x4{0, 0, 0, 0};
                return z;
            };
            if constexpr (T == T_F32) {
                // Eight loads in flight.
#pragma unroll 1
                for (int q0 = 0; q0 < kWeightRows / 4; q0 += 8) {
                    if (4 * q0 >= left) break;
                    u32x4 z[8];
#pragma unroll
                    for (int q = 0; q < 8; q++) z[q] = load_z(4 * (q0 + q) + g);
#pragma unroll
                    for (int q = 0; q < 8; q++)
#pragma unroll
                        for (int n = 0; n < RB; n++) {
                            const float v = reinterpret_cast<const float*>(vs)[(4 * (q0 + q) + g) * RN + 16 * n + i];
#pragma unroll
                            for (int e = 0; e < V; e++)
                                acc[e][n] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, __uint_as_float(z[q][e]), acc[e][n], 0, 0, 0);
                        }
                }
            } else {
#pragma unroll
                for (int q = 0; q < kWeightRows / 32; q++) {
                    if (32 * q >= left) break;
                    u32x4 z[8];
#pragma unroll
                    for (int y = 0; y < 8; y++) z[y] = load_z(32 * q + 8 * g + y);
                    u32x4 x[V];  // column e of the lane's 8 x 8
#pragma unroll
                    for (int e = 0; e < V; e++)
#pragma unroll
                        for (int y = 0; y < 4; y++)
                            x[e][y] = __builtin_amdgcn_perm(z[2 * y + 1][e / 2], z[2 * y][e / 2], e % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
                    for (int n = 0; n < RB; n++) {
                        const char* const at = vs + ((16 * n + i) * VP + 32 * q + 8 * g) * 2;
                        u32x4 part[3];
#pragma unroll
                        for (int z = 0; z < 3; z++) part[z] = *reinterpret_cast<const u32x4*>(at + z * RN * VP * 2);
#pragma unroll
                        for (int z = 0; z < 3; z++)
#pragma unroll
                            for (int e = 0; e < V; e++) acc[e][n] = mma16<T>(part[z], x[e], acc[e][n]);
                    }
                }
            }
        }
        if (c0 >= sd.C) continue;
        // The lane has ranks 4 g .. 4 g + 3 of each 16 at its V columns.
        const int64_t slot = slot_of(a, tile);
#pragma unroll
        for (int n = 0; n < RB; n++)
#pragma unroll
            for (int y = 0; y < 4; y++) {
                const int r = 16 * n + 4 * g + y;
                if (r0 + r >= a.R) continue;
                float f = s;
                if constexpr (T == T_F16) f = undone(s, half_factor(__uint_as_float(top[r])));
                if (slot >= 0) {
                    float* const at = sd.partial + (slot * a.R + r0 + r) * sd.C + c;
#pragma unroll
                    for (int e = 0; e < V; e += 4) {
                        const v4f w = {acc[e][n][y] * f, acc[e + 1][n][y] * f, acc[e + 2][n][y] * f, acc[e + 3][n][y] * f};
                        if constexpr (!NARROW) __builtin_memcpy(at + e, &w, 16);
                        else
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                if (c + e + q < sd.C) at[e + q] = w[q];
                    }
                } else {
                    E* const out = static_cast<E*>(sd.out) + tile.adapter * sd.so;
#pragma unroll
                    for (int e = 0; e < V; e++)
                        if (!NARROW || c + e < sd.C)
                            out[sd.turned ? (c + e) * sd.ldo + r0 + r : (r0 + r) * sd.ldo + c + e] = E(acc[e][n][y] * f);
                }
            }
    }
}

// The partial sums of an adapter added, in order, and zeros where no row has it:
// 16 ranks x 64 columns a workgroup, four neighbours a lane (16 slots of 64 x 6144:
// 6.6 us for 25 MB).
template <int T>
__global__ void __launch_bounds__(256) lora_weights_sum(WeightArgs a, int64_t tiles0, int64_t tiles) {
    using E = typename Elem<T>::type;
    __shared__ float part[64][17];
    const int rt = (a.R + 15) / 16;
    for (int64_t t0 = blockIdx.x; t0 < tiles; t0 += gridDim.x) {
        const bool second = t0 >= tiles0;
        const SideArgs& sd = a.side[second];
        const int64_t t = second ? t0 - tiles0 : t0, ct = (sd.C + 63) / 64;
        const int l = int(t / (rt * ct));
        const int r0 = int(t / ct % rt) * 16;
        const int64_t c0 = t % ct * 64;
        int64_t first, last;
        bool some;
        if (a.rows.mode == RowPlan::SORTED) {
            first = a.slot_start[l], last = a.slot_start[l + 1];
            some = a.chunk_start[l + 1] > a.chunk_start[l];
        } else {
            some = a.rows.M > 0 && l == 0;
            first = 0, last = some && a.rows.M > a.chunk ? (a.rows.M + a.chunk - 1) / a.chunk : 0;
        }
        if (some && first == last) continue;  // written by its only chunk
        __syncthreads();
        const int r = threadIdx.x / 16, x = threadIdx.x % 16 * 4;
        const int64_t c = c0 + x;
        const bool in = r0 + r < a.R && c < sd.C;
        v4f v = {0, 0, 0, 0};
        if (in) {
            const float* at = sd.partial + (first * a.R + r0 + r) * sd.C + c;
            if (c + 4 <= sd.C) {
#pragma unroll 4
                for (int64_t q = first; q < last; q++, at += int64_t(a.R) * sd.C) {
                    v4f w;
                    __builtin_memcpy(&w, at, 16);
                    v += w;
                }
            } else {
                for (int64_t q = first; q < last; q++, at += int64_t(a.R) * sd.C)
#pragma unroll
                    for (int e = 0; e < 3; e++)
                        if (c + e < sd.C) v[e] += at[e];
            }
        }
        E* const out = static_cast<E*>(sd.out) + l * sd.so;
        if (!sd.turned) {
            if (in)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (c + e < sd.C) out[(r0 + r) * sd.ldo + c + e] = E(v[e]);
            continue;
        }
#pragma unroll
        for (int e = 0; e < 4; e++) part[x + e][r] = v[e];
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; u++) {
            const int y = u * 16 + int(threadIdx.x) / 16, q = threadIdx.x % 16;
            if (r0 + q < a.R && c0 + y < sd.C) out[(c0 + y) * sd.ldo + r0 + q] = E(part[y][q]);
        }
    }
}

struct BackwardPlan {
    PassPlan pass;  // dH and dX: rows of N sums, K results
    int chunk;
    int64_t chunks, slots;
    int64_t pitch_a, pitch_b;
    size_t chunks_at, chunk_start_at, slot_start_at, a_at, b_at, pa_at, pb_at, bytes;
};

BackwardPlan backward_plan(int type, bool ids, int64_t M, int64_t N, int64_t K, int R, int L) {
    BackwardPlan p{};
    p.pass = pass_plan(type, ids, false, M, K, N, R, L);
    p.chunk = M > 4096 ? 512 : M > 2048 ? 256 : M > 512 ? 128 : 64;
    p.chunks = ceil_div(M, p.chunk) + (ids ? (L < M ? L : M) : 0);
    // Adapters with more than one chunk have at most two for each `chunk` rows.
    p.slots = 2 * ceil_div(M, p.chunk);
    p.pitch_a = (R + 7) / 8 * 8;
    p.pitch_b = (N + 7) / 8 * 8;
    size_t at = align_up(p.pass.bytes);
    auto take = [&](size_t n) {
        const size_t here = at;
        at += align_up(n);
        return here;
    };
    const size_t es = type == T_F32 ? 4 : 2;
    p.chunks_at = take(size_t(4 + 4 * (p.chunks + 1)) * sizeof(int));
    p.chunk_start_at = take(size_t(L + 1) * sizeof(int));
    p.slot_start_at = take(size_t(L + 1) * sizeof(int));
    p.a_at = take(size_t(L) * K * p.pitch_a * es);
    p.b_at = take(size_t(L) * R * p.pitch_b * es);
    p.pa_at = take(size_t(p.slots) * R * K * sizeof(float));
    p.pb_at = take(size_t(p.slots) * R * N * sizeof(float));
    p.bytes = at;
    return p;
}

template <int T>
hipError_t weights(const LoraGradArgs& b, const BackwardPlan& p, const RowPlan& rows, const float* dH, hipStream_t s) {
    const LoraArgs& g = b.f;
    char* const ws = static_cast<char*>(g.ws);
    WeightArgs a{};
    a.R = g.R;
    a.chunk = p.chunk;
    a.rows = rows;
    a.chunks = p.chunks;
    a.slot_start = reinterpret_cast<const int*>(ws + p.slot_start_at);
    a.chunk_start = reinterpret_cast<const int*>(ws + p.chunk_start_at);
    const int64_t wide = 4 * kGroupCols<T>;
    SideArgs& x = a.side[0];
    x = {g.X, g.ldx, b.dA ? g.K : 0, dH, lora_pitch(g.R), true,
         reinterpret_cast<float*>(ws + p.pa_at), b.dA, b.ldda, b.sda, false, nullptr, 1.0f, false, 0};
    SideArgs& y = a.side[1];
    y = {g.Y, g.ldy, b.dB ? g.N : 0, g.H, g.ldh, false,
         reinterpret_cast<float*>(ws + p.pb_at), b.dB, b.lddb, b.sdb, true, g.scales, g.alpha, true, 0};
    x.groups = ceil_div(x.C, wide);
    y.groups = ceil_div(y.C, wide);
    if (x.groups + y.groups == 0) return hipSuccess;
    const bool narrow = (x.C > 0 && x.C < kVec<T>) || (y.C > 0 && y.C < kVec<T>);
    auto run = [&](auto rb) {
        constexpr int RB = decltype(rb)::value;
        const dim3 grid(grid_for(p.chunks * (x.groups + y.groups)), 1, (g.R + 16 * RB - 1) / (16 * RB));
        if (narrow) hipLaunchKernelGGL((lora_weights<T, RB, true>), grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL((lora_weights<T, RB, false>), grid, dim3(256), 0, s, a);
    };
    if (g.M > 0) {
        if (g.R <= 16) run(std::integral_constant<int, 1>{});
        else if (g.R <= 32) run(std::integral_constant<int, 2>{});
        else run(std::integral_constant<int, 4>{});
    }
    const int64_t rt = (g.R + 15) / 16, t0 = g.L * rt * ceil_div(x.C, 64), t1 = g.L * rt * ceil_div(y.C, 64);
    hipLaunchKernelGGL(lora_weights_sum<T>, dim3(grid_for(t0 + t1)), dim3(256), 0, s, a, t0, t0 + t1);
    return hipGetLastError();
}

}  // namespace

size_t lora_backward_bytes(int type, bool ids, int64_t M, int64_t N, int64_t K, int R, int L) {
    return backward_plan(type, ids, M, N, K, R, L).bytes;
}

hipError_t launch_lora_backward(const LoraGradArgs& b, hipStream_t s) {
    const LoraArgs& g = b.f;
    hipError_t e = hipSuccess;
    BackwardPlan p{};
    RowPlan rows{RowPlan::UNIFORM, nullptr, false, int(g.M), g.L, nullptr, nullptr}, chunks = rows;
    char* const ws = static_cast<char*>(g.ws);
    float* dH = nullptr;
    if (g.M > 0) {
        p = backward_plan(g.type, g.ids != nullptr, g.M, g.N, g.K, g.R, g.L);
        dH = reinterpret_cast<float*>(ws + p.pass.p_at);
        GroupArgs group{};
        group.L = g.L;
        if (g.ids) {
            int* const order = reinterpret_cast<int*>(ws + p.pass.order_at);
            int* const head = reinterpret_cast<int*>(ws + p.pass.tiles_at);
            int* const ch = reinterpret_cast<int*>(ws + p.chunks_at);
            group = {g.ids, g.id64, int(g.M), g.L, 0, order, p.pass.tmb == 1 ? 4 : 6, head,
                     __builtin_ctz(p.chunk), ch,
                     reinterpret_cast<int*>(ws + p.chunk_start_at), reinterpret_cast<int*>(ws + p.slot_start_at)};
            rows = {RowPlan::SORTED, g.ids, g.id64, int(g.M), g.L, order, head};
            chunks = rows;
            chunks.head = ch;
        }
        // The adapters transposed: A for dX, B for dH.
        TurnArgs ta{g.A, g.lda, g.sa, g.R, b.dX ? g.K : 0, ws + p.a_at, p.pitch_a, ceil_div(p.pitch_a, 64), 0};
        TurnArgs tb{g.B, g.ldb, g.sb, g.N, b.dX || b.dA ? g.R : 0, ws + p.b_at, p.pitch_b, ceil_div(p.pitch_b, 64), 0};
        ta.tiles_c = ceil_div(ta.cols, 64);
        tb.tiles_c = ceil_div(tb.cols, 64);
        if ((e = launch_lora_prepare(g.type, group, ta, tb, s)) != hipSuccess) return e;
        const int64_t plane = g.M * lora_pitch(g.R);
        if (b.dX || b.dA) {
            const ShrinkArgs sh{g.Y, g.ldy, ws + p.b_at, p.pitch_b, g.R * p.pitch_b, g.N, g.R, g.scales, g.alpha, true,
                                dH, plane, p.pass.kshare, rows, p.pass.tiles};
            if ((e = launch_shrink(g.type, sh, p.pass, s)) != hipSuccess) return e;
            if (p.pass.planes > 1 && (e = launch_join(dH, plane, p.pass.planes, s)) != hipSuccess) return e;
        }
        if (b.dX && g.K > 0) {
            const ExpandArgs ex{dH, plane, 1, g.R, ws + p.a_at, p.pitch_a, g.K * p.pitch_a, g.K, nullptr,
                                1.0f, false, g.base, g.ldbase, b.dX, b.lddx, nullptr, 0, p.pass.nshare, rows, p.pass.tiles};
            if ((e = launch_expand(g.type, ex, p.pass, s)) != hipSuccess) return e;
        }
    }
    if (g.type == T_F32) return weights<T_F32>(b, p, chunks, dH, s);
    if (g.type == T_F16) return weights<T_F16>(b, p, chunks, dH, s);
    return weights<T_BF16>(b, p, chunks, dH, s);
}

}  // namespace sgemm
