// Rows of one adapter brought together: a stable counting sort of the ids, and
// the tiles of rows that the adapter kernels take.
#include "lora.h"

namespace sgemm {
namespace {

constexpr int kGroupThreads = 1024;
constexpr int kHeld = 8192;

// Exclusive prefix sums of n ints in LDS; returns the total.  Every thread of the
// workgroup calls it.
__device__ __forceinline__ int scan(int* v, int n) {
    __shared__ int part[kGroupThreads / 64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int each = (n + kGroupThreads - 1) / kGroupThreads;
    const int lo = min(int(threadIdx.x) * each, n), hi = min(lo + each, n);
    int sum = 0;
#pragma unroll 1
    for (int e = lo; e < hi; e++) sum += v[e];
    int incl = sum;
#pragma unroll 1
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(incl, d);
        if (lane >= d) incl += up;
    }
    if (lane == 63) part[wave] = incl;
    __syncthreads();
    // The waves' sums, added the same way by every wave.
    int waves = part[lane & (kGroupThreads / 64 - 1)];
#pragma unroll 1
    for (int d = 1; d < kGroupThreads / 64; d *= 2) {
        const int up = __shfl_up(waves, d, kGroupThreads / 64);
        if ((lane & (kGroupThreads / 64 - 1)) >= d) waves += up;
    }
    const int total = __shfl(waves, kGroupThreads / 64 - 1), before_wave = wave ? __shfl(waves, wave - 1) : 0;
    int before = before_wave + incl - sum;
#pragma unroll 1
    for (int e = lo; e < hi; e++) {
        const int x = v[e];
        v[e] = before;
        before += x;
    }
    __syncthreads();
    return total;
}

// One workgroup.  Each of `waves` waves has a run of rows of its own: it counts
// its ids, the counts' prefix sums over (adapter, wave) are where its rows of an
// adapter go, and it deals them out in order, 64 rows at a time, a row's place
// among equal ids of the 64 from ballots; the last of the equals counts for all
// (LDS atomics on one address take their turns).  Rows without adapter come last.
// Up to kHeld rows' groups and places stay in LDS between the two passes.  The
// loops are not unrolled and the code is short: it runs once, on one CU, and is
// fetched from memory first (64 rows 6 us, 1025 rows 7, 8192 rows 12: bound by the
// latency of one step after another; 32768 rows 52, 65536 rows 90 with the copies of
// lora_prepare: the ids past kHeld are fetched in each pass, 64 a wave at a time).
__device__ __forceinline__ void group_rows(const GroupArgs& a, int* lds) {
    const int groups = a.L + 1;           // the last: no adapter
    int* const first = lds;               // groups + 1: tiles before a group's
    int* const table = lds + groups + 1;  // groups x waves
    __shared__ uint16_t held[kHeld], place[kHeld];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t run = ((int64_t(a.M) + a.waves - 1) / a.waves + 63) / 64 * 64;
    const int64_t begin = wave * run, end = wave >= a.waves ? 0 : begin + run < a.M ? begin + run : a.M;
    auto group_of = [&](int64_t m) {
        const int l = adapter_of(a.ids, a.id64, a.L, m);
        return l < 0 ? a.L : l;
    };
    const int h = a.M < kHeld ? a.M : kHeld;
#pragma unroll 1
    for (int m = threadIdx.x; m < h; m += 4 * kGroupThreads) {
        // Four in flight; past the end the last one again.
        int l[4];
#pragma unroll
        for (int u = 0; u < 4; u++) l[u] = group_of(min(m + u * kGroupThreads, h - 1));
#pragma unroll
        for (int u = 0; u < 4; u++) held[min(m + u * kGroupThreads, h - 1)] = uint16_t(l[u]);
    }
#pragma unroll 1
    for (int e = threadIdx.x; e < a.waves * groups; e += kGroupThreads) table[e] = 0;
    // The wave's own counts, written by any lane of it: a barrier to the compiler
    // orders the accesses (volatile ones would leave the LDS instructions: they took
    // 1.4 us for each 1024 rows).
    int* const mine = table + wave;
    const int w = a.waves;
    // Pass 0 counts, pass 1 deals out (without counting again where all places are
    // held).
#pragma unroll 1
    for (int pass = 0; pass < 2; pass++) {
        __syncthreads();
#pragma unroll 1
        for (int64_t m0 = begin; m0 < end; m0 += 64) {
            const int64_t m = m0 + lane;
            const bool in = m < end;
            const int l = !in ? 0 : m < kHeld ? held[m] : group_of(m);
            if (pass && a.M <= kHeld) {
                if (in) a.order[mine[l * w] + place[m]] = int(m);
                continue;
            }
            // Lanes with the same id: of up to three ids one by one (runs of rows), else
            // from the ids' bits.
            uint64_t same = 0, todo = __ballot(in);
#pragma unroll 1
            for (int q = 0; todo && q < 3; q++) {
                const uint64_t m = __ballot(in && l == __builtin_amdgcn_readlane(l, __builtin_ctzll(todo)));
                same = m >> lane & 1 ? m : same;
                todo &= ~m;
            }
            if (todo) {
                same = __ballot(in);
#pragma unroll 1
                for (int b = 0; (groups - 1) >> b; b++) {
                    const uint64_t set = __ballot(l >> b & 1);
                    same &= l >> b & 1 ? set : ~set;
                }
            }
            const int at = in ? mine[l * w] + __popcll(same & ((uint64_t(1) << lane) - 1)) : 0;
            asm volatile("" ::: "memory");
            if (in && pass) a.order[at] = int(m);
            if (in && m < kHeld) place[m] = uint16_t(at);
            if (in && same >> lane == 1) mine[l * w] = at + 1;
            asm volatile("" ::: "memory");
        }
        if (pass) break;
        // Where every wave's rows of every group start; then tiles, chunks, and the
        // chunks of adapters that have more than one.  table[l w] is where l's rows start.
        auto start_of = [&](int l) { return l < groups ? table[l * w] : a.M; };
#pragma unroll 1
        for (int kind = -1; kind < 3; kind++) {
            const int shift = kind > 0 ? a.chunk_shift : a.tile_shift, size = 1 << shift;
            int* const head = kind > 0 ? a.chunks : a.tiles;
            if (!head) continue;
            const int last = kind > 0 ? a.L : groups;  // chunks are of adapters only
            if (kind >= 0)
#pragma unroll 1
                for (int l = threadIdx.x; l < last; l += kGroupThreads) {
                    const int n = int((uint32_t(start_of(l + 1) - start_of(l)) + size - 1) >> shift);
                    first[l] = kind == 2 && n == 1 ? 0 : n;
                }
            __syncthreads();
            const int total = scan(kind < 0 ? table : first, kind < 0 ? w * groups : last);
            if (kind < 0) continue;
            int* const starts = kind == 1 ? a.chunk_start : kind == 2 ? a.slot_start : nullptr;
            if (starts)
                for (int l = threadIdx.x; l <= last; l += kGroupThreads) starts[l] = l < last ? first[l] : total;
#pragma unroll 1
            for (int t = threadIdx.x; kind < 2 && t < total; t += kGroupThreads) {
                int lo = 0, hi = last - 1;  // the last l with first[l] <= t
#pragma unroll 1
                while (lo < hi) {
                    const int mid = (lo + hi + 1) / 2;
                    if (first[mid] <= t) lo = mid;
                    else hi = mid - 1;
                }
                const int s = start_of(lo) + ((t - first[lo]) << shift), n = start_of(lo + 1) - s;
                reinterpret_cast<int4*>(head)[1 + int64_t(t)] =
                    int4{lo < a.L ? lo : -1, s, n < size ? n : size, t - first[lo]};
            }
            if (threadIdx.x == 0 && kind < 2) head[0] = total;
            __syncthreads();
        }
    }
}

__global__ void __launch_bounds__(kGroupThreads) lora_group(GroupArgs a) {
    extern __shared__ int lds[];
    group_rows(a, lds);
}

// A 64 x 64 tile of a transposed matrix a workgroup.  (The sort takes longer than the
// copies of all adapters: 8192 rows with 8 adapters of rank 16 15 us together.)
template <typename E>
__device__ void turn_tile(const TurnArgs& a, int64_t t, E* tile) {
    constexpr int PITCH = 64 + 4 / sizeof(E);
    const int64_t l = t / (a.tiles_r * a.tiles_c), q = t % (a.tiles_r * a.tiles_c);
    const int64_t r0 = q / a.tiles_c * 64, c0 = q % a.tiles_c * 64;
    const E* const w = static_cast<const E*>(a.W) + l * a.sw;
    E v[4096 / kGroupThreads];
#pragma unroll
    for (int u = 0; u < 4096 / kGroupThreads; u++) {
        const int e = u * kGroupThreads + int(threadIdx.x);
        const int64_t r = r0 + e / 64, c = c0 + e % 64;
        const bool in = r < a.rows && c < a.cols;
        v[u] = w[in ? r * a.ldw + c : 0];
        if (!in) v[u] = E(0);
    }
#pragma unroll
    for (int u = 0; u < 4096 / kGroupThreads; u++) {
        const int e = u * kGroupThreads + int(threadIdx.x);
        tile[e / 64 * PITCH + e % 64] = v[u];
    }
    __syncthreads();
    E* const out = static_cast<E*>(a.out) + l * a.cols * a.pitch;
#pragma unroll
    for (int u = 0; u < 4096 / kGroupThreads; u++) {
        const int e = u * kGroupThreads + int(threadIdx.x);
        const int64_t c = c0 + e / 64, r = r0 + e % 64;
        if (c < a.cols && r < a.pitch) out[c * a.pitch + r] = tile[e % 64 * PITCH + e / 64];
    }
    __syncthreads();
}

// Workgroup 0 sorts, the others transpose meanwhile.
template <typename E>
__global__ void __launch_bounds__(kGroupThreads) lora_prepare(GroupArgs g, TurnArgs a, TurnArgs b, int64_t tiles_a,
                                                              int64_t tiles) {
    extern __shared__ int lds[];
    const int first = g.order ? 1 : 0;
    if (first && blockIdx.x == 0) {
        group_rows(g, lds);
        return;
    }
    for (int64_t t = int64_t(blockIdx.x) - first; t < tiles; t += int64_t(gridDim.x) - first) {
        if (t < tiles_a) turn_tile<E>(a, t, reinterpret_cast<E*>(lds));
        else turn_tile<E>(b, t - tiles_a, reinterpret_cast<E*>(lds));
    }
}

// Waves that sort, by the tables of all of them and the tiles' prefix sums in what
// held, place and scan leave of 64 KiB; and these tables' bytes.  From 3949 adapters
// on one wave's table passes that, by up to 1.2 KiB (65612 bytes with held, place and
// scan at 4096): a CU has 160 KiB, and one such workgroup runs.
size_t group_waves(GroupArgs& a) {
    const int groups = a.L + 1, ints = 7900;
    a.waves = (ints - groups - 1) / groups;
    a.waves = a.waves > kGroupThreads / 64 ? kGroupThreads / 64 : a.waves < 1 ? 1 : a.waves;
    return size_t(a.waves * groups + groups + 1) * sizeof(int);
}

}  // namespace

hipError_t launch_lora_group(const GroupArgs& in, hipStream_t s) {
    GroupArgs a = in;
    const size_t bytes = group_waves(a);
    hipLaunchKernelGGL(lora_group, dim3(1), dim3(kGroupThreads), bytes, s, a);
    return hipGetLastError();
}

hipError_t launch_lora_prepare(int type, const GroupArgs& in, const TurnArgs& a, const TurnArgs& b, hipStream_t s) {
    GroupArgs g = in;
    size_t bytes = g.order ? group_waves(g) : 0;
    const int64_t na = g.L * a.tiles_r * a.tiles_c, n = na + g.L * b.tiles_r * b.tiles_c;
    const int64_t grid = (g.order ? 1 : 0) + n;
    if (grid == 0) return hipSuccess;
    if (n > 0 && bytes < 64 * 68 * 4) bytes = 64 * 68 * 4;
    // 1024 lanes a workgroup: 2^20 of them stay within the 32-bit dispatch size.
    const dim3 blocks(grid_for(grid)), lanes(kGroupThreads);
    if (type == T_F32) hipLaunchKernelGGL(lora_prepare<uint32_t>, blocks, lanes, bytes, s, g, a, b, na, n);
    else hipLaunchKernelGGL(lora_prepare<uint16_t>, blocks, lanes, bytes, s, g, a, b, na, n);
    return hipGetLastError();
}

}  // namespace sgemm
