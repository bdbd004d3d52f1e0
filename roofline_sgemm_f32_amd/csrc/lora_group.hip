// Rows of one adapter brought together: a stable counting sort of the ids, and
// the tiles of rows that the adapter kernels take.
#include "lora.h"

namespace sgemm {
namespace {

constexpr int kGroupThreads = 1024;

// Exclusive prefix sums of n ints in LDS, in the order at(0), at(1), ...; returns
// the total.  Every thread of the workgroup calls it.
template <class At>
__device__ int scan(int n, At at) {
    __shared__ int part[kGroupThreads / 64];
    const int each = (n + kGroupThreads - 1) / kGroupThreads;
    const int lo = min(int(threadIdx.x) * each, n), hi = min(lo + each, n);
    int sum = 0;
    for (int e = lo; e < hi; e++) sum += at(e);
    int incl = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int up = __shfl_up(incl, d);
        if (int(threadIdx.x & 63) >= d) incl += up;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 63) part[threadIdx.x >> 6] = incl;
    __syncthreads();
    int before = incl - sum, total = 0;
    for (int w = 0; w < kGroupThreads / 64; w++) {
        if (w < int(threadIdx.x >> 6)) before += part[w];
        total += part[w];
    }
    for (int e = lo; e < hi; e++) {
        const int v = at(e);
        at(e) = before;
        before += v;
    }
    __syncthreads();
    return total;
}

// One workgroup.  Each of `waves` waves has a run of rows of its own: it counts
// its ids in a table of its own, the tables' prefix sums over (adapter, wave)
// are where its rows of an adapter go, and it deals them out in order, 64 rows
// at a time, a row's place among equal ids of the 64 from one ballot per bit of
// the id.  Rows without adapter come last.  One workgroup because the whole
// is small beside the products (8192 rows: 5 us), and no launch follows it.
__global__ void __launch_bounds__(kGroupThreads) lora_group(GroupArgs a) {
    extern __shared__ int lds[];
    const int groups = a.L + 1;                 // the last: no adapter
    int* const table = lds;                     // waves x groups
    int* const first = lds + a.waves * groups;  // groups + 1: tiles before a group's
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t run = ((a.M + a.waves - 1) / a.waves + 63) / 64 * 64;
    const int64_t begin = wave * run, end = begin + run < a.M ? begin + run : a.M;
    auto group_of = [&](int64_t m) {
        const int l = adapter_of(a.ids, a.id64, a.L, m);
        return l < 0 ? a.L : l;
    };
    for (int e = threadIdx.x; e < a.waves * groups; e += kGroupThreads) table[e] = 0;
    __syncthreads();
    if (wave < a.waves)
        for (int64_t m = begin + lane; m < end; m += 64) atomicAdd(&table[wave * groups + group_of(m)], 1);
    __syncthreads();
    scan(a.waves * groups, [&](int e) -> int& { return table[e % a.waves * groups + e / a.waves]; });
    // table[l] is now where adapter l's rows start.
    auto start_of = [&](int l) { return l < groups ? table[l] : a.M; };
    for (int kind = 0; kind < 2; kind++) {
        const int size = kind ? a.chunk : a.tile;
        int* const head = kind ? a.chunks : a.tiles;
        if (!head) continue;
        const int last = kind ? a.L : groups;  // chunks are of adapters only
        for (int l = threadIdx.x; l < last; l += kGroupThreads)
            first[l] = (start_of(l + 1) - start_of(l) + size - 1) / size;
        __syncthreads();
        const int total = scan(last, [&](int e) -> int& { return first[e]; });
        for (int t = threadIdx.x; t < total; t += kGroupThreads) {
            int lo = 0, hi = last - 1;  // the last l with first[l] <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (first[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int s = start_of(lo) + (t - first[lo]) * size, n = start_of(lo + 1) - s;
            int* const at = head + 4 + 4 * int64_t(t);
            at[0] = lo < a.L ? lo : -1;
            at[1] = s;
            at[2] = n < size ? n : size;
        }
        if (threadIdx.x == 0) head[0] = total;
        if (kind)
            for (int l = threadIdx.x; l <= last; l += kGroupThreads) a.chunk_start[l] = l < last ? first[l] : total;
        __syncthreads();
    }
    if (wave < a.waves) {
        volatile int* const next = table + wave * groups;  // other lanes write it
        for (int64_t m0 = begin; m0 < end; m0 += 64) {
            const bool in = m0 + lane < end;
            const int l = in ? group_of(m0 + lane) : 0;
            uint64_t same = __ballot(in);
            for (int b = 0; (groups - 1) >> b; b++) {
                const uint64_t set = __ballot(l >> b & 1);
                same &= l >> b & 1 ? set : ~set;
            }
            const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
            const int at = in ? next[l] : 0;
            __builtin_amdgcn_wave_barrier();
            if (in) {
                a.order[at + rank] = int(m0 + lane);
                if (same >> lane == 1) next[l] = at + rank + 1;  // the last of its equals
            }
            __builtin_amdgcn_wave_barrier();
        }
    }
}

}  // namespace

hipError_t launch_lora_group(const GroupArgs& in, hipStream_t s) {
    GroupArgs a = in;
    // Tables of all waves and the tiles' prefix sums in 64 KiB less what scan takes.
    const int groups = a.L + 1, ints = 16000;
    a.waves = (ints - groups - 1) / groups;
    a.waves = a.waves > kGroupThreads / 64 ? kGroupThreads / 64 : a.waves < 1 ? 1 : a.waves;
    const size_t bytes = size_t(a.waves * groups + groups + 1) * sizeof(int);
    hipLaunchKernelGGL(lora_group, dim3(1), dim3(kGroupThreads), bytes, s, a);
    return hipGetLastError();
}

}  // namespace sgemm
