// What the sources of the adapter kernels share.
#pragma once
#include "lora_rows.h"

namespace sgemm {

// The sort of the rows by adapter (lora_group.hip).
struct GroupArgs {
    const void* ids;
    bool id64;
    int M, L;
    int waves;         // set by the launcher
    int* order;        // M
    int tile_shift;    // a tile's rows: 2^tile_shift
    int* tiles;        // number of tiles, 3 unused, then adapter, start, count, place among
                       // its adapter's of each
    int chunk_shift;   // the same for chunks of 2^chunk_shift rows, rows without adapter left out
    int* chunks;       // (null: none)
    int* chunk_start;  // L + 1: chunks before an adapter's
    int* slot_start;   // L + 1: the same of adapters with more than one
};
hipError_t launch_lora_group(const GroupArgs& a, hipStream_t s);

// Adapters transposed.
struct TurnArgs {
    const void* W;  // L matrices of rows x cols
    int64_t ldw, sw;
    int64_t rows, cols;
    void* out;      // L matrices of cols x pitch, zero past `rows`
    int64_t pitch;
    int64_t tiles_r, tiles_c;
};

// The sort (unless group.order is null) and two stacks transposed, in one launch.
hipError_t launch_lora_prepare(int type, const GroupArgs& group, const TurnArgs& a, const TurnArgs& b, hipStream_t s);

// Sizes of a pass's launches (rows of K sums, N results a row) and of its
// workspace.
struct PassPlan {
    RowPlan::Mode mode;
    int tmb;        // 16-row blocks of a tile
    int64_t tiles;  // at most this many
    int planes;
    int64_t kshare, nshare;
    size_t p_at, order_at, tiles_at, bytes;
};
PassPlan pass_plan(int type, bool ids, bool single, int64_t M, int64_t N, int64_t K, int R, int L);
inline size_t align_up(size_t n) { return (n + 255) / 256 * 256; }

// Floats of a row of a plane of H: R rounded up so that rows are 64-byte pieces,
// zero past R.
__host__ __device__ constexpr int lora_pitch(int R) { return (R + 15) / 16 * 16; }

struct ShrinkArgs {
    const void* X;      // rows of K elements
    int64_t ldx;
    const void* W;      // L x R x K
    int64_t ldw, sw;
    int64_t K;
    int R;
    const float* scales;  // with scaled: the sums times alpha scales[l]
    float alpha;
    bool scaled;
    float* P;           // planes of M rows of lora_pitch(R) floats, in the order of positions, one for each K share
    int64_t plane;
    int64_t kshare;     // K per grid.y
    RowPlan rows;
    int64_t tiles;
};

struct ExpandArgs {
    const float* P;     // H: the sum of `planes` planes, as ShrinkArgs
    int64_t plane;
    int planes, R;
    const void* W;      // L x N x R
    int64_t ldw, sw;
    int64_t N;
    const float* scales;
    float alpha;
    bool scaled;
    const void* base;
    int64_t ldbase;
    void* Y;
    int64_t ldy;
    float* H;           // also store H here
    int64_t ldh;
    int64_t nshare;     // N per grid.y, a multiple of 64
    RowPlan rows;
    int64_t tiles;
};

// The two products (lora.hip), of element type T.
hipError_t launch_shrink(int type, const ShrinkArgs& a, const PassPlan& p, hipStream_t s);
hipError_t launch_expand(int type, const ExpandArgs& a, const PassPlan& p, hipStream_t s);
// The planes of H added into the first.
hipError_t launch_join(float* P, int64_t plane, int planes, hipStream_t s);
size_t lora_backward_bytes(int type, bool ids, int64_t M, int64_t N, int64_t K, int R, int L);

}  // namespace sgemm
