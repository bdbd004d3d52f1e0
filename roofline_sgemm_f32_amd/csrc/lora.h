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
    int tile;          // rows of a tile
    int* tiles;        // number of tiles, 3 unused, then adapter, start, count, unused of each
    int chunk;         // the same for chunks of `chunk` rows, rows without adapter left out
    int* chunks;       // (null: none)
    int* chunk_start;  // L + 1: chunks before an adapter's
};
hipError_t launch_lora_group(const GroupArgs& a, hipStream_t s);

}  // namespace sgemm
