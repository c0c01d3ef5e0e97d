// q4k_groups.h -- rows grouped by a matrix (an expert, an adapter): how a
// workgroup finds the rows of its tile.  Internal.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q4k {

// Rows begin .. begin + count - 1 (positions) of one group, at most one
// tile's.  count = 0: the tile does not exist.
struct GroupTile {
    int group, begin, count;
};

__device__ __forceinline__ int wave_scan_add(int v, int lane)
{
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(v, off, 64);
        v += lane >= off ? o : 0;
    }
    return v;
}

// Tile t when every group's positions are cut into tiles of ROWS.  Group g
// holds positions offsets[g] .. offsets[g + 1] - 1, cut to 0 .. rows - 1
// whatever the offsets say (a range that ends before it begins is empty).
// Every wave of the workgroup finds the same tile by itself: 64 groups at a
// time, a scan of their tile counts and one ballot.
template <int ROWS>
__device__ __forceinline__ GroupTile find_tile(const int* offsets, int groups, int rows, int t)
{
    const int lane = threadIdx.x & 63;
    int before = 0;                        // tiles of the groups already passed
    GroupTile r = {0, 0, 0};
    for (int base = 0; base < groups; base += 64) {
        const int g = base + lane;
        int lo = 0, hi = 0;
        if (g < groups) {
            lo = min(max(offsets[g], 0), rows);
            hi = min(max(offsets[g + 1], 0), rows);
        }
        const int tiles = hi > lo ? (hi - lo - 1) / ROWS + 1 : 0;
        const int upto = wave_scan_add(tiles, lane);
        const uint64_t past = __ballot(t < before + upto);
        if (past != 0) {
            const int l = __builtin_ctzll(past);
            const int first = __builtin_amdgcn_readlane(before + upto - tiles, l);
            const int glo = __builtin_amdgcn_readlane(lo, l);
            const int ghi = __builtin_amdgcn_readlane(hi, l);
            r.group = base + l;
            r.begin = glo + (t - first) * ROWS;
            r.count = min(ROWS, ghi - r.begin);
            return r;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return r;
}

// The most tiles of `tile` rows that `rows` positions in `groups` groups can
// take: every group that has any may end inside a tile.
inline int64_t most_tiles(int64_t rows, int64_t groups, int64_t tile)
{
    const int64_t some = rows < groups ? rows : groups;
    return (rows + some * (tile - 1)) / tile;
}

}  // namespace q4k
