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

// The group that holds tile t when every group's positions are cut into tiles
// of ROWS: its positions begin .. end - 1, its first tile and its tiles (0: no
// such tile).  Group g holds positions offsets[g] .. offsets[g + 1] - 1, cut to
// 0 .. rows - 1 whatever the offsets say (a range that ends before it begins
// is empty).  Every wave of the workgroup finds the same by itself: 64 groups
// at a time, a scan of their tile counts and one ballot.
struct GroupSpan {
    int group, begin, end, first, tiles;
};

template <int ROWS>
__device__ __forceinline__ GroupSpan find_span(const int* offsets, int groups, int rows, int t)
{
    const int lane = threadIdx.x & 63;
    int before = 0;                        // tiles of the groups already passed
    GroupSpan r = {0, 0, 0, 0, 0};
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
            r.group = base + l;
            r.begin = __builtin_amdgcn_readlane(lo, l);
            r.end = __builtin_amdgcn_readlane(hi, l);
            r.tiles = __builtin_amdgcn_readlane(tiles, l);
            r.first = __builtin_amdgcn_readlane(before + upto, l) - r.tiles;
            return r;
        }
        before += __builtin_amdgcn_readlane(upto, 63);
    }
    return r;
}

// Tile t itself; count = 0: it does not exist.
template <int ROWS>
__device__ __forceinline__ GroupTile find_tile(const int* offsets, int groups, int rows, int t)
{
    const GroupSpan s = find_span<ROWS>(offsets, groups, rows, t);
    GroupTile r = {0, 0, 0};
    if (s.tiles > 0) {
        r.group = s.group;
        r.begin = s.begin + (t - s.first) * ROWS;
        r.count = min(ROWS, s.end - r.begin);
    }
    return r;
}

// The tile that holds position p (the first group's that has it); count = 0:
// it is in no group.
template <int ROWS>
__device__ __forceinline__ GroupTile tile_of(const int* offsets, int groups, int rows, int p)
{
    const int lane = threadIdx.x & 63;
    GroupTile r = {0, 0, 0};
    for (int base = 0; base < groups; base += 64) {
        const int g = base + lane;
        int lo = 0, hi = 0;
        if (g < groups) {
            lo = min(max(offsets[g], 0), rows);
            hi = min(max(offsets[g + 1], 0), rows);
        }
        const uint64_t has = __ballot(lo <= p && p < hi);
        if (has != 0) {
            const int l = __builtin_ctzll(has);
            const int begin = __builtin_amdgcn_readlane(lo, l);
            r.group = base + l;
            r.begin = begin + (p - begin) / ROWS * ROWS;
            r.count = min(ROWS, __builtin_amdgcn_readlane(hi, l) - r.begin);
            return r;
        }
    }
    return r;
}

// One workgroup's share of (tiles) x (column blocks).  Workgroup b runs on XCD
// b % 8, so XCD x takes the x-th eighth of the list that runs over the groups,
// their column blocks and, innermost, the group's tiles: every XCD gets as
// many, the tiles that share a column block's weights meet in one L2, and so
// do a group's rows.  tile.count = 0: nothing to do.
struct GroupWork {
    GroupTile tile;
    int block;
};

template <int ROWS>
__device__ __forceinline__ GroupWork find_work(const int* offsets, int groups, int rows, int blocks,
                                               int b)
{
    const int lane = threadIdx.x & 63;
    // offsets that decrease can name more tiles than the grid has: cut there, so
    // that no number below passes 32 bits
    const int most = (int)gridDim.x / blocks;
    int total = 0;
    for (int g = lane; g < groups; g += 64) {
        const int lo = min(max(offsets[g], 0), rows);
        const int hi = min(max(offsets[g + 1], 0), rows);
        total = min(total + (hi > lo ? (hi - lo - 1) / ROWS + 1 : 0), most);
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
        total += __shfl_xor(total, off, 64);
    }
    total = min(__builtin_amdgcn_readfirstlane(total), most) * blocks;
    const int share = (total + 7) / 8;
    const int at = (b & 7) * share + (b >> 3);
    GroupWork r = {{0, 0, 0}, 0};
    if ((b >> 3) >= share || at >= total) {
        return r;
    }
    const GroupSpan s = find_span<ROWS>(offsets, groups, rows, at / blocks);
    const int in = at - s.first * blocks;              // within the group
    r.block = in / s.tiles;
    r.tile.group = s.group;
    r.tile.begin = s.begin + in % s.tiles * ROWS;
    r.tile.count = min(ROWS, s.end - r.tile.begin);
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
