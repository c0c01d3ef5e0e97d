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

// v of the lanes up to this one, added up: shifts within rows of 16 lanes (DPP),
// then lanes 15 and 31 broadcast into the rows behind them.
template <int CTRL, int ROWS>
__device__ __forceinline__ int scan_step(int v)
{
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, true);
}

__device__ __forceinline__ int wave_scan_add(int v)
{
    v = scan_step<0x111, 0xF>(v);
    v = scan_step<0x112, 0xF>(v);
    v = scan_step<0x114, 0xF>(v);
    v = scan_step<0x118, 0xF>(v);
    v = scan_step<0x142, 0xA>(v);
    return scan_step<0x143, 0xC>(v);
}

// Lane l's group base + l: its positions lo .. hi - 1, cut to 0 .. rows - 1
// whatever the offsets say (a range that ends before it begins is empty), its
// tiles of ROWS, and the tiles of the lanes up to this one.  A whole wave.
struct GroupLanes {
    int lo, hi, tiles, upto;
};

template <int ROWS>
__device__ __forceinline__ GroupLanes group_lanes(const int* offsets, int groups, int rows,
                                                  int base)
{
    const int g = base + (int)(threadIdx.x & 63);
    GroupLanes r = {0, 0, 0, 0};
    if (g < groups) {
        r.lo = min(max(offsets[g], 0), rows);
        r.hi = min(max(offsets[g + 1], 0), rows);
    }
    r.tiles = r.hi > r.lo ? (r.hi - r.lo - 1) / ROWS + 1 : 0;
    r.upto = wave_scan_add(r.tiles);
    return r;
}

// The group that holds tile t when every group's positions are cut into tiles
// of ROWS: its positions begin .. end - 1, its first tile and its tiles (0: no
// such tile).  Every wave of the workgroup finds the same by itself: 64 groups
// at a time, a scan of their tile counts and one ballot.
struct GroupSpan {
    int group, begin, end, first, tiles;
};

// Tile t among the 64 groups from base on, `before` tiles before them
__device__ __forceinline__ bool span_in(const GroupLanes& v, int base, int before, int t,
                                        GroupSpan& r)
{
    const uint64_t past = __ballot(t < before + v.upto);
    if (past == 0) {
        return false;
    }
    const int l = __builtin_ctzll(past);
    r.group = base + l;
    r.begin = __builtin_amdgcn_readlane(v.lo, l);
    r.end = __builtin_amdgcn_readlane(v.hi, l);
    r.tiles = __builtin_amdgcn_readlane(v.tiles, l);
    r.first = before + __builtin_amdgcn_readlane(v.upto, l) - r.tiles;
    return true;
}

template <int ROWS>
__device__ __forceinline__ GroupSpan find_span(const int* offsets, int groups, int rows, int t)
{
    int before = 0;                        // tiles of the groups already passed
    GroupSpan r = {0, 0, 0, 0, 0};
    for (int base = 0; base < groups; base += 64) {
        const GroupLanes v = group_lanes<ROWS>(offsets, groups, rows, base);
        if (span_in(v, base, before, t, r)) {
            return r;
        }
        before += __builtin_amdgcn_readlane(v.upto, 63);
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

// Tiles of all groups, and the first 64 groups' lanes
struct GroupTiles {
    GroupLanes first;
    int tiles;
};

// most: as many tiles as the grid has (offsets that decrease can name more),
// so that no number below passes 32 bits
template <int ROWS>
__device__ __forceinline__ GroupTiles count_tiles(const int* offsets, int groups, int rows,
                                                  int most)
{
    GroupTiles r;
    r.first = group_lanes<ROWS>(offsets, groups, rows, 0);
    r.tiles = min(__builtin_amdgcn_readlane(r.first.upto, 63), most);
    for (int base = 64; base < groups; base += 64) {
        const GroupLanes o = group_lanes<ROWS>(offsets, groups, rows, base);
        r.tiles = min(r.tiles + __builtin_amdgcn_readlane(o.upto, 63), most);
    }
    return r;
}

template <int ROWS>
__device__ __forceinline__ GroupWork find_work(const GroupTiles& tiles, const int* offsets,
                                               int groups, int rows, int blocks, int b)
{
    const int total = tiles.tiles * blocks;
    const int share = (total + 7) / 8;
    const int at = (b & 7) * share + (b >> 3);
    GroupWork r = {{0, 0, 0}, 0};
    if ((b >> 3) >= share || at >= total) {
        return r;
    }
    // one look at the offsets is enough for 64 groups
    GroupSpan s = {0, 0, 0, 0, 0};
    if (!span_in(tiles.first, 0, 0, at / blocks, s)) {
        s = find_span<ROWS>(offsets, groups, rows, at / blocks);
    }
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
