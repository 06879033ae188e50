// expert_tiles.h -- the tiles of a grouped product, row tiles of the experts'
// segments x tiles of weight rows, and the order in which workgroups take them.
// A kernel's arguments hold the segments as offsets, S, E and max_tiles, the row
// tiles that S rows in E segments can make.
#pragma once

#include "experts_internal.h"

namespace ep {
namespace {

// Order of the tiles.  The 8 XCDs take contiguous shares of them (workgroups go
// to the XCDs in turn); within a share, groups of 8 row tiles x all n tiles, row
// tiles fastest: the 32 workgroups that an XCD runs at once read 8 row tiles and
// 4 weight tiles through its L2.
// Up to 64 experts each lane keeps one segment.  With more a tile's segment is found by a scan
// of the offsets, one load after another for every 64 experts, whose waits are also for the
// stores of the tile before and the loads into LDS of the next: MI355X, bf16, us for 64
// experts with rows / those and 1 / 64 / 192 / 960 without: 64 x 2048 x 1024, 600 rows 178 / 179
// / 178 / 180 / 183; 64 rows 49.3 / 50.5 / 50.5 / 50.8 / 53.0; 64 x 4096 x 128 (two steps a
// tile), 300 rows 62.7 / 66.6 / 67.5 / 67.8 / 71.6.
struct GemmTile {
    RowTile rows;    // rows.expert = -1: none
    int n;           // n tile
};
// Part of every XCD's share: its tiles from `first` to before `last`, their rows halved
// so many times.
struct GemmShare {
    int first, last, halved;
};
constexpr GemmShare kWholeShare = {0, 1 << 30, 0};
struct GemmTiles {
    int mt, nt;          // row tiles, n tiles
    int b, end, upto;    // up to 64 experts: lane's segment, and the tiles up to its end

    template <class Args>
    __device__ __forceinline__ GemmTiles(const Args& p, int TM, int n_tiles) : nt(n_tiles) {
        b = end = upto = 0;
        if (p.E <= kWave) {
            if (lane_id() < p.E) segment_of(p.offsets, lane_id(), p.S, b, end);
            int tiles = (end - b + TM - 1) / TM;
            tiles = tiles < (1 << 24) ? tiles : (1 << 24);
            upto = wave_inclusive_sum(tiles);
            mt = __builtin_amdgcn_readlane(upto, kWave - 1);
            mt = mt < p.max_tiles ? mt : p.max_tiles;
        } else {
            mt = count_row_tiles(p.offsets, p.E, p.S, TM, p.max_tiles);
        }
    }
    // Of segments that were looked at before: lane e's is [begin, past) (up to 64
    // experts), and they make `row_tiles` row tiles.
    __device__ __forceinline__ GemmTiles(int TM, int n_tiles, int row_tiles, int begin, int past)
        : mt(row_tiles), nt(n_tiles), b(begin), end(past)
    {
        int tiles = (end - b + TM - 1) / TM;
        tiles = tiles < (1 << 24) ? tiles : (1 << 24);
        upto = wave_inclusive_sum(tiles);
    }
    // The workgroup's tile number `turn`, of those of its XCD slot / 8 apart by
    // gridDim / 8.
    template <class Args>
    __device__ __forceinline__ GemmTile at(const Args& p, int TM, int turn) const {
        return at(p, TM, turn, kWholeShare);
    }
    // The same of the pieces, of TM rows, of a part of the share.  A piece behind its tile's
    // rows has none.
    template <class Args>
    __device__ __forceinline__ GemmTile at(const Args& p, int TM, int turn, const GemmShare& of) const {
        const int slot = int(blockIdx.x / 8) + turn * int(gridDim.x / 8);
        GemmTile t = find(p, TM << of.halved, of.first + (slot >> of.halved), of.last);
        const int row = t.rows.row0 + (slot & ((1 << of.halved) - 1)) * TM;
        t.rows.row0 = row < t.rows.end ? row : t.rows.end;
        return t;
    }
    template <class Args>
    __device__ __forceinline__ GemmTile find(const Args& p, int TM, int in_share, int last) const {
        GemmTile t;
        t.rows = RowTile{-1, 0, 0};
        t.n = 0;
        const int total = mt * nt, per = (total + 7) / 8;
        const int id = int(blockIdx.x % 8) * per + in_share;
        if (in_share >= (last < per ? last : per) || id >= total) return t;
        constexpr int kGroup = 8;
        const int group = id / (kGroup * nt);
        const int gsize = mt - group * kGroup < kGroup ? mt - group * kGroup : kGroup;
        const int in = id - group * kGroup * nt;
        t.n = in / gsize;
        const int index = group * kGroup + in % gsize;
        if (p.E > kWave) {
            t.rows = find_row_tile(p.offsets, p.E, p.S, TM, index);
            return t;
        }
        const uint64_t past = ballot(upto > index);
        if (!past) return t;
        const int l = __builtin_ctzll(past);
        const int before = l ? __builtin_amdgcn_readlane(upto, l - 1) : 0;
        t.rows.expert = l;
        t.rows.row0 = __builtin_amdgcn_readlane(b, l) + (index - before) * TM;
        t.rows.end = __builtin_amdgcn_readlane(end, l);
        return t;
    }
};

// Tiles of TM rows x TN weight rows (a multiple of 8, for the XCDs), 0 when a
// launch cannot hold them; sets p.max_tiles.
template <class Args>
uint32_t gemm_tiles(Args& p, int TM, int TN)
{
    const int64_t mt = p.S / TM + (p.E < p.S ? p.E : p.S);
    p.max_tiles = int(mt);
    const int64_t grid = (mt * ((p.N + TN - 1) / TN) + 7) / 8 * 8;
    return grid < (int64_t(1) << 30) ? uint32_t(grid) : 0;
}

}  // namespace
}  // namespace ep
