// Rows sorted by group (experts, adapters): a workgroup's lookup of its tile
// among tiles whose number per group the host does not know.
#pragma once

#include "iqp_internal.h"

namespace iqp {
namespace {
namespace groups {

// 8 and 16 bytes at any even address: the card's vector memory takes them there too, in one access
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(2)));
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));

// inclusive sum over the 64 lanes
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // lane 15 of each row to the next
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // lane 31 to the upper half
  return v;
}

__device__ __forceinline__ int clamp_place(const RowGroups& g, int v) { return v < 0 ? 0 : (v > (int)g.R ? (int)g.R : v); }

// Places begin .. begin + rows - 1 of the sorted rows, all of one group, at most
// tm of them; part `part` of the `parts` that share them. rows 0: no such tile.
struct Tile {
  int group, begin, rows, part;
};

// Tile number `item`, where every group's rows are cut into tiles of tm (the
// last one shorter) and each tile has `parts` parts. All lanes of all waves call it
// and get the same answer. Offsets are kept inside [0, R] whatever they hold. 256
// groups a round of loads. The tiles come group by group, and within a group `run`
// parts of a tile, the same of its next tile, until all have had them, then the next
// `run`: with 1 neighbours share weights, with all parts they share rows.
// large_first: all groups' whole tiles first, then those of more than tm / 2 rows,
// then the others, so that few tiles end together.
__device__ __forceinline__ Tile find_tile(const RowGroups& g, int tm, int parts, int run, int64_t item, bool large_first) {
  const int lane = threadIdx.x & 63;
  int64_t done = 0;
  for (int pass = 0; pass < (large_first ? 3 : 1); ++pass)
    for (int g0 = 0; g0 < g.G; g0 += 256) {
      int begin[4], end[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int e = g0 + 64 * q + lane, c = e < g.G ? e : g.G - 1;
        begin[q] = g.offsets[c];
        end[q] = g.offsets[c + 1];
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int b = clamp_place(g, begin[q]), d = clamp_place(g, end[q]) - b;
        const int n = d > 0 && g0 + 64 * q + lane < g.G ? d : 0;
        const int whole = (int)((unsigned)n / (unsigned)tm), rest = n - whole * tm;
        int tiles = whole + (rest > 0 ? 1 : 0), t0 = 0;
        if (large_first) {
          t0 = pass ? whole : 0;
          tiles = pass == 0 ? whole : (pass == 1 ? rest > tm / 2 : rest > 0 && rest <= tm / 2) ? 1 : 0;
        }
        const int upto = wave_scan(tiles);
        const int total = __builtin_amdgcn_readlane(upto, 63);
        if (item < (done + total) * parts) {
          const int at = 63 - __builtin_clzll(__ballot((done + upto - tiles) * parts <= item));
          const int mine = __builtin_amdgcn_readlane(tiles, at);
          const int local = (int)(item - (done + __builtin_amdgcn_readlane(upto, at) - mine) * parts);
          const int first = local / (mine * run) * run, width = parts - first < run ? parts - first : run;
          const int in = local - first * mine, down = in / width;
          const int part = first + in - down * width, t = __builtin_amdgcn_readlane(t0, at) + down;
          const int rows = __builtin_amdgcn_readlane(n, at) - t * tm;
          return {g0 + 64 * q + at, __builtin_amdgcn_readlane(b, at) + t * tm, rows < tm ? rows : tm, part};
        }
        done += total;
      }
    }
  return {0, 0, 0, 0};
}

// Work item of workgroup `id`: `chunk` consecutive items to an XCD (workgroup id
// mod 8) at a time. The grid is a multiple of 8 chunk.
__device__ __forceinline__ int64_t item_of(unsigned id, unsigned chunk) {
  const unsigned xcd = id & 7, j = id >> 3;
  return (int64_t)(j / chunk) * 8 * chunk + xcd * chunk + j % chunk;
}

}  // namespace groups
}  // namespace
}  // namespace iqp
