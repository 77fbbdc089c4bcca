// grouped.hpp - rows in groups: the offsets a grouped product reads on the device, and which tile
// of which group a workgroup works on.
//
// offsets holds n + 1 row numbers; group g is rows offsets[g] .. offsets[g + 1] - 1. The host does
// not see them (a router writes them on the device), so the grid covers the most tiles any split
// can have, ceil(rows / BM) summed over the groups <= rows / BM + min(n, rows), and every
// workgroup finds its own tile from the offsets: one load and one 64-lane scan per 64 groups, made
// by each wave for itself (no LDS, no barrier). Offsets are clamped to 0 .. rows and a decreasing
// pair is an empty group, so no offset leads outside the buffers.
#pragma once
#include "bsm_device.hpp"
#include "bsm_internal.hpp"

namespace bsm {
namespace grouped {

// First row and end of group i < n.
__device__ __forceinline__ void group_range(const GroupArgs& gr, int i, int& lo, int& hi) {
  lo = min(max(gr.offsets[i], 0), gr.rows);
  hi = max(min(max(gr.offsets[i + 1], 0), gr.rows), lo);
}

// Inclusive sum over the 64 lanes, in the vector unit's own lane shifts: within rows of 16, then the
// last lane of each row into the rows behind it.
__device__ __forceinline__ int wave_inclusive_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

struct Spot {
  int g, row0, rows;  // the group, its first row and its row count
  int tm, tn;         // the tile within the group
};

// Tile `li` of tiles_m x tiles_n in bands of GROUP_M tile rows walked column by column.
template <int GROUP_M>
__device__ __forceinline__ void band_tile(int li, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int per_band = GROUP_M * tiles_n, band = li / per_band, first = band * GROUP_M;
  const int size = min(tiles_m - first, GROUP_M), in = li - band * per_band;
  tm = first + in % size;
  tn = in / size;
}

// Tile `pid` of the launch (wave-uniform result; false: no such tile). Group g has count(rows of g) row
// tiles of tiles_n tiles each. Tiles are numbered group by group, inside a group in bands of GROUP_M
// tile rows walked column by column, and the numbers are dealt to the XCDs (workgroup p runs on XCD
// p % 8) in eight contiguous ranges, so that the workgroups of one XCD share a group's weight panels
// in its L2. On return `used` is the number of pids that the split at hand can have tiles for (a
// multiple of 8).
template <int GROUP_M, typename F>
__device__ __forceinline__ bool find_tile_of(const GroupArgs& gr, int pid, int tiles_n, int lane, F count, Spot& s,
                                             int& used) {
  auto tiles_of = [&](int i, int& lo, int& hi) {
    if (i < gr.n) group_range(gr, i, lo, hi);
    else lo = hi = 0;
    return count(hi - lo);
  };
  int lo, hi;
  int t = tiles_of(lane, lo, hi), incl = wave_inclusive_scan(t);
  int all = __builtin_amdgcn_readlane(incl, 63);
  for (int i0 = 64; i0 < gr.n; i0 += 64) {
    int l, h;
    all += __builtin_amdgcn_readlane(wave_inclusive_scan(tiles_of(i0 + lane, l, h)), 63);
  }
  const int total = all * tiles_n, chunk = (total + 7) >> 3;
  used = 8 * chunk;
  const int lid = (pid & 7) * chunk + (pid >> 3);
  if ((pid >> 3) >= chunk || lid >= total) return false;
  const int rt = lid / tiles_n;
  int before = 0;
  for (int i0 = 0; i0 < gr.n; i0 += 64) {
    if (i0 > 0) {
      t = tiles_of(i0 + lane, lo, hi);
      incl = wave_inclusive_scan(t);
    }
    const uint64_t past = __ballot(before + incl > rt);
    if (past) {
      const int at = __builtin_ctzll(past);
      s.g = i0 + at;
      s.row0 = __builtin_amdgcn_readlane(lo, at);
      s.rows = __builtin_amdgcn_readlane(hi, at) - s.row0;
      const int tiles_m = __builtin_amdgcn_readlane(t, at);
      const int first_tile = before + __builtin_amdgcn_readlane(incl, at) - tiles_m;
      const int li = lid - first_tile * tiles_n;
      if (li < 0 || li >= tiles_m * tiles_n) return false;  // (offsets that overlap beyond all counting)
      band_tile<GROUP_M>(li, tiles_m, tiles_n, s.tm, s.tn);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// With tiles of BM rows.
template <int BM, int GROUP_M>
__device__ __forceinline__ bool find_tile(const GroupArgs& gr, int pid, int tiles_n, int lane, Spot& s) {
  int used;
  return find_tile_of<GROUP_M>(gr, pid, tiles_n, lane, [](int rows) { return (int)(((int64_t)rows + BM - 1) / BM); }, s, used);
}

// Row tiles that `rows` rows in n groups can need at most.
inline int64_t most_row_tiles(int64_t rows, int64_t n, int64_t bm) { return rows / bm + (n < rows ? n : rows); }

}  // namespace grouped
}  // namespace bsm
