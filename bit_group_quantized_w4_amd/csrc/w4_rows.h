// Rows sorted by expert: which rows of x, and which expert's weight, a block
// multiplies.  The row counts are known on the GPU only (`offsets`, experts + 1
// values), so a launch covers the most row tiles that M rows of that many
// experts can make -- M / BM full ones and at most one partial one per expert
// that has rows -- and each block looks its own tile up; blocks past the last
// tile have nothing to do.
#pragma once

#include "w4_device.h"

namespace w4 {

struct RowTile {
  int expert;
  int r0, r1;  // rows r0 .. r1-1, at most BM of them, at least one
  bool alone;  // the expert has no other row tile
};

// Sum of v over this lane and the lanes before it, all 64 being active: prefix
// sums within rows of sixteen lanes, then the rows' totals handed on.  (Six vector
// instructions: a call of eight rows of 512 experts of 768 x 2048 takes 6.7 us, and
// 8.2 us with the sums exchanged through LDS.)
__device__ __forceinline__ int lanes_upto(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // from 1 lane before, in the row
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row 0's last lane to row 1, 2's to 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return v;
}

// Row tile `t` of BM rows each: expert by expert, each expert's rows cut from
// its first one on.  Offsets are clamped to [0, M] and a range that ends before
// it begins is empty, so whatever the buffer holds no row outside x is named.
// offsets == nullptr: one expert that has all M rows.  Every lane of the
// wavefront must call this; the result is the same in all of them.
__device__ __forceinline__ bool find_row_tile(const int* __restrict__ offsets, int experts, int M, int BM, int t,
                                              RowTile& o) {
  if (!offsets) {
    o.expert = 0;
    o.r0 = t * BM;
    o.r1 = min(M, o.r0 + BM);
    o.alone = M <= BM;
    return o.r0 < M;
  }
  const int lane = threadIdx.x & 63;
  int before = 0;  // tiles of the experts before e0
  auto load = [&](int e, int& a, int& b) {
    a = b = 0;
    if (e < experts) {
      a = offsets[e];
      b = offsets[e + 1];
    }
  };
  int a, b, next_a, next_b;
  load(lane, a, b);
  for (int e0 = 0; e0 < experts; e0 += 64) {
    load(e0 + 64 + lane, next_a, next_b);  // on their way while these are counted
    a = min(max(a, 0), M);
    b = min(max(b, 0), M);
    const int n = b > a ? (b - a + BM - 1) / BM : 0;
    const int s = lanes_upto(n);
    const uint64_t past = __ballot(before + s > t);
    if (past) {
      const int l = __builtin_ctzll(past);
      o.expert = e0 + l;
      o.r0 = __builtin_amdgcn_readlane(a, l) + (t - before - __builtin_amdgcn_readlane(s - n, l)) * BM;
      o.r1 = min(__builtin_amdgcn_readlane(b, l), o.r0 + BM);
      o.alone = __builtin_amdgcn_readlane(n, l) == 1;
      return true;
    }
    before += __builtin_amdgcn_readlane(s, 63);
    a = next_a;
    b = next_b;
  }
  return false;
}

// Row tiles there are in all.  Every lane of the wavefront must call this.
__device__ __forceinline__ int count_row_tiles(const int* __restrict__ offsets, int experts, int M, int BM) {
  if (!offsets) return (M + BM - 1) / BM;
  int n = 0;
  for (int e = threadIdx.x & 63; e < experts; e += 64) {
    const int a = min(max(offsets[e], 0), M), b = min(max(offsets[e + 1], 0), M);
    n += b > a ? (b - a + BM - 1) / BM : 0;
  }
  return __builtin_amdgcn_readlane(lanes_upto(n), 63);
}

// Which (row tile, panel of outputs) block b of tiles * panels runs.  Blocks go to
// the eight XCDs in turn, each with an L2 of its own, so each XCD is given a
// contiguous run of the work: bands of kBand row tiles, panel by panel within a
// band, so that the blocks that run at one time on an XCD share their rows and
// their panels.
constexpr int kXcds = 8, kBand = 4;
__device__ __forceinline__ void tile_of_block(int b, int tiles, int panels, int& t, int& p) {
  const int total = tiles * panels, xcd = b % kXcds;
  const int at = xcd * (total / kXcds) + min(xcd, total % kXcds) + b / kXcds;
  const int band = at / (kBand * panels), in = at - band * kBand * panels;
  const int height = min(kBand, tiles - band * kBand);
  p = in / height;
  t = band * kBand + in - p * height;
}

// Block b's place in the order of tiles * panels pieces of work, each XCD given a contiguous
// run of them (as tile_of_block does).
__device__ __forceinline__ int slot_of_block(int b, int total) {
  const int xcd = b % kXcds;
  return xcd * (total / kXcds) + min(xcd, total % kXcds) + b / kXcds;
}

// Piece of work `at` of tiles * panels: expert by expert, an expert's row tiles in bands of kBand
// (up to 2 kBand - 1 in the last), panel by panel within a band.  So blocks that run at one
// time share not only rows and panels but also the expert, whose weights the panels are of
// (tile_of_block's bands may hold several experts').  Returns whether there is such a piece.
struct BandTile {
  RowTile rt;
  int p;           // panel
  int in, height;  // of the band: the row tile's place and the number of them
};
__device__ __forceinline__ bool band_tile(const int* __restrict__ offsets, int experts, int M, int BM, int panels, int at,
                                          BandTile& o) {
  int t = at / panels, first, end, before, n;  // the expert's rows, the tiles before its own, and its own
  if (!offsets) {
    o.rt.expert = before = first = 0;
    end = M;
    n = (M + BM - 1) / BM;
    if (t >= n) return false;
  } else {
    if (!find_row_tile(offsets, experts, M, BM, t, o.rt)) return false;
    first = min(max(offsets[o.rt.expert], 0), M);
    end = min(max(offsets[o.rt.expert + 1], 0), M);
    n = (end - first + BM - 1) / BM;
    before = t - (o.rt.r0 - first) / BM;
  }
  const int local = at - before * panels, bands = n < kBand ? 1 : n / kBand;
  const int band = min(local / (kBand * panels), bands - 1), left = local - band * kBand * panels;
  o.height = band == bands - 1 ? n - band * kBand : kBand;
  o.p = left / o.height;
  o.in = left - o.p * o.height;
  o.rt.r0 = first + (band * kBand + o.in) * BM;
  o.rt.r1 = min(end, o.rt.r0 + BM);
  o.rt.alone = n == 1;
  return true;
}

// Row tiles a launch has to cover (see above).
inline int64_t max_row_tiles(int64_t M, int64_t experts, bool grouped, int BM) {
  if (!grouped) return (M + BM - 1) / BM;
  return M / BM + (experts < M ? experts : M);
}

}  // namespace w4
