// What the gated projections' tensor-core kernels (la_ffn_tc.cu in bf16, la_ffn_tc32.cu in float32)
// share: which tile of which product a pair of CTAs makes, how sums are cut, and tensor maps.
#pragma once

#include "la_checkpoint.cuh"
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace ffn {

using namespace tcx;

enum Kind { kForward, kGrads, kDx, kDw };

constexpr int kWarps = 8;          // warps of results: two for each 32 rows, half the columns each
constexpr int kTileBytes = 16384;  // 128 x 64 bf16
constexpr int kStore = 4096;       // a warp's staging tile: 32 rows of 128 bytes

struct Grid {
  int rows, cols;  // of the result (kForward, kGrads: T, F)
  int m_tiles, n_tiles, splits, tiles;
  int steps, per;  // k steps of 64 in the whole sum; kDx: of one of its two parts
};

struct Tile {
  int m, n, part, split;  // part: kDw: dwg or dwu
};

template <int KIND>
__device__ __forceinline__ Tile tile_of(const Grid& a, uint32_t t) {
  Tile r;
  const uint32_t row = t / (uint32_t)a.n_tiles, mat = row / (uint32_t)a.m_tiles;
  r.n = (int)(t - row * (uint32_t)a.n_tiles);
  r.m = (int)(row - mat * (uint32_t)a.m_tiles);
  r.part = KIND == kDw ? (int)(mat & 1) : 0;
  r.split = (int)(KIND == kDw ? mat >> 1 : mat);
  return r;
}

// Where a split's steps begin (the whole sum in kForward and kGrads, which are not cut). At most
// 2^18 steps and 16 parts.
template <int KIND>
__device__ __forceinline__ int first_step(const Grid& a, int split) {
  if (KIND == kForward || KIND == kGrads || a.splits == 1) return split ? a.steps : 0;
  return (int)((uint32_t)(a.steps * split) / (uint32_t)a.splits);
}

// Wait codes of these kernels (la_workspace_wait_site)
enum Site { kSiteEmpty = 81, kSiteFull, kSiteAccEmpty, kSiteAccFull, kSiteDhFull, kSiteDhEmpty, kSiteDrain };

inline int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

// Parts of a sum of `steps` steps of 64 that cost `step` SM clocks each: the ones with the least time
// by this count: behind a tile's last step about 3000 clocks until its results are out; a
// part's results are 8 bytes a value more to move (written and read again, at about 3500 bytes a
// clock over all SMs), by one more launch.
inline int splits_of(int tiles, int steps, int step, double values) {
  int best = 1;
  double least = 0;
  for (int s = 1; s <= 16 && s <= steps; ++s) {
    const int waves = ceil_div((long long)tiles * s, 76);  // (pairs of the 152 SMs)
    const double t = (double)waves * ceil_div(steps, s) * step + 3000 + (s > 1 ? 4000 + s * values * 8 / 3500 : 0);
    if (s == 1 || t < least) best = s, least = t;
  }
  return best;
}

// rows of `cols` bf16 `ld` elements apart, in boxes of b1 rows by 64 columns; `mats` such matrices
inline bool rows_map(CUtensorMap* m, const void* p, long long cols, long long rows, long long ld, int b1, int mats = 1) {
  // (a single row's distance is of no use, but has to be one that the map takes)
  return make_tmap_bf16_strided(m, p, cols, rows, mats, rows > 1 ? ld : cols, (size_t)rows * cols, 64, b1, 1);
}

// the same in float32, in boxes of 32 rows by 32 columns
inline bool rows_map_f32(CUtensorMap* m, const void* p, long long cols, long long rows, long long ld, int mats = 1) {
  return make_tmap_f32_strided(m, p, cols, rows, mats, rows > 1 ? ld : cols, (size_t)rows * cols, 32, 32, 1);
}

}  // namespace ffn
}  // namespace la
