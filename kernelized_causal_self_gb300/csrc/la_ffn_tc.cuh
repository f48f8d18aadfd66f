// What the gated projections' tensor-core kernels (la_ffn_tc.cu in bf16, la_ffn_tc32.cu in float32)
// share: which tile of which product a pair of CTAs makes, how sums are cut, and tensor maps.
#pragma once

#include <algorithm>

#include "la_checkpoint.cuh"
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_pair.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace ffn {

using namespace tcx;

// The products that one launch makes: a = x wg^T and u = x wu^T for h, or for da and du; or the sums
// behind those, dx = da wg + du wu and dwg = da^T x, dwu = du^T x
enum Kind { kForward, kGrads, kSums };

constexpr int kWarps = 8;          // warps of results: two for each 32 rows, half the columns each
constexpr int kTileBytes = 16384;  // 128 x 64 bf16
constexpr int kStore = 4096;       // a warp's staging tile: 32 rows of 128 bytes

struct Grid {
  int rows, cols;  // of the result (kForward, kGrads: T, F)
  int m_tiles, n_tiles, splits, tiles;
  int steps, per;  // k steps of 64 in the whole sum; dx: of one of its two parts
};

struct Grids {
  Grid g[2];  // kSums: dx's, then those of dwg and dwu; else the first alone
  int extra;  // tiles of dwg and dwu that pairs with one tile of dx less take first
};

// The i-th tile of pair p of `pairs`, -1 behind its last. Tiles are dealt in turn; dx's and the
// weights' take different times, so the pairs that get one of dx's less (from `more` on) take `extra`
// of the weights' before these are dealt to all, and are the first to be dealt the rest.
template <int KIND>
__device__ __forceinline__ int dealt(const Grids& a, int p, int pairs, int i) {
  if (KIND != kSums) {
    const int t = p + i * pairs;
    return t < a.g[0].tiles ? t : -1;
  }
  const int nx = a.g[0].tiles, more = nx % pairs, own = nx / pairs + (p < more);
  if (i < own) return p + i * pairs;
  i -= own;
  const int less = pairs - more, ahead = a.extra * less;
  int w;
  if (p < more)
    w = ahead + i * pairs + less + p;
  else
    w = i < a.extra ? i * less + (p - more) : ahead + (i - a.extra) * pairs + (p - more);
  return w < a.g[1].tiles ? nx + w : -1;
}

struct Tile {
  int dw;                 // which grid's
  int m, n, part, split;  // part: dwg or dwu
};

template <int KIND>
__device__ __forceinline__ Tile tile_of(const Grids& a, uint32_t t) {
  Tile r;
  r.dw = KIND == kSums && t >= (uint32_t)a.g[0].tiles;
  if (r.dw) t -= (uint32_t)a.g[0].tiles;
  const Grid& g = a.g[r.dw];
  const uint32_t row = t / (uint32_t)g.n_tiles, mat = row / (uint32_t)g.m_tiles;
  r.n = (int)(t - row * (uint32_t)g.n_tiles);
  r.m = (int)(row - mat * (uint32_t)g.m_tiles);
  r.part = r.dw ? (int)(mat & 1) : 0;
  r.split = (int)(r.dw ? mat >> 1 : mat);
  return r;
}

// Where a split's steps begin (kForward's and kGrads' sums are not cut). At most 2^18 steps and 512 parts.
__device__ __forceinline__ int first_step(const Grid& g, int split) {
  return g.splits == 1 ? (split ? g.steps : 0) : (int)((uint32_t)(g.steps * split) / (uint32_t)g.splits);
}

// Wait codes of these kernels (la_workspace_wait_site)
enum Site { kSiteEmpty = 81, kSiteFull, kSiteAccEmpty, kSiteAccFull, kSiteDhFull, kSiteDhEmpty, kSiteDrain };

inline int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

// What a tile of sums costs in SM clocks: 64 terms, and its results, which are written while the next tile
// is summed; and the most steps that a part may have
struct Costs {
  int step, results, most;
};

// The grids of dx and of dwg, dwu, whose tiles one launch deals to 76 pairs of CTAs, with the sums
// cut into the parts, and the tiles dealt, that take the least time by this count: a tile costs its
// steps and 500 clocks more, or its results if they take longer; a part's results are 8 bytes a value
// more to move (written and read again, at about 3500 bytes a clock over all SMs), by one more launch.
// T 25, C 1536, F 5120 in bf16: all pairs done after 19 to 20 us; not counting results some after 15 and
// some after 26.
inline Grids count_sums_grids(int T, int C, int F, Costs cost) {
  constexpr int P = 76;
  Grids r{};
  Grid &x = r.g[0], &w = r.g[1];
  x.rows = T, w.rows = F;
  x.cols = w.cols = C;
  x.m_tiles = ceil_div(T, 256), w.m_tiles = ceil_div(F, 256);
  x.n_tiles = w.n_tiles = ceil_div(C, 256);
  x.per = ceil_div(F, 64);
  x.steps = 2 * x.per, w.steps = ceil_div(T, 64);
  const long long nx = (long long)x.m_tiles * x.n_tiles, nw = 2LL * w.m_tiles * w.n_tiles;
  const int tried[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 14, 16, 24, 32};
  const int least_x = ceil_div(x.steps, cost.most), least_w = ceil_div(w.steps, cost.most);
  const auto tile = [&](const Grid& g, int splits) {
    const double sums = (double)ceil_div(g.steps, splits) * cost.step + 500;
    return sums > cost.results ? sums : cost.results;
  };
  double least = 0;
  for (int try_x : tried)
    for (int try_w : tried) {
      const int sx = std::max(try_x, least_x), sw = std::max(try_w, least_w);
      if (sx > x.steps || sw > w.steps) continue;
      const long long tx = nx * sx, tw = nw * sw, more = tx % P, less = P - more;
      const double cx = tile(x, sx), cw = tile(w, sw);
      double moved = 0;
      if (sx > 1 || sw > 1)
        moved = 4000 + ((sx > 1 ? (double)sx * T * C : 0) + (sw > 1 ? 2.0 * sw * F * C : 0)) * 8 / 3500;
      for (int up = 0; up < 2; ++up) {
        long long extra = more ? (long long)(cx / cw) + up : 0;
        if (extra * less > tw) extra = tw / less;
        const long long rest = tw - extra * less;
        const double b = (tx / P) * cx + (extra + (rest + P - 1) / P) * cw;
        const double a = more ? (tx / P + 1) * cx + (rest > less ? (rest - less + P - 1) / P : 0) * cw : 0;
        const double t = (a > b ? a : b) + moved;
        if (least == 0 || t < least) least = t, x.splits = sx, w.splits = sw, r.extra = (int)extra;
      }
    }
  x.tiles = (int)(nx * x.splits);
  w.tiles = (int)(nw * w.splits);
  return r;
}

// (counted once for a size: a call asks three times, 0.6 us each)
inline const Grids& sums_grids(int T, int C, int F, Costs cost) {
  thread_local struct {
    int T, C, F, step;
    Grids grids;
  } last{};
  if (last.T != T || last.C != C || last.F != F || last.step != cost.step)
    last = {T, C, F, cost.step, count_sums_grids(T, C, F, cost)};
  return last.grids;
}

// Floats of the parts of dx, then of dwg and dwu
inline size_t dx_parts(const Grids& g) { return g.g[0].splits > 1 ? (size_t)g.g[0].splits * g.g[0].rows * g.g[0].cols : 0; }
inline size_t dw_parts(const Grids& g) { return g.g[1].splits > 1 ? 2 * (size_t)g.g[1].splits * g.g[1].rows * g.g[1].cols : 0; }

// The one grid of a = x wg^T, u = x wu^T
inline Grids products_grid(int T, int C, int F) {
  Grids r{};
  Grid& g = r.g[0];
  g.rows = T, g.cols = F;
  g.m_tiles = ceil_div(T, 256), g.n_tiles = ceil_div(F, 128);
  g.splits = 1;
  g.tiles = g.m_tiles * g.n_tiles;
  g.steps = ceil_div(C, 64);
  return r;
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

// The cut ones of dx, dwg and dwu, joined from their parts
inline cudaError_t join_sums(const FfnGate& f, const Grids& g, const float* parts, cudaStream_t st) {
  Join j[3];
  int n = 0;
  const Grid &x = g.g[0], &w = g.g[1];
  if (x.splits > 1) j[n++] = Join{parts, f.dx, f.dx_stride, x.rows, x.splits};
  if (w.splits > 1) {
    const float* pw = parts + dx_parts(g);
    j[n++] = Join{pw, f.dwg, f.C, w.rows, w.splits};
    j[n++] = Join{pw + dw_parts(g) / 2, f.dwu, f.C, w.rows, w.splits};
  }
  return n ? ffn_join(j, n, f.C, f.dtype, st) : cudaSuccess;
}

}  // namespace ffn
}  // namespace la
