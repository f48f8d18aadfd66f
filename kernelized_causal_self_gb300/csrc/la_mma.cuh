// Warp-level matrix products (m16n8k16, bf16 operands in registers, float32 sums) and
// the swizzled shared-memory tiles that feed them.
//
// A tile is 64 rows of 64 or 128 bf16; 16-byte chunk c of row r lies at chunk
// c ^ (r & 7), so that the eight rows a matrix load reads touch eight different bank
// groups. Fragments, with l the lane: an accumulator's elements 0, 1 are row l / 4,
// columns 2 (l % 4) + {0, 1}, elements 2, 3 the same columns of row l / 4 + 8.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "la_tc.cuh"

namespace la {
namespace mma {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;  // rows (tokens) of a tile

template <int COLS>
__device__ __forceinline__ uint32_t tile_at(uint32_t base, int row, int chunk) {
  return base + (uint32_t)(row * COLS * 2 + ((chunk ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// The four matrix fragments, each 16 x 16 of a tile with origin (row, 8 * chunk):
// A, rows of the tile as rows of A
template <int COLS>
__device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t base, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm(r, tile_at<COLS>(base, row + (l & 15), chunk + (l >> 4)));
}
// A, columns of the tile as rows of A
template <int COLS>
__device__ __forceinline__ void load_a_t(uint32_t (&r)[4], uint32_t base, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm_t(r, tile_at<COLS>(base, row + (l & 7) + ((l >> 4) << 3), chunk + ((l >> 3) & 1)));
}
// B for two neighbouring column tiles (r[0], r[1] and r[2], r[3]), rows of the tile as
// columns of B
template <int COLS>
__device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t base, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm(r, tile_at<COLS>(base, row + (l & 7) + ((l >> 4) << 3), chunk + ((l >> 3) & 1)));
}
// the same, rows of the tile as rows of B
template <int COLS>
__device__ __forceinline__ void load_b_t(uint32_t (&r)[4], uint32_t base, int row, int chunk) {
  const int l = threadIdx.x & 31;
  ldsm_t(r, tile_at<COLS>(base, row + (l & 15), chunk + (l >> 4)));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two floats rounded to bf16, `lo` in the lower half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_of(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

// bf16 pair u times (x, y), as the sum of two bf16 pairs: the product to 16 bits
__device__ __forceinline__ void scale_split(uint32_t u, float x, float y, uint32_t& hi,
                                            uint32_t& lo) {
  const float a = lo_of(u) * x, b = hi_of(u) * y;
  hi = pack2(a, b);
  lo = pack2(a - lo_of(hi), b - hi_of(hi));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 64 rows of COLS columns, from column c0 of rows of `width` elements, to a tile;
// rows from `rows` on and columns past `width` become zero (nothing is read there).
template <int COLS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t base, const bf16* src, int rows, int width,
                                          int c0) {
  constexpr int PER = COLS / 8;
#pragma unroll
  for (int i = 0; i < kC * PER / THREADS; ++i) {
    const int at = threadIdx.x + i * THREADS, row = at / PER, chunk = at % PER;
    const bool live = row < rows && c0 + chunk * 8 < width;
    cp_async16(tile_at<COLS>(base, row, chunk),
               live ? src + (size_t)row * width + c0 + chunk * 8 : src, live);
  }
}

}  // namespace mma
}  // namespace la
