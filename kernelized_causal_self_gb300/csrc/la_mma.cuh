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

#include "la_tc_common.cuh"

namespace la {
namespace mma {

using bf16 = __nv_bfloat16;

constexpr int kC = 64;  // rows (tokens) of a tile

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

__device__ __forceinline__ void stsm(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(a), "r"(b), "r"(c), "r"(d)
               : "memory");
}

// A lane's offsets in a tile, for the accesses below. Chunk c of a row r of any eight is
// at (c ^ r) within its row, and tiles are aligned to their rows, so moving on by whole
// column pairs is one exclusive or of the lane's address, and by rows an immediate.
template <int COLS>
struct Lane {
  uint32_t a, b;
  __device__ __forceinline__ Lane() {
    const int l = threadIdx.x & 31, r = (l & 7) + ((l >> 4) << 3);
    a = (l & 15) * COLS * 2 + (((l >> 4) ^ (l & 7)) << 4);
    b = r * COLS * 2 + ((((l >> 3) & 1) ^ (l & 7)) << 4);
  }
  // the 16 x 16 fragments at (row, 16 * pair), row a multiple of 8:
  // A, rows of the tile as rows of A. (Also the layout of two neighbouring accumulator
  // tiles: r[0], r[1] are rows l / 4, l / 4 + 8 of the first, r[2], r[3] of the second.)
  __device__ __forceinline__ void load_a(uint32_t (&r)[4], uint32_t base, int row, int pair) const {
    ldsm(r, ((base + a) ^ (pair << 5)) + row * COLS * 2);
  }
  // A, columns of the tile as rows of A
  __device__ __forceinline__ void load_a_t(uint32_t (&r)[4], uint32_t base, int row, int pair) const {
    ldsm_t(r, ((base + b) ^ (pair << 5)) + row * COLS * 2);
  }
  // B for two neighbouring column tiles (r[0], r[1] and r[2], r[3]), rows of the tile as
  // columns of B
  __device__ __forceinline__ void load_b(uint32_t (&r)[4], uint32_t base, int row, int pair) const {
    ldsm(r, ((base + b) ^ (pair << 5)) + row * COLS * 2);
  }
  // the same, rows of the tile as rows of B
  __device__ __forceinline__ void load_b_t(uint32_t (&r)[4], uint32_t base, int row, int pair) const {
    ldsm_t(r, ((base + a) ^ (pair << 5)) + row * COLS * 2);
  }
  // two neighbouring accumulator tiles, packed as load_a has them
  __device__ __forceinline__ void store(uint32_t base, int row, int pair, const float (&c)[4],
                                        const float (&d)[4]) const;
};

// Two floats rounded to bf16, `lo` in the lower half.
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float lo_of(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_of(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ float2 both_of(uint32_t u) { return make_float2(lo_of(u), hi_of(u)); }

template <int COLS>
__device__ __forceinline__ void Lane<COLS>::store(uint32_t base, int row, int pair,
                                                  const float (&c)[4], const float (&d)[4]) const {
  stsm(((base + a) ^ (pair << 5)) + row * COLS * 2, pack2(c[0], c[1]), pack2(c[2], c[3]),
       pack2(d[0], d[1]), pack2(d[2], d[3]));
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the same from zero
__device__ __forceinline__ void mma16816_0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                           uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// The halves of an accumulator's row pairs (columns 2 (l % 4) + {0, 1} of rows l / 4 and
// l / 4 + 8), two float32 at a time
__device__ __forceinline__ float2& pair_of(float (&c)[4], int h) {
  return *reinterpret_cast<float2*>(&c[2 * h]);
}
using tcx::fma2;
using tcx::mul2;
using tcx::sub2;

template <int NT>
__device__ __forceinline__ void scale_rows(float (&c)[NT][4], float top, float bottom) {
  const float2 t = make_float2(top, top), b = make_float2(bottom, bottom);
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    pair_of(c[j], 0) = mul2(pair_of(c[j], 0), t);
    pair_of(c[j], 1) = mul2(pair_of(c[j], 1), b);
  }
}

// A pair of float32 weights as two bf16 pairs, whose sum has 16 bits of it
__device__ __forceinline__ uint2 split_pair(float2 w) {
  const uint32_t hi = pack2(w.x, w.y);
  const float2 r = sub2(w, both_of(hi));
  return make_uint2(hi, pack2(r.x, r.y));
}

__device__ __forceinline__ uint32_t fma_bf2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

// bf16 pair u times such weights as the sum of two bf16 pairs, 16 bits of the product:
// hi = u w.x, whose remainder has at most eight bits and is exact, plus u w.y.
__device__ __forceinline__ void scale_split(uint32_t u, uint2 w, uint32_t& hi, uint32_t& lo) {
  hi = fma_bf2(u, w.x, 0x80008000u);  // (-0: a product of -0 stays one)
  lo = fma_bf2(u, w.y, fma_bf2(u, w.x, hi ^ 0x80008000u));
}

// bf16 pair u times float32 weights as the sum of three bf16 pairs, 24 bits of the product
__device__ __forceinline__ void scale_split3(uint32_t u, float2 w, uint32_t& hi, uint32_t& mid,
                                             uint32_t& lo) {
  const float2 p = mul2(both_of(u), w);
  hi = pack2(p.x, p.y);
  float2 r = sub2(p, both_of(hi));
  mid = pack2(r.x, r.y);
  r = sub2(r, both_of(mid));
  lo = pack2(r.x, r.y);
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

// x, in a way that keeps what is computed from it where it is used: hoisted out of a
// chunk loop, the addresses would hold registers through it.
__device__ __forceinline__ int here(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// 64 rows of COLS columns, from column c0 of rows of `width` elements, to a tile;
// rows from `rows` on and columns past `width` become zero (nothing is read there).
template <int COLS, int THREADS>
__device__ __forceinline__ void load_tile(uint32_t base, const bf16* src, int rows, int width,
                                          int c0) {
  constexpr int PER = COLS / 8, STEP = THREADS / PER;  // rows the threads cover at once
  static_assert(STEP % 8 == 0, "a thread's chunk stays where it is in its rows");
  const int tid = here(threadIdx.x), row = tid / PER, chunk = tid % PER;
  const uint32_t to = base + row * COLS * 2 + ((chunk ^ (row & 7)) << 4);
  const bf16* from = src + (size_t)row * width + c0 + chunk * 8;
  const bool wide = c0 + chunk * 8 < width;
  if (rows >= kC && c0 + COLS <= width) {  // (uniform: every chunk but a sequence's last)
#pragma unroll
    for (int i = 0; i < kC / STEP; ++i)
      cp_async16(to + i * STEP * COLS * 2, from + (uint32_t)(i * STEP * width), true);
    return;
  }
#pragma unroll
  for (int i = 0; i < kC / STEP; ++i) {
    const bool live = wide && row + i * STEP < rows;
    cp_async16(to + i * STEP * COLS * 2, live ? from + (size_t)i * STEP * width : src, live);
  }
}

// Rows r0 .. r0 + 15 of such a tile by one warp, from src on; `rows` of them, the others zero
template <int COLS>
__device__ __forceinline__ void load_rows(uint32_t base, int r0, const bf16* src, int rows, int width) {
  constexpr int PER = COLS / 8, STEP = 32 / PER;
  const int l = here(threadIdx.x & 31), row = l / PER, chunk = l % PER;
#pragma unroll
  for (int i = 0; i < 16 / STEP; ++i) {
    const int r = row + i * STEP;
    const bool live = chunk * 8 < width && r < rows;
    cp_async16(base + (r0 + r) * COLS * 2 + ((chunk ^ (r & 7)) << 4),
               live ? src + (size_t)r * width + chunk * 8 : src, live);
  }
}

// Rows r0 .. r0 + 15 of a warp's 16 x 64 result, through those rows of the tile at `tile`
// (the warp's own meanwhile), written in 16-byte pieces to rows of `width` elements at
// dst; `live` rows of them, columns up to `width`.
template <int COLS>
__device__ __forceinline__ void store_rows(const Lane<COLS>& ln, uint32_t tile, int r0,
                                           const float (&c)[8][4], bf16* dst, int live, int width,
                                           int stride) {
  const int l = here(threadIdx.x & 31), r = l >> 3, ch = l & 7;
  __syncwarp();
#pragma unroll
  for (int jp = 0; jp < 4; ++jp) ln.store(tile, r0, jp, c[2 * jp], c[2 * jp + 1]);
  __syncwarp();
  const uint32_t at = tile + (r0 + r) * COLS * 2 + ((ch ^ r) << 4);
  bf16* to = dst + (size_t)r * stride + ch * 8;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"((at ^ ((e & 1) << 6)) + e * 4 * COLS * 2));
    if (e * 4 + r < live && ch * 8 < width)
      __stcs(reinterpret_cast<uint4*>(to + (size_t)e * 4 * stride), v);
  }
}

// Rows r0.. of a tile's first 64 columns times c, summed over the columns: rows l / 4 and
// l / 4 + 8
template <int COLS>
__device__ __forceinline__ float2 row_dots(const Lane<COLS>& ln, uint32_t tile, int r0,
                                           float (&c)[8][4]) {
  float2 top = make_float2(0.f, 0.f), bottom = top;
#pragma unroll
  for (int jp = 0; jp < 4; ++jp) {
    uint32_t r[4];
    ln.load_a(r, tile, r0, jp);
    top = fma2(both_of(r[0]), pair_of(c[2 * jp], 0), top);
    bottom = fma2(both_of(r[1]), pair_of(c[2 * jp], 1), bottom);
    top = fma2(both_of(r[2]), pair_of(c[2 * jp + 1], 0), top);
    bottom = fma2(both_of(r[3]), pair_of(c[2 * jp + 1], 1), bottom);
  }
  float2 s = make_float2(top.x + top.y, bottom.x + bottom.y);
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
  }
  return s;
}

// An accumulator tile kept for the thread's own later use, and its dot with another's
__device__ __forceinline__ float4 keep_tile(const float (&a)[4]) {
  return make_float4(a[0], a[1], a[2], a[3]);
}
__device__ __forceinline__ float2 dot_kept(float4 kept, float (&a)[4], float2 s) {
  s = fma2(make_float2(kept.x, kept.y), pair_of(a, 0), s);
  return fma2(make_float2(kept.z, kept.w), pair_of(a, 1), s);
}

// What is left of a, b behind their bf16 pair
__device__ __forceinline__ float2 rest_of(float2 w, uint32_t hi) { return sub2(w, both_of(hi)); }

// A state's rows r0 .. as an operand, or (REST) what that operand's rounding leaves
template <bool REST = false, int NT>
__device__ __forceinline__ void store_op(const Lane<64>& ln, uint32_t op, int r0, int c0,
                                         const float (&x)[NT][4]) {
#pragma unroll
  for (int jp = 0; jp < NT / 2; ++jp) {
    float y[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int h = 0; h < 4; h += 2) {
        const float2 w = make_float2(x[2 * jp + t][h], x[2 * jp + t][h + 1]);
        const float2 v = REST ? rest_of(w, pack2(w.x, w.y)) : w;
        y[t][h] = v.x;
        y[t][h + 1] = v.y;
      }
    ln.store(op, r0, c0 / 16 + jp, y[0], y[1]);
  }
}

// x += (columns 16 col16.. of tile `a`, weighted along its rows)^T (columns c0.. of tile
// `b`), over 64 rows. The weights: a table of split_pair's of neighbouring rows; EXACT: of
// float32 pairs, and x is begun from zero.
template <bool EXACT, int COLS, int NT>
__device__ __forceinline__ void add_outer(const Lane<COLS>& la, const Lane<64>& lb, float (&x)[NT][4],
                                          uint32_t a, const float* weights, int col16, uint32_t b, int c0) {
  const uint2* w = reinterpret_cast<const uint2*>(weights) + (threadIdx.x & 3);
#pragma unroll
  for (int at = 0; at < kC; at += 16) {
    uint32_t f[4], hi[4], lo[4], last[4], y[NT / 2][4];
    la.load_a_t(f, a, at, col16);
#pragma unroll
    for (int jp = 0; jp < NT / 2; ++jp) lb.load_b_t(y[jp], b, at, c0 / 16 + jp);
    const uint2 w0 = w[at / 2], w8 = w[at / 2 + 4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint2 v = e < 2 ? w0 : w8;
      if (EXACT)
        scale_split3(f[e], make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), hi[e], lo[e], last[e]);
      else
        scale_split(f[e], v, hi[e], lo[e]);
    }
#pragma unroll
    for (int jp = 0; jp < NT / 2; ++jp) {
      if (EXACT && at == 0) {
        mma16816_0(x[2 * jp], hi, y[jp][0], y[jp][1]);
        mma16816_0(x[2 * jp + 1], hi, y[jp][2], y[jp][3]);
      } else {
        mma16816(x[2 * jp], hi, y[jp][0], y[jp][1]);
        mma16816(x[2 * jp + 1], hi, y[jp][2], y[jp][3]);
      }
    }
#pragma unroll
    for (int jp = 0; jp < NT / 2; ++jp) {
      mma16816(x[2 * jp], lo, y[jp][0], y[jp][1]);
      mma16816(x[2 * jp + 1], lo, y[jp][2], y[jp][3]);
    }
    if (EXACT)
#pragma unroll
      for (int jp = 0; jp < NT / 2; ++jp) {
        mma16816(x[2 * jp], last, y[jp][0], y[jp][1]);
        mma16816(x[2 * jp + 1], last, y[jp][2], y[jp][3]);
      }
  }
}

// c = A B, or (ADD) c += A B, for A's fragments of 16 rows by 16 KS and the 64 columns of
// B, which are the rows of the tile, or (TRANS) B's rows are
template <bool TRANS, bool ADD = false, int KS>
__device__ __forceinline__ void product(const Lane<64>& ln, float (&c)[8][4],
                                        const uint32_t (&a)[KS][4], uint32_t tile) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int jp = 0; jp < 4; ++jp) {
      uint32_t b[4];
      if (TRANS)
        ln.load_b_t(b, tile, 16 * ks, jp);
      else
        ln.load_b(b, tile, 16 * jp, ks);
      if (ks == 0 && !ADD) {
        mma16816_0(c[2 * jp], a[ks], b[0], b[1]);
        mma16816_0(c[2 * jp + 1], a[ks], b[2], b[3]);
      } else {
        mma16816(c[2 * jp], a[ks], b[0], b[1]);
        mma16816(c[2 * jp + 1], a[ks], b[2], b[3]);
      }
    }
}

// A block of 16 x 16 of A B^T: A's fragments, B the rows 16 cb.. of a tile
template <int COLS, int KS>
__device__ __forceinline__ void block_product(const Lane<COLS>& ln, float (&p)[2][4],
                                              const uint32_t (&a)[KS][4], uint32_t tile, int cb) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    uint32_t b[4];
    ln.load_b(b, tile, 16 * cb, ks);
    if (ks == 0) {
      mma16816_0(p[0], a[ks], b[0], b[1]);
      mma16816_0(p[1], a[ks], b[2], b[3]);
    } else {
      mma16816(p[0], a[ks], b[0], b[1]);
      mma16816(p[1], a[ks], b[2], b[3]);
    }
  }
}

// A pair of such a block as element e of an A operand of TERMS bf16 terms
template <int TERMS>
__device__ __forceinline__ void keep_terms(uint32_t (&out)[TERMS][4], int e, float2 w) {
#pragma unroll
  for (int i = 0; i < TERMS; ++i) {
    out[i][e] = pack2(w.x, w.y);
    w = rest_of(w, out[i][e]);
  }
}

// The block times weights that are a product of one of the column, from `cols`, and one of
// A's rows l / 4 and l / 4 + 8
template <int COLS, int KS, int TERMS>
__device__ __forceinline__ void weighted_block(const Lane<COLS>& ln, uint32_t (&out)[TERMS][4],
                                               const uint32_t (&a)[KS][4], uint32_t tile, int cb,
                                               const float* cols, const float (&rows)[2]) {
  const int col = (threadIdx.x & 3) * 2;
  float p[2][4];
  block_product(ln, p, a, tile, cb);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float2 c = *reinterpret_cast<const float2*>(cols + 16 * cb + 8 * t + col);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      keep_terms(out, 2 * t + h, mul2(pair_of(p[t], h), mul2(c, make_float2(rows[h], rows[h]))));
  }
}

// The block where A's rows and B's are the same tokens, times exp2 of the gates between a
// row's token and a column's (hi + lo: their sums up to each token), half of it zero. LOWER:
// A's rows are the later tokens, else B's are.
template <bool LOWER, int COLS, int KS, int TERMS>
__device__ __forceinline__ void diagonal_block(const Lane<COLS>& ln, uint32_t (&out)[TERMS][4],
                                               const uint32_t (&a)[KS][4], uint32_t tile, int cb,
                                               const float* hi, const float* lo) {
  const int l = threadIdx.x & 31, row = l >> 2, col = (l & 3) * 2;
  float p[2][4];
  block_product(ln, p, a, tile, cb);
  hi += 16 * cb;
  lo += 16 * cb;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float2 ch = *reinterpret_cast<const float2*>(hi + 8 * t + col),
                 cl = *reinterpret_cast<const float2*>(lo + 8 * t + col);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float gh = hi[row + 8 * h], gl = lo[row + 8 * h];
      const float2 rh = make_float2(gh, gh), rl = make_float2(gl, gl);
      const float2 d = LOWER ? sub2(rh, ch) : sub2(ch, rh), r = LOWER ? sub2(rl, cl) : sub2(cl, rl);
      float2 w = mul2(pair_of(p[t], h), make_float2(ex2(d.x + r.x), ex2(d.y + r.y)));
      const int c = 8 * t + col, i = row + 8 * h;
      w.x = (LOWER ? c <= i : c >= i) ? w.x : 0.f;
      w.y = (LOWER ? c + 1 <= i : c + 1 >= i) ? w.y : 0.f;
      keep_terms(out, 2 * t + h, w);
    }
  }
}

// c += the block's product with the rows 16 cb.. of a tile of 64 columns
template <int TERMS>
__device__ __forceinline__ void add_block(const Lane<64>& ln, float (&c)[8][4],
                                          const uint32_t (&a)[TERMS][4], uint32_t tile, int cb) {
#pragma unroll
  for (int jp = 0; jp < 4; ++jp) {
    uint32_t b[4];
    ln.load_b_t(b, tile, 16 * cb, jp);
#pragma unroll
    for (int i = 0; i < TERMS; ++i) {
      mma16816(c[2 * jp], a[i], b[0], b[1]);
      mma16816(c[2 * jp + 1], a[i], b[2], b[3]);
    }
  }
}

}  // namespace mma
}  // namespace la
