// Gated recurrence's backward in bf16 on tensor cores (D, M up to 64).
//
// Per chunk of 64 tokens, with S the state before it and E the loss's gradient with
// respect to the state after it (G, L as in the forward; W_ij = exp(G - G_j)):
//   dQ = ((dO V^T) * L) K + diag(exp(G_i)) dO S^T
//   dK = ((dO V^T) * L)^T Q + diag(exp(G - G_j)) V E^T
//   dV = ((Q K^T) * L)^T dO + diag(exp(G - G_j)) K E
//   S' = exp(G) S + (diag(exp(G - G_j)) K)^T V,  E' = exp(G) E + (diag(exp(G_i)) Q)^T dO
// A gate g_t scales what passes from tokens before t to tokens from t on:
//   dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} a_i + sum_{j < t} b_j + exp(G) <S, E>
//   X = (Q K^T) * (dO V^T) * L,  a_i = exp(G_i) q_i S dO_i,  b_j = exp(G - G_j) k_j E v_j
// X's sum is one over s >= t of its strict row sums less its column sums: both of the
// same float32 products, which cancel to float32 where they have to.
//
// S is known going forward and E going back, so a CTA walks its segment of a few chunks
// forward (dQ, a, and each chunk's S in bf16 to scratch of the CTA's own) and then back
// (dK, dV, dg). Segments are short enough (up to 8 chunks) that the tiles' second read
// comes from L2. Both walks keep their state in float32 accumulators; rounded to bf16
// are the operands (L's products, the copies of S and E that are multiplied) and the
// gradients.
#include "la_gated.cuh"
#include "la_gated_mma.cuh"
#include "la_mma.cuh"
#include "la_tc_common.cuh"

namespace la {

using namespace mma;

namespace {

constexpr int kThreads = 128, kResident = 2, kMaxChunks = 8;
constexpr int kTile = kC * 64 * 2;
constexpr int kStage = 4 * kTile;  // Q, K, V, dO
constexpr int kOp = kTile;         // S or E in bf16, [d][m], one of two
// floats: per-warp G, W, V tables; a of the segment; per parity: row sums of X by warp,
// column sums, b, <S, E> by warp
constexpr int kTables = 4 * 3 * kC, kAlpha = kMaxChunks * kC, kParts = 4 * kC + kC + kC + 4;
constexpr int kSmem = 2 * kStage + 2 * kOp + 4 * (kTables + kAlpha + 2 * kParts);

struct BwdArgs {
  const bf16 *q, *k, *v, *g, *dout;
  bf16 *dq, *dk, *dv, *dg;
  int D, M, N, BH, len, n_seg;
  const float *S, *E;    // per-segment entries (nullptr: one segment)
  const float *S0, *dS;  // one segment: the caller's (nullptr: zero)
  uint4* scratch;        // [CTA][kMaxChunks][4][kThreads]
};

// Rows 16 r.. of a tile of accumulators as bf16, through this warp's rows of the tile
// at `at`, in 16-byte pieces.
__device__ __forceinline__ void store_rows(uint8_t* tile, int r0, const float (&c)[8][4],
                                           bf16* dst, int live, int width) {
  const int lane = threadIdx.x & 31, row = lane >> 2, col = (lane & 3) * 2;
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint32_t*>(tile + tile_at<64>(0, r0 + row + 8 * h, j) + col * 2) =
          pack2(c[j][2 * h], c[j][2 * h + 1]);
  __syncwarp();
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int r = e * 4 + (lane >> 3), ch = lane & 7;
    if (r < live && ch * 8 < width)
      *reinterpret_cast<uint4*>(dst + (size_t)r * width + ch * 8) =
          *reinterpret_cast<const uint4*>(tile + tile_at<64>(0, r0 + r, ch));
  }
}

__device__ __forceinline__ void load_state(float (&x)[8][4], const float* from, int r0, int D,
                                           int M) {
  const int lane = threadIdx.x & 31, row = lane >> 2, col = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = r0 + row + 8 * h, m = 8 * j + col;
      float2 v = make_float2(0.f, 0.f);
      if (from && d < D && m < M) v = *reinterpret_cast<const float2*>(from + (size_t)d * M + m);
      x[j][2 * h] = v.x;
      x[j][2 * h + 1] = v.y;
    }
}

__device__ __forceinline__ void store_op(uint8_t* op, int r0, const float (&x)[8][4]) {
  const int lane = threadIdx.x & 31, row = lane >> 2, col = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<uint32_t*>(op + tile_at<64>(0, r0 + row + 8 * h, j) + col * 2) =
          pack2(x[j][2 * h], x[j][2 * h + 1]);
}

// this warp's rows of `tile` times c, summed over the columns: rows row, row + 8
__device__ __forceinline__ float2 row_dots(const uint8_t* tile, int r0, const float (&c)[8][4]) {
  const int lane = threadIdx.x & 31, row = lane >> 2, col = (lane & 3) * 2;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(tile + tile_at<64>(0, r0 + row, j) + col * 2);
    const uint32_t b = *reinterpret_cast<const uint32_t*>(tile + tile_at<64>(0, r0 + row + 8, j) + col * 2);
    s.x = fmaf(lo_of(a), c[j][0], fmaf(hi_of(a), c[j][1], s.x));
    s.y = fmaf(lo_of(b), c[j][2], fmaf(hi_of(b), c[j][3], s.y));
  }
#pragma unroll
  for (int o = 1; o < 4; o <<= 1) {
    s.x += __shfl_xor_sync(0xffffffffu, s.x, o);
    s.y += __shfl_xor_sync(0xffffffffu, s.y, o);
  }
  return s;
}

__device__ __forceinline__ void zero(float (&c)[8][4]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
}

__device__ __forceinline__ void scale_rows(float (&c)[8][4], float a, float b) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c[j][0] *= a;
    c[j][1] *= a;
    c[j][2] *= b;
    c[j][3] *= b;
  }
}

__global__ void __launch_bounds__(kThreads, kResident) gated_backward_kernel(const BwdArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = lane >> 2, col = (lane & 3) * 2;
  uint8_t* ops = smem + 2 * kStage;
  float* tables = reinterpret_cast<float*>(ops + 2 * kOp);
  float* Gs = tables + warp * 3 * kC;
  float *Ws = Gs + kC, *Vs = Ws + kC;
  float* alpha = tables + kTables;
  float* parts = alpha + kAlpha;
  const int r0 = ((warp + blockIdx.x) & 3) * 16, rb = r0 >> 4;
  uint4* scratch = a.scratch + (size_t)blockIdx.x * kMaxChunks * 4 * kThreads + tid;

  tc::pdl_wait();
  const int items = a.BH * a.n_seg;
  for (int item = blockIdx.x; item < items; item += gridDim.x) {
    const int bh = item / a.n_seg, seg = item % a.n_seg;
    const int tb = seg * a.len, te = min(tb + a.len, a.N);
    const int chunks = (te - tb + kC - 1) / kC;
    const size_t seq = (size_t)bh * a.N;
    const size_t DM = (size_t)a.D * a.M;
    auto load_chunk = [&](int c) {
      const int t0 = tb + c * kC, rows = min(kC, te - t0);
      const uint32_t at = base + (c & 1) * kStage;
      load_tile<64, kThreads>(at, a.q + (seq + t0) * a.D, rows, a.D, 0);
      load_tile<64, kThreads>(at + kTile, a.k + (seq + t0) * a.D, rows, a.D, 0);
      load_tile<64, kThreads>(at + 2 * kTile, a.v + (seq + t0) * a.M, rows, a.M, 0);
      load_tile<64, kThreads>(at + 3 * kTile, a.dout + (seq + t0) * a.M, rows, a.M, 0);
    };

    __syncthreads();  // the tiles of the item before are done with
    load_chunk(0);
    cp_async_commit();
    float2 g_next = load_gates(a.g + seq, tb, te);
    float x[8][4];  // S, then E
    load_state(x, a.S ? a.S + ((size_t)bh * (a.n_seg + 1) + seg) * DM : a.S0 ? a.S0 + bh * DM : nullptr,
               r0, a.D, a.M);
    store_op(ops, r0, x);

    // ---- forward: dQ, a
    for (int c = 0; c < chunks; ++c) {
      cp_async_wait<0>();
      __syncthreads();
      const float2 g = g_next;
      if (c + 1 < chunks) {
        load_chunk(c + 1);
        g_next = load_gates(a.g + seq, tb + (c + 1) * kC, te);
      }
      cp_async_commit();
      const float total = chunk_gates<false>(g, Gs, Ws);
      const float dec = gated_decay(total * kLn2);
      const uint32_t q_at = base + (c & 1) * kStage, k_at = q_at + kTile, v_at = k_at + kTile,
                     do_at = v_at + kTile, op = base + 2 * kStage + (c & 1) * kOp;
      // S of this chunk, for the way back
#pragma unroll
      for (int e = 0; e < 4; ++e)
        scratch[(c * 4 + e) * kThreads] =
            make_uint4(pack2(x[2 * e][0], x[2 * e][1]), pack2(x[2 * e][2], x[2 * e][3]),
                       pack2(x[2 * e + 1][0], x[2 * e + 1][1]), pack2(x[2 * e + 1][2], x[2 * e + 1][3]));
      uint32_t da[4][4];
      float dq[8][4];
      zero(dq);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) load_a<64>(da[ks], do_at, r0, 2 * ks);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
          uint32_t b[4];
          load_b<64>(b, op, 16 * jp, 2 * ks);
          mma16816(dq[2 * jp], da[ks], b[0], b[1]);
          mma16816(dq[2 * jp + 1], da[ks], b[2], b[3]);
        }
      const float gi[2] = {Gs[r0 + row], Gs[r0 + row + 8]};
      scale_rows(dq, ex2(gi[0]), ex2(gi[1]));
      const float2 al = row_dots(smem + (q_at - base), r0, dq);
      if ((lane & 3) == 0) {
        alpha[c * kC + r0 + row] = al.x;
        alpha[c * kC + r0 + row + 8] = al.y;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] *= dec;
#pragma unroll
      for (int jb = 0; jb < 4; ++jb) {
        if (jb <= rb) {
          float p[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            uint32_t b[4];
            load_b<64>(b, v_at, 16 * jb, 2 * ks);
            mma16816(p[0], da[ks], b[0], b[1]);
            mma16816(p[1], da[ks], b[2], b[3]);
          }
          uint32_t pa[4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float2 gj = *reinterpret_cast<const float2*>(&Gs[16 * jb + 8 * t + col]);
            float w[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int j = 8 * t + col, r = row + 8 * h;
              w[2 * h] = jb < rb || j <= r ? p[t][2 * h] * ex2(gi[h] - gj.x) : 0.f;
              w[2 * h + 1] = jb < rb || j + 1 <= r ? p[t][2 * h + 1] * ex2(gi[h] - gj.y) : 0.f;
            }
            pa[2 * t] = pack2(w[0], w[1]);
            pa[2 * t + 1] = pack2(w[2], w[3]);
          }
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {
            uint32_t b[4];
            load_b_t<64>(b, k_at, 16 * jb, 2 * jp);
            mma16816(dq[2 * jp], pa, b[0], b[1]);
            mma16816(dq[2 * jp + 1], pa, b[2], b[3]);
          }
        }
        if (c + 1 < chunks) {
          uint32_t ka[4], hi[4], lo[4];
          load_a_t<64>(ka, k_at, 16 * jb, 2 * rb);
          const float2 w0 = *reinterpret_cast<const float2*>(&Ws[16 * jb + col]);
          const float2 w8 = *reinterpret_cast<const float2*>(&Ws[16 * jb + 8 + col]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = e < 2 ? w0 : w8;
            scale_split(ka[e], w.x, w.y, hi[e], lo[e]);
          }
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {
            uint32_t b[4];
            load_b_t<64>(b, v_at, 16 * jb, 2 * jp);
            mma16816(x[2 * jp], hi, b[0], b[1]);
            mma16816(x[2 * jp + 1], hi, b[2], b[3]);
            mma16816(x[2 * jp], lo, b[0], b[1]);
            mma16816(x[2 * jp + 1], lo, b[2], b[3]);
          }
        }
      }
      if (c + 1 < chunks) store_op(ops + ((c + 1) & 1) * kOp, r0, x);
      const int t0 = tb + c * kC + r0;
      store_rows(smem + (do_at - base), r0, dq, a.dq + (seq + t0) * a.D, te - t0, a.D);
    }

    // ---- back: dK, dV, dg
    __syncthreads();
    load_chunk(chunks - 1);  // (its dO rows were written over)
    cp_async_commit();
    g_next = load_gates(a.g + seq, tb + (chunks - 1) * kC, te);
    load_state(x, a.E ? a.E + ((size_t)bh * (a.n_seg + 1) + seg + 1) * DM : a.dS ? a.dS + bh * DM : nullptr,
               r0, a.D, a.M);
    store_op(ops, r0, x);
    // dg of chunk c from the parts its warps left (one warp)
    auto finish = [&](int c) {
      const float* at = parts + (c & 1) * kParts;
      const int t = 2 * lane;
      float xs[2], bs[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float rows = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) rows += at[w * kC + t + e];
        xs[e] = rows - at[4 * kC + t + e] + alpha[c * kC + t + e];
        bs[e] = at[5 * kC + t + e];
      }
      float down = xs[0] + xs[1], up = bs[0] + bs[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float d = __shfl_down_sync(0xffffffffu, down, o);
        const float u = __shfl_up_sync(0xffffffffu, up, o);
        if (lane + o < 32) down += d;
        if (lane >= o) up += u;
      }
      float after = __shfl_down_sync(0xffffffffu, down, 1), before = __shfl_up_sync(0xffffffffu, up, 1);
      if (lane == 31) after = 0.f;
      if (lane == 0) before = 0.f;
      const float se = at[6 * kC] + at[6 * kC + 1] + at[6 * kC + 2] + at[6 * kC + 3];
      const int tok = tb + c * kC + t;
      if (tok < te) a.dg[seq + tok] = __float2bfloat16_rn(se + down + before);
      if (tok + 1 < te) a.dg[seq + tok + 1] = __float2bfloat16_rn(se + (xs[1] + after) + (before + bs[0]));
    };

    for (int c = chunks - 1; c >= 0; --c) {
      cp_async_wait<0>();
      __syncthreads();
      const float2 g = g_next;
      if (c > 0) {
        load_chunk(c - 1);
        g_next = load_gates(a.g + seq, tb + (c - 1) * kC, te);
      }
      cp_async_commit();
      if (c + 1 < chunks && warp == (c & 3)) finish(c + 1);
      chunk_gates<true>(g, Gs, Vs);  // Vs: exp(G_i)
      const float total = chunk_gates<false>(g, Gs, Ws);
      const float dec = gated_decay(total * kLn2);
      const int step = chunks - 1 - c;
      const uint32_t q_at = base + (c & 1) * kStage, k_at = q_at + kTile, v_at = k_at + kTile,
                     do_at = v_at + kTile, op = base + 2 * kStage + (step & 1) * kOp;
      float* part = parts + (c & 1) * kParts;
      {
        float se = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint4 s = scratch[(c * 4 + e) * kThreads];
          se = fmaf(lo_of(s.x), x[2 * e][0], fmaf(hi_of(s.x), x[2 * e][1], se));
          se = fmaf(lo_of(s.y), x[2 * e][2], fmaf(hi_of(s.y), x[2 * e][3], se));
          se = fmaf(lo_of(s.z), x[2 * e + 1][0], fmaf(hi_of(s.z), x[2 * e + 1][1], se));
          se = fmaf(lo_of(s.w), x[2 * e + 1][2], fmaf(hi_of(s.w), x[2 * e + 1][3], se));
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) se += __shfl_xor_sync(0xffffffffu, se, o);
        if (lane == 0) part[6 * kC + warp] = se * dec;
      }
      uint32_t ka[4][4], va[4][4];
      float dk[8][4], dv[8][4];
      zero(dk);
      zero(dv);
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        load_a<64>(ka[ks], k_at, r0, 2 * ks);
        load_a<64>(va[ks], v_at, r0, 2 * ks);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) {
          uint32_t b[4];
          load_b<64>(b, op, 16 * jp, 2 * ks);  // E^T
          mma16816(dk[2 * jp], va[ks], b[0], b[1]);
          mma16816(dk[2 * jp + 1], va[ks], b[2], b[3]);
          load_b_t<64>(b, op, 16 * ks, 2 * jp);
          mma16816(dv[2 * jp], ka[ks], b[0], b[1]);
          mma16816(dv[2 * jp + 1], ka[ks], b[2], b[3]);
        }
      {
        const float w0 = Ws[r0 + row], w1 = Ws[r0 + row + 8];
        scale_rows(dk, w0, w1);
        scale_rows(dv, w0, w1);
        const float2 be = row_dots(smem + (v_at - base), r0, dv);
        if ((lane & 3) == 0) {
          part[5 * kC + r0 + row] = be.x;
          part[5 * kC + r0 + row + 8] = be.y;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] *= dec;
      const float gj[2] = {Gs[r0 + row], Gs[r0 + row + 8]};
      float cols[2] = {0.f, 0.f};
#pragma unroll
      for (int ib = 0; ib < 4; ++ib) {
        uint32_t db[4][4];
#pragma unroll
        for (int jp = 0; jp < 4; ++jp) load_b_t<64>(db[jp], do_at, 16 * ib, 2 * jp);
        if (ib >= rb) {
          float p[2][4] = {}, dp[2][4] = {};
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            uint32_t b[4];
            load_b<64>(b, q_at, 16 * ib, 2 * ks);
            mma16816(p[0], ka[ks], b[0], b[1]);
            mma16816(p[1], ka[ks], b[2], b[3]);
            load_b<64>(b, do_at, 16 * ib, 2 * ks);
            mma16816(dp[0], va[ks], b[0], b[1]);
            mma16816(dp[1], va[ks], b[2], b[3]);
          }
          uint32_t pa[4], dpa[4];
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const float2 gi = *reinterpret_cast<const float2*>(&Gs[16 * ib + 8 * t + col]);
            float w[4], dw[4], rows[2] = {0.f, 0.f};
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int i = 8 * t + col + e, j = row + 8 * h, at = 2 * h + e;
                const float L = ib > rb || i >= j ? ex2((e ? gi.y : gi.x) - gj[h]) : 0.f;
                w[at] = p[t][at] * L;
                dw[at] = dp[t][at] * L;
                const float xx = ib > rb || i > j ? p[t][at] * dw[at] : 0.f;
                rows[e] += xx;
                cols[h] += xx;
              }
            pa[2 * t] = pack2(w[0], w[1]);
            pa[2 * t + 1] = pack2(w[2], w[3]);
            dpa[2 * t] = pack2(dw[0], dw[1]);
            dpa[2 * t + 1] = pack2(dw[2], dw[3]);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
              rows[0] += __shfl_xor_sync(0xffffffffu, rows[0], o);
              rows[1] += __shfl_xor_sync(0xffffffffu, rows[1], o);
            }
            if (row == 0)
              *reinterpret_cast<float2*>(part + warp * kC + 16 * ib + 8 * t + col) =
                  make_float2(rows[0], rows[1]);
          }
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {
            mma16816(dv[2 * jp], pa, db[jp][0], db[jp][1]);
            mma16816(dv[2 * jp + 1], pa, db[jp][2], db[jp][3]);
            uint32_t b[4];
            load_b_t<64>(b, q_at, 16 * ib, 2 * jp);
            mma16816(dk[2 * jp], dpa, b[0], b[1]);
            mma16816(dk[2 * jp + 1], dpa, b[2], b[3]);
          }
        } else if (row == 0) {
          *reinterpret_cast<float2*>(part + warp * kC + 16 * ib + col) = make_float2(0.f, 0.f);
          *reinterpret_cast<float2*>(part + warp * kC + 16 * ib + 8 + col) = make_float2(0.f, 0.f);
        }
        if (c > 0) {
          uint32_t qa[4], hi[4], lo[4];
          load_a_t<64>(qa, q_at, 16 * ib, 2 * rb);
          const float2 w0 = *reinterpret_cast<const float2*>(&Vs[16 * ib + col]);
          const float2 w8 = *reinterpret_cast<const float2*>(&Vs[16 * ib + 8 + col]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 w = e < 2 ? w0 : w8;
            scale_split(qa[e], w.x, w.y, hi[e], lo[e]);
          }
#pragma unroll
          for (int jp = 0; jp < 4; ++jp) {
            mma16816(x[2 * jp], hi, db[jp][0], db[jp][1]);
            mma16816(x[2 * jp + 1], hi, db[jp][2], db[jp][3]);
            mma16816(x[2 * jp], lo, db[jp][0], db[jp][1]);
            mma16816(x[2 * jp + 1], lo, db[jp][2], db[jp][3]);
          }
        }
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        cols[0] += __shfl_xor_sync(0xffffffffu, cols[0], o);
        cols[1] += __shfl_xor_sync(0xffffffffu, cols[1], o);
      }
      if ((lane & 3) == 0) {
        part[4 * kC + r0 + row] = cols[0];
        part[4 * kC + r0 + row + 8] = cols[1];
      }
      if (c > 0) store_op(ops + ((step + 1) & 1) * kOp, r0, x);
      const int t0 = tb + c * kC + r0;
      store_rows(smem + (k_at - base), r0, dk, a.dk + (seq + t0) * a.D, te - t0, a.D);
      store_rows(smem + (v_at - base), r0, dv, a.dv + (seq + t0) * a.M, te - t0, a.M);
    }
    __syncthreads();
    if (warp == 0) finish(0);
  }
}

int backward_grid(const GatedPlan& p) {
  const long long items = (long long)p.BH * p.n_seg;
  return (int)(items < 152 * kResident ? items : 152 * kResident);
}

}  // namespace

bool gated_mma_backward_supported(int D, int M) { return D <= 64 && M <= 64; }

// Segments of up to kMaxChunks chunks, of a length that fills whole waves of the
// resident CTAs.
GatedPlan gated_mma_backward_plan(int BH, int N) {
  const long long chunks = (N + kC - 1) / kC, total = chunks * BH, slots = 152 * kResident;
  long long waves = (total + slots * kMaxChunks - 1) / (slots * kMaxChunks);
  if (waves < 1) waves = 1;
  long long len = (total + slots * waves - 1) / (slots * waves);
  if (len > kMaxChunks) len = kMaxChunks;
  if (len > chunks) len = chunks;
  if (len < 1) len = 1;
  const long long n_seg = (chunks + len - 1) / len;
  return GatedPlan{BH, N, (int)(len * kC), n_seg < 1 ? 1 : (int)n_seg};
}

size_t gated_mma_backward_scratch(const GatedPlan& p) {
  return sizeof(uint4) * (size_t)backward_grid(p) * kMaxChunks * 4 * kThreads;
}

cudaError_t gated_mma_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                               cudaStream_t st) {
  cudaError_t e;
  BwdArgs a{};
  if (p.n_seg > 1 || f.dS0) {
    if ((e = gated_mma_states(p, f.k, f.v, f.q, f.dout, f.g, f.D, f.M, nullptr, f.H, w, st)) !=
        cudaSuccess)
      return e;
    const GatedGradients back{f.dS, f.dS0};
    if ((e = gated_scan(p, w, f.S0, nullptr, GatedEntries{nullptr, 0, f.H}, f.D * f.M, st, &back)) !=
        cudaSuccess)
      return e;
    a.S = w.S;
    a.E = w.E;
  }
  a.q = static_cast<const bf16*>(f.q);
  a.k = static_cast<const bf16*>(f.k);
  a.v = static_cast<const bf16*>(f.v);
  a.g = static_cast<const bf16*>(f.g);
  a.dout = static_cast<const bf16*>(f.dout);
  a.dq = static_cast<bf16*>(f.dq);
  a.dk = static_cast<bf16*>(f.dk);
  a.dv = static_cast<bf16*>(f.dv);
  a.dg = static_cast<bf16*>(f.dg);
  a.D = f.D;
  a.M = f.M;
  a.N = f.N;
  a.BH = p.BH;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.S0 = f.S0;
  a.dS = f.dS;
  a.scratch = static_cast<uint4*>(w.scratch);
  if ((e = tcx::configure(gated_backward_kernel, kSmem)) != cudaSuccess) return e;
  e = tcx::launch_pdl(gated_backward_kernel, dim3((unsigned)backward_grid(p)), dim3(kThreads), kSmem,
                      st, a);
  count_launches(1);
  return e;
}

}  // namespace la
