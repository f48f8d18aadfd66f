// Gated recurrence's backward in bf16 on tensor cores (D, M up to 64).
//
// Per chunk of 64 tokens, with S the state before it and E the loss's gradient with
// respect to the state after it (G, L as in the forward):
//   dQ = ((dO V^T) * L) K + diag(exp(G_i)) dO S^T
//   dK = ((dO V^T) * L)^T Q + diag(exp(G - G_j)) V E^T
//   dV = ((Q K^T) * L)^T dO + diag(exp(G - G_j)) K E
//   S' = exp(G) S + (diag(exp(G - G_j)) K)^T V,  E' = exp(G) E + (diag(exp(G_i)) Q)^T dO
// A gate g_t scales what passes from tokens before t to tokens from t on:
//   dg_t = sum_{i >= t > j} X_ij + sum_{i >= t} a_i + sum_{j < t} b_j + exp(G) <S, E>
//   X = (Q K^T) * (dO V^T) * L,  a_i = exp(G_i) q_i S dO_i,  b_j = exp(G - G_j) k_j E v_j
// X's sum is one over s >= t of its row sums less its column sums, and those are what
// the products within the chunk add to q_s . dQ_s and to k_s . dK_s. Both products take
// the same operand (dO V^T) * L, to 16 bits, so what has to cancel in the difference does.
//
// S is known going forward and E going back, so a CTA walks its segment of a few chunks
// forward (dQ; each chunk's S to scratch of the CTA's own, in float32 for <S, E>) and then
// back (dK, dV, dg). Both walks keep their state in float32 accumulators; operands that are
// not inputs (L's products, the copies of S and E that are multiplied, weighted rows) are
// two bf16 terms, and only the gradients are rounded to one.
//
// Four warps share a chunk, warp r with its rows 16 r.. of the outputs and of the states.
// Going back, dV is finished before dK is begun, so that one set of output accumulators is
// live at a time. What bounds it is what bounds the forward: 490 products (3900 cycles) and
// about 1700 other instructions a chunk and warp, which do not overlap, in 8700 cycles.
// Measured and not kept: a third CTA per SM in 168 registers (214 to 225 us for 196, more
// barriers), eight warps in roles with half the registers each (248 us), two tiles of rows
// a warp (298 us, spills).
//
// B4 H8 N16384 D = M = 64: states and gradients of segments 61 us, scans 11 us, this
// kernel 246 us (888 MB moved: the second read of the tiles mostly misses L2, which
// segments of 7 chunks avoid at the same time); the call 318 us against 70 us for reading
// four tensors and writing four. With one bf16 term of each operand it took 269 us, and
// gradients were off by 2.35e-3 (2-norm) instead of 1.66e-3, their own rounding.
#include "la_gated.cuh"
#include "la_gated_mma.cuh"
#include "la_mma.cuh"
#include "la_tc_common.cuh"

namespace la {

using namespace mma;

namespace {

constexpr int kThreads = 128, kResident = 2, kMaxChunks = 16;
constexpr int kTile = kC * 64 * 2;
constexpr int kStage = 4 * kTile;  // Q, K, V, dO
constexpr int kOp = kTile;         // a bf16 term of S or E, [d][m]
// floats per parity of the chunk: the parts of dg (sums of X's columns, b, <S, E> by warp)
constexpr int kParts = 2 * kC + 4;
// two stages of tiles, the operand's two in two terms each, outputs on their way out
constexpr int kSmem = 2 * kStage + 4 * kOp + kTile + 2 * ((int)sizeof(GateTables) + 4 * kParts);
static_assert(kResident * (kSmem + 1024) <= 228 * 1024, "CTAs per SM");
// scratch of a CTA for each chunk of a segment: S as the warps hold it, and q . dQ of each
// token
constexpr size_t kKept = 8 * kThreads * sizeof(float4), kScratch = kKept + kC * sizeof(float);

struct BwdArgs {
  const bf16 *q, *k, *v, *g, *dout;
  bf16 *dq, *dk, *dv, *dg;
  int D, M, N, BH, len, n_seg;
  const float *S, *E;    // per-segment entries (nullptr: one segment)
  const float *S0, *dS;  // one segment: the caller's (nullptr: zero)
  char* scratch;
};

// Rows r0.. of a state, 8 NT columns from c0 on
template <int NT>
__device__ __forceinline__ void load_state(float (&x)[NT][4], const float* from, int r0, int c0,
                                           int D, int M) {
  const int lane = threadIdx.x & 31, row = lane >> 2, col = (lane & 3) * 2;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int d = r0 + row + 8 * h, m = c0 + 8 * j + col;
      float2 v = make_float2(0.f, 0.f);
      if (from && d < D && m < M) v = *reinterpret_cast<const float2*>(from + (size_t)d * M + m);
      x[j][2 * h] = v.x;
      x[j][2 * h + 1] = v.y;
    }
}

__global__ void __launch_bounds__(kThreads, kResident) gated_backward_kernel(const BwdArgs a) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = lane >> 2;
  // the causal products give a chunk's rows unequal work: turn their order from CTA to
  // CTA, so that no scheduler gets all of the most
  const int rb = (warp + blockIdx.x) & 3, r0 = rb * 16;
  const Lane<64> ln;
  uint8_t* op_mem = smem + 2 * kStage;
  const uint32_t op_base = base + 2 * kStage, out_at = op_base + 4 * kOp;
  GateTables* tables = reinterpret_cast<GateTables*>(op_mem + 4 * kOp + kTile);
  float* parts = reinterpret_cast<float*>(tables + 2);
  char* own = a.scratch + (size_t)blockIdx.x * (a.len / kC) * kScratch;
  float4* states = reinterpret_cast<float4*>(own) + tid;  // [chunk][8][thread]
  float* alpha = reinterpret_cast<float*>(own + (a.len / kC) * kKept);  // [chunk][64]: q . dQ

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
    // A chunk's tables are made by one warp while the chunk before it is worked on. Going
    // forward K is weighted, going back Q.
    auto raw_gates = [&](int c) { return load_gates(a.g + seq, tb + c * kC, te); };

    __syncthreads();  // the item before is done with
    load_chunk(0);
    cp_async_commit();
    if (warp == 0) chunk_gates<false, false>(raw_gates(0), tables[0]);

    // ---- forward: dQ
    float x[8][4];  // S, then E
    auto keep_op = [&](int buf) {
      store_op(ln, op_base + buf * kOp, r0, 0, x);
      store_op<true>(ln, op_base + (2 + buf) * kOp, r0, 0, x);
    };
    load_state(x, a.S ? a.S + ((size_t)bh * (a.n_seg + 1) + seg) * DM : a.S0 ? a.S0 + bh * DM : nullptr,
               r0, 0, a.D, a.M);
    keep_op(0);
    for (int c = 0; c < chunks; ++c) {
      cp_async_wait<0>();
      __syncthreads();
      if (c + 1 < chunks) load_chunk(c + 1);
      cp_async_commit();
      const GateTables& t = tables[c & 1];
      const uint32_t q_at = base + (c & 1) * kStage, k_at = q_at + kTile, v_at = k_at + kTile,
                     do_at = v_at + kTile;
      const bool maker = c + 1 < chunks && rb == 0;  // (the warp with one block of the product)
      ushort2 raw = make_ushort2(0, 0);
      if (maker) raw = raw_gates(c + 1);
#pragma unroll
      for (int j = 0; j < 8; ++j) states[(c * 8 + j) * kThreads] = keep_tile(x[j]);
      uint32_t f[4][4], p[2][4];
      float d[8][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) ln.load_a(f[ks], do_at, r0, ks);
      product<false>(ln, d, f, op_base + (c & 1) * kOp);
      product<false, true>(ln, d, f, op_base + (2 + (c & 1)) * kOp);
      float wi[2] = {t.in[r0 + row], t.in[r0 + row + 8]};
      scale_rows(d, wi[0] * t.before[rb], wi[1] * t.before[rb]);
      diagonal_block<true>(ln, p, f, v_at, rb, t.hi, t.lo);
      add_block(ln, d, p, k_at, rb);
#pragma unroll 1
      for (int jb = rb - 1; jb >= 0; --jb) {
        weighted_block(ln, p, f, v_at, jb, t.out, wi);
        add_block(ln, d, p, k_at, jb);
        wi[0] *= t.total[jb];
        wi[1] *= t.total[jb];
      }
      const float2 dots = row_dots(ln, q_at, r0, d);
      if ((lane & 3) == 0) {
        alpha[c * kC + r0 + row] = dots.x;
        alpha[c * kC + r0 + row + 8] = dots.y;
      }
      const int t0 = tb + c * kC + r0;
      store_rows(ln, out_at, r0, d, a.dq + (seq + t0) * a.D, te - t0, a.D, a.D);
      if (c + 1 < chunks) {
        scale_rows(x, t.decay, t.decay);
        add_outer<false>(ln, ln, x, k_at, t.X, rb, v_at, 0);
        keep_op((c + 1) & 1);
      }
      if (maker) chunk_gates<false, false>(raw, tables[(c + 1) & 1]);
    }

    // ---- back: dV, dK, dg. The last two chunks' tiles are still there.
    load_state(x, a.E ? a.E + ((size_t)bh * (a.n_seg + 1) + seg + 1) * DM : a.dS ? a.dS + bh * DM : nullptr,
               r0, 0, a.D, a.M);
    __syncthreads();
    keep_op(0);
    if (warp == 0) chunk_gates<true, false>(raw_gates(chunks - 1), tables[(chunks - 1) & 1]);
    // dg of chunk c from the parts its warps left (one warp)
    auto finish = [&](int c) {
      const float* at = parts + (c & 1) * kParts;
      const float2 rows = *reinterpret_cast<const float2*>(alpha + c * kC + 2 * lane);
      const float2 cols = *reinterpret_cast<const float2*>(at + 2 * lane);
      const float2 be = *reinterpret_cast<const float2*>(at + kC + 2 * lane);
      const float x0 = rows.x - cols.x, x1 = rows.y - cols.y;
      float down = x0 + x1, up = be.x + be.y;
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
      const float se = at[2 * kC] + at[2 * kC + 1] + at[2 * kC + 2] + at[2 * kC + 3];
      const int tok = tb + c * kC + 2 * lane;
      if (tok < te) a.dg[seq + tok] = __float2bfloat16_rn(se + down + before);
      if (tok + 1 < te) a.dg[seq + tok + 1] = __float2bfloat16_rn(se + (x1 + after) + (before + be.x));
    };

    for (int c = chunks - 1; c >= 0; --c) {
      cp_async_wait<0>();
      __syncthreads();
      if (c > 0 && c + 1 < chunks) load_chunk(c - 1);
      cp_async_commit();
      const int step = chunks - 1 - c;
      const GateTables& t = tables[c & 1];
      float* part = parts + (c & 1) * kParts;
      const uint32_t q_at = base + (c & 1) * kStage, k_at = q_at + kTile, v_at = k_at + kTile,
                     do_at = v_at + kTile, op = op_base + (step & 1) * kOp;
      const bool maker = c > 0 && warp == (c & 3);
      ushort2 raw = make_ushort2(0, 0);
      if (maker) raw = raw_gates(c - 1);
      float4 sc[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sc[j] = states[(c * 8 + j) * kThreads];
      if (c + 1 < chunks && warp == ((c + 1) & 3)) finish(c + 1);
      const float dec = t.decay;
      const int t0 = tb + c * kC + r0;
      uint32_t f[4][4], p[2][4];
      float d[8][4];
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) ln.load_a(f[ks], k_at, r0, ks);
      product<true>(ln, d, f, op);
      product<true, true>(ln, d, f, op + 2 * kOp);
      float wj[2] = {t.out[r0 + row], t.out[r0 + row + 8]};
      scale_rows(d, wj[0] * t.behind[rb], wj[1] * t.behind[rb]);
      diagonal_block<false>(ln, p, f, q_at, rb, t.hi, t.lo);
      add_block(ln, d, p, do_at, rb);
#pragma unroll 1
      for (int ib = rb + 1; ib < 4; ++ib) {
        weighted_block(ln, p, f, q_at, ib, t.in, wj);
        add_block(ln, d, p, do_at, ib);
        wj[0] *= t.total[ib];
        wj[1] *= t.total[ib];
      }
      store_rows(ln, out_at, r0, d, a.dv + (seq + t0) * a.M, te - t0, a.M, a.M);
      {
        float2 se = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < 8; ++j) se = dot_kept(sc[j], x[j], se);
        float s = se.x + se.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) part[2 * kC + warp] = s * dec;
      }
      // dK by the rows from the other end: the two causal halves add up to the same for
      // every warp
      const int kb = 3 - rb, k0 = kb * 16, tk = tb + c * kC + k0;
      float wk[2] = {t.out[k0 + row], t.out[k0 + row + 8]};
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) ln.load_a(f[ks], v_at, k0, ks);
      product<false>(ln, d, f, op);
      product<false, true>(ln, d, f, op + 2 * kOp);
      scale_rows(d, wk[0] * t.behind[kb], wk[1] * t.behind[kb]);
      const float2 be = row_dots(ln, k_at, k0, d);
      diagonal_block<false>(ln, p, f, do_at, kb, t.hi, t.lo);
      add_block(ln, d, p, q_at, kb);
#pragma unroll 1
      for (int ib = kb + 1; ib < 4; ++ib) {
        weighted_block(ln, p, f, do_at, ib, t.in, wk);
        add_block(ln, d, p, q_at, ib);
        wk[0] *= t.total[ib];
        wk[1] *= t.total[ib];
      }
      const float2 all = row_dots(ln, k_at, k0, d);
      if ((lane & 3) == 0) {
        part[k0 + row] = all.x - be.x;
        part[k0 + row + 8] = all.y - be.y;
        part[kC + k0 + row] = be.x;
        part[kC + k0 + row + 8] = be.y;
      }
      // (through V's rows, which no other warp reads)
      store_rows(ln, v_at, k0, d, a.dk + (seq + tk) * a.D, te - tk, a.D, a.D);
      if (c > 0) {
        scale_rows(x, dec, dec);
        add_outer<false>(ln, ln, x, q_at, t.X, rb, do_at, 0);
        keep_op((step + 1) & 1);
      }
      if (maker) chunk_gates<true, false>(raw, tables[(c - 1) & 1]);
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

GatedPlan gated_mma_backward_plan(int BH, int N) {
  return gated_mma_plan(BH, N, 1, GatedCosts{152 * kResident, kMaxChunks, 4.f, 8.7f, 7.f, 3.4f});
}

size_t gated_mma_backward_scratch(const GatedPlan& p) {
  return (size_t)backward_grid(p) * (p.len / kC) * kScratch;
}

cudaError_t gated_mma_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                               cudaStream_t st) {
  cudaError_t e;
  BwdArgs a{};
  if (p.n_seg > 1 || f.dS0) {
    if ((e = gated_mma_states(p, f.k, f.v, f.q, f.dout, f.g, f.D, f.M, nullptr, f.H, f.dS0 != nullptr,
                              w, st)) !=
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
  a.scratch = static_cast<char*>(w.scratch);
  const dim3 grid((unsigned)backward_grid(p));
  return gated_launch<gated_backward_kernel>(kSmem, grid, kThreads, st, a);
}

}  // namespace la
