// Gated recurrence in bf16 on tensor cores: forward, and the states of segments.
//
// A chunk of 64 tokens is a masked product and a rank-64 update. With G_i the sum of
// the chunk's g up to and including token i, G the whole chunk's, L_ij = exp(G_i - G_j)
// for j <= i and 0 above:
//   O = diag(exp(G_i)) (Q S) + ((Q K^T) * L) V
//   S = exp(G) S + (diag(exp(G - G_j)) K)^T V
// All exponents are <= 0 for g <= 0, so nothing overflows, and sums that reach a
// weight are taken from the end that weight decays from (chunk_gates), so that a strong
// gate elsewhere in the chunk costs no digits.
//
// Four warps share a chunk: warp r has its rows 16 r.. of Q and O and rows 16 r.. of
// S (of each 64), S in float32 accumulators that stay in registers over the whole
// segment. What is multiplied by an input's rows and is not an input itself (Q K^T * L,
// the copy of S in shared memory that Q multiplies, K's weighted rows in the update of S)
// is taken as two bf16 terms, 16 bits: an output shows its own rounding only (1.66e-3 in
// the 2-norm of random data). With one term of the first two, outputs were off by 2.35e-3,
// in 106 us for the longest forward instead of 124; with one of the third too by 2.8e-3.
//
// Why warp-level products and not tcgen05: at 64 columns a chunk's products are small
// next to its element-wise work (masks, weights, splits), which here happens in the
// registers that hold the fragments, with no round trip through tensor memory and no
// barrier between a product and its use. The price is that these instructions hold up
// their scheduler's others: the products' 1504 cycles a chunk and warp (at the 600
// TFLOP/s they reach) and some 600 other instructions add up rather than overlap, to
// 3000 cycles with three CTAs of four warps per SM.
//
// B4 H8 N16384 D = M = 64: states 33 us (138 MB moved: half of what HBM gives, tensor
// pipe 49%), scan 6 us, outputs 85 us (252 MB); the whole call 124 us against 40 us for
// reading q, k, v and writing out once.
#include "la_gated.cuh"
#include "la_gated_mma.cuh"
#include "la_mma.cuh"
#include "la_tc_common.cuh"

namespace la {

using namespace mma;

namespace {

constexpr int kThreads = 128;

// One walk over a segment's chunks, with a state X [ZD][UD]:
//   forward   out_i = z_i (exp(G_i) X) + sum over j <= i of L_ij (z_i . w_j) u_j
//             X = exp(G) X + sum over j of exp(G - G_j) w_j u_j^T
//   reverse   out_j = z_j (exp(G - G_j) X) + sum over i >= j of L_ij (z_j . w_i) u_i
//             X = exp(G) X + sum over i of exp(G_i) w_i u_i^T,  last chunk first
//   out  forward, z = q,    w = k,    u = v,    X = S
//   dQ   forward, z = dout, w = v,    u = k,    X = S^T
//   dK   reverse, z = v,    w = dout, u = q,    X = E^T
//   dV   reverse, z = k,    w = q,    u = dout, X = E
// (the gradients this way only for D or M over 64; up to 64, la_gated_mma_bwd.cu has
// them in one kernel). A CTA has 64 of u's columns.
struct WalkArgs {
  const bf16 *z, *w, *u, *g;
  bf16* out;
  int ZD, UD, N, BH, len, n_seg;
  int rs, cs;            // X's element (r, c) of an entry is at r * rs + c * cs
  const int* lens;
  int H;
  const float* seg_in;   // segments' entries of X (nullptr: one segment, `init`)
  float *seg_out, *decay;
  const float* init;
  float* fin;
  GatedEntries entries;
  WorkspaceHeader* hdr;
  // for the gates' gradient: p . out by token and column block (forward; reverse: of what
  // the chunk itself adds, and in `inter` of X's part); X of every chunk as the threads
  // hold it (forward: written; reverse: read, and `ends` the warps' sums of X times it,
  // decayed over the chunk)
  const bf16* p;
  float *dots, *inter, *ends;
  float4* kept;
};

template <int DZ, bool OUT>
struct WalkSmem {
  // z: each warp its own rows, which it asks for as soon as it is done with the chunk before
  static constexpr int kZ = OUT ? kC * DZ * 2 : 0, kW = kC * DZ * 2, kU = kC * 64 * 2;
  static constexpr int kStage = kW + kU;
  // the state pass has little to do on a chunk, so it asks for two ahead; the outputs'
  // walk is longer on a chunk than a load takes
  static constexpr int kStages = OUT ? 2 : 3;
  // X's two bf16 terms; heads over 64 have no room for the next chunk's beside them
  static constexpr int kX = OUT ? DZ * 64 * 2 : 0, kOps = DZ == 64 ? 2 : 1;
  static constexpr int kTables = kZ + kStages * kStage + 2 * kOps * kX;
  static constexpr int kBytes = kTables + 2 * (int)sizeof(GateTables);
};

// OUT: outputs (and, with one segment, the final state), else the state pass: the
// segment's own X from zero.
// EXACT: a chunk's update of X is summed apart, with its operand to 24 bits, and added in
// float32 arithmetic that rounds (the tensor cores' own sums truncate, which over
// thousands of chunks would leave a bias in a state that hardly decays). Taken where X
// leaves the kernel as a float32 result and in long segments; where it only goes on as an
// operand of two bf16 terms, 16 bits and sums in place do, and leave registers for more
// CTAs per SM.
// DOTS: the parts of the gates' gradient.
template <int DZ, bool OUT, bool REV, bool EXACT, bool DOTS = false>
__device__ __forceinline__ void walk_chunks(const WalkArgs& a) {
  using Sm = WalkSmem<DZ, OUT>;
  constexpr int KS = DZ / 16, DT = DZ / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem), stages = base + Sm::kZ,
                 x_op = stages + Sm::kStages * Sm::kStage;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = lane >> 2, col = (lane & 3) * 2;  // of an accumulator
  GateTables* tables = reinterpret_cast<GateTables*>(smem + Sm::kTables);
  const Lane<DZ> ln;
  const Lane<64> ln64;

  tc::pdl_wait();
  const int bh = blockIdx.x / a.n_seg, seg = blockIdx.x % a.n_seg;
  const int c0 = blockIdx.y * 64;
  // the causal product gives a chunk's rows unequal work: turn their order from CTA to
  // CTA, so that no scheduler gets all of the most
  const int rb = (warp + blockIdx.x) & 3;
  const int n = gated_length(a.lens, a.H, bh, a.N);
  const int tb = min(seg * a.len, n), te = min(tb + a.len, n);
  const int chunks = (te - tb + kC - 1) / kC;
  const size_t seq = (size_t)bh * a.N;
  const long long entry = a.entries.at(bh);
  if (entry < 0 && seg == 0 && c0 == 0 && tid == 0 && a.hdr) a.hdr->status = LA_ERR_INVALID_ARG;
  const size_t entry_size = (size_t)a.ZD * a.UD;

  float x[DT][8][4];
  auto x_at = [&](int i) { return x_op + (Sm::kOps == 2 ? 2 * (i & 1) * Sm::kX : 0); };
  auto keep_op = [&](int i) {  // X before the i-th chunk
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      store_op(ln64, x_at(i), dt * 64 + rb * 16, 0, x[dt]);
      store_op<true>(ln64, x_at(i) + Sm::kX, dt * 64 + rb * 16, 0, x[dt]);
    }
  };
  auto load_chunk = [&](int c) {
    const int t0 = tb + c * kC, rows = min(kC, te - t0);
    const uint32_t at = stages + (c % Sm::kStages) * Sm::kStage;
    load_tile<DZ, kThreads>(at, a.w + (seq + t0) * a.ZD, rows, a.ZD, 0);
    load_tile<64, kThreads>(at + Sm::kW, a.u + (seq + t0) * a.UD, rows, a.UD, c0);
  };
  auto load_z = [&](int c) {
    const int t0 = tb + c * kC + rb * 16;
    load_rows<DZ>(base, rb * 16, a.z + (seq + min(t0, te - 1)) * a.ZD, te - t0, a.ZD);
  };
  auto chunk_of = [&](int i) { return REV ? chunks - 1 - i : i; };
  auto raw_gates = [&](int c) { return load_gates(a.g + seq, tb + c * kC, te); };

  // A chunk's tables are made by the warp whose rows have the fewest blocks in the causal product
  const bool makes = rb == (REV ? 3 : 0);
  float all = 0.f;  // (its own:) sum of the segment's gates, base 2
  constexpr int kAhead = Sm::kStages - 1;
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    if (i < chunks) load_chunk(chunk_of(i));
    if (OUT && i < chunks) load_z(chunk_of(i));
    cp_async_commit();
  }
  if (chunks > 0 && makes) all = chunk_gates<REV, EXACT>(raw_gates(chunk_of(0)), tables[0]);
  {
    const float* in = nullptr;
    if (OUT && a.seg_in)
      in = a.seg_in + ((size_t)bh * (a.n_seg + 1) + seg + (REV ? 1 : 0)) * entry_size;
    else if (OUT && a.init && entry >= 0)
      in = a.init + (size_t)entry * entry_size;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = dt * 64 + rb * 16 + row + 8 * h, c = c0 + 8 * j + col;
          float2 v = make_float2(0.f, 0.f);
          if (in && r < a.ZD && c < a.UD) {
            const float* at = in + (size_t)r * a.rs + (size_t)c * a.cs;
            if (a.cs == 1)
              v = *reinterpret_cast<const float2*>(at);
            else
              v = make_float2(at[0], at[a.cs]);
          }
          x[dt][j][2 * h] = v.x;
          x[dt][j][2 * h + 1] = v.y;
        }
  }
  if (OUT) keep_op(0);

  for (int i = 0; i < chunks; ++i) {
    const int c = chunk_of(i);
    cp_async_wait<kAhead - 1>();
    __syncthreads();  // chunk i has landed; every warp is done with chunk i - 1
    const uint32_t z_at = base, w_at = stages + (c % Sm::kStages) * Sm::kStage, u_at = w_at + Sm::kW;
    const int r0 = rb * 16, t0 = tb + c * kC + r0;
    uint32_t f[OUT ? KS : 1][4];
    if (OUT) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) ln.load_a(f[ks], z_at, r0, ks);
    }
    if (DOTS) {  // z's rows are this warp's alone and read: p's take their place
      __syncwarp();
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e * 4 + (lane >> 3), ch = lane & 7;
        const bool live = t0 + r < te && c0 + ch * 8 < a.UD;
        cp_async16(z_at + (r0 + r) * DZ * 2 + ((ch ^ (r & 7)) << 4),
                   live ? a.p + (seq + t0 + r) * a.UD + c0 + ch * 8 : a.p, live);
      }
      cp_async_commit();
    }
    if (i + kAhead < chunks) load_chunk(chunk_of(i + kAhead));
    cp_async_commit();
    // the next chunk's, from gates asked for here
    const bool maker = makes && i + 1 < chunks;
    ushort2 raw = make_ushort2(0, 0);
    if (maker) raw = raw_gates(chunk_of(i + 1));
    const GateTables& t = tables[i & 1];
    const float dec = t.decay;

    if (OUT) {
      const size_t kept_at = ((((size_t)blockIdx.y * a.BH + bh) * ((a.N + kC - 1) / kC) + tb / kC + c) *
                              DT * 8) * kThreads + tid;
      if (DOTS && !REV) {
#pragma unroll
        for (int e = 0; e < DT * 8; ++e) a.kept[kept_at + (size_t)e * kThreads] = keep_tile(x[e >> 3][e & 7]);
      }
      if (DOTS && REV) {
        float2 se = make_float2(0.f, 0.f);
#pragma unroll
        for (int e = 0; e < DT * 8; ++e)
          se = dot_kept(a.kept[kept_at + (size_t)e * kThreads], x[e >> 3][e & 7], se);
        float sum = se.x + se.y;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0)
          a.ends[(((size_t)blockIdx.y * a.BH + bh) * ((a.N + kC - 1) / kC) + tb / kC + c) * 4 + warp] =
              sum * dec;
      }
      float o[8][4];
      // of this warp's rows: what its own block of tokens leaves of them, or lets through
      float wr[2] = {(REV ? t.out : t.in)[r0 + row], (REV ? t.out : t.in)[r0 + row + 8]};
      product<true>(ln64, o, f, x_at(i));
      product<true, true>(ln64, o, f, x_at(i) + Sm::kX);
      const float others = (REV ? t.behind : t.before)[rb];
      scale_rows(o, wr[0] * others, wr[1] * others);
      const size_t dots_at = ((size_t)blockIdx.y * a.BH + bh) * a.N + t0 + row;
      float2 inter = make_float2(0.f, 0.f);
      if (DOTS && REV) {
        cp_async_wait<1>();
        __syncwarp();
        inter = row_dots(ln, z_at, r0, o);
      }
      uint32_t p[2][4];
      diagonal_block<!REV>(ln, p, f, w_at, rb, t.hi, t.lo);
      add_block(ln64, o, p, u_at, rb);
#pragma unroll 1
      for (int b = REV ? rb + 1 : rb - 1; REV ? b < 4 : b >= 0; b += REV ? 1 : -1) {
        weighted_block(ln, p, f, w_at, b, REV ? t.in : t.out, wr);
        add_block(ln64, o, p, u_at, b);
        wr[0] *= t.total[b];
        wr[1] *= t.total[b];
      }
      if (DOTS) {
        if (!REV) {
          cp_async_wait<1>();
          __syncwarp();
        }
        float2 d = row_dots(ln, z_at, r0, o);
        if (REV) {
          d.x -= inter.x;
          d.y -= inter.y;
        }
        if ((lane & 3) == 0) {
          if (t0 + row < te) {
            a.dots[dots_at] = d.x;
            if (REV) a.inter[dots_at] = inter.x;
          }
          if (t0 + row + 8 < te) {
            a.dots[dots_at + 8] = d.y;
            if (REV) a.inter[dots_at + 8] = inter.y;
          }
        }
      }
      // through this warp's rows of z's tile, which no other warp reads
      store_rows(ln, z_at, r0, o, a.out + (seq + t0) * a.UD + c0, te - t0, a.UD - c0, a.UD);
      __syncwarp();
      if (i + 1 < chunks) load_z(chunk_of(i + 1));
      cp_async_commit();
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      if (EXACT) {
        float y[8][4];
        add_outer<true>(ln, ln64, y, w_at, t.X, 4 * dt + rb, u_at, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pair_of(x[dt][j], h) = fma2(make_float2(dec, dec), pair_of(x[dt][j], h), pair_of(y[j], h));
      } else {
        scale_rows(x[dt], dec, dec);
        add_outer<false>(ln, ln64, x[dt], w_at, t.X, 4 * dt + rb, u_at, 0);
      }
    }
    if (OUT && Sm::kOps == 1) __syncthreads();  // every warp has multiplied X
    if (OUT && i + 1 < chunks) keep_op(i + 1);
    if (maker) all += chunk_gates<REV, EXACT>(raw, tables[(i + 1) & 1]);
  }

  float* to = nullptr;
  if (!OUT)
    to = a.seg_out + ((size_t)bh * (a.n_seg + 1) + seg) * entry_size;
  else if (a.fin && entry >= 0)
    to = a.fin + (size_t)entry * entry_size;
  if (to)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = dt * 64 + rb * 16 + row + 8 * h, m = c0 + 8 * j + col;
          if (r < a.ZD && m < a.UD)  // (only S and E leave: rs = UD, cs = 1)
            *reinterpret_cast<float2*>(to + (size_t)r * a.UD + m) =
                make_float2(x[dt][j][2 * h], x[dt][j][2 * h + 1]);
        }
  if (!OUT && a.decay && c0 == 0 && makes && lane == 0)
    a.decay[(size_t)bh * a.n_seg + seg] = gated_decay(all * kLn2);
}

template <int DZ, bool EXACT>
__global__ void __launch_bounds__(kThreads, DZ == 64 ? 3 : 2)
gated_forward_kernel(const WalkArgs a) {
  walk_chunks<DZ, true, false, EXACT>(a);
}

// blockIdx.z: the segments' states, or their gradients
template <int DZ, bool EXACT>
__global__ void __launch_bounds__(kThreads, DZ == 64 ? 3 : 2)
gated_states_kernel(const WalkArgs a, const WalkArgs back) {
  if (blockIdx.z == 0)
    walk_chunks<DZ, false, false, EXACT>(a);
  else
    walk_chunks<DZ, false, true, EXACT>(back);
}

template <int DZ, bool REV, bool DOTS>
__global__ void __launch_bounds__(kThreads, DZ == 64 ? 3 : 2)
gated_gradient_kernel(const WalkArgs a) {
  walk_chunks<DZ, true, REV, false, DOTS>(a);
}

dim3 walk_grid(const WalkArgs& a, int z = 1) {
  return dim3((unsigned)(a.BH * a.n_seg), (unsigned)((a.UD + 63) / 64), (unsigned)z);
}

template <int DZ, bool EXACT>
cudaError_t launch_forward(const WalkArgs& a, cudaStream_t st) {
  return gated_launch<gated_forward_kernel<DZ, EXACT>>(WalkSmem<DZ, true>::kBytes, walk_grid(a), kThreads,
                                                       st, a);
}

template <bool EXACT>
cudaError_t launch_states(const WalkArgs& a, const WalkArgs& back, int jobs, cudaStream_t st) {
  return a.ZD <= 64
             ? gated_launch<gated_states_kernel<64, EXACT>>(WalkSmem<64, false>::kBytes, walk_grid(a, jobs), kThreads, st, a, back)
             : gated_launch<gated_states_kernel<128, EXACT>>(WalkSmem<128, false>::kBytes, walk_grid(a, jobs), kThreads, st, a, back);
}

template <bool REV, bool DOTS>
cudaError_t launch_gradient(const WalkArgs& a, cudaStream_t st) {
  return a.ZD <= 64 ? gated_launch<gated_gradient_kernel<64, REV, DOTS>>(WalkSmem<64, true>::kBytes,
                                                                         walk_grid(a), kThreads, st, a)
                    : gated_launch<gated_gradient_kernel<128, REV, DOTS>>(WalkSmem<128, true>::kBytes,
                                                                          walk_grid(a), kThreads, st, a);
}

// dg of a chunk from its dots (see la_gated_mma_bwd.cu): a warp each, two tokens a lane.
__global__ void __launch_bounds__(kThreads)
gated_chunk_dg_kernel(const float* __restrict__ dot_q, const float* __restrict__ dot_k,
                      const float* __restrict__ inter, const float* __restrict__ ends,
                      bf16* __restrict__ dg, int BH, int N, int blocks) {
  tc::pdl_wait();
  const int chunks = (N + kC - 1) / kC, lane = threadIdx.x & 31;
  const long long at = (long long)blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  if (at >= (long long)BH * chunks) return;
  const long long bh = at / chunks;
  const int t0 = (int)(at % chunks) * kC + 2 * lane;
  float x[2] = {0.f, 0.f}, b[2] = {0.f, 0.f}, se = 0.f;
  for (int y = 0; y < blocks; ++y) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const size_t i = ((size_t)y * BH + bh) * N + t0 + e;
      if (t0 + e < N) {
        x[e] += dot_q[i] - dot_k[i];
        b[e] += inter[i];
      }
    }
    const float4 w = *reinterpret_cast<const float4*>(ends + (((size_t)y * BH + bh) * chunks + at % chunks) * 4);
    se += w.x + w.y + w.z + w.w;
  }
  float down = x[0] + x[1], up = b[0] + b[1];
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
  if (t0 < N) dg[bh * N + t0] = __float2bfloat16_rn(se + down + before);
  if (t0 + 1 < N) dg[bh * N + t0 + 1] = __float2bfloat16_rn(se + (x[1] + after) + (before + b[0]));
}

}  // namespace

// One of several segments has at most 64 chunks, 4096 tokens: its decay is one float32, which has
// to be finite where gates are positive, and its state is summed in place by the tensor cores.
constexpr int kJoined = 64;

GatedPlan gated_mma_plan(int BH, int N, int blocks, const GatedCosts& k) {
  const long long chunks = N > 0 ? (N + kC - 1) / kC : 1, per = (long long)BH * blocks;
  GatedPlan best{BH, N, (int)chunks * kC, 1};
  float shortest = -1.f;
  // one segment; what fills 1, 2, .. waves; segments of 16, 8, .. chunks (16 is within
  // every bound); and the fewest that the bound allows
  for (int w = 0; w < 38; ++w) {
    long long n_seg = w == 0 ? 1 : w * (long long)k.slots / per;
    if (w > 32) n_seg = (chunks + (512 >> (w - 28)) - 1) / (512 >> (w - 28));
    if (k.most > 0 && n_seg * k.most < chunks) n_seg = (chunks + k.most - 1) / k.most;
    if (n_seg < 1) n_seg = 1;
    if (n_seg > 1 && n_seg * kJoined < chunks) n_seg = (chunks + kJoined - 1) / kJoined;
    if (n_seg > chunks) n_seg = chunks;
    const long long len = (chunks + n_seg - 1) / n_seg;
    n_seg = (chunks + len - 1) / len;
    const long long waves = (per * n_seg + k.slots - 1) / k.slots;
    const float each = (float)(per * chunks) / (3 * 152), pass_chunks = each > len ? each : (float)len;
    // (an SM's only CTA takes less than half as long on a chunk as one of three)
    const float full = per * n_seg < k.slots ? (float)(per * n_seg) / k.slots : 1.f;
    const float t = waves * (k.fixed + len * k.chunk * (0.45f + 0.55f * full)) +
                    (n_seg > 1 ? k.pass + pass_chunks * k.pass_chunk + 0.1f * n_seg : 0.f);
    if (shortest < 0.f || t < shortest) {
      shortest = t;
      best.len = (int)(len * kC);
      best.n_seg = (int)n_seg;
    }
  }
  return best;
}

GatedPlan gated_mma_forward_plan(int BH, int N, int D, int M) {
  const int blocks = (M + 63) / 64;
  return gated_mma_plan(BH, N, blocks, D <= 64 ? GatedCosts{3 * 152, 0, 3.f, 4.f, 9.f, 1.7f}
                                               : GatedCosts{2 * 152, 0, 3.f, 4.9f, 9.f, 2.5f});
}

cudaError_t gated_mma_states(const GatedPlan& p, const void* k, const void* v, const void* q,
                             const void* dout, const void* g, int D, int M, const int* lens, int H,
                             bool exact, const GatedWorkspace& w, cudaStream_t st) {
  WalkArgs s{};
  s.w = static_cast<const bf16*>(k);
  s.u = static_cast<const bf16*>(v);
  s.g = static_cast<const bf16*>(g);
  s.ZD = D;
  s.UD = M;
  s.N = p.N;
  s.BH = p.BH;
  s.len = p.len;
  s.n_seg = p.n_seg;
  s.lens = lens;
  s.H = H;
  s.entries.H = H;
  s.seg_out = w.S;
  s.decay = w.decay;
  WalkArgs back = s;
  back.w = static_cast<const bf16*>(q);
  back.u = static_cast<const bf16*>(dout);
  back.seg_out = w.E;
  back.decay = nullptr;
  const int jobs = dout ? 2 : 1;
  return exact ? launch_states<true>(s, back, jobs, st) : launch_states<false>(s, back, jobs, st);
}

cudaError_t gated_mma_forward(const GatedForward& f, const GatedPlan& p, const GatedWorkspace& w,
                              cudaStream_t st) {
  WalkArgs a{};
  a.z = static_cast<const bf16*>(f.q);
  a.w = static_cast<const bf16*>(f.k);
  a.u = static_cast<const bf16*>(f.v);
  a.g = static_cast<const bf16*>(f.g);
  a.out = static_cast<bf16*>(f.out);
  a.ZD = f.D;
  a.UD = f.M;
  a.rs = f.M;
  a.cs = 1;
  a.N = f.N;
  a.BH = p.BH;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.lens = f.lens;
  a.H = f.H;
  a.entries = GatedEntries{f.slots, f.pool, f.H};
  a.hdr = w.hdr;
  if (p.n_seg > 1) {
    cudaError_t e = gated_mma_states(p, f.k, f.v, nullptr, nullptr, f.g, f.D, f.M, f.lens, f.H,
                                     f.S != nullptr, w, st);
    if (e != cudaSuccess) return e;
    if ((e = gated_scan(p, w, f.S0, f.S, a.entries, f.D * f.M, st)) != cudaSuccess) return e;
    a.seg_in = w.S;
  } else {
    a.init = f.S0;
    a.fin = f.S;
  }
  // A sequence of one segment may be of any length: from 16384 tokens on its state is summed as a
  // result is. (456 sequences of positive terms, hardly forgotten: with sums in place outputs were
  // 3e-5 too small there, 3.6e-4 at 65536 and 5.4e-4 at 131072 tokens; 17% of the time.)
  const bool exact = a.fin || (p.n_seg == 1 && p.N > 16384);
  if (f.D <= 64) return exact ? launch_forward<64, true>(a, st) : launch_forward<64, false>(a, st);
  return exact ? launch_forward<128, true>(a, st) : launch_forward<128, false>(a, st);
}

// ---- the backward for D or M over 64: states, scans, then dQ, dK and dV a walk each

GatedPlan gated_mma_wide_plan(int BH, int N, int D, int M) {
  return gated_mma_plan(BH, N, ((D > M ? D : M) + 63) / 64, GatedCosts{2 * 152, kJoined, 9.f, 18.5f, 12.f, 5.f});
}

namespace {
int wide_blocks(int D) { return (D + 63) / 64; }
size_t wide_kept(const GatedPlan& p, int D, int M) {  // X of every chunk: rows of M, columns of D
  return sizeof(float4) * 8 * kThreads * (size_t)wide_blocks(D) * wide_blocks(M) * p.BH * ((p.N + kC - 1) / kC);
}
}  // namespace

size_t gated_mma_wide_scratch(const GatedPlan& p, int D, int M) {
  const size_t blocks = wide_blocks(D), bh = p.BH;
  return wide_kept(p, D, M) + 16 * blocks * bh * ((p.N + kC - 1) / kC) + 3 * align_up(4 * blocks * bh * p.N, 16);
}

cudaError_t gated_mma_wide_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                                    cudaStream_t st) {
  const size_t blocks = wide_blocks(f.D), chunks = (p.N + kC - 1) / kC, dots = align_up(4 * blocks * p.BH * p.N, 16);
  char* at = static_cast<char*>(w.scratch);
  float4* kept = reinterpret_cast<float4*>(at);
  float* ends = reinterpret_cast<float*>(at += wide_kept(p, f.D, f.M));
  float* dot_q = reinterpret_cast<float*>(at += 16 * blocks * p.BH * chunks);
  float* dot_k = reinterpret_cast<float*>(at += dots);
  float* inter = reinterpret_cast<float*>(at += dots);
  cudaError_t e = gated_mma_states(p, f.k, f.v, f.q, f.dout, f.g, f.D, f.M, nullptr, f.H,
                                   f.dS0 != nullptr, w, st);
  if (e != cudaSuccess) return e;
  const GatedGradients back{f.dS, f.dS0};
  if ((e = gated_scan(p, w, f.S0, nullptr, GatedEntries{nullptr, 0, f.H}, f.D * f.M, st, &back)) != cudaSuccess)
    return e;
  WalkArgs a{};
  a.g = static_cast<const bf16*>(f.g);
  a.N = f.N;
  a.BH = p.BH;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.H = f.H;
  a.entries.H = f.H;
  a.kept = kept;
  a.ends = ends;
  a.inter = inter;
  WalkArgs dq = a, dk = a, dv = a;
  dq.z = dk.w = dv.u = static_cast<const bf16*>(f.dout);
  dq.w = dk.z = static_cast<const bf16*>(f.v);
  dq.u = dk.p = dv.z = static_cast<const bf16*>(f.k);
  dq.p = dk.u = dv.w = static_cast<const bf16*>(f.q);
  dq.out = static_cast<bf16*>(f.dq);
  dk.out = static_cast<bf16*>(f.dk);
  dv.out = static_cast<bf16*>(f.dv);
  dq.ZD = dk.ZD = dv.UD = f.M;
  dq.UD = dk.UD = dv.ZD = f.D;
  dq.rs = dk.rs = dv.cs = 1;
  dq.cs = dk.cs = dv.rs = f.M;
  dq.seg_in = w.S;
  dk.seg_in = dv.seg_in = w.E;
  dq.dots = dot_q;
  dk.dots = dot_k;
  e = launch_gradient<false, true>(dq, st);
  if (e == cudaSuccess) e = launch_gradient<true, true>(dk, st);
  if (e == cudaSuccess) e = launch_gradient<true, false>(dv, st);
  if (e != cudaSuccess) return e;
  const long long warps = (long long)p.BH * (long long)chunks;
  e = tcx::launch_pdl(gated_chunk_dg_kernel, dim3((unsigned)((warps + 3) / 4)), dim3(kThreads), 0, st,
                      (const float*)dot_q, (const float*)dot_k, (const float*)inter, (const float*)ends,
                      static_cast<bf16*>(f.dg), p.BH, f.N, (int)blocks);
  count_launches(1);
  return e;
}

}  // namespace la
