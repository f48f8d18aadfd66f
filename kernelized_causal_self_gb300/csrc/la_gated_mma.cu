// Gated recurrence in bf16 on tensor cores: forward, and the states of segments.
//
// A chunk of 64 tokens is a masked product and a rank-64 update. With G_i the sum of
// the chunk's g up to and including token i, G the whole chunk's, L_ij = exp(G_i - G_j)
// for j <= i and 0 above:
//   O = diag(exp(G_i)) (Q S) + ((Q K^T) * L) V
//   S = exp(G) S + (diag(exp(G - G_j)) K)^T V
// All exponents are <= 0 for g <= 0, so nothing overflows, and sums that reach a
// weight are taken from the end that weight decays from (G - G_j as a sum from the
// chunk's end), so that a strong gate elsewhere in the chunk costs no digits.
//
// Four warps share a chunk: warp r has its rows 16 r.. of Q and O and rows 16 r.. of
// S (of each 64), S in float32 accumulators that stay in registers over the whole
// segment. What is rounded to bf16: Q K^T * L as an operand, and the copy of S in
// shared memory that Q multiplies; the outputs, bf16 too, cannot show more. The update
// of S takes K's weighted rows as two bf16 terms (16 bits), since S itself is summed
// over the whole sequence and may be returned in float32.
//
// Why warp-level products and not tcgen05: at 64 columns a chunk's products are small
// next to its element-wise work (masks, weights, splits), which here happens in the
// registers that hold the fragments, with no round trip through tensor memory, no
// barrier between the product and its use, and three CTAs of four warps per SM to
// hide one another's waits. The products of the longest case take ~31 us of the
// tensor pipe at the 600 TFLOP/s these instructions reach; reading and writing
// q, k, v and out takes 40 us.
#include "la_gated.cuh"
#include "la_gated_mma.cuh"
#include "la_mma.cuh"
#include "la_tc_common.cuh"

namespace la {

using namespace mma;

namespace {

constexpr int kThreads = 128;

struct FwdArgs {
  const bf16 *q, *k, *v, *g;  // state pass: k, v are the pair whose outer products are summed
  bf16* out;
  int D, M, N, len, n_seg;
  const int* lens;
  int H;
  const float* seg_in;
  float *seg_out, *decay;
  const float* init;
  float* fin;
  GatedEntries entries;
  WorkspaceHeader* hdr;
};

template <int DZ, bool OUT>
struct FwdSmem {
  static constexpr int kQ = OUT ? kC * DZ * 2 : 0, kK = kC * DZ * 2, kV = kC * 64 * 2;
  static constexpr int kStage = kQ + kK + kV;
  static constexpr int kS = OUT ? DZ * 64 * 2 : 0;  // S in bf16, [d][m], one of two
  static constexpr int kBytes = 2 * kStage + 2 * kS + 4 * kC * 4 * 2;
};

// OUT: outputs (and, with one segment, the final state). Otherwise the state pass: the
// segment's own S from zero, over k, v with weights exp(G - G_j), or (REV) its own
// gradient of the incoming state from zero, over q, dout with weights exp(G_i), chunks
// from the last to the first.
// FRESH: a chunk's update of S is summed apart and then added, in float32 arithmetic that
// rounds; the tensor cores' own sums truncate, which over thousands of chunks would
// leave a bias in a state that hardly decays. Taken wherever S leaves the kernel in
// float32; where it only goes on as a bf16 operand, it is summed in place, which leaves
// registers for a third CTA per SM.
template <int DZ, bool OUT, bool REV, bool FRESH>
__device__ __forceinline__ void walk_chunks(const FwdArgs& a) {
  using Sm = FwdSmem<DZ, OUT>;
  constexpr int KS = DZ / 16, DT = DZ / 64;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t base = tc::smem_u32(smem);
  const uint32_t s_op = base + 2 * Sm::kStage;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float* Gs = reinterpret_cast<float*>(smem + 2 * Sm::kStage + 2 * Sm::kS) + warp * 2 * kC;
  float* Ws = Gs + kC;

  tc::pdl_wait();
  const int bh = blockIdx.x / a.n_seg, seg = blockIdx.x % a.n_seg;
  const int m0 = blockIdx.y * 64;
  // the causal product gives a chunk's last rows the most work: turn the rows' order
  // from CTA to CTA, so that no scheduler gets all of them
  const int rb = (warp + blockIdx.x) & 3;
  const int n = gated_length(a.lens, a.H, bh, a.N);
  const int tb = min(seg * a.len, n), te = min(tb + a.len, n);
  const int chunks = (te - tb + kC - 1) / kC;
  const size_t seq = (size_t)bh * a.N;
  const long long entry = a.entries.at(bh);
  if (entry < 0 && seg == 0 && m0 == 0 && tid == 0 && a.hdr) a.hdr->status = LA_ERR_INVALID_ARG;

  const int row = lane >> 2, col = (lane & 3) * 2;  // of an accumulator
  const Lane<DZ> ln;
  const Lane<64> ln64;
  float s[DT][8][4];
  {
    const float* in = nullptr;
    if (OUT && a.seg_in)
      in = a.seg_in + ((size_t)bh * (a.n_seg + 1) + seg) * a.D * a.M;
    else if (OUT && a.init && entry >= 0)
      in = a.init + (size_t)entry * a.D * a.M;
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = dt * 64 + rb * 16 + row + 8 * h, m = m0 + 8 * j + col;
          float2 x = make_float2(0.f, 0.f);
          if (in && d < a.D && m < a.M) x = *reinterpret_cast<const float2*>(in + (size_t)d * a.M + m);
          s[dt][j][2 * h] = x.x;
          s[dt][j][2 * h + 1] = x.y;
        }
  }
  auto keep_op = [&](int buf) {
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) store_op(ln64, s_op + buf * Sm::kS, dt * 64 + rb * 16, 0, s[dt]);
  };
  auto load_chunk = [&](int c) {
    const int t0 = tb + c * kC, rows = min(kC, te - t0);
    const uint32_t at = base + (c & 1) * Sm::kStage;
    if (OUT) load_tile<DZ, kThreads>(at, a.q + (seq + t0) * a.D, rows, a.D, 0);
    load_tile<DZ, kThreads>(at + Sm::kQ, a.k + (seq + t0) * a.D, rows, a.D, 0);
    load_tile<64, kThreads>(at + Sm::kQ + Sm::kK, a.v + (seq + t0) * a.M, rows, a.M, m0);
  };
  auto chunk_of = [&](int i) { return REV ? chunks - 1 - i : i; };
  auto raw_gates = [&](int c) { return load_gates(a.g + seq, tb + c * kC, te); };

  ushort2 g_next = make_ushort2(0, 0);
  float dec_all = 0.f;  // sum of the segment's g, base 2
  if (chunks > 0) {
    load_chunk(chunk_of(0));
    g_next = raw_gates(chunk_of(0));
  }
  cp_async_commit();
  if (OUT) keep_op(0);

  for (int i = 0; i < chunks; ++i) {
    const int c = chunk_of(i);
    cp_async_wait<0>();
    __syncthreads();  // chunk i has landed; every warp is done with chunk i - 1
    const float2 g = gates_of(g_next);
    if (i + 1 < chunks) {
      load_chunk(chunk_of(i + 1));
      g_next = raw_gates(chunk_of(i + 1));
    }
    cp_async_commit();
    const float total = chunk_gates<REV>(g, Gs, Ws);
    const float dec = gated_decay(total * kLn2);
    dec_all += total;

    const uint32_t q_at = base + (c & 1) * Sm::kStage, k_at = q_at + Sm::kQ, v_at = k_at + Sm::kK;
    float o[8][4];
    if (OUT) {
      uint32_t qa[KS][4];
      const float gi[2] = {Gs[rb * 16 + row], Gs[rb * 16 + row + 8]};
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) ln.load_a(qa[ks], q_at, rb * 16, ks);
      product<true>(ln64, o, qa, s_op + (i & 1) * Sm::kS);
      scale_rows(o, ex2(gi[0]), ex2(gi[1]));
      uint32_t p[4];
#pragma unroll 1
      for (int jb = 0; jb < rb; ++jb) {
        masked_block<true, false>(ln, p, qa, k_at, jb, gi, Gs);
        add_block(ln64, o, p, v_at, jb);
      }
      masked_block<true, true>(ln, p, qa, k_at, rb, gi, Gs);
      add_block(ln64, o, p, v_at, rb);
      // through this warp's rows of the Q tile, which no other warp reads
      const int t0 = tb + c * kC + rb * 16;
      store_rows(ln, q_at, rb * 16, o, a.out + (seq + t0) * a.M + m0, te - t0, a.M - m0, a.M);
    }
#pragma unroll
    for (int dt = 0; dt < DT; ++dt) {
      if (FRESH) {
        float u[8][4];
        add_outer<DZ, 8, true>(ln, ln64, u, k_at, Ws, 4 * dt + rb, v_at, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            pair_of(s[dt][j], h) = fma2(make_float2(dec, dec), pair_of(s[dt][j], h), pair_of(u[j], h));
      } else {
        scale_rows(s[dt], dec, dec);
        add_outer<DZ, 8>(ln, ln64, s[dt], k_at, Ws, 4 * dt + rb, v_at, 0);
      }
    }
    if (OUT && i + 1 < chunks) keep_op((i + 1) & 1);
  }

  float* to = nullptr;
  if (!OUT)
    to = a.seg_out + ((size_t)bh * (a.n_seg + 1) + seg) * a.D * a.M;
  else if (a.fin && entry >= 0)
    to = a.fin + (size_t)entry * a.D * a.M;
  if (to)
#pragma unroll
    for (int dt = 0; dt < DT; ++dt)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int d = dt * 64 + rb * 16 + row + 8 * h, m = m0 + 8 * j + col;
          if (d < a.D && m < a.M)
            *reinterpret_cast<float2*>(to + (size_t)d * a.M + m) =
                make_float2(s[dt][j][2 * h], s[dt][j][2 * h + 1]);
        }
  if (!OUT && a.decay && m0 == 0 && tid == 0)
    a.decay[(size_t)bh * a.n_seg + seg] = gated_decay(dec_all * kLn2);
}

template <int DZ, bool FRESH>
__global__ void __launch_bounds__(kThreads, DZ == 64 && !FRESH ? 3 : 2)
gated_forward_kernel(const FwdArgs a) {
  walk_chunks<DZ, true, false, FRESH>(a);
}

// blockIdx.z: the segments' states, or their gradients
template <int DZ>
__global__ void __launch_bounds__(kThreads, DZ == 64 ? 3 : 2)
gated_states_kernel(const FwdArgs a, const FwdArgs back) {
  if (blockIdx.z == 0)
    walk_chunks<DZ, false, false, true>(a);
  else
    walk_chunks<DZ, false, true, true>(back);
}

template <int DZ, bool FRESH>
cudaError_t launch_forward(const FwdArgs& a, int BH, cudaStream_t st) {
  using Sm = FwdSmem<DZ, true>;
  auto kernel = gated_forward_kernel<DZ, FRESH>;
  cudaError_t e = tcx::configure(kernel, Sm::kBytes);
  if (e != cudaSuccess) return e;
  e = tcx::launch_pdl(kernel, dim3((unsigned)(BH * a.n_seg), (unsigned)((a.M + 63) / 64)),
                      dim3(kThreads), Sm::kBytes, st, a);
  count_launches(1);
  return e;
}

template <int DZ>
cudaError_t launch_states(const FwdArgs& a, const FwdArgs* back, int BH, cudaStream_t st) {
  using Sm = FwdSmem<DZ, false>;
  auto kernel = gated_states_kernel<DZ>;
  cudaError_t e = tcx::configure(kernel, Sm::kBytes);
  if (e != cudaSuccess) return e;
  e = tcx::launch_pdl(kernel, dim3((unsigned)(BH * a.n_seg), (unsigned)((a.M + 63) / 64), back ? 2 : 1),
                      dim3(kThreads), Sm::kBytes, st, a, back ? *back : a);
  count_launches(1);
  return e;
}

}  // namespace

// Segments: one wave of the 152 SMs' resident CTAs, but no segment under four chunks
// (each costs the state pass and the scan).
GatedPlan gated_mma_plan(int BH, int N, int M, int resident) {
  const long long per = (long long)BH * ((M + 63) / 64);
  const long long chunks = (N + kC - 1) / kC;
  long long n_seg = (long long)152 * resident / per;
  if (n_seg > (chunks + 3) / 4) n_seg = (chunks + 3) / 4;
  if (n_seg < 1) n_seg = 1;
  long long len = (chunks + n_seg - 1) / n_seg;
  if (len < 1) len = 1;
  n_seg = (chunks + len - 1) / len;
  return GatedPlan{BH, N, (int)(len * kC), n_seg < 1 ? 1 : (int)n_seg};
}

GatedPlan gated_mma_forward_plan(int BH, int N, int D, int M) {
  return gated_mma_plan(BH, N, M, D <= 64 ? 3 : 2);
}

cudaError_t gated_mma_states(const GatedPlan& p, const void* k, const void* v, const void* q,
                             const void* dout, const void* g, int D, int M, const int* lens, int H,
                             const GatedWorkspace& w, cudaStream_t st) {
  FwdArgs s{};
  s.k = static_cast<const bf16*>(k);
  s.v = static_cast<const bf16*>(v);
  s.g = static_cast<const bf16*>(g);
  s.D = D;
  s.M = M;
  s.N = p.N;
  s.len = p.len;
  s.n_seg = p.n_seg;
  s.lens = lens;
  s.H = H;
  s.entries.H = H;
  s.seg_out = w.S;
  s.decay = w.decay;
  FwdArgs back = s;
  back.k = static_cast<const bf16*>(q);
  back.v = static_cast<const bf16*>(dout);
  back.seg_out = w.E;
  back.decay = nullptr;
  const FwdArgs* b = dout ? &back : nullptr;
  return D <= 64 ? launch_states<64>(s, b, p.BH, st) : launch_states<128>(s, b, p.BH, st);
}

cudaError_t gated_mma_forward(const GatedForward& f, const GatedWorkspace& w, cudaStream_t st) {
  const GatedPlan p = gated_mma_forward_plan(f.B * f.H, f.N, f.D, f.M);
  FwdArgs a{};
  a.q = static_cast<const bf16*>(f.q);
  a.k = static_cast<const bf16*>(f.k);
  a.v = static_cast<const bf16*>(f.v);
  a.g = static_cast<const bf16*>(f.g);
  a.out = static_cast<bf16*>(f.out);
  a.D = f.D;
  a.M = f.M;
  a.N = f.N;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.lens = f.lens;
  a.H = f.H;
  a.entries = GatedEntries{f.slots, f.pool, f.H};
  a.hdr = w.hdr;
  if (p.n_seg > 1) {
    cudaError_t e = gated_mma_states(p, f.k, f.v, nullptr, nullptr, f.g, f.D, f.M, f.lens, f.H, w, st);
    if (e != cudaSuccess) return e;
    if ((e = gated_scan(p, w, f.S0, f.S, a.entries, f.D * f.M, st)) != cudaSuccess) return e;
    a.seg_in = w.S;
  } else {
    a.init = f.S0;
    a.fin = f.S;
  }
  if (a.fin)
    return f.D <= 64 ? launch_forward<64, true>(a, p.BH, st) : launch_forward<128, true>(a, p.BH, st);
  return f.D <= 64 ? launch_forward<64, false>(a, p.BH, st) : launch_forward<128, false>(a, p.BH, st);
}

}  // namespace la
