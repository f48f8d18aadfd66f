// Gated recurrence in float32 on CUDA cores (tensor cores would round its inputs; D
// and M multiples of 8 up to 128), the scan over segments, and the decode step.
//
// One kernel carries every direction. With X a state and u, w, z three of the
// inputs, it walks a segment's tokens updating X by an outer product and reading
// it out along its columns:
//   forward   X = a_t X + u_t w_t^T;  y_t = X z_t
//   reverse   X = X + u_t w_t^T;  y_t = X z_t;  X = a_t X       (a_t = exp(g_t))
//   out   forward, X = S^T:  u = v,    w = k,    z = q
//   dq    forward, X = S:    u = k,    w = v,    z = dout
//   dk    reverse, X = dS:   u = q,    w = dout, z = v
//   dv    reverse, X = dS^T: u = dout, w = q,    z = k
// (dS_t is the loss's gradient with respect to S_t: dS_t = q_t dout_t^T + a_{t+1}
// dS_{t+1}.) The rows of X are independent of each other, so they are split over
// threads and CTAs freely, and the sum over columns stays within a thread and its
// neighbours.
//
// The token's own term is read out apart, y_t = X' z_t + u_t (w_t . z_t) with X' the
// state without it.
//
// The decay's gradient is dg_t = <dS_t, a_t S_{t-1}>. Its differences are two dots,
//   dg_t - dg_{t+1} = q_t . (a_t S_{t-1} dout_t) - k_t . (a_{t+1} dS_{t+1} v_t),
// with the token's own term left out of both (it would cancel, and outweighs the rest
// under a strong gate). So dg is a sum from a segment's last token back, begun there
// with <a S, E> of the segment's two states. It restarts in every segment, so that
// rounding errors do not pile up over the sequence.
//
// B2 H8 N4096 D = M = 64: forward 113 us, backward 288 us; B16 H16 N512 181 and 410. Bound by
// the reads of w and z from shared memory (two 16-byte words for six packed multiply-adds) and
// their waits. (Tiles of 4 rows by 16 columns a thread, which read a fourth as much, took 115
// and 312 us when this layout took 113 and 281: fewer and longer chains.)
#include "la_gated.cuh"
#include "la_gated_mma.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace {

using tcx::fma2;
using tcx::mul2;

constexpr int kThreads = 128;
constexpr int kTok = 16;       // tokens staged at a time

template <typename T>
struct RecurArgs {
  const T *u, *w, *z, *g;
  T* y;                  // outputs [BH][N][NR] (nullptr: state pass)
  const T* p;            // [BH][N][NR]: dots[rb][bh][t] = sum over rows of p (X' z) (nullptr: none)
  float* dots;
  // forward: ends[rb][bh][seg] = <X', E> at the segment's last token (nullptr: none); E is
  // entry seg + 1 of E's, or with one segment the caller's entry (nullptr: zero)
  const float* E;
  float* ends;
  int NR, NC, N, BH, len, n_seg;
  bool reverse;
  const int* lens;
  int H;
  // states: element (r, c) of an entry at r * rs + c * cs
  int rs, cs, DM;
  const float* seg_in;   // per-segment entries the walk starts from (nullptr: `init`)
  float* seg_out;        // state pass: per-segment entries it leaves
  float* decay;          // state pass: exp(sum of g) per segment
  const float* init;     // one segment: the caller's state (nullptr: zero)
  float* fin;            // one segment: the caller's final state (nullptr: not kept)
  GatedEntries entries;
  WorkspaceHeader* hdr;
};

// CP threads share a row, each with COLS of its columns (c = 4 (i CP + p) + 0..3, so
// that the lanes of a warp read neighbouring 16-byte words). 16 tokens are staged at a
// time, the next 16 on their way in registers meanwhile.
template <int CP, int COLS, bool REV, typename T>
__device__ __forceinline__ void recur_walk(const RecurArgs<T>& a) {
  constexpr int RB = kThreads / CP, ALL = COLS * CP;
  constexpr int PC = kTok * ALL / kThreads, PR = kTok * RB / kThreads;  // staged per thread
  __shared__ __align__(16) float sw[kTok][ALL], sz[kTok][ALL];
  __shared__ float su[kTok][RB], sy[kTok][RB + 1], sa[kTok], swz[kTok];
  __shared__ unsigned slow_tokens;  // bit t: sa[t] is exp(g_t) - 1, else exp(g_t)
  const int tid = threadIdx.x, part = tid % CP, row = tid / CP;
  const int bh = blockIdx.x / a.n_seg, seg = blockIdx.x % a.n_seg;
  const int r0 = blockIdx.y * RB, nr = min(RB, a.NR - r0);
  if (nr <= 0) return;
  const int n = gated_length(a.lens, a.H, bh, a.N);
  const int tb = min(seg * a.len, n), te = min(tb + a.len, n);
  const size_t seq = (size_t)bh * a.N;
  const T* u = a.u + seq * a.NR + r0;
  const T* w = a.w + seq * a.NC;
  const T* z = a.z + seq * a.NC;
  const T* g = a.g + seq;
  T* y = a.y + (a.y ? seq * a.NR + r0 : 0);

  float nw[PC], nz[PC], nu[PR], ng = 0.f;
  // the tile `done` tokens into the walk: its first token and count
  auto tile = [&](int done, int& t0) {
    const int m = min(kTok, te - tb - done);
    t0 = REV ? te - done - m : tb + done;
    return m;
  };
  auto fetch = [&](int done) {
    int t0;
    const int m = tile(done, t0);
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      const int at = tid + i * kThreads, t = at / ALL, c = at % ALL;
      const bool in = t < m && c < a.NC;
      nw[i] = in ? to_f32<T>(w[(size_t)(t0 + t) * a.NC + c]) : 0.f;
      nz[i] = in && a.y ? to_f32<T>(z[(size_t)(t0 + t) * a.NC + c]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < PR; ++i) {
      const int at = tid + i * kThreads, t = at / RB, r = at % RB;
      nu[i] = t < m && r < nr ? to_f32<T>(u[(size_t)(t0 + t) * a.NR + r]) : 0.f;
    }
    if (tid < kTok) ng = tid < m ? to_f32<T>(g[t0 + tid]) : 0.f;
  };
  if (tb < te) fetch(0);

  const long long entry = a.entries.at(bh);
  if (entry < 0 && seg == 0 && blockIdx.y == 0 && tid == 0 && a.hdr)
    a.hdr->status = LA_ERR_INVALID_ARG;
  const float* xin = nullptr;
  if (a.seg_in)
    xin = a.seg_in + ((size_t)bh * (a.n_seg + 1) + seg + (REV ? 1 : 0)) * a.DM;
  else if (a.init && entry >= 0)
    xin = a.init + (size_t)entry * a.DM;
  float2 x[COLS / 2];
#pragma unroll
  for (int i = 0; i < COLS / 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = 4 * (i * CP + part) + j;
      const bool in = xin && row < nr && c < a.NC;
      (&x[2 * i + j / 2].x)[j % 2] = in ? xin[(size_t)(r0 + row) * a.rs + (size_t)c * a.cs] : 0.f;
    }

  float end = 0.f;
  double gates = 0.0;  // a token of each tile (a product of float32 factors drifts by its roundings)
  for (int done = 0; done < te - tb; done += kTok) {
    int t0;
    const int m = tile(done, t0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      const int at = tid + i * kThreads;
      sw[at / ALL][at % ALL] = nw[i];
      sz[at / ALL][at % ALL] = nz[i];
    }
#pragma unroll
    for (int i = 0; i < PR; ++i) {
      const int at = tid + i * kThreads;
      su[at / RB][at % RB] = nu[i];
    }
    if (tid < 32) {
      const bool slow = tid < kTok && ng > -0.5f && ng < 0.5f;
      if (tid < kTok) {
        sa[tid] = slow ? expm1f(ng) : expf(ng);
        gates += (double)ng;
      }
      const unsigned bits = __ballot_sync(0xffffffffu, slow);
      if (tid == 0) slow_tokens = bits;
    }
    __syncthreads();
    if (done + kTok < te - tb) fetch(done + kTok);
    if (a.y) {  // w_t . z_t, eight threads a token
      float s = 0.f;
      for (int c = tid % 8; c < a.NC; c += 8) s = fmaf(sw[tid / 8][c], sz[tid / 8][c], s);
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tid % 8 == 0) swz[tid / 8] = s;
    }
    const unsigned slow_bits = slow_tokens;
    for (int k = 0; k < m; ++k) {
      const int t = REV ? m - 1 - k : k;
      const bool slow = slow_bits >> t & 1;
      const float at = sa[t], ut = su[t][row];
      const float2 a2 = make_float2(at, at), u2 = make_float2(ut, ut);
      // X + X (exp(g) - 1) near 1: exp(g) itself would keep too little of g, and with the same
      // gate at every token its rounding does not average out (1200 tokens of g = -3.1e-4:
      // final states off by 5.0e-6 instead of 8e-7). A branch a token, forward 5 to 10%.
      // Measured and not kept: X c + X e with c 0 or 1 (forward 14%, backward 10%), both
      // factors by predicates (spills; 20 to 30%), a loop of its own for tiles of slow gates
      // (spills; no faster than the branch). A token rounds X twice, here and by its outer
      // product; e X + (e' X + u w) with e + e' = exp(g) rounds it once, 1.4 times as exact,
      // and took up to 14% longer forward and 23% back; X kept as exp(sum of g) Y 2 to 11%, with
      // the terms under fast gates less exact instead.
      auto forget = [&]() {
        if (slow) {
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) x[i] = fma2(a2, x[i], x[i]);
        } else {
#pragma unroll
          for (int i = 0; i < COLS / 2; ++i) x[i] = mul2(a2, x[i]);
        }
      };
      if (!REV && a.E && t0 + t == te - 1) {
        const float* E = a.E + (a.seg_in ? (size_t)bh * (a.n_seg + 1) + seg + 1 : bh) * a.DM;
        if (row < nr)
#pragma unroll
          for (int i = 0; i < COLS / 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int c = 4 * (i * CP + part) + j;
              if (c < a.NC)
                end = fmaf((slow ? 1.f + at : at) * (&x[2 * i + j / 2].x)[j % 2],
                           E[(size_t)(r0 + row) * a.rs + (size_t)c * a.cs], end);
            }
      }
      if (!REV) forget();
      float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < COLS / 4; ++i) {
        const int c = 4 * (i * CP + part);
        const float4 wv = *reinterpret_cast<const float4*>(&sw[t][c]);
        if (a.y) {
          const float4 zv = *reinterpret_cast<const float4*>(&sz[t][c]);
          s2 = fma2(x[2 * i], make_float2(zv.x, zv.y), s2);
          s2 = fma2(x[2 * i + 1], make_float2(zv.z, zv.w), s2);
        }
        x[2 * i] = fma2(u2, make_float2(wv.x, wv.y), x[2 * i]);
        x[2 * i + 1] = fma2(u2, make_float2(wv.z, wv.w), x[2 * i + 1]);
      }
      if (REV) forget();
      if (a.y) {
        float s = s2.x + s2.y;
#pragma unroll
        for (int o = 1; o < CP; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (part == 0) sy[t][row] = s;
      }
    }
    if (a.y) {
      __syncthreads();
      for (int i = tid; i < m * RB; i += kThreads) {
        const int t = i / RB, r = i % RB;
        if (r < nr) y[(size_t)(t0 + t) * a.NR + r] = from_f32<T>(fmaf(su[t][r], swz[t], sy[t][r]));
      }
      if (a.p) {
        const T* p = a.p + seq * a.NR + r0;
        const int t = tid / 8;
        float s = 0.f;
        if (t < m)
          for (int r = tid % 8; r < nr; r += 8) s = fmaf(sy[t][r], to_f32<T>(p[(size_t)(t0 + t) * a.NR + r]), s);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (t < m && tid % 8 == 0)
          a.dots[((size_t)blockIdx.y * a.BH + bh) * a.N + t0 + t] = s;
      }
    }
  }

  if (!REV && a.ends) {
    for (int o = 16; o > 0; o >>= 1) end += __shfl_xor_sync(0xffffffffu, end, o);
    __syncthreads();
    if (tid % 32 == 0) sa[tid / 32] = end;
    __syncthreads();
    if (tid == 0)
      a.ends[((size_t)blockIdx.y * a.BH + bh) * a.n_seg + seg] = sa[0] + sa[1] + sa[2] + sa[3];
  }

  float* xout = nullptr;
  if (a.seg_out)
    xout = a.seg_out + ((size_t)bh * (a.n_seg + 1) + seg) * a.DM;
  else if (a.fin && entry >= 0)
    xout = a.fin + (size_t)entry * a.DM;
  if (xout && row < nr)
#pragma unroll
    for (int i = 0; i < COLS / 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 4 * (i * CP + part) + j;
        if (c < a.NC) xout[(size_t)(r0 + row) * a.rs + (size_t)c * a.cs] = (&x[2 * i + j / 2].x)[j % 2];
      }
  if (a.decay && blockIdx.y == 0 && tid < 32) {
#pragma unroll
    for (int o = kTok / 2; o > 0; o >>= 1) gates += __shfl_down_sync(0xffffffffu, gates, o);
    if (tid == 0) a.decay[(size_t)bh * a.n_seg + seg] = gated_decay((float)gates);
  }
}

constexpr int walks_per_sm(int cp, int cols) { return cols == 8 ? 5 : cp == 2 || cols < 32 ? 4 : 3; }

// blockIdx.z: one of up to three walks that do not depend on each other
template <typename T>
struct RecurJobs {
  RecurArgs<T> job[3];
};
template <int CP, int COLS, typename T>
__global__ void __launch_bounds__(kThreads, walks_per_sm(CP, COLS))
gated_recur_kernel(const __grid_constant__ RecurJobs<T> jobs) {
  const RecurArgs<T>& a = jobs.job[blockIdx.z];
  tc::pdl_wait();
  if (a.reverse)
    recur_walk<CP, COLS, true, T>(a);
  else
    recur_walk<CP, COLS, false, T>(a);
}

// Joins the segments: forward X[s + 1] = decay[s] X[s] + U[s] from X[0] = init,
// reverse X[s] = decay[s] X[s + 1] + U[s] from X[n_seg] = init; U[s] is read from
// entry s and replaced there. One thread per state element, its loads four segments
// ahead of their use (the walk is bound by their latency). blockIdx.z: which of the
// two jobs (states, gradients).
struct ScanJob {
  float* X;
  const float* init;
  float* fin;
  bool reverse;
};
__global__ void __launch_bounds__(256)
gated_scan_kernel(const ScanJob first, const ScanJob second, const float* __restrict__ decay,
                  const GatedEntries entries, int n_seg, int DM, WorkspaceHeader* hdr) {
  constexpr int kAhead = 4;
  const ScanJob& job = blockIdx.z == 0 ? first : second;
  const int bh = blockIdx.x;
  const int i = blockIdx.y * 256 + threadIdx.x;
  tc::pdl_wait();
  const long long entry = entries.at(bh);
  if (entry < 0 && i == 0) hdr->status = LA_ERR_INVALID_ARG;
  if (i >= DM) return;
  float* x = job.X + (size_t)bh * (n_seg + 1) * DM + i;
  const float* dec = decay + (size_t)bh * n_seg;
  float s = job.init && entry >= 0 ? job.init[(size_t)entry * DM + i] : 0.f;
  // segment k of the walk; a forward walk leaves the state before it there, a reverse
  // one the gradient behind it one entry further on
  auto at = [&](int k) { return job.reverse ? n_seg - 1 - k : k; };
  float u[kAhead], d[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    u[j] = j < n_seg ? x[(size_t)at(j) * DM] : 0.f;
    d[j] = j < n_seg ? dec[at(j)] : 0.f;
  }
  if (job.reverse) x[(size_t)n_seg * DM] = s;
  for (int k0 = 0; k0 < n_seg; k0 += kAhead) {
    float un[kAhead], dn[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + kAhead + j;
      un[j] = k < n_seg ? x[(size_t)at(k) * DM] : 0.f;
      dn[j] = k < n_seg ? dec[at(k)] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int k = k0 + j;
      if (k >= n_seg) break;
      const float before = s;
      s = fmaf(d[j], s, u[j]);
      x[(size_t)at(k) * DM] = job.reverse ? s : before;
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      u[j] = un[j];
      d[j] = dn[j];
    }
  }
  if (!job.reverse) x[(size_t)n_seg * DM] = s;
  if (job.fin && entry >= 0) job.fin[(size_t)entry * DM + i] = s;
}

// dg of one segment: from <X', E> at its last token back,
//   dg_t = <X', E> + sum over s >= t of dot_q[s] - sum over t <= s < last of dot_k[s],
// 256 tokens at a time (each dot the sum of its row blocks').
template <typename T>
__global__ void __launch_bounds__(256)
gated_dg_kernel(const float* __restrict__ ends, const float* __restrict__ dot_q,
                const float* __restrict__ dot_k, T* __restrict__ dg, int BH, int N, int len,
                int n_seg, int rb) {
  __shared__ float part[8];
  const int bh = blockIdx.x / n_seg, seg = blockIdx.x % n_seg, tid = threadIdx.x;
  const int tb = seg * len, te = min(tb + len, N);
  tc::pdl_wait();
  float carry = 0.f;
  for (int r = 0; r < rb; ++r) carry += ends[((size_t)r * BH + bh) * n_seg + seg];
  for (int hi = te; hi > tb; hi -= 256) {
    const int t = hi - 1 - tid;
    float s = 0.f;
    if (t >= tb) {
      for (int r = 0; r < rb; ++r) s += dot_q[((size_t)r * BH + bh) * N + t];
      float k = 0.f;
      if (t < te - 1)
        for (int r = 0; r < rb; ++r) k += dot_k[((size_t)r * BH + bh) * N + t];
      s -= k;
    }
    for (int o = 1; o < 32; o <<= 1) {
      const float other = __shfl_up_sync(0xffffffffu, s, o);
      if (tid % 32 >= o) s += other;
    }
    __syncthreads();
    if (tid % 32 == 31) part[tid / 32] = s;
    __syncthreads();
    float before = carry;
    for (int i = 0; i < tid / 32; ++i) before += part[i];
    if (t >= tb) dg[(size_t)bh * N + t] = from_f32<T>(before + s);
    for (int i = 0; i < 8; ++i) carry += part[i];
  }
}

// Threads per row and columns per thread: the widest of a call's states decides, so that its
// walks share launches. Few columns and rows are left idle, and more than 16 columns a thread
// pay where there are as many (two threads of 32 for 64: 500 tokens of 60 sequences forward 74
// us, four of 16 95). Against 32 columns for all: D = M = 32, 600 sequences of 300 tokens
// forward 186 to 92 us, backward 487 to 285; 48, 60 sequences 40 to 35 and 96 to 83; 72, 60
// sequences of 500 tokens 216 to 165 and 498 to 265.
struct Columns {
  int parts, each;
};
Columns columns(int D, int M) {
  const int nc = D > M ? D : M;
  return nc <= 32   ? Columns{4, 8}
         : nc <= 48 ? Columns{2, 24}
         : nc <= 64 ? Columns{2, 32}
         : nc <= 80 ? Columns{4, 20}
         : nc <= 96 ? Columns{4, 24}
                    : Columns{4, 32};
}

int row_blocks(int NR, int cp) { return (NR * cp + kThreads - 1) / kThreads; }

template <typename T>
cudaError_t launch_recur(const RecurJobs<T>& jobs, int count, int D, int M, cudaStream_t st) {
  const RecurArgs<T>& a = jobs.job[0];
  const Columns c = columns(D, M);
  const dim3 grid((unsigned)(a.BH * a.n_seg), (unsigned)row_blocks(D > M ? D : M, c.parts), count);
  auto launch = [&](auto kernel) { return tcx::launch_pdl(kernel, grid, dim3(kThreads), 0, st, jobs); };
  const cudaError_t e = c.each == 8    ? launch(gated_recur_kernel<4, 8, T>)
                        : c.each == 20 ? launch(gated_recur_kernel<4, 20, T>)
                        : c.parts == 2 ? c.each == 24 ? launch(gated_recur_kernel<2, 24, T>)
                                                      : launch(gated_recur_kernel<2, 32, T>)
                        : c.each == 24 ? launch(gated_recur_kernel<4, 24, T>)
                                       : launch(gated_recur_kernel<4, 32, T>);
  count_launches(1);
  return e;
}

// A walk of `ctas` CTAs over `len` tokens in microseconds, as measured: the slower on a
// token the more of them share an SM.
float walk_time(long long ctas, int per_sm, int len) {
  auto token = [](long long on_sm) { return 0.16f + 0.09f * (float)on_sm; };
  const long long full = ctas / (152 * per_sm), rest = ctas % (152 * per_sm);
  return (float)len * ((float)full * token(per_sm) + (rest ? token((rest + 151) / 152) : 0.f));
}

// The segments with which the walks take least: several fill the GPU, but cost the state
// passes (0.65 of a walk of outputs) and the scan first. At least 32 tokens each, one of
// several at most 4096 (its decay is one float32, which has to be finite where gates are
// positive), a backward's at most 512, over which dg's sum from the segment's end back keeps
// float32's accuracy. 128 tokens, D = M = 64, several segments and one: backward of 8 sequences 29 and
// 45 us, of 152 109 and 67, of 600 363 and 208; forward of 60 28 and 36, of 600 143 and 68.
GatedPlan plan_simt(int BH, int N, int D, int M, bool backward) {
  const Columns c = columns(D, M);
  const int per_sm = walks_per_sm(c.parts, c.each);
  const long long per = (long long)BH * row_blocks(D > M ? D : M, c.parts);
  const long long most = N > 0 ? (N + 31) / 32 : 1, fewest = backward && N > 512 ? (N + 511) / 512 : 1;
  GatedPlan best{BH, N, kTok, 1};
  float shortest = -1.f;
  for (int k = 0; k <= 16; ++k) {
    long long n_seg = k == 0 ? 1 : k * 152LL / per;
    if (n_seg > 1 && n_seg * 4096 < N) n_seg = (N + 4095) / 4096;
    if (n_seg > most) n_seg = most;
    if (n_seg < fewest) n_seg = fewest;
    const int len = N > 0 ? (int)(((N + n_seg - 1) / n_seg + kTok - 1) / kTok * kTok) : kTok;
    n_seg = N > 0 ? (N + len - 1) / len : 1;
    float t = walk_time((backward ? 3 : 1) * per * n_seg, per_sm, len);
    if (n_seg > 1)
      t += 7.f + 0.1f * (float)n_seg + 0.65f * walk_time((backward ? 2 : 1) * per * n_seg, per_sm, len);
    if (shortest < 0.f || t < shortest) {
      shortest = t;
      best.len = len;
      best.n_seg = (int)n_seg;
    }
  }
  return best;
}

GatedWorkspace carve(void* ws, const GatedPlan& p, int D, int M, bool backward, int dots,
                     size_t scratch = 0) {
  GatedWorkspace w{};
  const uintptr_t base = reinterpret_cast<uintptr_t>(ws);
  size_t at = kHeaderBytes;
  const size_t dm = (size_t)D * M, seq = (size_t)p.BH;
  auto take = [&](size_t floats) {
    float* r = reinterpret_cast<float*>(base + at);
    at += align_up(sizeof(float) * floats, 256);
    return r;
  };
  w.hdr = static_cast<WorkspaceHeader*>(ws);
  if (backward || p.n_seg > 1) {
    w.decay = take(seq * p.n_seg);
    w.S = take(seq * (p.n_seg + 1) * dm);
  }
  if (backward) {
    w.E = take(seq * (p.n_seg + 1) * dm);
    w.scratch = take(scratch / sizeof(float));
    w.dot_q = take((size_t)dots * seq * p.N);
    w.dot_k = take((size_t)dots * seq * p.N);
    w.ends = take((size_t)dots * seq * p.n_seg);
  }
  w.bytes = at;
  return w;
}

cudaError_t simt_forward(const GatedForward& f, const GatedPlan& p, const GatedWorkspace& w,
                         cudaStream_t st) {
  RecurJobs<float> jobs{};
  RecurArgs<float>& a = jobs.job[0];
  a.g = static_cast<const float*>(f.g);
  a.N = f.N;
  a.BH = p.BH;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.lens = f.lens;
  a.H = f.H;
  a.DM = f.D * f.M;
  a.entries = GatedEntries{f.slots, f.pool, f.H};
  a.hdr = w.hdr;
  cudaError_t e;
  if (p.n_seg > 1) {
    RecurJobs<float> states = jobs;  // X = S: rows d
    RecurArgs<float>& s = states.job[0];
    s.u = static_cast<const float*>(f.k);
    s.w = s.z = static_cast<const float*>(f.v);
    s.NR = f.D;
    s.NC = f.M;
    s.rs = f.M;
    s.cs = 1;
    s.seg_out = w.S;
    s.decay = w.decay;
    if ((e = launch_recur(states, 1, f.D, f.M, st)) != cudaSuccess) return e;
    if ((e = gated_scan(p, w, f.S0, f.S, a.entries, a.DM, st)) != cudaSuccess) return e;
    a.seg_in = w.S;
  } else {
    a.init = f.S0;
    a.fin = f.S;
  }
  a.u = static_cast<const float*>(f.v);  // X = S^T: rows m
  a.w = static_cast<const float*>(f.k);
  a.z = static_cast<const float*>(f.q);
  a.y = static_cast<float*>(f.out);
  a.NR = f.M;
  a.NC = f.D;
  a.rs = 1;
  a.cs = f.M;
  return launch_recur(jobs, 1, f.D, f.M, st);
}

int backward_dots(int D, int M) { return row_blocks(D, columns(D, M).parts); }

template <typename T>
cudaError_t simt_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                          cudaStream_t st) {
  const int rb = backward_dots(f.D, f.M);
  const T *q = static_cast<const T*>(f.q), *k = static_cast<const T*>(f.k),
              *v = static_cast<const T*>(f.v), *dout = static_cast<const T*>(f.dout);
  RecurArgs<T> a{};  // X = S, dS: rows d
  a.g = static_cast<const T*>(f.g);
  a.N = f.N;
  a.BH = p.BH;
  a.len = p.len;
  a.n_seg = p.n_seg;
  a.H = f.H;
  a.DM = f.D * f.M;
  a.entries = GatedEntries{nullptr, 0, f.H};
  a.NR = f.D;
  a.NC = f.M;
  a.rs = f.M;
  a.cs = 1;
  // One segment starts from the caller's states (unless dS0 takes the place of dS, which the
  // other walks still read).
  const bool whole = p.n_seg == 1 && (f.dS0 == nullptr || f.dS0 != f.dS);
  cudaError_t e;
  if (!whole) {  // the segments' own states and gradients
    RecurJobs<T> states{{a, a, a}};
    RecurArgs<T> &s = states.job[0], &r = states.job[1];
    s.u = k;
    s.w = s.z = v;
    s.seg_out = w.S;
    s.decay = w.decay;
    r.reverse = true;
    r.u = q;
    r.w = r.z = dout;
    r.seg_out = w.E;
    if ((e = launch_recur(states, 2, f.D, f.M, st)) != cudaSuccess) return e;
    const GatedGradients back{f.dS, f.dS0};
    if ((e = gated_scan(p, w, f.S0, nullptr, a.entries, a.DM, st, &back)) != cudaSuccess) return e;
  }
  RecurJobs<T> grads{{a, a, a}};
  RecurArgs<T> &dq = grads.job[0], &dk = grads.job[1], &dv = grads.job[2];
  dq.u = k;
  dq.w = v;
  dq.z = dout;
  dq.y = static_cast<T*>(f.dq);
  dq.p = q;
  dq.dots = w.dot_q;
  dq.ends = w.ends;
  dk.reverse = dv.reverse = true;
  dk.u = q;
  dk.w = dout;
  dk.z = v;
  dk.y = static_cast<T*>(f.dk);
  dk.p = k;
  dk.dots = w.dot_k;
  dv.u = dout;  // rows m: dS^T
  dv.w = q;
  dv.z = k;
  dv.y = static_cast<T*>(f.dv);
  dv.NR = f.M;
  dv.NC = f.D;
  dv.rs = 1;
  dv.cs = f.M;
  if (whole) {
    dq.init = f.S0;
    dq.E = dk.init = dv.init = f.dS;
    dk.fin = f.dS0;
  } else {
    dq.seg_in = w.S;
    dq.E = dk.seg_in = dv.seg_in = w.E;
  }
  if ((e = launch_recur(grads, 3, f.D, f.M, st)) != cudaSuccess) return e;
  e = tcx::launch_pdl(gated_dg_kernel<T>, dim3((unsigned)(p.BH * p.n_seg)), dim3(256), 0, st,
                      (const float*)w.ends, (const float*)w.dot_q, (const float*)w.dot_k,
                      static_cast<T*>(f.dg), p.BH, p.N, p.len, p.n_seg, rb);
  count_launches(1);
  return e;
}

// Decode step: one CTA per (stream, head). Bound by the state's read and write
// (2 D M 4 bytes; 256 streams of 8 heads, D = M = 64: 12.9 us for 67 MB, 9.9 at HBM's rate); a thread owns a float4 column group in every rgs-th row, and asks
// for up to eight of its rows before it uses the first.
template <typename T>
__global__ void __launch_bounds__(kThreads)
gated_decode_kernel(const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                    const T* __restrict__ g, float* S, T* __restrict__ out,
                    const GatedEntries entries, int D, int M) {
  __shared__ float fq[128], fk[128];
  __shared__ __align__(16) float vs[128];
  __shared__ __align__(16) float red[kThreads * 4];
  const size_t sh = blockIdx.x;
  const int tid = threadIdx.x;
  tc::pdl_wait();
  const long long entry = entries.at((int)sh);
  const int cg = M >> 2, rgs = kThreads / cg, col = tid % cg, rg = tid / cg;
  float4* S4 = reinterpret_cast<float4*>(S + (size_t)(entry < 0 ? 0 : entry) * D * M);
  constexpr int kBatch = 8;
  float4 s[kBatch];
#pragma unroll
  for (int j = 0; j < kBatch; ++j) {
    const int d = rg + j * rgs;
    s[j] = entry >= 0 && rg < rgs && d < D ? S4[d * cg + col] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const float a = gated_decay(to_f32<T>(g[sh]));
  if (tid < D) {
    fq[tid] = to_f32<T>(q[sh * D + tid]);
    fk[tid] = to_f32<T>(k[sh * D + tid]);
  }
  if (tid < M) vs[tid] = to_f32<T>(v[sh * M + tid]);
  __syncthreads();
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (rg < rgs) {
    const float4 v4 = *reinterpret_cast<const float4*>(&vs[4 * col]);
    for (int d0 = rg; d0 < D; d0 += kBatch * rgs) {
      if (d0 != rg)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const int d = d0 + j * rgs;
          s[j] = entry >= 0 && d < D ? S4[d * cg + col] : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int d = d0 + j * rgs;
        if (d >= D) break;
        const float kd = fk[d], qd = fq[d];
        s[j].x = fmaf(a, s[j].x, kd * v4.x);
        s[j].y = fmaf(a, s[j].y, kd * v4.y);
        s[j].z = fmaf(a, s[j].z, kd * v4.z);
        s[j].w = fmaf(a, s[j].w, kd * v4.w);
        if (entry >= 0) S4[d * cg + col] = s[j];
        acc.x = fmaf(qd, s[j].x, acc.x);
        acc.y = fmaf(qd, s[j].y, acc.y);
        acc.z = fmaf(qd, s[j].z, acc.z);
        acc.w = fmaf(qd, s[j].w, acc.w);
      }
    }
    *reinterpret_cast<float4*>(&red[rg * M + 4 * col]) = acc;
  }
  __syncthreads();
  if (tid < M) {
    float o = 0.f;
    for (int r = 0; r < rgs; ++r) o += red[r * M + tid];
    out[sh * M + tid] = from_f32<T>(o);
  }
}

}  // namespace

cudaError_t gated_scan(const GatedPlan& p, const GatedWorkspace& w, const float* S0, float* S,
                       const GatedEntries& e, int DM, cudaStream_t st, const GatedGradients* back) {
  const ScanJob first{w.S, S0, S, false};
  const ScanJob second = back ? ScanJob{w.E, back->dS, back->dS0, true} : first;
  const cudaError_t err =
      tcx::launch_pdl(gated_scan_kernel, dim3((unsigned)p.BH, (unsigned)((DM + 255) / 256), back ? 2 : 1),
                      dim3(256), 0, st, first, second, w.decay, e, p.n_seg, DM, w.hdr);
  count_launches(1);
  return err;
}

// float32, which the tensor cores would round, walks token by token.
static GatedPlan forward_plan(int BH, int N, int D, int M, int dtype) {
  return dtype == LA_F32 ? plan_simt(BH, N, D, M, false) : gated_mma_forward_plan(BH, N, D, M);
}

size_t gated_forward_workspace(int BH, int N, int D, int M, int dtype) {
  return carve(nullptr, forward_plan(BH, N, D, M, dtype), D, M, false, 0).bytes;
}

// A backward of a few tokens does too, where the tensor cores take several launches: their
// chunks cost the same for 1 token as for 64. Up to 64 columns and without dS0 they take one,
// and are faster for 2 tokens on. 512 sequences of 1, 4 and 16 tokens, us (on the tensor cores):
// D = M = 64 without dS0 16, 20, 35 (17, 17, 17), with it 27, 31, 48 (65, 65, 66); 128 60, 85,
// 184 (268, 268, 271). One sequence: 6, 8, 12 (7, 7, 7), 8, 10, 14 (11, 12, 12) and 6, 8, 13
// (27, 27, 28).
constexpr int kShort = 16;
static bool one_launch(int D, int M) { return D <= 64 && M <= 64; }
static bool backward_walks(int N, int D, int M, int dtype, bool dS0) {
  return dtype == LA_F32 || (N <= kShort && (N == 1 || dS0 || !one_launch(D, M)));
}

static GatedPlan backward_plan(int BH, int N, int D, int M, bool walks) {
  if (walks) return plan_simt(BH, N, D, M, true);
  return one_launch(D, M) ? gated_mma_backward_plan(BH, N) : gated_mma_wide_plan(BH, N, D, M);
}

static GatedWorkspace backward_workspace(void* ws, const GatedPlan& p, int D, int M, bool walks) {
  if (walks) return carve(ws, p, D, M, true, backward_dots(D, M));
  return carve(ws, p, D, M, true, 0,
               one_launch(D, M) ? gated_mma_backward_scratch(p) : gated_mma_wide_scratch(p, D, M));
}

size_t gated_backward_workspace(int BH, int N, int D, int M, int dtype) {
  size_t most = 0;
  for (const bool dS0 : {false, true}) {
    const bool walks = backward_walks(N, D, M, dtype, dS0);
    const size_t bytes = backward_workspace(nullptr, backward_plan(BH, N, D, M, walks), D, M, walks).bytes;
    if (bytes > most) most = bytes;
  }
  return most;
}

cudaError_t gated_forward(const GatedForward& f, void* ws, cudaStream_t st) {
  const GatedPlan p = forward_plan(f.B * f.H, f.N, f.D, f.M, f.dtype);
  const GatedWorkspace w = carve(ws, p, f.D, f.M, false, 0);
  return f.dtype == LA_F32 ? simt_forward(f, p, w, st) : gated_mma_forward(f, p, w, st);
}

cudaError_t gated_backward(const GatedBackward& f, void* ws, cudaStream_t st) {
  const bool walks = backward_walks(f.N, f.D, f.M, f.dtype, f.dS0 != nullptr);
  const GatedPlan p = backward_plan(f.B * f.H, f.N, f.D, f.M, walks);
  const GatedWorkspace w = backward_workspace(ws, p, f.D, f.M, walks);
  if (walks)
    return f.dtype == LA_F32 ? simt_backward<float>(f, p, w, st)
                             : simt_backward<__nv_bfloat16>(f, p, w, st);
  return one_launch(f.D, f.M) ? gated_mma_backward(f, p, w, st) : gated_mma_wide_backward(f, p, w, st);
}

cudaError_t gated_decode(const void* q, const void* k, const void* v, const void* g, float* S,
                         const int* slots, void* out, int pool, int n_streams, int H, int D, int M,
                         int dtype, cudaStream_t st) {
  const GatedEntries entries{slots, pool, H};
  const dim3 grid((unsigned)(n_streams * H)), block(kThreads);
  cudaError_t e;
  if (dtype == LA_F32)
    e = tcx::launch_pdl(gated_decode_kernel<float>, grid, block, 0, st, (const float*)q, (const float*)k,
                        (const float*)v, (const float*)g, S, (float*)out, entries, D, M);
  else
    e = tcx::launch_pdl(gated_decode_kernel<__nv_bfloat16>, grid, block, 0, st, (const __nv_bfloat16*)q,
                        (const __nv_bfloat16*)k, (const __nv_bfloat16*)v, (const __nv_bfloat16*)g, S,
                        (__nv_bfloat16*)out, entries, D, M);
  count_launches(1);
  return e;
}

}  // namespace la
