// The gates of a 64-token chunk, as the tensor-core kernels use them.
#pragma once

#include <atomic>

#include "la_gated.cuh"
#include "la_mma.cuh"
#include "la_tc_common.cuh"

namespace la {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Gates of tokens t0 + 2 l, t0 + 2 l + 1 (l the lane) as they are stored; 0 from token
// `end` on. (Converted where they are used, so that the load's latency is not waited for
// where it is issued.)
__device__ __forceinline__ ushort2 load_gates(const mma::bf16* g, int t0, int end) {
  const int t = t0 + 2 * (threadIdx.x & 31);
  const unsigned short* p = reinterpret_cast<const unsigned short*>(g);
  return make_ushort2(t < end ? p[t] : 0, t + 1 < end ? p[t + 1] : 0);
}

// Base 2, and no lower than -200: 2^-200 is zero in float32, and -inf less -inf is not.
__device__ __forceinline__ float2 gates_of(ushort2 g) {
  const float a = __uint_as_float((uint32_t)g.x << 16) * kLog2e;
  const float b = __uint_as_float((uint32_t)g.y << 16) * kLog2e;
  return make_float2(a < -200.f ? -200.f : a, b < -200.f ? -200.f : b);
}

// a + b as the nearest float32, and what that leaves (exactly)
__device__ __forceinline__ float two_sum(float a, float b, float& rest) {
  const float s = a + b, from_b = s - a;
  rest = (a - (s - from_b)) + (b - from_b);
  return s;
}

// From a lane's two gates, tables of the chunk (made by one warp for all). Every weight is
// made of sums within a block of 16 tokens, begun at the end that it decays from, and of the
// sums of whole blocks: what a strong gate adds to another token's sum costs no digits.
//   hi + lo [i]  the block's gates up to and including token i. In two terms, since weights
//         within a block are made of differences of them (of one term, 40 resets before a
//         chunk's other tokens left those weights off by 2e-3)
//   in[i] = 2^(that), out[i] = 2^(the block's gates behind i), total[b] = 2^(block b's), so
//         that token j's weight for token i of a later block is out[j] times the blocks
//         between times in[i]
//   before[b], behind[b] = 2^(the chunk's other blocks on that side of b)
//   X[i]  weights of an operand's rows: 2^(sum of the chunk's gates behind i), what is left
//         of i's outer product in the state after the chunk, with REV 2^(sum up to and
//         including i); as split_pair's, or if EXACT as float32
//   decay of the whole chunk; its sum is returned
struct GateTables {
  float hi[mma::kC], lo[mma::kC], in[mma::kC], out[mma::kC], X[mma::kC];
  float total[4], before[4], behind[4], decay, pad[3];
};
template <bool REV, bool EXACT>
__device__ __forceinline__ float chunk_gates(ushort2 raw, GateTables& t) {
  const int lane = threadIdx.x & 31, block = lane >> 3, at = lane & 7;
  const float2 g = gates_of(raw);
  float hi, lo, rest, down = g.x + g.y;
  hi = two_sum(g.x, g.y, lo);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    const float uh = __shfl_up_sync(0xffffffffu, hi, o, 8), ul = __shfl_up_sync(0xffffffffu, lo, o, 8);
    const float d = __shfl_down_sync(0xffffffffu, down, o, 8);
    if (at >= o) {
      hi = two_sum(hi, uh, rest);
      lo += ul + rest;
    }
    if (at + o < 8) down += d;
  }
  float first_hi = __shfl_up_sync(0xffffffffu, hi, 1, 8), first_lo = __shfl_up_sync(0xffffffffu, lo, 1, 8);
  float after = __shfl_down_sync(0xffffffffu, down, 1, 8);
  if (at == 0) first_hi = first_lo = 0.f;
  if (at == 7) after = 0.f;
  first_hi = two_sum(first_hi, g.x, rest);
  first_lo += rest;
  const float2 upto = make_float2(first_hi + first_lo, hi + lo), left = make_float2(after + g.y, after);
  const float t0 = __shfl_sync(0xffffffffu, upto.y, 7), t1 = __shfl_sync(0xffffffffu, upto.y, 15),
              t2 = __shfl_sync(0xffffffffu, upto.y, 23), t3 = __shfl_sync(0xffffffffu, upto.y, 31);
  const float before = block == 0 ? 0.f : block == 1 ? t0 : block == 2 ? t0 + t1 : t0 + t1 + t2;
  const float behind = block == 3 ? 0.f : block == 2 ? t3 : block == 1 ? t2 + t3 : t1 + (t2 + t3);
  const float2 w = REV ? make_float2(mma::ex2(before + upto.x), mma::ex2(before + upto.y))
                       : make_float2(mma::ex2(left.x + behind), mma::ex2(left.y + behind));
  reinterpret_cast<float2*>(t.hi)[lane] = make_float2(first_hi, hi);
  reinterpret_cast<float2*>(t.lo)[lane] = make_float2(first_lo, lo);
  reinterpret_cast<float2*>(t.in)[lane] = make_float2(mma::ex2(upto.x), mma::ex2(upto.y));
  reinterpret_cast<float2*>(t.out)[lane] = make_float2(mma::ex2(left.x), mma::ex2(left.y));
  if (EXACT)
    reinterpret_cast<float2*>(t.X)[lane] = w;
  else
    reinterpret_cast<uint2*>(t.X)[lane] = mma::split_pair(w);
  if (at == 7) {
    t.total[block] = mma::ex2(upto.y);
    t.before[block] = mma::ex2(before);
    t.behind[block] = mma::ex2(behind);
  }
  const float whole = t0 + t1 + (t2 + t3);
  if (lane == 0) t.decay = gated_decay(whole * kLn2);
  return whole;
}

// tcx::configure, once per kernel and device (its two calls of the runtime cost as much as a
// launch). The mask is the library's own state, as its launch count is.
template <auto KERNEL>
cudaError_t gated_configure(int smem) {
  static std::atomic<unsigned long long> done{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = device < 64 ? 1ull << device : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = tcx::configure(KERNEL, smem);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

template <auto KERNEL, typename... Args>
cudaError_t gated_launch(int smem, dim3 grid, int threads, cudaStream_t st, const Args&... args) {
  cudaError_t e = gated_configure<KERNEL>(smem);
  if (e != cudaSuccess) return e;
  e = tcx::launch_pdl(KERNEL, grid, dim3(threads), smem, st, args...);
  count_launches(1);
  return e;
}

// Tensor-core path: bf16 (la_gated_mma.cu, la_gated_mma_bwd.cu)
// The cut of BH sequences of N tokens (each `blocks` CTAs wide) that the costs below, in
// microseconds as measured, make the shortest: CTAs run in waves of `slots`, each for
// `fixed` + `chunk` a chunk of its segment; several segments need the state pass (three
// CTAs an SM, `pass_chunk` a chunk) and the scan (0.1 a segment) first, `pass` in all else.
struct GatedCosts {
  int slots, most;  // resident CTAs; chunks of a segment at most (0: any number)
  float fixed, chunk, pass, pass_chunk;
};
GatedPlan gated_mma_plan(int BH, int N, int blocks, const GatedCosts& k);
GatedPlan gated_mma_forward_plan(int BH, int N, int D, int M);
// each segment's own state from zero and its decay, and (dout not nullptr) its own
// gradient of the incoming state from zero. exact: to float32's digits, for results.
cudaError_t gated_mma_states(const GatedPlan& p, const void* k, const void* v, const void* q,
                             const void* dout, const void* g, int D, int M, const int* lens, int H,
                             bool exact, const GatedWorkspace& w, cudaStream_t st);
cudaError_t gated_mma_forward(const GatedForward& f, const GatedPlan& p, const GatedWorkspace& w,
                              cudaStream_t st);
// The backward, D and M up to 64 in one kernel, over that a kernel for each gradient.
// scratch: bytes behind the plan's states.
GatedPlan gated_mma_backward_plan(int BH, int N);
size_t gated_mma_backward_scratch(const GatedPlan& p);
cudaError_t gated_mma_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                               cudaStream_t st);
GatedPlan gated_mma_wide_plan(int BH, int N, int D, int M);
size_t gated_mma_wide_scratch(const GatedPlan& p, int D, int M);
cudaError_t gated_mma_wide_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                                    cudaStream_t st);

}  // namespace la
