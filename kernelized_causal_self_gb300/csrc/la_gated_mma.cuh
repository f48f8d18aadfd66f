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

// From a lane's two gates, tables of the chunk (made by one warp for all):
//   G[i]  the gates' sums up to and including token i
//   W[i]  2^(sum of those behind i), what is left of i's outer product in the state after
//         the chunk; and with REV V[i] = 2^G[i]. The one of the two that weights operands
//         (V with REV, else W) is kept as split_pair's in X, or if EXACT as float32.
//   decay of the whole chunk; its sum is returned
struct GateTables {
  float G[mma::kC], W[mma::kC], X[mma::kC], decay, pad[3];
};
template <bool REV, bool EXACT>
__device__ __forceinline__ float chunk_gates(ushort2 raw, GateTables& t) {
  const int lane = threadIdx.x & 31;
  const float2 g = gates_of(raw);
  const float both = g.x + g.y;
  float up = both, down = both;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float u = __shfl_up_sync(0xffffffffu, up, o);
    const float d = __shfl_down_sync(0xffffffffu, down, o);
    if (lane >= o) up += u;
    if (lane + o < 32) down += d;
  }
  float before = __shfl_up_sync(0xffffffffu, up, 1);
  float after = __shfl_down_sync(0xffffffffu, down, 1);
  if (lane == 0) before = 0.f;
  if (lane == 31) after = 0.f;
  const float2 incl = make_float2(before + g.x, up);
  const float2 left = make_float2(mma::ex2(after + g.y), mma::ex2(after));
  const float2 w = REV ? make_float2(mma::ex2(incl.x), mma::ex2(incl.y)) : left;
  reinterpret_cast<float2*>(t.G)[lane] = incl;
  reinterpret_cast<float2*>(t.W)[lane] = left;
  if (EXACT)
    reinterpret_cast<float2*>(t.X)[lane] = w;
  else
    reinterpret_cast<uint2*>(t.X)[lane] = mma::split_pair(w);
  const float total = __shfl_sync(0xffffffffu, up, 31);
  if (lane == 0) t.decay = gated_decay(total * kLn2);
  return total;
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

// FINE: two bf16 terms, not one, for what is multiplied by an input's rows and is not an
// input itself: the products * L, and the states. For calls of so few chunks (`blocks` CTAs
// wide) that each has a multiprocessor to itself, where it takes 3 to 17% longer (D = M = 64:
// forward of 16 heads and 64 tokens 4.2 us for 3.8, of 512 tokens 19 for 17; backward 6.6
// for 5.9 and 14.8 for 13.9), less than the host takes to issue the call. Their errors are
// averages over few values: with one term dg of 4 heads and 20 to 128 tokens was off by up to
// 2.9 times bf16's own rounding (2-norm; typically 1.5) and the other outputs by 1.4 times
// it, with two all by 1.00.
inline bool gated_fine(int blocks, int N) {
  return (long long)blocks * ((N + mma::kC - 1) / mma::kC) <= 152;
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
