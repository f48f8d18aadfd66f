// The gates of a 64-token chunk, as the tensor-core kernels use them.
#pragma once

#include "la_gated.cuh"
#include "la_mma.cuh"

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

// From a lane's two gates: G[i], their inclusive sums over the chunk, and W[i], the
// weights of the token's outer product in the chunk's state: 2^(sum of the gates behind
// it), or for the reverse direction 2^(sum up to and including it). Both are the
// warp's own tables. Returns the chunk's sum.
template <bool REV>
__device__ __forceinline__ float chunk_gates(float2 g, float* G, float* W) {
  const int lane = threadIdx.x & 31;
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
  __syncwarp();
  *reinterpret_cast<float2*>(G + 2 * lane) = incl;
  *reinterpret_cast<float2*>(W + 2 * lane) =
      REV ? make_float2(mma::ex2(incl.x), mma::ex2(incl.y))
          : make_float2(mma::ex2(after + g.y), mma::ex2(after));
  __syncwarp();
  return __shfl_sync(0xffffffffu, up, 31);
}

// Tensor-core path: bf16 (la_gated_mma.cu, la_gated_mma_bwd.cu)
GatedPlan gated_mma_plan(int BH, int N, int M, int resident);
GatedPlan gated_mma_forward_plan(int BH, int N, int D, int M);
// each segment's own state from zero and its decay, and (dout not nullptr) its own
// gradient of the incoming state from zero
cudaError_t gated_mma_states(const GatedPlan& p, const void* k, const void* v, const void* q,
                             const void* dout, const void* g, int D, int M, const int* lens, int H,
                             const GatedWorkspace& w, cudaStream_t st);
cudaError_t gated_mma_forward(const GatedForward& f, const GatedWorkspace& w, cudaStream_t st);
bool gated_mma_backward_supported(int D, int M);
GatedPlan gated_mma_backward_plan(int BH, int N);
// bytes of scratch behind the plan's states
size_t gated_mma_backward_scratch(const GatedPlan& p);
cudaError_t gated_mma_backward(const GatedBackward& f, const GatedPlan& p, const GatedWorkspace& w,
                               cudaStream_t st);

}  // namespace la
