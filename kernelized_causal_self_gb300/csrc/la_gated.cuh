// Shared pieces of the gated recurrence's kernels: how a sequence is cut into
// segments, where its states live in the workspace and in the caller's pool.
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   out_t = S_t^T q_t
//
// The recurrence is linear in the state, so a segment of tokens acts on the state
// it receives as S -> decay * S + U with decay = exp(sum of its g) and U the state
// it builds from zero. With few sequences the segments' U are formed in parallel
// (the state pass), joined in order by a scan over the segments, and the outputs
// then computed for all segments at once.
#pragma once

#include "la_common.cuh"
#include "la_internal.h"

namespace la {

// How the N tokens of each of BH sequences are cut: segment s holds tokens
// [s * len, (s + 1) * len).
struct GatedPlan {
  int BH, N, len, n_seg;
};

// Workspace: header | decay [BH][n_seg] | S [BH][n_seg + 1][D][M] and, for the
// backward, E [BH][n_seg + 1][D][M] | dots of q with dq, of k with
// dk, and the segments' ends (the decay's gradient is made of them; on the tensor-core
// path one scratch area in their place).
// S[.][s] is the state segment s receives (n_seg: the final one), E[.][s] the
// loss's gradient with respect to it.
struct GatedWorkspace {
  WorkspaceHeader* hdr;
  float *decay, *S, *E, *dot_q, *dot_k, *ends;
  void* scratch;
  size_t bytes;
};

// The state entry of sequence bh: bh itself, or its stream's pool entry; -1 for a
// slot outside the pool.
struct GatedEntries {
  const int* slots = nullptr;
  int pool = 0, H = 1;
  __device__ long long at(int bh) const {
    if (slots == nullptr) return bh;
    const int s = slots[bh / H];
    return s >= 0 && s < pool ? (long long)s * H + bh % H : -1;
  }
};

// exp(g) to half a step (2^-25) where it is close to 1: a slow gate multiplies the
// state thousands of times, and a few-ulp bias of each factor would grow with them.
__device__ __forceinline__ float gated_decay(float g) {
  return g > -0.5f && g < 0.5f ? 1.f + expm1f(g) : expf(g);
}

__device__ __forceinline__ int gated_length(const int* lens, int H, int bh, int N) {
  return lens ? max(0, min(lens[bh / H], N)) : N;
}

// The scan over the segments: of the states, from S0 to S (nullptr: zero, not wanted),
// and with `back` of the gradients too, from dS to dS0.
struct GatedGradients {
  const float* dS;
  float* dS0;
};
cudaError_t gated_scan(const GatedPlan& p, const GatedWorkspace& w, const float* S0, float* S,
                       const GatedEntries& e, int DM, cudaStream_t st,
                       const GatedGradients* back = nullptr);

}  // namespace la
