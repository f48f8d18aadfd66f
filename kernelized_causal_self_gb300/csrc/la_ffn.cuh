// The gated projections' activations: f = act(a) and its derivative.
//   silu       a s,  s = 1 / (1 + exp(-a));                  f' = s (1 + a (1 - s))
//   gelu       a P(a),  P(a) = erfc(-a / sqrt(2)) / 2;       f' = P + a exp(-a^2 / 2) / sqrt(2 pi)
//   gelu_tanh  a s(z),  z = c (a + 0.044715 a^3), c = 2 sqrt(2 / pi)  ((1 + tanh(y)) / 2 = s(2 y));
//              f' = s + a s (1 - s) z'
#pragma once

#include "la_common.cuh"
#include "la_internal.h"

namespace la {
namespace ffn {

enum Act { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// s = sigmoid(z) and 1 - s. FAST (results in bf16): by __expf, off by 2 + 1.17 |z| steps of
// 2^-23, and a quotient off by 2; past |z| = 87 the smaller one is 0 instead of below 2^-125.
// Otherwise from expf and a rounded quotient. 1 - s cancels nothing: both come from exp(-|z|).
template <bool FAST>
__device__ __forceinline__ void sigmoid(float z, float& s, float& rest) {
  const float e = FAST ? __expf(-fabsf(z)) : expf(-fabsf(z));
  const float large = FAST ? __fdividef(1.f, 1.f + e) : 1.f / (1.f + e);
  const float small = e * large;
  s = z < 0.f ? small : large;
  rest = z < 0.f ? large : small;
}

// P(a) of the gelu and e = exp(-a^2 / 2). FAST: with t = 1 / (1 + 0.375 |a| / sqrt(2)) a polynomial
// of t for erfc(|a| / sqrt(2)) / e, fitted (least squares, reweighted towards the largest error) to
// 6.4e-7 relative for |a| up to 13, past which e is 0: P(a) and 1 - P(a) keep their digits.
template <bool FAST>
__device__ __forceinline__ float normal(float a, float& e) {
  if constexpr (!FAST) {
    e = expf(-0.5f * a * a);
    return 0.5f * erfcf(-0.70710678118654752f * a);
  }
  e = __expf(-0.5f * a * a);
  const float t = __fdividef(1.f, fmaf(0.265165043f, fabsf(a), 1.f));
  float q = -0.06754790f;
  q = fmaf(q, t, 0.19396870f);
  q = fmaf(q, t, -0.06479833f);
  q = fmaf(q, t, 0.14153051f);
  q = fmaf(q, t, 0.08333239f);
  q = fmaf(q, t, 0.10784457f);
  q = fmaf(q, t, 0.10566973f);
  const float tail = q * t * e;  // of |a|
  return a < 0.f ? tail : 1.f - tail;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float act(float a) {
  if constexpr (ACT == kGelu) {
    float e;
    return a * normal<FAST>(a, e);
  }
  float z = a;
  if constexpr (ACT == kGeluTanh) z = 1.5957691216057308f * a * fmaf(0.044715f * a, a, 1.f);
  if constexpr (FAST) return a * __fdividef(1.f, 1.f + __expf(-z));  // (0 once exp(-z) is infinite)
  float s, rest;
  sigmoid<FAST>(z, s, rest);
  return a * s;
}

template <int ACT, bool FAST>
__device__ __forceinline__ void act_grad(float a, float& f, float& df) {
  if constexpr (ACT == kGelu) {
    float e;
    const float p = normal<FAST>(a, e);
    f = a * p;
    df = fmaf(0.3989422804014327f * a, e, p);
    return;
  }
  float z = a, dz = 1.f, s, rest;
  if constexpr (ACT == kGeluTanh) {
    const float q = 0.044715f * a * a;
    z = 1.5957691216057308f * a * (1.f + q);
    dz = 1.5957691216057308f * fmaf(3.f, q, 1.f);
  }
  sigmoid<FAST>(z, s, rest);
  f = a * s;
  df = s * fmaf(a * dz, rest, 1.f);
}

}  // namespace ffn

// out (and out2 with count 2): the sums over `splits` parts of partial [count][splits][rows][C],
// added in order
cudaError_t ffn_join(const float* partial, void* out, void* out2, long long out_stride, int rows, int count, int C,
                     int splits, int dtype, cudaStream_t st);
// dact [2][T][F]: da = dh u act'(a), du = dh act(a), a and u from f's checkpoint
cudaError_t ffn_kept_grads(const FfnGate& f, void* dact, cudaStream_t st);

}  // namespace la
