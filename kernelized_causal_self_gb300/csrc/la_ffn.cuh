// The gated projections' activations: f = act(a) and its derivative.
//   silu       a s,  s = 1 / (1 + exp(-a));                  f' = s (1 + a (1 - s))
//   gelu       a P(a),  P(a) = erfc(-a / sqrt(2)) / 2;       f' = P + a exp(-a^2 / 2) / sqrt(2 pi)
//   gelu_tanh  a s(z),  z = c (a + 0.044715 a^3), c = 2 sqrt(2 / pi)  ((1 + tanh(y)) / 2 = s(2 y));
//              f' = s + a s (1 - s) z'
#pragma once

#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace ffn {

enum Act { kSilu = 0, kGelu = 1, kGeluTanh = 2 };

// Two neighbours at once in packed float32 arithmetic, with the hardware's base-2 exponential
// and reciprocal, each off by 2 steps of 2^-23 at most, results below 2^-126 zero. An exponential's
// argument y is rounded, by |y| 2^-24: where s is small, at y = 20, it is off by 2^-19 of itself,
// and by less than 2^-22 of the largest s, as a sum that is off by 2^-22 makes of it.
__device__ __forceinline__ float2 ex2(float2 x) {
  float2 y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}
__device__ __forceinline__ float2 rcp(float2 x) {
  float2 y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(x.y));
  return y;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// s = 1 / (1 + 2^y), y = -z log2(e): 0 once 2^y is infinite
__device__ __forceinline__ float2 sigmoid2(float2 y) { return rcp(tcx::add2(ex2(y), both(1.f))); }

// y of the gelu_tanh's sigmoid, and q = 0.044715 a^2, of a within +-16, where s is 0 or 1
__device__ __forceinline__ float2 tanh_arg(float2 a, float2& q) {
  a = make_float2(fminf(fmaxf(a.x, -16.f), 16.f), fminf(fmaxf(a.y, -16.f), 16.f));
  q = tcx::mul2(tcx::mul2(a, both(0.044715f)), a);
  return tcx::mul2(tcx::mul2(a, both(-2.302208198f)), tcx::add2(q, both(1.f)));
}

// P(a) and e = exp(-a^2 / 2). With t = 1 / (1 + 0.33 |a| / sqrt(2)), a polynomial of t for
// erfc(|a| / sqrt(2)) / e, fitted (least squares, reweighted towards the largest error) to 9.1e-8
// relative for |a| up to 13, past which e is 0. The smaller of P(a) and 1 - P(a) is off by 4.5e-7 of
// itself for |a| up to 1 and by about a^2 2^-24 from 3 on (1.4e-6 at 5, 7.8e-6 at 13): the exponential's
// argument, a^2 / 2 log2(e), is rounded twice and its constant once. Of 1, all of it is 2^-22 at most.
__device__ __forceinline__ float2 normal2(float2 a, float2& e) {
  using namespace tcx;
  e = ex2(mul2(mul2(a, both(-0.72134752f)), a));
  const float2 t = rcp(fma2(make_float2(fabsf(a.x), fabsf(a.y)), both(0.233345238f), both(1.f)));
  float2 q = both(-0.0679643825f);
  q = fma2(q, t, both(0.231344029f));
  q = fma2(q, t, both(-0.17771931f));
  q = fma2(q, t, both(0.20627065f));
  q = fma2(q, t, both(0.0225054026f));
  q = fma2(q, t, both(0.100961886f));
  q = fma2(q, t, both(0.0914186239f));
  q = fma2(q, t, both(0.0931830555f));
  const float2 tail = mul2(mul2(q, t), e);  // of |a|
  const float2 rest = sub2(both(1.f), tail);
  return make_float2(a.x < 0.f ? tail.x : rest.x, a.y < 0.f ? tail.y : rest.y);
}

template <int ACT>
__device__ __forceinline__ float2 act2(float2 a) {
  float2 q;
  if constexpr (ACT == kGelu) return tcx::mul2(a, normal2(a, q));
  if constexpr (ACT == kGeluTanh) return tcx::mul2(a, sigmoid2(tanh_arg(a, q)));
  return tcx::mul2(a, sigmoid2(tcx::mul2(a, both(-1.44269504f))));
}

// (1 - s is a difference here, off by 2^-24 and 0 where s is 1)
template <int ACT>
__device__ __forceinline__ void act_grad2(float2 a, float2& f, float2& df) {
  using namespace tcx;
  float2 q;
  if constexpr (ACT == kGelu) {
    const float2 p = normal2(a, q);
    f = mul2(a, p);
    df = fma2(mul2(a, both(0.39894228f)), q, p);
  } else if constexpr (ACT == kGeluTanh) {
    const float2 s = sigmoid2(tanh_arg(a, q));
    f = mul2(a, s);
    const float2 dz = fma2(q, both(4.787307365f), both(1.595769122f));
    df = fma2(mul2(f, sub2(both(1.f), s)), dz, s);  // (f dz alone is past float32 from f = 6e36 on)
  } else {
    const float2 s = sigmoid2(mul2(a, both(-1.44269504f)));
    f = mul2(a, s);
    df = fma2(f, sub2(both(1.f), s), s);
  }
}

// The next of a float32's three bf16 parts, for two neighbours, which keep the rest: its top 16 bits,
// then what is left rounded, twice (each rest is exact). Cut, not rounded, at first, so that the
// largest values stay finite.
__device__ __forceinline__ uint32_t take_part(float& x, float& y, int part) {
  const uint32_t u = part == 0 ? __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632) : tc::pack_bf16(x, y);
  x -= tcx::bf16_lo_f(u);
  y -= tcx::bf16_hi_f(u);
  return u;
}

}  // namespace ffn

// A matrix `to` of `rows` rows `stride` apart: the sums over `splits` parts of from
// [splits][rows][C], added in order; `n` of them, of C columns each, at once
struct Join {
  const float* from;
  void* to;
  long long stride;
  int rows, splits;
};
cudaError_t ffn_join(const Join* j, int n, int C, int dtype, cudaStream_t st);
// dact: da = dh u act'(a), du = dh act(a), a and u from f's checkpoint; in bf16 [2][T][F], in float32
// as their three bf16 parts, [2][3][T][F]
cudaError_t ffn_kept_grads(const FfnGate& f, void* dact, cudaStream_t st);

}  // namespace la
