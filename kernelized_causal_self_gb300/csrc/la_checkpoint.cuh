// Activations in 8 bits: whole numbers of -127 .. 127 and, for each block of 32 neighbours of a
// row, a step that is a power of two: 2^(e - 127) for the block's byte e. The step is the
// smallest, from e = 1 on, for which the block's largest magnitude rounds to 127 or less, so a
// value is off by half a step at most, 1/127.5 of that magnitude (and 2^-127). Powers of two make
// every scaling exact: what is stored does not depend on the order or the type of the
// arithmetic. A block that holds an infinity or a NaN gets e = 255, which restores as NaN.
//
// From 63.75 2^122 on a magnitude is 64 steps of 2^122, and 2^128 is no float32: what a code stands
// for is bounded by the largest bf16, 2^128 - 2^120, which is closer than 2^120 to all of those
// values (so finite values restore finite, in both types as the same).
#pragma once

#include "la_common.cuh"

namespace la {
namespace q8 {

constexpr int kBlock = 32;  // values that share a step

__host__ __device__ inline int blocks_of(int n) { return (n + kBlock - 1) / kBlock; }

// The byte of a block, from the bits of its largest magnitude. 2^E of that magnitude is 64 steps,
// and from 127.5 / 64 of it on (a mantissa of 0x7F0000 or more) 32.
__device__ __forceinline__ uint32_t step_of(uint32_t top) {
  const int e = (int)((top + 0x10000u) >> 23) - 6;
  return top >= 0x7F800000u ? 255u : (uint32_t)max(e, 1);
}

// the largest magnitude of three, NaN if one is (whose bits are above infinity's)
__device__ __forceinline__ float top3(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// one over the step (any finite number for e = 255, whose codes are masked)
__device__ __forceinline__ float inverse_step(uint32_t e) {
  return __uint_as_float((e == 255u ? 127u : 254u - e) << 23);
}

__device__ __forceinline__ float step_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7FFFFFFFu : e << 23);
}

// round(x / step), ties to even, in the low byte: adding 1.5 2^23 leaves the whole number there
__device__ __forceinline__ uint32_t code_of(float x, float inverse) {
  return __float_as_uint(fmaf(x, inverse, 12582912.f));
}

__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// four codes of a block with byte e
__device__ __forceinline__ uint32_t codes4(const float* x, float inverse, uint32_t e) {
  const uint32_t c = pack4(code_of(x[0], inverse), code_of(x[1], inverse), code_of(x[2], inverse),
                           code_of(x[3], inverse));
  return e == 255u ? 0u : c;
}

// (the smaller magnitude of the two with the product's sign, NaN if the step is)
__device__ __forceinline__ float value_of(uint32_t codes, int i, float step) {
  float v;
  asm("min.NaN.xorsign.abs.f32 %0, %1, %2;"
      : "=f"(v)
      : "f"((float)(signed char)(codes >> (8 * i)) * step), "f"(__uint_as_float(0x7F7F0000u)));
  return v;
}

// Codes of V neighbours that a thread holds, as bytes in memory
template <int V> struct Codes;
template <> struct Codes<4> { using type = uint32_t; };
template <> struct Codes<8> { using type = uint2; };

template <int V>
__device__ __forceinline__ typename Codes<V>::type codes_of(const float* x, float inverse, uint32_t e) {
  if constexpr (V == 4)
    return codes4(x, inverse, e);
  else
    return make_uint2(codes4(x, inverse, e), codes4(x + 4, inverse, e));
}

template <int V>
__device__ __forceinline__ void values_of(const typename Codes<V>::type& c, float step, float* x) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (V == 4)
      x[i] = value_of(c, i, step);
    else
      x[i] = value_of(i < 4 ? c.x : c.y, i % 4, step);
  }
}

// The largest magnitude's bits over the 32 / V neighbouring lanes that hold a block
template <int V>
__device__ __forceinline__ uint32_t block_top(const float* x) {
  float most = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i + 1 < V; i += 2) most = top3(most, x[i], x[i + 1]);
  uint32_t top = __float_as_uint(top3(most, x[V - 1], x[V - 1]));
#pragma unroll
  for (int o = kBlock / V / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  return top;
}

}  // namespace q8
}  // namespace la
