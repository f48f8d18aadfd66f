// Activations put away in 8 bits (see la_checkpoint.cuh) and taken back.
//
// Bound by memory: a bf16 value costs 2 bytes on one side and 1 + 1/32 on the other. A thread
// has 16 bytes of a row at a time, so the 32 / V neighbouring lanes of a block find its largest
// magnitude by shuffles, and keeps kEach of them in flight. A row's pieces are counted up to
// whole blocks, so that a block never straddles lanes of two groups.
#include "la_checkpoint.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int kThreads = 256, kEach = 4;

struct Pieces {
  long long rows, x_stride;
  unsigned C, padded, n_blocks;  // padded: pieces of a row, up to whole blocks
};

template <typename T, bool PACK>
__global__ void __launch_bounds__(kThreads)
checkpoint_kernel(T* x, signed char* codes, unsigned char* exps, const Pieces p) {
  constexpr int V = 16 / sizeof(T), LANES = q8::kBlock / V;
  using Code = typename q8::Codes<V>::type;
  // the CTA's first piece: one 64-bit division, the rest are small
  const unsigned long long first = (unsigned long long)blockIdx.x * (kThreads * kEach);
  const long long row0 = (long long)(first / p.padded);
  const unsigned at0 = (unsigned)(first % p.padded) + threadIdx.x;
  tc::pdl_wait();
  long long row[kEach];
  unsigned piece[kEach];
  bool in[kEach];
  uint4 raw[kEach];
  Code code[kEach];
  uint32_t e[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const unsigned at = at0 + j * kThreads;
    row[j] = row0 + at / p.padded;
    piece[j] = at % p.padded;
    in[j] = row[j] < p.rows && piece[j] * V < p.C;
    const size_t c = (size_t)row[j] * p.C + piece[j] * V;
    if (PACK) {
      raw[j] = in[j] ? __ldcs(reinterpret_cast<const uint4*>(x + row[j] * p.x_stride + piece[j] * V))
                     : make_uint4(0, 0, 0, 0);
    } else if (in[j]) {
      code[j] = __ldcs(reinterpret_cast<const Code*>(codes + c));
      e[j] = exps[(size_t)row[j] * p.n_blocks + piece[j] / LANES];
    }
  }
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    float v[V];
    if (PACK) {
      const T* t = reinterpret_cast<const T*>(&raw[j]);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = to_f32<T>(t[i]);
      const uint32_t b = q8::step_of(q8::block_top<V>(v));
      if (!in[j]) continue;
      *reinterpret_cast<Code*>(codes + (size_t)row[j] * p.C + piece[j] * V) =
          q8::codes_of<V>(v, q8::inverse_step(b), b);
      if (piece[j] % LANES == 0)
        exps[(size_t)row[j] * p.n_blocks + piece[j] / LANES] = (unsigned char)b;
    } else if (in[j]) {
      q8::values_of<V>(code[j], q8::step_value(e[j]), v);
      uint4 u;
      T* t = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint4*>(x + row[j] * p.x_stride + piece[j] * V) = u;
    }
  }
}

template <typename T, bool PACK>
cudaError_t launch(const Checkpoint& c, cudaStream_t st) {
  constexpr unsigned V = 16 / sizeof(T), LANES = q8::kBlock / V;
  Pieces p;
  p.rows = c.rows;
  p.x_stride = c.x_stride;
  p.C = (unsigned)c.C;
  p.n_blocks = (unsigned)q8::blocks_of(c.C);
  p.padded = p.n_blocks * LANES;
  const unsigned long long all = (unsigned long long)c.rows * p.padded;
  const unsigned long long ctas = (all + kThreads * kEach - 1) / (kThreads * kEach);
  if (ctas > 0x7fffffffULL) return cudaErrorInvalidValue;
  const cudaError_t e = tcx::launch_pdl(checkpoint_kernel<T, PACK>, dim3((unsigned)ctas), dim3(kThreads),
                                        0, st, static_cast<T*>(c.x), c.codes, c.exps, p);
  count_launches(1);
  return e;
}

}  // namespace

cudaError_t checkpoint_pack(const Checkpoint& c, cudaStream_t st) {
  return c.dtype == LA_F32 ? launch<float, true>(c, st) : launch<__nv_bfloat16, true>(c, st);
}

cudaError_t checkpoint_restore(const Checkpoint& c, cudaStream_t st) {
  return c.dtype == LA_F32 ? launch<float, false>(c, st) : launch<__nv_bfloat16, false>(c, st);
}

}  // namespace la
