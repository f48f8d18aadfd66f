// Activations put away in 8 bits (see la_checkpoint.cuh) and taken back.
//
// Bound by memory: a bf16 value costs 2 bytes on one side and 1 + 1/32 on the other. A thread
// has 16 bytes of a row at a time, so the 32 / V neighbouring lanes of a block find its largest
// magnitude by shuffles, and keeps kEach of them in flight. A row's pieces are counted up to
// whole blocks, so that a block never straddles lanes of two groups; where rows are whole blocks
// one behind another (FLAT) they are not told apart. 65536 x 512 in bf16: 17.2 us (102 MB, 5.9 TB/s; with
// divisions 19.5), restored in 10.6.
#include "la_checkpoint.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int kThreads = 256, kEach = 4;

struct Pieces {
  long long rows, x_stride;
  unsigned long long all;        // pieces in all
  unsigned C, padded, n_blocks;  // padded: pieces of a row, up to whole blocks
};

template <typename T, bool PACK, bool FLAT>
__global__ void __launch_bounds__(kThreads)
checkpoint_kernel(T* x, signed char* codes, unsigned char* exps, const Pieces p) {
  constexpr int V = 16 / sizeof(T), LANES = q8::kBlock / V;
  using Code = typename q8::Codes<V>::type;
  const unsigned long long first = (unsigned long long)blockIdx.x * (kThreads * kEach);
  // the CTA's first row: one 64-bit division, the rest are small
  const long long row0 = FLAT ? 0 : (long long)(first / p.padded);
  const unsigned at0 = FLAT ? 0 : (unsigned)(first % p.padded) + threadIdx.x;
  tc::pdl_wait();
  long long xat[kEach];   // of x, of the codes, of the block's byte
  size_t cat[kEach], eat[kEach];
  bool in[kEach];
  uint4 raw[kEach];
  Code code[kEach];
  uint32_t e[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (FLAT) {
      const unsigned long long piece = first + j * kThreads + threadIdx.x;
      in[j] = piece < p.all;
      cat[j] = piece * V;
      xat[j] = (long long)cat[j];
      eat[j] = piece / LANES;
    } else {
      const unsigned at = at0 + j * kThreads, piece = at % p.padded;
      const long long row = row0 + at / p.padded;
      in[j] = row < p.rows && piece * V < p.C;
      xat[j] = row * p.x_stride + piece * V;
      cat[j] = (size_t)row * p.C + piece * V;
      eat[j] = (size_t)row * p.n_blocks + piece / LANES;
    }
    if (PACK) {
      raw[j] = in[j] ? __ldcs(reinterpret_cast<const uint4*>(x + xat[j])) : make_uint4(0, 0, 0, 0);
    } else if (in[j]) {
      code[j] = __ldcs(reinterpret_cast<const Code*>(codes + cat[j]));
      e[j] = exps[eat[j]];
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
      *reinterpret_cast<Code*>(codes + cat[j]) = q8::codes_of<V>(v, q8::inverse_step(b), b);
      if (threadIdx.x % LANES == 0) exps[eat[j]] = (unsigned char)b;
    } else if (in[j]) {
      q8::values_of<V>(code[j], q8::step_value(e[j]), v);
      uint4 u;
      T* t = reinterpret_cast<T*>(&u);
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = from_f32<T>(v[i]);
      *reinterpret_cast<uint4*>(x + xat[j]) = u;
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
  p.all = (unsigned long long)c.rows * p.padded;
  const unsigned long long ctas = (p.all + kThreads * kEach - 1) / (kThreads * kEach);
  if (ctas > 0x7fffffffULL) return cudaErrorInvalidValue;
  const bool flat = c.C % q8::kBlock == 0 && (c.x_stride == c.C || c.rows == 1);
  const cudaError_t e =
      flat ? tcx::launch_pdl(checkpoint_kernel<T, PACK, true>, dim3((unsigned)ctas), dim3(kThreads), 0, st,
                             static_cast<T*>(c.x), c.codes, c.exps, p)
           : tcx::launch_pdl(checkpoint_kernel<T, PACK, false>, dim3((unsigned)ctas), dim3(kThreads), 0, st,
                             static_cast<T*>(c.x), c.codes, c.exps, p);
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
