// What the gated projections' backward passes need beside their products: da = dh u act'(a) and
// du = dh act(a) from a checkpoint of a and u (rounded to bf16 once in bf16, as in la_ffn_tc.cu, three
// parts in float32), and the parts of cut sums added in order. Both are bound by memory.
#include "la_checkpoint.cuh"
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace tcx;
using namespace ffn;

// 4 neighbours as float32
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16_lo_f(u.x), bf16_hi_f(u.x), bf16_lo_f(u.y), bf16_hi_f(u.y));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(tc::pack_bf16(v.x, v.y), tc::pack_bf16(v.z, v.w));
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]),
                                            tc::pack_bf16(v[4], v[5]), tc::pack_bf16(v[6], v[7]));
}

struct Joins {
  Join j[3];
};

// Matrix blockIdx.y, EACH times 4 neighbours a thread. Eight loads are in flight together, of two parts
// (EACH 4) or, where that would leave SMs idle, of eight: C 512, F 1408 4.1 us and not 7.0; 16 parts of
// 32 x 480 3.2 and not 5.8.
template <typename T, int EACH>
__global__ void __launch_bounds__(256) ffn_join_kernel(const __grid_constant__ Joins all, int C) {
  const Join& m = all.j[blockIdx.y];
  const unsigned per = C / 4;
  const size_t n = (size_t)m.rows * per, plane = n * 4;
  const size_t at = (size_t)blockIdx.x * (256 * EACH) + threadIdx.x;
  if (at >= n) return;
  const size_t row0 = at / per;  // (one 64-bit division a thread)
  const unsigned c0 = (unsigned)(at - row0 * per);
  size_t from[EACH];  // (past the end the first again, which is not stored)
#pragma unroll
  for (int j = 0; j < EACH; ++j) from[j] = at + j * 256 < n ? j * 1024 : 0;
  pdl_wait();
  const float* p = m.from + at * 4;
  float4 s[EACH];
#pragma unroll
  for (int j = 0; j < EACH; ++j) s[j] = __ldcs(reinterpret_cast<const float4*>(p + from[j]));
  constexpr int K = 8 / EACH;
  for (int k = 1; k < m.splits; k += K) {
    float4 v[K][EACH];
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (k + i >= m.splits) continue;
#pragma unroll
      for (int j = 0; j < EACH; ++j) v[i][j] = __ldcs(reinterpret_cast<const float4*>(p + (k + i) * plane + from[j]));
    }
#pragma unroll
    for (int i = 0; i < K; ++i) {
      if (k + i >= m.splits) continue;
#pragma unroll
      for (int j = 0; j < EACH; ++j) s[j].x += v[i][j].x, s[j].y += v[i][j].y, s[j].z += v[i][j].z, s[j].w += v[i][j].w;
    }
  }
#pragma unroll
  for (int j = 0; j < EACH; ++j) {
    if (at + j * 256 >= n) continue;
    const unsigned i = c0 + j * 256;
    store4(static_cast<T*>(m.to) + (long long)(row0 + i / per) * m.stride + i % per * 4, s[j]);
  }
}

// da, du from a checkpoint of a and u: 8 neighbours a thread, all of a block's step. Bound by
// memory (T 4096, F 5632 in bf16: 186 MB).
struct Kept {
  const void* dh;
  const signed char* codes;
  const unsigned char* exps;
  __nv_bfloat16* dact;
  long long dh_stride;
  int T, F;
};

template <typename T, int ACT>
__global__ void __launch_bounds__(256) ffn_kept_grads_kernel(const Kept a) {
  const unsigned per = a.F / 8, nb = q8::blocks_of(a.F);
  const size_t part = (size_t)a.T * a.F;
  tc::pdl_wait();
  const unsigned long long at = (unsigned long long)blockIdx.x * 256;  // (one 64-bit division a CTA)
  const unsigned i = (unsigned)(at % per) + threadIdx.x;
  const size_t t = at / per + i / per;
  if (t >= a.T) return;
  const unsigned f = i % per * 8;
  const size_t row = 2 * t;
  const T* dh = static_cast<const T*>(a.dh) + (long long)t * a.dh_stride + f;
  const uint2 ca = __ldcs(reinterpret_cast<const uint2*>(a.codes + row * a.F + f));
  const uint2 cu = __ldcs(reinterpret_cast<const uint2*>(a.codes + (row + 1) * a.F + f));
  const float4 d0 = load4(dh), d1 = load4(dh + 4);
  float g[8], u[8];
  q8::values_of<8>(ca, q8::step_value(a.exps[row * nb + f / q8::kBlock]), g);
  q8::values_of<8>(cu, q8::step_value(a.exps[(row + 1) * nb + f / q8::kBlock]), u);
  const float dv[8] = {d0.x, d0.y, d0.z, d0.w, d1.x, d1.y, d1.z, d1.w};
  float da[8], du[8];
#pragma unroll
  for (int j = 0; j < 8; j += 2) {
    float2 fa, df;
    act_grad2<ACT>(make_float2(g[j], g[j + 1]), fa, df);
    da[j] = dv[j] * u[j] * df.x, da[j + 1] = dv[j + 1] * u[j + 1] * df.y;
    du[j] = dv[j] * fa.x, du[j + 1] = dv[j + 1] * fa.y;
  }
  __nv_bfloat16* to = a.dact + t * a.F + f;
  if constexpr (sizeof(T) == 2) {
    store8(to, da);
    store8(to + part, du);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        float* v = i ? du : da;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = take_part(v[2 * j], v[2 * j + 1], p);
        *reinterpret_cast<uint4*>(to + (i * 3 + p) * part) = make_uint4(o[0], o[1], o[2], o[3]);
      }
  }
}

template <typename T>
cudaError_t kept_grads(const Kept& a, int act, cudaStream_t st) {
  const dim3 grid((unsigned)(((long long)a.T * (a.F / 8) + 255) / 256));  // (T <= 2^24, F <= 2^16: an int)
  const cudaError_t e =
      act == kSilu   ? launch_pdl(ffn_kept_grads_kernel<T, kSilu>, grid, dim3(256), 0, st, a)
      : act == kGelu ? launch_pdl(ffn_kept_grads_kernel<T, kGelu>, grid, dim3(256), 0, st, a)
                     : launch_pdl(ffn_kept_grads_kernel<T, kGeluTanh>, grid, dim3(256), 0, st, a);
  count_launches(1);
  return e;
}

template <typename T>
cudaError_t join(const Joins& all, int n, long long rows, int C, cudaStream_t st) {
  const long long blocks = (rows * (C / 4) + 1023) / 1024;  // (rows <= 2^24, C <= 2^16: an int)
  return blocks * n >= sm_count() ? launch_pdl(ffn_join_kernel<T, 4>, dim3((unsigned)blocks, n), dim3(256), 0, st, all, C)
                                      : launch_pdl(ffn_join_kernel<T, 1>, dim3((unsigned)blocks * 4, n), dim3(256), 0, st, all, C);
}

}  // namespace

cudaError_t ffn_join(const Join* j, int n, int C, int dtype, cudaStream_t st) {
  Joins all{};
  long long most = 0;
  for (int i = 0; i < n; ++i) {
    all.j[i] = j[i];
    if (j[i].rows > most) most = j[i].rows;
  }
  const cudaError_t e = dtype == LA_F32 ? join<float>(all, n, most, C, st) : join<__nv_bfloat16>(all, n, most, C, st);
  count_launches(1);
  return e;
}

cudaError_t ffn_kept_grads(const FfnGate& f, void* dact, cudaStream_t st) {
  const Kept a{f.dh, f.codes, f.exps, static_cast<__nv_bfloat16*>(dact), f.dh_stride, f.T, f.F};
  return f.dtype == LA_F32 ? kept_grads<float>(a, f.act, st) : kept_grads<__nv_bfloat16>(a, f.act, st);
}

}  // namespace la
