// The gated projections of a few tokens (serving: one of each stream), h = act(x wg^T) (x wu^T).
// Bound by the weights' bytes, which are read once: a CTA takes some rows f of wg and the same of
// wu, its eight warps share their elements, and the sums are joined in shared memory in order, so
// that a and u meet in one thread.
//
// bf16: 8 rows of wg and 8 of wu are the 16 rows of mma.sync's m16n8k16 A, 8 tokens its columns.
// The order of the terms of a sum is free, so a lane loads 16 neighbouring bytes of its two rows
// and takes them as the terms of two products, and the same 16 bytes of its token's x: no
// shared memory, no transposition, every byte of a 64-byte piece of a row used at once.
// Measured, T 1 in bf16: C 4096, F 11008 29.9 us (180 MB, 6.0 TB/s), C 2048, F 5632 10.1 us (46 MB;
// four warps with twice the loads in flight 12.8, sixteen 13.9), C 512, F 1408 2.2 us.
// float32: 2 rows of each matrix and NT tokens are 4 NT sums a lane, which the warp's lanes add up by
// exchanging halves, each lane ending with one of them. C 2048, F 5632: 1 token 14.3 us (92 MB,
// 6.4 TB/s; with one piece in flight 15.7, four 17.8; as 8 tokens 19.3), 4 tokens 18.6, 8 25.7.
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace tcx;
using namespace ffn;

constexpr int kWarps = 8;

struct Args {
  const void *x, *wg, *wu;
  void* h;
  long long x_stride, h_stride;
  int T, C, F;
};

__device__ __forceinline__ uint4 load_once(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// (volatile, so that it stays behind all the loads of its pieces)
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// NT: groups of 8 tokens. U: pieces of 32 terms a warp has in flight.
template <int ACT, int NT, int U>
__global__ void __launch_bounds__(32 * kWarps) ffn_few_kernel(const Args a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int f0 = blockIdx.x * 8, steps = (a.C + 31) / 32;
  const size_t row = (size_t)(f0 + g) * a.C;  // (F is a multiple of 8)
  const __nv_bfloat16 *wg = static_cast<const __nv_bfloat16*>(a.wg) + row, *wu = static_cast<const __nv_bfloat16*>(a.wu) + row;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const __nv_bfloat16* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    x[n] = n * 8 + g < a.T ? static_cast<const __nv_bfloat16*>(a.x) + (n * 8 + g) * a.x_stride : nullptr;
  float d[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
  tc::pdl_wait();
  for (int s0 = warp; s0 < steps; s0 += U * kWarps) {
    uint4 p[U], q[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (s0 + j * kWarps) * 32 + t * 8;
      const bool in = k < a.C;
      p[j] = in ? load_once(wg + k) : none;
      q[j] = in ? load_once(wu + k) : none;
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (s0 + j * kWarps) * 32 + t * 8;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 v = k < a.C && x[n] != nullptr ? __ldg(reinterpret_cast<const uint4*>(x[n] + k)) : none;
        mma16816(d[n], p[j].x, q[j].x, p[j].y, q[j].y, v.x, v.y);
        mma16816(d[n], p[j].z, q[j].z, p[j].w, q[j].w, v.z, v.w);
      }
    }
  }
  __shared__ float4 sums[kWarps][NT][32];
#pragma unroll
  for (int n = 0; n < NT; ++n) sums[warp][n][lane] = make_float4(d[n][0], d[n][1], d[n][2], d[n][3]);
  __syncthreads();
  // a lane has a of tokens 2 t, 2 t + 1 (of its group) and row f0 + g, and u of the same
  for (int n = warp; n < NT; n += kWarps) {
    float4 s = sums[0][n][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = sums[w][n][lane];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const float2 h = mul2(act2<ACT>(make_float2(s.x, s.y)), make_float2(s.z, s.w));
    const int tok = n * 8 + t * 2;
    __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.h) + tok * a.h_stride + f0 + g;
    if (tok < a.T) to[0] = __float2bfloat16_rn(h.x);
    if (tok + 1 < a.T) to[a.h_stride] = __float2bfloat16_rn(h.y);
  }
}

// N values a lane, added over the warp: lane i ends with the sum of value i % N
template <int N>
__device__ __forceinline__ float sums_to_lanes(float (&v)[N]) {
  const int lane = threadIdx.x % 32;
#pragma unroll
  for (int o = 16; o >= N; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  return v[0];
}

// NT: tokens. U: pieces of 128 terms a warp has in flight.
template <int ACT, int NT, int U>
__global__ void __launch_bounds__(32 * kWarps) ffn_few_f32_kernel(const Args a) {
  constexpr int N = 4 * NT;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int f0 = blockIdx.x * 2;
  const float* w[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    w[r] = static_cast<const float*>(r < 2 ? a.wg : a.wu) + (size_t)(f0 + r % 2) * a.C;
  const float* x = static_cast<const float*>(a.x);
  float v[N];  // value r * NT + token
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = 0.f;
  tc::pdl_wait();
  for (int k0 = (warp * 32 + lane) * 4; k0 < a.C; k0 += U * kWarps * 128) {
    uint4 p[U][4];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = k0 + j * kWarps * 128;
        p[j][r] = k < a.C ? load_once(w[r] + k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = k0 + j * kWarps * 128;
      if (k >= a.C) continue;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (n >= a.T) continue;
        const float4 y = __ldg(reinterpret_cast<const float4*>(x + n * a.x_stride + k));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float& s = v[r * NT + n];
          s = fmaf(__uint_as_float(p[j][r].x), y.x, s);
          s = fmaf(__uint_as_float(p[j][r].y), y.y, s);
          s = fmaf(__uint_as_float(p[j][r].z), y.z, s);
          s = fmaf(__uint_as_float(p[j][r].w), y.w, s);
        }
      }
    }
  }
  __shared__ float sums[kWarps][N];
  const float mine = sums_to_lanes(v);
  if (lane < N) sums[warp][lane] = mine;
  __syncthreads();
  if (threadIdx.x < 2 * NT) {  // row f0 + threadIdx.x / NT of both matrices
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) g += sums[i][threadIdx.x], u += sums[i][2 * NT + threadIdx.x];
    const int n = threadIdx.x % NT;
    if (n < a.T)
      static_cast<float*>(a.h)[n * a.h_stride + f0 + threadIdx.x / NT] = act2<ACT>(make_float2(g, 0.f)).x * u;
  }
}

template <int ACT>
cudaError_t launch(const Args& a, int dtype, cudaStream_t st) {
  const dim3 block(32 * kWarps), grid(dtype == LA_F32 ? a.F / 2 : a.F / 8);
  const cudaError_t e = dtype == LA_F32 && a.T == 1   ? launch_pdl(ffn_few_f32_kernel<ACT, 1, 2>, grid, block, 0, st, a)
                        : dtype == LA_F32 && a.T <= 4 ? launch_pdl(ffn_few_f32_kernel<ACT, 4, 2>, grid, block, 0, st, a)
                        : dtype == LA_F32             ? launch_pdl(ffn_few_f32_kernel<ACT, 8, 2>, grid, block, 0, st, a)
                        : a.T <= 8      ? launch_pdl(ffn_few_kernel<ACT, 1, 4>, grid, block, 0, st, a)
                        : a.T <= 16     ? launch_pdl(ffn_few_kernel<ACT, 2, 4>, grid, block, 0, st, a)
                                        : launch_pdl(ffn_few_kernel<ACT, 4, 4>, grid, block, 0, st, a);
  count_launches(1);
  return e;
}

}  // namespace

// bf16: 32 tokens take 15.7 us at C 2048, F 5632 here and 16.0 in tiles of 256 tokens, 64 tokens 38.
// float32: 8 take 26 us, 9 take 100 in tiles.
int ffn_few_tokens(int dtype) { return dtype == LA_F32 ? 8 : 32; }

cudaError_t ffn_few_forward(const FfnGate& f, cudaStream_t st) {
  Args a;
  a.x = f.x;
  a.wg = f.wg;
  a.wu = f.wu;
  a.h = f.h;
  a.x_stride = f.x_stride;
  a.h_stride = f.h_stride;
  a.T = f.T;
  a.C = f.C;
  a.F = f.F;
  return f.act == kSilu   ? launch<kSilu>(a, f.dtype, st)
         : f.act == kGelu ? launch<kGelu>(a, f.dtype, st)
                          : launch<kGeluTanh>(a, f.dtype, st);
}

}  // namespace la
