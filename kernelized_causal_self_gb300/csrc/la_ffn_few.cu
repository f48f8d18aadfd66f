// The gated projections of a few tokens (serving: one of each stream), h = act(x wg^T) (x wu^T), and
// da, du of the backward pass from the same products (in bf16 rounded to it once, as in la_ffn_tc.cu).
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
// Groups of 32 tokens are CTAs of their own, whose weights come from L2.
// float32: one token on the CUDA cores, 2 rows of each matrix a CTA: C 2048, F 5632 14.5 us (92 MB, 6.4
// TB/s; one piece in flight 15.7, four 17.8). From two on as in bf16, with each value as three bf16
// parts and six products of them (la_ffn_tc32.cu), cut up in registers, 16 bytes of a row one product;
// the largest products' sums are taken out every 32 terms, and the others', 2^-8 of them, kept apart.
// The next pieces are asked for before one is used: 8, 16 and 32 tokens 19.7, 26.3, 36.1 us (all loads
// first 21.3, 30.9, 41.5), 64 67, which mma.sync's rate then bounds; on the CUDA cores 8 took 25.7.
// (Parts of an infinity are an infinity and NaN: only the CUDA cores' one token gives infinities.)
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace tcx;
using namespace ffn;

constexpr int kWarps = 8;

struct Args {
  const void *x, *wg, *wu, *dh;
  void* out;  // h, or da and du: [2][T][F], in float32 their parts, [2][3][T][F]
  long long x_stride, out_stride, dh_stride;
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

// Lane 4 g + t has in s what is a of tokens tok, tok + 1 and row f, and u of the same
template <typename T, int ACT, bool GRADS>
__device__ __forceinline__ void finish(const Args& a, float4 s, int tok, int f) {
  if constexpr (!GRADS) {
    const float2 h = mul2(act2<ACT>(make_float2(s.x, s.y)), make_float2(s.z, s.w));
    T* to = static_cast<T*>(a.out) + tok * a.out_stride + f;
    if (tok < a.T) to[0] = from_f32<T>(h.x);
    if (tok + 1 < a.T) to[a.out_stride] = from_f32<T>(h.y);
  } else {
    float2 fa, df;
    act_grad2<ACT>(make_float2(s.x, s.y), fa, df);
    const size_t plane = (size_t)a.T * a.F;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (tok + i >= a.T) continue;
      const float dh = to_f32(static_cast<const T*>(a.dh)[(tok + i) * a.dh_stride + f]);
      float da = dh * (i ? s.w : s.z) * (i ? df.y : df.x), du = dh * (i ? fa.y : fa.x);
      __nv_bfloat16* to = static_cast<__nv_bfloat16*>(a.out) + (size_t)(tok + i) * a.F + f;
      constexpr int P = sizeof(T) == 2 ? 1 : 3;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t u = P == 1 ? tc::pack_bf16(da, du) : take_part(da, du, p);
        to[p * plane] = __ushort_as_bfloat16((unsigned short)u);
        to[(P + p) * plane] = __ushort_as_bfloat16((unsigned short)(u >> 16));
      }
    }
  }
}

// NT: groups of 8 tokens. U: pieces of 32 terms a warp has in flight.
template <int ACT, bool GRADS, int NT, int U>
__global__ void __launch_bounds__(32 * kWarps) ffn_few_kernel(const Args a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int f0 = blockIdx.x * 8, steps = (a.C + 31) / 32, first = blockIdx.y * (NT * 8);
  const size_t row = (size_t)(f0 + g) * a.C;  // (F is a multiple of 8)
  const __nv_bfloat16 *wg = static_cast<const __nv_bfloat16*>(a.wg) + row, *wu = static_cast<const __nv_bfloat16*>(a.wu) + row;
  const uint4 none = make_uint4(0, 0, 0, 0);
  const __nv_bfloat16* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    x[n] = first + n * 8 + g < a.T ? static_cast<const __nv_bfloat16*>(a.x) + (first + n * 8 + g) * a.x_stride : nullptr;
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
  for (int n = warp; n < NT; n += kWarps) {
    float4 s = sums[0][n][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = sums[w][n][lane];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    finish<__nv_bfloat16, ACT, GRADS>(a, s, first + n * 8 + t * 2, f0 + g);
  }
}

// U: pieces of 128 terms a warp has in flight.
template <int ACT, int U>
__global__ void __launch_bounds__(32 * kWarps) ffn_one_f32_kernel(const Args a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int f0 = blockIdx.x * 2;
  const float* w[4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
    w[r] = static_cast<const float*>(r < 2 ? a.wg : a.wu) + (size_t)(f0 + r % 2) * a.C;
  const float* x = static_cast<const float*>(a.x);
  float v[4] = {0.f, 0.f, 0.f, 0.f};
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
      const float4 y = __ldg(reinterpret_cast<const float4*>(x + k));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        v[r] = fmaf(__uint_as_float(p[j][r].x), y.x, v[r]);
        v[r] = fmaf(__uint_as_float(p[j][r].y), y.y, v[r]);
        v[r] = fmaf(__uint_as_float(p[j][r].z), y.z, v[r]);
        v[r] = fmaf(__uint_as_float(p[j][r].w), y.w, v[r]);
      }
    }
  }
  __shared__ float sums[kWarps][4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
#pragma unroll
    for (int o = 16; o > 0; o /= 2) v[r] += __shfl_xor_sync(0xffffffffu, v[r], o);
    if (lane == r) sums[warp][r] = v[r];
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    float g = 0.f, u = 0.f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) g += sums[i][threadIdx.x], u += sums[i][2 + threadIdx.x];
    static_cast<float*>(a.out)[f0 + threadIdx.x] = act2<ACT>(make_float2(g, 0.f)).x * u;
  }
}

// NT: groups of 8 tokens. U: pieces of 16 terms a warp has in flight.
template <int ACT, bool GRADS, int NT, int U>
__global__ void __launch_bounds__(32 * kWarps, NT < 4 ? 3 : 2) ffn_few_parts_kernel(const Args a) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  const int f0 = blockIdx.x * 8, steps = (a.C + 15) / 16, first = blockIdx.y * (NT * 8);
  const size_t row = (size_t)(f0 + g) * a.C;  // (F is a multiple of 8)
  const float *wg = static_cast<const float*>(a.wg) + row, *wu = static_cast<const float*>(a.wu) + row;
  const float* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tok = first + n * 8 + g;
    x[n] = tok < a.T ? static_cast<const float*>(a.x) + tok * a.x_stride : nullptr;
  }
  float sum[NT][4], rest[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[n][i] = rest[n][i] = 0.f;
  tc::pdl_wait();
  uint4 p[U], q[U];  // pieces of 16 terms of the rows; the next ones are asked for when one is used
  auto ask = [&](int j, int step) {
    const int k = step * 16 + t * 4;
    p[j] = k < a.C ? load_once(wg + k) : make_uint4(0, 0, 0, 0);
    q[j] = k < a.C ? load_once(wu + k) : make_uint4(0, 0, 0, 0);
  };
#pragma unroll
  for (int j = 0; j < U; ++j) ask(j, warp + j * kWarps);
  for (int s0 = warp; s0 < steps; s0 += U * kWarps) {
    float d[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) d[n][0] = d[n][1] = d[n][2] = d[n][3] = 0.f;
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (s0 + j * kWarps) * 16 + t * 4;
      float v[8] = {__uint_as_float(p[j].x), __uint_as_float(p[j].y), __uint_as_float(q[j].x), __uint_as_float(q[j].y),
                    __uint_as_float(p[j].z), __uint_as_float(p[j].w), __uint_as_float(q[j].z), __uint_as_float(q[j].w)};
      ask(j, s0 + (U + j) * kWarps);
      uint32_t w[3][4];
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) w[i][r] = take_part(v[2 * r], v[2 * r + 1], i);
      uint32_t b[NT][3][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float4 y = k < a.C && x[n] != nullptr ? __ldg(reinterpret_cast<const float4*>(x[n] + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 3; ++i) b[n][i][0] = take_part(y.x, y.y, i), b[n][i][1] = take_part(y.z, y.w, i);
      }
      // (products on other accumulators do not wait for one another)
#pragma unroll
      for (int i = 0; i < 6; ++i) {
        constexpr int of_w[6] = {0, 2, 0, 1, 1, 0}, of_x[6] = {0, 0, 2, 1, 0, 1};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint32_t* m = w[of_w[i]];
          mma16816(i == 0 ? d[n] : rest[n], m[0], m[1], m[2], m[3], b[n][of_x[i]][0], b[n][of_x[i]][1]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] += d[n][i];
  }
  __shared__ float4 sums[kWarps][NT][32];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[n][i] += rest[n][i];
    sums[warp][n][lane] = make_float4(sum[n][0], sum[n][1], sum[n][2], sum[n][3]);
  }
  __syncthreads();
  for (int n = warp; n < NT; n += kWarps) {
    float4 s = sums[0][n][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const float4 v = sums[w][n][lane];
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    finish<float, ACT, GRADS>(a, s, first + n * 8 + t * 2, f0 + g);
  }
}

template <int ACT, bool GRADS>
cudaError_t launch(const Args& a, int dtype, cudaStream_t st) {
  const dim3 block(32 * kWarps), grid(a.F / 8, a.T <= 16 ? 1 : (a.T + 31) / 32);
  count_launches(1);
  if (dtype != LA_F32)
    return a.T <= 8    ? launch_pdl(ffn_few_kernel<ACT, GRADS, 1, 4>, grid, block, 0, st, a)
           : a.T <= 16 ? launch_pdl(ffn_few_kernel<ACT, GRADS, 2, 4>, grid, block, 0, st, a)
                       : launch_pdl(ffn_few_kernel<ACT, GRADS, 4, 4>, grid, block, 0, st, a);
  if (a.T == 1 && !GRADS) return launch_pdl(ffn_one_f32_kernel<ACT, 2>, dim3(a.F / 2), block, 0, st, a);
  return a.T <= 8    ? launch_pdl(ffn_few_parts_kernel<ACT, GRADS, 1, 2>, grid, block, 0, st, a)
         : a.T <= 16 ? launch_pdl(ffn_few_parts_kernel<ACT, GRADS, 2, 2>, grid, block, 0, st, a)
                     : launch_pdl(ffn_few_parts_kernel<ACT, GRADS, 4, 2>, grid, block, 0, st, a);
}

template <bool GRADS>
cudaError_t launch_act(const FfnGate& f, void* out, long long out_stride, cudaStream_t st) {
  const Args a{f.x, f.wg, f.wu, f.dh, out, f.x_stride, out_stride, f.dh_stride, f.T, f.C, f.F};
  return f.act == kSilu   ? launch<kSilu, GRADS>(a, f.dtype, st)
         : f.act == kGelu ? launch<kGelu, GRADS>(a, f.dtype, st)
                          : launch<kGeluTanh, GRADS>(a, f.dtype, st);
}

}  // namespace

// Few tokens, or a small product, of which the tiles of 256 tokens leave most tensor cores idle.
// bf16, here and in tiles: 32 tokens at C 2048, F 5632 15.7 and 16.0 us, 64 38 and 16; at C 512, F 1408
// 64 4.1 and 8.0; at C 64, F 168 300 2.5 and 6.3. float32: 64 tokens at C 2048, F 5632 67 and 100 us; at
// C 512, F 1408 186 14.7 and 22.9; at C 256, F 680 382 9.5 and 15.6. da and du: bf16 32 tokens at C 480,
// F 1920 3.8 and 8.6, at C 2048, F 5632 20.4 and 20.3; float32 186 at C 512, F 1408 17.3 and 24.9.
bool ffn_few(int T, int F, int dtype) {
  const bool f32 = dtype == LA_F32;
  return T <= (f32 ? 64 : 32) || (long long)T * F <= (f32 ? 1 << 18 : 1 << 17);
}

cudaError_t ffn_few_forward(const FfnGate& f, cudaStream_t st) { return launch_act<false>(f, f.h, f.h_stride, st); }

cudaError_t ffn_few_grads(const FfnGate& f, void* dact, cudaStream_t st) { return launch_act<true>(f, dact, f.F, st); }

}  // namespace la
