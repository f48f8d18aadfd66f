// The gated projections on the CUDA cores: a = x wg^T, u = x wu^T, h = act(a) u, and the backward
// pass da = dh u act'(a), du = dh act(a), dx = da wg + du wu, dwg = da^T x, dwu = du^T x.
//
// One tiled product for all of them: a CTA makes a BM x BN tile of D = sum_k A(m, k) B(n, k),
// 8 x 8 of it a thread, with operands that are contiguous along k or along m / n, staged through
// two shared-memory tiles of kK steps of k while the next ones are on their way to registers:
//   projections  A = x (along k), B = half a tile's rows of wg and the same rows of wu (along k),
//                so that a thread's 8 columns are 4 of a and the same 4 of u;
//   dx           A = da, then du (along k = f), B = wg, then wu (along n = c);
//   dw           A = da or du (along m = f), B = x (along n = c), k the tokens.
// Bound by the float32 pipes (two lanes a packed multiply-add): 64 of them for 4 reads of 16
// bytes. Products with few tiles and long sums (dx, dw) are cut along k, the parts written in
// float32 and added in a fixed order by a second kernel.
#include "la_checkpoint.cuh"
#include "la_ffn.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

using namespace tcx;
using namespace ffn;

constexpr int kK = 16;

enum Kind { kForward, kGrads, kDx, kDw };

struct Args {
  const void *x, *wg, *wu, *dh;
  void* out;                // h, dx or dwg
  void* out2;               // dwu
  void* dact;               // [2][T][F]: da, du (written by kGrads, read by kDx and kDw)
  float* partial;           // split sums: [splits][matrix]
  signed char* codes;       // checkpoint of a, u: [T][2][F], nullptr: not wanted
  unsigned char* exps;
  long long x_stride, dh_stride, out_stride;
  int T, C, F, splits;
  unsigned n_tiles;  // tiles along n, which move fastest
};

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

__device__ __forceinline__ void store8(float* p, const float* v) {
  store4(p, make_float4(v[0], v[1], v[2], v[3]));
  store4(p + 4, make_float4(v[4], v[5], v[6], v[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(tc::pack_bf16(v[0], v[1]), tc::pack_bf16(v[2], v[3]),
                                            tc::pack_bf16(v[4], v[5]), tc::pack_bf16(v[6], v[7]));
}

template <typename T, int KIND, int ACT, int BM, int BN>
__global__ void __launch_bounds__(BM * BN / 64, BM == 128 ? 2 : 8) ffn_simt_kernel(const Args a) {
  constexpr int THREADS = BM * BN / 64, TX = BN / 8, PAD = 4;
  constexpr bool DUAL = KIND == kForward || KIND == kGrads;
  constexpr int LA = BM * kK / 4 / THREADS, LB = BN * kK / 4 / THREADS;  // 4-element loads a thread
  __shared__ float As[2][kK][BM + PAD], Bs[2][kK][BN + PAD];
  const int tid = threadIdx.x, tx = tid % TX, ty = tid / TX;
  const T* x = static_cast<const T*>(a.x);
  const T* dact = static_cast<const T*>(a.dact);
  const size_t part = (size_t)a.T * a.F;
  // the tile, the sum's range
  const int m0 = (int)(blockIdx.x / a.n_tiles) * BM, n0 = (int)(blockIdx.x % a.n_tiles) * (DUAL ? BN / 2 : BN);
  const int which = KIND == kDw ? blockIdx.z / a.splits : 0;
  const int split = KIND == kDw ? blockIdx.z % a.splits : blockIdx.z;
  const int per = KIND == kDx ? (a.F + kK - 1) / kK : 0;  // k steps of each of dx's two parts
  const int steps = KIND == kDx ? 2 * per : ((KIND == kDw ? a.T : a.C) + kK - 1) / kK;
  const int begin = DUAL ? 0 : (int)((long long)steps * split / a.splits);
  const int end = DUAL ? steps : (int)((long long)steps * (split + 1) / a.splits);
  tc::pdl_wait();

  float4 ra[LA], rb[LB];
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  auto ask = [&](int s) {
    const int p = KIND == kDx ? s / per : 0, k0 = (KIND == kDx ? s % per : s) * kK;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      const int i = tid + j * THREADS;
      if constexpr (KIND == kDw) {
        const int k = k0 + i / (BM / 4), m = m0 + i % (BM / 4) * 4;
        ra[j] = k < a.T && m < a.F ? load4(dact + which * part + (size_t)k * a.F + m) : zero;
      } else {
        const int m = m0 + i / (kK / 4), k = k0 + i % (kK / 4) * 4;
        if constexpr (KIND == kDx)
          ra[j] = m < a.T && k < a.F ? load4(dact + p * part + (size_t)m * a.F + k) : zero;
        else
          ra[j] = m < a.T && k < a.C ? load4(x + m * a.x_stride + k) : zero;
      }
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int i = tid + j * THREADS;
      if constexpr (DUAL) {
        const int row = i / (kK / 4), k = k0 + i % (kK / 4) * 4, f = n0 + row % (BN / 2);
        const T* w = static_cast<const T*>(row < BN / 2 ? a.wg : a.wu);
        rb[j] = f < a.F && k < a.C ? load4(w + (size_t)f * a.C + k) : zero;
      } else {
        const int k = k0 + i / (BN / 4), n = n0 + i % (BN / 4) * 4;
        if constexpr (KIND == kDx)
          rb[j] = k < a.F && n < a.C ? load4(static_cast<const T*>(p ? a.wu : a.wg) + (size_t)k * a.C + n) : zero;
        else
          rb[j] = k < a.T && n < a.C ? load4(x + k * a.x_stride + n) : zero;
      }
    }
  };
  auto put = [&](int b) {
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      const int i = tid + j * THREADS;
      if constexpr (KIND == kDw) {
        *reinterpret_cast<float4*>(&As[b][i / (BM / 4)][i % (BM / 4) * 4]) = ra[j];
      } else {
        const int m = i / (kK / 4), k = i % (kK / 4) * 4;
        As[b][k][m] = ra[j].x, As[b][k + 1][m] = ra[j].y, As[b][k + 2][m] = ra[j].z, As[b][k + 3][m] = ra[j].w;
      }
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int i = tid + j * THREADS;
      if constexpr (!DUAL) {
        *reinterpret_cast<float4*>(&Bs[b][i / (BN / 4)][i % (BN / 4) * 4]) = rb[j];
      } else {
        const int n = i / (kK / 4), k = i % (kK / 4) * 4;
        Bs[b][k][n] = rb[j].x, Bs[b][k + 1][n] = rb[j].y, Bs[b][k + 2][n] = rb[j].z, Bs[b][k + 3][n] = rb[j].w;
      }
    }
  };

  float2 acc[8][4];  // rows ty * 4 + {0..3}, BM / 2 + the same; columns likewise
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
  if (begin < end) {
    ask(begin);
    put(0);
  }
  __syncthreads();
  for (int s = begin; s < end; ++s) {
    const int b = (s - begin) & 1;
    if (s + 1 < end) ask(s + 1);
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const float4 a0 = *reinterpret_cast<const float4*>(&As[b][k][ty * 4]);
      const float4 a1 = *reinterpret_cast<const float4*>(&As[b][k][BM / 2 + ty * 4]);
      const float4 b0 = *reinterpret_cast<const float4*>(&Bs[b][k][tx * 4]);
      const float4 b1 = *reinterpret_cast<const float4*>(&Bs[b][k][BN / 2 + tx * 4]);
      const float av[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      const float2 bv[4] = {make_float2(b0.x, b0.y), make_float2(b0.z, b0.w), make_float2(b1.x, b1.y),
                            make_float2(b1.z, b1.w)};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fma2(make_float2(av[i], av[i]), bv[j], acc[i][j]);
    }
    if (s + 1 < end) put(b ^ 1);
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int m = m0 + (i < 4 ? 0 : BM / 2) + ty * 4 + i % 4;
    const float lo[4] = {acc[i][0].x, acc[i][0].y, acc[i][1].x, acc[i][1].y};
    const float hi[4] = {acc[i][2].x, acc[i][2].y, acc[i][3].x, acc[i][3].y};
    if constexpr (DUAL) {
      const int f = n0 + tx * 4;
      const bool in = m < a.T && f < a.F;
      float o[4], o2[4];
      float4 d = zero;
      if (KIND == kGrads && in) d = load4(static_cast<const T*>(a.dh) + m * a.dh_stride + f);
      const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (KIND == kForward) {
          o[j] = act<ACT>(lo[j]) * hi[j];
        } else {
          float fa, df;
          act_grad<ACT>(lo[j], fa, df);
          o[j] = dv[j] * hi[j] * df;
          o2[j] = dv[j] * fa;
        }
      }
      if constexpr (KIND == kForward) {
        if (in) store4(static_cast<T*>(a.out) + m * a.out_stride + f, make_float4(o[0], o[1], o[2], o[3]));
        if (a.codes != nullptr) {
          // 8 neighbouring lanes hold a block of 32 columns (columns past F are sums of zeros)
          const int nb = q8::blocks_of(a.F);
          const uint32_t ea = q8::step_of(q8::block_top<4>(lo)), eu = q8::step_of(q8::block_top<4>(hi));
          if (in) {
            const size_t row = 2 * (size_t)m;
            *reinterpret_cast<uint32_t*>(a.codes + row * a.F + f) = q8::codes4(lo, q8::inverse_step(ea), ea);
            *reinterpret_cast<uint32_t*>(a.codes + (row + 1) * a.F + f) = q8::codes4(hi, q8::inverse_step(eu), eu);
            if (f % q8::kBlock == 0) {
              a.exps[row * nb + f / q8::kBlock] = (unsigned char)ea;
              a.exps[(row + 1) * nb + f / q8::kBlock] = (unsigned char)eu;
            }
          }
        }
      } else if (in) {
        T* to = static_cast<T*>(a.dact) + (size_t)m * a.F + f;
        store4(to, make_float4(o[0], o[1], o[2], o[3]));
        store4(to + part, make_float4(o2[0], o2[1], o2[2], o2[3]));
      }
    } else {
      const int rows = KIND == kDx ? a.T : a.F;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int c = n0 + half * (BN / 2) + tx * 4;
        if (m >= rows || c >= a.C) continue;
        const float* v = half ? hi : lo;
        const float4 o = make_float4(v[0], v[1], v[2], v[3]);
        if (a.splits > 1)
          store4(a.partial + ((size_t)(KIND == kDw ? which * a.splits + split : split) * rows + m) * a.C + c, o);
        else if (KIND == kDx)
          store4(static_cast<T*>(a.out) + m * a.out_stride + c, o);
        else
          store4(static_cast<T*>(which ? a.out2 : a.out) + (size_t)m * a.C + c, o);
      }
    }
  }
}

// The parts of split sums, added in order: matrix blockIdx.y of [.][splits][rows][C]
template <typename T>
__global__ void __launch_bounds__(256) ffn_join_kernel(const float* partial, T* out, T* out2, long long out_stride,
                                                       int rows, int C, int splits) {
  const long long n = (long long)rows * C / 4;
  const float* p = partial + (size_t)blockIdx.y * splits * rows * C;
  T* to = blockIdx.y ? out2 : out;
  tc::pdl_wait();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    float4 s = load4(p + 4 * i);
    for (int k = 1; k < splits; ++k) {
      const float4 v = load4(p + (size_t)k * rows * C + 4 * i);
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    const long long row = 4 * i / C;
    store4(to + row * out_stride + (4 * i - row * C), s);
  }
}

// da, du from a checkpoint of a and u: 8 neighbours a thread, all of a block's step. Bound by
// memory (T 4096, F 5632 in bf16: 186 MB).
template <typename T, int ACT>
__global__ void __launch_bounds__(256) ffn_kept_grads_kernel(const Args a) {
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
    if constexpr (sizeof(T) == 2) {
      act_grad2<ACT>(make_float2(g[j], g[j + 1]), fa, df);
    } else {
      act_grad<ACT>(g[j], fa.x, df.x);
      act_grad<ACT>(g[j + 1], fa.y, df.y);
    }
    da[j] = dv[j] * u[j] * df.x, da[j + 1] = dv[j + 1] * u[j + 1] * df.y;
    du[j] = dv[j] * fa.x, du[j + 1] = dv[j + 1] * fa.y;
  }
  T* to = static_cast<T*>(a.dact) + t * a.F + f;
  store8(to, da);
  store8(to + part, du);
}

constexpr int kSms = 152;

int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

// Tiles of 128 x 128 where they fill the SMs, else of 64 x 64
bool wide(long long m, long long n, int count) {
  return (long long)ceil_div(m, 128) * ceil_div(n, 128) * count >= kSms;
}

// Parts of a sum of k terms, so that its tiles' CTAs are about two per SM and a part is no
// shorter than 128 terms
int splits_of(long long m, long long n, long long k, int count) {
  const int b = wide(m, n, count) ? 128 : 64;
  const long long tiles = (long long)ceil_div(m, b) * ceil_div(n, b) * count;
  const long long want = b == 128 ? 2 * kSms : 6 * kSms;
  long long s = want / tiles;
  if (s > k / 128) s = k / 128;
  if (s > 32) s = 32;
  return s < 1 ? 1 : (int)s;
}

template <typename T, int KIND, int ACT>
cudaError_t launch(Args a, cudaStream_t st) {
  const long long m = KIND == kDw ? a.F : a.T, n = KIND == kForward || KIND == kGrads ? 2LL * a.F : a.C;
  const int count = KIND == kDw ? 2 : 1, z = KIND == kForward || KIND == kGrads ? 1 : count * a.splits;
  cudaError_t e;
  const bool big = wide(m, n, count);
  const int b = big ? 128 : 64;
  a.n_tiles = ceil_div(n, b);
  const dim3 grid(a.n_tiles * (unsigned)ceil_div(m, b), 1, z);  // (T <= 2^24, C, F <= 2^16: an int)
  e = big ? launch_pdl(ffn_simt_kernel<T, KIND, ACT, 128, 128>, grid, dim3(256), 0, st, a)
          : launch_pdl(ffn_simt_kernel<T, KIND, ACT, 64, 64>, grid, dim3(64), 0, st, a);
  count_launches(1);
  return e;
}

template <typename T>
cudaError_t grads(const Args& a, int act, cudaStream_t st) {
  return act == kSilu   ? launch<T, kGrads, kSilu>(a, st)
         : act == kGelu ? launch<T, kGrads, kGelu>(a, st)
                        : launch<T, kGrads, kGeluTanh>(a, st);
}

template <typename T>
cudaError_t kept_grads(const Args& a, int act, cudaStream_t st) {
  const dim3 grid((unsigned)(((long long)a.T * (a.F / 8) + 255) / 256));  // (T <= 2^24, F <= 2^16: an int)
  const cudaError_t e =
      act == kSilu   ? launch_pdl(ffn_kept_grads_kernel<T, kSilu>, grid, dim3(256), 0, st, a)
      : act == kGelu ? launch_pdl(ffn_kept_grads_kernel<T, kGelu>, grid, dim3(256), 0, st, a)
                     : launch_pdl(ffn_kept_grads_kernel<T, kGeluTanh>, grid, dim3(256), 0, st, a);
  count_launches(1);
  return e;
}

template <typename T>
cudaError_t join(const float* partial, void* out, void* out2, long long stride, int rows, int count, int C, int splits,
                 cudaStream_t st) {
  const long long n = (long long)rows * C / 4;
  const int ctas = (int)((n + 255) / 256 < 8 * kSms ? (n + 255) / 256 : 8 * kSms);
  const cudaError_t e = launch_pdl(ffn_join_kernel<T>, dim3(ctas, count), dim3(256), 0, st, partial,
                                   static_cast<T*>(out), static_cast<T*>(out2), stride, rows, C, splits);
  count_launches(1);
  return e;
}

Args args_of(const FfnGate& f) {
  Args a{};
  a.x = f.x, a.wg = f.wg, a.wu = f.wu, a.dh = f.dh;
  a.codes = f.codes, a.exps = f.exps;
  a.x_stride = f.x_stride, a.dh_stride = f.dh_stride;
  a.T = f.T, a.C = f.C, a.F = f.F, a.splits = 1;
  return a;
}

template <typename T>
cudaError_t backward(const FfnGate& f, void* ws, cudaStream_t st) {
  Args a = args_of(f);
  char* at = static_cast<char*>(ws) + kHeaderBytes;
  a.dact = at;
  a.partial = reinterpret_cast<float*>(at + align_up(2 * sizeof(T) * (size_t)f.T * f.F, 256));
  cudaError_t e = f.codes != nullptr ? ffn_kept_grads(f, a.dact, st) : grads<T>(a, f.act, st);
  if (e != cudaSuccess) return e;
  a.out = f.dx, a.out_stride = f.dx_stride;
  a.splits = splits_of(f.T, f.C, 2LL * f.F, 1);
  e = launch<T, kDx, kSilu>(a, st);
  if (e == cudaSuccess && a.splits > 1) e = join<T>(a.partial, a.out, nullptr, f.dx_stride, f.T, 1, f.C, a.splits, st);
  if (e != cudaSuccess) return e;
  a.out = f.dwg, a.out2 = f.dwu;
  a.splits = splits_of(f.F, f.C, f.T, 2);
  e = launch<T, kDw, kSilu>(a, st);
  if (e == cudaSuccess && a.splits > 1) e = join<T>(a.partial, a.out, a.out2, f.C, f.F, 2, f.C, a.splits, st);
  return e;
}

template <typename T>
cudaError_t forward(const FfnGate& f, cudaStream_t st) {
  Args a = args_of(f);
  a.out = f.h, a.out_stride = f.h_stride;
  return f.act == kSilu   ? launch<T, kForward, kSilu>(a, st)
         : f.act == kGelu ? launch<T, kForward, kGelu>(a, st)
                          : launch<T, kForward, kGeluTanh>(a, st);
}

}  // namespace

cudaError_t ffn_join(const float* partial, void* out, void* out2, long long out_stride, int rows, int count, int C,
                     int splits, int dtype, cudaStream_t st) {
  return dtype == LA_F32 ? join<float>(partial, out, out2, out_stride, rows, count, C, splits, st)
                         : join<__nv_bfloat16>(partial, out, out2, out_stride, rows, count, C, splits, st);
}

cudaError_t ffn_kept_grads(const FfnGate& f, void* dact, cudaStream_t st) {
  Args a = args_of(f);
  a.dact = dact;
  return f.dtype == LA_F32 ? kept_grads<float>(a, f.act, st) : kept_grads<__nv_bfloat16>(a, f.act, st);
}

size_t ffn_simt_backward_workspace(int T, int C, int F, int dtype) {
  const int sx = splits_of(T, C, 2LL * F, 1), sw = splits_of(F, C, T, 2);
  const size_t dx = sx > 1 ? (size_t)sx * T * C : 0, dw = sw > 1 ? 2 * (size_t)sw * F * C : 0;
  return kHeaderBytes + align_up(2 * (size_t)(dtype == LA_F32 ? 4 : 2) * T * F, 256) +
         sizeof(float) * (dx > dw ? dx : dw);
}

cudaError_t ffn_simt_forward(const FfnGate& f, cudaStream_t st) {
  return f.dtype == LA_F32 ? forward<float>(f, st) : forward<__nv_bfloat16>(f, st);
}

cudaError_t ffn_simt_backward(const FfnGate& f, void* ws, cudaStream_t st) {
  return f.dtype == LA_F32 ? backward<float>(f, ws, st) : backward<__nv_bfloat16>(f, ws, st);
}

}  // namespace la
