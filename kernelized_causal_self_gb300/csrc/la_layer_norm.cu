// Layer norm over the C elements of each row, y = n w + b with n = (x - mean) r,
// r = 1 / sqrt(mean((x - mean)^2) + eps); and its gradients, with g = dy w:
//   dx = r (g - mean(g) - n mean(g n)),  dw = sum over rows of dy n,  db = sum over rows of dy.
// x may be read from an 8-bit checkpoint (la_checkpoint.cuh) in the backward pass, and one may
// be written in the forward pass, from the row that is in registers anyway.
//
// Bound by memory: every row is read once and stays in registers, as P pieces of 16 bytes in
// each of the G threads that share it; its sums go through shuffles and, where G is more than
// a warp, shared memory. The deviations are summed behind the mean, not as a difference of two
// large sums. A thread keeps its columns of w and b, and its sums of dw and db, over all rows
// that it takes; rows are asked for one ahead. The sums of the CTAs are joined in a fixed order
// by a second kernel (no atomics: results repeat bit for bit). Everything is float32, rounded once.
#include "la_checkpoint.cuh"
#include "la_internal.h"
#include "la_pair.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace {

struct Args {
  const void *x, *w, *b, *dy;
  const signed char* codes_in;
  const unsigned char* exps_in;
  void* out;  // y or dx
  signed char* codes;
  unsigned char* exps;
  float* partial;  // backward: [2][CTAs][C], dw's sums and db's
  long long rows, x_stride, dy_stride, out_stride;
  int C, n_blocks;
  float eps;
};

// Sums of N values over the G threads of a row, in a fixed order
template <int G, int THREADS, int N>
struct RowSum {
  static constexpr int kWarps = THREADS / 32;
  float (*slots)[N][kWarps];  // two of them in turn, so that one barrier a sum is enough
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&s)[N]) {
    constexpr int L = G < 32 ? G : 32;
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
    if constexpr (G > 32) {
      const int warp = threadIdx.x / 32;
      if (threadIdx.x % 32 == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) slots[turn][i][warp] = s[i];
      __syncthreads();
      const int w0 = threadIdx.x / G * (G / 32);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        s[i] = 0.f;
#pragma unroll
        for (int w = 0; w < G / 32; ++w) s[i] += slots[turn][i][w0 + w];
      }
      turn ^= 1;
    }
  }
};

enum Mode { kForward, kForwardKeep, kBackward, kBackwardKept };

template <typename T, int G, int P, int MODE>
__global__ void __launch_bounds__(G > 256 ? G : 256, G > 256 ? 1 : MODE < kBackward ? 3 : 2)
layer_norm_kernel(const Args a) {
  constexpr int V = 16 / sizeof(T), THREADS = G > 256 ? G : 256, ROWS = THREADS / G;
  constexpr bool BWD = MODE == kBackward || MODE == kBackwardKept;
  constexpr int LANES = q8::kBlock / V;
  using Code = typename q8::Codes<V>::type;
  __shared__ float slots1[2][1][THREADS / 32], slots2[2][2][THREADS / 32];
  RowSum<G, THREADS, 1> sum1{slots1};
  RowSum<G, THREADS, 2> sum2{slots2};
  const int group = threadIdx.x / G, lane = threadIdx.x % G;
  const float inv_c = 1.f / a.C;
  int col[P];
  bool live[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    col[p] = (p * G + lane) * V;
    live[p] = col[p] < a.C;
    if (!live[p]) col[p] = 0;
  }
  tc::pdl_wait();
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 wu[P], bu[P];  // as they are stored: converted where they are used
  // sums of dw and db: in registers, or (rows of 1024 threads, which have 64 each) in shared memory
  constexpr bool SHARED = BWD && G == 1024;
  constexpr int PR = SHARED ? 1 : P;
  float dw[PR][V], db[PR][V];
  extern __shared__ float4 acc[];  // [dw, db][P][V / 4][G]
  float4* mine = acc + threadIdx.x;
  auto piece = [&](const void* base, long long at) {
    return *reinterpret_cast<const uint4*>(static_cast<const T*>(base) + at);
  };
  auto values = [](const uint4& u, float (&to)[V]) {
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) to[i] = to_f32<T>(t[i]);
  };
#pragma unroll
  for (int p = 0; p < P; ++p) {
    wu[p] = live[p] ? piece(a.w, col[p]) : none;
    bu[p] = !BWD && live[p] && a.b != nullptr ? piece(a.b, col[p]) : none;
  }
#pragma unroll
  for (int p = 0; p < PR; ++p)
#pragma unroll
    for (int i = 0; i < V; ++i) dw[p][i] = db[p][i] = 0.f;
  if (SHARED)
    for (int i = 0; i < 2 * P * (V / 4); ++i) mine[i * G] = make_float4(0.f, 0.f, 0.f, 0.f);

  uint4 nx[P], ndy[P];
  Code ncode[P];
  uint32_t ne[P];
  auto ask = [&](long long row) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const bool in = live[p] && row < a.rows;
      if constexpr (MODE == kBackwardKept) {
        ncode[p] = Code{};
        ne[p] = 127;
        if (in) {
          ncode[p] = __ldcs(reinterpret_cast<const Code*>(a.codes_in + row * a.C + col[p]));
          ne[p] = a.exps_in[row * a.n_blocks + col[p] / q8::kBlock];
        }
      } else {
        nx[p] = in ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) +
                                                           row * a.x_stride + col[p]))
                   : none;
      }
      if (BWD)
        ndy[p] = in ? __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(a.dy) +
                                                            row * a.dy_stride + col[p]))
                    : none;
    }
  };
  const long long step = (long long)gridDim.x * ROWS;
  long long row = (long long)blockIdx.x * ROWS + group;
  ask(row);
  // (every group of the CTA runs as often as the first, whose row is the smallest)
  for (long long r0 = (long long)blockIdx.x * ROWS; r0 < a.rows; r0 += step, row += step) {
    float x[P][V], dy[P][V];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if constexpr (MODE == kBackwardKept) {
        q8::values_of<V>(ncode[p], q8::step_value(ne[p]), x[p]);
      } else {
        values(nx[p], x[p]);
      }
      if (BWD) values(ndy[p], dy[p]);
    }
    ask(row + step);
    if constexpr (MODE == kForwardKeep) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const uint32_t e = q8::step_of(q8::block_top<V>(x[p]));
        if (live[p] && row < a.rows) {
          *reinterpret_cast<Code*>(a.codes + row * a.C + col[p]) =
              q8::codes_of<V>(x[p], q8::inverse_step(e), e);
          if (lane % LANES == 0)
            a.exps[row * a.n_blocks + col[p] / q8::kBlock] = (unsigned char)e;
        }
      }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) s[0] += x[p][i];
    sum1(s);
    const float mean = s[0] / a.C;  // (rounded once: a flat row of short values has no deviations)
    s[0] = 0.f;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[p][i] = live[p] ? x[p][i] - mean : 0.f;
        s[0] = fmaf(x[p][i], x[p][i], s[0]);
      }
    sum1(s);
    // (a row past the end adds nothing to dw, whatever eps)
    const float r = row < a.rows ? rsqrtf(fmaf(s[0], inv_c, a.eps)) : 0.f;
    if (!BWD) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float w[V], b[V];
        values(wu[p], w);
        values(bu[p], b);
        uint4 u;
        T* t = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = from_f32<T>(fmaf(x[p][i] * r, w[i], b[i]));
        if (live[p] && row < a.rows)
          *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.out_stride + col[p]) = u;
      }
    } else {
      float m[2] = {0.f, 0.f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        float w[V];
        values(wu[p], w);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          x[p][i] *= r;
          if constexpr (!SHARED) {
            dw[p][i] = fmaf(dy[p][i], x[p][i], dw[p][i]);
            db[p][i] += dy[p][i];
          }
        }
        if constexpr (SHARED) {
#pragma unroll
          for (int i = 0; i < V; i += 4) {
            float4 *tw = mine + (p * (V / 4) + i / 4) * G, *tb = tw + P * (V / 4) * G;
            float4 sw = *tw, sb = *tb;
            sw.x = fmaf(dy[p][i], x[p][i], sw.x), sw.y = fmaf(dy[p][i + 1], x[p][i + 1], sw.y);
            sw.z = fmaf(dy[p][i + 2], x[p][i + 2], sw.z), sw.w = fmaf(dy[p][i + 3], x[p][i + 3], sw.w);
            sb.x += dy[p][i], sb.y += dy[p][i + 1], sb.z += dy[p][i + 2], sb.w += dy[p][i + 3];
            *tw = sw;
            *tb = sb;
          }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
          dy[p][i] *= w[i];
          m[0] += dy[p][i];
          m[1] = fmaf(dy[p][i], x[p][i], m[1]);
        }
      }
      sum2(m);
      const float m0 = m[0] * inv_c, m1 = m[1] * inv_c;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        uint4 u;
        T* t = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < V; ++i) t[i] = from_f32<T>(r * (dy[p][i] - m0 - x[p][i] * m1));
        if (live[p] && row < a.rows)
          *reinterpret_cast<uint4*>(static_cast<T*>(a.out) + row * a.out_stride + col[p]) = u;
      }
    }
  }
  if constexpr (BWD) {
    // the groups' sums, in order, through shared memory
    __shared__ float sums[ROWS > 1 ? ROWS : 1][ROWS > 1 ? G * P * V : 1];
    float* to = a.partial + (size_t)blockIdx.x * a.C;
    const size_t half = (size_t)gridDim.x * a.C;
    for (int which = 0; which < 2; ++which, to += half) {
      if constexpr (ROWS > 1) {
        __syncthreads();
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int i = 0; i < V; ++i)
            sums[group][(p * G + lane) * V + i] = which ? db[p % PR][i] : dw[p % PR][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.C; c += THREADS) {
          float t = 0.f;
          for (int g = 0; g < ROWS; ++g) t += sums[g][c];
          to[c] = t;
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (live[p])
#pragma unroll
            for (int i = 0; i < V; i += 4) {
              float4 v;
              if constexpr (SHARED) {
                v = mine[((which * P + p) * (V / 4) + i / 4) * G];
              } else {
                const float* s = which ? &db[p][i] : &dw[p][i];
                v = make_float4(s[0], s[1], s[2], s[3]);
              }
              *reinterpret_cast<float4*>(to + col[p] + i) = v;
            }
      }
    }
  }
}

// dw (blockIdx.y == 0) and db: sums of the CTAs' sums, 32 columns by 32 strided rows a CTA
template <typename T>
__global__ void __launch_bounds__(1024)
layer_norm_sums_kernel(const float* __restrict__ partial, T* dw, T* db, int rows, int C) {
  __shared__ float sums[32][33];
  int c = blockIdx.x * 32 + threadIdx.x;
  const float* p = partial + (size_t)blockIdx.y * rows * C;
  T* to = blockIdx.y ? db : dw;
  tc::pdl_wait();
  float s = 0.f;
  if (c < C)
    for (int r = threadIdx.y; r < rows; r += 32 * 5) {  // (five loads in flight: 304 rows are two turns)
      float v[5];
#pragma unroll
      for (int i = 0; i < 5; ++i) v[i] = r + 32 * i < rows ? p[(size_t)(r + 32 * i) * C + c] : 0.f;
#pragma unroll
      for (int i = 0; i < 5; ++i) s += v[i];
    }
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  s = sums[threadIdx.x][threadIdx.y];  // (a warp has a column now)
#pragma unroll
  for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
  c = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && c < C) to[c] = from_f32<T>(s);
}

// Threads that share a row, and the rows that a CTA of 256 (or G, if more) has at once
int threads_per_row(int C) {
  for (int g = 8; g < 32; g *= 2)
    if (C <= 8 * g) return g;
  int g = 32;
  while (C > 16 * g) g *= 2;
  return g;
}

// CTAs: twice the three that an SM holds, the backward pass's two (whose sums cost per CTA), fewer
// where rows are few. 65536 x 512 in bf16: 24.6 us (5.5 TB/s) with three CTAs of 80 registers an SM,
// 27.5 with four of 64 or two, 27 with two rows asked for ahead, 28 to 34 with none; backward 37.6
// (5.3 TB/s), 81 with three CTAs an SM. In float32, whose rows of 264 to 4096 spill 8 to 36 bytes a thread
// at 80 registers, 42.3 us (6.3 TB/s) and backward 60.0 (6.7); 20000 x 1000 26.6 and 40.0 (6.0 TB/s both),
// 32.4 with a checkpoint, 38.3 from one. What would be a wave and a part of one is one of CTAs that
// take two: 2001 x 1000 in float32 kept in 8 bits 7.1 -> 6.3 us, 4096 x 512 in bf16 4.7 -> 4.2.
int ctas_of(long long rows, int C, bool bwd) {
  const int g = threads_per_row(C), at_once = g < 256 ? 256 / g : 1;
  const long long all = (rows + at_once - 1) / at_once;
  int each = bwd ? 2 : 6;
  if (g > 256) each = g == 512 ? each / 2 : 1;
  if (!bwd && g <= 256 && all > 3 * 152 && all <= 6 * 152) return (int)((all + 1) / 2);
  return (int)(all < (long long)each * 152 ? all : each * 152);
}

template <typename T, int G, int P, int MODE>
cudaError_t launch_one(const Args& a, int ctas, cudaStream_t st) {
  constexpr int smem = (MODE == kBackward || MODE == kBackwardKept) && G == 1024 ? 2 * P * (16 / sizeof(T) / 4) * G * 16 : 0;
  cudaError_t e = cudaSuccess;
  if (smem > 0) e = tcx::configure_once<layer_norm_kernel<T, G, P, MODE>>(smem);
  if (e != cudaSuccess) return e;
  e = tcx::launch_pdl(layer_norm_kernel<T, G, P, MODE>, dim3(ctas), dim3(G > 256 ? G : 256), smem, st, a);
  count_launches(1);
  return e;
}

template <typename T, int MODE>
cudaError_t launch(const Args& a, cudaStream_t st) {
  constexpr int E = sizeof(T) / 2;  // pieces of 8 elements
  const int n = ctas_of(a.rows, a.C, MODE == kBackward || MODE == kBackwardKept);
  const int g = threads_per_row(a.C);
  if (g == 8) return launch_one<T, 8, E, MODE>(a, n, st);
  if (g == 16) return launch_one<T, 16, E, MODE>(a, n, st);
  if (g == 32)
    return a.C <= 256 ? launch_one<T, 32, E, MODE>(a, n, st) : launch_one<T, 32, 2 * E, MODE>(a, n, st);
  if (g == 64) return launch_one<T, 64, 2 * E, MODE>(a, n, st);
  if (g == 128) return launch_one<T, 128, 2 * E, MODE>(a, n, st);
  if (g == 256) return launch_one<T, 256, 2 * E, MODE>(a, n, st);
  if (g == 512) return launch_one<T, 512, 2 * E, MODE>(a, n, st);
  return launch_one<T, 1024, 2 * E, MODE>(a, n, st);
}

Args args_of(const LayerNorm& n) {
  Args a{};
  a.x = n.x;
  a.w = n.w;
  a.b = n.b;
  a.dy = n.dy;
  a.rows = n.rows;
  a.x_stride = n.x_stride;
  a.C = n.C;
  a.n_blocks = q8::blocks_of(n.C);
  a.eps = n.eps;
  return a;
}

}  // namespace

size_t layer_norm_workspace(long long rows, int C) {
  return kHeaderBytes + sizeof(float) * 2 * (size_t)ctas_of(rows, C, true) * C;
}

cudaError_t layer_norm(const LayerNorm& n, cudaStream_t st) {
  Args a = args_of(n);
  a.out = n.y;
  a.out_stride = n.y_stride;
  a.codes = n.codes;
  a.exps = n.exps;
  if (n.dtype == LA_F32)
    return n.codes ? launch<float, kForwardKeep>(a, st) : launch<float, kForward>(a, st);
  return n.codes ? launch<__nv_bfloat16, kForwardKeep>(a, st) : launch<__nv_bfloat16, kForward>(a, st);
}

cudaError_t layer_norm_backward(const LayerNorm& n, void* ws, cudaStream_t st) {
  Args a = args_of(n);
  a.codes_in = n.codes;
  a.exps_in = n.exps;
  a.dy_stride = n.dy_stride;
  a.out = n.dx;
  a.out_stride = n.dx_stride;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes);
  cudaError_t e;
  if (n.dtype == LA_F32)
    e = n.codes ? launch<float, kBackwardKept>(a, st) : launch<float, kBackward>(a, st);
  else
    e = n.codes ? launch<__nv_bfloat16, kBackwardKept>(a, st) : launch<__nv_bfloat16, kBackward>(a, st);
  if (e != cudaSuccess) return e;
  const int rows = ctas_of(n.rows, n.C, true);
  const dim3 grid((n.C + 31) / 32, 2), block(32, 32);
  const float* partial = a.partial;
  e = n.dtype == LA_F32
          ? tcx::launch_pdl(layer_norm_sums_kernel<float>, grid, block, 0, st, partial, (float*)n.dw,
                            (float*)n.db, rows, n.C)
          : tcx::launch_pdl(layer_norm_sums_kernel<__nv_bfloat16>, grid, block, 0, st, partial,
                            (__nv_bfloat16*)n.dw, (__nv_bfloat16*)n.db, rows, n.C);
  count_launches(1);
  return e;
}

}  // namespace la
