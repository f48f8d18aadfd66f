// Gated head norm: y = n * w * silu(z) with n = x r, r = 1 / sqrt(mean(x^2) + eps)
// over a head's M elements and silu(z) = z sigmoid(z); and its gradients, with
// s = sigmoid(z):
//   dn = dy w z s        dx = r (dn - n mean(dn n))
//   dz = dy w n s (1 + z (1 - s))                       dw = sum over rows of dy n z s
//
// Bound by memory: each row is read and written once, 16 bytes a thread, a row by
// M / V neighbouring lanes (V elements of 16 bytes) that share its sums by shuffles.
// A CTA's rows are of one head, so a thread keeps its piece of w in registers and
// sums its piece of dw over its rows; the CTAs' sums are joined in a fixed order by
// a second kernel (no atomics: the result repeats bit for bit). All arithmetic and
// sums are float32; results are rounded once.
#include "la_common.cuh"
#include "la_internal.h"

namespace la {
namespace {

constexpr int kThreads = 256;

struct NormArgs {
  const void *x, *z, *w, *dy;
  void *y, *dx, *dz;
  float* partial;  // backward: [H][tiles][M]
  long long zs[3], ys[3], dys[3], dzs[3];  // strides in elements: batch, head, token
  int B, H, N, M, w_stride, tiles, rows_per_tile;
  float eps;
};

template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T);
  float e[V];
  __device__ void load(const T* p) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = to_f32<T>(t[i]);
  }
  __device__ void store(T* p) const {
    uint4 u;
    T* t = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = from_f32<T>(e[i]);
    *reinterpret_cast<uint4*>(p) = u;
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// (the division's approximation is off by 2 steps of 2^-23; exp's overflow gives 0)
__device__ __forceinline__ float sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// LANES: threads per row, the power of two that holds M / V pieces.
template <typename T, int LANES, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_gate_kernel(const NormArgs a) {
  constexpr int V = Piece<T>::V, ROWS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
  const int h = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const bool live = lane * V < a.M;
  const unsigned n_rows = (unsigned)a.B * (unsigned)a.N;
  const unsigned begin = (unsigned)tile * (unsigned)a.rows_per_tile;
  const unsigned end = min(begin + (unsigned)a.rows_per_tile, n_rows);
  const int c = live ? lane * V : 0;
  Piece<T> w, dw;
  w.load(static_cast<const T*>(a.w) + (size_t)h * a.w_stride + c);
#pragma unroll
  for (int i = 0; i < V; ++i) dw.e[i] = 0.f;
  const float inv_m = 1.f / a.M;
  // AT rows a thread at once: their loads are all asked for before the first is used
  constexpr int AT = BWD ? 1 : 2;
  for (unsigned r0 = begin; r0 < end; r0 += AT * ROWS) {
    Piece<T> x[AT], z[AT], dy[AT];
    size_t xo[AT];
    long long b[AT], t[AT];
    bool in[AT];
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      const unsigned row = r0 + k * ROWS + row0;
      in[k] = live && row < end;
      b[k] = row / (unsigned)a.N;
      t[k] = row % (unsigned)a.N;
      xo[k] = (((size_t)b[k] * a.H + h) * a.N + t[k]) * a.M + c;
      if (in[k]) {
        x[k].load(static_cast<const T*>(a.x) + xo[k]);
        z[k].load(static_cast<const T*>(a.z) + b[k] * a.zs[0] + h * a.zs[1] + t[k] * a.zs[2] + c);
        if (BWD)
          dy[k].load(static_cast<const T*>(a.dy) + b[k] * a.dys[0] + h * a.dys[1] + t[k] * a.dys[2] + c);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) x[k].e[i] = z[k].e[i] = dy[k].e[i] = 0.f;
      }
    }
#pragma unroll
    for (int k = 0; k < AT; ++k) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(x[k].e[i], x[k].e[i], ss);
      const float r = rsqrtf(fmaf(row_sum<LANES>(ss), inv_m, a.eps));
      if (!BWD) {
        Piece<T> y;
#pragma unroll
        for (int i = 0; i < V; ++i)
          y.e[i] = x[k].e[i] * r * w.e[i] * (z[k].e[i] * sigmoid(z[k].e[i]));
        if (in[k]) y.store(static_cast<T*>(a.y) + b[k] * a.ys[0] + h * a.ys[1] + t[k] * a.ys[2] + c);
      } else {
        float dot = 0.f;
        Piece<T> dn, dz;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float zi = z[k].e[i], s = sigmoid(zi), n = x[k].e[i] * r, gate = zi * s;
          const float dyn = dy[k].e[i] * n;
          dn.e[i] = dy[k].e[i] * w.e[i] * gate;
          dz.e[i] = dyn * w.e[i] * (s * fmaf(zi, 1.f - s, 1.f));
          if (in[k]) dw.e[i] = fmaf(dyn, gate, dw.e[i]);
          dot = fmaf(dn.e[i], n, dot);
        }
        const float mean = row_sum<LANES>(dot) * inv_m;
#pragma unroll
        for (int i = 0; i < V; ++i) dn.e[i] = r * fmaf(-x[k].e[i] * r, mean, dn.e[i]);
        if (in[k]) {
          dn.store(static_cast<T*>(a.dx) + xo[k]);
          dz.store(static_cast<T*>(a.dz) + b[k] * a.dzs[0] + h * a.dzs[1] + t[k] * a.dzs[2] + c);
        }
      }
    }
  }
  if (BWD) {
    __shared__ float sums[ROWS][LANES * V + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) sums[row0][lane * V + i] = dw.e[i];
    __syncthreads();
    for (int m = threadIdx.x; m < a.M; m += kThreads) {
      float s = 0.f;
      for (int i = 0; i < ROWS; ++i) s += sums[i][m];
      a.partial[(size_t)blockIdx.x * a.M + m] = s;
    }
  }
}

// dw: sums of the CTAs' sums, one head's (w [H][M]) or all heads' (w [M]). 32
// columns by 32 strided rows a CTA.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_dw_kernel(const float* __restrict__ partial, T* __restrict__ dw, int rows, int M) {
  __shared__ float sums[32][33];
  const int m = blockIdx.x * 32 + threadIdx.x;
  const float* p = partial + (size_t)blockIdx.y * rows * M;
  float s = 0.f;
  if (m < M)
    for (int r = threadIdx.y; r < rows; r += 32) s += p[(size_t)r * M + m];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && m < M) {
    for (int i = 1; i < 32; ++i) s += sums[i][threadIdx.x];
    dw[(size_t)blockIdx.y * M + m] = from_f32<T>(s);
  }
}

// Tiles per head: about eight CTAs for each of the 152 SMs over all heads, but no
// fewer than 64 rows each (the weight's piece and the sums are paid per CTA).
int tiles_per_head(long long rows, int H) {
  long long t = (8 * 152 + H - 1) / H;
  const long long most = (rows + 63) / 64;
  if (t > most) t = most;
  return t < 1 ? 1 : (int)t;
}

template <typename T, bool BWD>
cudaError_t launch(const NormArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)a.H * a.tiles;
  const int pieces = (a.M + Piece<T>::V - 1) / Piece<T>::V;
  if (pieces <= 4)
    norm_gate_kernel<T, 4, BWD><<<grid, kThreads, 0, st>>>(a);
  else if (pieces <= 8)
    norm_gate_kernel<T, 8, BWD><<<grid, kThreads, 0, st>>>(a);
  else if (pieces <= 16)
    norm_gate_kernel<T, 16, BWD><<<grid, kThreads, 0, st>>>(a);
  else
    norm_gate_kernel<T, 32, BWD><<<grid, kThreads, 0, st>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

NormArgs args_of(const NormGate& n) {
  NormArgs a{};
  a.x = n.x;
  a.z = n.z;
  a.w = n.w;
  a.y = n.y;
  a.dy = n.dy;
  a.dx = n.dx;
  a.dz = n.dz;
  for (int d = 0; d < 3; ++d) {
    a.zs[d] = n.z_strides[d];
    if (n.y) a.ys[d] = n.y_strides[d];
    if (n.dy) {
      a.dys[d] = n.dy_strides[d];
      a.dzs[d] = n.dz_strides[d];
    }
  }
  a.B = n.B;
  a.H = n.H;
  a.N = n.N;
  a.M = n.M;
  a.w_stride = n.w_per_head ? n.M : 0;
  a.eps = n.eps;
  const long long rows = (long long)n.B * n.N;
  a.tiles = tiles_per_head(rows, n.H);
  a.rows_per_tile = (int)((rows + a.tiles - 1) / a.tiles);
  return a;
}

}  // namespace

size_t norm_gate_workspace(int B, int H, int N, int M) {
  return kHeaderBytes + sizeof(float) * (size_t)H * tiles_per_head((long long)B * N, H) * M;
}

cudaError_t norm_gate(const NormGate& n, cudaStream_t st) {
  const NormArgs a = args_of(n);
  return n.dtype == LA_F32 ? launch<float, false>(a, st) : launch<__nv_bfloat16, false>(a, st);
}

cudaError_t norm_gate_backward(const NormGate& n, void* ws, cudaStream_t st) {
  NormArgs a = args_of(n);
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes);
  cudaError_t e =
      n.dtype == LA_F32 ? launch<float, true>(a, st) : launch<__nv_bfloat16, true>(a, st);
  if (e != cudaSuccess) return e;
  const int rows = n.w_per_head ? a.tiles : a.tiles * n.H;
  const dim3 grid((n.M + 31) / 32, n.w_per_head ? n.H : 1), block(32, 32);
  if (n.dtype == LA_F32)
    norm_dw_kernel<float><<<grid, block, 0, st>>>(a.partial, (float*)n.dw, rows, n.M);
  else
    norm_dw_kernel<__nv_bfloat16><<<grid, block, 0, st>>>(a.partial, (__nv_bfloat16*)n.dw, rows, n.M);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace la
