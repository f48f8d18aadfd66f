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
// sums are float32, with functions as exact as the type shows; results are rounded once.
// B4 H8 N16384 M64 bf16: forward 33 us for 201 MB (6.1 TB/s). Two rows a thread at once with
// their addresses worked out anew took 43 us, with 222 instructions a row and thread.
// B2 H6 N2001 M96 float32: backward 10.3 + 2.3 us for 46 MB (6.8 us at HBM's rate).
#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

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

// 16 bytes of a row as float32
template <typename T>
struct Piece {
  static constexpr int V = 16 / sizeof(T);
  float e[V];
  __device__ void set(const uint4& u) {
    const T* t = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = to_f32<T>(t[i]);
  }
  __device__ void store(T* p) const {
    uint4 u;
    T* t = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < V; ++i) t[i] = from_f32<T>(e[i]);
    __stcs(reinterpret_cast<uint4*>(p), u);
  }
};

// A thread's piece of the rows (b, h, t) of one head that it visits, `step` rows of t
// apart: the address moves by additions (divisions only where t passes N).
template <typename T>
struct Rows {
  T* p;
  long long move, wrap;  // per step; from the end of a batch entry to the next
  __device__ void start(const void* base, long long b, long long t, long long sb, long long st,
                        long long at, int N, int step) {
    p = const_cast<T*>(static_cast<const T*>(base)) + b * sb + t * st + at;
    move = st * step;
    wrap = sb - N * st;
  }
  __device__ void next(unsigned wraps) {
    p += move;
    if (wraps) p += wraps * wrap;
  }
};

template <int LANES>
__device__ __forceinline__ float row_sum(float s) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// s = sigmoid(z) and 1 - s, from exp(-|z|): nothing overflows and nothing cancels. In bf16
// __expf, off by 2 + 1.17 |z| steps of 2^-23 and zero past |z| = 87.3; in float32 that would
// show, and expf costs 3% (backward of B4 H8 N8192 M64 59.4 to 61.4 us). The quotient's
// divisor is within [1, 2], where __fdividef is off by at most 2 steps.
template <typename T>
__device__ __forceinline__ void sigmoid(float z, float& s, float& rest) {
  const float e = sizeof(T) == 4 ? expf(-fabsf(z)) : __expf(-fabsf(z));
  const float large = __fdividef(1.f, 1.f + e), small = e * large;
  s = z < 0.f ? small : large;
  rest = z < 0.f ? large : small;
}

// LANES: threads per row, the power of two that holds M / V pieces. A row's loads are
// asked for while the row before it is worked on.
template <typename T, int LANES, bool BWD>
__global__ void __launch_bounds__(kThreads) norm_gate_kernel(const NormArgs a) {
  constexpr int V = Piece<T>::V, ROWS = kThreads / LANES;
  const int lane = threadIdx.x % LANES, row0 = threadIdx.x / LANES;
  // heads in neighbouring CTAs: a token-major tensor's rows of one token then move together
  const int h = blockIdx.x % a.H, tile = blockIdx.x / a.H;
  const bool live = lane * V < a.M;
  const unsigned n_rows = (unsigned)a.B * (unsigned)a.N, N = a.N;
  const unsigned begin = (unsigned)tile * (unsigned)a.rows_per_tile;
  const unsigned end = min(begin + (unsigned)a.rows_per_tile, n_rows);
  const int c = live ? lane * V : 0;
  tc::pdl_wait();
  Piece<T> w, dw;
  w.set(*reinterpret_cast<const uint4*>(static_cast<const T*>(a.w) + (size_t)h * a.w_stride + c));
#pragma unroll
  for (int i = 0; i < V; ++i) dw.e[i] = 0.f;
  const float inv_m = 1.f / a.M;

  unsigned row = begin + row0;
  const long long b0 = row / N;
  unsigned t = row % N;  // of the row that is asked for next
  const long long sb = (long long)a.H * a.N * a.M;
  Rows<T> xr, zr, dyr, out, dzr;
  xr.start(a.x, b0, t, sb, a.M, (long long)h * a.N * a.M + c, N, ROWS);
  zr.start(a.z, b0, t, a.zs[0], a.zs[2], h * a.zs[1] + c, N, ROWS);
  if (BWD) {
    dyr.start(a.dy, b0, t, a.dys[0], a.dys[2], h * a.dys[1] + c, N, ROWS);
    out.start(a.dx, b0, t, sb, a.M, (long long)h * a.N * a.M + c, N, ROWS);
    dzr.start(a.dz, b0, t, a.dzs[0], a.dzs[2], h * a.dzs[1] + c, N, ROWS);
  } else {
    out.start(a.y, b0, t, a.ys[0], a.ys[2], h * a.ys[1] + c, N, ROWS);
  }
  const uint4 none = make_uint4(0, 0, 0, 0);
  uint4 nx = none, nz = none, ndy = none;
  auto ask = [&]() {
    const bool in = live && row < end;
    nx = in ? __ldcs(reinterpret_cast<const uint4*>(xr.p)) : none;
    nz = in ? __ldcs(reinterpret_cast<const uint4*>(zr.p)) : none;
    if (BWD) ndy = in ? __ldcs(reinterpret_cast<const uint4*>(dyr.p)) : none;
  };
  ask();
  for (unsigned r0 = begin; r0 < end; r0 += ROWS) {
    const bool in = live && row < end;
    Piece<T> x, z, dy;
    x.set(nx);
    z.set(nz);
    if (BWD) dy.set(ndy);
    // on to the next row
    row += ROWS;
    t += ROWS;
    unsigned wraps = 0;
    if (t >= N) {
      wraps = t / N;
      t -= wraps * N;
    }
    xr.next(wraps);
    zr.next(wraps);
    if (BWD) dyr.next(wraps);
    ask();

    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) ss = fmaf(x.e[i], x.e[i], ss);
    const float r = rsqrtf(fmaf(row_sum<LANES>(ss), inv_m, a.eps));
    if (!BWD) {
      Piece<T> y;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s, rest;
        sigmoid<T>(z.e[i], s, rest);
        y.e[i] = x.e[i] * r * w.e[i] * (z.e[i] * s);
      }
      if (in) y.store(out.p);
    } else {
      float dot = 0.f;
      Piece<T> dn, dz;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s, rest;
        sigmoid<T>(z.e[i], s, rest);
        const float zi = z.e[i], n = x.e[i] * r, gate = zi * s;
        const float dyn = dy.e[i] * n;
        dn.e[i] = dy.e[i] * w.e[i] * gate;
        dz.e[i] = dyn * w.e[i] * (s * fmaf(zi, rest, 1.f));
        if (in) dw.e[i] = fmaf(dyn, gate, dw.e[i]);
        dot = fmaf(dn.e[i], n, dot);
      }
      const float mean = row_sum<LANES>(dot) * inv_m;
#pragma unroll
      for (int i = 0; i < V; ++i) dn.e[i] = r * fmaf(-x.e[i] * r, mean, dn.e[i]);
      if (in) {
        dn.store(out.p);
        dz.store(dzr.p);
      }
      dzr.next(wraps);
    }
    out.next(wraps);
  }
  if (BWD) {
    __shared__ float sums[ROWS][LANES * V + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) sums[row0][lane * V + i] = dw.e[i];
    __syncthreads();
    for (int m = threadIdx.x; m < a.M; m += kThreads) {
      float s = 0.f;
      for (int i = 0; i < ROWS; ++i) s += sums[i][m];
      a.partial[((size_t)h * a.tiles + tile) * a.M + m] = s;
    }
  }
}

// dw: sums of the CTAs' sums, one head's (w [H][M]) or all heads' (w [M]). 32
// columns (blockIdx.y) of a head (blockIdx.x) by 32 strided rows a CTA.
template <typename T>
__global__ void __launch_bounds__(1024)
norm_dw_kernel(const float* __restrict__ partial, T* __restrict__ dw, int rows, int M) {
  __shared__ float sums[32][33];
  const int m = blockIdx.y * 32 + threadIdx.x;
  const float* p = partial + (size_t)blockIdx.x * rows * M;
  tc::pdl_wait();
  float s = 0.f;
  if (m < M)
    for (int r = threadIdx.y; r < rows; r += 32) s += p[(size_t)r * M + m];
  sums[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && m < M) {
    for (int i = 1; i < 32; ++i) s += sums[i][threadIdx.x];
    dw[(size_t)blockIdx.x * M + m] = from_f32<T>(s);
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
  const dim3 grid((unsigned)a.H * a.tiles), block(kThreads);
  const int pieces = (a.M + Piece<T>::V - 1) / Piece<T>::V;
  const cudaError_t e =
      pieces <= 4    ? tcx::launch_pdl(norm_gate_kernel<T, 4, BWD>, grid, block, 0, st, a)
      : pieces <= 8  ? tcx::launch_pdl(norm_gate_kernel<T, 8, BWD>, grid, block, 0, st, a)
      : pieces <= 16 ? tcx::launch_pdl(norm_gate_kernel<T, 16, BWD>, grid, block, 0, st, a)
                     : tcx::launch_pdl(norm_gate_kernel<T, 32, BWD>, grid, block, 0, st, a);
  count_launches(1);
  return e;
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
  const dim3 grid(n.w_per_head ? n.H : 1, (n.M + 31) / 32), block(32, 32);
  const float* partial = a.partial;
  e = n.dtype == LA_F32
          ? tcx::launch_pdl(norm_dw_kernel<float>, grid, block, 0, st, partial, (float*)n.dw, rows, n.M)
          : tcx::launch_pdl(norm_dw_kernel<__nv_bfloat16>, grid, block, 0, st, partial,
                            (__nv_bfloat16*)n.dw, rows, n.M);
  count_launches(1);
  return e;
}

}  // namespace la
