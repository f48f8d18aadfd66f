// Rotary positions on q and k.
//
// Pair i of a head's first R elements, (a, b), is turned by the angle
// pos * freq_i and scaled: (a, b) -> mscale (a cos - b sin, a sin + b cos). The
// pair is elements (2i, 2i + 1) in the interleaved layout, (i, i + R/2) in the half
// layout; elements from R on are copied. The rotation's transpose (its gradient, and
// its inverse but for mscale) is the same with the angle's sign turned.
//
// Angles: a float32 product pos * freq loses the angle at far positions (2^-24 of
// 10^6 radians is 0.06). Here a frequency is a fraction of a turn in 64-bit fixed
// point, so the phase pos * freq modulo one turn is one wrapping integer product,
// off by at most |pos| 2^-54 turns (the float64 frequency's own rounding); of its top
// 32 bits, what is left of the nearest quarter turn goes to sincospif (of a whole half
// turn, float32 keeps 9e-8 radians; of an eighth of a turn 2.3e-8).
//
// Bound by memory: q and k are read and written once. A thread owns a few pairs of
// one token, works out their cosines and sines once and applies them to up to 8 heads of
// q and k. B4 H8 + 8 N16384 D64 bf16, token-major in, head-major out: 49 us for 268 MB
// (5.5 TB/s; 40 us at the rate of a plain copy). With the frequencies' float64 products
// per thread and not per CTA it was 61 us; 4 heads a thread 50.6, 16 heads 49.2.
#include "la_common.cuh"
#include "la_internal.h"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ unsigned long long turn_step(double freq) {
  const double t = freq * 0.15915494309189533577;  // 1 / (2 pi)
  return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

__device__ __forceinline__ void turn(unsigned long long step, long long pos, float mscale,
                                     float& c, float& s) {
  const unsigned top = (unsigned)(step * (unsigned long long)pos >> 32);
  const unsigned quarters = (top + 0x20000000u) >> 30;  // the nearest: an eighth of a turn is left
  const int rest = (int)(top - (quarters << 30));
  float rc, rs;
  sincospif((float)rest * 4.656612873077393e-10f, &rs, &rc);  // 2^-31 half turns
  c = quarters & 1 ? -rs : rc;
  s = quarters & 1 ? rc : rs;
  const float scale = quarters & 2 ? -mscale : mscale;
  c *= scale;
  s *= scale;
}

struct RotaryArgs {
  const void* x[2];  // q, k
  void* y[2];
  long long xs[2][3], ys[2][3];  // strides in elements: batch, head, token
  int heads[2];
  const double* freqs;
  const int* positions;
  long long pos_stride_b, offset;
  int N, D, R, per_thread;
  float mscale;
  bool interleaved, inverse;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

// V elements, read or written once: 16 bytes at a time are marked to leave the cache first
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> read(const T* p) {
  if constexpr (sizeof(T) * V == 16) {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
    return *reinterpret_cast<const Vec<T, V>*>(&u);
  }
  return *reinterpret_cast<const Vec<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void write(T* p, const Vec<T, V>& v) {
  if constexpr (sizeof(T) * V == 16)
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(&v));
  else
    *reinterpret_cast<Vec<T, V>*>(p) = v;
}

// V elements at a time (16 bytes; one element where a layout or an address does not
// allow that). An item is V elements of each half of the pairs (half layout), V / 2
// neighbouring pairs (interleaved; one pair for V = 1) or V copied elements.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int PAIRS = !INTER ? V : V > 1 ? V / 2 : 1;
  constexpr int W = INTER && V == 1 ? 2 : V;  // elements of one access of a turned item
  // a CTA works its frequencies out once: float64 is slow here (two lanes a clock per SM)
  __shared__ unsigned long long steps[64];
  tc::pdl_wait();
  if (threadIdx.x < a.R / 2) steps[threadIdx.x] = turn_step(a.freqs[threadIdx.x]);
  __syncthreads();
  const int turned = INTER ? a.R / W : a.R / (2 * V);
  const int items = turned + (a.D - a.R) / V;
  // (the thread's token and item, with the 64-bit division once per CTA)
  const long long first_item = (long long)blockIdx.x * kThreads, first_token = first_item / items;
  const unsigned in_cta = (unsigned)(first_item - first_token * items) + threadIdx.x;
  const long long t = first_token + in_cta / (unsigned)items;
  const int item = (int)(in_cta % (unsigned)items);
  if (t >= a.N) return;
  const int b = blockIdx.z;
  const int first = blockIdx.y * a.per_thread;
  const int last = min(first + a.per_thread, a.heads[0] + a.heads[1]);
  if (item >= turned) {
    const int at = a.R + (item - turned) * V;
    for (int i = first; i < last; ++i) {
      const int which = i >= a.heads[0], h = which ? i - a.heads[0] : i;
      const T* x = static_cast<const T*>(a.x[which]) + b * a.xs[which][0] + h * a.xs[which][1] + t * a.xs[which][2];
      T* y = static_cast<T*>(a.y[which]) + b * a.ys[which][0] + h * a.ys[which][1] + t * a.ys[which][2];
      write<T, V>(y + at, read<T, V>(x + at));
    }
    return;
  }
  const long long pos = a.positions ? (long long)a.positions[b * a.pos_stride_b + t] : a.offset + t;
  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int j = 0; j < PAIRS; ++j) {
    turn(steps[item * PAIRS + j], pos, a.mscale, c[j], s[j]);
    if (a.inverse) s[j] = -s[j];
  }
  const int at = item * W;
#pragma unroll 4
  for (int i = first; i < last; ++i) {
    const int which = i >= a.heads[0], h = which ? i - a.heads[0] : i;
    const T* x = static_cast<const T*>(a.x[which]) + b * a.xs[which][0] + h * a.xs[which][1] + t * a.xs[which][2];
    T* y = static_cast<T*>(a.y[which]) + b * a.ys[which][0] + h * a.ys[which][1] + t * a.ys[which][2];
    if constexpr (INTER && V == 1) {
      const float lo = to_f32<T>(x[at]), hi = to_f32<T>(x[at + 1]);
      y[at] = from_f32<T>(lo * c[0] - hi * s[0]);
      y[at + 1] = from_f32<T>(lo * s[0] + hi * c[0]);
    } else if constexpr (INTER) {
      Vec<T, V> w = read<T, V>(x + at);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const float lo = to_f32<T>(w.e[2 * j]), hi = to_f32<T>(w.e[2 * j + 1]);
        w.e[2 * j] = from_f32<T>(lo * c[j] - hi * s[j]);
        w.e[2 * j + 1] = from_f32<T>(lo * s[j] + hi * c[j]);
      }
      write<T, V>(y + at, w);
    } else {
      Vec<T, V> wa = read<T, V>(x + at);
      Vec<T, V> wb = read<T, V>(x + at + a.R / 2);
#pragma unroll
      for (int j = 0; j < PAIRS; ++j) {
        const float lo = to_f32<T>(wa.e[j]), hi = to_f32<T>(wb.e[j]);
        wa.e[j] = from_f32<T>(lo * c[j] - hi * s[j]);
        wb.e[j] = from_f32<T>(lo * s[j] + hi * c[j]);
      }
      write<T, V>(y + at, wa);
      write<T, V>(y + at + a.R / 2, wb);
    }
  }
}

template <typename T, int V, bool INTER>
cudaError_t launch(RotaryArgs a, int B, cudaStream_t st) {
  constexpr int W = INTER && V == 1 ? 2 : V;
  const int items = (INTER ? a.R / W : a.R / (2 * V)) + (a.D - a.R) / V;
  const long long tiles = ((long long)a.N * items + kThreads - 1) / kThreads;
  const int heads = a.heads[0] + a.heads[1];
  // heads per thread: as many as leave eight CTAs for each of the 152 SMs, up to 8
  int per = 8;
  while (per > 1 && tiles * B * ((heads + per - 1) / per) < 8 * 152) per /= 2;
  a.per_thread = per;
  // the grid's y and z end at 65535
  if (B > 65535 || (heads + per - 1) / per > 65535 || tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const cudaError_t e = tcx::launch_pdl(rotary_kernel<T, V, INTER>,
                                        dim3((unsigned)tiles, (heads + per - 1) / per, B),
                                        dim3(kThreads), 0, st, a);
  count_launches(1);
  return e;
}

template <typename T>
cudaError_t rotary_t(const RotaryArgs& a, int B, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  // 16-byte accesses where every row, the pairs and the copied rest allow them
  bool wide = (a.interleaved ? a.R : a.R / 2) % V == 0 && (a.D - a.R) % V == 0;
  for (int i = 0; i < 2 && wide; ++i) {
    if (a.heads[i] == 0) continue;
    wide = (reinterpret_cast<uintptr_t>(a.x[i]) | reinterpret_cast<uintptr_t>(a.y[i])) % 16 == 0;
    for (int d = 0; d < 3; ++d) wide = wide && a.xs[i][d] % V == 0 && a.ys[i][d] % V == 0;
  }
  if (wide) return a.interleaved ? launch<T, V, true>(a, B, st) : launch<T, V, false>(a, B, st);
  return a.interleaved ? launch<T, 1, true>(a, B, st) : launch<T, 1, false>(a, B, st);
}

}  // namespace

cudaError_t rotary(const Rotary& r, cudaStream_t st) {
  RotaryArgs a{};
  a.x[0] = r.q;
  a.x[1] = r.k;
  a.y[0] = r.q_out;
  a.y[1] = r.k_out;
  const long long* in[2] = {r.q_strides, r.k_strides};
  const long long* out[2] = {r.q_out_strides, r.k_out_strides};
  a.heads[0] = r.H;
  a.heads[1] = r.Hk;
  for (int i = 0; i < 2; ++i)
    for (int d = 0; d < 3 && a.heads[i]; ++d) {
      a.xs[i][d] = in[i][d];
      a.ys[i][d] = out[i][d];
    }
  a.freqs = r.freqs;
  a.positions = r.positions;
  a.pos_stride_b = r.pos_stride_b;
  a.offset = r.offset;
  a.N = r.N;
  a.D = r.D;
  a.R = r.R;
  a.mscale = r.mscale;
  a.interleaved = r.interleaved;
  a.inverse = r.inverse;
  return r.dtype == LA_F32 ? rotary_t<float>(a, r.B, st) : rotary_t<__nv_bfloat16>(a, r.B, st);
}

}  // namespace la
