// C-ABI entry points of the gated recurrence, rotary positions and the gated head
// norm: argument validation on the host, then the kernels on the caller's stream.
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "la_common.cuh"
#include "la_internal.h"

namespace {

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

bool ptrs_ok(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr || !aligned(p, 16)) return false;
  return true;
}

bool dim_ok(int d) { return d >= 8 && d <= 128 && d % 8 == 0; }

bool shape_ok(int B, int H, int N) {
  return B >= 1 && H >= 1 && N >= 0 && (long long)B * H <= 0x7fffffffLL;
}

bool dtype_ok(int dtype) { return dtype == LA_F32 || dtype == LA_BF16; }

bool gated_ok(int B, int H, int N, int D, int M, int dtype) {
  // (token indices are ints, also past a segment's end)
  return shape_ok(B, H, N) && N <= 1 << 30 && dim_ok(D) && dim_ok(M) && dtype_ok(dtype);
}

bool strides_ok(const long long* s, int per) {
  return s != nullptr && s[0] % per == 0 && s[1] % per == 0 && s[2] % per == 0;
}

// Whether two arrays of float32 states share memory without being the same array.
bool overlap(const float* a, const float* b, size_t floats) {
  if (a == nullptr || b == nullptr || a == b) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x > y ? x - y : y - x) < sizeof(float) * floats;
}

int from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

// the state of no tokens: `from`, or zero
int copy_state(float* to, const float* from, size_t floats, cudaStream_t st) {
  if (to == nullptr || to == from) return LA_OK;
  return from_cuda(from ? cudaMemcpyAsync(to, from, sizeof(float) * floats,
                                          cudaMemcpyDeviceToDevice, st)
                        : cudaMemsetAsync(to, 0, sizeof(float) * floats, st));
}

}  // namespace

extern "C" {

size_t la_gated_workspace_bytes(int B, int H, int N, int D, int M, int dtype) {
  if (!gated_ok(B, H, N, D, M, dtype)) return la::kHeaderBytes;
  return la::gated_forward_workspace(B * H, N, D, M, dtype);
}

size_t la_gated_backward_workspace_bytes(int B, int H, int N, int D, int M, int dtype) {
  if (!gated_ok(B, H, N, D, M, dtype)) return la::kHeaderBytes;
  return la::gated_backward_workspace(B * H, N, D, M, dtype);
}

int la_forward_gated(const void* q, const void* k, const void* v, const void* g, void* out,
                     const float* S0, float* S, int B, int H, int N, int D, int M, int dtype,
                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!gated_ok(B, H, N, D, M, dtype)) return LA_ERR_INVALID_ARG;
  if (!aligned(S0, 16) || !aligned(S, 16)) return LA_ERR_INVALID_ARG;
  if (overlap(S0, S, (size_t)B * H * D * M)) return LA_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (N == 0) return copy_state(S, S0, (size_t)B * H * D * M, st);
  if (!ptrs_ok({q, k, v, g, out})) return LA_ERR_INVALID_ARG;
  // (the header alone is not used: there is no slot that could be outside a pool)
  const size_t need = la::gated_forward_workspace(B * H, N, D, M, dtype);
  if (need > la::kHeaderBytes &&
      (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
    return LA_ERR_WORKSPACE;
  const la::GatedForward f{q, k, v, g, out, S0, S, nullptr, nullptr, B, B, H, N, D, M, dtype};
  return from_cuda(la::gated_forward(f, workspace, st));
}

int la_extend_gated(const void* q, const void* k, const void* v, const void* g, void* out,
                    float* S_pool, const int* slots, const int* lens, int pool_size, int B, int H,
                    int N, int D, int M, int dtype, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (!gated_ok(B, H, N, D, M, dtype)) return LA_ERR_INVALID_ARG;
  if (!ptrs_ok({S_pool}) || !aligned(slots, 4) || !aligned(lens, 4)) return LA_ERR_INVALID_ARG;
  if (slots == nullptr ? pool_size < B : pool_size < 1) return LA_ERR_INVALID_ARG;
  if (N == 0) return LA_OK;
  if (!ptrs_ok({q, k, v, g, out})) return LA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < la::gated_forward_workspace(B * H, N, D, M, dtype))
    return LA_ERR_WORKSPACE;
  cudaStream_t st = as_stream(stream);
  // the status word, which only a slot outside the pool sets
  if (cudaMemsetAsync(workspace, 0, la::kHeaderBytes, st) != cudaSuccess) return LA_ERR_CUDA;
  const la::GatedForward f{q, k, v, g, out, S_pool, S_pool, slots, lens, pool_size,
                           B, H, N, D, M, dtype};
  return from_cuda(la::gated_forward(f, workspace, st));
}

int la_decode_step_gated(const void* q, const void* k, const void* v, const void* g, float* S_pool,
                         const int* slots, void* out, int pool_size, int n_streams, int H, int D,
                         int M, int dtype, void* stream) {
  if (!gated_ok(n_streams, H, 1, D, M, dtype)) return LA_ERR_INVALID_ARG;
  if (!ptrs_ok({q, k, v, g, S_pool, out}) || !aligned(slots, 4)) return LA_ERR_INVALID_ARG;
  if (slots == nullptr ? pool_size < n_streams : pool_size < 1) return LA_ERR_INVALID_ARG;
  return from_cuda(la::gated_decode(q, k, v, g, S_pool, slots, out, pool_size, n_streams, H, D, M,
                                    dtype, as_stream(stream)));
}

int la_backward_gated(const void* q, const void* k, const void* v, const void* g, const void* dout,
                      const float* S0, const float* dS, void* dq, void* dk, void* dv, void* dg,
                      float* dS0, int B, int H, int N, int D, int M, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!gated_ok(B, H, N, D, M, dtype)) return LA_ERR_INVALID_ARG;
  if (!aligned(S0, 16) || !aligned(dS, 16) || !aligned(dS0, 16)) return LA_ERR_INVALID_ARG;
  // dS0 is written while S0 is still read from (the states and their gradients are joined at
  // once); each element of dS is read by the thread that writes its dS0.
  const size_t floats = (size_t)B * H * D * M;
  if ((dS0 != nullptr && dS0 == S0) || overlap(dS0, S0, floats) || overlap(dS0, dS, floats))
    return LA_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (N == 0) return copy_state(dS0, dS, (size_t)B * H * D * M, st);
  if (!ptrs_ok({q, k, v, g, dout, dq, dk, dv, dg})) return LA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < la::gated_backward_workspace(B * H, N, D, M, dtype))
    return LA_ERR_WORKSPACE;
  const la::GatedBackward f{q, k, v, g, dout, S0, dS, dq, dk, dv, dg, dS0, B, H, N, D, M, dtype};
  return from_cuda(la::gated_backward(f, workspace, st));
}

int la_rotary(const void* q, const long long* q_strides, void* q_out, const long long* q_out_strides,
              const void* k, const long long* k_strides, void* k_out, const long long* k_out_strides,
              const double* freqs, const int* positions, long long pos_stride_b, long long offset,
              int B, int H, int Hk, int N, int D, int R, int interleaved, int inverse, float mscale,
              int dtype, void* stream) {
  if (!dtype_ok(dtype) || B < 1 || B > 65535 || H < 1 || Hk < 0 || N < 0 || !dim_ok(D) || R < 2 ||
      R > D || R % 2 != 0 || (long long)H + Hk > 65535)
    return LA_ERR_INVALID_ARG;
  // (a position is offset + token)
  if (offset > 1LL << 62 || offset < -(1LL << 62)) return LA_ERR_INVALID_ARG;
  if (N == 0) return LA_OK;
  const uintptr_t e = dtype == LA_F32 ? 4 : 2;
  if (q == nullptr || q_out == nullptr || !aligned(q, e) || !aligned(q_out, e) ||
      q_strides == nullptr || q_out_strides == nullptr || freqs == nullptr || !aligned(freqs, 8) ||
      !aligned(positions, 4))
    return LA_ERR_INVALID_ARG;
  if (Hk > 0 && (k == nullptr || k_out == nullptr || !aligned(k, e) || !aligned(k_out, e) ||
                 k_strides == nullptr || k_out_strides == nullptr))
    return LA_ERR_INVALID_ARG;
  la::Rotary r{};
  r.q = q;
  r.k = k;
  r.q_out = q_out;
  r.k_out = k_out;
  r.q_strides = q_strides;
  r.q_out_strides = q_out_strides;
  r.k_strides = k_strides;
  r.k_out_strides = k_out_strides;
  r.freqs = freqs;
  r.positions = positions;
  r.pos_stride_b = pos_stride_b;
  r.offset = offset;
  r.B = B;
  r.H = H;
  r.Hk = Hk;
  r.N = N;
  r.D = D;
  r.R = R;
  r.dtype = dtype;
  r.interleaved = interleaved != 0;
  r.inverse = inverse != 0;
  r.mscale = mscale;
  return from_cuda(la::rotary(r, as_stream(stream)));
}

static bool norm_ok(int B, int H, int N, int M, float eps, int dtype) {
  return shape_ok(B, H, N) && dim_ok(M) && dtype_ok(dtype) && eps >= 0.f &&
         (long long)B * N <= 0x7fffffffLL;
}

int la_norm_gate(const void* x, const void* z, const long long* z_strides, const void* w, void* y,
                 const long long* y_strides, int B, int H, int N, int M, int w_per_head, float eps,
                 int dtype, void* stream) {
  if (!norm_ok(B, H, N, M, eps, dtype)) return LA_ERR_INVALID_ARG;
  if (N == 0) return LA_OK;
  const int per = dtype == LA_F32 ? 4 : 8;
  if (!ptrs_ok({x, z, w, y}) || !strides_ok(z_strides, per) || !strides_ok(y_strides, per))
    return LA_ERR_INVALID_ARG;
  la::NormGate n{};
  n.x = x;
  n.z = z;
  n.w = w;
  n.y = y;
  n.z_strides = z_strides;
  n.y_strides = y_strides;
  n.B = B;
  n.H = H;
  n.N = N;
  n.M = M;
  n.dtype = dtype;
  n.w_per_head = w_per_head != 0;
  n.eps = eps;
  return from_cuda(la::norm_gate(n, as_stream(stream)));
}

size_t la_norm_gate_workspace_bytes(int B, int H, int N, int M) {
  if (!norm_ok(B, H, N, M, 0.f, LA_F32)) return la::kHeaderBytes;
  return la::norm_gate_workspace(B, H, N, M);
}

int la_norm_gate_backward(const void* x, const void* z, const long long* z_strides, const void* w,
                          const void* dy, const long long* dy_strides, void* dx, void* dz,
                          const long long* dz_strides, void* dw, int B, int H, int N, int M,
                          int w_per_head, float eps, int dtype, void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!norm_ok(B, H, N, M, eps, dtype) || !ptrs_ok({dw})) return LA_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  if (N == 0)
    return from_cuda(cudaMemsetAsync(
        dw, 0, (size_t)(dtype == LA_F32 ? 4 : 2) * M * (w_per_head ? H : 1), st));
  const int per = dtype == LA_F32 ? 4 : 8;
  if (!ptrs_ok({x, z, w, dy, dx, dz}) || !strides_ok(z_strides, per) ||
      !strides_ok(dy_strides, per) || !strides_ok(dz_strides, per))
    return LA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) ||
      workspace_bytes < la::norm_gate_workspace(B, H, N, M))
    return LA_ERR_WORKSPACE;
  la::NormGate n{};
  n.x = x;
  n.z = z;
  n.w = w;
  n.dy = dy;
  n.dx = dx;
  n.dz = dz;
  n.dw = dw;
  n.z_strides = z_strides;
  n.dy_strides = dy_strides;
  n.dz_strides = dz_strides;
  n.B = B;
  n.H = H;
  n.N = N;
  n.M = M;
  n.dtype = dtype;
  n.w_per_head = w_per_head != 0;
  n.eps = eps;
  return from_cuda(la::norm_gate_backward(n, workspace, st));
}

}  // extern "C"
