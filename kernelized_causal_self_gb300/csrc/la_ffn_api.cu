// C-ABI entry points of a layer's feed-forward half (layer norm, gated projections) and of the
// 8-bit checkpoints: argument validation on the host, then the kernels on the caller's stream.
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

bool dtype_ok(int dtype) { return dtype == LA_F32 || dtype == LA_BF16; }

size_t size_of(int dtype) { return dtype == LA_F32 ? 4 : 2; }

// n elements a row, rows `stride` elements apart: 16-byte pieces that do not overlap
bool stride_ok(long long stride, int n, int dtype) {
  return stride >= n && stride <= 1LL << 37 && stride % (dtype == LA_F32 ? 4 : 8) == 0;
}

bool rows_ok(long long rows, int C, int dtype) {
  return rows >= 0 && rows <= 0x7fffffffLL && C >= 8 && C % 8 == 0 && C <= 1 << 16 && dtype_ok(dtype);
}

bool norm_ok(long long rows, int C, float eps, int dtype) {
  return rows_ok(rows, C, dtype) && C <= 1 << 14 && eps >= 0.f;
}

bool ffn_ok(int T, int C, int F, int act, int dtype) {
  return rows_ok(T, C, dtype) && T <= 1 << 24 && F >= 8 && F % 8 == 0 && F <= 1 << 16 && act >= LA_SILU &&
         act <= LA_GELU_TANH;
}

// codes and exps: both or neither; 8 codes at a time are written
bool kept_ok(const void* codes, const void* exps, bool needed) {
  if ((codes == nullptr) != (exps == nullptr)) return false;
  return codes != nullptr ? aligned(codes, 16) : !needed;
}

// `rows` rows of `width` bytes, `stride` bytes apart
struct Span {
  const void* p;
  size_t width, stride, rows;
};

Span span(const void* p, size_t bytes) { return {p, bytes, bytes, bytes > 0 ? 1u : 0u}; }

Span span(const void* p, long long rows, long long stride, int n, int dtype) {
  return {p, size_of(dtype) * n, size_of(dtype) * (size_t)stride, (size_t)rows};
}

bool meet(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (x >= y + (b.rows - 1) * b.stride + b.width || y >= x + (a.rows - 1) * a.stride + a.width) return false;
  // rows equally far apart, each in columns of its own of one buffer
  if (a.rows > 1 && b.rows > 1 && a.stride == b.stride) {
    const uintptr_t at = y >= x ? (y - x) % a.stride : a.stride - 1 - (x - y - 1) % a.stride;
    return at < a.width || at + b.width > a.stride;
  }
  return true;
}

// Whether memory that is written is no other argument's.
bool apart(std::initializer_list<Span> written, std::initializer_list<Span> read) {
  for (const Span& w : written) {
    for (const Span& r : read)
      if (meet(w, r)) return false;
    for (const Span& o : written)
      if (&o != &w && meet(w, o)) return false;
  }
  return true;
}

size_t exps_of(int n) { return (size_t)(n + 31) / 32; }

int from_cuda(cudaError_t e) { return e == cudaSuccess ? LA_OK : LA_ERR_CUDA; }

cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }

bool few(int T, int F, bool kept, int dtype) { return !kept && la::ffn_few(T, F, dtype); }

// (bf16: the tensor-core kernels' status header)
size_t ffn_workspace(int T, int C, int F, bool kept, int dtype) {
  if (few(T, F, kept, dtype)) return 0;
  return dtype == LA_F32 ? la::ffn_tc32_workspace(T, C, F, false) : la::kHeaderBytes;
}

size_t ffn_backward_workspace(int T, int C, int F, int dtype) {
  return dtype == LA_F32 ? la::ffn_tc32_workspace(T, C, F, true) : la::ffn_tc_backward_workspace(T, C, F);
}

}  // namespace

extern "C" {

int la_checkpoint(const void* x, long long x_stride, signed char* codes, unsigned char* exps, long long rows,
                  int C, int dtype, void* stream) {
  if (!rows_ok(rows, C, dtype)) return LA_ERR_INVALID_ARG;
  if (rows == 0) return LA_OK;
  if (!ptrs_ok({x}) || !stride_ok(x_stride, C, dtype) || !kept_ok(codes, exps, true) ||
      !apart({span(codes, (size_t)rows * C), span(exps, (size_t)rows * exps_of(C))}, {span(x, rows, x_stride, C, dtype)}))
    return LA_ERR_INVALID_ARG;
  const la::Checkpoint c{const_cast<void*>(x), codes, exps, rows, x_stride, C, dtype};
  return from_cuda(la::checkpoint_pack(c, as_stream(stream)));
}

int la_checkpoint_restore(const signed char* codes, const unsigned char* exps, void* x, long long x_stride,
                          long long rows, int C, int dtype, void* stream) {
  if (!rows_ok(rows, C, dtype)) return LA_ERR_INVALID_ARG;
  if (rows == 0) return LA_OK;
  if (!ptrs_ok({x}) || !stride_ok(x_stride, C, dtype) || !kept_ok(codes, exps, true) ||
      !apart({span(x, rows, x_stride, C, dtype)}, {span(codes, (size_t)rows * C), span(exps, (size_t)rows * exps_of(C))}))
    return LA_ERR_INVALID_ARG;
  const la::Checkpoint c{x, const_cast<signed char*>(codes), const_cast<unsigned char*>(exps), rows, x_stride, C, dtype};
  return from_cuda(la::checkpoint_restore(c, as_stream(stream)));
}

int la_layer_norm(const void* x, long long x_stride, const void* w, const void* b, void* y, long long y_stride,
                  signed char* codes, unsigned char* exps, long long rows, int C, float eps, int dtype,
                  void* stream) {
  if (!norm_ok(rows, C, eps, dtype)) return LA_ERR_INVALID_ARG;
  if (rows == 0) return LA_OK;
  if (!ptrs_ok({x, w, y}) || !aligned(b, 16) || !stride_ok(x_stride, C, dtype) || !stride_ok(y_stride, C, dtype) ||
      !kept_ok(codes, exps, false))
    return LA_ERR_INVALID_ARG;
  const size_t e = size_of(dtype) * C;
  const Span xs = span(x, rows, x_stride, C, dtype), ys = span(y, rows, y_stride, C, dtype), none = span(nullptr, 0);
  // y may be x itself: a row is in registers before it is written
  const bool itself = y == x && y_stride == x_stride;
  if (!apart({ys, span(codes, (size_t)rows * C), span(exps, (size_t)rows * exps_of(C))}, {span(w, e), span(b, e)}) ||
      !apart({itself ? none : ys, span(codes, (size_t)rows * C), span(exps, (size_t)rows * exps_of(C))}, {xs}))
    return LA_ERR_INVALID_ARG;
  la::LayerNorm n{};
  n.x = x;
  n.w = w;
  n.b = b;
  n.y = y;
  n.codes = codes;
  n.exps = exps;
  n.rows = rows;
  n.x_stride = x_stride;
  n.y_stride = y_stride;
  n.C = C;
  n.dtype = dtype;
  n.eps = eps;
  return from_cuda(la::layer_norm(n, as_stream(stream)));
}

size_t la_layer_norm_workspace_bytes(long long rows, int C) {
  if (!norm_ok(rows, C, 0.f, LA_F32) || rows == 0) return la::kHeaderBytes;
  return la::layer_norm_workspace(rows, C);
}

int la_layer_norm_backward(const void* x, long long x_stride, const signed char* codes, const unsigned char* exps,
                           const void* w, const void* dy, long long dy_stride, void* dx, long long dx_stride,
                           void* dw, void* db, long long rows, int C, float eps, int dtype, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!norm_ok(rows, C, eps, dtype) || !ptrs_ok({dw, db})) return LA_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  const size_t e = size_of(dtype) * C;
  if (rows == 0) {
    if (!apart({span(dw, e), span(db, e)}, {})) return LA_ERR_INVALID_ARG;
    const cudaError_t r = cudaMemsetAsync(dw, 0, e, st);
    return from_cuda(r == cudaSuccess ? cudaMemsetAsync(db, 0, e, st) : r);
  }
  if ((x == nullptr) == (codes == nullptr) || !kept_ok(codes, exps, x == nullptr) || !ptrs_ok({w, dy, dx}) ||
      !aligned(x, 16) || (x != nullptr && !stride_ok(x_stride, C, dtype)) || !stride_ok(dy_stride, C, dtype) ||
      !stride_ok(dx_stride, C, dtype))
    return LA_ERR_INVALID_ARG;
  const Span xs = span(x, rows, x_stride, C, dtype), ys = span(dy, rows, dy_stride, C, dtype),
             ds = span(dx, rows, dx_stride, C, dtype), none = span(nullptr, 0);
  // dx may be x or dy itself, as y may be x
  const bool is_x = dx == x && dx_stride == x_stride, is_dy = dx == dy && dx_stride == dy_stride;
  if (!apart({ds, span(dw, e), span(db, e)}, {span(w, e), span(codes, (size_t)rows * C), span(exps, (size_t)rows * exps_of(C)),
                                            is_x ? none : xs, is_dy ? none : ys}) ||
      !apart({span(dw, e), span(db, e)}, {xs, ys}))
    return LA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < la::layer_norm_workspace(rows, C))
    return LA_ERR_WORKSPACE;
  la::LayerNorm n{};
  n.x = x;
  n.codes = const_cast<signed char*>(codes);
  n.exps = const_cast<unsigned char*>(exps);
  n.w = w;
  n.dy = dy;
  n.dx = dx;
  n.dw = dw;
  n.db = db;
  n.rows = rows;
  n.x_stride = x_stride;
  n.dy_stride = dy_stride;
  n.dx_stride = dx_stride;
  n.C = C;
  n.dtype = dtype;
  n.eps = eps;
  return from_cuda(la::layer_norm_backward(n, workspace, st));
}

size_t la_ffn_gate_workspace_bytes(int T, int C, int F, int checkpoint, int dtype) {
  if (!ffn_ok(T, C, F, LA_SILU, dtype)) return la::kHeaderBytes;
  return ffn_workspace(T, C, F, checkpoint != 0, dtype);
}

size_t la_ffn_gate_backward_workspace_bytes(int T, int C, int F, int dtype) {
  if (!ffn_ok(T, C, F, LA_SILU, dtype) || T == 0) return la::kHeaderBytes;
  return ffn_backward_workspace(T, C, F, dtype);
}

int la_ffn_gate(const void* x, long long x_stride, const void* wg, const void* wu, void* h, long long h_stride,
                signed char* codes, unsigned char* exps, int T, int C, int F, int act, int dtype, void* workspace,
                size_t workspace_bytes, void* stream) {
  if (!ffn_ok(T, C, F, act, dtype)) return LA_ERR_INVALID_ARG;
  if (T == 0) return LA_OK;
  if (!ptrs_ok({x, wg, wu, h}) || !stride_ok(x_stride, C, dtype) || !stride_ok(h_stride, F, dtype) ||
      !kept_ok(codes, exps, false))
    return LA_ERR_INVALID_ARG;
  const size_t w = size_of(dtype) * C * F, kept = 2 * (size_t)T;
  if (!apart({span(h, T, h_stride, F, dtype), span(codes, kept * F), span(exps, kept * exps_of(F))},
             {span(x, T, x_stride, C, dtype), span(wg, w), span(wu, w)}))
    return LA_ERR_INVALID_ARG;
  const size_t need = ffn_workspace(T, C, F, codes != nullptr, dtype);
  if (need > 0 && (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need))
    return LA_ERR_WORKSPACE;
  la::FfnGate f{};
  f.x = x;
  f.wg = wg;
  f.wu = wu;
  f.h = h;
  f.codes = codes;
  f.exps = exps;
  f.x_stride = x_stride;
  f.h_stride = h_stride;
  f.T = T;
  f.C = C;
  f.F = F;
  f.act = act;
  f.dtype = dtype;
  if (few(T, F, codes != nullptr, dtype)) return from_cuda(la::ffn_few_forward(f, as_stream(stream)));
  return from_cuda(dtype == LA_F32 ? la::ffn_tc32_forward(f, workspace, as_stream(stream))
                                   : la::ffn_tc_forward(f, workspace, as_stream(stream)));
}

int la_ffn_gate_backward(const void* x, long long x_stride, const void* wg, const void* wu, const void* dh,
                         long long dh_stride, const signed char* codes, const unsigned char* exps, void* dx,
                         long long dx_stride, void* dwg, void* dwu, int T, int C, int F, int act, int dtype,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (!ffn_ok(T, C, F, act, dtype) || !ptrs_ok({dwg, dwu})) return LA_ERR_INVALID_ARG;
  cudaStream_t st = as_stream(stream);
  const size_t w = size_of(dtype) * C * F, kept = 2 * (size_t)T;
  if (T == 0) {
    if (!apart({span(dwg, w), span(dwu, w)}, {})) return LA_ERR_INVALID_ARG;
    const cudaError_t e = cudaMemsetAsync(dwg, 0, w, st);
    return from_cuda(e == cudaSuccess ? cudaMemsetAsync(dwu, 0, w, st) : e);
  }
  if (!ptrs_ok({x, wg, wu, dh, dx}) || !stride_ok(x_stride, C, dtype) || !stride_ok(dh_stride, F, dtype) ||
      !stride_ok(dx_stride, C, dtype) || !kept_ok(codes, exps, false))
    return LA_ERR_INVALID_ARG;
  if (!apart({span(dx, T, dx_stride, C, dtype), span(dwg, w), span(dwu, w)},
             {span(x, T, x_stride, C, dtype), span(wg, w), span(wu, w), span(dh, T, dh_stride, F, dtype),
              span(codes, kept * F), span(exps, kept * exps_of(F))}))
    return LA_ERR_INVALID_ARG;
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < ffn_backward_workspace(T, C, F, dtype))
    return LA_ERR_WORKSPACE;
  la::FfnGate f{};
  f.x = x;
  f.wg = wg;
  f.wu = wu;
  f.dh = dh;
  f.dx = dx;
  f.dwg = dwg;
  f.dwu = dwu;
  f.codes = const_cast<signed char*>(codes);
  f.exps = const_cast<unsigned char*>(exps);
  f.x_stride = x_stride;
  f.dh_stride = dh_stride;
  f.dx_stride = dx_stride;
  f.T = T;
  f.C = C;
  f.F = F;
  f.act = act;
  f.dtype = dtype;
  return from_cuda(dtype == LA_F32 ? la::ffn_tc32_backward(f, workspace, st) : la::ffn_tc_backward(f, workspace, st));
}

}  // extern "C"
