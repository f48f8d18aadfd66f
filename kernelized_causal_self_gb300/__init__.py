"""Thin Python binding over the C ABI in ``include/la.h``.

Argument marshalling only: every tensor is checked for shape and dtype against
the layouts of ``include/la.h`` (sizes taken from ``q`` and ``v``), then for
being a contiguous CUDA tensor on ``q``'s device, since the library sees only
raw pointers; their ``data_ptr()`` and the current CUDA stream are handed to the
shared library, and outputs/workspaces are allocated with PyTorch (the caller's
allocator). Every step of the computation runs in the library's CUDA kernels;
there is no fallback. If the library is missing the calls raise.
"""

import contextlib
import ctypes
import functools
import os

__all__ = [
    "la_forward", "la_prefill", "la_extend", "la_extend_packed", "la_backward", "la_decode_step",
    "la_forward_workspace_bytes", "la_backward_workspace_bytes",
    "la_workspace_status", "la_status_string", "la_kernel_launches", "library_path",
    "load_library",
    "LAError", "LA_OK", "LA_ERR_INVALID_ARG", "LA_ERR_WORKSPACE", "LA_ERR_CUDA",
    "LA_ERR_TIMEOUT", "LA_ERR_TOO_LARGE", "LA_F32", "LA_BF16", "la_forward_noalloc",
    "la_forward_noalloc_status", "la_workspace_wait_site",
    "la_state_sums", "la_forward_shard", "la_backward_shard_q", "la_backward_shard_kv",
    "la_forward_poly2", "la_poly2_workspace_bytes", "la_forward_rff", "la_rff_workspace_bytes",
    "LA_SITE_FORWARD_LOAD", "LA_SITE_BACKWARD_LOAD",
    "la_forward_gated", "la_prefill_gated", "la_extend_gated", "la_decode_step_gated",
    "la_backward_gated", "la_gated_workspace_bytes", "la_gated_backward_workspace_bytes",
    "la_rotary", "la_rotary_freqs", "la_norm_gate", "la_norm_gate_backward",
    "la_norm_gate_workspace_bytes",
]

LA_OK, LA_ERR_INVALID_ARG, LA_ERR_WORKSPACE, LA_ERR_CUDA, LA_ERR_TIMEOUT = 0, 1, 2, 3, 4
LA_ERR_TOO_LARGE = 5
LA_F32, LA_BF16 = 0, 1
LA_SITE_FORWARD_LOAD, LA_SITE_FORWARD_FUSED_LOAD, LA_SITE_BACKWARD_LOAD = 11, 16, 21

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "_build", "liblagb300.so")
_lib = None

_c_int, _c_size, _vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p

_SIGNATURES = {
    "la_status_string": (ctypes.c_char_p, [_c_int]),
    "la_version": (_c_int, []),
    "la_kernel_launches": (ctypes.c_ulonglong, []),
    "la_forward_workspace_bytes": (_c_size, [_c_int] * 7),
    "la_backward_workspace_bytes": (_c_size, [_c_int] * 7),
    "la_forward": (_c_int, [_vp] * 4 + [_c_int] * 7 + [_vp, _c_size, _vp]),
    "la_prefill": (_c_int, [_vp] * 6 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_extend": (_c_int, [_vp] * 8 + [_c_int] * 7 + [_vp, _c_size, _vp]),
    "la_extend_packed": (_c_int, [_vp] * 8 + [_c_int] * 8 + [_vp, _c_size, _vp]),
    "la_backward": (_c_int, [_vp] * 7 + [_c_int] * 7 + [_vp, _c_size, _vp]),
    "la_decode_step": (_c_int, [_vp] * 6 + [_c_int] * 5 + [_vp]),
    "la_workspace_status": (_c_int, [_vp, _c_size, _vp]),
    "la_forward_noalloc": (_c_int, [_vp] * 4 + [_c_int] * 7 + [_vp]),
    "la_forward_noalloc_status": (_c_int, [_vp]),
    "la_state_sums": (_c_int, [_vp] * 4 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_poly2_workspace_bytes": (_c_size, [_c_int] * 7),
    "la_rff_workspace_bytes": (_c_size, [_c_int] * 8),
    "la_forward_rff": (_c_int, [_vp] * 6 + [_c_int] * 8 + [_vp, _c_size, _vp]),
    "la_backward_from_forward": (_c_int, [_vp] * 7 + [_c_int] * 7 + [_vp, _c_size, _vp, _c_size,
                                                                     _vp]),
    "la_forward_poly2": (_c_int, [_vp] * 4 + [_c_int] * 7 + [_vp, _c_size, _vp]),
    "la_forward_shard": (_c_int, [_vp] * 6 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_backward_shard_q": (_c_int, [_vp] * 9 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_backward_shard_kv": (_c_int, [_vp] * 8 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_gated_workspace_bytes": (_c_size, [_c_int] * 6),
    "la_gated_backward_workspace_bytes": (_c_size, [_c_int] * 6),
    "la_forward_gated": (_c_int, [_vp] * 7 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_extend_gated": (_c_int, [_vp] * 8 + [_c_int] * 7 + [_vp, _c_size, _vp]),
    "la_decode_step_gated": (_c_int, [_vp] * 7 + [_c_int] * 6 + [_vp]),
    "la_backward_gated": (_c_int, [_vp] * 12 + [_c_int] * 6 + [_vp, _c_size, _vp]),
    "la_rotary": (_c_int, [_vp] * 10 + [ctypes.c_longlong] * 2 + [_c_int] * 8
                  + [ctypes.c_float, _c_int, _vp]),
    "la_norm_gate": (_c_int, [_vp] * 6 + [_c_int] * 5 + [ctypes.c_float, _c_int, _vp]),
    "la_norm_gate_workspace_bytes": (_c_size, [_c_int] * 4),
    "la_norm_gate_backward": (_c_int, [_vp] * 10 + [_c_int] * 5
                              + [ctypes.c_float, _c_int, _vp, _c_size, _vp]),
    "la_debug_noalloc_set_status": (_c_int, [_c_int, _c_int, _vp]),
    "la_workspace_wait_site": (_c_int, [_vp, _c_size, _vp]),
    "la_debug_forward_fault": (_c_int, [_vp] * 4 + [_c_int] * 7 + [_vp, _c_size, _c_int,
                                                                    ctypes.c_ulonglong, _vp]),
    "la_debug_forward_fused_fault": (_c_int, [_vp] * 4 + [_c_int] * 7 + [_vp, _c_size, _c_int,
                                                                          ctypes.c_ulonglong, _vp]),
    "la_debug_backward_fault": (_c_int, [_vp] * 7 + [_c_int] * 7 + [_vp, _c_size, _c_int,
                                                                     ctypes.c_ulonglong, _vp]),
}


class LAError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn}: {la_status_string(status)} (status {status})")


def library_path():
    return _LIB_PATH


def load_library():
    """Load the shared library (ctypes); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"CUDA library not built: {_LIB_PATH} is missing "
                "(run `python -c 'import __graft_entry__ as g; g.build()'`)")
        lib = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype, fn.argtypes = res, args
        _lib = lib
    return _lib


def la_status_string(status):
    return load_library().la_status_string(int(status)).decode()


def _check(fn, status):
    if status != LA_OK:
        raise LAError(fn, status)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return LA_F32
    if t.dtype == torch.bfloat16:
        return LA_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (float32 or bfloat16)")


def _on_device(device):
    """Context that makes `device` current around a library call: the library looks up
    per-device state (la_forward_noalloc's fixed scratch) on the current device, and the
    stream it is handed belongs to `device`."""
    import torch
    if device.index is not None and torch.cuda.current_device() == device.index:
        return _ALREADY
    return torch.cuda.device(device)


_ALREADY = contextlib.nullcontext()


def _stream_ptr(device):
    """The current stream of `device`, as the library takes it (without the Stream object that
    torch.cuda.current_stream would build, which costs as much as a small launch)."""
    import torch
    if device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _need_cuda(*ts, device=None):
    """Contiguous CUDA tensors, all on `device` (default: the first one's)."""
    index = None if device is None else device.index
    for t in ts:
        at = t.get_device()  # (an index: a device object costs more than the comparison)
        if at < 0:
            raise ValueError("tensors must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
        if index is None:
            index, device = at, t.device
        elif at != index:
            raise ValueError(f"tensors must all be on {device}, got one on {t.device}")


def _expect(fn, name, t, shape, dtype):
    """`t` has exactly `shape` and `dtype` (the library reads and writes that many elements)."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{fn}: {name} must be {dtype} of shape {tuple(shape)}, "
                         f"got {t.dtype} of shape {tuple(t.shape)}")


def _dims(fn, q, v, rank):
    """(leading sizes of q, D, M) for q [..., D], v [..., M] of the given rank."""
    if q.dim() != rank or v.dim() != rank:
        raise ValueError(f"{fn}: q and v must have {rank} dimensions")
    return tuple(q.shape[:-1]), q.shape[-1], v.shape[-1]


def _workspace(nbytes, device, workspace):
    import torch
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError("workspace too small")
        _need_cuda(workspace, device=device)
        return workspace
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def la_kernel_launches():
    """Kernels launched by the library in this process so far."""
    return int(load_library().la_kernel_launches())


def la_forward_workspace_bytes(B, H, N, D, M, causal=True, dtype=LA_BF16):
    return load_library().la_forward_workspace_bytes(B, H, N, D, M, int(bool(causal)), dtype)


def la_backward_workspace_bytes(B, H, N, D, M, causal=True, dtype=LA_BF16):
    return load_library().la_backward_workspace_bytes(B, H, N, D, M, int(bool(causal)), dtype)


def la_forward(q, k, v, causal=True, out=None, workspace=None):
    """out[B,H,N,M] = kernelized attention of q, k [B,H,N,D] and v [B,H,N,M]."""
    import torch
    (B, H, N), D, M = _dims("la_forward", q, v, 4)
    _expect("la_forward", "k", k, q.shape, q.dtype)
    _expect("la_forward", "v", v, (B, H, N, M), q.dtype)
    if out is not None:
        _expect("la_forward", "out", out, (B, H, N, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, *([] if out is None else [out]))
    lib = load_library()
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    nbytes = lib.la_forward_workspace_bytes(B, H, N, D, M, int(bool(causal)), dt)
    ws = _workspace(nbytes, q.device, workspace)
    with _on_device(q.device):
        st = lib.la_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H, N, D,
                            M, int(bool(causal)), dt, ws.data_ptr(),
                            ws.numel() * ws.element_size(), _stream_ptr(q.device))
    _check("la_forward", st)
    return out


def la_forward_noalloc(q, k, v, causal=True, out=None):
    """la_forward without a workspace: the library's fixed device scratch array is used.

    For callers that cannot allocate device memory. Calls that overlap on the
    GPU share that array and race; the first call on a device must not be
    made during stream capture.
    """
    import torch
    (B, H, N), D, M = _dims("la_forward_noalloc", q, v, 4)
    _expect("la_forward_noalloc", "k", k, q.shape, q.dtype)
    _expect("la_forward_noalloc", "v", v, (B, H, N, M), q.dtype)
    if out is not None:
        _expect("la_forward_noalloc", "out", out, (B, H, N, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, *([] if out is None else [out]))
    lib = load_library()
    if out is None:
        out = torch.empty((B, H, N, M), dtype=q.dtype, device=q.device)
    with _on_device(q.device):
        st = lib.la_forward_noalloc(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H,
                                    N, D, M, int(bool(causal)), dt, _stream_ptr(q.device))
    _check("la_forward_noalloc", st)
    return out


def la_prefill(q, k, v, out=None, S=None, Z=None, workspace=None):
    """Causal forward plus the final float32 state S [B,H,D,M], Z [B,H,D]."""
    import torch
    fn, f32 = "la_prefill", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    given = [(n, t) for n, t in (("out", out), ("S", S), ("Z", Z)) if t is not None]
    for name, t in given:
        _expect(fn, name, t, {"out": (B, H, N, M), "S": (B, H, D, M), "Z": (B, H, D)}[name],
                q.dtype if name == "out" else f32)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, *[t for _, t in given])
    lib = load_library()
    dev = q.device
    out = torch.empty((B, H, N, M), dtype=q.dtype, device=dev) if out is None else out
    S = torch.empty((B, H, D, M), dtype=f32, device=dev) if S is None else S
    Z = torch.empty((B, H, D), dtype=f32, device=dev) if Z is None else Z
    nbytes = lib.la_forward_workspace_bytes(B, H, N, D, M, 1, dt)
    ws = _workspace(nbytes, dev, workspace)
    with _on_device(dev):
        st = lib.la_prefill(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), S.data_ptr(),
                            Z.data_ptr(), B, H, N, D, M, dt, ws.data_ptr(),
                            ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check("la_prefill", st)
    return out, S, Z


def la_extend(q, k, v, S_pool, Z_pool, slots=None, lens=None, out=None, workspace=None):
    """Causal forward over new tokens of B streams continuing from stored state.

    S_pool [P,H,D,M], Z_pool [P,H,D] float32 hold per-stream states; stream b uses
    entry slots[b] (int32 device tensor of B distinct entries; None: entry b) and
    its entry is advanced past its tokens in place: the first lens[b] of the N
    (int32 device tensor; None: all N). Returns out [B,H,N,M]; rows at or past
    lens[b] are unspecified.
    """
    import torch
    fn, f32 = "la_extend", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    if S_pool.dim() != 4:
        raise ValueError(f"{fn}: S_pool must be [pool, H, D, M]")
    P = S_pool.shape[0]
    _expect(fn, "S_pool", S_pool, (P, H, D, M), f32)
    _expect(fn, "Z_pool", Z_pool, (P, H, D), f32)
    if out is not None:
        _expect(fn, "out", out, (B, H, N, M), q.dtype)
    for name, t in (("slots", slots), ("lens", lens)):
        if t is not None and (t.dtype != torch.int32 or t.numel() != B):
            raise ValueError(f"{name} must be a contiguous int32 tensor of B entries")
    dt = _dtype_code(q)
    _need_cuda(q, k, v, S_pool, Z_pool,
               *[t for t in (out, slots, lens) if t is not None])
    lib = load_library()
    dev = q.device
    out = torch.empty((B, H, N, M), dtype=q.dtype, device=dev) if out is None else out
    nbytes = lib.la_forward_workspace_bytes(B, H, N, D, M, 1, dt)
    ws = _workspace(nbytes, dev, workspace)
    with _on_device(dev):
        st = lib.la_extend(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                           S_pool.data_ptr(), Z_pool.data_ptr(),
                           0 if slots is None else slots.data_ptr(),
                           0 if lens is None else lens.data_ptr(), P,
                           B, H, N, D, M, dt, ws.data_ptr(), ws.numel() * ws.element_size(),
                           _stream_ptr(dev))
    _check("la_extend", st)
    return out


def la_extend_packed(q, k, v, S_pool, Z_pool, cu_seqlens, max_len, slots=None, out=None,
                     workspace=None):
    """la_extend on a packed batch: q, k [T,H,D] and v [T,H,M], stream b in rows
    cu_seqlens[b] .. cu_seqlens[b+1]-1 (int32 device tensor of B + 1 offsets), each
    stream at most max_len tokens. Returns out [T,H,M] (rows of no stream are left
    as they were in `out`, uninitialised if it is None).
    """
    import torch
    fn, f32 = "la_extend_packed", torch.float32
    (T, H), D, M = _dims(fn, q, v, 3)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (T, H, M), q.dtype)
    if S_pool.dim() != 4:
        raise ValueError(f"{fn}: S_pool must be [pool, H, D, M]")
    P = S_pool.shape[0]
    _expect(fn, "S_pool", S_pool, (P, H, D, M), f32)
    _expect(fn, "Z_pool", Z_pool, (P, H, D), f32)
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be a contiguous int32 tensor of B + 1 offsets")
    B = cu_seqlens.numel() - 1
    if slots is not None and (slots.dtype != torch.int32 or slots.numel() != B):
        raise ValueError("slots must be a contiguous int32 tensor of B entries")
    if out is not None:
        _expect(fn, "out", out, (T, H, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, S_pool, Z_pool, cu_seqlens,
               *[t for t in (out, slots) if t is not None])
    lib = load_library()
    dev = q.device
    out = torch.empty((T, H, M), dtype=q.dtype, device=dev) if out is None else out
    nbytes = lib.la_forward_workspace_bytes(B, H, max_len, D, M, 1, dt)
    ws = _workspace(nbytes, dev, workspace)
    with _on_device(dev):
        st = lib.la_extend_packed(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  S_pool.data_ptr(), Z_pool.data_ptr(),
                                  0 if slots is None else slots.data_ptr(),
                                  cu_seqlens.data_ptr(), P, B, H, T, int(max_len), D, M, dt,
                                  ws.data_ptr(), ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check(fn, st)
    return out


def la_backward(q, k, v, dout, causal=True, dq=None, dk=None, dv=None, workspace=None,
                fwd_workspace=None):
    """float32 gradients (dq, dk, dv) of sum(dout * la_forward(q, k, v)).

    fwd_workspace: the workspace of a la_forward call on the same q, k, v (and causal), not
    reused since; its segment states are then read instead of recomputed
    (la_backward_from_forward)."""
    import torch
    fn, f32 = "la_backward", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    _expect(fn, "dout", dout, (B, H, N, M), q.dtype)
    given = [(n, t) for n, t in (("dq", dq), ("dk", dk), ("dv", dv)) if t is not None]
    for name, t in given:
        _expect(fn, name, t, (B, H, N, M) if name == "dv" else (B, H, N, D), f32)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, dout, *[t for _, t in given])
    lib = load_library()
    dev = q.device
    dq = torch.empty((B, H, N, D), dtype=f32, device=dev) if dq is None else dq
    dk = torch.empty((B, H, N, D), dtype=f32, device=dev) if dk is None else dk
    dv = torch.empty((B, H, N, M), dtype=f32, device=dev) if dv is None else dv
    nbytes = lib.la_backward_workspace_bytes(B, H, N, D, M, int(bool(causal)), dt)
    ws = _workspace(nbytes, dev, workspace)
    if fwd_workspace is not None:
        _need_cuda(fwd_workspace, device=dev)
    with _on_device(dev):
        if fwd_workspace is None:
            st = lib.la_backward(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                 dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, H, N, D, M,
                                 int(bool(causal)), dt, ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream_ptr(dev))
        else:
            st = lib.la_backward_from_forward(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(), dq.data_ptr(),
                dk.data_ptr(), dv.data_ptr(), B, H, N, D, M, int(bool(causal)), dt,
                fwd_workspace.data_ptr(), fwd_workspace.numel() * fwd_workspace.element_size(),
                ws.data_ptr(), ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check("la_backward", st)
    return dq, dk, dv


def la_decode_step(q, k, v, S, Z, out=None):
    """One recurrent step: q, k [S,H,D], v [S,H,M]; S, Z updated in place; returns out."""
    import torch
    fn, f32 = "la_decode_step", torch.float32
    (n, H), D, M = _dims(fn, q, v, 3)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (n, H, M), q.dtype)
    _expect(fn, "S", S, (n, H, D, M), f32)
    _expect(fn, "Z", Z, (n, H, D), f32)
    if out is not None:
        _expect(fn, "out", out, (n, H, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, S, Z, *([] if out is None else [out]))
    lib = load_library()
    out = torch.empty((n, H, M), dtype=q.dtype, device=q.device) if out is None else out
    with _on_device(q.device):
        st = lib.la_decode_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), S.data_ptr(),
                                Z.data_ptr(), out.data_ptr(), n, H, D, M, dt,
                                _stream_ptr(q.device))
    _check("la_decode_step", st)
    return out


def la_workspace_status(workspace):
    """Synchronise and read (then clear) the status word a call left in `workspace`."""
    lib = load_library()
    with _on_device(workspace.device):
        return lib.la_workspace_status(workspace.data_ptr(),
                                       workspace.numel() * workspace.element_size(),
                                       _stream_ptr(workspace.device))


def la_workspace_wait_site(workspace):
    """Synchronise and read the code of the bounded wait that last gave up in the call that
    used `workspace` (0: none). Nothing is cleared."""
    lib = load_library()
    with _on_device(workspace.device):
        return lib.la_workspace_wait_site(workspace.data_ptr(),
                                          workspace.numel() * workspace.element_size(),
                                          _stream_ptr(workspace.device))


def la_forward_noalloc_status(device=None):
    """Synchronise and read (then clear) the status word of la_forward_noalloc's fixed
    scratch on `device` (default: the current CUDA device)."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    lib = load_library()
    with _on_device(dev):
        return lib.la_forward_noalloc_status(_stream_ptr(dev))


# ------------------------------------------------------------ sequence shards

def _state_shapes(B, H, D, M):
    return (B, H, D, M), (B, H, D)


def la_state_sums(k, v, S=None, Z=None, workspace=None):
    """A shard's own sums S = sum_j phi(k_j) v_j^T [B,H,D,M], Z = sum_j phi(k_j) [B,H,D]."""
    import torch
    fn, f32 = "la_state_sums", torch.float32
    (B, H, N), D, M = _dims(fn, k, v, 4)
    _expect(fn, "v", v, (B, H, N, M), k.dtype)
    sS, sZ = _state_shapes(B, H, D, M)
    for name, t, shp in (("S", S, sS), ("Z", Z, sZ)):
        if t is not None:
            _expect(fn, name, t, shp, f32)
    dt = _dtype_code(k)
    _need_cuda(k, v, *[t for t in (S, Z) if t is not None])
    lib = load_library()
    dev = k.device
    S = torch.empty(sS, dtype=f32, device=dev) if S is None else S
    Z = torch.empty(sZ, dtype=f32, device=dev) if Z is None else Z
    ws = _workspace(lib.la_forward_workspace_bytes(B, H, N, D, M, 1, dt), dev, workspace)
    with _on_device(dev):
        st = lib.la_state_sums(k.data_ptr(), v.data_ptr(), S.data_ptr(), Z.data_ptr(), B, H, N, D,
                               M, dt, ws.data_ptr(), ws.numel() * ws.element_size(),
                               _stream_ptr(dev))
    _check(fn, st)
    return S, Z


def la_forward_shard(q, k, v, S0, Z0, out=None, workspace=None):
    """Causal forward of a shard's tokens after the state (S0, Z0) of the tokens before them."""
    import torch
    fn, f32 = "la_forward_shard", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    sS, sZ = _state_shapes(B, H, D, M)
    _expect(fn, "S0", S0, sS, f32)
    _expect(fn, "Z0", Z0, sZ, f32)
    if out is not None:
        _expect(fn, "out", out, (B, H, N, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, S0, Z0, *([] if out is None else [out]))
    lib = load_library()
    dev = q.device
    out = torch.empty((B, H, N, M), dtype=q.dtype, device=dev) if out is None else out
    ws = _workspace(lib.la_forward_workspace_bytes(B, H, N, D, M, 1, dt), dev, workspace)
    with _on_device(dev):
        st = lib.la_forward_shard(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                                  S0.data_ptr(), Z0.data_ptr(), B, H, N, D, M, dt, ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check(fn, st)
    return out


def la_backward_shard_q(q, k, v, dout, S0, Z0, dq=None, R_own=None, r_own=None, workspace=None):
    """First backward pass of a shard: (dq, R_own, r_own, workspace); pass the workspace on
    to la_backward_shard_kv."""
    import torch
    fn, f32 = "la_backward_shard_q", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    _expect(fn, "dout", dout, (B, H, N, M), q.dtype)
    sS, sZ = _state_shapes(B, H, D, M)
    _expect(fn, "S0", S0, sS, f32)
    _expect(fn, "Z0", Z0, sZ, f32)
    given = [(n, t, shp) for n, t, shp in (("dq", dq, (B, H, N, D)), ("R_own", R_own, sS),
                                           ("r_own", r_own, sZ)) if t is not None]
    for name, t, shp in given:
        _expect(fn, name, t, shp, f32)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, dout, S0, Z0, *[t for _, t, _ in given])
    lib = load_library()
    dev = q.device
    dq = torch.empty((B, H, N, D), dtype=f32, device=dev) if dq is None else dq
    R_own = torch.empty(sS, dtype=f32, device=dev) if R_own is None else R_own
    r_own = torch.empty(sZ, dtype=f32, device=dev) if r_own is None else r_own
    ws = _workspace(lib.la_backward_workspace_bytes(B, H, N, D, M, 1, dt), dev, workspace)
    with _on_device(dev):
        st = lib.la_backward_shard_q(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                     dq.data_ptr(), S0.data_ptr(), Z0.data_ptr(), R_own.data_ptr(),
                                     r_own.data_ptr(), B, H, N, D, M, dt, ws.data_ptr(),
                                     ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check(fn, st)
    return dq, R_own, r_own, ws


def la_backward_shard_kv(q, k, v, dout, R0, r0, workspace, dk=None, dv=None):
    """Second backward pass of a shard: (dk, dv) given the reverse sums (R0, r0) of the tokens
    after it and the workspace of its la_backward_shard_q call."""
    import torch
    fn, f32 = "la_backward_shard_kv", torch.float32
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    _expect(fn, "dout", dout, (B, H, N, M), q.dtype)
    sS, sZ = _state_shapes(B, H, D, M)
    _expect(fn, "R0", R0, sS, f32)
    _expect(fn, "r0", r0, sZ, f32)
    given = [(n, t, shp) for n, t, shp in (("dk", dk, (B, H, N, D)), ("dv", dv, (B, H, N, M)))
             if t is not None]
    for name, t, shp in given:
        _expect(fn, name, t, shp, f32)
    dt = _dtype_code(q)
    lib = load_library()
    nbytes = lib.la_backward_workspace_bytes(B, H, N, D, M, 1, dt)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise ValueError(f"{fn}: workspace too small")
    _need_cuda(q, k, v, dout, R0, r0, workspace, *[t for _, t, _ in given])
    dev = q.device
    dk = torch.empty((B, H, N, D), dtype=f32, device=dev) if dk is None else dk
    dv = torch.empty((B, H, N, M), dtype=f32, device=dev) if dv is None else dv
    with _on_device(dev):
        st = lib.la_backward_shard_kv(q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                                      dk.data_ptr(), dv.data_ptr(), R0.data_ptr(), r0.data_ptr(),
                                      B, H, N, D, M, dt, workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream_ptr(dev))
    _check(fn, st)
    return dk, dv


# ---------------------------------------------- degree-2 polynomial feature map

def la_poly2_workspace_bytes(B, H, N, D, M, causal=True, dtype=LA_BF16):
    return load_library().la_poly2_workspace_bytes(B, H, N, D, M, int(bool(causal)), dtype)


def la_forward_poly2(q, k, v, causal=True, out=None, workspace=None):
    """out[B,H,N,M] = causal attention with sim(q, k) = (q . k)^2 (feature map vec(x x^T))."""
    import torch
    fn = "la_forward_poly2"
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    if out is not None:
        _expect(fn, "out", out, (B, H, N, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, *([] if out is None else [out]))
    lib = load_library()
    dev = q.device
    out = torch.empty((B, H, N, M), dtype=q.dtype, device=dev) if out is None else out
    ws = _workspace(lib.la_poly2_workspace_bytes(B, H, N, D, M, int(bool(causal)), dt), dev,
                    workspace)
    with _on_device(dev):
        st = lib.la_forward_poly2(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), B, H,
                                  N, D, M, int(bool(causal)), dt, ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check(fn, st)
    return out


# ------------------------------------------------------ random Fourier features

def la_rff_workspace_bytes(B, H, N, D, M, F, causal=True, dtype=LA_BF16):
    return load_library().la_rff_workspace_bytes(B, H, N, D, M, F, int(bool(causal)), dtype)


def la_forward_rff(q, k, v, W, bias, causal=True, out=None, workspace=None):
    """out[B,H,N,M] = attention with phi(x) = sqrt(2/F) cos(W x + bias) (random Fourier
    features of the RBF kernel); W [F, D] in q's dtype, bias [F] float32."""
    import torch
    fn = "la_forward_rff"
    (B, H, N), D, M = _dims(fn, q, v, 4)
    _expect(fn, "k", k, q.shape, q.dtype)
    _expect(fn, "v", v, (B, H, N, M), q.dtype)
    if W.dim() != 2:
        raise ValueError(f"{fn}: W must be [F, D]")
    F = W.shape[0]
    _expect(fn, "W", W, (F, D), q.dtype)
    _expect(fn, "bias", bias, (F,), torch.float32)
    if out is not None:
        _expect(fn, "out", out, (B, H, N, M), q.dtype)
    dt = _dtype_code(q)
    _need_cuda(q, k, v, W, bias, *([] if out is None else [out]))
    lib = load_library()
    dev = q.device
    out = torch.empty((B, H, N, M), dtype=q.dtype, device=dev) if out is None else out
    ws = _workspace(lib.la_rff_workspace_bytes(B, H, N, D, M, F, int(bool(causal)), dt), dev,
                    workspace)
    with _on_device(dev):
        st = lib.la_forward_rff(q.data_ptr(), k.data_ptr(), v.data_ptr(), W.data_ptr(),
                                bias.data_ptr(), out.data_ptr(), B, H, N, D, M, F,
                                int(bool(causal)), dt, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream_ptr(dev))
    _check(fn, st)
    return out


# ---------------------------------------------------------- gated recurrence

def la_gated_workspace_bytes(B, H, N, D, M, dtype=LA_BF16):
    return load_library().la_gated_workspace_bytes(B, H, N, D, M, dtype)


def la_gated_backward_workspace_bytes(B, H, N, D, M, dtype=LA_BF16):
    return load_library().la_gated_backward_workspace_bytes(B, H, N, D, M, dtype)


@functools.lru_cache(maxsize=4096)
def _bytes(query, *dims):
    """A workspace query's answer (it depends on the sizes alone)."""
    return getattr(load_library(), query)(*dims)


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _scratch(like, nbytes, workspace):
    """(workspace, its bytes): the caller's, or one of `nbytes` if any are needed."""
    if workspace is not None:
        workspace = _workspace(nbytes, like.device, workspace)
        return workspace, workspace.numel() * workspace.element_size()
    import torch
    return (torch.empty(nbytes, dtype=torch.uint8, device=like.device) if nbytes else None), nbytes


def _check_gated(fn, q, k, v, g, rank):
    lead, last, dt = q.shape, v.shape, q.dtype
    if len(lead) != rank or len(last) != rank:
        raise ValueError(f"{fn}: q and v must have {rank} dimensions")
    if k.shape != lead or k.dtype != dt:
        _expect(fn, "k", k, lead, dt)
    dims = (*lead, last[-1])
    lead = lead[:-1]
    if last[:-1] != lead or v.dtype != dt:
        _expect(fn, "v", v, (*lead, last[-1]), dt)
    if g.shape != lead or g.dtype != dt:
        _expect(fn, "g", g, lead, dt)
    return dims, _dtype_code(q)


def _apart(fn, name, t, other, o, same_ok):
    """Two float32 states do not share memory (same_ok: or are the same)."""
    at, to = t.data_ptr(), o.data_ptr()
    if abs(at - to) < 4 * t.numel() and not (same_ok and at == to):
        raise ValueError(f"{fn}: {name} shares memory with {other}")


def _forward_gated(fn, q, k, v, g, S0, out, S, want_state, workspace):
    import torch
    (B, H, N, D, M), dt = _check_gated(fn, q, k, v, g, 4)
    given = []
    for name, t in (("S0", S0), ("S", S)):
        if t is not None:
            _expect(fn, name, t, (B, H, D, M), torch.float32)
            given.append(t)
    if S0 is not None and S is not None:
        _apart(fn, "S", S, "S0", S0, True)
    if out is not None:
        _expect(fn, "out", out, v.shape, q.dtype)
        given.append(out)
    _need_cuda(q, k, v, g, *given)
    lib = load_library()
    dev = q.device
    out = torch.empty_like(v) if out is None else out
    if want_state and S is None:
        S = torch.empty((B, H, D, M), dtype=torch.float32, device=dev)
    need = _bytes("la_gated_workspace_bytes", B, H, N, D, M, dt)
    ws, nbytes = _scratch(q, need if need > 256 else 0, workspace)  # (256: a header it leaves alone)
    with _on_device(dev):
        st = lib.la_forward_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                  out.data_ptr(), _ptr(S0), _ptr(S), B, H, N, D, M, dt, _ptr(ws),
                                  nbytes, _stream_ptr(dev))
    _check(fn, st)
    return out, S


def la_forward_gated(q, k, v, g, S0=None, out=None, workspace=None):
    """out[B,H,N,M]: out_t = S_t^T q_t with S_t = exp(g_t) S_{t-1} + k_t v_t^T.

    q, k [B,H,N,D], v [B,H,N,M]; g [B,H,N], in q's dtype: log-decays, normally <= 0.
    S0 [B,H,D,M] float32: the state before the first token (None: zero)."""
    return _forward_gated("la_forward_gated", q, k, v, g, S0, out, None, False, workspace)[0]


def la_prefill_gated(q, k, v, g, S0=None, out=None, S=None, workspace=None):
    """la_forward_gated plus the state S [B,H,D,M] (float32) after the last token; S may be S0."""
    return _forward_gated("la_prefill_gated", q, k, v, g, S0, out, S, True, workspace)


def _check_pool(fn, S_pool, H, D, M, B, slots):
    import torch
    shape = S_pool.shape
    if len(shape) != 4:
        raise ValueError(f"{fn}: S_pool must be [pool, H, D, M]")
    if shape[1:] != (H, D, M) or S_pool.dtype != torch.float32:
        _expect(fn, "S_pool", S_pool, (shape[0], H, D, M), torch.float32)
    if slots is not None and (slots.dtype != torch.int32 or slots.numel() != B):
        raise ValueError("slots must be a contiguous int32 tensor of B entries")
    return shape[0]


def la_extend_gated(q, k, v, g, S_pool, slots=None, lens=None, out=None, workspace=None):
    """la_forward_gated over new tokens of B streams, from and to their states in a pool.

    S_pool [P,H,D,M] float32; stream b uses entry slots[b] (int32 device tensor of B distinct
    entries; None: entry b), advanced in place past the first lens[b] of the N tokens (int32
    device tensor; None: all N). Returns out [B,H,N,M]; its rows at or past lens[b] are left
    as they were (uninitialised if `out` is None)."""
    import torch
    fn = "la_extend_gated"
    (B, H, N, D, M), dt = _check_gated(fn, q, k, v, g, 4)
    pool = _check_pool(fn, S_pool, H, D, M, B, slots)
    if lens is not None and (lens.dtype != torch.int32 or lens.numel() != B):
        raise ValueError("lens must be a contiguous int32 tensor of B entries")
    if out is not None:
        _expect(fn, "out", out, v.shape, q.dtype)
    _need_cuda(q, k, v, g, S_pool, *[t for t in (out, slots, lens) if t is not None])
    lib = load_library()
    dev = q.device
    out = torch.empty_like(v) if out is None else out
    ws, nbytes = _scratch(q, max(_bytes("la_gated_workspace_bytes", B, H, N, D, M, dt), 256), workspace)
    with _on_device(dev):
        st = lib.la_extend_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                 out.data_ptr(), S_pool.data_ptr(), _ptr(slots), _ptr(lens), pool,
                                 B, H, N, D, M, dt, ws.data_ptr(), nbytes, _stream_ptr(dev))
    _check(fn, st)
    return out


def la_decode_step_gated(q, k, v, g, S_pool, slots=None, out=None):
    """One token of each of n streams: q, k [n,H,D], v [n,H,M], g [n,H]; the states in S_pool
    [P,H,D,M] (entries slots, as in la_extend_gated) are updated in place; returns out [n,H,M]."""
    import torch
    fn = "la_decode_step_gated"
    (n, H, D, M), dt = _check_gated(fn, q, k, v, g, 3)
    pool = _check_pool(fn, S_pool, H, D, M, n, slots)
    if out is None:
        _need_cuda(q, k, v, g, S_pool)
        out = torch.empty_like(v)
    else:
        if out.shape != v.shape or out.dtype != v.dtype:
            _expect(fn, "out", out, v.shape, q.dtype)
        _need_cuda(q, k, v, g, S_pool, out)
    if slots is not None:
        _need_cuda(slots, device=q.device)
    lib = load_library()
    dev = q.device
    with _on_device(dev):
        st = lib.la_decode_step_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                      S_pool.data_ptr(), _ptr(slots), out.data_ptr(), pool, n, H,
                                      D, M, dt, _stream_ptr(dev))
    _check(fn, st)
    return out


def la_backward_gated(q, k, v, g, dout, S0=None, dS=None, dq=None, dk=None, dv=None, dg=None,
                      dS0=None, workspace=None):
    """Gradients of sum(dout * out) + sum(dS * S) of la_prefill_gated(q, k, v, g, S0): (dq, dk,
    dv, dg) in the inputs' dtype, and dS0 [B,H,D,M] (float32) behind them if S0 is given.

    dS [B,H,D,M] float32: the gradient with respect to the final state (None: zero). dS0 may be
    dS itself."""
    import torch
    fn, f32 = "la_backward_gated", torch.float32
    (B, H, N, D, M), dt = _check_gated(fn, q, k, v, g, 4)
    if dout.shape != v.shape or dout.dtype != v.dtype:
        _expect(fn, "dout", dout, v.shape, v.dtype)
    given = []
    for name, t in (("S0", S0), ("dS", dS), ("dS0", dS0)):
        if t is not None:
            _expect(fn, name, t, (B, H, D, M), f32)
            given.append(t)
    if dS0 is not None:
        if S0 is None:
            raise ValueError(f"{fn}: dS0 without S0")
        _apart(fn, "dS0", dS0, "S0", S0, False)
        if dS is not None:
            _apart(fn, "dS0", dS0, "dS", dS, True)
    for name, t, like in (("dq", dq, q), ("dk", dk, q), ("dv", dv, v), ("dg", dg, g)):
        if t is not None:
            _expect(fn, name, t, like.shape, q.dtype)
            given.append(t)
    _need_cuda(q, k, v, g, dout, *given)
    lib = load_library()
    dev = q.device
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    dg = torch.empty_like(g) if dg is None else dg
    if S0 is not None and dS0 is None:
        dS0 = torch.empty_like(S0)
    ws, nbytes = _scratch(q, _bytes("la_gated_backward_workspace_bytes", B, H, N, D, M, dt), workspace)
    with _on_device(dev):
        st = lib.la_backward_gated(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
                                   dout.data_ptr(), _ptr(S0), _ptr(dS), dq.data_ptr(),
                                   dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), _ptr(dS0), B, H,
                                   N, D, M, dt, _ptr(ws), nbytes, _stream_ptr(dev))
    _check(fn, st)
    return (dq, dk, dv, dg) if S0 is None else (dq, dk, dv, dg, dS0)


# ------------------------------------------- rotary positions, gated head norm

def _need_rows(*ts, device):
    """CUDA tensors on `device` whose last dimension is contiguous (the others strided)."""
    index = device.index
    for t in ts:
        at = t.get_device()
        if at < 0:
            raise ValueError("tensors must be on a CUDA device")
        if at != index:
            raise ValueError(f"tensors must all be on {device}, got one on {t.device}")


@functools.lru_cache(maxsize=1024)
def _long3(a, b, c):
    return (ctypes.c_longlong * 3)(a, b, c)


def _row_strides(fn, name, t, packed=False, written=False):
    """The strides of the batch, head and token of t [B,H,N,*] (packed: [N,H,*]), for the library
    (0 where a dimension has one entry); rows that are written must not overlap."""
    size, stride = t.shape, t.stride()
    if stride[-1] != 1 and size[-1] > 1 and t.numel():
        raise ValueError(f"{fn}: {name}'s last dimension must be contiguous")
    if written and not t.is_contiguous():
        reach = size[-1]
        for st, n in sorted((st, n) for st, n in zip(stride[:-1], size[:-1]) if n > 1):
            if st < reach:
                raise ValueError(f"{fn}: rows of {name} overlap in memory")
            reach = st * (n - 1) + reach
    if packed:
        (n, h, _), (sn, sh, _) = size, stride
        return _long3(0, sh if h > 1 else 0, sn if n > 1 else 0)
    (b, h, n, _), (sb, sh, sn, _) = size, stride
    return _long3(sb if b > 1 else 0, sh if h > 1 else 0, sn if n > 1 else 0)


def la_rotary_freqs(rot_dim, base=10000.0, scaling=None, factor=1.0, original_len=None, slow=1.0,
                    fast=32.0, device="cuda"):
    """(freqs, mscale) for la_rotary: float64 [rot_dim/2] radians per token, base^(-2i/rot_dim),
    for contexts `factor` times longer than those trained on by one of

    scaling=None       as they are;
    scaling="linear"   every frequency divided by factor (positions interpolated);
    scaling="base"     base * factor^(rot_dim/(rot_dim-2)): the slowest pair is divided by
                       factor, the fastest kept;
    scaling="ramp"     pairs that make fewer than `slow` turns in original_len tokens divided
                       by factor, those of more than `fast` turns kept, a linear ramp between;
                       mscale = 0.1 ln(factor) + 1 (1 for the others).
    """
    import math
    import torch
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError("la_rotary_freqs: rot_dim must be even and at least 2")
    if not base > 0 or not factor > 0:
        raise ValueError("la_rotary_freqs: base and factor must be positive")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"la_rotary_freqs: unknown scaling {scaling!r}")
    mscale = 1.0
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2.0))
    freqs = torch.tensor([base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)],
                         dtype=torch.float64)
    if scaling == "linear":
        freqs = freqs / factor
    elif scaling == "ramp":
        if original_len is None or not fast > slow:
            raise ValueError("la_rotary_freqs: a ramp needs original_len and slow < fast")
        turns = original_len * freqs / (2.0 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        freqs = freqs * keep + freqs / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return freqs.to(device), mscale


def la_rotary(q, k, freqs, positions=None, offset=0, interleaved=False, mscale=1.0, inverse=False,
              q_out=None, k_out=None):
    """q and k with the first 2 * len(freqs) elements of each head rotated by their positions.

    q [B,H,N,D] and k [B,Hk,N,D] (or None), or packed [T,H,D] and [T,Hk,D]; any strides with a
    contiguous last dimension. freqs: float64 [R/2] radians per token (la_rotary_freqs). Pairs
    are elements (2i, 2i+1) if interleaved, else (i, i + R/2). positions: int32 [N] or [B,N]
    (packed: [T]); None: offset, offset + 1, ... mscale scales the rotated elements. inverse
    turns the other way: la_rotary(dq, dk, ..., inverse=True) is the gradient. Outputs may be
    the inputs themselves. Returns (q_out, k_out), contiguous unless passed in."""
    import torch
    fn = "la_rotary"
    dt, shape, dtype, dev = _dtype_code(q), q.shape, q.dtype, q.device
    packed = len(shape) == 3
    if packed:
        B = 1
        N, H, D = shape
    elif len(shape) == 4:
        B, H, N, D = shape
    else:
        raise ValueError(f"{fn}: q must have 3 or 4 dimensions")
    qs = _row_strides(fn, "q", q, packed)
    if k is None:
        if k_out is not None:
            raise ValueError(f"{fn}: k_out without k")
        Hk, ks, kos = 0, None, None
    else:
        kshape = k.shape
        Hk = kshape[1] if len(kshape) == len(shape) else -1
        if kshape[0] != shape[0] or kshape[2:] != shape[2:] or Hk < 0 or k.dtype != dtype:
            _expect(fn, "k", k, (shape[0], Hk, *shape[2:]), dtype)
        ks = _row_strides(fn, "k", k, packed)
    if freqs.dtype != torch.float64 or len(freqs.shape) != 1 or not freqs.is_contiguous():
        raise ValueError(f"{fn}: freqs must be a contiguous float64 tensor of R/2 entries")
    if not -2 ** 62 <= offset <= 2 ** 62 or offset != int(offset):
        raise ValueError(f"{fn}: offset must be a whole number within +-2^62")
    pos_b = 0
    if positions is not None:
        p = positions.shape
        if p != (N,):
            pos_b = N
        if (pos_b and (packed or p != (B, N))) or positions.dtype != torch.int32 \
                or not positions.is_contiguous():
            raise ValueError(f"{fn}: positions must be a contiguous int32 tensor of [N] or [B, N]")
    if q_out is not None:
        _expect(fn, "q_out", q_out, shape, dtype)
        qos = _row_strides(fn, "q_out", q_out, packed, True)
    if k_out is not None:
        _expect(fn, "k_out", k_out, kshape, dtype)
        kos = _row_strides(fn, "k_out", k_out, packed, True)
    _need_rows(q, freqs, *[t for t in (k, positions, q_out, k_out) if t is not None], device=dev)
    lib = load_library()
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=torch.contiguous_format)
        qos = _row_strides(fn, "q_out", q_out, packed)
    if k is not None and k_out is None:
        k_out = torch.empty_like(k, memory_format=torch.contiguous_format)
        kos = _row_strides(fn, "k_out", k_out, packed)
    with _on_device(dev):
        st = lib.la_rotary(q.data_ptr(), qs, q_out.data_ptr(), qos, _ptr(k), ks, _ptr(k_out), kos,
                           freqs.data_ptr(), _ptr(positions), pos_b, int(offset), B, H, Hk, N, D,
                           2 * freqs.shape[0], 1 if interleaved else 0, 1 if inverse else 0,
                           float(mscale), dt, _stream_ptr(dev))
    if st:
        _check(fn, st)
    return q_out, k_out


def la_norm_gate_workspace_bytes(B, H, N, M):
    return load_library().la_norm_gate_workspace_bytes(B, H, N, M)


def _norm_checks(fn, x, z, w):
    shape, dt = x.shape, x.dtype
    if len(shape) != 4:
        raise ValueError(f"{fn}: x must have 4 dimensions")
    if z.shape != shape or z.dtype != dt:
        _expect(fn, "z", z, shape, dt)
    if w.dim() not in (1, 2):
        raise ValueError(f"{fn}: w must be [M] or [H, M]")
    if w.dtype != dt or w.shape != (shape[3:] if w.dim() == 1 else shape[1::2]):
        _expect(fn, "w", w, tuple(shape[3:] if w.dim() == 1 else shape[1::2]), dt)
    return shape, _dtype_code(x)


def la_norm_gate(x, z, w, eps=1e-6, out=None):
    """out = x / sqrt(mean(x^2) + eps) * w * z sigmoid(z), the mean over each head's M elements.

    x [B,H,N,M] contiguous (la_forward_gated's output), w [M] or [H,M]; z and out [B,H,N,M] with
    any strides that are multiples of 16 bytes and a contiguous last dimension, so that out can
    be a token-major [B,N,H,M] buffer's transpose. out: contiguous unless passed in."""
    import torch
    fn = "la_norm_gate"
    (B, H, N, M), dt = _norm_checks(fn, x, z, w)
    dev = x.device
    zs = _row_strides(fn, "z", z)
    if out is None:
        _need_cuda(x, w)
        _need_rows(z, device=dev)
        out = torch.empty_like(x)
        outs = _row_strides(fn, "out", out)
    else:
        _expect(fn, "out", out, x.shape, x.dtype)
        outs = _row_strides(fn, "out", out, False, True)
        _need_cuda(x, w)
        _need_rows(z, out, device=dev)
    lib = load_library()
    with _on_device(dev):
        st = lib.la_norm_gate(x.data_ptr(), z.data_ptr(), zs, w.data_ptr(), out.data_ptr(), outs,
                              B, H, N, M, w.dim() - 1, float(eps), dt, _stream_ptr(dev))
    if st:
        _check(fn, st)
    return out


def la_norm_gate_backward(x, z, w, dy, eps=1e-6, dx=None, dz=None, dw=None, workspace=None):
    """Gradients (dx, dz, dw) of sum(dy * la_norm_gate(x, z, w, eps)), in the inputs' dtype; dw
    has w's shape. dy and dz are strided as z is (dz: contiguous unless passed in)."""
    import torch
    fn = "la_norm_gate_backward"
    (B, H, N, M), dt = _norm_checks(fn, x, z, w)
    shape, dtype, dev = x.shape, x.dtype, x.device
    if dy.shape != shape or dy.dtype != dtype:
        _expect(fn, "dy", dy, shape, dtype)
    for name, t, like in (("dx", dx, shape), ("dz", dz, shape), ("dw", dw, w.shape)):
        if t is not None:
            _expect(fn, name, t, like, dtype)
    zs, dys = _row_strides(fn, "z", z), _row_strides(fn, "dy", dy)
    if dz is not None:
        dzs = _row_strides(fn, "dz", dz, False, True)
    _need_cuda(x, w, *[t for t in (dx, dw) if t is not None])
    _need_rows(z, dy, *([] if dz is None else [dz]), device=dev)
    lib = load_library()
    if dx is None:
        dx = torch.empty_like(x)
    if dz is None:
        dz = torch.empty_like(x)
        dzs = _row_strides(fn, "dz", dz)
    if dw is None:
        dw = torch.empty_like(w)
    ws, nbytes = _scratch(x, _bytes("la_norm_gate_workspace_bytes", B, H, N, M), workspace)
    with _on_device(dev):
        st = lib.la_norm_gate_backward(x.data_ptr(), z.data_ptr(), zs, w.data_ptr(), dy.data_ptr(),
                                       dys, dx.data_ptr(), dz.data_ptr(), dzs, dw.data_ptr(),
                                       B, H, N, M, w.dim() - 1, float(eps), dt, ws.data_ptr(),
                                       nbytes, _stream_ptr(dev))
    if st:
        _check(fn, st)
    return dx, dz, dw
