"""Refusals of the gated recurrence's, the rotary's and the gated norm's entry points, in the
binding and in the C ABI, without a GPU."""

import ctypes
import math

import pytest
import torch

import kernelized_causal_self_gb300 as la
from kernelized_causal_self_gb300 import build as labuild

BF, F32 = torch.bfloat16, torch.float32
FAKE, ODD = 0x10000, 0x10008  # never dereferenced: every call below returns before a launch


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def test_forward_and_backward_check_every_tensor():
    q, v, g, S = _t(2, 3, 10, 16), _t(2, 3, 10, 8), _t(2, 3, 10), _t(2, 3, 16, 8, dtype=F32)
    for fn in (la.la_forward_gated, la.la_prefill_gated):
        _raises("k must be", fn, q, _t(2, 3, 9, 16), v, g)
        _raises("v must be", fn, q, q, _t(2, 1, 10, 8), g)
        _raises("g must be", fn, q, q, v, _t(2, 3, 10, dtype=F32))
        _raises("g must be", fn, q, q, v, _t(2, 3, 10, 1))
        _raises("S0 must be", fn, q, q, v, g, S0=_t(2, 3, 16, 8))
        _raises("out must be", fn, q, q, v, g, out=q)
        _raises("4 dimensions", fn, q[0], q[0], v[0], g[0])
        _raises("CUDA device", fn, q, q, v, g, S0=S)
    _raises("S must be", la.la_prefill_gated, q, q, v, g, S=_t(2, 3, 8, 16, dtype=F32))
    with pytest.raises(TypeError):
        la.la_forward_gated(*(x.half() for x in (q, q, v, g)))
    back = la.la_backward_gated
    _raises("dout must be", back, q, q, v, g, q)
    _raises("g must be", back, q, q, v, _t(2, 3), v)
    _raises("dS must be", back, q, q, v, g, v, dS=_t(2, 3, 16, 16, dtype=F32))
    _raises("dS0 without S0", back, q, q, v, g, v, dS0=S)
    _raises("dq must be", back, q, q, v, g, v, dq=_t(2, 3, 10, 16, dtype=F32))
    _raises("dg must be", back, q, q, v, g, v, dg=_t(2, 3, 10, dtype=F32))
    _raises("CUDA device", back, q, q, v, g, v, S0=S, dS=S)


def test_pool_calls_check_pool_and_indices():
    q, v, g, S = _t(2, 3, 4, 16), _t(2, 3, 4, 8), _t(2, 3, 4), _t(5, 3, 16, 8, dtype=F32)
    ext, dec = la.la_extend_gated, la.la_decode_step_gated
    _raises("S_pool must be", ext, q, q, v, g, _t(5, 2, 16, 8, dtype=F32))
    _raises("S_pool must be", ext, q, q, v, g, S[0])
    _raises("S_pool must be", ext, q, q, v, g, _t(5, 3, 16, 8))
    _raises("slots must be", ext, q, q, v, g, S, slots=torch.zeros(2, dtype=torch.int64))
    _raises("lens must be", ext, q, q, v, g, S, lens=torch.zeros(3, dtype=torch.int32))
    _raises("out must be", ext, q, q, v, g, S, out=q)
    _raises("CUDA device", ext, q, q, v, g, S)
    one = [x[:, :, 0] for x in (q, q, v, g)]
    _raises("3 dimensions", dec, q, q, v, g, S)
    _raises("g must be", dec, *one[:3], _t(2, 4), S)
    _raises("slots must be", dec, *one, S, slots=torch.zeros(3, dtype=torch.int32))
    _raises("out must be", dec, *one, S, out=one[0])
    _raises("CUDA device", dec, *one, S)


def test_rotary_checks():
    q, k, f = _t(2, 4, 10, 16), _t(2, 2, 10, 16), torch.zeros(4, dtype=torch.float64)
    rot = la.la_rotary
    _raises("3 or 4", rot, q[0, 0], None, f)
    _raises("k must be", rot, q, _t(2, 2, 9, 16), f)
    _raises("k must be", rot, q, k[0], f)
    _raises("k must be", rot, q, k.float(), f)
    _raises("freqs must be", rot, q, k, f.float())
    _raises("freqs must be", rot, q, k, torch.zeros(8, dtype=torch.float64)[::2])
    _raises("positions must be", rot, q, k, f, positions=torch.zeros(10, dtype=torch.int64))
    _raises("positions must be", rot, q, k, f, positions=torch.zeros(9, dtype=torch.int32))
    _raises("positions must be", rot, q, k, f, positions=torch.zeros(10, 2, dtype=torch.int32).t())
    _raises("last dimension", rot, q.transpose(2, 3).contiguous().transpose(2, 3), None, f)
    _raises("q_out must be", rot, q, k, f, q_out=k)
    _raises("overlap", rot, q, None, f, q_out=_t(1, 1, 10, 16).expand(2, 4, 10, 16))
    _raises("k_out without k", rot, q, None, f, k_out=k)
    _raises("CUDA device", rot, q, k, f)
    with pytest.raises(TypeError):
        rot(q.half(), None, f)


def test_rotary_freqs():
    f, ms = la.la_rotary_freqs(8, base=100.0, device="cpu")
    assert ms == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([100.0 ** (-i / 4) for i in range(4)], dtype=torch.float64), rtol=1e-15)
    lin, _ = la.la_rotary_freqs(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(lin, f / 4)
    b, _ = la.la_rotary_freqs(8, base=100.0, scaling="base", factor=4.0, device="cpu")
    assert b[0] == f[0] and torch.allclose(b[-1], f[-1] / 4, rtol=1e-14)
    r, ms = la.la_rotary_freqs(64, scaling="ramp", factor=4.0, original_len=2048, device="cpu")
    plain, _ = la.la_rotary_freqs(64, device="cpu")
    turns = 2048 * plain / (2 * math.pi)
    assert torch.equal(r[turns >= 32], plain[turns >= 32])
    assert torch.allclose(r[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    assert torch.all(r[1:] < r[:-1]) and math.isclose(ms, 0.1 * math.log(4) + 1)
    for kw in ({"rot_dim": 7}, {"rot_dim": 0}, {"rot_dim": 8, "scaling": "other"}, {"rot_dim": 8, "base": 0.0},
               {"rot_dim": 8, "scaling": "ramp"}, {"rot_dim": 8, "factor": -1.0},
               {"rot_dim": 8, "scaling": "ramp", "original_len": 10, "slow": 2.0, "fast": 2.0}):
        with pytest.raises(ValueError):
            la.la_rotary_freqs(**kw, device="cpu")


def test_norm_gate_checks():
    x, w = _t(2, 3, 5, 16), _t(16)
    fwd, back = la.la_norm_gate, la.la_norm_gate_backward
    _raises("4 dimensions", fwd, x[0], x[0], w)
    _raises("z must be", fwd, x, x.float(), w)
    _raises("w must be", fwd, x, x, _t(2, 16))
    _raises("w must be", fwd, x, x, _t(16, dtype=F32))
    _raises("out must be", fwd, x, x, w, out=_t(2, 3, 5, 8))
    _raises("overlap", fwd, x, x, w, out=_t(1, 3, 5, 16).expand(2, 3, 5, 16))
    _raises("last dimension", fwd, x, x.transpose(2, 3).contiguous().transpose(2, 3), w)
    _raises("CUDA device", fwd, x, x, w)
    _raises("dy must be", back, x, x, w, x[0])
    _raises("dw must be", back, x, x, w, x, dw=_t(3, 16))
    _raises("overlap", back, x, x, w, x, dz=_t(1, 3, 5, 16).expand(2, 3, 5, 16))
    _raises("CUDA device", back, x, x, w, x)


def test_abi_refuses_before_a_launch(lib):
    bad, ws = la.LA_ERR_INVALID_ARG, la.LA_ERR_WORKSPACE

    def fwd(q=FAKE, g=FAKE, S0=None, S=None, B=1, H=1, N=16, D=64, M=64, dt=1, w=FAKE, wb=1 << 20):
        return lib.la_forward_gated(q, FAKE, FAKE, g, FAKE, S0, S, B, H, N, D, M, dt, w, wb, None)
    assert fwd(q=0) == bad and fwd(g=ODD) == bad and fwd(S0=ODD) == bad and fwd(S=ODD) == bad
    assert fwd(D=12) == bad and fwd(M=136) == bad and fwd(B=0) == bad and fwd(N=-1) == bad and fwd(dt=2) == bad
    assert fwd(B=1 << 16, H=1 << 16) == bad
    assert fwd(N=0, q=0) == la.LA_OK
    need = la.la_gated_workspace_bytes(1, 1, 4000, 64, 64)
    assert need > 256 and fwd(N=4000, wb=need - 1) == ws and fwd(N=4000, w=None, wb=need) == ws
    assert fwd(N=4000, w=ODD, wb=need) == ws

    def ext(pool=FAKE, slots=None, lens=None, P=4, B=2, N=8, w=FAKE):
        return lib.la_extend_gated(FAKE, FAKE, FAKE, FAKE, FAKE, pool, slots, lens, P, B, 2, N, 64, 64, 1,
                                   w, 1 << 24, None)
    assert ext(pool=0) == bad and ext(pool=ODD) == bad and ext(slots=FAKE + 2) == bad and ext(lens=FAKE + 1) == bad
    assert ext(P=1) == bad and ext(slots=FAKE, P=0) == bad and ext(w=None) == ws and ext(N=0) == la.LA_OK

    def dec(q=FAKE, pool=FAKE, slots=None, P=4, n=2, D=64):
        return lib.la_decode_step_gated(q, FAKE, FAKE, FAKE, pool, slots, FAKE, P, n, 2, D, 64, 1, None)
    assert dec(q=ODD) == bad and dec(pool=0) == bad and dec(P=1) == bad and dec(D=4) == bad
    assert dec(slots=FAKE, P=0) == bad and dec(n=0) == bad

    def back(do=FAKE, dg=FAKE, S0=None, N=16, w=FAKE, wb=1 << 24):
        return lib.la_backward_gated(FAKE, FAKE, FAKE, FAKE, do, S0, None, FAKE, FAKE, FAKE, dg, None,
                                     1, 1, N, 64, 64, 1, w, wb, None)
    assert back(do=0) == bad and back(dg=ODD) == bad and back(S0=ODD) == bad
    assert back(w=0) == ws and back(wb=la.la_gated_backward_workspace_bytes(1, 1, 16, 64, 64) - 1) == ws
    assert back(N=0, do=0) == la.LA_OK

    s = (ctypes.c_longlong * 3)(64, 64, 64)

    def rot(q=FAKE, qs=s, k=FAKE, ks=s, f=FAKE, B=1, H=1, Hk=1, N=4, D=64, R=64, dt=1):
        return lib.la_rotary(q, qs, FAKE, s, k, ks, FAKE, s, f, None, 0, 0, B, H, Hk, N, D, R, 0, 0, 1.0, dt, None)
    assert rot(q=0) == bad and rot(q=FAKE + 1) == bad and rot(qs=None) == bad and rot(f=FAKE + 4) == bad
    assert rot(k=0) == bad and rot(ks=None) == bad and rot(R=63) == bad and rot(R=66) == bad and rot(R=0) == bad
    assert rot(D=60) == bad and rot(B=65536) == bad and rot(Hk=-1) == bad and rot(dt=3) == bad
    assert rot(N=0, q=0) == la.LA_OK

    def norm(x=FAKE, zs=s, eps=1e-6, B=1, N=4, M=64, dt=1):
        return lib.la_norm_gate(x, FAKE, zs, FAKE, FAKE, s, B, 2, N, M, 0, eps, dt, None)
    odd = (ctypes.c_longlong * 3)(64, 64, 60)
    assert norm(x=ODD) == bad and norm(zs=None) == bad and norm(zs=odd) == bad and norm(eps=-1.0) == bad
    assert norm(eps=math.nan) == bad and norm(M=60) == bad and norm(B=1 << 16, N=1 << 15) == bad
    assert norm(N=0, x=0) == la.LA_OK

    def nback(dw=FAKE, dy=FAKE, w=FAKE, wb=1 << 20):
        return lib.la_norm_gate_backward(FAKE, FAKE, s, FAKE, dy, s, FAKE, FAKE, s, dw, 1, 2, 4, 64, 0, 1e-6, 1,
                                         w, wb, None)
    assert nback(dw=0) == bad and nback(dy=0) == bad and nback(w=0) == ws and nback(wb=300) == ws


def test_abi_refuses_states_that_share_memory(lib):
    """A gradient of the initial state may take the place of the final state's gradient, and a final
    state that of the initial one, but no other two of them may touch: the walks from the two ends
    run at once."""
    bad, bytes_ = la.LA_ERR_INVALID_ARG, 4 * 3 * 16 * 8
    far = FAKE + bytes_

    def back(S0, dS, dS0, N=40, dt=1):
        return lib.la_backward_gated(FAKE, FAKE, FAKE, FAKE, FAKE, S0, dS, FAKE, FAKE, FAKE, FAKE, dS0,
                                     1, 3, N, 16, 8, dt, FAKE, 16, None)

    for dt in (0, 1):
        for N in (1, 40, 4000):
            assert back(FAKE, None, FAKE, N, dt) == bad and back(FAKE, far, FAKE, N, dt) == bad
            assert back(FAKE, None, FAKE + 16, N, dt) == bad and back(FAKE + 16, None, FAKE, N, dt) == bad
            assert back(FAKE, None, far - 16, N, dt) == bad and back(None, FAKE, FAKE + 16, N, dt) == bad
            # (a workspace that is too small is the next refusal)
            assert back(FAKE, None, far, N, dt) == la.LA_ERR_WORKSPACE
            assert back(far, FAKE, FAKE, N, dt) == la.LA_ERR_WORKSPACE

    def fwd(S0, S):
        return lib.la_forward_gated(FAKE, FAKE, FAKE, FAKE, FAKE, S0, S, 1, 3, 4000, 16, 8, 1, FAKE, 16, None)
    assert fwd(FAKE, FAKE + 16) == bad and fwd(far - 16, FAKE) == bad
    assert fwd(FAKE, FAKE) == la.LA_ERR_WORKSPACE and fwd(FAKE, far) == la.LA_ERR_WORKSPACE


def test_rotary_refuses_offsets_that_are_no_position(lib):
    q, f, s = _t(1, 2, 4, 16), torch.zeros(4, dtype=torch.float64), (ctypes.c_longlong * 3)(64, 64, 64)
    for offset in (2 ** 64, 2 ** 62 + 1, -2 ** 62 - 1, -2 ** 70):
        _raises("offset", la.la_rotary, q, None, f, offset=offset)
    _raises("offset", la.la_rotary, q, None, f, offset=1.5)
    _raises("CUDA device", la.la_rotary, q, None, f, offset=2 ** 62)

    def rot(offset, N):
        return lib.la_rotary(FAKE, s, FAKE, s, None, None, None, None, FAKE, None, 0, offset, 1, 1, 0, N, 64, 64,
                             0, 0, 1.0, 1, None)
    assert rot(2 ** 62 + 1, 0) == la.LA_ERR_INVALID_ARG and rot(-2 ** 63, 0) == la.LA_ERR_INVALID_ARG
    assert rot(2 ** 62, 0) == la.LA_OK and rot(-2 ** 62, 0) == la.LA_OK


@pytest.mark.parametrize("BH,N", [(1, 8192), (16, 1 << 18), (16, 1 << 20), (8, 1 << 20), (3, 1 << 24), (200, 1 << 20)])
def test_one_of_several_segments_has_at_most_4096_tokens(lib, BH, N):
    """So that exp() of a segment's gates is finite where la.h says so, and a state's sums are short.
    The workspace tells the segments: a state of each and one more of every sequence."""
    for dt, D, M in ((la.LA_BF16, 64, 64), (la.LA_BF16, 128, 128), (la.LA_F32, 64, 64), (la.LA_F32, 128, 128)):
        bytes_ = la.la_gated_workspace_bytes(1, BH, N, D, M, dt)
        segments = 1 if bytes_ == 256 else bytes_ // (4 * BH * D * M) - 1
        assert segments == 1 or segments * 4096 >= N, (dt, D, segments)
    D = 128  # the backward of wide heads joins states and gradients, however few the segments
    bytes_ = la.la_gated_backward_workspace_bytes(1, BH, N, D, D, la.LA_BF16)
    chunks = (N + 63) // 64
    scratch = BH * (chunks * (4 * 64 * 1024 // 4 + 32) + 3 * 2 * 4 * N)
    assert (bytes_ - scratch) // (2 * 4 * BH * D * D) - 1 >= N // 4096


def test_binding_refuses_states_that_share_memory():
    q, v, g, S = _t(2, 3, 10, 16), _t(2, 3, 10, 8), _t(2, 3, 10), _t(3, 3, 16, 8, dtype=F32)
    _raises("dS0 shares memory with S0", la.la_backward_gated, q, q, v, g, v, S0=S[:2], dS0=S[:2])
    _raises("dS0 shares memory with S0", la.la_backward_gated, q, q, v, g, v, S0=S[:2], dS0=S[1:])
    _raises("dS0 shares memory with dS", la.la_backward_gated, q, q, v, g, v, S0=_t(2, 3, 16, 8, dtype=F32),
            dS=S[:2], dS0=S[1:])
    _raises("S shares memory with S0", la.la_prefill_gated, q, q, v, g, S0=S[:2], S=S[1:])
    _raises("CUDA device", la.la_prefill_gated, q, q, v, g, S0=S[:2], S=S[:2])
    _raises("CUDA device", la.la_backward_gated, q, q, v, g, v, S0=_t(2, 3, 16, 8, dtype=F32), dS=S[:2], dS0=S[:2])


def test_workspace_queries_of_shapes_that_are_refused(lib):
    assert la.la_gated_workspace_bytes(0, 1, 1, 64, 64) == 256
    assert la.la_gated_backward_workspace_bytes(1, 1, 8, 63, 64) == 256
    assert la.la_norm_gate_workspace_bytes(1, 1, -1, 64) == 256


def test_every_new_call_runs_with_the_tensors_device_current(monkeypatch):
    events = []

    class Guard:
        def __init__(self, dev):
            self.dev = str(dev)

        def __enter__(self):
            events.append("enter " + self.dev)

        def __exit__(self, *exc):
            events.append("exit " + self.dev)

    class FakeLib:
        def __getattr__(self, name):
            def fn(*args):
                if name.endswith("_bytes"):
                    return 256
                events.append(name)
                return 0
            return fn

    monkeypatch.setattr(la, "_on_device", Guard)
    monkeypatch.setattr(la, "load_library", lambda: FakeLib())
    monkeypatch.setattr(la, "_need_cuda", lambda *a, **k: None)
    monkeypatch.setattr(la, "_need_rows", lambda *a, **k: None)
    monkeypatch.setattr(la, "_stream_ptr", lambda dev: 0)
    monkeypatch.setattr(la, "_bytes", lambda query, *dims: 256)
    q, v, g, S = _t(2, 3, 10, 16), _t(2, 3, 10, 8), _t(2, 3, 10), _t(2, 3, 16, 8, dtype=F32)
    assert la.la_forward_gated(q, q, v, g).shape == v.shape
    assert la.la_prefill_gated(q, q, v, g)[1].shape == S.shape
    la.la_extend_gated(q, q, v, g, S)
    la.la_decode_step_gated(*(x[:, :, 0] for x in (q, q, v, g)), S)
    assert len(la.la_backward_gated(q, q, v, g, v)) == 4
    assert la.la_backward_gated(q, q, v, g, v, S0=S)[4].shape == S.shape
    la.la_rotary(q, q[:, :1], torch.zeros(4, dtype=torch.float64))
    la.la_norm_gate(v, v, _t(8))
    la.la_norm_gate_backward(v, v, _t(3, 8), v)
    names = ["la_forward_gated", "la_forward_gated", "la_extend_gated", "la_decode_step_gated",
             "la_backward_gated", "la_backward_gated", "la_rotary", "la_norm_gate", "la_norm_gate_backward"]
    assert events == [e for n in names for e in ("enter cpu", n, "exit cpu")]
