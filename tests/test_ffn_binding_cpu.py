"""Refusals of the layer norm's, the gated projections' and the checkpoints' entry points, in the
binding and in the C ABI, without a GPU."""

import pytest
import torch

import kernelized_causal_self_gb300 as la
from kernelized_causal_self_gb300 import build as labuild

BF, F32 = torch.bfloat16, torch.float32
FAKE, ODD = 0x10000, 0x10008  # never dereferenced: every call below returns before a launch
FAR = [0x10000000 * (i + 1) for i in range(12)]


def _t(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def _raises(match, fn, *args, **kw):
    with pytest.raises(ValueError, match=match):
        fn(*args, **kw)


@pytest.fixture(scope="module")
def lib():
    labuild.build()
    return la.load_library()


def _pair(*shape):
    return _t(*shape, dtype=torch.int8), _t(*shape[:-1], -(-shape[-1] // 32), dtype=torch.uint8)


def test_checkpoint_checks():
    x = _t(4, 40)
    _raises("codes must be", la.la_checkpoint, x, checkpoint=_pair(4, 48))
    _raises("exps must be", la.la_checkpoint, x, checkpoint=(_pair(4, 40)[0], _pair(4, 72)[1]))
    _raises("pair", la.la_checkpoint, x, checkpoint=_pair(4, 40)[0])
    _raises("last dimension", la.la_checkpoint, _t(40, 4).t())
    _raises("evenly", la.la_checkpoint, _t(3, 5, 40)[:, :4])
    _raises("overlap", la.la_checkpoint, x[:1].expand(4, 40))
    _raises("CUDA device", la.la_checkpoint, x)
    codes, exps = _pair(4, 40)
    back = la.la_checkpoint_restore
    _raises("exps must be", back, codes, exps[:, :1])
    _raises("codes must be", back, codes.float(), exps)
    _raises("out must be", back, codes, exps, out=_t(4, 48))
    _raises("out must be", back, codes, exps, out=x, dtype=F32)
    _raises("CUDA device", back, codes, exps)
    for bad in (torch.float16, torch.float64):
        with pytest.raises(TypeError):
            back(codes, exps, dtype=bad)
        with pytest.raises(TypeError):
            la.la_checkpoint(x.to(bad))


def test_layer_norm_checks():
    x, w = _t(2, 5, 16), _t(16)
    fwd, back = la.la_layer_norm, la.la_layer_norm_backward
    _raises("w must be", fwd, x, _t(8))
    _raises("w must be", fwd, x, _t(16, dtype=F32))
    _raises("b must be", fwd, x, w, _t(1, 16))
    _raises("out must be", fwd, x, w, out=_t(10, 16))
    _raises("evenly", fwd, x, w, out=_t(2, 7, 16)[:, :5])
    _raises("codes must be", fwd, x, w, checkpoint=_pair(10, 16))
    _raises("CUDA device", fwd, x, w)
    with pytest.raises(TypeError):
        fwd(x.half(), w.half())
    _raises("x must be", back, x[0], w, x)
    _raises("x must be", back, x.float(), w, x)
    _raises("codes must be", back, _pair(2, 4, 16), w, x)
    _raises("pair", back, (x,), w, x)
    _raises("w must be", back, x, _t(15), x)
    _raises("dx must be", back, x, w, x, dx=x[0])
    _raises("dw must be", back, x, w, x, dw=_t(16, dtype=F32))
    _raises("db must be", back, x, w, x, db=_t(2, 16))
    _raises("CUDA device", back, x, w, x)


def test_ffn_checks():
    x, w, h = _t(3, 4, 16), _t(24, 16), _t(3, 4, 24)
    fwd, back = la.la_ffn_gate, la.la_ffn_gate_backward
    _raises("activation", fwd, x, w, w, activation="relu")
    _raises("wg must be", fwd, x, _t(24, 8), w)
    _raises("wg must be", fwd, x, w.float(), w)
    _raises("wu must be", fwd, x, w, _t(16, 16))
    _raises("x must be", fwd, x, w[0], w)
    _raises("out must be", fwd, x, w, w, out=x)
    _raises("codes must be", fwd, x, w, w, checkpoint=_pair(3, 4, 24))
    _raises("exps must be", fwd, x, w, w, checkpoint=(_t(3, 4, 2, 24, dtype=torch.int8), _t(3, 4, 2, 2, dtype=torch.uint8)))
    _raises("CUDA device", fwd, x, w, w)
    _raises("dh must be", back, x, w, w, x)
    _raises("dh must be", back, x, w, w, h.float())
    _raises("dx must be", back, x, w, w, h, dx=h)
    _raises("dwg must be", back, x, w, w, h, dwg=w.t())
    _raises("dwu must be", back, x, w, w, h, dwu=w.float())
    _raises("codes must be", back, x, w, w, h, checkpoint=_pair(3, 4, 24))
    _raises("CUDA device", back, x, w, w, h, checkpoint=_pair(3, 4, 2, 24))
    with pytest.raises(TypeError):
        fwd(x.half(), w.half(), w.half())


def test_abi_checkpoint(lib):
    bad = la.LA_ERR_INVALID_ARG

    def pack(x=FAR[0], ld=64, codes=FAR[1], exps=FAR[2], rows=4, C=64, dt=1):
        return lib.la_checkpoint(x, ld, codes, exps, rows, C, dt, None)

    def back(x=FAR[0], ld=64, codes=FAR[1], exps=FAR[2], rows=4, C=64, dt=1):
        return lib.la_checkpoint_restore(codes, exps, x, ld, rows, C, dt, None)
    for f in (pack, back):
        assert f(x=0) == bad and f(x=ODD) == bad and f(codes=0) == bad and f(exps=0) == bad and f(codes=ODD) == bad
        assert f(C=12) == bad and f(C=0) == bad and f(C=65544) == bad and f(dt=2) == bad
        assert f(rows=-1) == bad and f(rows=1 << 31) == bad
        assert f(ld=56) == bad and f(ld=68) == bad and f(ld=1 << 41) == bad and f(ld=66, dt=0) == bad
        assert f(codes=FAR[0] + 128) == bad and f(exps=FAR[0] + 511) == bad  # shared memory
        assert f(rows=0, x=0) == la.LA_OK


def test_abi_layer_norm(lib):
    bad, ws = la.LA_ERR_INVALID_ARG, la.LA_ERR_WORKSPACE

    def fwd(x=FAR[0], xs=64, w=FAR[1], b=FAR[2], y=FAR[3], ys=64, codes=0, exps=0, rows=4, C=64, eps=1e-5, dt=1):
        return lib.la_layer_norm(x, xs, w, b, y, ys, codes, exps, rows, C, eps, dt, None)
    assert fwd(x=0) == bad and fwd(w=0) == bad and fwd(y=0) == bad and fwd(b=ODD) == bad and fwd(x=ODD) == bad
    assert fwd(C=20) == bad and fwd(C=16392) == bad and fwd(dt=3) == bad and fwd(rows=-1) == bad
    assert fwd(eps=-1e-5) == bad and fwd(eps=float("nan")) == bad
    assert fwd(xs=63) == bad and fwd(ys=56) == bad and fwd(ys=68) == bad
    assert fwd(codes=FAR[4]) == bad and fwd(exps=FAR[4]) == bad
    # columns of one buffer: refused only where they meet
    assert fwd(xs=192, y=FAR[0] + 256, ys=192, w=0) == bad and fwd(xs=192, y=FAR[0] + 64, ys=192) == bad
    assert fwd(xs=192, y=FAR[0] + 320, ys=192) == bad and fwd(x=FAR[0] + 64, xs=192, y=FAR[0], ys=192) == bad
    assert fwd(y=FAR[0], ys=128) == bad and fwd(y=FAR[0] + 128) == bad and fwd(y=FAR[1]) == bad
    assert fwd(codes=FAR[0], exps=FAR[5]) == bad and fwd(codes=FAR[3], exps=FAR[5]) == bad
    assert fwd(rows=0, x=0) == la.LA_OK

    def back(x=FAR[0], xs=64, codes=0, exps=0, w=FAR[1], dy=FAR[2], dys=64, dx=FAR[3], dxs=64, dw=FAR[4], db=FAR[5],
             rows=4, C=64, eps=1e-5, dt=1, wsp=FAR[6], wsb=1 << 30):
        return lib.la_layer_norm_backward(x, xs, codes, exps, w, dy, dys, dx, dxs, dw, db, rows, C, eps, dt, wsp, wsb,
                                          None)
    assert back(x=0) == bad and back(codes=FAR[7], exps=FAR[8]) == bad and back(x=0, codes=FAR[7]) == bad
    assert back(dw=0) == bad and back(db=ODD) == bad and back(dx=0) == bad and back(dy=ODD) == bad and back(w=0) == bad
    assert back(xs=56) == bad and back(dys=56) == bad and back(dxs=60) == bad and back(eps=-1.0) == bad
    assert back(dw=FAR[5]) == bad and back(dw=FAR[0]) == bad and back(dx=FAR[1]) == bad and back(dx=FAR[2], dxs=72) == bad
    assert back(x=0, codes=FAR[3], exps=FAR[8]) == bad
    assert back(wsp=0) == ws and back(wsp=ODD) == ws and back(wsb=256) == ws
    need = lib.la_layer_norm_workspace_bytes(4, 64)
    assert back(wsb=need - 1) == ws and need >= 256 + 2 * 4 * 64
    assert lib.la_layer_norm_workspace_bytes(0, 64) == 256 and lib.la_layer_norm_workspace_bytes(4, 63) == 256


def test_abi_ffn(lib):
    bad, ws = la.LA_ERR_INVALID_ARG, la.LA_ERR_WORKSPACE

    def fwd(x=FAR[0], xs=64, wg=FAR[1], wu=FAR[2], h=FAR[3], hs=128, codes=0, exps=0, T=4, C=64, F=128, act=0, dt=1,
            wsp=FAR[4], wsb=1 << 27):
        return lib.la_ffn_gate(x, xs, wg, wu, h, hs, codes, exps, T, C, F, act, dt, wsp, wsb, None)
    assert fwd(x=0) == bad and fwd(wg=0) == bad and fwd(wu=ODD) == bad and fwd(h=0) == bad
    assert fwd(C=12) == bad and fwd(F=12) == bad and fwd(C=65544) == bad and fwd(F=65544) == bad and fwd(F=0) == bad
    assert fwd(T=-1) == bad and fwd(T=(1 << 24) + 1) == bad and fwd(act=3) == bad and fwd(act=-1) == bad and fwd(dt=2) == bad
    assert fwd(xs=56) == bad and fwd(hs=120) == bad and fwd(hs=132) == bad
    assert fwd(codes=FAR[5]) == bad and fwd(codes=ODD, exps=FAR[6]) == bad
    assert fwd(h=FAR[0]) == bad and fwd(h=FAR[1] + 1024) == bad and fwd(codes=FAR[3], exps=FAR[6]) == bad
    for many in ({"T": 4000}, {"codes": FAR[5], "exps": FAR[6]}):
        assert fwd(wsp=0, **many) == ws and fwd(wsb=128, **many) == ws and fwd(wsp=ODD, **many) == ws
    assert fwd(T=0, x=0, wsp=0) == la.LA_OK

    def back(x=FAR[0], xs=64, wg=FAR[1], wu=FAR[2], dh=FAR[3], dhs=128, codes=0, exps=0, dx=FAR[4], dxs=64, dwg=FAR[5],
             dwu=FAR[6], T=4, C=64, F=128, act=0, dt=1, wsp=FAR[7], wsb=1 << 27):
        return lib.la_ffn_gate_backward(x, xs, wg, wu, dh, dhs, codes, exps, dx, dxs, dwg, dwu, T, C, F, act, dt, wsp,
                                        wsb, None)
    assert back(x=0) == bad and back(dh=0) == bad and back(dx=ODD) == bad and back(dwg=0) == bad and back(dwu=ODD) == bad
    assert back(dhs=120) == bad and back(dxs=56) == bad and back(exps=FAR[8]) == bad and back(act=9) == bad
    assert back(dx=FAR[0]) == bad and back(dx=FAR[3]) == bad and back(dwg=FAR[6]) == bad and back(dwg=FAR[1]) == bad
    need = lib.la_ffn_gate_backward_workspace_bytes(4, 64, 128, 1)
    assert need > 256 and back(wsb=need - 1) == ws and back(wsp=0) == ws
    assert lib.la_ffn_gate_backward_workspace_bytes(4, 63, 128, 1) == 256
    need = lib.la_ffn_gate_workspace_bytes
    assert need(4000, 64, 128, 0, 1) == need(4, 64, 128, 1, 1) == need(-1, 64, 128, 0, 1) == 256
    assert need(4, 64, 128, 0, 1) == need(4, 64, 128, 0, 0) == need(100, 64, 128, 0, 0) == 0
    assert need(4000, 64, 128, 0, 0) >= 256 + 6 * 64 * (4000 + 2 * 128)


def test_marshalling_leaves_what_it_does_not_do(lib):
    """The C++ marshalling answers NotImplemented, and launches nothing, for anything but plain CUDA
    tensors; its functions are the library's."""
    m = la._marshal()
    assert set(m.names()) <= set(la._SIGNATURES)
    x, w, h = _t(4, 40), _t(40), _t(8, 40)
    pair = _pair(4, 40)
    before = la.la_kernel_launches()
    for args in ((x, None), (x, pair), (None, None), (x,), (3, None)):
        assert m.checkpoint(*args) is NotImplemented
    for args in ((*pair, 0), (*pair, 7), (x, pair[1], 0), (None, None, 0)):
        assert m.checkpoint_restore(*args) is NotImplemented
    for args in ((x, w, None, 1e-5, None, None), (x, w, w, 0, None, pair), (x, w, w, 1e-5, x), ([1], w, w, 1e-5, None, None)):
        assert m.layer_norm(*args) is NotImplemented
    for args in ((x, w, x, 1e-5), (pair, w, x, 1e-5), (None, w, x, 1e-5), (x, w, x)):
        assert m.layer_norm_backward(*args) is NotImplemented
    for args in ((x, h, h, 0, None, None), (x, h, h, -1, x, pair), (x, h[0], h, 0, None, None), (x, h, h)):
        assert m.ffn_gate(*args) is NotImplemented
    for args in ((x, h, h, 0, _t(4, 8), None), (x, h, h, 0, _t(4, 8), pair), (x, h, h, 0, None)):
        assert m.ffn_gate_backward(*args) is NotImplemented
    assert la.la_kernel_launches() == before
    with pytest.raises(ValueError):
        m.connect(1, 2)
    with pytest.raises(ValueError):
        m.connect(*[0] * len(m.names()))


def test_missing_marshalling_module_raises(monkeypatch):
    monkeypatch.setattr(la, "_fast", None)
    monkeypatch.setattr(la, "_MARSHAL_PATH", "/nowhere/la_marshal.so")
    with pytest.raises(RuntimeError, match="not built"):
        la.la_layer_norm(_t(4, 40), _t(40))
