"""la_rotary, la_norm_gate and la_norm_gate_backward on the GPU against the fp64 oracle.

Tolerances. Half a step of the type, u (bf16 2^-8, float32 2^-24), of each result for its
rounding. Rotary in float32: the angle is off by 2^-32 turns of its top 32 bits, 2^-25 half turns
of the conversion to float32 and |pos| 2^-54 turns (the frequency), together below 2^-21 radians
for |pos| < 2^31, cos and sin by a few 2^-24, the products and the sum by 2^-24 each: 2^-20 of
|a| + |b| in all. The norm: the sum of M squares (M 2^-24), the exponential of the sigmoid
(__expf: 2 + |1.173 z| ulp of 2^-23), divisions and products: (M + 64 + 4 |z|) 2^-24 of the sum
of absolute terms; its gradients pass through two such sums, and dw through the sum of the rows.
"""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
BF, FL = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, FL: 2.0 ** -24}


@pytest.fixture(scope="module")
def la():
    from kernelized_causal_self_gb300 import build
    build.build()
    import kernelized_causal_self_gb300 as pkg
    pkg.load_library()
    return pkg


def _f64(t):
    return t.double().cpu().numpy()


def _randn(seed, *shape, dtype=FL):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


# ------------------------------------------------------------------------- rotary

def _rotary_close(got, x, pos, freqs, dtype, **kw):
    want = oracle.rotary(_f64(x), pos, _f64(freqs), **kw)
    ms = abs(kw.get("mscale", 1.0))
    half = len(freqs)
    reach = np.abs(_f64(x)).copy()
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if kw.get("interleaved") else (i, i + half)
    reach[..., lo] = reach[..., hi] = ms * (reach[..., lo] + reach[..., hi])
    assert got.dtype == dtype and got.shape == x.shape
    off = np.abs(_f64(got) - want)
    assert np.all(off <= HALF[dtype] * np.abs(want) + 2.0 ** -20 * reach + 1e-37)
    rest = slice(2 * half, None)
    assert torch.equal(got[..., rest], x[..., rest])


@pytest.mark.parametrize("inverse", [False, True], ids=["turn", "inverse"])
@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 64, 64), (2, 4, 2, 33, 64, 64), (3, 3, 1, 70, 80, 20),
                                   (1, 5, 5, 129, 128, 64), (2, 2, 2, 9, 8, 2), (16, 8, 8, 1, 96, 96),
                                   (1, 2, 2, 40, 72, 48), (1, 16, 2, 700, 64, 32)],
                         ids=lambda s: "b%dh%dk%dn%dd%dr%d" % s)
def test_rotary(la, shape, dtype, interleaved, inverse):
    B, H, Hk, N, D, R = shape
    q, k = _randn(1, B, H, N, D, dtype=dtype), _randn(2, B, Hk, N, D, dtype=dtype)
    freqs, _ = la.la_rotary_freqs(R, device=DEV)
    kw = dict(interleaved=interleaved, inverse=inverse, mscale=1.25)
    rq, rk = la.la_rotary(q, k, freqs, offset=5, **kw)
    pos = np.arange(N) + 5
    _rotary_close(rq, q, pos, freqs, dtype, **kw)
    _rotary_close(rk, k, pos, freqs, dtype, **kw)
    each = torch.randint(-1000, 2 ** 31 - 1, (B, N), device=DEV, dtype=torch.int32,
                         generator=torch.Generator(device=DEV).manual_seed(4))
    rq, rk = la.la_rotary(q, k, freqs, positions=each, **kw)
    pos = each.cpu().numpy()[:, None]
    _rotary_close(rq, q, pos, freqs, dtype, **kw)
    _rotary_close(rk, k, pos, freqs, dtype, **kw)


@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
def test_rotary_layouts_and_places(la, dtype):
    B, H, N, D, R = 2, 3, 50, 64, 32
    freqs, _ = la.la_rotary_freqs(R, device=DEV)
    both = _randn(3, B, N, H, 2 * D + 1, dtype=dtype)    # odd strides, q and k in one buffer
    q, k = both[..., :D].transpose(1, 2), both[..., D + 1:].transpose(1, 2)
    assert q.stride(1) % 8 == 1
    pos = torch.arange(N, dtype=torch.int32, device=DEV) * 3
    rq, rk = la.la_rotary(q, k, freqs, positions=pos)
    assert rq.is_contiguous() and rk.is_contiguous()
    want = la.la_rotary(q.contiguous(), k.contiguous(), freqs, positions=pos)
    assert torch.equal(rq, want[0]) and torch.equal(rk, want[1])
    _rotary_close(rq, q, pos.cpu().numpy(), freqs, dtype)
    # in place, and only q
    edge = both[..., D].clone()
    got = la.la_rotary(q, k, freqs, positions=pos, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, rq) and torch.equal(k, rk) and torch.equal(both[..., D], edge)
    c = rq.clone()
    only = la.la_rotary(c, None, freqs, positions=pos, inverse=True)
    assert only[1] is None
    _rotary_close(only[0], c, pos.cpu().numpy(), freqs, dtype, inverse=True)
    # packed [T, H, D]
    p = _randn(5, 40, H, D, dtype=dtype)
    pp = torch.randint(0, 4000, (40,), device=DEV, dtype=torch.int32)
    rp, rk = la.la_rotary(p, p[:, :1], freqs, positions=pp)
    _rotary_close(rp.transpose(0, 1), p.transpose(0, 1), pp.cpu().numpy(), freqs, dtype)
    assert torch.equal(rk, rp[:, :1])
    # no tokens; a broadcast input
    e, _ = la.la_rotary(p[:0], None, freqs)
    assert e.shape == (0, H, D)
    one = _randn(6, 1, 1, N, D, dtype=dtype)
    rb, _ = la.la_rotary(one.expand(B, H, N, D), None, freqs)
    assert torch.equal(rb, la.la_rotary(one, None, freqs)[0].expand(B, H, N, D))


@pytest.mark.parametrize("scaling", ["linear", "base", "ramp"])
def test_rotary_scaled_for_long_contexts(la, scaling):
    freqs, ms = la.la_rotary_freqs(64, scaling=scaling, factor=16.0, original_len=4096, device=DEV)
    q = _randn(7, 1, 2, 64, 64)
    pos = torch.arange(10 ** 6, 10 ** 6 + 64, dtype=torch.int32, device=DEV)
    rq, _ = la.la_rotary(q, None, freqs, positions=pos, mscale=ms)
    _rotary_close(rq, q, pos.cpu().numpy(), freqs, FL, mscale=ms)
    far, _ = la.la_rotary(q, None, freqs, offset=2 ** 40)
    # the float64 frequency's rounding, 2^40 2^-54 turns, is 4e-4 radians
    want = oracle.rotary(_f64(q), np.arange(64) + 2 ** 40, _f64(freqs))
    assert np.all(np.abs(_f64(far) - want) <= 1e-3 * np.abs(_f64(q)).max())


@pytest.mark.parametrize("interleaved", [False, True], ids=["half", "interleaved"])
def test_rotary_turns_by_the_angle_to_float32s_digits(la, interleaved):
    """float32, pairs (a, 0), whose results are a cos and a sin. In half steps, 2^-24: 2 of the
    function, 1 of the product. The angle: its top 32 bits (2^-32 turns), 2^-27 half turns where an
    eighth of a turn is converted to float32, and 2^-54 turns a token: below 2^-25.2 radians."""
    N, D = 3000, 64
    q = _randn(11, 1, 2, N, D)
    q[..., (slice(1, None, 2) if interleaved else slice(D // 2, None))] = 0.0
    freqs, _ = la.la_rotary_freqs(D, device=DEV)
    pos = torch.randint(-2 ** 20, 2 ** 20, (N,), device=DEV, dtype=torch.int32,
                        generator=torch.Generator(device=DEV).manual_seed(3))
    got = _f64(la.la_rotary(q, None, freqs, positions=pos, interleaved=interleaved)[0])
    kw = dict(interleaved=interleaved)
    want = oracle.rotary(_f64(q), pos.cpu().numpy(), _f64(freqs), **kw)
    pairs = (lambda x: (x[..., 0::2], x[..., 1::2])) if interleaved else (lambda x: (x[..., :D // 2], x[..., D // 2:]))
    (c, s), (gc, gs) = pairs(want), pairs(got)
    for g, w, other in ((gc, c, s), (gs, s, c)):
        assert np.all(np.abs(g - w) <= 3 * 2.0 ** -24 * np.abs(w) + 2.0 ** -25.2 * np.abs(other) + 1e-37)


def test_rotary_past_32_bits(la):
    """The last tokens of a tensor of more than 2^31 elements, in place."""
    N = 2 ** 31 // 128 + 100
    q = torch.zeros(1, 1, N, 128, dtype=BF, device=DEV)
    tail = _randn(8, 1, 1, 50, 128, dtype=BF)
    q[:, :, -50:] = tail
    freqs, _ = la.la_rotary_freqs(128, device=DEV)
    la.la_rotary(q, None, freqs, q_out=q)
    _rotary_close(q[:, :, -50:], tail, np.arange(N - 50, N), freqs, BF)
    assert not q[:, :, :100].any()


# ---------------------------------------------------------------- gated head norm

def _norm_inputs(seed, B, H, N, M, dtype, heads, token_major):
    def rows(s):
        r = _randn(s, B, N, H, M, dtype=dtype)
        return r.transpose(1, 2) if token_major else r.transpose(1, 2).contiguous()
    x = _randn(seed, B, H, N, M, dtype=dtype)
    w = (1 + 0.2 * _randn(seed + 1, *((H, M) if heads else (M,)))).to(dtype)
    return x, rows(seed + 2) * 2, w, rows(seed + 3)


NORM_SHAPES = [(1, 1, 1, 64), (2, 3, 77, 64), (1, 2, 300, 128), (3, 5, 41, 96), (2, 1, 129, 8),
               (70, 4, 1, 72), (1, 16, 700, 24)]


@pytest.mark.parametrize("token_major", [False, True], ids=["head", "token"])
@pytest.mark.parametrize("heads", [False, True], ids=["shared", "each"])
@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", NORM_SHAPES, ids=lambda s: "b%dh%dn%dm%d" % s)
def test_norm_gate_and_gradients(la, shape, dtype, heads, token_major):
    B, H, N, M = shape
    x, z, w, dy = _norm_inputs(sum(shape), *shape, dtype, heads, token_major)
    if N > 1:
        x[0, 0, 1] = 0      # a row of zeros
        z[0, 0, 0] = -200.0  # a closed gate
    out = torch.empty(B, N, H, M, dtype=dtype, device=DEV).transpose(1, 2) if token_major else None
    y = la.la_norm_gate(x, z, w, out=out)
    u, f = HALF[dtype], 2.0 ** -24
    want = oracle.norm_gate(*map(_f64, (x, z, w)))
    grow = (M + 64 + 4 * np.abs(_f64(z))) * f
    assert np.all(np.abs(_f64(y) - want) <= (u + grow) * np.abs(want) + 1e-37)
    dz = torch.empty_like(dy)
    got = la.la_norm_gate_backward(x, z, w, dy, dz=dz)
    assert got[1] is dz
    wdx, wdz, wdw = oracle.norm_gate_backward(*map(_f64, (x, z, w, dy)))
    x6, z6, dy6 = map(_f64, (x, z, dy))
    w6 = _f64(w) if w.dim() == 1 else _f64(w)[None, :, None]
    r = 1 / np.sqrt(np.mean(x6 * x6, -1, keepdims=True) + 1e-6)
    s = 1 / (1 + np.exp(-z6))
    n = np.abs(x6 * r)
    dn = np.abs(dy6 * w6 * z6 * s)
    size = r * (dn + n * np.mean(dn * n, -1, keepdims=True))
    grow = (2 * M + 128 + 8 * np.max(np.abs(z6) * (np.abs(z6) < 50))) * f
    assert np.all(np.abs(_f64(got[0]) - wdx) <= u * np.abs(wdx) + grow * size + 1e-37)
    size = np.abs(dy6 * w6) * n * s * (1 + np.abs(z6) * (1 - s))
    assert np.all(np.abs(_f64(dz) - wdz) <= u * np.abs(wdz) + grow * size + 1e-30)
    size = np.sum(np.abs(dy6) * n * np.abs(z6) * s, axis=(0, 2) if heads else (0, 1, 2))
    rows = B * N * (1 if heads else H)
    assert got[2].shape == w.shape
    assert np.all(np.abs(_f64(got[2]) - wdw) <= u * np.abs(wdw) + (grow + min(rows, 4096) * f) * size + 1e-37)
    again = la.la_norm_gate_backward(x, z, w, dy)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


def test_float32_norm_gate_keeps_its_digits_at_every_gate(la):
    """Gates from -86 to 86 (where z sigmoid(z) is a normal float32). In half steps of 2^-24: the mean
    of M squares (M + 1 roundings, halved by the root), rsqrt (4), expf (4), the sigmoid's sum and
    quotient (5), products and the result (6): M / 2 + 20 in all; dz's sum of two terms and its
    factor 1 - s add 8, of the absolute terms."""
    H, M = 173, 8
    x, _, w, dy = _norm_inputs(9, 1, H, 1, M, FL, True, False)
    z = torch.linspace(-86, 86, H * M, device=DEV).view(1, H, 1, M)
    y = la.la_norm_gate(x, z, w)
    dx, dz, dw = la.la_norm_gate_backward(x, z, w, dy)
    x6, z6, w6, dy6 = map(_f64, (x, z, w, dy))
    f, grow = 2.0 ** -24, M / 2 + 20
    want = oracle.norm_gate(x6, z6, w6)
    assert np.all(np.abs(_f64(y) - want) <= grow * f * np.abs(want))
    wdx, wdz, wdw = oracle.norm_gate_backward(x6, z6, w6, dy6)
    assert np.all(np.abs(_f64(dw) - wdw) <= grow * f * np.abs(wdw))
    n = np.abs(x6) / np.sqrt(np.mean(x6 * x6, -1, keepdims=True) + 1e-6)
    s = np.where(z6 > 0, 1.0 / (1.0 + np.exp(-np.abs(z6))), np.exp(-np.abs(z6)) / (1.0 + np.exp(-np.abs(z6))))
    size = np.abs(dy6 * w6[None, :, None]) * n * s * (1.0 + np.abs(z6) / (1.0 + np.exp(z6)))
    assert np.all(np.abs(_f64(dz) - wdz) <= (grow + 8) * f * size)


def test_gates_that_are_all_but_closed(la):
    """As far as exp(z) is a normal float32 (in bf16 its next step down is not)."""
    for dtype, low in ((FL, -87.3), (BF, -87.0)):
        x, _, w, _ = _norm_inputs(3, 1, 1, 40, 64, dtype, False, False)
        z = torch.linspace(low, -86.0, 40 * 64, device=DEV).view(1, 1, 40, 64).to(dtype)
        want = oracle.norm_gate(*map(_f64, (x, z, w)))
        got = _f64(la.la_norm_gate(x, z, w))
        assert np.all(np.abs(got - want) <= (HALF[dtype] + 2.0 ** -14) * np.abs(want) + 2.0 ** -125)


def test_norm_gate_of_more_heads_than_a_grid_is_high(la):
    """w's gradient per head: one term each, dy n z s; a dozen float32 operations."""
    x, z, w, dy = _norm_inputs(4, 1, 70001, 1, 8, FL, True, False)
    dw = la.la_norm_gate_backward(x, z, w, dy)[2]
    want = oracle.norm_gate_backward(*map(_f64, (x, z, w, dy)))[2]
    grow = (8 + 64 + 8 * np.abs(_f64(z))[0, :, 0]) * 2.0 ** -24
    assert np.all(np.abs(_f64(dw) - want) <= grow * np.abs(want) + 1e-37)


def test_norm_gate_edges(la):
    x, z, w, dy = _norm_inputs(1, 2, 2, 6, 64, FL, False, False)
    e = x[:, :, :0].contiguous()
    assert la.la_norm_gate(e, e, w).shape == e.shape
    dx, dz, dw = la.la_norm_gate_backward(e, e, w, e)
    assert dx.shape == e.shape and dw.shape == w.shape and not dw.any()
    # an input that every head shares, and an eps of the caller's
    one = z[:, :1].expand(2, 2, 6, 64)
    assert torch.equal(la.la_norm_gate(x, one, w, eps=0.5), la.la_norm_gate(x, one.contiguous(), w, eps=0.5))
    want = oracle.norm_gate(_f64(x), _f64(one), _f64(w), eps=0.5)
    assert np.all(np.abs(_f64(la.la_norm_gate(x, one, w, eps=0.5)) - want) <= 2.0 ** -16 * np.abs(want))
    with pytest.raises(la.LAError):  # rows that do not start on 16 bytes
        bad = torch.zeros(2, 2, 6, 65, device=DEV)[..., :64]
        la.la_norm_gate(x, bad, w)
    with pytest.raises(la.LAError):
        la.la_norm_gate(x, z, w, eps=-1.0)


def test_rotary_and_norm_in_a_graph_on_two_streams(la):
    """Two graphs with their own workspaces replayed at once."""
    freqs, _ = la.la_rotary_freqs(64, device=DEV)
    runs = []
    for seed in (1, 2):
        x, z, w, dy = _norm_inputs(seed, 2, 4, 500, 64, BF, False, True)

        def step(x=x, z=z, w=w, dy=dy):
            q, k = la.la_rotary(x, z, freqs)
            return (q, k, *la.la_norm_gate_backward(q, k, w, dy))
        want = step()
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
        runs.append((graph, stream, got, want, (x, z, w, dy)))
    for _ in range(3):
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)
