"""la_layer_norm, la_ffn_gate, their gradients and the 8-bit checkpoints on the GPU against the
float64 oracle.

Tolerances, from the arithmetic. A result's own rounding is half a step of its type, HALF = eps / 2.
A float32 sum of n terms is off by n 2^-24 of the sum of magnitudes, on the tensor cores by n 2^-23
(their adder may cut off instead of rounding).

Layer norm: the mean is off by C 2^-24 mean|x|, the deviations by a rounding more, r by half of
(C + 8) 2^-24 and 2^-22 of the root, so n = (x - mean) r by N = (C + 16) 2^-23 (|n| + r mean|x|).
y: N |w| and two roundings more. The gradients: g = dy w, its mean and that of g n are off by
(C + 4) 2^-24 of their magnitudes and by N; dw and db by sums over the T rows.

Projections: a and u are off by A = C 2^-23 sum|x w|; |act'| <= 1.13, |act''| <= 1.13. The functions:
exponentials are off by 2 + 1.17 |z| steps of 2^-23, quotients and products by a few; for |z| below
30 all of it is below 2^-17 relative (erfc of the gelu: 2^-19). So da is off by
dh (1.13 (|u| A + U) + 2^-17 |u|) + HALF |da|, du by dh (1.13 A + 2^-17 |f|) + HALF |du|, each being
rounded to the inputs' type once (HALF), and the sums behind them add those up, with theirs.
The bounds add magnitudes; the errors have both signs, so that their 2-norms are compared too: a
result and the factor before it, rounded independently, are within 2 HALF / sqrt(3) of the 2-norm,
and the test allows 2 HALF (float32, whose sums' roundings count as well: sqrt(terms) 2^-24).
"""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
BF, FL = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, FL: 2.0 ** -24}
TYPES = pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
ACTS = pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])


@pytest.fixture(scope="module")
def la():
    from kernelized_causal_self_gb300 import build
    build.build()
    import kernelized_causal_self_gb300 as pkg
    pkg.load_library()
    return pkg


def _f64(t):
    return t.double().cpu().numpy()


def _randn(seed, *shape, dtype=FL, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)


def _within(got, want, tol, what=""):
    got = _f64(got)
    assert got.shape == want.shape, what
    off = np.abs(got - want)
    assert np.all(off <= tol + 1e-37), f"{what}: {np.max(off / (tol + 1e-37))} of the tolerance"


def _kept_like(*shape):
    return (torch.empty(shape, dtype=torch.int8, device=DEV),
            torch.empty((*shape[:-1], -(-shape[-1] // 32)), dtype=torch.uint8, device=DEV))


# --------------------------------------------------------------------- checkpoints

def _kept_equal(pair, x):
    codes, exps, values = oracle.checkpoint(_f64(x))
    assert np.array_equal(pair[1].cpu().numpy(), exps)
    assert np.array_equal(pair[0].cpu().numpy(), codes)
    return values


@TYPES
@pytest.mark.parametrize("shape", [(1, 8), (1, 32), (3, 40), (5, 7, 24), (2001, 96), (70, 1000), (300, 2248), (4, 65536)],
                         ids=str)
def test_checkpoint(la, shape, dtype):
    x = _randn(1, *shape, dtype=dtype) * torch.exp(8 * _randn(2, *shape[:-1], 1)).to(dtype)
    pair = la.la_checkpoint(x)
    values = _kept_equal(pair, x)
    for out in (BF, FL):
        back = la.la_checkpoint_restore(*pair, dtype=out)
        assert back.dtype == out and np.array_equal(_f64(back), values)  # (7 bits: exact in bf16)
    assert la.la_checkpoint_restore(*pair).dtype == BF
    again = la.la_checkpoint(la.la_checkpoint_restore(*pair, dtype=FL))
    assert np.array_equal(_f64(la.la_checkpoint_restore(*again, dtype=FL)), values)


@TYPES
def test_checkpoint_of_values_at_the_borders(la, dtype):
    x = torch.zeros(9, 72, device=DEV)
    x[0, :4] = torch.tensor([127.0, 64.5, -63.5, 0.5])       # ties
    x[1, :3] = torch.tensor([127.5, 1.0, 3.0])
    x[2, :3] = torch.tensor([1e-38, -1e-40, 2.0 ** -127])    # below the smallest step, or near it
    x[3, 40], x[3, 3] = float("inf"), 5.0
    x[4, 71], x[4, 3] = float("nan"), 5.0
    x[5, :2] = torch.tensor([3.3e38, -1e38])
    x[6] = float("-inf")
    x[7, 64:] = torch.tensor([255.0, 254.0, 253.0, 1.0, 2.0, 3.0, -255.0, 128.0])
    x = x.to(dtype)
    pair = la.la_checkpoint(x)
    values = _kept_equal(pair, x)
    back = _f64(la.la_checkpoint_restore(*pair, dtype=dtype))
    assert np.array_equal(back, values, equal_nan=True)
    assert np.isnan(back[3, 32:64]).all() and back[3, 3] == 5.0 and np.isnan(back[4, 64:]).all()


@TYPES
def test_checkpoint_layouts(la, dtype):
    big = _randn(3, 6, 11, 3, 48, dtype=dtype)
    x = big[:, :, 1]                                   # rows 144 apart
    assert not x.is_contiguous()
    pair = _kept_like(6, 11, 48)
    got = la.la_checkpoint(x, checkpoint=pair)
    assert got[0] is pair[0] and got[1] is pair[1]
    values = _kept_equal(pair, x)
    keep = big.clone()
    out = la.la_checkpoint_restore(*pair, out=x)
    assert out is x and np.array_equal(_f64(x), values)
    assert torch.equal(big[:, :, 0], keep[:, :, 0]) and torch.equal(big[:, :, 2], keep[:, :, 2])
    none = la.la_checkpoint(x[:0])
    assert none[0].shape == (0, 11, 48) and la.la_checkpoint_restore(*none, dtype=dtype).shape == (0, 11, 48)
    one = la.la_checkpoint(x[0, 0])
    assert torch.equal(one[0], pair[0][0, 0]) and torch.equal(one[1], pair[1][0, 0])


# ---------------------------------------------------------------------- layer norm

def _norm_parts(x, w, eps):
    x, w = _f64(x), _f64(w)
    C = x.shape[-1]
    d = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n = d * r
    return n, r, (C + 16) * 2.0 ** -23 * (np.abs(n) + r * np.abs(x).mean(-1, keepdims=True))


def _norm_close(got, x, w, b, dtype, eps=1e-5):
    want = oracle.layer_norm(_f64(x), _f64(w), None if b is None else _f64(b), eps)
    n, _, off = _norm_parts(x, w, eps)
    wb = np.abs(n * _f64(w)) + (0 if b is None else np.abs(_f64(b)))
    assert got.dtype == dtype
    _within(got, want, HALF[dtype] * np.abs(want) + off * np.abs(_f64(w)) + 2.0 ** -22 * wb, "y")


def _norm_grads_close(got, x, w, dy, dtype, eps=1e-5):
    """x: the norm's input in float64 or a tensor"""
    x = x if torch.is_tensor(x) else torch.from_numpy(x)
    n, r, off = _norm_parts(x, w, eps)
    x, w, dy = _f64(x), _f64(w), _f64(dy)
    C, T = x.shape[-1], x.size // x.shape[-1]
    want = oracle.layer_norm_backward(x, w, dy, eps)
    g = np.abs(dy * w)
    mean = lambda t: t.mean(-1, keepdims=True)  # noqa: E731
    n = np.abs(n)
    s = (C + 16) * 2.0 ** -23
    tol = s * (g + mean(g) + n * mean(g * n)) + off * mean(g * n) + n * mean(g * off)
    rows = tuple(range(x.ndim - 1))
    u = HALF[dtype]
    assert all(t.dtype == dtype for t in got)
    _within(got[0], want[0], u * np.abs(want[0]) + r * tol, "dx")
    sums = (T + 8) * 2.0 ** -24
    _within(got[1], want[1], u * np.abs(want[1]) + (np.abs(dy) * (off + sums * n)).sum(rows), "dw")
    _within(got[2], want[2], u * np.abs(want[2]) + sums * np.abs(dy).sum(rows), "db")


@TYPES
@pytest.mark.parametrize("shape", [(1, 8), (1, 512), (3, 64), (2, 5, 72), (129, 128), (33, 136), (300, 256), (40, 264),
                                   (257, 512), (65, 520), (19, 1000), (7, 2048), (10, 2056), (6, 4104), (5, 8192),
                                   (3, 8200), (2, 16384), (4001, 64)], ids=str)
def test_layer_norm(la, shape, dtype):
    C = shape[-1]
    x = _randn(1, *shape, dtype=dtype, scale=2.0) + 1.5
    w, b, dy = _randn(2, C, dtype=dtype), _randn(3, C, dtype=dtype), _randn(4, *shape, dtype=dtype)
    _norm_close(la.la_layer_norm(x, w, b), x, w, b, dtype)
    _norm_close(la.la_layer_norm(x, w, eps=0.5), x, w, None, dtype, 0.5)
    grads = la.la_layer_norm_backward(x, w, dy)
    _norm_grads_close(grads, x, w, dy, dtype)
    again = la.la_layer_norm_backward(x, w, dy)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))
    # through a checkpoint: written on the way, read instead of x
    pair = _kept_like(*shape)
    y = la.la_layer_norm(x, w, b, checkpoint=pair)
    assert torch.equal(y, la.la_layer_norm(x, w, b))
    values = _kept_equal(pair, x)
    _norm_grads_close(la.la_layer_norm_backward(pair, w, dy), values, w, dy, dtype)


@TYPES
def test_layer_norm_layouts(la, dtype):
    big, w, b = _randn(1, 9, 4, 3, 96, dtype=dtype), _randn(2, 96, dtype=dtype), _randn(3, 96, dtype=dtype)
    x, keep = big[:, :, 1], big.clone()
    want = la.la_layer_norm(x.contiguous(), w, b)
    assert torch.equal(la.la_layer_norm(x, w, b), want)
    dybig = _randn(4, 9, 4, 2, 96, dtype=dtype)
    dy = dybig[:, :, 0]
    grads = la.la_layer_norm_backward(x.contiguous(), w, dy.contiguous())
    dx = torch.full((9, 4, 200), 3.0, device=DEV, dtype=dtype)
    dw, db = torch.empty_like(w), torch.empty_like(w)
    got = la.la_layer_norm_backward(x, w, dy, dx=dx[..., :96], dw=dw, db=db)
    assert all(torch.equal(p, q) for p, q in zip(got, grads)) and got[1] is dw and got[2] is db
    assert torch.all(dx[..., 96:] == 3.0)
    # over dy, over x, and in place
    over = dybig.clone()
    got = la.la_layer_norm_backward(x, w, over[:, :, 0], dx=over[:, :, 0])
    assert torch.equal(over[:, :, 0], grads[0]) and torch.equal(over[:, :, 1], dybig[:, :, 1])
    assert torch.equal(got[1], grads[1])
    over = big.clone()
    la.la_layer_norm_backward(over[:, :, 1], w, dy, dx=over[:, :, 1])
    assert torch.equal(over[:, :, 1], grads[0]) and torch.equal(over[:, :, 2], keep[:, :, 2])
    la.la_layer_norm(x, w, b, out=x)
    assert torch.equal(x, want) and torch.equal(big[:, :, 0], keep[:, :, 0]) and torch.equal(big[:, :, 2], keep[:, :, 2])
    # no rows
    none = la.la_layer_norm_backward(x[:0], w, dy[:0])
    assert none[0].shape == (0, 4, 96) and not none[1].any() and not none[2].any()
    assert la.la_layer_norm(x[:0], w, b).shape == (0, 4, 96)


@TYPES
def test_layer_norm_of_rows_that_are_not_finite_or_flat(la, dtype):
    x, w, dy = _randn(1, 70, 264, dtype=dtype), _randn(2, 264, dtype=dtype), _randn(3, 70, 264, dtype=dtype)
    clean = la.la_layer_norm(x, w)
    x[3, 5], x[40, 7] = float("nan"), float("inf")
    x[50] = 2.5
    y = la.la_layer_norm(x, w)
    others = [i for i in range(70) if i not in (3, 40, 50)]
    assert torch.equal(y[others], clean[others]) and y[3].isnan().all() and y[40].isnan().all()
    assert not y[50].any()
    # eps 0: a flat row is 0 / 0 as in the formula, and the rows past the last add nothing
    y = la.la_layer_norm(x, w, eps=0.0)
    assert y[50].isnan().all() and y[others].isfinite().all()
    keep = others[:67]
    grads = la.la_layer_norm_backward(x[keep], w, dy[keep], eps=0.0)
    _norm_grads_close(grads, x[keep], w, dy[keep], dtype, 0.0)


def test_layer_norm_of_a_far_mean(la):
    """Deviations are summed behind the mean: one of 4096 costs 2^12 of the digits, not its square."""
    x = _randn(1, 50, 512) + 4096.0
    w = torch.ones(512, device=DEV)
    _norm_close(la.la_layer_norm(x, w), x, w, None, FL)
    n, _, off = _norm_parts(x, w, 1e-5)
    got = _f64(la.la_layer_norm(x, w))
    assert np.abs(got - n).max() < 2e-3


# ------------------------------------------------------------------------ projections

def _ffn_parts(x, wg, wu, act):
    x, wg, wu = (_f64(t) for t in (x, wg, wu))
    c = x.shape[-1] * 2.0 ** -23
    A, U = c * (np.abs(x) @ np.abs(wg).T), c * (np.abs(x) @ np.abs(wu).T)
    a, u = x @ wg.T, x @ wu.T
    f, df = oracle.activation(a, act)
    return a, u, f, df, A, U


def _norm2(got, want, limit, what):
    rel = np.linalg.norm(_f64(got) - want) / max(np.linalg.norm(want), 1e-300)
    assert rel <= limit, f"{what}: {rel} of its 2-norm, {limit} allowed"


def _ffn_close(h, x, wg, wu, act, dtype):
    a, u, f, df, A, U = _ffn_parts(x, wg, wu, act)
    want = f * u
    tol = HALF[dtype] * np.abs(want) + 1.13 * A * np.abs(u) + (np.abs(f) + 1.13 * A) * U + 2.0 ** -17 * np.abs(a * u)
    assert h.dtype == dtype
    _within(h, want, tol, "h")
    # (2^-17 a: the functions' own bound, of which float32 takes a small part)
    terms = np.sqrt(x.shape[-1]) + 16
    _norm2(h, want, 2 * HALF[BF] if dtype == BF else 4 * terms * 2.0 ** -24, "h")


def _ffn_grads_close(grads, x, wg, wu, dh, act, dtype, kept=None):
    a, u, f, df, A, U = _ffn_parts(x, wg, wu, act)
    if kept is not None:
        (a, u), A, U = kept, 0 * A, 0 * U
        f, df = oracle.activation(a, act)
    want = oracle.ffn_gate_backward(_f64(x), _f64(wg), _f64(wu), _f64(dh), act, kept)
    x, wg, wu, dh = (np.abs(_f64(t)) for t in (x, wg, wu, dh))
    half = HALF[dtype]
    da, du = dh * np.abs(u * df), dh * np.abs(f)
    eda = dh * (1.13 * (np.abs(u) * A + U) + 2.0 ** -17 * np.abs(u)) + half * da
    edu = dh * (1.13 * A + 2.0 ** -17 * np.abs(a)) + half * du
    T, F = da.shape
    c = 2.0 ** -23
    tols = (eda @ wg + edu @ wu + 2 * F * c * (da @ wg + du @ wu),
            eda.T @ x + T * c * (da.T @ x), edu.T @ x + T * c * (du.T @ x))
    terms = np.sqrt(max(2 * F, T, x.shape[-1])) + 16
    for name, g, w, tol in zip(("dx", "dwg", "dwu"), grads, want, tols):
        assert g.dtype == dtype
        _within(g, w, tol + half * np.abs(w), name)
        _norm2(g, w, 2 * HALF[BF] if dtype == BF else 4 * terms * 2.0 ** -24, name)


def _ffn_inputs(T, C, F, dtype, seed=1):
    return (_randn(seed, T, C, dtype=dtype), _randn(seed + 1, F, C, dtype=dtype, scale=C ** -0.5),
            _randn(seed + 2, F, C, dtype=dtype, scale=C ** -0.5), _randn(seed + 3, T, F, dtype=dtype))


FFN_SIZES = [(1, 8, 8), (1, 64, 128), (1, 2048, 1032), (2, 72, 40), (5, 136, 264), (7, 1000, 24), (8, 256, 680), (9, 520, 72), (16, 64, 64), (17, 200, 96), (33, 64, 1032),
             (64, 512, 256), (65, 128, 136), (127, 64, 128), (128, 128, 256), (129, 264, 136), (200, 1032, 8),
             (256, 256, 512), (300, 8, 520), (513, 104, 280), (777, 256, 680), (1500, 264, 1032),
             (2100, 136, 520), (512, 72, 256), (513, 72, 256), (1024, 72, 256), (1025, 72, 256),
             (1032, 264, 264)]


@TYPES
@pytest.mark.parametrize("size", FFN_SIZES, ids=lambda s: "t%dc%df%d" % s)
def test_ffn_gate(la, size, dtype):
    act = ("silu", "gelu", "gelu_tanh")[sum(size) // 8 % 3]
    x, wg, wu, dh = _ffn_inputs(*size, dtype)
    h = la.la_ffn_gate(x, wg, wu, activation=act)
    _ffn_close(h, x, wg, wu, act, dtype)
    grads = la.la_ffn_gate_backward(x, wg, wu, dh, activation=act)
    _ffn_grads_close(grads, x, wg, wu, dh, act, dtype)
    assert torch.equal(h, la.la_ffn_gate(x, wg, wu, activation=act))
    again = la.la_ffn_gate_backward(x, wg, wu, dh, activation=act)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


@TYPES
@ACTS
@pytest.mark.parametrize("size", [(1, 64, 72), (40, 256, 264), (300, 72, 136), (256, 128, 384)], ids=lambda s: "t%dc%df%d" % s)
def test_ffn_gate_with_a_checkpoint(la, size, act, dtype):
    T, C, F = size
    x, wg, wu, dh = _ffn_inputs(*size, dtype)
    pair = _kept_like(T, 2, F)
    h = la.la_ffn_gate(x, wg, wu, activation=act, checkpoint=pair)
    _ffn_close(h, x, wg, wu, act, dtype)
    # the stored products are within half a step, and what the sums are off, of the exact ones
    a, u, _, _, A, U = _ffn_parts(x, wg, wu, act)
    codes, exps = (t.cpu().numpy() for t in pair)
    step = np.repeat(2.0 ** (exps.astype(float) - 127), 32, -1)[..., :F]
    kept = codes * step
    for i, (want, off) in enumerate(((a, A), (u, U))):
        assert np.all(np.abs(kept[:, i] - want) <= step[:, i] / 2 + off)
        top = np.abs(np.pad(want, ((0, 0), (0, -F % 32))).reshape(T, -1, 32)).max(-1)
        slack = np.abs(np.pad(off, ((0, 0), (0, -F % 32))).reshape(T, -1, 32)).max(-1)
        unit = 2.0 ** (exps[:, i].astype(float) - 127)
        assert np.all(top - slack < 127.5 * unit) and np.all(top + slack >= 127.5 * unit / 2)
    assert np.abs(codes.astype(int)).max() <= 127
    grads = la.la_ffn_gate_backward(x, wg, wu, dh, activation=act, checkpoint=pair)
    _ffn_grads_close(grads, x, wg, wu, dh, act, dtype, (kept[:, 0], kept[:, 1]))


@TYPES
@ACTS
def test_ffn_gradients_by_differences(la, act, dtype):
    """Along a direction in each argument: (f(+) - f(-)) / 2 of the float64 definition."""
    x, wg, wu, dh = _ffn_inputs(48, 72, 104, dtype)
    grads = la.la_ffn_gate_backward(x, wg, wu, dh, activation=act)
    args = [_f64(t) for t in (x, wg, wu)]
    rng = np.random.default_rng(3)
    for k, g in enumerate(grads):
        d = rng.normal(size=args[k].shape)
        d /= np.linalg.norm(d)
        f = lambda t: (_f64(dh) * oracle.ffn_gate(*args[:k], t, *args[k + 1:], act)).sum()  # noqa: E731
        slope = (f(args[k] + 1e-5 * d) - f(args[k] - 1e-5 * d)) / 2e-5
        # a unit direction meets the gradient's error by its 2-norm at most
        off = abs(slope - (_f64(g) * d).sum()) / np.linalg.norm(_f64(g))
        assert off <= (2 * HALF[BF] if dtype == BF else 4 * 32 * 2.0 ** -24) + 1e-9


@TYPES
@pytest.mark.parametrize("a, b", [(9, 10), (45, 50)])
def test_ffn_layouts(la, a, b, dtype):
    T = a * b
    x, wg, wu, dh = _ffn_inputs(T, 72, 136, dtype)
    want = la.la_ffn_gate(x, wg, wu)
    grads = la.la_ffn_gate_backward(x, wg, wu, dh)
    xs = torch.full((a, b, 200), 7.0, device=DEV, dtype=dtype)
    xs[..., 64:136] = x.view(a, b, 72)
    hs = torch.full((a, b, 3, 136), 5.0, device=DEV, dtype=dtype)
    xv = xs[..., 64:136]
    h = la.la_ffn_gate(xv, wg, wu, out=hs[:, :, 1])
    assert h.shape == (a, b, 136) and torch.equal(h.reshape(T, 136), want)
    assert torch.all(hs[:, :, 0] == 5.0) and torch.all(hs[:, :, 2] == 5.0)
    hs[:, :, 1] = dh.view(a, b, 136)
    dxs = torch.full((a, b, 80), 5.0, device=DEV, dtype=dtype)
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    got = la.la_ffn_gate_backward(xv, wg, wu, hs[:, :, 1], dx=dxs[..., :72], dwg=dwg, dwu=dwu)
    assert torch.equal(got[0].reshape(T, 72), grads[0]) and torch.equal(dwg, grads[1]) and torch.equal(dwu, grads[2])
    assert torch.all(dxs[..., 72:] == 5.0)
    pair = _kept_like(a, b, 2, 136)
    la.la_ffn_gate(xv, wg, wu, checkpoint=pair)
    flat = _kept_like(T, 2, 136)
    la.la_ffn_gate(x, wg, wu, checkpoint=flat)
    assert torch.equal(pair[0].reshape(T, 2, 136), flat[0]) and torch.equal(pair[1].reshape(T, 2, 5), flat[1])
    one = la.la_ffn_gate(x[4], wg, wu)
    assert one.shape == (136,)
    _ffn_close(one[None], x[4:5], wg, wu, "silu", dtype)
    none = la.la_ffn_gate_backward(x[:0], wg, wu, dh[:0])
    assert none[0].shape == (0, 72) and not none[1].any() and not none[2].any()
    assert la.la_ffn_gate(x[:0], wg, wu).shape == (0, 136)


@TYPES
@pytest.mark.parametrize("T", [3, 40, 300, 1600])
def test_ffn_rows_that_are_not_finite_stay_alone(la, T, dtype):
    x, wg, wu, dh = _ffn_inputs(T, 136, 200, dtype)
    bad = T // 2
    y = x.clone()
    y[bad, 3] = float("nan")
    rows = [i for i in range(T) if i != bad]
    for pair in (None, _kept_like(T, 2, 200)):  # (few tokens without one take another kernel, and order)
        clean = la.la_ffn_gate(x, wg, wu, checkpoint=pair)
        h = la.la_ffn_gate(y, wg, wu, checkpoint=pair)
        assert h[bad].isnan().all() and torch.equal(h[rows], clean[rows])
    assert torch.all(pair[1][bad] == 255) and torch.all(pair[1][rows] != 255)
    grads = la.la_ffn_gate_backward(x, wg, wu, dh)
    got = la.la_ffn_gate_backward(y, wg, wu, dh)
    assert got[0][bad].isnan().all() and torch.equal(got[0][rows], grads[0][rows])
    assert got[1].isnan().all()  # da of the row is NaN, so every sum over the rows is
    # large values: exponentials over- and underflow without a NaN
    big = la.la_ffn_gate(x * 300, wg, wu)
    assert big.isfinite().all()


@TYPES
@pytest.mark.parametrize("T", [70, 2100])
def test_columns_of_one_buffer(la, T, dtype):
    """Inputs and outputs may be columns of one buffer, which share no memory."""
    C, F = 72, 136
    x, wg, wu, dh = _ffn_inputs(T, C, F, dtype)
    w = _randn(9, C, dtype=dtype)
    buf = torch.full((T, 2 * C + 2 * F), 2.0, dtype=dtype, device=DEV)
    xv, yv, hv, dhv = buf[:, :C], buf[:, C:2 * C], buf[:, 2 * C:2 * C + F], buf[:, 2 * C + F:]
    xv.copy_(x)
    dhv.copy_(dh)
    y = la.la_layer_norm(x, w)
    h = la.la_ffn_gate(y, wg, wu)
    la.la_layer_norm(xv, w, out=yv)
    la.la_ffn_gate(yv, wg, wu, out=hv)
    want = la.la_ffn_gate_backward(y, wg, wu, dh)
    got = la.la_ffn_gate_backward(yv, wg, wu, dhv, dx=xv)
    for p, q in ((yv, y), (hv, h), (dhv, dh), *zip(got, want)):
        assert torch.equal(p, q)


def test_more_elements_than_32_bits_count(la):
    """270000 rows of 8192: the last rows' results are those of the rows alone, bit for bit."""
    T, C, F, n = 270000, 64, 8192, 300
    x, wg, wu, _ = _ffn_inputs(T, C, F, BF)
    last = x[-n:].contiguous()
    pair, own = _kept_like(T, 2, F), _kept_like(n, 2, F)
    h, hl = la.la_ffn_gate(x, wg, wu, checkpoint=pair), la.la_ffn_gate(last, wg, wu, checkpoint=own)
    assert h.numel() > 2 ** 31 and torch.equal(h[-n:], hl)
    assert torch.equal(pair[0][-n:], own[0]) and torch.equal(pair[1][-n:], own[1])
    for kept, kl in ((None, None), (pair, own)):
        grads, gl = la.la_ffn_gate_backward(x, wg, wu, h, checkpoint=kept), la.la_ffn_gate_backward(last, wg, wu, hl, checkpoint=kl)
        # (dx's sums may be cut at other places)
        _norm2(grads[0][-n:], _f64(gl[0]), HALF[BF], "dx")
        del grads
    w, b = _randn(8, F, dtype=BF), _randn(9, F, dtype=BF)
    del pair
    pair = _kept_like(T, F)
    y = la.la_layer_norm(h, w, b, checkpoint=pair)
    kl = la.la_checkpoint(hl)
    assert torch.equal(y[-n:], la.la_layer_norm(hl, w, b))
    assert torch.equal(pair[0][-n:], kl[0]) and torch.equal(pair[1][-n:], kl[1])
    again = la.la_checkpoint(h)
    assert torch.equal(again[0], pair[0]) and torch.equal(again[1], pair[1])
    assert torch.equal(la.la_checkpoint_restore(*again)[-n:], la.la_checkpoint_restore(*kl))
    for xin, xl in ((h, hl), (pair, kl)):
        dx = la.la_layer_norm_backward(xin, w, y)[0]
        assert torch.equal(dx[-n:], la.la_layer_norm_backward(xl, w, y[-n:].contiguous())[0])


@pytest.mark.parametrize("T", [300, 600])
def test_calls_on_another_stream_and_in_a_graph(la, T):
    """A norm, projections and the way back, captured and replayed on new inputs in two graphs, with
    workspaces of their own, and on two streams at once."""
    C, F = 136, 264
    x, wg, wu, dh = _ffn_inputs(T, C, F, BF)
    w, b = _randn(9, C, dtype=BF), _randn(10, C, dtype=BF)

    def step(x):
        pair = _kept_like(T, 2, F)
        y = la.la_layer_norm(x, w, b)
        h = la.la_ffn_gate(y, wg, wu, checkpoint=pair)
        dy, dwg, dwu = la.la_ffn_gate_backward(y, wg, wu, dh, checkpoint=pair)
        again = la.la_ffn_gate_backward(y, wg, wu, dh)
        return (h, dwg, dwu, *la.la_layer_norm_backward(x, w, dy), *again, la.la_ffn_gate(y, wg, wu))
    ins = [_randn(20 + i, T, C, dtype=BF) for i in range(4)]
    want = [[t.clone() for t in step(v)] for v in ins]
    torch.cuda.synchronize()
    graphs, outs, held = [], [], []
    for _ in range(2):
        held.append(ins[0].clone())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(held[-1]))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for turn in range(2):
        for i, (g, s) in enumerate(zip(graphs, streams)):
            with torch.cuda.stream(s):
                held[i].copy_(ins[2 * turn + i])
                g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            for got, ref in zip(outs[i], want[2 * turn + i]):
                assert torch.equal(got, ref)
    results = []
    for s, v in zip(streams, ins):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            results.append(step(v))
    torch.cuda.synchronize()
    for got, ref in zip(results, want):
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


class _Nothing:
    """A marshalling module that does no call itself."""

    def __getattr__(self, name):
        return lambda *args: NotImplemented


@TYPES
def test_calls_marshalled_in_cpp_are_those_in_python(la, monkeypatch, dtype):
    T, C, F = 50, 72, 136
    x, wg, wu, dh = _ffn_inputs(T, C, F, dtype)
    w, b, big = _randn(7, C, dtype=dtype), _randn(8, C, dtype=dtype), x.reshape(5, 10, C)

    def calls():
        pair, both = la.la_checkpoint(big), (torch.zeros(T, 2, F, dtype=torch.int8, device=DEV),
                                             torch.zeros(T, 2, 5, dtype=torch.uint8, device=DEV))
        kept, out = la.la_checkpoint(x), torch.zeros_like(big)
        h = la.la_ffn_gate(x, wg, wu, "gelu", checkpoint=both)
        assert la.la_layer_norm(big, w, b, out=out) is out
        return [*pair, la.la_checkpoint_restore(*pair), la.la_checkpoint_restore(*pair, dtype=FL), out,
                la.la_layer_norm(big, w, eps=0.25), la.la_layer_norm(x, w, b, checkpoint=kept), *kept,
                *la.la_layer_norm_backward(big, w, big), *la.la_layer_norm_backward(kept, w, x, eps=0.5),
                h, *both, la.la_ffn_gate(big, wg, wu), la.la_ffn_gate(x[0], wg, wu, out=torch.zeros(F, dtype=dtype, device=DEV)),
                *la.la_ffn_gate_backward(big, wg, wu, dh.view(5, 10, F)),
                *la.la_ffn_gate_backward(x, wg, wu, dh, "gelu", checkpoint=both)]
    n0 = la.la_kernel_launches()
    fast, n1 = calls(), la.la_kernel_launches()
    monkeypatch.setattr(la, "_fast", _Nothing())
    slow, n2 = calls(), la.la_kernel_launches()
    assert n1 - n0 == n2 - n1
    for p, q in zip(fast, slow):
        assert p.shape == q.shape and p.dtype == q.dtype and p.device == q.device and torch.equal(p, q)


def test_a_status_is_left_in_the_workspace(la):
    """The tensor-core calls clear the status header of a workspace of any contents."""
    for dtype in (BF, FL):
        x, wg, wu, dh = _ffn_inputs(2000, 64, 136, dtype)
        dt = la.LA_BF16 if dtype == BF else la.LA_F32
        assert la.la_ffn_gate_workspace_bytes(2000, 64, 136, False, dt) > 0
        for pair in (None, _kept_like(2000, 2, 136)):
            ws = torch.full((la.la_ffn_gate_workspace_bytes(2000, 64, 136, pair is not None, dt),), 3, dtype=torch.uint8,
                            device=DEV)
            la.la_ffn_gate(x, wg, wu, checkpoint=pair, workspace=ws)
            assert la.la_workspace_status(ws) == la.LA_OK
            ws = torch.full((la.la_ffn_gate_backward_workspace_bytes(2000, 64, 136, dt),), 3, dtype=torch.uint8, device=DEV)
            la.la_ffn_gate_backward(x, wg, wu, dh, checkpoint=pair, workspace=ws)
            assert la.la_workspace_status(ws) == la.LA_OK


def test_outputs_that_share_memory_are_refused(la):
    x, wg, wu, dh = _ffn_inputs(40, 72, 72, BF)
    w = _randn(5, 72, dtype=BF)
    for call in (lambda: la.la_ffn_gate(x, wg, wu, out=x), lambda: la.la_ffn_gate(x, wg, wu, out=wg[:40]),
                 lambda: la.la_ffn_gate_backward(x, wg, wu, dh, dx=x), lambda: la.la_ffn_gate_backward(x, wg, wu, dh, dwg=wu),
                 lambda: la.la_layer_norm(x[:39], w, out=x[1:]), lambda: la.la_layer_norm(x[:1], w, out=w[None]),
                 lambda: la.la_layer_norm_backward(x, w, dh, dw=w)):
        before = la.la_kernel_launches()
        with pytest.raises(la.LAError, match="invalid argument"):
            call()
        assert la.la_kernel_launches() == before


def test_a_workspace_of_the_callers(la):
    T, C, F = 200, 128, 264
    x, wg, wu, dh = _ffn_inputs(T, C, F, BF)
    ws = torch.full((la.la_ffn_gate_backward_workspace_bytes(T, C, F),), 255, dtype=torch.uint8, device=DEV)
    got = la.la_ffn_gate_backward(x, wg, wu, dh, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(got, la.la_ffn_gate_backward(x, wg, wu, dh)))
    fws = torch.full((la.la_ffn_gate_workspace_bytes(T, C, F),), 255, dtype=torch.uint8, device=DEV)
    assert torch.equal(la.la_ffn_gate(x, wg, wu, workspace=fws), la.la_ffn_gate(x, wg, wu))
    nws = torch.full((la.la_layer_norm_workspace_bytes(T, C),), 255, dtype=torch.uint8, device=DEV)
    w = _randn(7, C, dtype=BF)
    got = la.la_layer_norm_backward(x, w, x, workspace=nws)
    assert all(torch.equal(p, q) for p, q in zip(got, la.la_layer_norm_backward(x, w, x)))
    with pytest.raises(ValueError, match="workspace too small"):
        la.la_ffn_gate_backward(x, wg, wu, dh, workspace=ws[:-1])
    with pytest.raises(la.LAError):
        la.la_layer_norm(x[:, 4:124], w[:120])  # rows that do not begin at 16 bytes


@TYPES
def test_the_feed_forward_half_of_a_layer(la, dtype):
    """norm -> projections -> back, everything kept in 8 bits, against the same chain in float64 on
    the values that the checkpoints stand for."""
    T, C, F = 150, 128, 344
    x, wg, wu, dh = _ffn_inputs(T, C, F, dtype)
    w, b = 1 + _randn(8, C, dtype=dtype, scale=0.1), _randn(9, C, dtype=dtype, scale=0.1)
    kx, kau = _kept_like(T, C), _kept_like(T, 2, F)
    y = la.la_layer_norm(x, w, b, checkpoint=kx)
    h = la.la_ffn_gate(y, wg, wu, activation="gelu", checkpoint=kau)
    dy, dwg, dwu = la.la_ffn_gate_backward(y, wg, wu, dh, activation="gelu", checkpoint=kau)
    dx, dw, db = la.la_layer_norm_backward(kx, w, dy)
    _norm_close(y, x, w, b, dtype)
    _ffn_close(h, y, wg, wu, "gelu", dtype)
    au = _f64(la.la_checkpoint_restore(*kau, dtype=FL))
    _ffn_grads_close((dy, dwg, dwu), y, wg, wu, dh, "gelu", dtype, (au[:, 0], au[:, 1]))
    _norm_grads_close((dx, dw, db), _f64(la.la_checkpoint_restore(*kx, dtype=FL)), w, dy, dtype)
    # and the whole against the exact gradients: a block's values are off by 2^-7 of its largest at
    # most, 2^-8 of their 2-norm and less (a uniform error of half a step, the largest a few norms)
    yx = oracle.layer_norm(_f64(x), _f64(w), _f64(b))
    want = oracle.ffn_gate_backward(yx, _f64(wg), _f64(wu), _f64(dh), "gelu")
    for got, ref in zip((dy, dwg, dwu), want):
        _norm2(got, ref, 0.05, "chain")
