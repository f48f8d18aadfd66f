"""The gated recurrence on the GPU (la_forward_gated, la_prefill_gated, la_extend_gated,
la_decode_step_gated, la_backward_gated) against the fp64 oracle.

Tolerances. Let u be half a step of the outputs' type (bf16 2^-8, float32 2^-24) and A the
oracle's result for the absolute values of the inputs: the sum of the absolute terms that an
output sums.
 - A bf16 output is rounded once (u |want|), and in each of its terms one operand may have been
   rounded to bf16 (a chunk's weights, or the state; u A together, being one or the other, and
   u of the product of two more at most: u^2, absorbed by the float32 share).
 - Float32 arithmetic: a term passes through at most N + D + M + 64 roundings of 2^-24 each
   (the walk over the tokens, the sums over a head, an exponential).
 - A final state is float32; from bf16 inputs its products carry at least 16 bits (2^-17).
 - dg sums differences of q . dq and k . dk over up to all N tokens, whose own float32 errors do
   not cancel: 2^-24 (N + D + M + 64) of the sum over the tokens of the absolute dots.
With inputs of random signs the roundings are independent, which bounds the 2-norm of the error
more tightly than A does: at most three roundings (operand, state, output), each of 2-norm at
most u / sqrt(3) of the result's: sqrt(3) u / sqrt(3) = u in all, and for float32 the walk's
roundings add up as sqrt(N + D + M + 64) u.
"""

import numpy as np
import pytest

import oracle

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

DEV = "cuda:0"
F32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: F32}


@pytest.fixture(scope="module")
def la():
    from kernelized_causal_self_gb300 import build
    build.build()
    import kernelized_causal_self_gb300 as pkg
    pkg.load_library()
    return pkg


def _f64(t):
    return t.detach().double().cpu().numpy()


def _gates(gen, shape, kind):
    x = torch.randn(shape, generator=gen, device=DEV)
    if kind == "none":
        return torch.zeros(shape, device=DEV)
    if kind == "slow":
        return torch.nn.functional.logsigmoid(x + 2.0) / 16.0
    if kind == "strong":
        return -5.0 * torch.exp(0.5 * x)
    g = -torch.exp(torch.linspace(-6.0, 1.0, shape[1], device=DEV).view(1, -1, *[1] * (len(shape) - 2)) + 0.5 * x)
    if kind == "resets":  # empties the state now and then: -inf, and the type's lowest value
        g = torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.05, -torch.inf, g)
        g = torch.where(torch.rand(shape, generator=gen, device=DEV) < 0.03,
                        torch.finfo(torch.bfloat16).min, g)
    return g


def _inputs(seed, B, H, N, D, M, dtype, gate="mixed"):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    r = lambda d: (torch.randn((B, H, N, d), generator=gen, device=DEV) * d ** -0.5).to(dtype)  # noqa: E731
    q, k, v, do = r(D), r(D), r(M), r(M)
    S0, dS = (torch.randn((B, H, D, M), generator=gen, device=DEV) * 0.3 for _ in range(2))
    return q, k, v, _gates(gen, (B, H, N), gate).to(dtype), do, S0, dS


def _close(got, want, absolute, dtype, chain, what, extra=0.0, state=False):
    """The elementwise and, where the result is large enough for statistics, the 2-norm bound."""
    got = _f64(got)
    assert got.shape == want.shape
    assert np.all(np.isfinite(got)), what
    low = dtype == torch.bfloat16
    u = HALF[dtype]
    if state:
        each = (2.0 ** -17 if low else 0.0) * absolute + chain * F32 * absolute
        norm = (2.0 ** -17 if low else 0.0) + chain ** 0.5 * F32
    else:
        each = u * np.abs(want) + (u if low else 0.0) * absolute + chain * F32 * absolute
        norm = u + chain ** 0.5 * F32
    off = np.abs(got - want)
    bad = off > each + extra + 1e-30
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(off - each)}"
    if want.size >= 512 and np.any(want):
        rel = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert rel <= norm, f"{what}: 2-norm {rel:.3g} over {norm:.3g}"


def _abs(*ts):
    return [None if t is None else np.abs(_f64(t)) for t in ts]


BF, FL = torch.bfloat16, torch.float32
SHAPES = [  # B, H, N, D, M
    (1, 1, 1, 64, 64), (2, 3, 2, 64, 64), (1, 2, 15, 64, 64), (1, 1, 63, 64, 64), (2, 1, 64, 64, 64),
    (1, 3, 65, 64, 64), (1, 2, 128, 64, 64), (2, 2, 129, 64, 64), (1, 2, 1301, 64, 64),
    (3, 7, 200, 64, 64), (1, 2, 77, 128, 128), (1, 1, 700, 128, 128), (2, 2, 130, 40, 72),
    (1, 2, 90, 8, 128), (2, 1, 333, 128, 16), (1, 1, 257, 96, 64), (1, 2, 100, 64, 96),
    (40, 8, 70, 64, 64), (1, 1, 2500, 64, 64), (2, 20, 1100, 64, 64), (1, 3, 1000, 96, 128),
]
ids = lambda s: "b%dh%dn%dd%dm%d" % s  # noqa: E731


@pytest.mark.parametrize("states", [False, True], ids=["zero", "states"])
@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_forward_and_final_state(la, shape, dtype, states):
    B, H, N, D, M = shape
    q, k, v, g, _, S0, _ = _inputs(sum(shape), *shape, dtype)
    S0 = S0 if states else None
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    assert torch.equal(out, la.la_forward_gated(q, k, v, g, S0=S0)) or dtype == BF
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g)), None if S0 is None else _f64(S0))
    aq, ak, av, aS = _abs(q, k, v, S0)
    ao, aS = oracle.gated_forward(aq, ak, av, _f64(g), aS)
    chain = N + D + M + 64
    _close(out, want, ao, dtype, chain, "out")
    _close(la.la_forward_gated(q, k, v, g, S0=S0), want, ao, dtype, chain, "out without state")
    _close(S, wS, aS, dtype, chain, "S", state=True)


@pytest.mark.parametrize("gate", ["none", "slow", "strong", "resets"])
@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 3, 300, 64, 64), (1, 2, 150, 32, 48)], ids=ids)
def test_gates_from_none_to_emptying_the_state(la, shape, dtype, gate):
    B, H, N, D, M = shape
    q, k, v, g, do, S0, dS = _inputs(5, *shape, dtype, gate)
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g, S0)))
    ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g), np.abs(_f64(S0)))
    chain = N + D + M + 64
    _close(out, want, ao, dtype, chain, "out")
    _close(S, wS, aS, dtype, chain, "S", state=True)
    _backward_close(la, q, k, v, g, do, S0, dS, dtype)


def _backward_close(la, q, k, v, g, do, S0, dS, dtype):
    B, H, N, D = q.shape
    M = v.shape[-1]
    got = la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)
    assert len(got) == (4 if S0 is None else 5)
    n64 = lambda t: None if t is None else _f64(t)  # noqa: E731
    want = oracle.gated_backward(*map(n64, (q, k, v, g, do, S0, dS)))
    aq, ak, av, ado, aS0, adS = _abs(q, k, v, do, S0, dS)
    bound = oracle.gated_backward(aq, ak, av, _f64(g), ado, aS0, adS)
    chain = N + D + M + 64
    dots = np.sum(aq * bound[0] + ak * bound[1], axis=(-1, -2)) + np.sum(np.abs(bound[4]), axis=(-1, -2))
    for name, o, w, a in zip(("dq", "dk", "dv", "dg", "dS0"), got, want, bound):
        extra = chain * F32 * dots[..., None] if name == "dg" else 0.0
        _close(o, w, a, dtype, chain, name, extra=extra, state=name == "dS0")


@pytest.mark.parametrize("states", [False, True], ids=["zero", "states"])
@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", SHAPES, ids=ids)
def test_backward(la, shape, dtype, states):
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 1, *shape, dtype)
    _backward_close(la, q, k, v, g, do, S0 if states else None, dS if states else None, dtype)


@pytest.mark.parametrize("gate", ["mixed", "slow"])
@pytest.mark.parametrize("shape", [(1, 4, 5, 64, 64), (1, 2, 16, 128, 40), (1, 3, 17, 64, 64),
                                   (2, 8, 64, 64, 64), (19, 8, 40, 64, 64), (1, 2, 200, 128, 96),
                                   (1, 1, 700, 40, 72), (1, 2, 90, 8, 128), (1, 4, 1025, 64, 64)],
                         ids=ids)
def test_calls_of_few_chunks_show_only_their_outputs_rounding(la, shape, gate):
    """bf16, up to 152 chunks: no operand is rounded to one bf16 term. A term keeps 16 bits in
    each of two places (its chunk's operand or state, the state's own update), 2^-16 each."""
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 2, *shape, BF, gate)
    B, H, N, D, M = shape
    chain, u = N + D + M + 64, HALF[BF]
    n64 = [_f64(t) for t in (q, k, v, g, do, S0, dS)]
    size = [np.abs(x) for x in n64]
    size[3] = n64[3]
    bound = oracle.gated_backward(*size)
    dots = np.sum(size[0] * bound[0] + size[1] * bound[1], axis=(-1, -2)) + \
        np.sum(bound[4], axis=(-1, -2))
    names = ("out", "dq", "dk", "dv", "dg")
    outs = (la.la_forward_gated(q, k, v, g, S0=S0), *la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)[:4])
    wants = (oracle.gated_forward(*n64[:4], n64[5])[0], *oracle.gated_backward(*n64)[:4])
    sizes = (oracle.gated_forward(*size[:4], size[5])[0], *bound[:4])
    for name, got, want, a in zip(names, outs, wants, sizes):
        each = u * np.abs(want) + (2.0 ** -15 + chain * F32) * a
        if name == "dg":
            each = each + chain * F32 * dots[..., None]
        assert np.all(np.abs(_f64(got) - want) <= each), name


@pytest.mark.parametrize("dims", [(8, 8), (32, 24), (16, 48), (56, 64), (80, 72), (96, 88), (104, 8)],
                         ids=str)
def test_float32_heads_of_every_width(la, dims):
    for B, H, N in ((1, 2, 33), (2, 1, 600), (40, 16, 40)):
        D, M = dims
        q, k, v, g, do, S0, dS = _inputs(D + N, B, H, N, D, M, FL)
        out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
        want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g, S0)))
        ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g), np.abs(_f64(S0)))
        _close(out, want, ao, FL, N + D + M + 64, "out")
        _close(S, wS, aS, FL, N + D + M + 64, "S", state=True)
        _backward_close(la, q, k, v, g, do, S0, dS, FL)


@pytest.mark.parametrize("states", [False, True], ids=["zero", "states"])
@pytest.mark.parametrize("shape", [(2, 8, 700, 128, 128), (4, 10, 333, 96, 64), (3, 8, 450, 40, 128),
                                   (40, 4, 65, 128, 72), (1, 2, 5003, 128, 128), (1, 3, 4100, 64, 64)], ids=ids)
def test_calls_that_fill_the_multiprocessors(la, shape, states):
    """bf16, forward and backward: more than 152 blocks of 64 tokens by 64 columns, the last of a
    sequence a part of one, as a training step has them."""
    B, H, N, D, M = shape
    assert B * H * ((N + 63) // 64) * ((max(D, M) + 63) // 64) > 152 or N > 4000
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 3, *shape, BF)
    S0, dS = (S0, dS) if states else (None, None)
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g)), None if S0 is None else _f64(S0))
    ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g), None if S0 is None else np.abs(_f64(S0)))
    chain = N + D + M + 64
    _close(out, want, ao, BF, chain, "out")
    _close(la.la_forward_gated(q, k, v, g, S0=S0), want, ao, BF, chain, "out without state")
    _close(S, wS, aS, BF, chain, "S", state=True)
    _backward_close(la, q, k, v, g, do, S0, dS, BF)


def _half_step(x):
    """Half a step of bf16 at |x|."""
    return np.exp2(np.floor(np.log2(np.maximum(np.abs(x), 1e-37))) - 8)


@pytest.mark.parametrize("gate", ["slow", "many resets", "some resets"])
@pytest.mark.parametrize("shape", [(1, 4, 63, 64, 64), (1, 3, 700, 64, 64), (1, 2, 200, 128, 96)], ids=ids)
def test_resets_cost_the_tokens_behind_them_no_digits(la, shape, gate):
    """bf16, up to 152 chunks. A term of an output is rounded in no more than two operands of two
    bf16 terms each, 2^-17 of it, and in weights whose gates are summed to float32's digits, however
    often the state is emptied among the same 64 tokens: 2^-15 of the absolute terms in all; then
    the output by half a step of its own."""
    B, H, N, D, M = shape
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 7, *shape, BF, "slow")
    at = torch.arange(N, device=DEV) % 64
    if gate == "many resets":  # 40 in every 64, then tokens that forget very little
        g[...] = torch.where(at < 40, -torch.inf, -1e-4)
        q, k, v, do = (x.abs() for x in (q, k, v, do))  # (so that a weight off everywhere shows)
    elif gate == "some resets":  # between tokens that forget little
        g[..., at % 8 == 2] = torch.finfo(BF).min
        g[..., at % 8 == 3] = -40.0
    chain = N + D + M + 64
    n64 = [_f64(t) for t in (q, k, v, g, do, S0, dS)]
    size = [np.abs(x) for x in n64]
    size[3] = n64[3]
    bound = oracle.gated_backward(*size)
    dots = np.sum(size[0] * bound[0] + size[1] * bound[1], axis=(-1, -2)) + \
        np.sum(bound[4], axis=(-1, -2))
    names = ("out", "dq", "dk", "dv", "dg")
    outs = (la.la_forward_gated(q, k, v, g, S0=S0), *la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)[:4])
    wants = (oracle.gated_forward(*n64[:4], n64[5])[0], *oracle.gated_backward(*n64)[:4])
    sizes = (oracle.gated_forward(*size[:4], size[5])[0], *bound[:4])
    for name, got, want, a in zip(names, outs, wants, sizes):
        off = (2.0 ** -15 + chain * F32) * a
        if name == "dg":
            off = off + chain * F32 * dots[..., None]
        each = np.abs(_f64(got) - want) - _half_step(np.abs(want) + off) - off
        assert np.all(each <= 0), (name, (each > 0).mean(), np.max(each / (a + 1e-30)))


@pytest.mark.parametrize("gate", ["mixed", "slow"])
@pytest.mark.parametrize("shape", [(2, 8, 1025, 64, 64), (20, 8, 130, 64, 64), (160, 8, 20, 64, 64),
                                   (2, 8, 700, 128, 128), (4, 10, 333, 96, 64)], ids=ids)
def test_calls_that_fill_the_multiprocessors_show_only_their_outputs_rounding(la, shape, gate):
    """bf16: a sequence's outputs are as exact in a large batch as alone. A term keeps 16 bits in each
    of two places, 2^-16 each (its chunk's operand or state, the state's own update); then the output
    is rounded by half a step."""
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 2, *shape, BF, gate)
    B, H, N, D, M = shape
    chain = N + D + M + 64
    n64 = [_f64(t) for t in (q, k, v, g, do, S0, dS)]
    size = [np.abs(x) for x in n64]
    size[3] = n64[3]
    bound = oracle.gated_backward(*size)
    dots = np.sum(size[0] * bound[0] + size[1] * bound[1], axis=(-1, -2)) + \
        np.sum(bound[4], axis=(-1, -2))
    names = ("out", "out with S", "dq", "dk", "dv", "dg")
    outs = (la.la_forward_gated(q, k, v, g, S0=S0), la.la_prefill_gated(q, k, v, g, S0=S0)[0],
            *la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)[:4])
    want, a = oracle.gated_forward(*n64[:4], n64[5])[0], oracle.gated_forward(*size[:4], size[5])[0]
    wants, sizes = (want, want, *oracle.gated_backward(*n64)[:4]), (a, a, *bound[:4])
    for name, got, want, a in zip(names, outs, wants, sizes):
        off = (2.0 ** -15 + chain * F32) * a
        if name == "dg":
            off = off + chain * F32 * dots[..., None]
        each = np.abs(_f64(got) - want) - _half_step(np.abs(want) + off) - off
        assert np.all(each <= 0), (name, (each > 0).mean(), np.max(each / (a + 1e-30)))


def test_backward_with_only_one_of_the_states(la):
    q, k, v, g, do, S0, dS = _inputs(3, 1, 2, 100, 64, 64, BF)
    _backward_close(la, q, k, v, g, do, S0, None, BF)
    _backward_close(la, q, k, v, g, do, None, dS, BF)


def test_backward_against_differences_of_the_forward(la):
    """float32, along random directions, in chunks of a loss whose float32 evaluation is good to
    ~2^-20: a step of 2^-5 leaves 2^-15 relative to the loss's scale. What the central difference
    itself is off by at that step (its third-order term: exp of a sum of up to 70 moved gates) is
    taken from the oracle's difference and derivative at the same step and direction."""
    q, k, v, g, do, S0, dS = _inputs(11, 1, 2, 70, 32, 32, FL)
    grads = la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)

    def loss(*a):
        out, S = la.la_prefill_gated(*a[:4], S0=a[4])
        return float((out.double() * do.double()).sum() + (S.double() * dS.double()).sum())
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    xs = [q, k, v, g, S0]
    scale = abs(loss(*xs)) + 1.0
    for i, x in enumerate(xs):
        d = torch.randn(x.shape, generator=gen, device=DEV) * x.abs().mean()
        h = 2.0 ** -5
        up, down = [y + h * d if j == i else y for j, y in enumerate(xs)], [y - h * d if j == i else y for j, y in enumerate(xs)]
        diff = (loss(*up) - loss(*down)) / (2 * h)
        exact = [oracle.gated_forward(*map(_f64, y)) for y in (up, down)]
        exact = [np.sum(o * _f64(do)) + np.sum(S * _f64(dS)) for o, S in exact]
        exact_grad = oracle.gated_backward(*map(_f64, (q, k, v, g, do, S0, dS)))[i]
        diff -= (exact[0] - exact[1]) / (2 * h) - np.sum(exact_grad * _f64(d))
        want = float((grads[i].double() * d.double()).sum())
        size = float((grads[i].double().abs() * d.double().abs()).sum())
        assert abs(diff - want) <= 2.0 ** -10 * size + 2.0 ** -15 * scale, (i, diff, want)


def test_the_same_slow_gate_at_every_token(la):
    """float32. A state is rounded twice a token (the decay, the outer product), each time by at
    most half a step, 2-norm 2^-24 / sqrt(3), of either sign: sqrt(2 N) of those over N tokens
    that it hardly forgets, and sqrt(D + M) more in an output. A rounded exp(g) would be off the
    same way at every token: up to N 2^-25."""
    B, H, N, D, M = 13, 16, 1200, 32, 32
    q, k, v, _, do, S0, dS = _inputs(8, B, H, N, D, M, FL)
    g = torch.full((B, H, N), -3.1e-4, device=DEV)
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    grads = la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g, S0)))
    wants = oracle.gated_backward(*map(_f64, (q, k, v, g, do, S0, dS)))
    step = F32 / 3 ** 0.5
    for name, o, w, count in (("out", out, want, 2 * N + D + M), ("S", S, wS, 2 * N),
                              ("dq", grads[0], wants[0], 2 * N + D + M),
                              ("dk", grads[1], wants[1], 2 * N + D + M),
                              ("dv", grads[2], wants[2], 2 * N + D + M),
                              ("dS0", grads[4], wants[4], 2 * N)):
        rel = np.linalg.norm(_f64(o) - w) / np.linalg.norm(w)
        assert rel <= count ** 0.5 * step, (name, rel)


@pytest.mark.parametrize("gate", [-1e-6, 0.02], ids=["hardly forgotten", "growing"])
def test_long_sequences_in_few_segments(la, gate):
    """bf16. Sums that truncate would leave every output of a state that hardly decays too small: the
    outputs' mean relative error is that of n roundings of either sign, each below 2^-8 / sqrt(3),
    and of operands that are rounded at 2^-17. Growing: the gates of 4096 tokens sum to 82, those of
    the call to far more than a float32 exponential takes."""
    if gate < 0:  # as many sequences as fill the GPU, each one segment
        few, B, N = 4, 456, 1 << 16
    else:
        few, B, N = 1, 16, 1 << 18
    gen = torch.Generator(device=DEV).manual_seed(7)
    q, k, v = (torch.rand((few, 1, N, 64), generator=gen, device=DEV).to(BF) for _ in range(3))
    g = torch.full((few, 1, N), gate, device=DEV).to(BF)
    if gate > 0:
        # the state is emptied in the end, so that the results are finite
        g[:, :, -5] = -torch.inf
        k[:, :, :-5], q[:, :, :-5] = 0, 0
    want = oracle.gated_forward(*(_f64(x[:, :, -8192:]) for x in (q, k, v, g)),
                                None if gate > 0 else _early_state(k, v, g, N - 8192))[0]
    rows = [x.expand(B // few, few, *x.shape[1:]).reshape(B, *x.shape[1:]).contiguous() for x in (q, k, v, g)]
    out = la.la_forward_gated(*rows)
    assert torch.isfinite(out).all()
    tail = _f64(out[:few, :, -64:]) if gate < 0 else _f64(out[:few, :, -5:])
    want = want[:, :, -tail.shape[2]:]
    off = (tail - want) / want
    assert np.all(np.abs(off) <= 2.0 ** -8 + 2.0 ** -12)
    assert abs(off.mean()) <= 2.0 ** -16 + 5 * 2.0 ** -8 / (3 * off.size) ** 0.5
    for b in range(few, B, few):
        assert torch.equal(out[b:b + few], out[:few])


def _early_state(k, v, g, n):
    """The state after the first n tokens in float64: sums of k_t v_t^T, each left to decay."""
    k, v, g = (x[:, :, :n].double() for x in (k, v, g))
    left = torch.exp(g.flip(2).cumsum(2).flip(2) - g)
    return torch.einsum("bhnd,bhnm->bhdm", k * left[..., None], v).cpu().numpy()


# ------------------------------------------------------------------------ serving

@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (24, 40)], ids=str)
@pytest.mark.parametrize("N", [1, 70, 400])
def test_extend_ragged_batch_from_a_pool(la, N, dims, dtype):
    D, M = dims
    B, H, P = 6, 3, 9
    q, k, v, g, *_ = _inputs(N, B, H, N, D, M, dtype)
    lens = torch.tensor([0, 1, N, N // 2, N + 5, -3], dtype=torch.int32, device=DEV)
    n = lens.clamp(0, N).tolist()
    for b in range(B):  # padding rows may hold anything
        for t in (q, k, v, g):
            t[b, :, n[b]:] = torch.nan
    slots = torch.tensor([4, 0, 8, 2, 5, 7], dtype=torch.int32, device=DEV)
    pool = torch.randn(P, H, D, M, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)) * 0.3
    before, out = pool.clone(), torch.full((B, H, N, M), 7.0, dtype=dtype, device=DEV)
    la.la_extend_gated(q, k, v, g, pool, slots=slots, lens=lens, out=out)
    chain = N + D + M + 64
    for b, s in enumerate(slots.tolist()):
        a = [x[b:b + 1, :, :n[b]] for x in (q, k, v, g)]
        want, wS = oracle.gated_forward(*map(_f64, a), _f64(before[s:s + 1]))
        ao, aS = oracle.gated_forward(*_abs(*a[:3]), _f64(a[3]), np.abs(_f64(before[s:s + 1])))
        _close(out[b:b + 1, :, :n[b]], want, ao, dtype, chain, f"out of stream {b}")
        _close(pool[s:s + 1], wS, aS, dtype, chain, f"state of stream {b}", state=True)
        assert torch.all(out[b, :, n[b]:] == 7.0), "rows behind a stream's end"
    for s in (1, 3, 6):
        assert torch.equal(pool[s], before[s]), "an entry of no stream"


def test_extend_reports_a_slot_outside_the_pool(la):
    B, H, N = 3, 2, 200
    q, k, v, g, *_ = _inputs(1, B, H, N, 64, 64, BF)
    pool = torch.ones(4, H, 64, 64, device=DEV)
    before = pool.clone()
    ws = torch.empty(la.la_gated_workspace_bytes(B, H, N, 64, 64), dtype=torch.uint8, device=DEV)
    slots = torch.tensor([2, 4, -1], dtype=torch.int32, device=DEV)
    out = la.la_extend_gated(q, k, v, g, pool, slots=slots, workspace=ws)
    assert la.la_workspace_status(ws) == la.LA_ERR_INVALID_ARG
    zero = la.la_forward_gated(q[1:], k[1:], v[1:], g[1:])
    aq = oracle.gated_forward(*_abs(q[1:], k[1:], v[1:]), _f64(g[1:]))[0]
    assert np.all(np.abs(_f64(out[1:]) - _f64(zero)) <= 2 * HALF[BF] * aq)
    assert torch.equal(pool[[0, 1, 3]], before[[0, 1, 3]])
    la.la_extend_gated(q, k, v, g, pool, slots=torch.tensor([2, 3, 0], dtype=torch.int32, device=DEV), workspace=ws)
    assert la.la_workspace_status(ws) == la.LA_OK


@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (8, 8), (24, 104), (128, 8)], ids=str)
def test_decode_step(la, dims, dtype):
    D, M = dims
    n, H, P = 5, 3, 8
    q, k, v, g, *_ = _inputs(9, n, H, 1, D, M, dtype, "resets")
    pool = torch.randn(P, H, D, M, device=DEV, generator=torch.Generator(device=DEV).manual_seed(3))
    before = pool.clone()
    slots = torch.tensor([7, 0, 3, 6, 99], dtype=torch.int32, device=DEV)  # the last: no entry
    out = la.la_decode_step_gated(*(x[:, :, 0].contiguous() for x in (q, k, v, g)), pool, slots=slots)
    start = torch.cat((before[slots[:4].long()], torch.zeros(1, H, D, M, device=DEV)))
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g, start)))
    ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g), np.abs(_f64(start)))
    u = HALF[dtype]
    assert np.all(np.abs(_f64(out) - want[:, :, 0]) <= u * np.abs(want[:, :, 0]) + (D + 8) * F32 * ao[:, :, 0])
    assert np.all(np.abs(_f64(pool[slots[:4].long()]) - wS[:4]) <= 4 * F32 * aS[:4])
    assert torch.equal(pool[[1, 2, 4, 5]], before[[1, 2, 4, 5]])


def test_prompt_then_tokens_equals_the_whole_sequence(la):
    B, H, N, D, M = 2, 3, 150, 64, 64
    q, k, v, g, *_ = _inputs(21, B, H, N, D, M, BF)
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g)))
    ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g))
    cut = lambda i, j: [x[:, :, i:j].contiguous() for x in (q, k, v, g)]  # noqa: E731
    out, S = la.la_prefill_gated(*cut(0, 101))
    outs = [out, la.la_extend_gated(*cut(101, 141), S)]
    for t in range(141, N):
        outs.append(la.la_decode_step_gated(*(x[:, :, t].contiguous() for x in (q, k, v, g)), S)[:, :, None])
    _close(torch.cat(outs, 2), want, ao, BF, N + D + M + 64, "out")
    _close(S, wS, aS, BF, N + D + M + 64, "S", state=True)


def test_final_state_may_replace_the_initial_one(la):
    for N in (40, 900):
        q, k, v, g, _, S0, _ = _inputs(N, 2, 2, N, 64, 64, BF)
        out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
        both = S0.clone()
        out2, S2 = la.la_prefill_gated(q, k, v, g, S0=both, S=both)
        assert S2 is both and torch.equal(S2, S) and torch.equal(out2, out)


@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 2, 7, 64, 64), (2, 40, 20, 32, 48), (2, 3, 700, 64, 64), (1, 2, 300, 128, 96)],
                         ids=ids)
def test_initial_states_gradient_may_replace_the_final_ones(la, shape, dtype):
    q, k, v, g, do, S0, dS = _inputs(sum(shape) + 5, *shape, dtype)
    want = la.la_backward_gated(q, k, v, g, do, S0, dS)
    both = dS.clone()
    got = la.la_backward_gated(q, k, v, g, do, S0, both, dS0=both)
    assert got[4] is both
    B, H, N, D, M = shape
    n64 = [_f64(t) for t in (q, k, v, g, do, S0, dS)]
    size = [np.abs(x) for x in n64]
    size[3] = n64[3]
    bound = oracle.gated_backward(*size)
    for name, a, b, x in zip(("dq", "dk", "dv", "dg", "dS0"), got, want, bound):
        # (the two may sum in other orders: each is within its own bound)
        u = 2 * (HALF[dtype] if name != "dS0" else 2.0 ** -17 if dtype == BF else F32)
        dots = np.sum(size[0] * bound[0] + size[1] * bound[1], axis=(-1, -2)) + np.sum(bound[4], axis=(-1, -2))
        extra = 2 * (N + D + M + 64) * F32 * dots[..., None] if name == "dg" else 0.0
        assert np.all(np.abs(_f64(a) - _f64(b)) <= 2 * (u + (N + D + M + 64) * F32) * x + extra), name


def test_no_tokens(la):
    q, k, v, g, do, S0, dS = _inputs(1, 2, 2, 0, 64, 64, BF)
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    assert out.shape == (2, 2, 0, 64) and torch.equal(S, S0)
    _, S = la.la_prefill_gated(q, k, v, g)
    assert not S.any()
    *_, dS0 = la.la_backward_gated(q, k, v, g, do, S0=S0, dS=dS)
    assert torch.equal(dS0, dS)
    *_, dS0 = la.la_backward_gated(q, k, v, g, do, S0=S0)
    assert not dS0.any()


def test_pool_entries_past_32_bits(la):
    """The last entry of a pool of more than 2^31 elements."""
    H, D = 8, 64
    P = 2 ** 31 // (H * D * D) + 3
    pool = torch.empty(P, H, D, D, device=DEV)
    pool[-1], pool[0] = 0.5, 2.0
    q, k, v, g, *_ = _inputs(4, 1, H, 70, D, D, BF)
    start = pool[-1:].clone()
    slots = torch.tensor([P - 1], dtype=torch.int32, device=DEV)
    cut = lambda i, j: [x[:, :, i:j].contiguous() for x in (q, k, v, g)]  # noqa: E731
    out = la.la_extend_gated(*cut(0, 69), pool, slots=slots)
    one = la.la_decode_step_gated(*(x[:, :, 69].contiguous() for x in (q, k, v, g)), pool, slots=slots)
    want, wS = oracle.gated_forward(*map(_f64, (q, k, v, g, start)))
    ao, aS = oracle.gated_forward(*_abs(q, k, v), _f64(g), _f64(start))
    _close(torch.cat((out, one[:, :, None]), 2), want, ao, BF, 70 + 2 * D + 64, "out")
    _close(pool[-1:], wS, aS, BF, 70 + 2 * D + 64, "S", state=True)
    assert torch.all(pool[0] == 2.0)


# -------------------------------------------------------- streams, graphs, repeats

def test_two_calls_at_once_on_two_streams(la):
    sets = [_inputs(s, 2, 4, 700, 64, 64, BF) for s in (41, 42)]
    run = lambda q, k, v, g, do, S0, dS: (*la.la_prefill_gated(q, k, v, g, S0=S0),  # noqa: E731
                                          *la.la_backward_gated(q, k, v, g, do, S0, dS))
    want = [run(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(4):
        got = []
        for s, stream in zip(sets, streams):
            with torch.cuda.stream(stream):
                got.append(run(*s))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_outputs_and_workspaces_of_the_callers(la):
    q, k, v, g, do, S0, dS = _inputs(6, 2, 3, 333, 64, 64, BF)
    out, S = la.la_prefill_gated(q, k, v, g, S0=S0)
    grads = la.la_backward_gated(q, k, v, g, do, S0, dS)
    ws = torch.full((la.la_gated_workspace_bytes(2, 3, 333, 64, 64),), 255, dtype=torch.uint8, device=DEV)
    bws = torch.full((la.la_gated_backward_workspace_bytes(2, 3, 333, 64, 64),), 255, dtype=torch.uint8, device=DEV)
    o2, s2 = torch.full_like(out, torch.nan), torch.full_like(S, torch.nan)
    got = la.la_prefill_gated(q, k, v, g, S0=S0, out=o2, S=s2, workspace=ws)
    assert got[0] is o2 and got[1] is s2 and torch.equal(o2, out) and torch.equal(s2, S)
    into = [torch.full_like(x, torch.nan) for x in grads]
    got = la.la_backward_gated(q, k, v, g, do, S0, dS, *into, workspace=bws)
    assert all(a is b for a, b in zip(got, into)) and all(torch.equal(a, b) for a, b in zip(got, grads))
    z = torch.zeros(1, 1, 4000, 64, dtype=BF, device=DEV)
    with pytest.raises(ValueError):
        la.la_forward_gated(z, z, z, z[..., 0].contiguous(), workspace=ws[:100])


def test_repeats_bit_for_bit_and_on_another_stream(la):
    q, k, v, g, do, S0, dS = _inputs(8, 2, 4, 1000, 64, 64, BF)
    first = (*la.la_prefill_gated(q, k, v, g, S0=S0), *la.la_backward_gated(q, k, v, g, do, S0, dS))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = (*la.la_prefill_gated(q, k, v, g, S0=S0), *la.la_backward_gated(q, k, v, g, do, S0, dS))
    side.synchronize()
    for a, b in zip(first, again):
        assert torch.equal(a, b)


def test_captured_and_replayed_on_new_inputs(la):
    a, b = (_inputs(s, 1, 3, 500, 64, 64, BF) for s in (31, 32))
    held = [x.clone() for x in a]
    q, k, v, g, do, S0, dS = held

    def step():
        return (*la.la_prefill_gated(q, k, v, g, S0=S0), *la.la_backward_gated(q, k, v, g, do, S0, dS))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for src in (b, a):
        for h, x in zip(held, src):
            h.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        want = (*la.la_prefill_gated(*src[:4], S0=src[5]), *la.la_backward_gated(*src[:5], src[5], src[6]))
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", [BF, FL], ids=["bf16", "f32"])
def test_serving_calls_captured_and_replayed_at_once(la, dtype):
    """Two graphs, each of an extend and a decode step on its own pool, replayed on two streams with
    new tokens, slots and lengths: the same as the calls themselves."""
    B, H, N, D, P = 6, 4, 90, 64, 20
    runs = []
    for seed in (1, 2):
        q, k, v, g, *_ = _inputs(seed, B, H, N, D, D, dtype)
        q1, k1, v1, g1 = (x[:, :, 0].contiguous() for x in _inputs(seed + 10, B, H, 1, D, D, dtype)[:4])
        gen = torch.Generator(device=DEV).manual_seed(seed)
        pool = torch.randn((P, H, D, D), generator=gen, device=DEV)
        slots = torch.arange(B, dtype=torch.int32, device=DEV)
        lens = torch.full((B,), N, dtype=torch.int32, device=DEV)
        out = torch.zeros_like(v)

        def step(q=q, k=k, v=v, g=g, one=(q1, k1, v1, g1), pool=pool, slots=slots, lens=lens, out=out):
            la.la_extend_gated(q, k, v, g, pool, slots=slots, lens=lens, out=out)
            return out, la.la_decode_step_gated(*one, pool, slots=slots)
        start = pool.clone()
        step()
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step()
        # what the replay finds: other tokens, slots (one of no entry) and lengths
        q.copy_(_inputs(seed + 20, B, H, N, D, D, dtype)[0])
        slots.copy_(torch.tensor([7, 19, 3, -1, 0, 11], dtype=torch.int32))
        lens.copy_(torch.tensor([0, 1, 64, 65, N, 17], dtype=torch.int32))
        pool.copy_(start)
        out.fill_(3.0)
        want = [x.clone() for x in step()] + [pool.clone()]
        pool.copy_(start)
        out.fill_(3.0)
        runs.append((graph, stream, (*got, pool), want, step))  # (step holds the inputs)
    torch.cuda.synchronize()
    for graph, stream, *_ in runs:
        with torch.cuda.stream(stream):
            graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in runs:
        for a, b in zip(got, want):
            assert torch.equal(a, b)


# ------------------------------------------------------------ the layer as it is used

def test_layer_of_the_three_operators(la):
    """rotary -> gated recurrence -> gated norm written token-major, and the way back, against
    the oracle's chain fed with the GPU's own intermediates (so each stage keeps its bound)."""
    B, H, N, D = 2, 4, 300, 64
    gen = torch.Generator(device=DEV).manual_seed(77)
    proj = (torch.randn((4, B, N, H, D), generator=gen, device=DEV) * 0.5).to(BF)
    q, k, v, z = (p.transpose(1, 2) for p in proj)
    g = _gates(gen, (B, H, N), "mixed").to(BF)
    w = (1 + 0.1 * torch.randn((D,), generator=gen, device=DEV)).to(BF)
    freqs, mscale = la.la_rotary_freqs(32, device=DEV)
    rq, rk = la.la_rotary(q, k, freqs, mscale=mscale)
    vc = v.contiguous()
    out = la.la_forward_gated(rq, rk, vc, g)
    y = torch.empty(B, N, H, D, dtype=BF, device=DEV)
    la.la_norm_gate(out, z, w, out=y.transpose(1, 2))
    u, pos = HALF[BF], np.arange(N)
    wq = oracle.rotary(_f64(q), pos, _f64(freqs))
    assert np.all(np.abs(_f64(rq) - wq) <= u * np.abs(wq) + 1e-6)
    want, _ = oracle.gated_forward(*map(_f64, (rq, rk, vc, g)))
    ao, _ = oracle.gated_forward(*_abs(rq, rk, vc), _f64(g))
    _close(out, want, ao, BF, N + 2 * D + 64, "out")
    wy = oracle.norm_gate(_f64(out), _f64(z), _f64(w))
    assert np.all(np.abs(_f64(y.transpose(1, 2)) - wy) <= (u + 1e-5) * np.abs(wy) + 1e-30)
    dy = (torch.randn((B, N, H, D), generator=gen, device=DEV)).to(BF).transpose(1, 2)
    dout, dz, dw = la.la_norm_gate_backward(out, z, w, dy)
    dq, dk, dv, dg = la.la_backward_gated(rq, rk, vc, g, dout)
    iq, ik = la.la_rotary(dq, dk, freqs, mscale=mscale, inverse=True)
    wd = oracle.gated_backward(*map(_f64, (rq, rk, vc, g, dout)))
    ad = oracle.gated_backward(*_abs(rq, rk, vc), _f64(g), np.abs(_f64(dout)))
    for name, o, x, a in zip(("dq", "dk", "dv"), (dq, dk, dv), wd, ad):
        _close(o, x, a, BF, N + 2 * D + 64, name)
    wi = oracle.rotary(_f64(dq), pos, _f64(freqs), inverse=True)
    assert np.all(np.abs(_f64(iq) - wi) <= u * np.abs(wi) + 1e-6 * np.abs(_f64(dq)).max())
