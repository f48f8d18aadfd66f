"""The fp64 definitions of oracle/gated.py, each against something other than itself: the
masked quadratic form, the ungated limit, complex multiplication, and central finite
differences for every gradient."""

import numpy as np
import pytest

import oracle


def _draw(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def _case(seed=0, B=2, H=2, N=7, D=3, M=4):
    q, k, v, do = (_draw(seed + i, B, H, N, d) for i, d in enumerate((D, D, M, M)))
    g = -np.exp(_draw(seed + 9, B, H, N))
    S0, dS = _draw(seed + 5, B, H, D, M), _draw(seed + 6, B, H, D, M)
    return q, k, v, g, do, S0, dS


def test_forward_is_the_masked_quadratic_form():
    q, k, v, g, _, S0, _ = _case()
    out, S = oracle.gated_forward(q, k, v, g, S0)
    G = np.cumsum(g, -1)
    L = np.tril(np.exp(G[..., :, None] - G[..., None, :]))
    want = np.einsum("bhij,bhij,bhjm->bhim", np.einsum("bhid,bhjd->bhij", q, k), L, v)
    want += np.exp(G)[..., None] * np.einsum("bhid,bhdm->bhim", q, S0)
    np.testing.assert_allclose(out, want, rtol=1e-12, atol=1e-12)
    last = np.einsum("bhj,bhjd,bhjm->bhdm", L[:, :, -1], k, v) + np.exp(G[..., -1:, None]) * S0
    np.testing.assert_allclose(S, last, rtol=1e-12, atol=1e-12)


def test_forward_without_decay_sums_and_with_full_decay_forgets():
    q, k, v, g, *_ = _case(1)
    _, S = oracle.gated_forward(q, k, v, 0 * g)
    np.testing.assert_allclose(S, np.einsum("bhnd,bhnm->bhdm", k, v), rtol=1e-12)
    out, S = oracle.gated_forward(q, k, v, np.full_like(g, -np.inf), S0=_draw(3, 2, 2, 3, 4))
    np.testing.assert_allclose(out, np.einsum("bhnd,bhnd,bhnm->bhnm", q, k, v), rtol=1e-12, atol=1e-14)


def test_forward_stops_each_stream_at_its_length():
    q, k, v, g, _, S0, _ = _case(2)
    out, S = oracle.gated_forward(q, k, v, g, S0, lens=[3, 0])
    short, S3 = oracle.gated_forward(q[:1, :, :3], k[:1, :, :3], v[:1, :, :3], g[:1, :, :3], S0[:1])
    np.testing.assert_array_equal(out[0, :, :3], short[0])
    np.testing.assert_array_equal(S[0], S3[0])
    np.testing.assert_array_equal(S[1], S0[1])
    assert not out[0, :, 3:].any() and not out[1].any()


def _differences(f, x, h=1e-6):
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        d[i] = (f(up) - f(down)) / (2 * h)
    return d


def test_gated_backward_against_differences():
    args = _case(3, B=1, N=5)
    q, k, v, g, do, S0, dS = args
    grads = oracle.gated_backward(*args)

    def loss(**kw):
        a = {"q": q, "k": k, "v": v, "g": g, "S0": S0, **kw}
        out, S = oracle.gated_forward(**a)
        return np.sum(out * do) + np.sum(S * dS)
    for got, (name, x) in zip(grads, (("q", q), ("k", k), ("v", v), ("g", g), ("S0", S0))):
        # central differences of a smooth loss: O(h^2) = 1e-12 and rounding 1e-16 / h = 1e-10
        np.testing.assert_allclose(got, _differences(lambda y: loss(**{name: y}), x),
                                   rtol=1e-7, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_complex_multiplication(interleaved):
    x, f, pos = _draw(4, 2, 3, 5, 10), np.array([1.0, 0.3, 0.01]), np.arange(7, 12)
    y = oracle.rotary(x, pos, f, interleaved, mscale=1.5)
    pair = (lambda u: u[..., 0:6:2] + 1j * u[..., 1:6:2]) if interleaved else \
        (lambda u: u[..., :3] + 1j * u[..., 3:6])
    np.testing.assert_allclose(pair(y), 1.5 * pair(x) * np.exp(1j * pos[:, None] * f), atol=1e-13)
    np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
    back = oracle.rotary(y, pos, f, interleaved, mscale=1 / 1.5, inverse=True)
    np.testing.assert_allclose(back, x, atol=1e-13)
    # the inverse turn is the transpose: <rotary(x), y'> = <x, inverse(y')>
    u = _draw(6, *x.shape)
    np.testing.assert_allclose(np.sum(y * u),
                               np.sum(x * oracle.rotary(u, pos, f, interleaved, 1.5, inverse=True)))


@pytest.mark.parametrize("heads", [False, True])
def test_norm_gate_backward_against_differences(heads):
    x, z, dy = (_draw(7 + i, 2, 2, 3, 4) for i in range(3))
    w = _draw(11, 2, 4) if heads else _draw(11, 4)
    for got, (i, a) in zip(oracle.norm_gate_backward(x, z, w, dy), enumerate((x, z, w))):
        def loss(u):
            args = [x, z, w]
            args[i] = u
            return np.sum(dy * oracle.norm_gate(*args))
        np.testing.assert_allclose(got, _differences(loss, a), rtol=1e-6, atol=1e-7)
    n = oracle.norm_gate(x, np.full_like(z, 50.0), np.ones(4), eps=0.0) / 50.0
    np.testing.assert_allclose(np.mean(n * n, -1), 1.0)
