"""The float64 definitions of the layer norm, the gated projections and the checkpoints against
closed forms, central differences and brute force."""

import math

import numpy as np
import pytest

import oracle

RNG = np.random.default_rng(5)


def _slope(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_layer_norm_has_mean_zero_and_variance_one():
    x = RNG.normal(3.0, 2.0, (4, 50))
    y = oracle.layer_norm(x, np.ones(50), eps=0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-14) and np.allclose((y * y).mean(-1), 1, rtol=1e-14)
    w, b = RNG.normal(size=50), RNG.normal(size=50)
    assert np.allclose(oracle.layer_norm(7 * x + 2, w, b, eps=0.0), y * w + b, rtol=1e-13, atol=1e-13)


def test_layer_norm_gradients_by_differences():
    x, w, b, dy = (RNG.normal(size=s) for s in ((3, 5, 24), (24,), (24,), (3, 5, 24)))
    grads = oracle.layer_norm_backward(x, w, dy)
    f = lambda *a: (dy * oracle.layer_norm(*a)).sum()  # noqa: E731
    for k, g in enumerate(grads):
        args = [x, w, b]
        d = RNG.normal(size=args[k].shape)
        slope = _slope(lambda t: f(*args[:k], t, *args[k + 1:]), args[k], d)
        assert math.isclose(slope, (g * d).sum(), rel_tol=1e-7)


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_activations(kind):
    a = np.linspace(-9, 9, 401)
    f, df = oracle.activation(a, kind)
    exact = {"silu": lambda t: t / (1 + math.exp(-t)),
             "gelu": lambda t: t * (1 + math.erf(t / math.sqrt(2))) / 2,
             "gelu_tanh": lambda t: t / 2 * (1 + math.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t ** 3)))}[kind]
    assert np.allclose(f, [exact(t) for t in a], rtol=1e-9, atol=1e-15)
    slope = _slope(lambda t: oracle.activation(t, kind)[0], a, np.ones_like(a))
    assert np.allclose(df, slope, atol=1e-9)
    assert oracle.activation(np.array([-800.0, 800.0]), kind)[0].tolist() == [0.0, 800.0]


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_ffn_gradients_by_differences(kind):
    x, wg, wu, dh = (RNG.normal(size=s) for s in ((6, 8), (10, 8), (10, 8), (6, 10)))
    grads = oracle.ffn_gate_backward(x, wg, wu, dh, kind)
    for k, g in enumerate(grads):
        args = [x, wg, wu]
        d = RNG.normal(size=args[k].shape)
        slope = _slope(lambda t: (dh * oracle.ffn_gate(*args[:k], t, *args[k + 1:], kind)).sum(), args[k], d)
        assert math.isclose(slope, (g * d).sum(), rel_tol=1e-7)


def test_checkpoint_by_hand():
    x = np.zeros((6, 40))
    x[0, :3] = 127.49, 64.5, -63.5        # step 1; ties to the even number
    x[1, :3] = 127.5, 1.0, 3.0            # step 2
    x[2, :2], x[2, 32] = (1e-40, 0), 1.0  # below the smallest step; another block
    x[3, 1], x[3, 2], x[3, 33] = np.inf, 5.0, 5.0
    x[4, 0] = np.nan
    x[5, :2] = 3.4e38, -1e38
    codes, exps, values = oracle.checkpoint(x)
    assert codes[0, :3].tolist() == [127, 64, -64] and exps[0].tolist() == [127, 1]
    assert codes[1, :3].tolist() == [64, 0, 2] and exps[1, 0] == 128
    assert codes[2, :2].tolist() == [0, 0] and exps[2].tolist() == [1, 121] and values[2, 32] == 1.0
    assert exps[3].tolist() == [255, 123] and np.isnan(values[3, :32]).all() and values[3, 33] == 5.0
    assert exps[4, 0] == 255 and not codes[4].any()
    assert codes[5, 0] == 64 and exps[5, 0] == 249 and np.isfinite(values[5]).all()


def test_checkpoint_is_within_half_a_step():
    x = RNG.normal(size=(50, 77)) * np.exp(5 * RNG.normal(size=(50, 1)))
    codes, exps, values = oracle.checkpoint(x)
    step = np.repeat(2.0 ** (exps.astype(float) - 127), 32, -1)[:, :77]
    assert np.all(np.abs(values - x) <= step / 2) and np.abs(codes.astype(int)).max() <= 127
    top = np.maximum.reduceat(np.abs(codes.astype(int)), [0, 32, 64], -1)
    assert top.min() >= 64  # half the step would not have done
    again = oracle.checkpoint(values)
    assert np.array_equal(again[2], values)


def test_checkpoint_of_the_largest_values():
    """2^128 is no float32: what codes stand for ends at the largest bfloat16, within half a step."""
    most = 2.0 ** 128 - 2.0 ** 120
    x = np.zeros((4, 32))
    x[0, 0], x[1, 0], x[2, 0], x[3, 0] = most, -63.75 * 2.0 ** 122, 2.0 ** 128 - 2.0 ** 104, 127.25 * 2.0 ** 121
    codes, exps, values = oracle.checkpoint(x)
    assert codes[:, 0].tolist() == [64, -64, 64, 127] and exps[:, 0].tolist() == [249, 249, 249, 248]
    assert values[:, 0].tolist() == [most, -most, most, 127 * 2.0 ** 121]
    assert np.all(np.abs(values - x) <= 2.0 ** (exps.astype(float) - 128))
