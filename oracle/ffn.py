"""float64 definitions of the layer norm, the gated projections and the 8-bit checkpoints."""

import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def layer_norm(x, w, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    d = x - x.mean(-1, keepdims=True)
    y = d / np.sqrt((d * d).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
    return y if b is None else y + np.asarray(b, np.float64)


def layer_norm_backward(x, w, dy, eps=1e-5):
    """(dx, dw, db) of sum(dy * layer_norm(x, w, b, eps)); dw and db summed over all rows."""
    x, w, dy = (np.asarray(t, np.float64) for t in (x, w, dy))
    d = x - x.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((d * d).mean(-1, keepdims=True) + eps)
    n, g = d * r, dy * w
    dx = r * (g - g.mean(-1, keepdims=True) - n * (g * n).mean(-1, keepdims=True))
    rows = tuple(range(x.ndim - 1))
    return dx, (dy * n).sum(rows), dy.sum(rows)


def activation(a, kind):
    """(act(a), act'(a))."""
    a = np.asarray(a, np.float64)
    if kind == "gelu":
        p = 0.5 * _erfc(-a / math.sqrt(2.0))
        return a * p, p + a * np.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)
    z, dz = a, np.ones_like(a)
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        z, dz = c * (a + 0.044715 * a ** 3), c * (1.0 + 3.0 * 0.044715 * a * a)
    elif kind != "silu":
        raise ValueError(kind)
    e = np.exp(-np.abs(z))
    s = np.where(z < 0, e, 1.0) / (1.0 + e)
    return a * s, s + a * s * (1.0 - s) * dz


def ffn_gate(x, wg, wu, kind="silu"):
    x, wg, wu = (np.asarray(t, np.float64) for t in (x, wg, wu))
    return activation(x @ wg.T, kind)[0] * (x @ wu.T)


def ffn_gate_backward(x, wg, wu, dh, kind="silu", kept=None):
    """(dx, dwg, dwu) of sum(dh * ffn_gate(x, wg, wu, kind)), x [T, C]; kept: the pair of products
    to be taken instead of x wg^T and x wu^T."""
    x, wg, wu, dh = (np.asarray(t, np.float64) for t in (x, wg, wu, dh))
    a, u = (x @ wg.T, x @ wu.T) if kept is None else kept
    f, df = activation(a, kind)
    da, du = dh * u * df, dh * f
    return da @ wg + du @ wu, da.T @ x, du.T @ x


def checkpoint(x):
    """(codes, exps, values) of x [..., C] in blocks of 32: the step 2^(exp - 127) is the smallest,
    from exp = 1 on, with every |value| / step below 127.5; exp = 255 and NaN for a block that is
    not finite. Values are bounded by the largest bf16, 2^128 - 2^120."""
    x = np.asarray(x, np.float64)
    n = x.shape[-1]
    v = np.concatenate([x, np.zeros((*x.shape[:-1], -n % 32))], -1).reshape(*x.shape[:-1], -1, 32)
    top = np.abs(v).max(-1)
    bad = ~np.isfinite(top)
    step = np.full(top.shape, 2.0 ** -126)
    for _ in range(260):
        step = np.where(~bad & (top / step >= 127.5), 2.0 * step, step)
    with np.errstate(invalid="ignore"):
        codes = np.where(bad[..., None], 0.0, np.rint(v / step[..., None]))
    exps = np.where(bad, 255, np.log2(step) + 127).astype(np.uint8)
    most = 2.0 ** 128 - 2.0 ** 120
    values = np.clip(codes * np.where(bad, np.nan, step)[..., None], -most, most)
    cut = lambda t: t.reshape(*x.shape[:-1], -1)[..., :n]  # noqa: E731
    return cut(codes).astype(np.int8), exps, cut(values)
