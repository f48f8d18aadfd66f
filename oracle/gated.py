"""fp64 definitions of the gated recurrence, rotary positions and the gated head norm.

Each is written token by token or element by element from its formula, over numpy
arrays; the gradients are derived by hand and checked against central finite
differences in ``tests/test_gated_oracle.py``.
"""

import numpy as np


def _f64(x):
    return np.asarray(x, dtype=np.float64)


def gated_forward(q, k, v, g, S0=None, lens=None):
    """(out, S): S_t = exp(g_t) S_{t-1} + k_t v_t^T, out_t = S_t^T q_t, for q, k [B,H,N,D],
    v [B,H,N,M], g [B,H,N]. Stream b stops after lens[b] tokens; its later rows of out are 0."""
    q, k, v, g = map(_f64, (q, k, v, g))
    B, H, N, D = q.shape
    S = np.zeros((B, H, D, v.shape[-1])) if S0 is None else _f64(S0).copy()
    out = np.zeros(v.shape)
    for t in range(N):
        on = np.ones(B, bool) if lens is None else t < np.asarray(lens)
        a = np.exp(g[on, :, t])[..., None, None]
        S[on] = a * S[on] + k[on, :, t, :, None] * v[on, :, t, None, :]
        out[on, :, t] = np.einsum("bhd,bhdm->bhm", q[on, :, t], S[on])
    return out, S


def gated_backward(q, k, v, g, dout, S0=None, dS=None):
    """(dq, dk, dv, dg, dS0) of sum(dout * out) + sum(dS * S): with E_t the gradient with respect
    to S_t, E_t = q_t dout_t^T + exp(g_{t+1}) E_{t+1} (E_{N-1} has dS in place of the latter),
    dq_t = S_t dout_t, dk_t = E_t v_t, dv_t = E_t^T k_t, dg_t = <E_t, exp(g_t) S_{t-1}>."""
    q, k, v, g, dout = map(_f64, (q, k, v, g, dout))
    B, H, N, D = q.shape
    states = [np.zeros((B, H, D, v.shape[-1])) if S0 is None else _f64(S0)]
    for t in range(N):
        states.append(np.exp(g[:, :, t])[..., None, None] * states[-1]
                      + k[:, :, t, :, None] * v[:, :, t, None, :])
    dq, dk, dv, dg = (np.zeros(x.shape) for x in (q, k, v, g))
    E = np.zeros(states[0].shape) if dS is None else _f64(dS).copy()
    for t in range(N - 1, -1, -1):
        dq[:, :, t] = np.einsum("bhdm,bhm->bhd", states[t + 1], dout[:, :, t])
        E = E + q[:, :, t, :, None] * dout[:, :, t, None, :]
        dk[:, :, t] = np.einsum("bhdm,bhm->bhd", E, v[:, :, t])
        dv[:, :, t] = np.einsum("bhd,bhdm->bhm", k[:, :, t], E)
        E = np.exp(g[:, :, t])[..., None, None] * E
        dg[:, :, t] = np.sum(E * states[t], axis=(-1, -2))
    return dq, dk, dv, dg, E


def rotary(x, positions, freqs, interleaved=False, mscale=1.0, inverse=False):
    """x [..., N, D] with pair i of its first 2 len(freqs) elements turned by positions * freqs[i];
    positions broadcast against x's leading dimensions and N."""
    x, freqs = _f64(x), _f64(freqs)
    y, half = x.copy(), len(freqs)
    i = np.arange(half)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    angle = np.asarray(positions)[..., None].astype(np.longdouble) * freqs
    c, s = (mscale * f(angle).astype(np.float64) for f in (np.cos, np.sin))
    s = -s if inverse else s
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., lo] * s + x[..., hi] * c
    return y


def _weight(w):
    w = _f64(w)
    return w if w.ndim == 1 else w[None, :, None, :]


def norm_gate(x, z, w, eps=1e-6):
    """x / sqrt(mean(x^2) + eps) * w * z sigmoid(z) over the last axis; w [M] or [H, M]."""
    x, z = _f64(x), _f64(z)
    n = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    return n * _weight(w) * z / (1.0 + np.exp(-z))


def norm_gate_backward(x, z, w, dy, eps=1e-6):
    """(dx, dz, dw) of sum(dy * norm_gate(x, z, w, eps))."""
    x, z, dy = map(_f64, (x, z, dy))
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    n, s, wide = x * r, 1.0 / (1.0 + np.exp(-z)), _weight(w)
    dn = dy * wide * z * s
    dx = r * (dn - n * np.mean(dn * n, axis=-1, keepdims=True))
    dz = dy * wide * n * (s + z * s * (1.0 - s))
    dw = np.sum(dy * n * z * s, axis=(0, 1, 2) if np.ndim(w) == 1 else (0, 2))
    return dx, dz, dw
