"""The feed-forward half's calls at the ends of what they take, on the GPU against the float64 oracle.
Bounds as in test_ffn_gpu.py where no others are given."""

import threading
import time

import numpy as np
import pytest

import oracle
from tests.test_ffn_gpu import (ACTS, BF, DEV, FL, HALF, TYPES, _f64, _ffn_close, _ffn_grads_close, _ffn_inputs,  # noqa: F401
                                _kept_equal, _kept_like, _randn, la)

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


# --------------------------------------------------------------------- checkpoints

def _largest(dtype):
    """Rows with the largest finite values of either type, and the values about the border 63.75 2^122
    from which on a block's step is 2^122."""
    x = _randn(1, 12, 72, dtype=FL)
    big = [torch.finfo(BF).max, 63.75 * 2.0 ** 122, 0.5 * (127 + 127.5) * 2.0 ** 121, 127 * 2.0 ** 121]
    big += [torch.finfo(FL).max if dtype == FL else 2.0 ** 127]
    for i, v in enumerate(big):
        x[2 * i, 3], x[2 * i + 1, 40] = v, -v
        x[2 * i, 5] = 1e38
    assert x.isfinite().all()
    return x.to(dtype)


@TYPES
def test_a_checkpoint_of_the_largest_values_restores_finite(la, dtype):
    x = _largest(dtype)
    if dtype == BF:  # (what lies between two bf16 rounds to one of them: infinity above the largest)
        assert x.isfinite().all()
    pair = la.la_checkpoint(x)
    values = _kept_equal(pair, x)
    assert np.isfinite(values).all()
    unit = np.repeat(2.0 ** (pair[1].cpu().numpy().astype(float) - 127), 32, -1)[:, :72]
    assert np.all(np.abs(values - _f64(x)) <= unit / 2)
    for out in (BF, FL):
        back = la.la_checkpoint_restore(*pair, dtype=out)
        assert np.array_equal(_f64(back), values)
    again = la.la_checkpoint(la.la_checkpoint_restore(*pair, dtype=FL))
    assert torch.equal(again[0], pair[0]) and torch.equal(again[1], pair[1])


def test_restored_bytes_of_any_kind(la):
    """code * step, its magnitude no more than the largest bf16; e = 0 a step of zero, e = 255 NaN."""
    gen = torch.Generator(device=DEV).manual_seed(5)
    codes = torch.randint(-128, 128, (512, 64), generator=gen, device=DEV, dtype=torch.int8)
    exps = torch.arange(1024, device=DEV).remainder(256).to(torch.uint8).view(512, 2)
    e = exps.cpu().numpy().astype(float)
    step = np.repeat(np.where(e == 255, np.nan, np.where(e == 0, 0.0, 2.0 ** (e - 127))), 32, -1)
    most = 2.0 ** 128 - 2.0 ** 120
    want = np.clip(codes.cpu().numpy() * step, -most, most)
    for out in (BF, FL):
        back = _f64(la.la_checkpoint_restore(codes, exps, dtype=out))
        assert np.array_equal(back, want, equal_nan=True)


@TYPES
@ACTS
def test_gradients_through_a_checkpoint_of_the_largest_values(la, act, dtype):
    """a and u up to the largest finite values: da = dh u act'(a) with dh so small that it is finite. What
    the blocks hold are whole multiples of 2^122 and 2^117: act(a) is 0 or a, its derivative 0, 1 or, at 0, 1/2."""
    T, C, F = 4, 8, 64
    a = torch.zeros(F, device=DEV)
    a[0:32:4], a[1:32:4], a[2:32:4] = torch.finfo(BF).max, -3e38, 1e37
    a[32::4], a[33::4], a[34::4] = 1e37, -9e36, 7e36
    u = a.flip(0)
    both = torch.stack((a, u))[None].expand(T, 2, F).contiguous()
    pair = la.la_checkpoint(both)
    kept = oracle.checkpoint(_f64(both))[2]
    x, wg, wu, _ = _ffn_inputs(T, C, F, dtype)
    dh = _randn(9, T, F, dtype=dtype, scale=2.0 ** -118)
    got = la.la_ffn_gate_backward(x, wg, wu, dh, act, checkpoint=pair)
    assert all(g.isfinite().all() for g in got)
    f, df = np.maximum(kept[:, 0], 0.0), 0.5 + 0.5 * np.sign(kept[:, 0])
    X, WG, WU, DH = (_f64(t) for t in (x, wg, wu, dh))
    da, du = DH * kept[:, 1] * df, DH * f
    want = da @ WG + du @ WU, da.T @ X, du.T @ X
    tols = (np.abs(da) @ np.abs(WG) + np.abs(du) @ np.abs(WU), np.abs(da).T @ np.abs(X), np.abs(du).T @ np.abs(X))
    for g, w, t in zip(got, want, tols):
        # da, du rounded once, two products and the sum of at most 2 F terms before it, the result
        assert np.all(np.abs(_f64(g) - w) <= HALF[dtype] * np.abs(w) + (HALF[dtype] + (2 * F + 8) * 2.0 ** -23) * t)


@TYPES
def test_norm_gradients_through_a_checkpoint_of_the_largest_values(la, dtype):
    """Finite blocks stay finite: such a row's squares are past float32, its root zero, and dx with it."""
    x, w, dy = _largest(dtype), _randn(2, 72, dtype=dtype), _randn(3, 12, 72, dtype=dtype)
    x[:10, 5] = 0.0  # (a second large value, with which the row's sum is past float32 too)
    kept = la.la_checkpoint(x)
    dx, dw, db = la.la_layer_norm_backward(kept, w, dy)
    assert not any(t.isnan().any() for t in (dx, dw, db))
    plain = [10, 11]  # rows of ordinary values
    alone = la.la_layer_norm_backward((kept[0][plain], kept[1][plain]), w, dy[plain])
    assert torch.equal(dx[plain], alone[0])


# ------------------------------------------------------------------------ projections

@TYPES
@ACTS
@pytest.mark.parametrize("T", [1, 40, 2100])
def test_gradients_of_the_largest_products(la, T, act, dtype):
    """a of 1e34 to 3e38 and their negatives: act'(a) is 1 or 0, so that da = dh u (u = 1) or 0, finite
    as the formula has it."""
    F, C = 136, 16
    a = torch.tensor([1e34, 2e36, 7e36, 3e37, 1e38, 3e38, 20.0, 1e20], device=DEV).repeat(F // 8)
    a[::3] *= -1
    x, wg, wu = (torch.zeros(n, C, dtype=dtype, device=DEV) for n in (T, F, F))
    x[:, 0], wu[:, 0] = 1.0, 1.0
    wg[:, 0] = a.to(dtype)
    a = _f64(wg[:, 0])
    dh = torch.zeros(T, F, dtype=dtype, device=DEV)
    dh[0] = 0.5
    _, dwg, dwu = la.la_ffn_gate_backward(x, wg, wu, dh, act)
    f, df = np.maximum(a, 0.0), (a > 0).astype(float)  # (at +-20 to 4e-8)
    assert np.all(np.abs(_f64(dwg[:, 0]) - 0.5 * df) <= HALF[dtype] + 1e-7)
    assert np.all(np.abs(_f64(dwu[:, 0]) - 0.5 * f) <= (2 * HALF[dtype] + 2.0 ** -22) * f + 1e-7)


@TYPES
@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
@pytest.mark.parametrize("size, act", [((2600, 520, 2056), "silu"), ((3000, 456, 2184), "gelu"), ((2313, 392, 2824), "gelu_tanh")],
                         ids=["t2600c520f2056", "t3000c456f2184", "t2313c392f2824"])
def test_many_tiles_for_each_pair(la, size, act, kept, dtype):
    """More than two tiles of h, and of da and du, for each of 76 pairs of CTAs, and more steps of 64 than
    stages: accumulators, stages, staging tiles and dh's tiles are all used again. Every row is compared."""
    T, C, F = size
    assert -(-T // 256) * -(-F // 128) > 2 * 76 and C > 6 * 64
    x, wg, wu, dh = _ffn_inputs(*size, dtype)
    pair = _kept_like(T, 2, F) if kept else None
    h = la.la_ffn_gate(x, wg, wu, act, checkpoint=pair)
    _ffn_close(h, x, wg, wu, act, dtype)
    values = None
    if kept:
        au = _f64(la.la_checkpoint_restore(*pair, dtype=FL))
        values = au[:, 0], au[:, 1]
        unit = np.repeat(2.0 ** (pair[1].cpu().numpy().astype(float) - 127), 32, -1)[..., :F]
        X = _f64(x)
        for i, w in enumerate((wg, wu)):
            off = C * 2.0 ** -23 * (np.abs(X) @ np.abs(_f64(w)).T)
            assert np.all(np.abs(au[:, i] - X @ _f64(w).T) <= unit[:, i] / 2 + off)
    grads = la.la_ffn_gate_backward(x, wg, wu, dh, act, checkpoint=pair)
    _ffn_grads_close(grads, x, wg, wu, dh, act, dtype, values)
    again = la.la_ffn_gate_backward(x, wg, wu, dh, act, checkpoint=pair)
    assert all(torch.equal(p, q) for p, q in zip(grads, again))


def test_sums_of_many_tokens_do_not_drift(la):
    """dwu of T equal positive terms, T = 3 * 2^18. The tensor cores' adder cuts off towards zero: an
    addition of 16 terms loses one to two units, 2^-23 of the sum so far, which grows evenly. A part of
    n terms is n / 16 * 2^-23 of itself too small, by two units, and parts are added in float32, rounded
    (24 of them: 2^-20). With n = 32768 at most the mean loss is 2^-12. The results' own rounding to bf16 is up
    as often as down: 128 x 128 different products, each off by up to 2^-8, evenly, are off by 2^-8 / sqrt(3 2^14) =
    2^-15.8 in the mean, and four times that is 2^-13.8. One part of 2^18 terms or more loses 1.3e-3 > 2^-10."""
    T, C, F = 3 << 18, 512, 1408
    gen = torch.Generator(device=DEV).manual_seed(1)
    v, d = ((torch.rand(n, generator=gen, device=DEV) + 1).to(BF) for n in (C, F))
    v[0] = 1.0
    x, dh = v.expand(T, C).contiguous(), d.expand(T, F).contiguous()
    wg, wu = torch.zeros(F, C, dtype=BF, device=DEV), torch.zeros(F, C, dtype=BF, device=DEV)
    wg[:, 0] = 32.0  # a = 32, silu(a) = 32 to 2^-45, u = 0
    dx, dwg, dwu = la.la_ffn_gate_backward(x, wg, wu, dh)
    rel = dwu.double() / (32.0 * T * d.double()[:, None] * v.double()[None]) - 1
    assert abs(rel.mean().item()) <= 2.0 ** -12 + 2.0 ** -13
    assert rel.abs().max().item() <= HALF[BF] + 32768 * 2.0 ** -23
    assert not dwg.any() and torch.equal(dx[0], dx[-1])


def _grid(act):
    """Whole multiples of a power of two, 8 bits each: exact in bf16, and as x w with x = 1."""
    top, step = (80.0, 0.5) if act == "silu" else (13.0, 0.0625) if act == "gelu" else (5.0, 0.03125)
    a = np.arange(-top, top + step, step)
    return np.concatenate([a, np.full(-len(a) % 8, 1.0)])


def _act_bound(a, act):
    """Relative error of act(a) in float32, in steps of 2^-24, by the roundings on the way. A base-2
    exponential and a reciprocal are off by 4, a product, sum or constant by 1.
    silu: the exponent by 2 |a| (constant, product), the sigmoid by that, 4 + 1 + 4, and two products.
    gelu_tanh: z by 6 of itself (constants and products), then the same.
    gelu: a^2 / 2 by 3 of itself (constant, two products), exponential 4, reciprocal 4 + 3 of its
    argument; the polynomial of 8 terms, 2 for its fit, 2 roundings a term of twice its sum at most; 3
    products behind it."""
    if act == "silu":
        return 2 * np.abs(a) + 12
    if act == "gelu":
        return 1.5 * a * a + 4 + 7 * 2 + 2 + 32 + 3
    z = 2 * np.sqrt(2 / np.pi) * (a + 0.044715 * a ** 3)
    return 6 * np.abs(z) + 12


@TYPES
@ACTS
@pytest.mark.parametrize("T", [1, 5, 1000])
def test_activations_far_from_zero_keep_their_digits(la, T, act, dtype):
    """h, da and du where act(a) is small: with x = (1, 0, ...) and wu = (1, 0, ...) a is wg's first column
    and u = 1 in every kernel, without an error, and dwg = da, dwu = du of the first token."""
    a = _grid(act)
    F, C = len(a), 16
    x, wg, wu = (torch.zeros(n, C, dtype=dtype, device=DEV) for n in (T, F, F))
    x[:, 0], wu[:, 0] = 1.0, 1.0
    wg[:, 0] = torch.from_numpy(a).to(DEV).to(dtype)
    assert np.array_equal(_f64(wg[:, 0]), a)
    dh = torch.zeros(T, F, dtype=dtype, device=DEV)
    dh[0] = 1.0
    h = la.la_ffn_gate(x, wg, wu, act)
    _, dwg, dwu = la.la_ffn_gate_backward(x, wg, wu, dh, act)
    f, df = oracle.activation(a, act)
    off = _act_bound(a, act) * 2.0 ** -24
    least = 100 * 2.0 ** -126  # what is below is zero
    half = HALF[dtype]
    assert np.all(np.abs(_f64(h) - f) <= (half + off) * np.abs(f) + least)
    # (sums of one term and zeros, in bf16 of rounded da and du; the result's own rounding; 2^-22 as a sum)
    own = 2 * half + 2.0 ** -22
    assert np.all(np.abs(_f64(dwu[:, 0]) - f) <= (own + off) * np.abs(f) + least)
    # act' is a sum s + a s (1 - s) z' (gelu: P + a e), whose terms are off by `off` and three products, and
    # 1 - s by 1 step of 1
    s = np.where(a == 0, 0.5, f / np.where(a == 0, 1.0, a))
    terms = np.abs(s) + np.abs(df - s)
    one = np.abs(f) * (1.0 if act != "gelu_tanh" else 1.6 * (1 + 0.14 * a * a))
    tol = own * np.abs(df) + (off + 4 * 2.0 ** -24) * terms + 2.0 ** -24 * one + least
    assert np.all(np.abs(_f64(dwg[:, 0]) - df) <= tol)
    assert not dwg[:, 1:].any() and not dwu[:, 1:].any()


@TYPES
@pytest.mark.parametrize("T", [1, 2, 40, 1600])
@pytest.mark.parametrize("kept", [False, True], ids=["recomputed", "kept"])
def test_a_row_with_an_infinity(la, T, kept, dtype):
    """bf16 gives what the formula gives: a = +inf and u = +-inf multiply to infinities, a = -inf gives NaN.
    float32 gives NaN for those infinities, but for a call of one token without a checkpoint. The other rows stay
    as they were."""
    C, F = 136, 200
    x, wg, wu, dh = _ffn_inputs(T, C, F, dtype)
    bad = T // 2
    for value in (float("inf"), -float("inf")):
        y = x.clone()
        y[bad, 3] = value
        pair, clean = (_kept_like(T, 2, F) if kept else None for _ in range(2))
        want = la.la_ffn_gate(x, wg, wu, checkpoint=clean)
        h = la.la_ffn_gate(y, wg, wu, checkpoint=pair)
        rows = [i for i in range(T) if i != bad]
        assert torch.equal(h[rows], want[rows])
        a, u = (value * np.sign(_f64(w[:, 3])) for w in (wg, wu))
        due = np.where(a > 0, u, np.nan)
        got = _f64(h[bad])
        assert not np.isfinite(got).any()
        if dtype == BF or (T == 1 and not kept):
            assert np.array_equal(got, due, equal_nan=True)
        else:
            assert np.isnan(got).all()
        if kept:
            assert torch.all(pair[1][bad] == 255) and torch.equal(pair[1][rows], clean[1][rows])
            assert torch.equal(pair[0][rows], clean[0][rows])
        ref = la.la_ffn_gate_backward(x, wg, wu, dh, checkpoint=clean)
        dx, dwg, dwu = la.la_ffn_gate_backward(y, wg, wu, dh, checkpoint=pair)
        assert torch.equal(dx[rows], ref[0][rows])
        assert not dx[bad].isfinite().any() and not dwg.isfinite().any()


# ------------------------------------------------------------------------------ threads

def test_other_threads_run_while_a_call_waits(la):
    """A launch waits while the stream's queue is full: here behind a kernel of about a second, which ends
    by itself. Another Python thread goes on meanwhile."""
    x = _randn(1, 4, 64, dtype=BF)
    la.la_checkpoint(x)
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)
    other = threading.Thread(target=tick)
    other.start()
    try:
        torch.cuda._sleep(2_000_000_000)
        start = time.perf_counter()
        longest = 0.0
        for _ in range(20000):
            t = time.perf_counter()
            la.la_checkpoint(x)
            longest = max(longest, time.perf_counter() - t)
            if longest > 0.3 or time.perf_counter() - start > 5.0:
                break
    finally:
        stop.set()
        other.join()
        torch.cuda.synchronize()
    if longest <= 0.3:
        pytest.skip("the stream's queue did not fill")
    gaps = np.diff(ticks)
    assert gaps.max() < longest / 2, (gaps.max(), longest)
