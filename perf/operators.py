"""The operators of a gated linear-attention layer, as cases that can be timed and compared.

A layer of this kind rotates q and k by their positions, runs the gated recurrence
S_t = exp(g_t) S_{t-1} + k_t v_t^T, out_t = q_t S_t over them, and normalises each head's
output, weighted and gated, on its way to the output projection:

  rotary            la_rotary                                     (its own gradient: inverse)
  gated recurrence  la_forward_gated, la_prefill_gated, la_extend_gated,
                    la_decode_step_gated, la_backward_gated
  gated head norm   la_norm_gate, la_norm_gate_backward

`run` computes them in plain torch where `own` is false and through the library where it is
true; `exact` has the same results in 64 bits, token by token from the definitions.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
CHUNK = 128  # tokens per chunk of the plain form


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # the training step of this repository's benchmark (B4 H8 N16384, D = M = 64), gated
        {"name": "forward long", "op": "forward", "B": 4, "H": 8, "N": 16384, "D": 64, "M": 64,
         "type": "bf16", "gate": "slow", "states": False},
        {"name": "backward long", "op": "backward", "B": 4, "H": 8, "N": 16384, "D": 64, "M": 64,
         "type": "bf16", "gate": "slow", "states": False},
        # prompts of a ragged length, continued from a cached prefix, heads of 128
        {"name": "prefill wide odd", "op": "forward", "B": 3, "H": 5, "N": 1237, "D": 128, "M": 128,
         "type": "bf16", "gate": "mixed", "states": True},
        # one window of truncated backpropagation through time: states in, their gradients out
        {"name": "backward odd with states", "op": "backward", "B": 2, "H": 3, "N": 2085, "D": 64,
         "M": 64, "type": "bf16", "gate": "mixed", "states": True},
        # a small float32 model with a head of other sizes, as a gradient check trains it
        {"name": "backward float32", "op": "backward", "B": 2, "H": 4, "N": 777, "D": 32, "M": 48,
         "type": "f32", "gate": "mixed", "states": False},
        # a serving batch that takes up to 300 new tokens a stream, states in a pool
        {"name": "extend ragged", "op": "extend", "B": 64, "H": 8, "N": 300, "D": 64, "M": 64,
         "type": "bf16", "gate": "slow"},
        # one token of each of 256 streams (this repository's decode workload), and of a single one
        {"name": "decode many", "op": "decode", "B": 256, "H": 8, "D": 64, "M": 64, "type": "bf16",
         "gate": "slow"},
        {"name": "decode one", "op": "decode", "B": 1, "H": 8, "D": 64, "M": 64, "type": "bf16",
         "gate": "slow"},
        # q and k of the training step, cut out of token-major projections
        {"name": "rotary long", "op": "rotary", "B": 4, "H": 8, "Hk": 8, "N": 16384, "D": 64, "R": 64,
         "type": "bf16", "interleaved": False, "token_major": True, "inverse": False,
         "scaling": "none", "each": False},
        # the next tokens of 16 streams, each far into its context, a part of an odd head
        {"name": "rotary decode", "op": "rotary", "B": 16, "H": 8, "Hk": 2, "N": 1, "D": 80, "R": 20,
         "type": "f32", "interleaved": True, "token_major": False, "inverse": False,
         "scaling": "ramp", "each": True},
        # the training step's head outputs, gated and written token-major for the projection
        {"name": "norm long", "op": "norm", "B": 4, "H": 8, "N": 16384, "M": 64, "type": "bf16",
         "shared": True, "token_major": True},
        # and the way back, at an odd size in float32 with a weight of each head's own
        {"name": "norm backward odd", "op": "norm_backward", "B": 2, "H": 6, "N": 2001, "M": 96,
         "type": "f32", "shared": False, "token_major": True},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("forward", "forward", "backward", "backward", "extend", "decode", "rotary",
                     "norm", "norm_backward"))
    bf16 = rng.random() < 0.75
    case = {"op": op, "type": "bf16" if bf16 else "f32", "H": rng.randint(1, 16)}
    if op in ("forward", "backward", "extend", "decode"):
        wide = (64, 64, 64, 64, 128, 40, 96) if bf16 else (64, 32, 48, 72)
        case["D"] = rng.choice(wide)
        case["M"] = case["D"] if rng.random() < 0.7 else rng.choice(wide)
        case["gate"] = rng.choice(("slow", "mixed"))
        each = case["H"] * case["D"] * case["M"]
        most = 4 * 8 * 16384 * 64 * 64 // (1 if bf16 else 8)
    if op in ("forward", "backward"):
        case["N"] = _spread(rng, 1, 16384)
        case["B"] = _spread(rng, 1, max(1, min(16, most // (each * case["N"]))))
        case["N"] = min(case["N"], most // (each * case["B"]))
        case["states"] = rng.random() < 0.5
    elif op == "extend":
        case["N"] = _spread(rng, 2, 512)
        case["B"] = _spread(rng, 1, max(1, min(256, most // (4 * each * case["N"]))))
    elif op == "decode":
        case["B"] = _spread(rng, 1, 512)
    elif op == "rotary":
        case["N"] = _spread(rng, 1, 16384)
        case["D"] = rng.choice((64, 64, 128, 80, 96))
        case["R"] = case["D"] if rng.random() < 0.6 else rng.choice((16, 20, 32, 48, 64))
        case["Hk"] = rng.choice([h for h in range(1, case["H"] + 1) if case["H"] % h == 0])
        most = 4 * 16 * 16384 * 64 // (1 if bf16 else 2)
        case["B"] = _spread(rng, 1, max(1, min(32, most // ((case["H"] + case["Hk"]) * case["N"]
                                                            * case["D"]))))
        case["interleaved"] = rng.random() < 0.5
        case["token_major"] = rng.random() < 0.5
        case["inverse"] = rng.random() < 0.3
        case["scaling"] = rng.choice(("none", "linear", "base", "ramp"))
        case["each"] = rng.random() < 0.5
    else:
        case["N"] = _spread(rng, 1, 16384)
        case["M"] = rng.choice((64, 64, 128, 32, 96, 72))
        most = 4 * 8 * 16384 * 64 // (1 if bf16 else 4)
        case["B"] = _spread(rng, 1, max(1, min(32, most // (case["H"] * case["N"] * case["M"]))))
        case["shared"] = rng.random() < 0.5
        case["token_major"] = rng.random() < 0.5
    return case


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, B, H = case["op"], case["B"], case["H"]
    if op == "rotary":
        rows = B * case["N"] * (H + case["Hk"])
        pos = 4 * case["N"] * (B if case["each"] else 1)
        return {"bytes": 2 * rows * case["D"] * e + pos, "flops": 6 * rows * case["R"] // 2}
    if op in ("norm", "norm_backward"):
        n = B * H * case["N"] * case["M"]
        return {"bytes": (3 if op == "norm" else 5) * n * e, "flops": (10 if op == "norm" else 24) * n}
    D, M = case["D"], case["M"]
    state = 4 * B * H * D * M
    if op == "decode":
        return {"bytes": 2 * state + B * H * (2 * D + 2 * M + 1) * e, "flops": 4 * B * H * D * M}
    if op == "extend":
        rows = H * sum(_lens(case))
        return {"bytes": 2 * state + rows * (2 * D + 2 * M + 1) * e, "flops": 4 * rows * D * M}
    rows = B * H * case["N"]
    if op == "forward":
        return {"bytes": rows * (2 * D + 2 * M + 1) * e + (2 * state if case["states"] else 0),
                "flops": 4 * rows * D * M}
    return {"bytes": rows * (4 * D + 3 * M + 2) * e + (3 * state if case["states"] else 0),
            "flops": 10 * rows * D * M}


def _lens(case):
    """Token counts of the streams: ragged, among them none, one and all N."""
    n = case["N"]
    lens = [(i * 7919 + 5) % n + 1 for i in range(case["B"])]
    lens[-1] = n
    if case["B"] > 2:
        lens[0], lens[1] = 0, 1
    return lens


# ----------------------------------------------------------------------- inputs

def _gates(gen, shape, kind, dtype):
    """Log-decays, below zero: a sigmoid gate with a long memory ("slow"), or heads that run
    from hardly forgetting to forgetting within a few tokens ("mixed")."""
    x = torch.randn(shape, generator=gen, device=DEV)
    if kind == "slow":
        g = torch.nn.functional.logsigmoid(x + 2.0) / 16.0
    else:
        heads = torch.linspace(-8.0, 0.5, shape[1], device=DEV).view(1, -1, *([1] * (len(shape) - 2)))
        g = -torch.exp(heads + 0.5 * x)
    return g.to(dtype)


def freqs_of(case):
    """Radians per token of each rotated pair, in 64 bits, and the factor on cos and sin."""
    pairs = case["R"] // 2
    i = torch.arange(pairs, dtype=torch.float64)
    factor, base, mscale = 8.0, 10000.0, 1.0
    if case["scaling"] == "base" and case["R"] > 2:
        base = base * factor ** (case["R"] / (case["R"] - 2.0))
    f = base ** (-2.0 * i / case["R"])
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "ramp":
        turns = 4096 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        mscale = 0.1 * math.log(factor) + 1.0
    return f.to(DEV), mscale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    op, B, H = case["op"], case["B"], case["H"]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dtype)

    s = {"case": case}
    if op == "rotary":
        N, D = case["N"], case["D"]
        for name, h in (("q", H), ("k", case["Hk"])):
            s[name] = normal(B, N, h, D).transpose(1, 2) if case["token_major"] else normal(B, h, N, D)
        s["freqs"], s["mscale"] = freqs_of(case)
        start = torch.randint(0, 100000, (B if case["each"] else 1, 1), generator=gen, device=DEV)
        pos = (start + torch.arange(N, device=DEV)).to(torch.int32)
        s["positions"] = pos if case["each"] else pos[0]
        return s
    if op in ("norm", "norm_backward"):
        N, M = case["N"], case["M"]

        def rows():
            return normal(B, N, H, M).transpose(1, 2) if case["token_major"] else normal(B, H, N, M)
        s["x"], s["z"] = normal(B, H, N, M), rows()
        s["w"] = (1 + 0.1 * torch.randn((M,) if case["shared"] else (H, M), generator=gen,
                                        device=DEV)).to(t)
        if op == "norm_backward":
            s["dy"] = rows()
        return s
    D, M = case["D"], case["M"]
    lead = (B, H) if op == "decode" else (B, H, case["N"])
    s["q"], s["k"], s["v"] = (normal(*lead, d, scale=d ** -0.5) for d in (D, D, M))
    s["g"] = _gates(gen, lead, case["gate"], t)
    if op in ("decode", "extend"):
        s["pool"] = normal(B + 3, H, D, M, scale=0.1, dtype=torch.float32)
        order = torch.randperm(B + 3, generator=gen, device=DEV)[:B]
        s["slots"] = order.to(torch.int32)
        s["out"] = torch.zeros((*lead, M), dtype=t, device=DEV)
    if op == "extend":
        s["lens"] = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
    if op in ("forward", "backward"):
        s["S0"] = normal(B, H, D, M, scale=0.1, dtype=torch.float32) if case["states"] else None
    if op == "backward":
        s["dout"] = normal(*lead, M, scale=M ** -0.5)
        s["dS"] = normal(B, H, D, M, scale=0.01, dtype=torch.float32) if case["states"] else None
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import kernelized_causal_self_gb300 as la
    case = s["case"]
    op = case["op"]
    if op == "rotary":
        return la.la_rotary(s["q"], s["k"], s["freqs"], positions=s["positions"],
                            interleaved=case["interleaved"], mscale=s["mscale"],
                            inverse=case["inverse"])
    if op == "norm":
        out = _like(s["z"])
        return la.la_norm_gate(s["x"], s["z"], s["w"], out=out)
    if op == "norm_backward":
        return la.la_norm_gate_backward(s["x"], s["z"], s["w"], s["dy"], dz=_like(s["z"]))
    qkvg = (s["q"], s["k"], s["v"], s["g"])
    if op == "forward" and case["states"]:
        return la.la_prefill_gated(*qkvg, S0=s["S0"])
    if op == "forward":
        return la.la_forward_gated(*qkvg)
    if op == "backward":
        return la.la_backward_gated(*qkvg, s["dout"], S0=s["S0"], dS=s["dS"])
    if op == "extend":
        out = la.la_extend_gated(*qkvg, s["pool"], slots=s["slots"], lens=s["lens"], out=s["out"])
    else:
        out = la.la_decode_step_gated(*qkvg, s["pool"], slots=s["slots"], out=s["out"])
    return out, s["pool"]


def _like(z):
    """An output with z's order of dimensions in memory."""
    return torch.empty_like(z.transpose(1, 2)).transpose(1, 2) if z.transpose(1, 2).is_contiguous() \
        else torch.empty_like(z)


def _plain(s):
    op, t = s["case"]["op"], TYPES[s["case"]["type"]]
    if op == "rotary":
        return _plain_rotary(s, s["q"]), _plain_rotary(s, s["k"])
    if op == "norm":
        x, z, r = _plain_rows(s)
        return (x * r * _weight(s) * (z * torch.sigmoid(z))).to(t)
    if op == "norm_backward":
        x, z, r = _plain_rows(s)
        dy, w, sig = s["dy"].float(), _weight(s), torch.sigmoid(z)
        n = x * r
        dn = dy * w * (z * sig)
        dx = r * (dn - n * (dn * n).mean(-1, keepdim=True))
        dz = dy * w * n * (sig * (1 + z * (1 - sig)))
        dw = (dy * n * (z * sig)).sum((0, 1, 2) if s["w"].dim() == 1 else (0, 2))
        return dx.to(t), dz.to(t), dw.to(t)
    if op == "decode":
        at = s["slots"].long()
        a = torch.exp(s["g"].float())[..., None, None]
        S = s["pool"][at] * a + s["k"].float()[..., :, None] * s["v"].float()[..., None, :]
        s["pool"][at] = S
        s["out"].copy_((s["q"].float()[..., :, None] * S).sum(-2).to(t))
        return s["out"], s["pool"]
    if op == "extend":
        at, n = s["slots"].long(), s["case"]["N"]
        live = (torch.arange(n, device=DEV)[None] < s["lens"][:, None])[:, None]
        k, v, g = s["k"].float(), s["v"].float(), s["g"].float()
        k, g = k * live[..., None], g.masked_fill(~live, 0.0)
        out, S = _plain_forward(s["q"].float(), k, v, g, s["pool"][at])[:2]
        s["pool"][at] = S[:, :, -1]
        s["out"].copy_(torch.where(live[..., None], out.to(t), s["out"]))
        return s["out"], s["pool"]
    q, k, v, g = (s[n].float() for n in ("q", "k", "v", "g"))
    out, S, f = _plain_forward(q, k, v, g, s["S0"])
    if op == "forward":
        return (out.to(t), S[:, :, -1].contiguous()) if s["case"]["states"] else out.to(t)
    dq, dk, dv, dg, dS0 = _plain_backward(q, k, v, s["dout"].float(), S, s["dS"], f)
    grads = (dq.to(t), dk.to(t), dv.to(t), dg.to(t))
    return grads + (dS0,) if s["case"]["states"] else grads


def _plain_rotary(s, x):
    case = s["case"]
    pos = s["positions"].double()
    ang = pos[..., None] * s["freqs"]
    ang = ang[:, None] if case["each"] else ang
    c, n = (torch.cos(ang) * s["mscale"]).float(), (torch.sin(ang) * s["mscale"]).float()
    n = -n if case["inverse"] else n
    R, xf = case["R"], x.float()
    if case["interleaved"]:
        a, b = xf[..., 0:R:2], xf[..., 1:R:2]
        y = torch.stack((a * c - b * n, a * n + b * c), -1).flatten(-2)
    else:
        a, b = xf[..., :R // 2], xf[..., R // 2:R]
        y = torch.cat((a * c - b * n, a * n + b * c), -1)
    return torch.cat((y, xf[..., R:]), -1).to(x.dtype).contiguous()


def _plain_rows(s):
    x, z = s["x"].float(), s["z"].float()
    return x, z, torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)


def _weight(s):
    w = s["w"].float()
    return w if w.dim() == 1 else w[None, :, None]


def _split(x, n):
    """[B, H, N, ...] as [B, H, chunks, CHUNK, ...], zeros behind the last token."""
    pad = -n % CHUNK
    if pad:
        x = torch.cat((x, x.new_zeros((*x.shape[:2], pad, *x.shape[3:]))), 2)
    return x.reshape(*x.shape[:2], -1, CHUNK, *x.shape[3:])


def _plain_forward(q, k, v, g, S0):
    """Outputs, the states before each chunk and after the last, and the chunks' factors."""
    n = q.shape[2]
    q, k, v = (_split(x, n) for x in (q, k, v))
    cum = _split(g.double().clamp(min=-400.0), n).cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=q.device).tril()
    L = torch.where(low, (cum[..., :, None] - cum[..., None, :]).float(), -math.inf).exp()
    tot = cum[..., -1]
    end = tot.cumsum(-1)
    begin = torch.nn.functional.pad(end, (1, 0))  # the log-decay up to each chunk, and to the end
    into, out_of = torch.exp(cum.float())[..., None], torch.exp((tot[..., None] - cum).float())[..., None]
    U = (k * out_of).transpose(-1, -2) @ v
    nc = U.shape[2]
    before = torch.ones(nc + 1, nc, dtype=torch.bool, device=q.device).tril(-1)
    W = torch.where(before, (begin[..., :, None] - end[..., None, :]).float(), -math.inf).exp()
    S = (W @ U.flatten(-2)).unflatten(-1, U.shape[-2:])
    if S0 is not None:
        S = S + torch.exp(begin.float())[..., None, None] * S0[:, :, None]
    P = q @ k.transpose(-1, -2) * L
    out = into * (q @ S[:, :, :-1]) + P @ v
    f = {"n": n, "q": q, "k": k, "v": v, "L": L, "P": P, "into": into, "out_of": out_of, "begin": begin}
    return out.flatten(2, 3)[:, :, :n], S, f


def _plain_backward(q, k, v, dout, S, dS, f):
    n, q, k, v, begin = f["n"], f["q"], f["k"], f["v"], f["begin"]
    do = _split(dout, n)
    R = (q * f["into"]).transpose(-1, -2) @ do
    nc = R.shape[2]
    later = torch.ones(nc + 1, nc, dtype=torch.bool, device=q.device).triu()
    W = torch.where(later, (begin[..., None, :-1] - begin[..., :, None]).float(), -math.inf).exp()
    E = (W @ R.flatten(-2)).unflatten(-1, R.shape[-2:])
    if dS is not None:
        E = E + torch.exp((begin[..., -1:] - begin).float())[..., None, None] * dS[:, :, None]
    dP = do @ v.transpose(-1, -2) * f["L"]
    after = E[:, :, 1:]
    dq = dP @ k + f["into"] * (do @ S[:, :, :-1].transpose(-1, -2))
    dk = dP.transpose(-1, -2) @ q + f["out_of"] * (v @ after.transpose(-1, -2))
    dv = f["P"].transpose(-1, -2) @ do + f["out_of"] * (k @ after)
    # dg_t: what the state after t gives to its gradient less what t's own token adds, from the
    # end of each chunk back
    step = ((q * dq).sum(-1) - (k * dk).sum(-1)).double()
    dg = (S[:, :, 1:] * after).sum((-1, -2)).double()[..., None] + step.flip(-1).cumsum(-1).flip(-1)
    dq, dk, dv, dg = (x.flatten(2, 3)[:, :, :n].contiguous() for x in (dq, dk, dv, dg))
    return dq, dk, dv, dg, E[:, :, 0].contiguous()


# -------------------------------------------------------------- 64 bits, by definition

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rotary":
        turn = torch.polar(torch.full_like(s["freqs"], s["mscale"])[None],
                           s["positions"].double().reshape(-1, 1) * s["freqs"])
        turn = turn.conj() if case["inverse"] else turn
        turn = turn.reshape(-1, 1, case["N"], case["R"] // 2)

        def rotated(x):
            y, half = x.double().clone(), case["R"] // 2
            at = torch.arange(half, device=DEV)
            i, j = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
            z = torch.complex(y[..., i], y[..., j]) * turn
            y[..., i], y[..., j] = z.real, z.imag
            return y
        return rotated(s["q"]), rotated(s["k"])
    if op in ("norm", "norm_backward"):
        x, z, w = (s[n].double().requires_grad_() for n in ("x", "z", "w"))
        rms = ((x ** 2).sum(-1, keepdim=True) / case["M"] + 1e-6) ** 0.5
        y = x / rms * (w if w.dim() == 1 else w.reshape(1, case["H"], 1, -1)) * z / (1 + torch.exp(-z))
        if op == "norm":
            return y.detach()
        return torch.autograd.grad(y, (x, z, w), s["dy"].double())
    q, k, v, a = (s[n].double() for n in ("q", "k", "v", "g"))
    a = a.exp()
    if op == "decode":
        q, k, v, a = (x.unsqueeze(2) for x in (q, k, v, a))
    B, H, N, D, M = *q.shape, v.shape[-1]
    n_b = s["lens"].tolist() if op == "extend" else [N] * B
    S = q.new_zeros(B, H, D, M)
    if op in ("decode", "extend"):
        S = s["pool"].double()[s["slots"].long()]
    elif s["S0"] is not None:
        S = s["S0"].double()
    live = (torch.arange(N, device=DEV)[:, None] < torch.tensor(n_b, device=DEV)).double()
    out, every = q.new_zeros(B, H, N, M), []
    for t in range(N):
        if op == "backward":
            every.append(S)
        here = live[t][:, None, None, None]
        decay = 1 + here * (a[:, :, t, None, None] - 1)
        S = decay * S + here * k[:, :, t, :, None] * v[:, :, t, None, :]
        out[:, :, t] = (q[:, :, t, None] @ S)[:, :, 0] * here[..., 0]
    if op == "forward":
        return (out, S) if case["states"] else out
    if op in ("decode", "extend"):
        pool = s["pool"].double()
        pool[s["slots"].long()] = S
        return (out[:, :, 0] if op == "decode" else out), pool
    do = s["dout"].double()
    dq, dk, dv, dg = (torch.empty_like(x) for x in (q, k, v, a))
    E = s["dS"].double() if s["dS"] is not None else torch.zeros_like(S)
    for t in reversed(range(N)):
        dq[:, :, t] = (S @ do[:, :, t, :, None])[..., 0]
        E = E + q[:, :, t, :, None] * do[:, :, t, None, :]
        dk[:, :, t] = (E @ v[:, :, t, :, None])[..., 0]
        dv[:, :, t] = (k[:, :, t, None] @ E)[:, :, 0]
        S = every.pop()
        E = a[:, :, t, None, None] * E
        dg[:, :, t] = (E * S).sum((-1, -2))
    return (dq, dk, dv, dg, E) if case["states"] else (dq, dk, dv, dg)
