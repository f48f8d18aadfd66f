"""The feed-forward half of a layer, as cases that can be timed and compared.

Behind the attention a layer normalises the residual stream and passes it through a gated
feed-forward network; its training keeps what the backward pass needs, in 8 bits if memory is short:

  layer norm         la_layer_norm, la_layer_norm_backward       y = (x - mean) / sd * w + b
  gated projections  la_ffn_gate, la_ffn_gate_backward           h = act(x wg^T) * (x wu^T)
  8-bit checkpoints  la_checkpoint, la_checkpoint_restore; the norm and the projections write one
                     in their forward pass and read it in their backward pass

A checkpoint holds whole numbers of -127 .. 127 and a power of two, the step, for each block of
32 neighbours of a row: the smallest step, at least 2^-126, for which every |value| / step is
below 127.5. What it stands for is round(value / step) * step, ties to the even number.

`run` computes them in plain torch where `own` is false and through the library where it is
true; `exact` has the same results in 64 bits, from the definitions.
"""

import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BLOCK = 32
EPS = 1e-5
MOST = {"bf16": 65536 * 512 * 1408, "f32": 2048 * 512 * 1408}  # T * C * F of a case


# ------------------------------------------------------------------------ cases

def listed():
    return [
        # the 4 x 16384 tokens of this repository's training step, 8 heads of 64 wide
        {"name": "projections long", "op": "ffn", "T": 65536, "C": 512, "F": 1408, "act": "silu", "type": "bf16"},
        {"name": "projections long backward", "op": "ffn_backward", "T": 65536, "C": 512, "F": 1408, "act": "silu",
         "type": "bf16"},
        # the training step of a wider layer that keeps both products in 8 bits
        {"name": "step of a wide layer, 8 bits", "op": "ffn_step", "T": 4096, "C": 2048, "F": 5632, "act": "silu",
         "type": "bf16"},
        # a ragged batch through a layer of odd sizes, nothing kept
        {"name": "projections odd backward", "op": "ffn_backward", "T": 1237, "C": 840, "F": 2248, "act": "gelu",
         "type": "bf16"},
        # one token of each of 256 streams (this repository's decode workload), and of a single one
        {"name": "projections of 256 tokens", "op": "ffn", "T": 256, "C": 2048, "F": 5632, "act": "silu", "type": "bf16"},
        {"name": "projections of one token", "op": "ffn", "T": 1, "C": 2048, "F": 5632, "act": "silu", "type": "bf16"},
        # a small float32 model, as a gradient check trains it
        {"name": "projections float32 backward", "op": "ffn_backward", "T": 777, "C": 256, "F": 680, "act": "gelu",
         "type": "f32"},
        # the norm in front of the training step's projections, and its way back
        {"name": "norm long", "op": "norm", "T": 65536, "C": 512, "type": "bf16"},
        {"name": "norm long backward", "op": "norm_backward", "T": 65536, "C": 512, "type": "bf16"},
        # a float32 norm of an odd size that keeps its input in 8 bits
        {"name": "norm step odd, 8 bits", "op": "norm_step", "T": 2001, "C": 1000, "type": "f32"},
        # activations put away in 8 bits and taken back, at the training step's size and a ragged one
        {"name": "checkpoint long", "op": "checkpoint", "T": 65536, "C": 512, "type": "bf16"},
        {"name": "checkpoint odd", "op": "checkpoint", "T": 333, "C": 2248, "type": "f32"},
    ]


def _spread(rng, low, high):
    """A whole number between low and high, even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("ffn", "ffn", "ffn", "ffn_backward", "ffn_backward", "ffn_step", "norm", "norm_backward",
                     "norm_step", "checkpoint"))
    # (in float32 two exact enough sums that fall on either side of a checkpoint's rounding are a step apart,
    # which float32 results would show: the step that keeps its products is drawn in bf16)
    case = {"op": op, "type": "bf16" if op == "ffn_step" or rng.random() < 0.7 else "f32"}
    if op in ("ffn", "ffn_backward", "ffn_step"):
        most = MOST[case["type"]]
        case["C"] = 8 * _spread(rng, 8, 256)
        case["F"] = 8 * max(8, int(case["C"] * rng.choice((1.5, 2, 8 / 3, 8 / 3, 4)) / 8 + rng.random()))
        case["T"] = _spread(rng, 1 if op == "ffn" else 16, min(65536, most // (case["C"] * case["F"])))
        case["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh"))
    else:
        case["C"] = 8 * _spread(rng, 8, 1024)
        case["T"] = _spread(rng, 1, min(65536, 65536 * 512 // (case["C"] * (1 if case["type"] == "bf16" else 2))))
    return case


def work(case):
    e = 2 if case["type"] == "bf16" else 4
    op, T, C = case["op"], case["T"], case["C"]
    n = T * C
    kept = T * (C + -(-C // BLOCK))  # a checkpoint of [T, C]
    if op == "norm":
        return {"bytes": 2 * n * e + 2 * C * e, "flops": 8 * n}
    if op == "norm_backward":
        return {"bytes": 3 * n * e + 3 * C * e, "flops": 16 * n}
    if op == "norm_step":  # x, y, the checkpoint twice, dy, dx
        return {"bytes": 4 * n * e + 2 * kept + 4 * C * e, "flops": 26 * n}
    if op == "checkpoint":
        return {"bytes": 2 * n * e + 2 * kept, "flops": 4 * n}
    F = case["F"]
    product, kept = 2 * T * C * F, 2 * T * (F + -(-F // BLOCK))
    if op == "ffn":
        return {"bytes": (n + 2 * C * F + T * F) * e, "flops": 2 * product}
    if op == "ffn_backward":  # both products again, two products each for dx and the weights
        return {"bytes": (2 * n + 4 * C * F + T * F) * e, "flops": 6 * product}
    return {"bytes": (2 * n + 4 * C * F + 2 * T * F) * e + 2 * kept, "flops": 6 * product}


# ----------------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    t = TYPES[case["type"]]
    T, C = case["T"], case["C"]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(t)

    s = {"case": case}
    if case["op"].startswith("ffn"):
        F = case["F"]
        s["x"] = normal(T, C)
        s["wg"], s["wu"] = normal(F, C, scale=C ** -0.5), normal(F, C, scale=C ** -0.5)
        if case["op"] != "ffn":
            s["dh"] = normal(T, F, scale=0.1)
        return s
    # a residual stream: a few channels are much larger than the rest, and off zero
    size = torch.exp(0.7 * torch.randn(C, generator=gen, device=DEV))
    mean = 0.3 * torch.randn(C, generator=gen, device=DEV)
    s["x"] = (torch.randn(T, C, generator=gen, device=DEV) * size + mean).to(t)
    if case["op"] != "checkpoint":
        s["w"], s["b"] = 1 + normal(C, scale=0.1), normal(C, scale=0.1)
    if case["op"] in ("norm_backward", "norm_step"):
        s["dy"] = normal(T, C, scale=0.1)
    return s


# ------------------------------------------------------------------ the operators

def run(s):
    return _library(s) if own else _plain(s)


def _library(s):
    import kernelized_causal_self_gb300 as la
    case, x = s["case"], s["x"]
    op = case["op"]
    if op == "ffn":
        return la.la_ffn_gate(x, s["wg"], s["wu"], activation=case["act"])
    if op == "ffn_backward":
        return la.la_ffn_gate_backward(x, s["wg"], s["wu"], s["dh"], activation=case["act"])
    if op == "ffn_step":
        kept = _room(case["T"], 2, case["F"])
        h = la.la_ffn_gate(x, s["wg"], s["wu"], activation=case["act"], checkpoint=kept)
        return (h, *la.la_ffn_gate_backward(x, s["wg"], s["wu"], s["dh"], activation=case["act"],
                                            checkpoint=kept))
    if op == "norm":
        return la.la_layer_norm(x, s["w"], s["b"], eps=EPS)
    if op == "norm_backward":
        return la.la_layer_norm_backward(x, s["w"], s["dy"], eps=EPS)
    if op == "norm_step":
        kept = _room(case["T"], case["C"])
        y = la.la_layer_norm(x, s["w"], s["b"], eps=EPS, checkpoint=kept)
        return (y, *la.la_layer_norm_backward(kept, s["w"], s["dy"], eps=EPS))
    return la.la_checkpoint_restore(*la.la_checkpoint(x), dtype=x.dtype)


def _room(*shape):
    return (torch.empty(shape, dtype=torch.int8, device=DEV),
            torch.empty((*shape[:-1], -(-shape[-1] // BLOCK)), dtype=torch.uint8, device=DEV))


def _plain(s):
    case = s["case"]
    op, t, x = case["op"], TYPES[case["type"]], s["x"].float()
    if op == "checkpoint":
        return _plain_kept(x).to(t)
    if op == "norm":
        return _plain_norm(x, s).to(t)
    if op == "norm_backward":
        return _plain_norm_backward(x, s)
    if op == "norm_step":
        return (_plain_norm(x, s).to(t), *_plain_norm_backward(_plain_kept(x), s))
    wg, wu = s["wg"].float(), s["wu"].float()
    a, u = x @ wg.t(), x @ wu.t()
    if op == "ffn":
        return (_plain_act(a, case["act"])[0] * u).to(t)
    h = ()
    if op == "ffn_step":
        h = ((_plain_act(a, case["act"])[0] * u).to(t),)
        a, u = _plain_kept(a), _plain_kept(u)
    dh = s["dh"].float()
    f, df = _plain_act(a, case["act"])
    da, du = dh * u * df, dh * f
    return (*h, (da @ wg + du @ wu).to(t), (da.t() @ x).to(t), (du.t() @ x).to(t))


def _plain_act(a, act):
    """The activation and its derivative."""
    if act == "silu":
        s = torch.sigmoid(a)
        return a * s, s * (1 + a * (1 - s))
    if act == "gelu_tanh":  # (1 + tanh(z)) / 2 = sigmoid(2 z)
        c = 2 * (2 / math.pi) ** 0.5
        s = torch.sigmoid(c * (a + 0.044715 * a ** 3))
        return a * s, s + a * s * (1 - s) * c * (1 + 3 * 0.044715 * a * a)
    p = 0.5 * (1 + torch.erf(a * 0.5 ** 0.5))
    return a * p, p + a * torch.exp(-0.5 * a * a) * (2 * math.pi) ** -0.5


def _plain_kept(x):
    """What the checkpoint of x stands for."""
    n = x.shape[-1]
    blocks = torch.nn.functional.pad(x, (0, -n % BLOCK)).unflatten(-1, (-1, BLOCK))
    m, k = torch.frexp(blocks.abs().amax(-1, keepdim=True))  # m * 2^k, m in [0.5, 1)
    k = (k + (m >= 127.5 / 128) - 7).clamp(min=-126)
    step, inverse = (((127 + e) << 23).view(torch.float32) for e in (k, -k))
    return (torch.round(blocks * inverse) * step).flatten(-2)[..., :n]


def _plain_norm(x, s):
    d = x - x.mean(-1, keepdim=True)
    return d * torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS) * s["w"].float() + s["b"].float()


def _plain_norm_backward(x, s):
    t, dy, w = s["dy"].dtype, s["dy"].float(), s["w"].float()
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + EPS)
    n, g = d * r, dy * w
    dx = r * (g - g.mean(-1, keepdim=True) - n * (g * n).mean(-1, keepdim=True))
    return dx.to(t), (dy * n).sum(0).to(t), dy.sum(0).to(t)


# -------------------------------------------------------------- 64 bits, by definition

def _exact_kept(x):
    out = x.clone()
    for at in range(0, x.shape[-1], BLOCK):
        v = x[..., at:at + BLOCK]
        top = v.abs().max(-1, keepdim=True).values / 127.5
        power = torch.floor(torch.log2(top.clamp(min=2.0 ** -300)) + 1).long()
        step = ((1023 + power) << 52).view(torch.float64)
        # (a logarithm next to a whole number may fall on either side of it)
        step = torch.where(top >= step, step * 2, torch.where(top < step / 2, step / 2, step))
        step = step.clamp(min=2.0 ** -126)
        out[..., at:at + BLOCK] = torch.round(v / step) * step
    return out


def _exact_act(a, act):
    if act == "silu":
        return a / (1 + torch.exp(-a))
    if act == "gelu_tanh":
        return a / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3)))
    return a * torch.erfc(-a / math.sqrt(2.0)) / 2


def _exact_norm(x, w, b):
    mean = x.sum(-1, keepdim=True) / x.shape[-1]
    var = ((x - mean) ** 2).sum(-1, keepdim=True) / x.shape[-1]
    return (x - mean) / (var + EPS) ** 0.5 * w + b


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"].double()
    if op == "checkpoint":
        return _exact_kept(x)
    if op.startswith("norm"):
        w, b = s["w"].double().requires_grad_(), s["b"].double().requires_grad_()
        y = _exact_norm(x, w, b).detach()
        if op == "norm":
            return y
        z = (_exact_kept(x) if op == "norm_step" else x).requires_grad_()
        grads = torch.autograd.grad(_exact_norm(z, w, b), (z, w, b), s["dy"].double())
        return (y, *grads) if op == "norm_step" else grads
    wg, wu = s["wg"].double(), s["wu"].double()
    a, u = x @ wg.T, x @ wu.T
    h = _exact_act(a, case["act"]) * u
    if op == "ffn":
        return h
    if op == "ffn_step":
        a, u = _exact_kept(a), _exact_kept(u)
    a, u = a.requires_grad_(), u.requires_grad_()
    da, du = torch.autograd.grad(_exact_act(a, case["act"]) * u, (a, u), s["dh"].double())
    grads = (torch.cat((da, du), 1) @ torch.cat((wg, wu)), (x.T @ da).T, (x.T @ du).T)
    return (h, *grads) if op == "ffn_step" else grads
