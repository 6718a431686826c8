"""The INT8 (W8A8) layer operators as they are measured: each in a plain form of elementary torch
operations, and as a user calls it from this package.

  linear   y = (xq . wq^T) * scale_w * scale_a (+ bias): the product of per-token INT8 activation codes and
           per-channel INT8 weights
  gated    h = act(g) * u with g and u two such products on the same codes (a gated feed-forward's first half)
  norm     b = post-norm of a block's output, r = res_scale * residual + gate * branch_scale * b, n = the next
           block's norm of r; r and n, or r and the INT8 codes and scales of n
"""
import math

import torch

own = False

# the widths of the decode and prefill workloads this package is measured on: hidden 2048, intermediate 8192;
# the MoE layer's experts have intermediate 1024
HIDDEN, INTER, EXPERT = 2048, 8192, 1024
MOST = 2 * 4096 * INTER * HIDDEN          # multiply-adds of the largest listed product


def _linear(name, m, n, k, out="bf16", bias=False):
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "out": out, "bias": bias}


def _gated(name, m, n, k, act="silu", out="bf16"):
    return {"name": name, "op": "gated", "m": m, "n": n, "k": k, "act": act, "out": out}


def _norm(name, t, h, x="bf16", res="bf16", post=False, gates=0, res_scale=1.0, branch_scale=1.0, out="bf16", quant=True):
    return {"name": name, "op": "norm", "t": t, "h": h, "x": x, "res": res, "post": post, "gates": gates,
            "res_scale": res_scale, "branch_scale": branch_scale, "out": out, "quant": quant}


def listed():
    return [
        # one token through the output projection of a decode step: latency
        _linear("linear_decode_1", 1, HIDDEN, HIDDEN),
        # a small decode batch through the down projection, whose fp32 output joins an fp32 residual
        _linear("linear_decode_16", 16, HIDDEN, INTER, out="f32"),
        # a chunk of a prompt whose length and output width are no multiples of anything, with a bias
        _linear("linear_ragged_333", 333, 1003, 1040, bias=True),
        # a prefill chunk through an up projection
        _linear("linear_prefill_512", 512, INTER, HIDDEN),
        # a long prompt through the down projection
        _linear("linear_prefill_4096", 4096, HIDDEN, INTER),
        # one token through gate and up
        _gated("gated_decode_1", 1, INTER, HIDDEN),
        # the tokens one expert gets of a batch, expert widths, GELU
        _gated("gated_expert_200", 200, EXPERT, HIDDEN, act="gelu"),
        # a long prompt through gate and up: the largest product
        _gated("gated_prefill_4096", 4096, INTER, HIDDEN),
        # the block boundary of one decoded token
        _norm("norm_decode_1", 1, HIDDEN),
        # a prompt's block boundary with every part: norm after, gate per channel, both scales
        _norm("norm_prefill_4096", 4096, HIDDEN, post=True, gates=1, res_scale=0.9, branch_scale=0.25),
        # an odd width, gates per sequence, 16-bit floats of the other kind, the normed rows kept
        _norm("norm_odd_1111", 1111, 1001, x="f16", res="f32", post=True, gates=11, out="f16", quant=False),
        # a long batch of wide rows with an fp32 block output and residual
        _norm("norm_wide_8192", 8192, INTER, x="f32", res="f32", out="bf16", quant=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "gated", "norm"))
    if op == "norm":
        h = _log_int(rng, 64, INTER)
        if rng.random() < 0.5:
            h = max(64, h // 64 * 64)                 # the widths that models have
        t = _log_int(rng, 1, max(2, min(32768, 8192 * INTER // h)))
        gates = rng.choice((0, 1, t, 2))
        gates = 2 if gates == 2 and t % 2 == 0 else min(gates, 1) if gates == 2 else gates
        quant = rng.random() < 0.6
        return {"op": "norm", "t": t, "h": h, "x": rng.choice(("bf16", "bf16", "f16", "f32")),
                "res": rng.choice(("bf16", "bf16", "f16", "f32")), "post": rng.random() < 0.5, "gates": gates,
                "res_scale": rng.choice((1.0, 0.5, 0.9)), "branch_scale": rng.choice((1.0, 0.22)),
                "out": rng.choice(("bf16", "bf16", "f16", "f32")), "quant": quant}
    while True:
        m = _log_int(rng, 1, 4096)
        n = _log_int(rng, 64, INTER)
        if rng.random() < 0.5:
            n = max(64, n // 64 * 64)
        k = 16 * _log_int(rng, 4, INTER // 16)
        if m * n * k * (2 if op == "gated" else 1) <= MOST:
            break
    c = {"op": op, "m": m, "n": n, "k": k, "out": rng.choice(("bf16", "bf16", "f32"))}
    if op == "linear":
        c["bias"] = rng.random() < 0.3
    else:
        c["act"] = rng.choice(("silu", "silu", "gelu"))
    return c


_DTYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-5


def _codes(v):
    """Rows quantized to INT8: amax / 127 per row, round half to even."""
    scale = v.abs().amax(-1) / 127
    return (v / scale.clamp_min(1e-30)[:, None]).round().clamp(-128, 127).to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        # a residual stream with a few large channels, as trained models have
        big = 1 + 9 * (torch.rand(h, generator=gen, device="cuda") < 0.01).float()
        s = {"x": normal(t, h).to(_DTYPE[case["x"]]), "residual": (normal(t, h) * big * 4).to(_DTYPE[case["res"]]),
             "pre_w": 1 + 0.2 * normal(h), "post_w": 1 + 0.2 * normal(h) if case["post"] else None,
             "gate": normal(case["gates"], h) if case["gates"] else None}
        return {"case": case, **s}
    m, n, k = case["m"], case["n"], case["k"]
    # heavy-tailed activations (Student-t, 3 degrees of freedom), weights N(0, 0.02) with 0.1% outliers x20
    x = normal(m, k) / (normal(m, k).square() + normal(m, k).square() + normal(m, k).square()).div_(3).sqrt_().clamp_min_(0.05)
    xq, scale_a = _codes(x.to(torch.bfloat16).float())
    s = {"xq": xq, "scale_a": scale_a}
    for part in ("gate", "up") if case["op"] == "gated" else ("w",):
        w = 0.02 * normal(n, k)
        w.mul_(1 + 19 * (torch.rand((n, k), generator=gen, device="cuda") < 0.001).float())
        s["wq_" + part], s["scale_" + part] = _codes(w)
    s["bias"] = normal(n) if case.get("bias") else None
    return {"case": case, **s}


def _product(s, part):
    return (s["xq"].float() @ s["wq_" + part].float().t()) * s["scale_" + part] * s["scale_a"][:, None]


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _rstd(v):
    # the mean square of a row is a long sum, and codes lie next to rounding borders: 64 bits, rounded once
    return torch.rsqrt(v.double().square().mean(-1, keepdim=True) + EPS).float()


def _plain_norm(s):
    c = s["case"]
    b = s["x"].float()
    if s["post_w"] is not None:
        b = b * _rstd(b) * s["post_w"]
    b = b * c["branch_scale"]
    if s["gate"] is not None:
        b = (b.view(c["gates"], -1, c["h"]) * s["gate"][:, None, :]).view(c["t"], c["h"])
    r = s["residual"].float() * c["res_scale"] + b
    y = (r * _rstd(r) * s["pre_w"]).to(_DTYPE[c["out"]])
    out = {"residual": r.to(s["residual"].dtype)}
    if c["quant"]:
        # the codes are whole numbers: they have to be equal, and stand for codes * scale
        v = y.float()
        scale = v.abs().amax(-1, keepdim=True) / 127
        out["xq"] = torch.where(scale > 0, (v / scale).round().clamp(-128, 127), 0.0).to(torch.int8)
        out["scale_a"] = scale[:, 0]
    else:
        out["y"] = y
    return out


def run(state):
    s, c = state, state["case"]
    if own:
        from moe_linear_layers_b200 import q4
        if c["op"] == "linear":
            return q4.q8_linear_w8a8(s["xq"], s["scale_a"], s["wq_w"], s["scale_w"], bias=s["bias"], out_dtype=_DTYPE[c["out"]])
        if c["op"] == "gated":
            return q4.q8_linear_w8a8_gated(s["xq"], s["scale_a"], s["wq_gate"], s["scale_gate"], s["wq_up"], s["scale_up"],
                                           act=c["act"], out_dtype=_DTYPE[c["out"]])
        r, y, xq, scale_a = q4.block_norm(s["x"], s["residual"], s["pre_w"], post_w=s["post_w"], gate=s["gate"], eps=EPS,
                                          res_scale=c["res_scale"], branch_scale=c["branch_scale"],
                                          out_dtype=_DTYPE[c["out"]], quant=c["quant"], want_y=not c["quant"])
        return {"residual": r, "xq": xq, "scale_a": scale_a} if c["quant"] else {"residual": r, "y": y}
    if c["op"] == "linear":
        y = _product(s, "w")
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(_DTYPE[c["out"]])
    if c["op"] == "gated":
        return (_act(_product(s, "gate"), c["act"]) * _product(s, "up")).to(_DTYPE[c["out"]])
    return _plain_norm(s)


def work(case):
    if case["op"] == "norm":
        t, h = case["t"], case["h"]
        per = _SIZE[case["x"]] + 2 * _SIZE[case["res"]] + (1 if case["quant"] else _SIZE[case["out"]])
        vectors = h * (4 + (4 if case["post"] else 0) + 4 * case["gates"])
        return {"bytes": t * h * per + vectors + (4 * t if case["quant"] else 0), "flops": t * h * 12}
    m, n, k = case["m"], case["n"], case["k"]
    mats = 2 if case["op"] == "gated" else 1
    return {"bytes": m * k + mats * n * k + 4 * (m + mats * n) + m * n * _SIZE[case["out"]] + (4 * n if case.get("bias") else 0),
            "flops": 2 * mats * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "norm":
        h = case["h"]
        v = s["x"].to(f64)
        if s["post_w"] is not None:
            v = v / torch.sqrt((v * v).sum(1, keepdim=True) / h + EPS) * s["post_w"].to(f64)
        v = v * case["branch_scale"]
        if s["gate"] is not None:
            v = v * s["gate"].to(f64).repeat_interleave(case["t"] // case["gates"], 0)
        r = s["residual"].to(f64) * case["res_scale"] + v
        y = r / torch.sqrt((r * r).sum(1, keepdim=True) / h + EPS) * s["pre_w"].to(f64)
        if not case["quant"]:
            return {"residual": r, "y": y}
        # the codes are whole numbers, decided next to borders; the scale is that of the rows as they are rounded
        return {"residual": r, "xq": None, "scale_a": y.to(_DTYPE[case["out"]]).to(f64).abs().amax(1) / 127}
    x = s["xq"].to(f64) * s["scale_a"].to(f64).unsqueeze(1)
    if case["op"] == "linear":
        y = torch.einsum("mk,nk->mn", x, s["wq_w"].to(f64) * s["scale_w"].to(f64).unsqueeze(1))
        return y if s["bias"] is None else y + s["bias"].to(f64)
    g = torch.einsum("mk,nk->mn", x, s["wq_gate"].to(f64) * s["scale_gate"].to(f64).unsqueeze(1))
    u = torch.einsum("mk,nk->mn", x, s["wq_up"].to(f64) * s["scale_up"].to(f64).unsqueeze(1))
    if case["act"] == "silu":
        return g * torch.sigmoid(g) * u
    return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * u
