"""The experts' products as a user calls them, each beside its plain form.

Three calls that stand between the MoE dispatch and combine of this library: the product of fp8 rows, as the fp8
dispatch writes them, with fp8 weights that have a scale for each block of 128 x 128 (serving), and the gated
feed-forward block of the experts in 16 bits with its backward pass (training). `run` computes them with elementary
torch operations in 32 bits where `own` is false, and through the library where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
_BLOCK = 128
_E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _fp8(name, T, K, E, inner, outer, swiglu=False, x="e4m3", ue8m0=False, columns=False, dtype="bf16", skew=0.0):
    c = {"op": "fp8", "T": T, "K": K, "E": E, "inner": inner, "outer": outer, "swiglu": swiglu, "x": x, "ue8m0": ue8m0,
         "columns": columns, "dtype": dtype, "skew": skew}
    return c if name is None else {"name": name, **c}


def _fp8_ffn(name, T, K, E, hidden, inner, dtype="bf16", skew=0.0):
    c = {"op": "fp8_ffn", "T": T, "K": K, "E": E, "hidden": hidden, "inner": inner, "dtype": dtype, "skew": skew}
    return c if name is None else {"name": name, **c}


def _ffn(name, T, K, E, hidden, inner, dtype="bf16", skew=0.0, save=True, backward=False):
    c = {"op": "ffn_backward" if backward else "ffn", "T": T, "K": K, "E": E, "hidden": hidden, "inner": inner,
         "dtype": dtype, "skew": skew, "save": save}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one dense projection of a few sequences' tokens (latency alone)
        _fp8("fp8 projection", 4, 1, 1, 4096, 4096),
        # one token's eight experts, gate and up projection with the activation
        _fp8("fp8 one token", 1, 8, 256, 7168, 4096, swiglu=True),
        # a decode step of 256 tokens through both products, fp8 in between: every expert of the layer is read
        _fp8_ffn("fp8 block decode", 256, 8, 256, 7168, 2048),
        # a prompt of 8192 tokens, gate and up projection with the activation
        _fp8("fp8 prompt", 8192, 8, 256, 7168, 4096, swiglu=True),
        # the down projection of a prompt whose rows came in e5m2 with power-of-two scales, column by column; uneven experts
        _fp8("fp8 prompt down", 4096, 6, 64, 2048, 4096, x="e5m2", ue8m0=True, columns=True, skew=0.3),
        # a few tokens through 16-bit experts: the weights are read for a row or two each
        _ffn("block few tokens", 16, 6, 64, 4096, 2048, save=False),
        # a training micro-batch, uneven experts, odd sizes, fp16
        _ffn("block uneven fp16", 2048, 4, 60, 2056, 1368, dtype="fp16", skew=0.5),
        # a training step's 16384 tokens of 64 experts
        _ffn("block training", 16384, 6, 64, 4096, 2048),
        # the gradients of a small block: a few experts, few rows each
        _ffn("backward small", 64, 2, 8, 1024, 512, backward=True),
        # the micro-batch above
        _ffn("backward uneven fp16", 2048, 4, 60, 2056, 1368, dtype="fp16", skew=0.5, backward=True),
        # the training step above
        _ffn("backward training", 16384, 6, 64, 4096, 2048, backward=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("fp8", "fp8", "fp8_ffn", "ffn", "ffn_backward", "ffn_backward"))
    E = rng.choice((1, 1, 8, 32, 60, 64, 128))
    K = rng.randint(1, min(8, E))
    skew = rng.choice((0.0, 0.0, 0.3, 0.6)) if E > 1 else 0.0
    T = _log(rng, 1, 8192)
    dtype = rng.choice(("bf16", "bf16", "fp16"))
    if op == "fp8":
        swiglu = rng.random() < 0.5
        return _fp8(None, T, K, E, _BLOCK * _log(rng, 1, 32), _log(rng, 8, 2048) * (2 if swiglu else 1), swiglu,
                    rng.choice(("e4m3", "e4m3", "e5m2")), rng.random() < 0.3, rng.random() < 0.3, dtype, skew)
    if op == "fp8_ffn":
        return _fp8_ffn(None, T, K, E, _BLOCK * _log(rng, 1, 32), _BLOCK * _log(rng, 1, 16), dtype, skew)
    return _ffn(None, T, K, E, 8 * _log(rng, 4, 512), 8 * _log(rng, 4, 256), dtype, skew, rng.random() < 0.7,
                op == "ffn_backward")


def _used(case):
    """Experts with a row, on average."""
    return case["E"] * (1 - (1 - case["K"] / case["E"]) ** case["T"])


def work(case):
    rows = case["T"] * case["K"]
    if case["op"] == "fp8":
        i, o = case["inner"], case["outer"]
        cols, blocks = o // 2 if case["swiglu"] else o, i // _BLOCK
        return {"bytes": _used(case) * (o * i + 4 * -(-o // _BLOCK) * blocks)
                + rows * (i + (1 if case["ue8m0"] else 4) * blocks + 2 * cols) + 4 * (case["E"] + 1),
                "flops": 2 * rows * o * i}
    h, f = case["hidden"], case["inner"]
    if case["op"] == "fp8_ffn":   # (the fp8 rows between the products go through memory: written once and read once)
        return {"bytes": _used(case) * 3 * h * f * (1 + 4 / _BLOCK ** 2) + rows * (h * (1 + 4 / _BLOCK) + 2 * f * (1 + 4 / _BLOCK)
                                                                               + 2 * h) + 8 * (case["E"] + 1),
                "flops": 6 * rows * h * f}
    if case["op"] == "ffn":
        return {"bytes": 2 * (_used(case) * 3 * h * f + rows * (2 * h + f + (2 * f if case["save"] else 0))) + 4 * (case["E"] + 1),
                "flops": 6 * rows * h * f}
    return {"bytes": 2 * (_used(case) * 3 * h * f + case["E"] * 3 * h * f + rows * (3 * h + 5 * f)) + 4 * (case["E"] + 1),
            "flops": 12 * rows * h * f}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    made = {"fp8": _prepare_fp8, "fp8_ffn": _prepare_fp8_ffn, "ffn": _prepare_ffn, "ffn_backward": _prepare_ffn}[case["op"]]
    return {"case": case, "expert_offsets": _offsets(case, g), **made(case, g)}


def _offsets(case, g):
    """Rows by expert of T tokens with K experts each, some experts more popular than others."""
    T, K, E = case["T"], case["K"], case["E"]
    liking = torch.rand(T, E, device="cuda", generator=g) + case["skew"] * torch.rand(E, device="cuda", generator=g)
    chosen = liking.topk(K, dim=1).indices.reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(chosen, minlength=E).cumsum(0)
    return offsets


def _normal(g, shape, dtype, scale=1.0):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.split(-(-shape[0] // 16)):   # one large draw at a time
        part.copy_(torch.randn(part.shape, device="cuda", generator=g).mul_(scale).clamp_(-_E4M3_MAX, _E4M3_MAX))
    return out


def _fp8_weights(g, E, outer, inner):
    """Codes whose largest are near the format's, and scales that leave outputs of their inputs' size."""
    codes = _normal(g, (E, outer, inner), torch.float8_e4m3fn, 100.0)
    scales = torch.rand(E, -(-outer // _BLOCK), inner // _BLOCK, device="cuda", generator=g) + 0.5
    return codes, scales / (100.0 * math.sqrt(inner))


def _fp8_rows(g, rows, width, case):
    """Rows and scales as the fp8 dispatch writes them."""
    x = torch.randn(rows, width, device="cuda", generator=g)
    most = _E4M3_MAX if case.get("x", "e4m3") == "e4m3" else 57344.0
    scales = x.view(rows, -1, _BLOCK).abs().amax(2) / most
    if case.get("ue8m0"):
        power = torch.ceil(torch.log2(scales))
        codes, scales = x / torch.exp2(power).repeat_interleave(_BLOCK, 1), (power + 127).to(torch.uint8)
    else:
        codes = x / scales.repeat_interleave(_BLOCK, 1)
    codes = codes.clamp(-most, most).to(_DTYPES[case.get("x", "e4m3")])
    if case.get("columns"):
        scales = scales.t().contiguous().t()
    return codes, scales


def _prepare_fp8(case, g):
    rows, cols = case["T"] * case["K"], case["outer"] // 2 if case["swiglu"] else case["outer"]
    w, ws = _fp8_weights(g, case["E"], case["outer"], case["inner"])
    x, xs = _fp8_rows(g, rows, case["inner"], case)
    return {"x": x, "x_scales": xs, "weights": w, "weight_scales": ws,
            "y": torch.empty(rows, cols, dtype=_DTYPES[case["dtype"]], device="cuda")}


def _prepare_fp8_ffn(case, g):
    rows, h, f = case["T"] * case["K"], case["hidden"], case["inner"]
    up, ups = _fp8_weights(g, case["E"], 2 * f, h)
    down, downs = _fp8_weights(g, case["E"], h, f)
    x, xs = _fp8_rows(g, rows, h, case)
    return {"x": x, "x_scales": xs, "w_gate_up": up, "gate_up_scales": ups, "w_down": down, "down_scales": downs,
            "act": torch.empty(rows, f, dtype=torch.float8_e4m3fn, device="cuda"),
            "act_scales": torch.empty(rows, f // _BLOCK, device="cuda"),
            "y": torch.empty(rows, h, dtype=_DTYPES[case["dtype"]], device="cuda")}


def _prepare_ffn(case, g):
    rows, E, h, f, dt = case["T"] * case["K"], case["E"], case["hidden"], case["inner"], _DTYPES[case["dtype"]]
    s = {"x": _normal(g, (rows, h), dt), "w_gate_up": _normal(g, (E, 2 * f, h), dt, 1 / math.sqrt(h)),
         "w_down": _normal(g, (E, h, f), dt, 1 / math.sqrt(f))}
    if case["op"] == "ffn":
        return {**s, "act": torch.empty(rows, f, dtype=dt, device="cuda"), "y": torch.empty(rows, h, dtype=dt, device="cuda"),
                "gate_up": torch.empty(rows, 2 * f, dtype=dt, device="cuda") if case["save"] else None}
    gate_up = _normal(g, (rows, 2 * f), dt)   # (as such weights leave them)
    gate, up = gate_up.float().chunk(2, 1)
    return {**s, "gate_up": gate_up, "act": (gate / (1 + torch.exp(-gate)) * up).to(dt), "grad_y": _normal(g, (rows, h), dt),
            "grad_gate_up": torch.empty_like(gate_up), "grad_x": torch.empty_like(s["x"]),
            "grad_w_gate_up": torch.empty_like(s["w_gate_up"]), "grad_w_down": torch.empty_like(s["w_down"])}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"fp8": _own_fp8, "fp8_ffn": _own_fp8_ffn, "ffn": _own_ffn, "ffn_backward": _own_ffn_backward}[op](s)
    return {"fp8": _plain_fp8, "fp8_ffn": _plain_fp8_ffn, "ffn": _plain_ffn, "ffn_backward": _plain_ffn_backward}[op](s)


def _own_fp8(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_expert_fp8(s["x"], s["x_scales"], s["weights"], s["weight_scales"], s["y"], expert_offsets=s["expert_offsets"],
                     activation=ep.EP_ACT_SWIGLU if s["case"]["swiglu"] else ep.EP_ACT_NONE)
    return s["y"]


def _own_fp8_ffn(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_expert_fp8(s["x"], s["x_scales"], s["w_gate_up"], s["gate_up_scales"], s["act"], y_scales=s["act_scales"],
                     expert_offsets=s["expert_offsets"], activation=ep.EP_ACT_SWIGLU)
    ep.ep_expert_fp8(s["act"], s["act_scales"], s["w_down"], s["down_scales"], s["y"], expert_offsets=s["expert_offsets"])
    return s["y"]


def _own_ffn(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_expert_ffn(s["x"], s["w_gate_up"], s["w_down"], s["act"], s["y"], gate_up=s["gate_up"],
                     expert_offsets=s["expert_offsets"])
    return {"y": s["y"], "act": s["act"], "gate_up": s["gate_up"]}


def _own_ffn_backward(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_expert_ffn_backward(s["grad_y"], s["x"], s["gate_up"], s["act"], s["w_gate_up"], s["w_down"], s["grad_gate_up"],
                              grad_x=s["grad_x"], grad_w_gate_up=s["grad_w_gate_up"], grad_w_down=s["grad_w_down"],
                              expert_offsets=s["expert_offsets"])
    return {m: s[m] for m in ("grad_x", "grad_gate_up", "grad_w_gate_up", "grad_w_down")}


class _Groups:
    """The experts that have rows, and these rows as one [experts, most, width] with zeros behind an expert's last."""

    def __init__(self, offsets):
        offsets = offsets.long()
        counts = offsets[1:] - offsets[:-1]
        self.used = counts.nonzero()[:, 0]
        most = torch.arange(int(counts.max()), device="cuda")
        self.real = most < counts[self.used][:, None]
        self.rows = torch.where(self.real, offsets[self.used][:, None] + most, 0)

    def spread(self, x):
        return torch.where(self.real[..., None], x[self.rows], 0.0)

    def gather(self, y):
        return y[self.real]

    def weights(self, w):
        return w if len(self.used) == w.shape[0] else w[self.used]

    def whole(self, grad, like):
        """Gradients of all experts' weights: zeros for those without rows."""
        if len(self.used) == like.shape[0]:
            return grad.to(like.dtype)
        out = torch.zeros_like(like)
        out[self.used] = grad.to(like.dtype)
        return out


def _blocks(scales, width, axis):
    return scales.repeat_interleave(_BLOCK, axis).narrow(axis, 0, width)


def _plain_rows(x, scales):
    if scales.dtype == torch.uint8:
        scales = torch.exp2(scales.float() - 127)
    return x.float() * _blocks(scales, x.shape[1], 1)


def _plain_weights(groups, w, scales):
    code = groups.weights(w.view(torch.uint8)).view(w.dtype).float()
    s = groups.weights(scales)
    return code.mul_(_blocks(_blocks(s, code.shape[2], 2), code.shape[1], 1))


def _gated(y):
    gate, up = y.chunk(2, -1)
    return gate / (1 + torch.exp(-gate)) * up


def _plain_fp8(s):
    groups = _Groups(s["expert_offsets"])
    w = _plain_weights(groups, s["weights"], s["weight_scales"])
    y = groups.spread(_plain_rows(s["x"], s["x_scales"])) @ w.transpose(1, 2)
    return groups.gather(_gated(y) if s["case"]["swiglu"] else y).to(s["y"].dtype)


def _plain_fp8_ffn(s):
    groups = _Groups(s["expert_offsets"])
    w = _plain_weights(groups, s["w_gate_up"], s["gate_up_scales"])
    act = groups.gather(_gated(groups.spread(_plain_rows(s["x"], s["x_scales"])) @ w.transpose(1, 2)))
    del w
    parts = act.view(act.shape[0], -1, _BLOCK)
    scales = parts.abs().amax(2, keepdim=True) / _E4M3_MAX   # what lies between the products is 8 bits by definition
    codes = (parts / torch.where(scales > 0, scales, 1.0)).clamp(-_E4M3_MAX, _E4M3_MAX).to(torch.float8_e4m3fn)
    act = (codes.float() * scales).view(act.shape)
    w = _plain_weights(groups, s["w_down"], s["down_scales"])
    return groups.gather(groups.spread(act) @ w.transpose(1, 2)).to(s["y"].dtype)


def _plain_ffn(s):
    groups = _Groups(s["expert_offsets"])
    dt = s["x"].dtype
    gate_up = groups.spread(s["x"].float()) @ groups.weights(s["w_gate_up"]).float().transpose(1, 2)
    act = _gated(gate_up)
    y = groups.gather(act @ groups.weights(s["w_down"]).float().transpose(1, 2))
    return {"y": y.to(dt), "act": groups.gather(act).to(dt),
            "gate_up": groups.gather(gate_up).to(dt) if s["case"]["save"] else None}


def _plain_ffn_backward(s):
    groups = _Groups(s["expert_offsets"])
    dt = s["x"].dtype
    grad_y, w_down, w_up = groups.spread(s["grad_y"].float()), groups.weights(s["w_down"]), groups.weights(s["w_gate_up"])
    grad_act = grad_y @ w_down.float()
    gate, up = groups.spread(s["gate_up"].float()).chunk(2, 2)
    p = 1 / (1 + torch.exp(-gate))
    grad = torch.cat((grad_act * up * p * (1 + gate * (1 - p)), grad_act * gate * p), 2)
    del grad_act, gate, up, p
    grad_down = grad_y.transpose(1, 2) @ groups.spread(s["act"].float())
    grad_up = grad.transpose(1, 2) @ groups.spread(s["x"].float())
    return {"grad_x": groups.gather(grad @ w_up.float()).to(dt), "grad_gate_up": groups.gather(grad).to(dt),
            "grad_w_gate_up": groups.whole(grad_up, s["w_gate_up"]), "grad_w_down": groups.whole(grad_down, s["w_down"])}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if work(case)["flops"] > 12e12:   # (64-bit products run at about 1e12 a second)
        return None
    s = prepare(case, seed)
    offsets = s["expert_offsets"].tolist()
    parts = [_EXACT[case["op"]](s, e, slice(offsets[e], offsets[e + 1])) for e in range(case["E"])]
    whole = {}
    for name in parts[0]:   # rows one expert after the other, weights by expert
        values = [p[name] for p in parts]
        whole[name] = None if values[0] is None else torch.stack(values) if name.startswith("grad_w") else torch.cat(values)
    return whole["y"] if case["op"].startswith("fp8") else whole


def _exact_product(x, x_scales, w, w_scales):
    """Rows times one expert's weights, both in fp8, block by block."""
    x_scales = torch.ldexp(torch.ones_like(x_scales, dtype=torch.float64), x_scales.int() - 127) if x_scales.dtype == torch.uint8 \
        else x_scales.double()
    which = torch.arange(w.shape[0], device="cuda") // _BLOCK
    w = (w.double().unflatten(1, (-1, _BLOCK)) * w_scales.double()[which][..., None]).flatten(1)
    return (x.double().unflatten(1, (-1, _BLOCK)) * x_scales[..., None]).flatten(1) @ w.t()


def _exact_gate(y):
    half = y.shape[1] // 2
    return torch.nn.functional.silu(y[:, :half]) * y[:, half:]


def _exact_fp8(s, e, at):
    y = _exact_product(s["x"][at], s["x_scales"][at], s["weights"][e], s["weight_scales"][e])
    return {"y": _exact_gate(y) if s["case"]["swiglu"] else y}


def _exact_fp8_ffn(s, e, at):
    act = _exact_gate(_exact_product(s["x"][at], s["x_scales"][at], s["w_gate_up"][e], s["gate_up_scales"][e]))
    act = act.unflatten(1, (-1, _BLOCK))
    scales = (act.abs().amax(2) / _E4M3_MAX).float()   # a scale is an fp32 number
    codes = (act / scales.double().clamp(min=1e-300)[..., None]).clamp(-_E4M3_MAX, _E4M3_MAX)
    codes = codes.float().to(torch.float8_e4m3fn).flatten(1)
    return {"y": _exact_product(codes, scales, s["w_down"][e], s["down_scales"][e])}


def _exact_ffn(s, e, at):
    gate_up = s["x"][at].double() @ s["w_gate_up"][e].double().t()
    act = _exact_gate(gate_up)
    return {"y": act @ s["w_down"][e].double().t(), "act": act, "gate_up": gate_up if s["case"]["save"] else None}


def _exact_ffn_backward(s, e, at):
    gate_up = s["gate_up"][at].double().requires_grad_()
    grad_y = s["grad_y"][at].double()
    _exact_gate(gate_up).backward(grad_y @ s["w_down"][e].double())
    return {"grad_x": gate_up.grad @ s["w_gate_up"][e].double(), "grad_gate_up": gate_up.grad,
            "grad_w_gate_up": gate_up.grad.t() @ s["x"][at].double(), "grad_w_down": grad_y.t() @ s["act"][at].double()}


_EXACT = {"fp8": _exact_fp8, "fp8_ffn": _exact_fp8_ffn, "ffn": _exact_ffn, "ffn_backward": _exact_ffn_backward}
