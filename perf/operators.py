"""The decode-layer operators as a user calls them, each beside its plain form.

Five calls that stand around the MoE dispatch and combine of this library in a
transformer layer: the router that picks each token's experts (forward and
backward), the append of rotated keys and values to a paged cache, the
attention of one new token over that cache, and the experts' products with
4-bit weights. `run` computes them with elementary torch operations in 32 bits
where `own` is false, and through the library where it is true.
"""
from __future__ import annotations

import math

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}


# ------------------------------------------------------------------ cases

def _router(name, T, E, K, dtype="fp32", score="softmax", renorm=True, scale=1.0, groups=1, keep=1, masked=0.0,
            backward=False):
    c = {"op": "router_backward" if backward else "router", "T": T, "E": E, "K": K, "dtype": dtype, "score": score,
         "renorm": renorm, "scale": scale, "groups": groups, "keep": keep, "masked": masked}
    return c if name is None else {"name": name, **c}


def _append(name, T, heads, kv_heads, dim, page, pages, dtype="bf16", cache="bf16", rotary=None, interleaved=False,
            prefill=False):
    c = {"op": "append", "T": T, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "pages": pages,
         "dtype": dtype, "cache": cache, "rotary": dim if rotary is None else rotary, "interleaved": interleaved,
         "prefill": prefill}
    return c if name is None else {"name": name, **c}


def _attention(name, B, length, heads, kv_heads, dim, page, dtype="bf16", cache="bf16", ragged=False, heads_first=False,
               window=0):
    c = {"op": "attention", "B": B, "length": length, "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page,
         "dtype": dtype, "cache": cache, "ragged": ragged, "heads_first": heads_first, "window": window}
    return c if name is None else {"name": name, **c}


def _experts(name, T, K, E, inner, outer, group, dtype="bf16", zeros=False, swiglu=False):
    c = {"op": "experts", "T": T, "K": K, "E": E, "inner": inner, "outer": outer, "group": group, "dtype": dtype,
         "zeros": zeros, "swiglu": swiglu}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one decode step's routing: 256 sequences, 256 experts, top 8 (launch-bound)
        _router("router decode", 256, 256, 8),
        # routing of a long prompt, bf16 logits as a bf16 gate leaves them (many ties), experts in
        # groups of which each token may use some, a few experts out of service
        _router("router prompt groups", 16384, 64, 6, dtype="bf16", score="sigmoid", scale=2.5, groups=8, keep=4,
                masked=0.05),
        # the gradient of the top-k weights back to the logits, one training micro-batch
        _router("router backward", 8192, 256, 8, renorm=False, backward=True),
        # one decode step of 256 sequences: one row each to pages all over the cache
        _append("append decode", 256, 32, 8, 128, 16, 1024),
        # a prompt's keys and values into an fp8 cache, many query heads rotated on the way
        _append("append prompt e4m3", 8192, 64, 8, 128, 64, 256, cache="e4m3", prefill=True),
        # one chat sequence just begun (latency alone)
        _attention("attention short", 1, 129, 32, 8, 128, 16),
        # a serving batch: sequences of every length, some just begun
        _attention("attention batch", 64, 4096, 64, 8, 128, 64, ragged=True),
        # one long document: a single sequence has to fill the GPU
        _attention("attention long", 1, 131071, 32, 8, 128, 64),
        # a large batch over an fp8 cache laid out head by head, long contexts
        _attention("attention e4m3 batch", 128, 8192, 64, 8, 128, 64, cache="e4m3", ragged=True, heads_first=True),
        # a dense projection by 4-bit weights with zero points, a few sequences
        _experts("projection", 4, 1, 1, 4096, 4096, 128, dtype="fp16", zeros=True),
        # one token's eight experts, gate and up projection with the activation
        _experts("experts one token", 1, 8, 256, 7168, 4096, 128, swiglu=True),
        # a decode step of 256 tokens: every expert of the layer is read
        _experts("experts decode", 256, 8, 256, 7168, 4096, 128, swiglu=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("router", "router_backward", "append", "attention", "attention", "experts", "experts"))
    if op in ("router", "router_backward"):
        groups = rng.choice((1, 1, 2, 4, 8)) if op == "router" else 1
        E = groups * rng.choice((5, 8, 16, 20, 32)) if groups > 1 else rng.choice((8, 60, 64, 128, 160, 256, 384))
        keep = rng.randint(1, groups)
        K = rng.randint(1, min(10, keep * (E // groups)))
        return _router(None, _log(rng, 1, 16384 if E <= 128 else 8192), E, K, rng.choice(("fp32", "bf16", "fp16")),
                       rng.choice(("softmax", "sigmoid")), rng.random() < 0.5, rng.choice((1.0, 2.5)), groups, keep,
                       rng.choice((0.0, 0.05)), op == "router_backward")
    if op == "append":
        dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        page = rng.choice((1, 16, 24, 64, 256))
        T = _log(rng, 1, 8192 * 8 * 128 // (kv_heads * max(dim, 128)) if kv_heads == 8 else 8192)
        heads = min(64 * 128 // max(dim, 128), kv_heads * rng.choice((1, 3, 4, 8)))
        dtype = rng.choice(("bf16", "fp16"))
        return _append(None, T, heads, kv_heads, dim, page, -(-T // page) + rng.randint(1, 64), dtype,
                       rng.choice((dtype, "e4m3")), rng.choice((dim, dim // 2)), rng.random() < 0.5, rng.random() < 0.5)
    if op == "attention":
        B = _log(rng, 1, 128)
        dim = rng.choice((64, 80, 96, 128, 256))
        kv_heads = rng.choice((1, 2, 4, 8))
        most = min(131072, 96 * 4096 * 8 * 128 // (B * kv_heads * dim))
        length = _log(rng, 1, most)
        dtype = rng.choice(("bf16", "fp16"))
        return _attention(None, B, length, kv_heads * rng.choice((1, 2, 3, 4, 7, 8, 16)), kv_heads, dim,
                          rng.choice((1, 16, 24, 64, 256)), dtype, rng.choice((dtype, dtype, "e4m3")),
                          rng.random() < 0.7, rng.random() < 0.5, rng.choice((0, 0, 0, 777)))
    E = rng.choice((1, 1, 8, 32, 64))
    K = rng.randint(1, min(8, E))
    group = rng.choice((32, 64, 128))
    inner = group * rng.randint(max(1, 256 // group), 4096 // group)
    swiglu = rng.random() < 0.5
    outer = _log(rng, 32, 4096) * (2 if swiglu else 1)
    return _experts(None, _log(rng, 1, 128), K, E, inner, outer, group, rng.choice(("bf16", "fp16")),
                    rng.random() < 0.5, swiglu)


def work(case):
    op = case["op"]
    if op == "router":
        T, E, K = case["T"], case["E"], case["K"]
        return {"bytes": T * E * _BYTES[case["dtype"]] + T * K * 12, "flops": 4 * T * E}
    if op == "router_backward":
        T, E, K = case["T"], case["E"], case["K"]
        return {"bytes": 2 * T * E * _BYTES[case["dtype"]] + T * K * 12, "flops": 6 * T * E}
    if op == "append":
        T, d = case["T"], case["dim"]
        row = 2 * (2 * case["heads"] + 2 * case["kv_heads"]) * d + 2 * case["kv_heads"] * d * _BYTES[case["cache"]]
        return {"bytes": T * (row + 16 + 4 * case["rotary"]),
                "flops": 3 * T * (case["heads"] + case["kv_heads"]) * case["rotary"]}
    if op == "attention":
        B, h, g, d = case["B"], case["heads"], case["kv_heads"], case["dim"]
        mean = case["length"] / 2 if case["ragged"] else case["length"]
        if case["window"]:
            w, n = case["window"], case["length"]
            mean = min(w, n) if not case["ragged"] else (n / 2 if n <= w else w - w * w / (2 * n))
        return {"bytes": B * (2 * mean * g * d * _BYTES[case["cache"]] + 4 * h * d + 4 * h + 4 * mean / case["page"]),
                "flops": 4 * B * h * d * mean}
    T, K, E, i, o = case["T"], case["K"], case["E"], case["inner"], case["outer"]
    used = E * (1 - (1 - K / E) ** T)
    return {"bytes": used * o * (i // 2 + i // case["group"] * (3 if case["zeros"] else 2))
            + T * K * 2 * (i + (o // 2 if case["swiglu"] else o)) + 4 * (E + 1),
            "flops": 2 * T * K * o * i}


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    made = {"router": _prepare_router, "router_backward": _prepare_router, "append": _prepare_append,
            "attention": _prepare_attention, "experts": _prepare_experts}[op](case, g)
    return {"case": case, **made}


def _prepare_router(case, g):
    T, E, K, dt = case["T"], case["E"], case["K"], _DTYPES[case["dtype"]]
    logits = (2 * torch.randn(T, E, device="cuda", generator=g)).to(dt)
    if case["masked"]:
        logits[torch.rand(T, E, device="cuda", generator=g) < case["masked"]] = -math.inf
    s = {"logits": logits, "topk_idx": torch.empty(T, K, dtype=torch.int64, device="cuda"),
         "topk_weights": torch.empty(T, K, device="cuda")}
    if case["op"] == "router_backward":
        s["topk_idx"] = _select(logits.float(), case)
        s["grad_weights"] = torch.randn(T, K, device="cuda", generator=g)
        s["grad_logits"] = torch.empty_like(logits)
    return s


def _prepare_append(case, g):
    T, h, n, d, page, pages = (case[k] for k in ("T", "heads", "kv_heads", "dim", "page", "pages"))
    dt, ct, most = _DTYPES[case["dtype"]], _DTYPES[case["cache"]], max(8192, T)
    qkv = torch.randn(T, (h + 2 * n) * d, device="cuda", generator=g).to(dt)   # one fused projection's output
    q, k, v = qkv.split((h * d, n * d, n * d), dim=1)
    if case["prefill"]:   # the positions of one prompt, on pages in an order of their own
        positions = torch.arange(T, device="cuda")
        order = torch.randperm(pages, device="cuda", generator=g)
        slots = order[positions // page] * page + positions % page
    else:                 # one token of each of T sequences
        positions = torch.randint(0, most, (T,), device="cuda", generator=g)
        slots = torch.randperm(pages * page, device="cuda", generator=g)[:T]
    half = case["rotary"] // 2
    angle = torch.arange(most, device="cuda")[:, None] * 10000.0 ** (-torch.arange(half, device="cuda") / half)
    caches = [torch.randn(pages, page, n, d, device="cuda", generator=g).to(ct) for _ in range(2)]
    return {"q": q.view(T, h, d), "k": k.view(T, n, d), "v": v.view(T, n, d), "positions": positions, "slots": slots,
            "cos_sin": torch.cat((angle.cos(), angle.sin()), 1), "q_out": torch.empty(T, h, d, dtype=dt, device="cuda"),
            "k_cache": caches[0], "v_cache": caches[1], "k_scale": 0.02 if case["cache"] == "e4m3" else 1.0,
            "v_scale": 0.03 if case["cache"] == "e4m3" else 1.0}


def _prepare_attention(case, g):
    B, n, h, d, page, length = (case[k] for k in ("B", "kv_heads", "heads", "dim", "page", "length"))
    dt, ct = _DTYPES[case["dtype"]], _DTYPES[case["cache"]]
    lens = torch.full((B,), length, dtype=torch.int32, device="cuda")
    if case["ragged"]:
        lens = torch.randint(0, length + 1, (B,), dtype=torch.int32, device="cuda", generator=g)
    width = -(-length // page)
    pages = B * width + 3
    shape = (pages, n, page, d) if case["heads_first"] else (pages, page, n, d)
    caches = []
    for _ in range(2):   # one large draw at a time: the largest caches have a thousand million values
        c = torch.empty(shape, dtype=ct, device="cuda")
        for part in c.split(-(-pages // 16)):
            part.copy_(torch.randn(part.shape, device="cuda", generator=g))
        caches.append(c.transpose(1, 2) if case["heads_first"] else c)
    table = torch.randperm(pages, device="cuda", generator=g)[:B * width].to(torch.int32).view(B, width)
    table[torch.arange(width, device="cuda")[None] * page >= lens[:, None]] = -1   # no page behind the end
    return {"q": (1.5 * torch.randn(B, h, d, device="cuda", generator=g)).to(dt), "k_cache": caches[0],
            "v_cache": caches[1], "block_table": table, "seq_lens": lens,
            "out": torch.empty(B, h, d, dtype=dt, device="cuda"), "lse": torch.empty(B, h, device="cuda"),
            "scale": 1 / math.sqrt(d), "k_scale": 0.9 if case["cache"] == "e4m3" else 1.0,
            "v_scale": 1.1 if case["cache"] == "e4m3" else 1.0}


def _prepare_experts(case, g):
    T, K, E, i, o, dt = (case[k] for k in ("T", "K", "E", "inner", "outer", "dtype"))
    dt, groups = _DTYPES[dt], i // case["group"]
    chosen = torch.rand(T, E, device="cuda", generator=g).argsort(1)[:, :K].reshape(-1)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.bincount(chosen, minlength=E).cumsum(0)
    weights = torch.empty(E, o, i // 2, dtype=torch.uint8, device="cuda")
    for part in weights.split(-(-E // 16)):
        part.random_(0, 256, generator=g)
    scales = (torch.rand(E, groups, o, device="cuda", generator=g) + 0.5).mul_(1 / (4.6 * math.sqrt(i))).to(dt)
    zeros = torch.randint(6, 11, (E, groups, o), dtype=torch.uint8, device="cuda", generator=g) if case["zeros"] else None
    return {"x": torch.randn(T * K, i, device="cuda", generator=g).to(dt), "weights": weights, "scales": scales,
            "zeros": zeros, "expert_offsets": offsets,
            "y": torch.empty(T * K, o // 2 if case["swiglu"] else o, dtype=dt, device="cuda")}


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"router": _own_router, "router_backward": _own_router_backward, "append": _own_append,
                "attention": _own_attention, "experts": _own_experts}[op](s)
    return {"router": _plain_router, "router_backward": _plain_router_backward, "append": _plain_append,
            "attention": _plain_attention, "experts": _plain_experts}[op](s)


def _own_router(s):
    import combine_get_dispatch_layout_gb300 as ep
    c = s["case"]
    ep.ep_router_topk(s["logits"], s["topk_idx"], s["topk_weights"],
                      score=ep.EP_SCORE_SIGMOID if c["score"] == "sigmoid" else ep.EP_SCORE_SOFTMAX,
                      renormalize=c["renorm"], scale=c["scale"], num_groups=c["groups"], topk_groups=c["keep"])
    return s["topk_idx"], s["topk_weights"]


def _own_router_backward(s):
    import combine_get_dispatch_layout_gb300 as ep
    c = s["case"]
    ep.ep_router_topk_backward(s["logits"], s["topk_idx"], s["grad_weights"], s["grad_logits"],
                               score=ep.EP_SCORE_SIGMOID if c["score"] == "sigmoid" else ep.EP_SCORE_SOFTMAX,
                               renormalize=c["renorm"], scale=c["scale"])
    return s["grad_logits"]


def _own_append(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_kv_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cos_sin"], s["q_out"], s["k_cache"],
                    s["v_cache"], interleaved=s["case"]["interleaved"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_attention(s):
    import combine_get_dispatch_layout_gb300 as ep
    if "workspace" not in s:   # scratch that a serving program keeps beside its cache
        size = ep.ep_paged_attention_workspace(s["q"], s["k_cache"], s["block_table"])
        s["workspace"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    ep.ep_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], s["out"], s["workspace"],
                          lse=s["lse"], scale=s["scale"], window=s["case"]["window"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"])
    return s["out"], s["lse"]


def _own_experts(s):
    import combine_get_dispatch_layout_gb300 as ep
    ep.ep_expert_w4(s["x"], s["weights"], s["scales"], s["y"], expert_offsets=s["expert_offsets"], zeros=s["zeros"],
                    activation=ep.EP_ACT_SWIGLU if s["case"]["swiglu"] else ep.EP_ACT_NONE)
    return s["y"]


def _select(l, case):
    """Each row's K largest logits, the largest first, equal ones by index; -1 where all that is left is masked."""
    if case["groups"] > 1:
        T, E = l.shape
        best = l.view(T, case["groups"], -1).amax(2)
        first = best.sort(dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        allowed = torch.zeros_like(best, dtype=torch.bool).scatter_(1, first, True)
        l = torch.where(allowed.repeat_interleave(E // case["groups"], 1), l, -math.inf)
    values, idx = l.sort(dim=1, descending=True, stable=True)
    return torch.where(values == -math.inf, -1, idx)[:, :case["K"]]


def _plain_router(s):
    c, l = s["case"], s["logits"].float()
    idx = _select(l, c)
    p = 1 / (1 + torch.exp(-l)) if c["score"] == "sigmoid" else _softmax(l)
    w = torch.where(idx >= 0, p.gather(1, idx.clamp(min=0)), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return idx, w * c["scale"]


def _softmax(l):
    e = torch.exp(l - l.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_router_backward(s):
    c, l = s["case"], s["logits"].float()
    idx = s["topk_idx"].clamp(min=0)
    taken = s["topk_idx"] >= 0
    g = torch.where(taken, s["grad_weights"], 0.0) * c["scale"]
    p = 1 / (1 + torch.exp(-l)) if c["score"] == "sigmoid" else _softmax(l)
    if c["renorm"]:
        q = torch.where(taken, p.gather(1, idx), 0.0)
        q = q / q.sum(1, keepdim=True)
        d = q * (g - (g * q).sum(1, keepdim=True))
        if c["score"] == "sigmoid":
            d = d * (1 - p.gather(1, idx))
        grad = torch.zeros_like(l).scatter_add_(1, idx, d)
    else:
        dense = torch.zeros_like(l).scatter_add_(1, idx, g)
        grad = dense * p * (1 - p) if c["score"] == "sigmoid" else p * (dense - (dense * p).sum(1, keepdim=True))
    return grad.to(s["logits"].dtype)


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[1] values of each head turned by pairs, the rest as they are."""
    half = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = turned[..., :half], turned[..., half:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, rest), -1)


def _stored(x, cache):
    if cache.dtype == torch.float8_e4m3fn:
        return x.clamp(-448.0, 448.0).to(cache.dtype).view(torch.uint8)
    return x.to(cache.dtype)


def _plain_append(s):
    c = s["case"]
    cos, sin = s["cos_sin"][s["positions"]].chunk(2, 1)
    q = _rotate(s["q"].float(), cos, sin, c["interleaved"]).to(s["q_out"].dtype)
    k = _rotate(s["k"].float(), cos, sin, c["interleaved"])
    for x, scale, cache in ((k, s["k_scale"], s["k_cache"]), (s["v"].float(), s["v_scale"], s["v_cache"])):
        flat = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
        flat.view(-1, *cache.shape[2:])[s["slots"]] = _stored(x / scale, cache)
    return q, s["k_cache"], s["v_cache"]


def _plain_attention(s):
    c, q = s["case"], s["q"].float()
    B, h, d = q.shape
    n = c["kv_heads"]
    at = torch.arange(c["length"], device="cuda")
    page = s["block_table"][:, at // c["page"]].clamp(min=0).long()
    k = s["k_cache"][page, at % c["page"]].float().transpose(1, 2)           # [B, n, length, d]
    scores = (q.view(B, n, h // n, d) @ k.transpose(2, 3)) * (s["scale"] * s["k_scale"])
    del k
    lens = s["seq_lens"].long()[:, None]
    seen = at < lens
    if c["window"]:
        seen &= at >= lens - c["window"]
    scores = torch.where(seen[:, None, None], scores, -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    v = s["v_cache"][page, at % c["page"]].float().transpose(1, 2)
    out = (p / torch.where(total > 0, total, 1.0)) @ v * s["v_scale"]
    lse = (top + torch.log(total)).view(B, h)
    return out.view(B, h, d).to(s["out"].dtype), lse


def _plain_experts(s):
    c, x, offsets = s["case"], s["x"].float(), s["expert_offsets"].long()
    counts = offsets[1:] - offsets[:-1]
    used = counts.nonzero()[:, 0]
    code = s["weights"][used]
    n, o, i = code.shape[0], c["outer"], c["inner"]
    code = torch.stack((code & 15, code >> 4), -1)
    w = code.view(n, o, i // c["group"], c["group"]).float()
    del code
    w -= 8.0 if s["zeros"] is None else s["zeros"][used].float().transpose(1, 2)[..., None]
    w *= s["scales"][used].float().transpose(1, 2)[..., None]
    most = torch.arange(int(counts.max()), device="cuda")
    rows = offsets[used][:, None] + most
    real = most < counts[used][:, None]
    y = x[rows.clamp(max=x.shape[0] - 1)] @ w.view(n, o, i).transpose(1, 2)  # [n, most, o]
    if c["swiglu"]:
        gate, up = y.chunk(2, 2)
        y = gate / (1 + torch.exp(-gate)) * up
    return y[real].to(s["x"].dtype)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"router": _exact_router, "router_backward": _exact_router_backward, "append": _exact_append,
            "attention": _exact_attention, "experts": _exact_experts}[case["op"]](s)


def _exact_router(s):
    c, l = s["case"], s["logits"].double()
    idx = _select(s["logits"].float(), c)
    chosen = l.gather(1, idx.clamp(min=0)).masked_fill(idx < 0, -math.inf)
    if c["score"] == "sigmoid":
        w = torch.sigmoid(chosen)
        w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    else:
        w = torch.exp(chosen - torch.logsumexp(chosen if c["renorm"] else l, 1, keepdim=True))
    return None, w * c["scale"]


def _exact_router_backward(s):
    c = s["case"]
    l = s["logits"].double().requires_grad_()
    idx = s["topk_idx"]
    p = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    w = p.gather(1, idx.clamp(min=0)) * (idx >= 0)
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    (w * c["scale"] * s["grad_weights"].double()).sum().backward()
    return l.grad


def _exact_append(s):
    c = s["case"]
    half = c["rotary"] // 2
    table = s["cos_sin"].double()[s["positions"]]
    turn = torch.complex(table[:, :half], table[:, half:])[:, None]
    first = torch.arange(half, device="cuda") * (2 if c["interleaved"] else 1)
    second = first + (1 if c["interleaved"] else half)

    def turned(x):
        x = x.double()
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    caches = []
    for x, scale, cache in ((turned(s["k"]), s["k_scale"], s["k_cache"]), (s["v"].double(), s["v_scale"], s["v_cache"])):
        x = x / scale
        x = x.clamp(-448, 448) if c["cache"] == "e4m3" else x
        full = cache.double()
        full[s["slots"] // c["page"], s["slots"] % c["page"]] = x
        caches.append(full)
    return turned(s["q"]), caches[0], caches[1]


def _exact_attention(s):
    c, q = s["case"], s["q"].double()
    n = c["kv_heads"]
    out, lse = torch.zeros_like(q), torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["seq_lens"].tolist()):
        low = max(0, length - c["window"]) if c["window"] else 0
        if length == low:
            continue
        at = torch.arange(low, length, device="cuda")
        page = s["block_table"][b].long()[at // c["page"]]
        k, v = (s[m][page, at % c["page"]].double() for m in ("k_cache", "v_cache"))   # [keys, n, d]
        heads = q[b].view(n, -1, c["dim"])
        t = torch.einsum("ngd,knd->ngk", heads, k) * (s["scale"] * s["k_scale"])
        lse[b] = torch.logsumexp(t, 2).view(-1)
        out[b] = (torch.einsum("ngk,knd->ngd", torch.softmax(t, 2), v) * s["v_scale"]).reshape(-1, c["dim"])
    return out, lse


def _exact_experts(s):
    c = s["case"]
    offsets = s["expert_offsets"].tolist()
    parts = []
    for e in range(c["E"]):
        if offsets[e] == offsets[e + 1]:
            continue
        x = s["x"][offsets[e]:offsets[e + 1]].double()
        w = torch.empty(c["outer"], c["inner"], dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = s["weights"][e] & 15, s["weights"][e] >> 4
        spread = lambda t: t[e].double().t().repeat_interleave(c["group"], 1)  # noqa: E731
        w = (w - (8 if s["zeros"] is None else spread(s["zeros"]))) * spread(s["scales"])
        y = x @ w.t()
        if c["swiglu"]:
            half = c["outer"] // 2
            y = torch.nn.functional.silu(y[:, :half]) * y[:, half:]
        parts.append(y)
    return torch.cat(parts)
