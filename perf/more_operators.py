"""What the operators around the expert and projection products are measured on.

  route     which experts a token takes, by scores: logits l = x W^T, scores s = softmax(l) or
            sigmoid(l); chosen by s + bias among the best groups of experts, weighted by s
            (renormalized, scaled)
  norm      the residual stream around a block: x' = x + scale * gate * post(y), h = pre(x'),
            post and pre an RMS or a layer norm or nothing; h in 16 or 32 bits or in MXFP4
            (4-bit e2m1 codes with one power of two per 32 columns)
  adapters  low-rank adapters of many requests beside a shared projection's output y:
            y'[t] = y[t] + c[a] * B[a] (A[a] x[t]) for the adapter a of token t (or none)

listed() names the cases, prepare() makes a case's inputs, run() is one call of the operator
(in its plain form, or through the framework where `own` is set), exact() the result in 64
bits, work() the bytes and operations that the call cannot do without."""
import math

import numpy as np
import torch

own = False

BLOCK = 32          # columns that share one scale of the 4-bit form
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of one request: sigmoid scores, balance bias, the best 4 of 8 groups; latency
        {"name": "route T=1 sigmoid groups", "op": "route", "t": 1, "h": 2048, "e": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5},
        # a batch of decoding requests, softmax scores without groups
        {"name": "route T=37 softmax", "op": "route", "t": 37, "h": 2048, "e": 256, "k": 8,
         "score": "softmax", "bias": False, "groups": 1, "kept": 1, "best": 1, "renorm": True, "scale": 1.0},
        # a ragged prompt through a small router, groups ranked by their best expert, weights as they are
        {"name": "route T=300 softmax groups", "op": "route", "t": 300, "h": 1024, "e": 64, "k": 6,
         "score": "softmax", "bias": False, "groups": 8, "kept": 3, "best": 1, "renorm": False, "scale": 16.0},
        # a long prompt
        {"name": "route T=4096 sigmoid groups", "op": "route", "t": 4096, "h": 2048, "e": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "kept": 4, "best": 2, "renorm": True, "scale": 2.5},
        # one token between two blocks: the last one's output added, the next one's input normed; latency
        {"name": "norm T=1 bf16", "op": "norm", "t": 1, "h": 2048, "x": "bf16", "y": "bf16", "to": "bf16",
         "post": "none", "pre": "rms", "gate": "none", "scale": 1.0},
        # a ragged prompt on its way into a 4-bit product, the block's output gated per channel
        {"name": "norm T=300 gate mx4", "op": "norm", "t": 300, "h": 2048, "x": "bf16", "y": "bf16", "to": "mx4",
         "post": "none", "pre": "rms", "gate": "channel", "scale": 1.0},
        # a long prompt with norms on both sides of the block and a scaled residual: bandwidth
        {"name": "norm T=4096 sandwich", "op": "norm", "t": 4096, "h": 2048, "x": "bf16", "y": "bf16", "to": "bf16",
         "post": "rms", "pre": "rms", "gate": "none", "scale": 0.22},
        # a 32-bit residual stream of an odd width, layer norm, a gate for each value
        {"name": "norm T=2050 layer fp32", "op": "norm", "t": 2050, "h": 1056, "x": "fp32", "y": "bf16", "to": "fp16",
         "post": "none", "pre": "layer", "gate": "full", "scale": 1.0},
        # one token of one request beside a square projection: latency
        {"name": "adapters T=1 r=16", "op": "adapters", "t": 1, "k": 2048, "n": 2048, "count": 8, "rank": 16,
         "mixed": False, "y": "bf16", "packed": False, "none": 0.0},
        # a batch of decoding requests with adapters of several ranks, some requests without one
        {"name": "adapters T=37 mixed", "op": "adapters", "t": 37, "k": 2048, "n": 8192, "count": 16, "rank": 64,
         "mixed": True, "y": "bf16", "packed": False, "none": 0.2},
        # every request with an adapter of its own, through a long reduction: bandwidth
        {"name": "adapters T=64 own r=64", "op": "adapters", "t": 64, "k": 8192, "n": 2048, "count": 64, "rank": 64,
         "mixed": False, "y": "bf16", "packed": False, "none": 0.0},
        # packed prompts of several requests beside a wide projection
        {"name": "adapters T=4096 packed", "op": "adapters", "t": 4096, "k": 2048, "n": 8192, "count": 6, "rank": 32,
         "mixed": True, "y": "bf16", "packed": True, "none": 0.1},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["route", "norm", "adapters"])
    if op == "route":
        e = rng.choice([8, 16, 48, 64, 128, 160, 256])
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if e % g == 0 and e // g >= 4])
        kept = rng.randint(1, groups)
        room = kept * (e // groups)
        h = 64 * rng.randint(4, 32)
        return {"op": op, "t": _log(rng, 1, 4096), "h": h, "e": e, "k": rng.randint(1, min(8, room)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "kept": kept, "best": rng.choice([1, 2]), "renorm": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5])}
    if op == "norm":
        to = rng.choice(["bf16", "bf16", "fp16", "fp32", "mx4"])
        h = 32 * _log(rng, 2, 256)
        return {"op": op, "t": _log(rng, 1, min(4096, 4096 * 2048 // h)), "h": h, "x": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                "y": rng.choice(["bf16", "fp16", "fp32"]), "to": to, "post": rng.choice(["none", "rms", "layer"]),
                "pre": rng.choice(["rms", "rms", "layer"]), "gate": rng.choice(["none", "channel", "token", "full"]),
                "scale": rng.choice([1.0, 0.22])}
    k, n = 8 * _log(rng, 16, 1024), _log(rng, 64, 8192)
    count, rank, y = _log(rng, 1, 32), 8 * rng.randint(1, 8), rng.choice(["bf16", "bf16", "fp32"])
    room = 1.4e8 - 2 * count * rank * (k + n)  # bytes of x and y that keep a case below the largest listed one
    t = _log(rng, 1, min(4096, int(room / (2 * k + (4 if y == "bf16" else 8) * n))))
    return {"op": op, "t": t, "k": k, "n": n, "count": count, "rank": rank, "mixed": rng.random() < 0.5,
            "y": y, "packed": t > 64, "none": rng.choice([0.0, 0.2])}


# ------------------------------------------------------------------ inputs

def _gen(seed, *parts):
    g = torch.Generator(device="cuda")
    h = seed
    for p in parts:
        h = (h * 1000003 + int(p)) % (1 << 62)
    g.manual_seed(h)
    return g


def _randn(shape, seed, *tag):
    return torch.randn(shape, generator=_gen(seed, *tag), device="cuda")


def _route_inputs(c, seed):
    router = _randn((c["e"], c["h"]), seed, 1) * (2.2 * c["h"] ** -0.5)
    bias = _randn((c["e"],), seed, 2) * 0.05 if c["bias"] else None
    x = _randn((c["t"], c["h"]), seed, 3).to(torch.bfloat16)
    for attempt in range(60):  # a token whose choices are almost tied is drawn again
        logits = x.double() @ router.double().T
        s = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
        by = s if bias is None else s + bias.double()
        tied = torch.zeros(c["t"], dtype=torch.bool, device="cuda")
        if c["kept"] < c["groups"]:
            parts = by.reshape(c["t"], c["groups"], -1)
            value = torch.sort(parts, dim=2, descending=True).values[:, :, : c["best"]].sum(dim=2)
            order = torch.sort(value, dim=1, descending=True)
            tied |= order.values[:, c["kept"] - 1] - order.values[:, c["kept"]] < 1e-4 * order.values[:, 0].abs()
            keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order.indices[:, : c["kept"]], True)
            by = torch.where(keep[:, :, None], parts, -math.inf).reshape(c["t"], -1)
        top = torch.sort(by, dim=1, descending=True).values[:, : min(c["k"] + 1, c["e"])]
        gap = top[:, :-1] - top[:, 1:]
        tied |= (gap < 1e-4 * top[:, :-1].abs().clamp_max(0.25)).any(dim=1)
        if not bool(tied.any()):
            break
        x = torch.where(tied[:, None], _randn((c["t"], c["h"]), seed, 4, attempt).to(torch.bfloat16), x)
    return {"case": c, "x": x, "router": router, "bias": bias}


def _norm_inputs(c, seed):
    t, h = c["t"], c["h"]
    x = _randn((t, h), seed, 11) * 2
    big = torch.randint(0, h, (max(1, h // 512),), generator=_gen(seed, 12), device="cuda")
    x[:, big] *= 8.0  # a few columns of a residual stream are much larger than the rest
    shape = {"none": None, "channel": (h,), "token": (t, 1), "full": (t, h)}[c["gate"]]
    s = {"case": c, "x": x.to(DTYPES[c["x"]]), "y": (_randn((t, h), seed, 13) * 0.7).to(DTYPES[c["y"]]),
         "gate": None if shape is None else (1 + 0.3 * _randn(shape, seed, 14)).to(torch.float32 if c["gate"] == "token" else torch.bfloat16)}
    for n, name in enumerate(("post", "pre")):
        s[name + "_w"] = 1 + 0.2 * _randn((h,), seed, 15, n)
        s[name + "_b"] = 0.1 * _randn((h,), seed, 16, n)
    for attempt in range(12 if c["to"] == "mx4" else 0):  # a value on the border of two codes is moved off it
        b = _norm_exact(s)[1].reshape(t, -1, BLOCK)
        top = b.abs().amax(dim=2, keepdim=True)
        q = b.abs() / 2.0 ** (torch.floor(torch.log2(top)) - 2)
        border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device="cuda")
        near = ((q[..., None] / border - 1).abs() < 4e-6).any(dim=3)
        f = torch.frexp(top).mantissa  # 0.5 .. 1
        near |= (b.abs() == top) & ((f - 0.5 < 4e-6) | (1 - f < 4e-6))
        near = near.reshape(t, h)
        if not bool(near.any()):
            break
        # by more than a step of the type, up or down by turns
        step = 1 + (0.02 + 0.005 * attempt) * (1 if attempt % 2 == 0 else -1)
        s["x"] = torch.where(near, s["x"].float() * step + 0.01, s["x"].float()).to(s["x"].dtype)
    return s


def _ids(c, rng):
    """The adapter of each token: requests one after another where packed, else one a token."""
    t, count = c["t"], c["count"]
    if not c["packed"]:
        ids = rng.permutation(count)[:t] if t <= count else rng.integers(0, count, t)
    else:  # prompts of uneven lengths
        share = rng.dirichlet(np.ones(count + 2)) * t
        ends = np.minimum(np.cumsum(np.maximum(share.astype(int), 1)), t)
        ids = np.searchsorted(ends, np.arange(t), side="right") % count
        ids = np.where(rng.random(count)[ids] < c["none"], -1, ids)
        return ids
    return np.where(rng.random(t) < c["none"], -1, ids)


def _ranks(c, rng):
    return rng.integers(1, c["rank"] // 8 + 1, c["count"]) * 8 if c["mixed"] else np.full(c["count"], c["rank"])


def prepare(case, seed):
    c = case
    if c["op"] == "route":
        return _route_inputs(c, seed)
    if c["op"] == "norm":
        return _norm_inputs(c, seed)
    rng = np.random.default_rng([seed, 31])
    put = lambda a: torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()  # noqa: E731
    r, n = c["rank"], c["count"]
    return {"case": c, "x": _randn((c["t"], c["k"]), seed, 21).to(torch.bfloat16),
            "y": _randn((c["t"], c["n"]), seed, 22).to(DTYPES[c["y"]]),
            "a": (_randn((n, r, c["k"]), seed, 23) * c["k"] ** -0.5).to(torch.bfloat16),
            "b": (_randn((n, c["n"], r), seed, 24) * r ** -0.5).to(torch.bfloat16),
            "scale": torch.rand((n,), generator=_gen(seed, 25), device="cuda") + 0.5,
            "ranks": put(_ranks(c, rng)), "ids": put(_ids(c, rng))}


# ------------------------------------------------------------- plain forms

def _plain_route(s):
    c = s["case"]
    logits = torch.matmul(s["x"].float(), s["router"].T)
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        p = torch.exp(logits - logits.amax(dim=1, keepdim=True))
        score = p / p.sum(dim=1, keepdim=True)
    by = score if s["bias"] is None else score + s["bias"]
    if c["kept"] < c["groups"]:
        parts = by.reshape(c["t"], c["groups"], -1)
        value = torch.sort(parts, dim=2, descending=True).values[:, :, : c["best"]].sum(dim=2)
        kept = torch.sort(value, dim=1, descending=True, stable=True).indices[:, : c["kept"]]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, kept, True)
        by = torch.where(keep[:, :, None], parts, -math.inf).reshape(c["t"], -1)
    ids = torch.sort(by, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    weight = torch.gather(score, 1, ids)
    if c["renorm"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    return {"experts": ids.int(), "weights": weight * c["scale"]}


def _normed(v, kind, w, b):
    """v in 32 or 64 bits."""
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-6) * w
    return v + b if kind == "layer" else v


def _codes(h):
    """h [t, columns] replaced by what its 4-bit form stands for: per 32 columns a power of two
    two binades below the largest magnitude, the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times it
    (ties to the even code, those over 6 become 6)."""
    v = h.reshape(h.shape[0], -1, BLOCK)
    top = v.abs().amax(dim=2, keepdim=True)
    unit = torch.where(top > 0, torch.exp2(torch.frexp(top).exponent.to(h.dtype) - 3), torch.ones_like(top))
    q = (v / unit).abs()
    code = (q > 0.25).int() + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=h.dtype, device=h.device)
    return (torch.copysign(table[code], v) * unit).reshape(h.shape)


def _plain_norm(s):
    c = s["case"]
    wide = torch.float64 if c["to"] == "mx4" else torch.float32  # codes: values next to a border
    w = {n: s[n].to(wide) for n in ("post_w", "post_b", "pre_w", "pre_b")}
    d = _normed(s["y"].to(wide), c["post"], w["post_w"], w["post_b"])
    if s["gate"] is not None:
        d = d * s["gate"].to(wide)
    x = s["x"].to(wide) + c["scale"] * d
    h = _normed(x, c["pre"], w["pre_w"], w["pre_b"])
    h = _codes(h).to(torch.bfloat16) if c["to"] == "mx4" else h.to(DTYPES[c["to"]])
    return {"x": x.to(s["x"].dtype), "h": h}


def _plain_adapters(s):
    c, n, r = s["case"], s["case"]["count"], s["case"]["rank"]
    # every adapter on every token, zeroed where it is not the token's
    v = torch.matmul(s["x"].float(), s["a"].float().reshape(n * r, -1).T).reshape(-1, n, r)
    mine = s["ids"][:, None] == torch.arange(n, device="cuda")
    used = torch.arange(r, device="cuda") < s["ranks"][:, None]
    v = torch.where(mine[:, :, None] & used, v * s["scale"][:, None], 0.0)
    d = torch.matmul(v.reshape(-1, n * r), s["b"].float().transpose(1, 2).reshape(n * r, -1))
    return (s["y"].float() + d).to(s["y"].dtype)


# ----------------------------------------------------------- the framework

def _own_route(s):
    import quantized_sparse_moe_gb300 as q
    c = s["case"]
    if "plan" not in s:
        s["plan"] = q.MoERouter(s["router"], c["k"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                groups_kept=c["kept"], group_best=c["best"], renormalize=c["renorm"], scale=c["scale"])
    ids, weights = q.moe_route_scores(s["x"], s["plan"])
    return {"experts": ids, "weights": weights}


def _own_norm(s):
    import quantized_sparse_moe_gb300 as q
    c = s["case"]
    if "plan" not in s:
        norm = lambda n: None if c[n] == "none" else q.Norm(s[n + "_w"], s[n + "_b"] if c[n] == "layer" else None, kind=c[n], eps=1e-6)  # noqa: E731
        s["plan"] = q.ResidualNorm(c["h"], pre=norm("pre"), post=norm("post"), scale=c["scale"])
        s["h"] = q.Mx4Tensor.empty(c["t"], c["h"]) if c["to"] == "mx4" else torch.empty_like(s["x"], dtype=DTYPES[c["to"]])
        s["x_out"] = torch.empty_like(s["x"])  # the buffers that a program keeps
    x, h = s["plan"](s["x"], s["y"], s["gate"], x_out=s["x_out"], h=s["h"])
    return {"x": x, "h": q.mx4_dequantize(h) if c["to"] == "mx4" else h}


def _own_adapters(s):
    import quantized_sparse_moe_gb300 as q
    if "plan" not in s:
        s["plan"] = q.LoraAdapters(s["a"], s["b"], s["scale"], s["ranks"])
    return q.lora_add(s["x"], s["plan"], s["ids"], s["y"])


def run(state):
    op = state["case"]["op"]
    if own:
        return {"route": _own_route, "norm": _own_norm, "adapters": _own_adapters}[op](state)
    return {"route": _plain_route, "norm": _plain_norm, "adapters": _plain_adapters}[op](state)


# -------------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "route":
        return {"bytes": 2 * c["t"] * c["h"] + 4 * c["e"] * c["h"] + 8 * c["t"] * c["k"], "flops": 2 * c["t"] * c["e"] * c["h"]}
    size = {"bf16": 2, "fp16": 2, "fp32": 4, "mx4": 0.5 + 1 / BLOCK}
    if c["op"] == "norm":
        n = c["t"] * c["h"]
        # x, x', y and h, the gate; a 4-bit h is read again and comes back in 16 bits
        each = 2 * size[c["x"]] + size[c["y"]] + size[c["to"]] + (2 + size["mx4"] if c["to"] == "mx4" else 0) + (2 if c["gate"] == "full" else 0)
        return {"bytes": n * each + 8 * c["h"], "flops": 10 * n}
    # the adapters that such a batch touches, drawn once from a fixed seed
    rng = np.random.default_rng(0)
    ranks, ids = _ranks(c, rng), _ids(c, rng)
    used = ids[ids >= 0]
    weights = 2 * float(ranks[np.unique(used)].sum()) * (c["k"] + c["n"])
    return {"bytes": weights + 2 * c["t"] * c["k"] + 2 * size[c["y"]] * c["t"] * c["n"],
            "flops": 2 * float(ranks[used].sum()) * (c["k"] + c["n"]) + c["t"] * c["n"]}


# ------------------------------------------------------------ in 64 bits

def _norm_exact(s):
    """(x', h before its rounding)."""
    c = s["case"]

    def norm(v, which):
        if c[which] == "none":
            return v
        w = s[which + "_w"].double()
        if c[which] == "rms":
            return v * w * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + 1e-6)
        z = (v - v.mean(dim=1, keepdim=True)) * torch.rsqrt(v.var(dim=1, keepdim=True, unbiased=False) + 1e-6)
        return z * w + s[which + "_b"].double()

    gate = 1.0 if s["gate"] is None else s["gate"].double()
    x = s["x"].double() + c["scale"] * gate * norm(s["y"].double(), "post")
    return x, norm(x, "pre")


def _nearest(h):
    """h in 64 bits, each value replaced by what its MXFP4 form stands for."""
    b = h.reshape(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    unit = 2.0 ** (torch.floor(torch.log2(top.clamp_min(1e-300))) - 2)
    q = b / unit
    step = 2.0 ** (torch.floor(torch.log2(q.abs().clamp_min(1e-300))).clamp(0, 2) - 1)
    return ((torch.round(q / step) * step).clamp(-6, 6) * unit).reshape(h.shape)


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    if c["op"] == "norm":
        x, h = _norm_exact(s)
        return {"x": x, "h": _nearest(h) if c["to"] == "mx4" else h}
    if c["op"] == "adapters":
        y, ids, ranks = s["y"].double(), s["ids"], s["ranks"].tolist()
        for n in range(c["count"]):
            t = torch.nonzero(ids == n)[:, 0]
            if len(t):
                a, b = s["a"][n, : ranks[n]].double(), s["b"][n, :, : ranks[n]].double()
                y[t] += s["scale"][n].double() * ((s["x"][t].double() @ a.T) @ b.T)
        return y
    logits = s["x"].double() @ s["router"].double().T
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    by = score if s["bias"] is None else score + s["bias"].double()
    group = torch.arange(c["e"], device="cuda") // (c["e"] // c["groups"])
    value = torch.stack([torch.topk(by[:, group == g], c["best"], dim=1).values.sum(dim=1) for g in range(c["groups"])], dim=1)
    for g in range(c["groups"]):  # a group is kept when fewer than `kept` are better
        better = (value > value[:, g : g + 1]).sum(dim=1)
        by[:, group == g] = torch.where((better < c["kept"])[:, None], by[:, group == g], -math.inf)
    weight = torch.gather(score, 1, torch.topk(by, c["k"], dim=1).indices)
    if c["renorm"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    return {"experts": None, "weights": weight * c["scale"]}
