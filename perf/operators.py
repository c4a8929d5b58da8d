"""What the MXFP4 operators are measured on.

MXFP4 holds a matrix [rows, cols] as 4-bit floating-point codes (sign, two exponent bits, one
mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two to a byte along the columns, and one power of
two (an 8-bit exponent, 2^(s - 127)) for each block of 32 columns of a row.  Five operators:

  quantize   x -> codes and scales, and back to the values that they stand for
  gemm       y = A W^T with both operands in MXFP4
  gemv       y = x W^T for a few rows of 16-bit x and W in MXFP4
  moe16      a mixture-of-experts layer with MXFP4 weights and 16-bit activations (few tokens)
  moe4       the same layer with the activations quantized to MXFP4 as well (many tokens)

listed() names the cases, prepare() makes a case's inputs, run() is one call of the operator
(in its plain form, or through the framework where `own` is set), exact() the result in 64
bits, work() the bytes and operations that the call cannot do without."""
import math

import numpy as np
import torch

own = False

BLOCK = 32          # columns that share one scale
EXP = 127           # bias of the scale's exponent


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token's hidden state on its way into a 4-bit product: latency alone
        {"name": "quantize 1x2048 bf16", "op": "quantize", "rows": 1, "cols": 2048, "dtype": "bf16"},
        # a prompt's hidden states: bandwidth
        {"name": "quantize 4096x2048 bf16", "op": "quantize", "rows": 4096, "cols": 2048, "dtype": "bf16"},
        # weights on their way into the format, from 32-bit masters, with a ragged size
        {"name": "quantize 2050x1056 fp32", "op": "quantize", "rows": 2050, "cols": 1056, "dtype": "fp32"},
        # a short ragged prompt through an output projection
        {"name": "gemm 300x2048x2048", "op": "gemm", "m": 300, "n": 2048, "k": 2048},
        # a long prompt through a gate or up projection
        {"name": "gemm 4096x8192x2048", "op": "gemm", "m": 4096, "n": 8192, "k": 2048},
        # one token through the smallest projection (keys or values): latency alone
        {"name": "gemv 1x512x2048", "op": "gemv", "m": 1, "n": 512, "k": 2048},
        # five tokens (a short draft to verify) through a long reduction
        {"name": "gemv 5x2048x8192", "op": "gemv", "m": 5, "n": 2048, "k": 8192},
        # one token through the vocabulary's projection: bandwidth
        {"name": "gemv 1x128256x2048", "op": "gemv", "m": 1, "n": 128256, "k": 2048},
        # one token of one request through a layer: latency
        {"name": "moe16 T=1", "op": "moe16", "t": 1, "h": 2048, "i": 512, "e": 256, "k": 8, "zipf": False},
        # a batch of decoding requests: most experts are touched by a few tokens
        {"name": "moe16 T=37", "op": "moe16", "t": 37, "h": 2048, "i": 512, "e": 256, "k": 8, "zipf": False},
        # a short prompt
        {"name": "moe4 T=300", "op": "moe4", "t": 300, "h": 2048, "i": 512, "e": 256, "k": 8, "zipf": False},
        # a long prompt, with experts of uneven popularity, some of them empty
        {"name": "moe4 T=4096 zipf", "op": "moe4", "t": 4096, "h": 2048, "i": 512, "e": 256, "k": 8, "zipf": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "gemm", "gemv", "moe16", "moe4"])
    if op == "quantize":
        cols = 32 * _log(rng, 2, 256)
        return {"op": op, "rows": _log(rng, 1, min(4096, 4096 * 2048 // cols)), "cols": cols,
                "dtype": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "gemm":
        k = 32 * _log(rng, 4, 256)
        m = _log(rng, 33, 4096)
        return {"op": op, "m": m, "n": _log(rng, 64, min(8192, 4096 * 8192 * 2048 // (k * m))), "k": k}
    if op == "gemv":
        k = 32 * _log(rng, 8, 256)
        return {"op": op, "m": rng.randint(1, 32), "n": _log(rng, 64, 128256 * 2048 // k), "k": k}
    e = rng.choice([8, 16, 64, 128, 256])
    t = _log(rng, 1, 64) if op == "moe16" else _log(rng, 65, 4096)
    return {"op": op, "t": t, "h": 128 * rng.randint(2, 16), "i": 128 * rng.randint(1, 4), "e": e,
            "k": rng.randint(1, min(8, e)), "zipf": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs

def _gen(seed, *parts):
    g = torch.Generator(device="cuda")
    h = seed
    for p in parts:
        h = (h * 1000003 + int(p)) % (1 << 62)
    g.manual_seed(h)
    return g


def _weights(shape, seed, tag):
    """Codes [.., cols / 2] and scale bytes [.., cols / 32] of normal weights of variance
    1 / cols, and the scales laid out in the tiles of 128 rows x 4 blocks that the matrix
    units read (512 bytes: byte 16 (r % 32) + 4 (r / 32) + b; rows and blocks padded with 0)."""
    experts, rows, cols = shape
    w = torch.randn(shape, generator=_gen(seed, tag), device="cuda") * (cols ** -0.5)
    # a weight matrix's rows and columns differ in size by a few powers of two
    w *= torch.exp2(torch.randint(-1, 2, (experts, rows, 1), generator=_gen(seed, tag, 1), device="cuda").float())
    codes, scales = _quantize(w)
    return {"codes": codes, "scales": scales, "tiles": _tiles(scales), "rows": rows, "cols": cols, "experts": experts}


def _tiles(scales):
    experts, rows, blocks = scales.shape
    pad = torch.nn.functional.pad(scales, (0, -blocks % 4, 0, -rows % 128))
    t = pad.reshape(experts, -1, 4, 32, pad.shape[2] // 4, 4).permute(0, 1, 4, 3, 2, 5)
    return t.reshape(-1).contiguous()


def _hidden(rows, cols, seed, dtype):
    """Hidden states: normal, with a few columns much larger than the rest, as models have."""
    x = torch.randn((rows, cols), generator=_gen(seed, 11), device="cuda")
    big = torch.randint(0, cols, (max(1, cols // 512),), generator=_gen(seed, 12), device="cuda")
    x[:, big] *= 8.0
    return x.to(dtype)


def _router_bias(c, seed):
    """Offsets that make the experts' popularity fall off as 1 / rank, in a random order, in
    units of the logits' own spread."""
    if not c["zipf"]:
        return None
    rank = torch.randperm(c["e"], generator=_gen(seed, 21), device="cuda").float() + 1
    return -(0.05 * c["h"] ** 0.5) * torch.log(rank)


def prepare(case, seed):
    c = case
    if c["op"] == "quantize":
        dtype = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[c["dtype"]]
        return {"case": c, "x": _hidden(c["rows"], c["cols"], seed, dtype)}
    if c["op"] == "gemm":
        # the left operand is what a quantized activation looks like: blocks of both sizes
        codes, scales = _quantize(_hidden(c["m"], c["k"], seed, torch.float32)[None])
        a = {"codes": codes, "scales": scales, "tiles": _tiles(scales), "rows": c["m"], "cols": c["k"], "experts": 1}
        return {"case": c, "a": a, "w": _weights((1, c["n"], c["k"]), seed, 1)}
    if c["op"] == "gemv":
        return {"case": c, "x": _hidden(c["m"], c["k"], seed, torch.bfloat16), "w": _weights((1, c["n"], c["k"]), seed, 1)}
    h, i, e, k = c["h"], c["i"], c["e"], c["k"]
    router = torch.randn((e, h), generator=_gen(seed, 20), device="cuda") * 0.05
    bias = _router_bias(c, seed)
    x = torch.randn((c["t"], h), generator=_gen(seed, 22), device="cuda").to(torch.bfloat16)
    for attempt in range(40):  # a token whose best experts are almost tied is drawn again
        logits = x.float() @ router.T
        top = torch.topk(logits if bias is None else logits + bias, min(k + 1, e), dim=1).values
        tied = ((top[:, :-1] - top[:, 1:]) < 2e-4).any(dim=1) if top.shape[1] > 1 else torch.zeros(c["t"], dtype=torch.bool, device="cuda")
        if not bool(tied.any()):
            break
        again = torch.randn((c["t"], h), generator=_gen(seed, 23, attempt), device="cuda").to(torch.bfloat16)
        x = torch.where(tied[:, None], again, x)
    return {"case": c, "x": x, "router": router, "bias": bias,
            "gate_up": _weights((e, 2 * i, h), seed, 1), "down": _weights((e, h, i), seed, 2),
            "shared_gate_up": _weights((1, 2 * i, h), seed, 3), "shared_down": _weights((1, h, i), seed, 4)}


# ------------------------------------------------------------- plain forms

def _power(s):
    """2^(s - 127) in 32 bits for the scale byte s, from its bits."""
    return torch.where(s == 0, 1 << 22, s.int() << 23).view(torch.float32)


def _quantize(x):
    """Codes and scale bytes of x [.., cols]: the scale is the power of two two binades below
    the block's largest magnitude, a value the nearest of the eight (ties to the even code), those
    over 6 become 6."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // BLOCK, BLOCK)
    top = b.abs().amax(dim=-1)
    s = torch.where(top > 0, torch.frexp(top).exponent - 3 + EXP, 0).clamp(0, 254)
    v = b * _power(254 - s)[..., None]
    q = v.abs()
    code = ((q > 0.25).to(torch.uint8) + (q >= 0.75) + (q > 1.25) + (q >= 1.75) + (q > 2.5) + (q >= 3.5) + (q > 5.0))
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), s.to(torch.uint8)


def _values(codes, scales):
    """What codes [.., cols / 2] and scales [.., cols / 32] stand for, in 32 bits."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    pair = torch.stack((codes & 15, codes >> 4), dim=-1).int()
    v = table[pair].reshape(*scales.shape, BLOCK) * _power(scales)[..., None]
    return v.reshape(*codes.shape[:-1], -1)


def _silu(g):
    return g / (1 + torch.exp(-g))


def _experts(x, w, s, four):
    """The outputs [E, T, H] of the experts of w on x [E or 1, T, H]."""
    up = torch.matmul(x, _values(w[0]["codes"], w[0]["scales"]).transpose(1, 2))
    half = up.shape[2] // 2
    h = _silu(up[..., :half]) * up[..., half:]
    if four:
        h = _values(*_quantize(h))
    return torch.matmul(h, _values(w[1]["codes"], w[1]["scales"]).transpose(1, 2))


def _take(w, ids):
    return {"codes": w["codes"][ids], "scales": w["scales"][ids]}


def _plain_moe(s, four):
    c, x = s["case"], s["x"].float()
    logits = torch.matmul(x, s["router"].T)
    best = torch.topk(logits if s["bias"] is None else logits + s["bias"], c["k"], dim=1)
    weight = torch.exp(best.values - best.values[:, :1])
    weight = weight / weight.sum(dim=1, keepdim=True)
    if four:
        x = _values(*_quantize(x))
    if c["t"] * c["k"] <= c["e"]:  # few tokens: the chosen experts' weights, once for each choice
        ids = best.indices.reshape(-1)
        each = x[:, None].expand(-1, c["k"], -1).reshape(-1, 1, c["h"])
        y = _experts(each, (_take(s["gate_up"], ids), _take(s["down"], ids)), s, four)
        y = (y.reshape(c["t"], c["k"], -1) * weight[..., None]).sum(dim=1)
    else:  # every expert on every token, weighted with 0 where it was not chosen
        full = torch.zeros((c["t"], c["e"]), device=x.device).scatter_(1, best.indices, weight)
        y = _experts(x[None], (s["gate_up"], s["down"]), s, four)
        y = torch.matmul(full[:, None, :], y.transpose(0, 1))[:, 0]
    y = y + _experts(x[None], (s["shared_gate_up"], s["shared_down"]), s, four)[0]
    return {"y": y.to(torch.bfloat16), "experts": best.indices.int(), "weights": weight}


def _plain(s):
    op = s["case"]["op"]
    if op == "quantize":
        return _values(*_quantize(s["x"])).to(torch.bfloat16)
    if op == "gemm":
        a, w = _values(s["a"]["codes"], s["a"]["scales"])[0], _values(s["w"]["codes"], s["w"]["scales"])[0]
        return torch.matmul(a, w.T).to(torch.bfloat16)
    if op == "gemv":
        return torch.matmul(s["x"].float(), _values(s["w"]["codes"], s["w"]["scales"])[0].T).to(torch.bfloat16)
    return _plain_moe(s, op == "moe4")


# ----------------------------------------------------------- the framework

def _tensor(q, w):
    return q.Mx4Tensor(w["codes"], w["tiles"], w["rows"], w["cols"], w["experts"])


def _own(s):
    import quantized_sparse_moe_gb300 as q
    c = s["case"]
    if c["op"] == "quantize":
        if "out" not in s:  # the buffers that a program keeps
            s["out"] = q.Mx4Tensor.empty(c["rows"], c["cols"], device="cuda")
        return q.mx4_dequantize(q.mx4_quantize(s["x"], out=s["out"]))
    if c["op"] == "gemm":
        if "plan" not in s:
            s["plan"] = _tensor(q, s["a"]), _tensor(q, s["w"])
        return q.mx4_gemm(*s["plan"])
    if c["op"] == "gemv":
        if "plan" not in s:
            s["plan"] = _tensor(q, s["w"])
        return q.mx4_gemv(s["x"], s["plan"])
    if "plan" not in s:
        layer = q.Mx4Layer(c["h"], c["i"], c["e"], c["k"], *(_tensor(q, s[n]) for n in ("gate_up", "down", "shared_gate_up", "shared_down")),
                           s["router"], s["bias"])
        s["plan"] = q.Mx4Forward(layer, c["t"], acts="mx4" if c["op"] == "moe4" else "bf16")
    f = s["plan"]
    y = f(s["x"])
    return {"y": y, "experts": f.topk_idx, "weights": f.topk_w}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work

def _bytes(rows, cols):
    return rows * (cols / 2 + cols / BLOCK)


def _touched(c):
    """How many experts a routing like the case's touches (drawn once, from a fixed seed)."""
    r = np.random.default_rng(0)
    logits = r.standard_normal((c["t"], c["e"]))
    if c["zipf"]:
        logits -= np.log(r.permutation(c["e"]) + 1.0)
    return len(np.unique(np.argsort(-logits, axis=1)[:, : c["k"]]))


def work(case):
    c = case
    if c["op"] == "quantize":
        n, each = c["rows"] * c["cols"], 4 if c["dtype"] == "fp32" else 2
        # x, the codes and scales, the values
        return {"bytes": n * each + _bytes(c["rows"], c["cols"]) + 2 * n, "flops": 2 * n}
    if c["op"] in ("gemm", "gemv"):
        x = _bytes(c["m"], c["k"]) if c["op"] == "gemm" else 2 * c["m"] * c["k"]
        return {"bytes": x + _bytes(c["n"], c["k"]) + 2 * c["m"] * c["n"], "flops": 2 * c["m"] * c["n"] * c["k"]}
    t, h, i, e, k = c["t"], c["h"], c["i"], c["e"], c["k"]
    weights = (_touched(c) + 1) * (_bytes(2 * i, h) + _bytes(h, i))
    return {"bytes": weights + 4 * e * h + 4 * t * h + 8 * t * k, "flops": 2 * t * e * h + 6 * t * (k + 1) * h * i}


# ------------------------------------------------------------ in 64 bits

def _wide(codes, scales):
    """What codes and scales stand for, in 64 bits, from the format's definition."""
    n = torch.stack((codes % 16, codes // 16), dim=-1).reshape(*codes.shape[:-1], -1).double()
    sign, e, m = torch.floor(n / 8), torch.floor(n / 2) % 4, n % 2
    v = torch.where(e == 0, m / 2, (1 + m / 2) * 2.0 ** (e - 1)) * (1 - 2 * sign)
    return v * (2.0 ** (scales.double() - EXP)).repeat_interleave(BLOCK, dim=-1)


def _round(x):
    """x in 64 bits, each value replaced by what its MXFP4 form stands for."""
    b = x.double().reshape(-1, BLOCK)
    top = b.abs().amax(dim=1, keepdim=True)
    e = torch.where(top > 0, torch.floor(torch.log2(top.clamp_min(1e-300))) - 2, torch.full_like(top, -EXP)).clamp(-EXP, EXP)
    q = b / 2.0 ** e
    step = 2.0 ** (torch.floor(torch.log2(q.abs().clamp_min(1e-300))).clamp(0, 2) - 1)
    return ((torch.round(q / step) * step).clamp(-6, 6) * 2.0 ** e).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        return _round(s["x"])
    w = s["w"] if op in ("gemm", "gemv") else None
    if op == "gemm":
        return _wide(s["a"]["codes"][0], s["a"]["scales"][0]) @ _wide(w["codes"][0], w["scales"][0]).T
    if op == "gemv":
        parts = [s["x"].double() @ _wide(a, b).T for a, b in zip(w["codes"][0].split(16384), w["scales"][0].split(16384))]
        return torch.cat(parts, dim=1)
    x = s["x"].double()
    logits = x @ s["router"].double().T
    order = torch.sort(logits if s["bias"] is None else logits + s["bias"].double(), dim=1, descending=True, stable=True)
    ids = order.indices[:, : case["k"]]
    weight = torch.softmax(order.values[:, : case["k"]], dim=1)
    four = op == "moe4"
    x = _round(x) if four else x

    def expert(v, up, down, n):
        g = v @ _wide(up["codes"][n], up["scales"][n]).T
        h = g[:, : case["i"]] * torch.sigmoid(g[:, : case["i"]]) * g[:, case["i"]:]
        return (_round(h) if four else h) @ _wide(down["codes"][n], down["scales"][n]).T

    y = expert(x, s["shared_gate_up"], s["shared_down"], 0)
    for n in torch.unique(ids).tolist():
        t, j = torch.nonzero(ids == n, as_tuple=True)
        y[t] += weight[t, j, None] * expert(x[t], s["gate_up"], s["down"], n)
    return {"y": y, "experts": None, "weights": weight}
