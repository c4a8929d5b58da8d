"""MXFP4 and its products in 64 bits, from the definitions, for the tests
(nothing here calls the library)."""
from __future__ import annotations

import numpy as np
import torch

GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def quantize(x: torch.Tensor):
    """x [rows, cols] -> (codes [rows, cols / 2] uint8, scale bytes
    [rows, cols / 32] uint8) of finite values, by the rule of mx4_quantize."""
    rows, cols = x.shape
    b = x.double().cpu().reshape(rows, cols // 32, 32)
    top = b.abs().amax(dim=2)
    # floor(log2) from the binary exponent: exact, subnormals included
    e = np.frexp(top.numpy())[1].astype(np.int64) - 1
    s = np.where(top.numpy() > 0, np.clip(e - 2 + 127, 0, 254), 0)
    q = b / torch.from_numpy(np.exp2(s.astype(np.float64) - 127))[..., None]
    d = (q.abs()[..., None] - GRID).abs()
    lo = d.argmin(dim=3)                       # the lower code of a tie
    nxt = (lo + 1).clamp_max(7)
    tie = (d.gather(3, lo[..., None]) == d.gather(3, nxt[..., None]))[..., 0] & (nxt != lo)
    code = torch.where(tie & (lo % 2 == 1), nxt, lo)
    code = (code + 8 * torch.signbit(q)).to(torch.uint8).reshape(rows, cols // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), torch.from_numpy(s.astype(np.uint8))


def values(codes: torch.Tensor, scales: torch.Tensor) -> torch.Tensor:
    """[.., cols / 2] codes and [.., cols / 32] scale bytes -> [.., cols] float64."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1).long()
    v = GRID.to(codes.device)[c & 7] * torch.where(c >= 8, -1.0, 1.0)
    return v * torch.exp2(scales.double() - 127).repeat_interleave(32, dim=-1)


def untile(tiles: torch.Tensor, rows: int, cols: int) -> torch.Tensor:
    """The scale bytes [rows, cols / 32] of one matrix's tiles."""
    ct = -(-cols // 128)
    t = tiles.reshape(-(-rows // 128), ct, 32, 4, 4)  # row tile, column tile, r % 32, r / 32, block
    full = t.permute(0, 3, 2, 1, 4).reshape(-1, ct * 4)
    return full[:rows, :cols // 32]


def rounded(x: torch.Tensor) -> torch.Tensor:
    """The values of x's MXFP4 form, float64 on x's device."""
    c, s = quantize(x.reshape(-1, x.shape[-1]))
    return values(c, s).reshape(x.shape).to(x.device)


def draw(rows, cols, seed, spread=3.0, device="cuda"):
    """Normal values over a few binades (a random power of two per block)."""
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    x = torch.randn((rows, cols // 32, 32), generator=g)
    x *= torch.exp2(torch.randint(-int(spread), int(spread) + 1, (rows, cols // 32, 1), generator=g).float())
    return x.reshape(rows, cols).to(device)


def moe(x, idx, w, gate_up, down, shared_gate_up, shared_down, gate=None, four=False):
    """The layer's output [T, H] in float64 for the routing (idx, w); the
    weights are float64 [E, 2I, H], [E, H, I] (shared: E = 1)."""
    x = x.double()
    rnd = rounded if four else (lambda v: v)

    def expert(v, up, dn):
        g = v @ up.T
        half = g.shape[1] // 2
        h = g[:, :half] * torch.sigmoid(g[:, :half]) * g[:, half:]
        return rnd(h) @ dn.T

    xr = rnd(x)
    y = expert(xr, shared_gate_up[0], shared_down[0])
    if gate is not None:
        y = y * torch.sigmoid(x @ gate.double())[:, None]
    for e in torch.unique(idx).tolist():
        t, j = torch.nonzero(idx == e, as_tuple=True)
        y[t] += w[t, j].double()[:, None] * expert(xr[t], gate_up[e], down[e])
    return y
