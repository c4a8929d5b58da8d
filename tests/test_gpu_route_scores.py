"""Routing by scores on the GPU against its definition in 64 bits.

Tolerance of the logits (fixed before the first run): products are exact; a logit is at
most H / 8 + 8 fp32 additions (the tensor cores may truncate), each off by at most 2^-23 of
the largest partial sum, which for these inputs (independent, normal) lies within 8 standard
deviations, 8 |x w|_2: |dl| <= (H / 8 + 8) 2^-23 8 |x w|_2.  A sigmoid's error is s (1 - s) |dl|
and four roundings, a softmax's 2 s |dl| and twelve (the sum over E in a tree); a
renormalized weight collects the relative error of two scores and of the sum over k.
Ids are exact: the inputs are drawn so that no choice hangs on less than these errors."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def definition(x, w, bias, k, score, groups, kept, best, renorm, scale):
    """(ids, weights, bound on the weights' error, tokens whose choice is too close to call)."""
    xd, wd = x.double(), w.double()
    l = xd @ wd.T
    dl = (x.shape[1] / 8 + 8) * 2.0 ** -23 * 8 * (xd.square() @ wd.square().T).sqrt().amax(dim=1, keepdim=True)
    if score == "sigmoid":
        s = torch.sigmoid(l)
        ds = s * ((1 - s) * torch.expm1(dl) + 4 * U)
    else:
        s = torch.softmax(l, dim=1)
        ds = s * (torch.expm1(2 * dl) + 12 * U)
    c = s if bias is None else s + bias.double()
    if bias is not None:
        ds = ds + U * c.abs()
    T, E = c.shape
    close = torch.zeros(T, dtype=torch.bool, device=x.device)
    if kept < groups:
        part = c.reshape(T, groups, -1)
        value = part.topk(best, dim=2).values.sum(dim=2)
        order = torch.sort(value, dim=1, descending=True, stable=True)
        close |= order.values[:, kept - 1] - order.values[:, kept] < 2 * best * ds.amax(dim=1)
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, order.indices[:, :kept], True)
        c = torch.where(keep[:, :, None], part, -torch.inf).reshape(T, E)
    order = torch.sort(c, dim=1, descending=True, stable=True)
    n = min(k + 1, E)
    top, err = order.values[:, :n], ds.gather(1, order.indices[:, :n])
    close |= (top[:, :-1] - top[:, 1:] < err[:, :-1] + err[:, 1:]).any(dim=1)
    ids = order.indices[:, :k]
    wt, dw = s.gather(1, ids), ds.gather(1, ids)
    rel = dw / wt
    if renorm:
        rel = rel + rel.amax(dim=1, keepdim=True) + 8 * U
        wt = wt / wt.sum(dim=1, keepdim=True)
    return ids, wt * scale, (wt * scale).abs() * (torch.expm1(rel) + 2 * U), close


def draw(T, H, E, seed, **kw):
    """x, w without a token whose choice is too close to call."""
    w = torch.randn((E, H), generator=gen(seed), device="cuda") * (2.0 * H ** -0.5)
    x = torch.randn((T, H), generator=gen(seed + 1), device="cuda").to(torch.bfloat16)
    for n in range(400):
        close = definition(x, w, **kw)[-1]
        if not bool(close.any()):
            return x, w
        x = torch.where(close[:, None], torch.randn((T, H), generator=gen(seed + 2 + n), device="cuda").to(torch.bfloat16), x)
    raise AssertionError("ties")


def router(qsm, w, bias, k, score, groups, kept, best, renorm, scale):
    return qsm.MoERouter(w, k, score, bias, groups=groups, groups_kept=kept, group_best=best,
                         renormalize=renorm, scale=scale)


def check(qsm, T, H, E, seed, **kw):
    x, w = draw(T, H, E, seed, **kw)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = router(qsm, w, **kw)
    ids, wt = qsm.moe_route_scores(x, r, dev_status=st)
    want, ww, bound, _ = definition(x, w, **kw)
    assert torch.equal(ids.long(), want)
    assert ((wt.double() - ww).abs() <= bound).all()
    assert st.item() == 0
    return x, r, ids, wt


def bias_of(E, seed=5):
    return 0.05 * torch.randn(E, generator=gen(seed), device="cuda")


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 64, 65, 255, 300, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens(qsm, T, score):
    check(qsm, T, 2048, 256, T, bias=bias_of(256), k=8, score=score, groups=8, kept=4, best=2, renorm=True, scale=2.5)


@pytest.mark.parametrize("H,E,k,groups,kept", [
    (64, 1, 1, 1, 1), (64, 5, 5, 1, 1), (192, 8, 3, 2, 1), (320, 48, 6, 6, 2), (1024, 64, 6, 8, 3),
    (448, 128, 32, 4, 4), (512, 129, 4, 3, 2), (2048, 160, 8, 8, 3), (640, 256, 8, 1, 1), (1024, 300, 10, 10, 4),
    (2048, 512, 10, 32, 8), (128, 512, 32, 16, 1), (4096, 384, 12, 12, 6)])
def test_shapes(qsm, H, E, k, groups, kept):
    for T, (score, best, renorm, b) in zip((3, 37, 130, 70), itertools.product(("softmax", "sigmoid"), (1, 2), (False,), (True,))):
        if best > E // groups:
            best = 1
        check(qsm, T, H, E, T, bias=bias_of(E) if b else None, k=k, score=score, groups=groups, kept=kept,
              best=best, renorm=renorm, scale=1.0)
    check(qsm, 20, H, E, 9, bias=None, k=k, score="softmax", groups=groups, kept=kept, best=1, renorm=True, scale=0.5)


def test_softmax_without_bias_is_the_other_router(qsm):
    T, H, E, k = 300, 2048, 256, 8
    x, w = draw(T, H, E, 3, bias=None, k=k, score="softmax", groups=1, kept=1, best=1, renorm=True, scale=1.0)
    for renorm in (True, False):
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, k, renormalize=renorm))
        want, ww = qsm.moe_route(x, w, k, renormalize=renorm)
        assert torch.equal(ids, want) and (wt - ww).abs().max() < 2e-5   # both within 1e-5 of the definition


def test_ties_go_to_the_lower_index(qsm):
    H, E = 128, 64
    x = torch.randn((5, H), generator=gen(1), device="cuda").to(torch.bfloat16)
    for score in ("softmax", "sigmoid"):
        w = torch.zeros(E, H, device="cuda")                              # every score the same
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 6, score))
        assert torch.equal(ids, torch.arange(6, device="cuda", dtype=torch.int32).expand(5, 6))
        assert torch.allclose(wt, torch.full_like(wt, 1 / 6), rtol=1e-6)
        ids, _ = qsm.moe_route_scores(x, qsm.MoERouter(w, 6, score, groups=8, groups_kept=2, group_best=2))
        assert torch.equal(ids, torch.arange(6, device="cuda", dtype=torch.int32).expand(5, 6))
        b = torch.zeros(E, device="cuda")
        b[40:48] = 0.25                                                   # group 5, then group 0
        ids, _ = qsm.moe_route_scores(x, qsm.MoERouter(w, 10, score, b, groups=8, groups_kept=2, group_best=2))
        assert ids[0].tolist() == [40, 41, 42, 43, 44, 45, 46, 47, 0, 1]


@pytest.mark.parametrize("E", [1, 5, 33, 48, 128, 130, 256, 300, 512])
def test_ties_of_many(qsm, E):
    """Equal and two-valued scores: the lanes of a warp run out of experts at different times."""
    H, T, k = 64, 21, min(E, 32)
    x = torch.zeros(T, H, device="cuda")
    x[:, 0] = 1
    x = x.bfloat16()
    w = torch.zeros(E, H, device="cuda")
    ids, _ = qsm.moe_route_scores(x, qsm.MoERouter(w, k))
    assert torch.equal(ids, torch.arange(k, device="cuda", dtype=torch.int32).expand(T, k))
    for seed in range(3):
        high = torch.rand(E, generator=gen(seed), device="cuda") < 0.3
        w[:, 0] = torch.where(high, 1.0, -1.0)
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, k, "sigmoid", renormalize=False))
        want = torch.sort((~high).int(), stable=True).indices[:k]
        assert torch.equal(ids.long(), want.expand(T, k))
        assert torch.allclose(wt[0], torch.sigmoid(w[want, 0]), rtol=1e-6)


def test_closed_experts(qsm):
    T, H, E = 4, 256, 16
    x = torch.randn((T, H), generator=gen(2), device="cuda").to(torch.bfloat16)
    w = torch.randn((E, H), generator=gen(3), device="cuda") * 0.1
    b = torch.full((E,), -torch.inf, device="cuda")
    b[3], b[9] = 0.0, 0.5
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for score in ("softmax", "sigmoid"):
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 4, score, b), dev_status=st)
        assert all(sorted(row[:2]) == [3, 9] and row[2:] == [0, 1] for row in ids.tolist())
        assert not wt[:, 2:].any() and torch.allclose(wt.sum(dim=1), torch.ones(T, device="cuda"))
        # all closed: the first of them, with weight 0
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 3, score, torch.full((E,), -torch.inf, device="cuda")), dev_status=st)
        assert ids.tolist() == [[0, 1, 2]] * T and not wt.any()
        # a kept group with too few open experts gives closed ones, not those of other groups
        c = torch.zeros(E, device="cuda")
        c[:3], c[4:] = -torch.inf, -4.0
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 2, score, c, groups=4, groups_kept=1), dev_status=st)
        assert ids.tolist() == [[3, 0]] * T and not wt[:, 1].any()
    assert st.item() == 0


def test_values_that_are_not_finite(qsm):
    T, H, E = 40, 128, 32
    x = torch.randn((T, H), generator=gen(4), device="cuda").to(torch.bfloat16)
    w = torch.randn((E, H), generator=gen(5), device="cuda") * 0.2
    for score in ("softmax", "sigmoid"):
        r = qsm.MoERouter(w, 4, score)
        want = qsm.moe_route_scores(x, r)
        y = x.clone()
        y[7, 3], y[20, 0] = float("nan"), float("inf")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        ids, wt = qsm.moe_route_scores(y, r, dev_status=st)
        good = [t for t in range(T) if t not in (7, 20)]
        assert torch.equal(ids[good], want[0][good]) and torch.equal(wt[good], want[1][good])
        assert ids[7].tolist() == [0, 1, 2, 3] and not wt[[7, 20]].any()     # every logit is lost
        assert st.item() == 2
        v = w.clone()
        v[want[0][0, 0].item()] = float("nan")                             # one expert is lost
        st.zero_()
        ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(v, 4, score), dev_status=st)
        assert st.item() == 2 and not (ids == want[0][0, 0]).any() and wt.isfinite().all()
        b = torch.zeros(E, device="cuda")
        b[want[0][0, 0].item()] = float("inf")
        st.zero_()
        ids, _ = qsm.moe_route_scores(x, qsm.MoERouter(w, 4, score, b), dev_status=st)
        assert st.item() == 2 and not (ids == want[0][0, 0]).any()


def test_scores_at_the_ends(qsm):
    """Logits of hundreds: sigmoid 1 (ties) and 0, a softmax with one expert left."""
    H, E = 64, 8
    w = torch.zeros(E, H, device="cuda")
    w[:, 0] = torch.tensor([-500.0, 300, 200, -90, 0, 300, 100, -500], device="cuda")
    x = torch.zeros(1, H, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = 1
    ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 4, "sigmoid", renormalize=False))
    assert ids.tolist() == [[1, 2, 5, 6]] and (wt == 1).all()
    ids, wt = qsm.moe_route_scores(x, qsm.MoERouter(w, 3, "softmax", renormalize=False))
    assert ids.tolist() == [[1, 5, 2]] and (wt[0, :2] == 0.5).all()
    # e^-100 / 2 = 1.86e-44: subnormal, in steps of 1.4e-45, rounded twice (the exponential, the quotient)
    assert abs(wt[0, 2].item() - 1.86e-44) <= 2 * 1.41e-45
    ids, wt = qsm.moe_route_scores(-x, qsm.MoERouter(w, 1, "sigmoid", torch.tensor([-3.0, 0, 0, -3, -3, 0, 0, -3], device="cuda")))
    assert ids.tolist() == [[1]] and not wt.any()                         # its score is 0: the sum is 0


def test_layouts_streams_and_a_graph(qsm):
    T, H, E, k = 50, 512, 64, 6
    kw = dict(bias=bias_of(E), k=k, score="sigmoid", groups=8, kept=3, best=2, renorm=True, scale=2.0)
    x, r, ids, wt = check(qsm, T, H, E, 11, **kw)
    m = torch.full((T, H + 24), float("nan"), dtype=torch.bfloat16, device="cuda")
    m[:, 8:8 + H] = x
    got = qsm.moe_route_scores(m[:, 8:8 + H], r)
    assert torch.equal(got[0], ids) and torch.equal(got[1], wt)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = qsm.moe_route_scores(x, r, stream=s)
    s.synchronize()
    assert torch.equal(got[0], ids) and torch.equal(got[1], wt)
    # outputs behind the last token stay
    bi, bw = torch.full((T + 3, k), -7, dtype=torch.int32, device="cuda"), torch.full((T + 3, k), 7.0, device="cuda")
    qsm.moe_route_scores(x, r, bi[:T], bw[:T])
    assert torch.equal(bi[:T], ids) and (bi[T:] == -7).all() and (bw[T:] == 7).all()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gi, gw = qsm.moe_route_scores(x, r)
    x2, _ = draw(T, H, E, 12, **kw)
    x.copy_(x2)
    g.replay()
    want = qsm.moe_route_scores(x, r)
    assert torch.equal(gi, want[0]) and torch.equal(gw, want[1])
    e = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    assert qsm.moe_route_scores(e, r)[0].shape == (0, k)


def test_the_weights_are_those_of_the_constructor(qsm):
    x = torch.randn((3, 64), generator=gen(6), device="cuda").to(torch.bfloat16)
    w = torch.randn((8, 64), generator=gen(7), device="cuda")
    r = qsm.MoERouter(w, 2)
    want = qsm.moe_route_scores(x, r)
    w.zero_()
    got = qsm.moe_route_scores(x, r)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals(qsm):
    w = torch.randn((16, 128), generator=gen(8), device="cuda")
    for kw in (dict(k=0), dict(k=17), dict(k=2, score="max"), dict(k=2, groups=3), dict(k=2, groups=4, groups_kept=5),
               dict(k=5, groups=4, groups_kept=1), dict(k=2, group_best=3), dict(k=1, groups=16, groups_kept=2, group_best=2),
               dict(k=2, scale=float("inf")), dict(k=2, bias=torch.zeros(15, device="cuda")), dict(k=2, bias=torch.zeros(16))):
        with pytest.raises(qsm.QSMError):
            qsm.MoERouter(w, **kw)
    for bad in (w.half(), w.cpu(), w[:, :96].contiguous(), w.t(), torch.zeros(513, 64, device="cuda")):
        with pytest.raises(qsm.QSMError):
            qsm.MoERouter(bad, 2)
    r = qsm.MoERouter(w, 2)
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    ids, wt = qsm.moe_route_scores(x, r)
    for f in (lambda: qsm.moe_route_scores(x.float(), r), lambda: qsm.moe_route_scores(x[:, :64], r),
              lambda: qsm.moe_route_scores(x.cpu(), r), lambda: qsm.moe_route_scores(x, r, ids[:2]),
              lambda: qsm.moe_route_scores(x, r, ids, wt.half()), lambda: qsm.moe_route_scores(x, r, ids.long()),
              lambda: qsm.moe_route_scores(torch.zeros(4, 132, dtype=torch.bfloat16, device="cuda")[:, 4:], r)):
        with pytest.raises(qsm.QSMError):
            f()
    with pytest.raises(AttributeError):
        r.k = 3


def test_offsets_that_pass_32_bits(qsm):
    """x and its row offsets past 2^32 elements; the last tokens as a call of their own."""
    T, H, E, k = (1 << 20) + 37, 4096, 48, 6
    r = qsm.MoERouter(torch.randn((E, H), generator=gen(70), device="cuda"), k, "sigmoid", groups=6, groups_kept=3)
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-40:] = (torch.randn((40, H), generator=gen(71), device="cuda") * H ** -0.5).bfloat16()
    ids, w = r.route(x)
    want, ww = r.route(x[-40:].clone())
    assert torch.equal(ids[-40:], want) and (w[-40:] - ww).abs().max().item() <= 1e-5
    assert torch.equal(ids[:1000], torch.arange(k, device="cuda", dtype=torch.int32).expand(1000, k))


def last_bits(E, H):
    """w [E, H] of 24 significant bits, whose order in each column lies in the last of them:
    4 + (2^14 + 8 p + 3) 2^-21 with p = (e + column) mod E.  The first 8 bits are 4, the next
    8 units of 2^-14, and p goes down to 2^-18."""
    p = (torch.arange(E)[:, None] + torch.arange(H)[None]) % E
    return p, (4 + (2 ** 14 + 8 * p + 3).double() * 2.0 ** -21).float()


@pytest.mark.parametrize("E", [5, 100, 128, 256, 300, 512])
@pytest.mark.parametrize("T,H", [(1, 64), (1, 2048), (37, 704), (300, 2048), (4096, 2048)])
def test_every_bit_of_the_weights_counts(qsm, T, H, E):
    """A token is a multiple of a unit vector: its logits are a column of w, exactly, so that ids and weights
    hang on the last bits alone.
    Softmax, logits of 64: neighbours are 2^-14 apart and all within 0.04 of the best one.  A weight collects
    4 roundings of the exponential (two units in the last place), 21 of the sum and the exponentials in it
    4 more, 4 of the quotient (two units), 1: 34 U; divided by the sum of k, twice that, k and 5 more.
    Sigmoid, logits of -8: neighbours 2^-17 apart; the exponential of 8 to 11 units in the last place (22 U),
    1, 4 of the quotient: 27 U.  Without the last 8 bits a weight would be off by up to 2^-11 and 2^-14."""
    k = min(E, 8)
    p, w = last_bits(E, H)
    col = torch.arange(T) * 37 % H
    r = w.cuda()
    for score, f, bound in (("softmax", 16.0, 34 * U), ("sigmoid", -2.0, 27 * U)):
        x = torch.zeros(T, H)
        x[torch.arange(T), col] = f
        l = f * w.double()[:, col].T                      # exact
        s = torch.softmax(l, dim=1) if score == "softmax" else torch.sigmoid(l)
        want = torch.sort(l, dim=1, descending=True).indices[:, :k]
        for renorm in (False, True):
            ids, wt = qsm.moe_route_scores(x.bfloat16().cuda(), qsm.MoERouter(r, k, score, renormalize=renorm))
            ww, tol = s.gather(1, want), bound
            if renorm:
                ww, tol = ww / ww.sum(dim=1, keepdim=True), 2 * bound + (k + 5) * U
            assert torch.equal(ids.cpu().long(), want)
            assert ((wt.cpu().double() - ww).abs() <= tol * ww).all()
