"""The residual stream and its norms on the GPU against the formulas in 64 bits.

Tolerance (fixed before the first run): the kernel's arithmetic is fp32 between the
loads and the stores, so each result is the rounding to its type of something within
the fp32 error that tests/_block_ref.py adds up for these very inputs (64 roundings for
a sum over a row, one for each operation).  An MXFP4 code is the code of something within
that error of h; in a block whose largest magnitude is that close to a power of two either
scale is right."""
import pytest
import torch

import _block_ref as ref
import _mx4_ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def draw(shape, seed, dtype=torch.float32):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def side(qsm, kind, H, seed, bias=True, eps=1e-6):
    """(Norm or None, the same for the reference)."""
    if kind is None:
        return None, (None, None, None, 0.0)
    w = 1 + 0.3 * draw((H,), seed)
    b = 0.2 * draw((H,), seed + 1) if bias else None
    return qsm.Norm(w, b, kind=kind, eps=eps), (w.cpu(), None if b is None else b.cpu(), kind, eps)


def gate_of(kind, T, H, seed, dtype=torch.bfloat16):
    shape = {"none": None, "channel": (H,), "token": (T, 1), "full": (T, H)}[kind]
    return None if shape is None else 1 + 0.5 * draw(shape, seed, dtype).to(dtype)


def check_codes(h, tiles, want, err):
    """h: an Mx4Tensor; every code that of something within err of want."""
    T, H = want.shape
    codes, scales = h.codes.cpu().reshape(T, H // 2), _mx4_ref.untile(h.scales.cpu(), T, H)
    lo, hi = want.abs() - err, want.abs() + err
    top_lo, top_hi = (t.reshape(T, -1, 32).amax(dim=2) for t in (lo, hi))
    e = lambda t: torch.clamp(torch.floor(torch.log2(t.clamp_min(1e-300))) - 2, -127, 127)  # noqa: E731
    s = scales.double() - 127
    assert ((s >= e(top_lo)) & (s <= e(top_hi))).all()
    got = _mx4_ref.values(codes, scales)
    unit = torch.exp2(s).repeat_interleave(32, dim=1)

    def nearest(v):  # of one magnitude, in units of its block's scale
        q = v / unit
        step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0)).double()
        return (torch.round(q / step) * step).clamp(max=6) * unit
    sign = torch.where(want < 0, -1.0, 1.0).double()
    a, b = nearest((want * sign - err).clamp_min(0)), nearest(want * sign + err)
    m = got * sign
    assert ((m >= a) & (m <= b) | (want.abs() <= err) & (m.abs() <= b)).all()
    full = _mx4_ref.untile(h.scales.cpu(), -(-T // 128) * 128, -(-H // 128) * 128)
    assert not full[T:].any() and not full[:, H // 32:].any()             # the padding holds 0


@pytest.mark.parametrize("post,pre", [(None, "rms"), ("rms", "rms"), ("layer", "layer"), ("rms", None), (None, "layer")])
@pytest.mark.parametrize("T,H", [(1, 2048), (1, 8), (5, 264), (3, 256), (160, 1056), (153, 8192), (300, 2048), (2, 16384), (200, 16384), (170, 128)])
def test_formula(qsm, T, H, post, pre):
    x, y = draw((T, H), T + H, torch.bfloat16) * 3, draw((T, H), T + H + 1, torch.bfloat16)
    npost, rpost = side(qsm, post, H, 10)
    npre, rpre = side(qsm, pre, H, 20, bias=pre == "layer")
    n = qsm.ResidualNorm(H, pre=npre, post=npost, scale=0.22)
    xo, h = n(x, y)
    (wx, ex), wh = ref.residual(x, y, None, n.scale, rpost, rpre)
    assert ref.lies_between(xo, wx, ex)
    assert (h is None) == (pre is None)
    if h is not None:
        assert ref.lies_between(h, *wh)


@pytest.mark.parametrize("xt", DT)
@pytest.mark.parametrize("yt", DT)
@pytest.mark.parametrize("ht", [*DT, "mx4"])
def test_types(qsm, xt, yt, ht):
    for T, H in ((3, 320), (161, 416)):
        x, y = draw((T, H), 1, DT[xt]) * 2, draw((T, H), 2, DT[yt])
        npre, rpre = side(qsm, "rms", H, 30, bias=False)
        n = qsm.ResidualNorm(H, pre=npre)
        st = status()
        xo, h = n(x, y, h="mx4" if ht == "mx4" else DT[ht], dev_status=st)
        (wx, ex), (wh, eh) = ref.residual(x, y, None, 1.0, (None,) * 3 + (0.0,), rpre)
        assert xo.dtype == DT[xt] and ref.lies_between(xo, wx, ex)
        if ht == "mx4":
            check_codes(h, None, wh, eh)
        else:
            assert h.dtype == DT[ht] and ref.lies_between(h, wh, eh)
        assert st.item() == 0


@pytest.mark.parametrize("kind", ["channel", "token", "full"])
@pytest.mark.parametrize("gt", DT)
@pytest.mark.parametrize("sigmoid", [False, True])
def test_gates(qsm, kind, gt, sigmoid):
    for T, H in ((1, 64), (7, 640), (200, 640)):
        x, y = draw((T, H), 3, torch.bfloat16), draw((T, H), 4, torch.float32)
        g = gate_of(kind, T, H, 5, DT[gt]).to(DT[gt])
        npre, rpre = side(qsm, "rms", H, 40)
        npost, rpost = side(qsm, "rms", H, 50)
        n = qsm.ResidualNorm(H, pre=npre, post=npost, scale=-1.5, sigmoid_gate=sigmoid)
        xo, h = n(x, y, g)
        (wx, ex), wh = ref.residual(x, y, g, -1.5, rpost, rpre, sigmoid)
        assert ref.lies_between(xo, wx, ex) and ref.lies_between(h, *wh)


@pytest.mark.parametrize("T,H", [(1, 32), (1, 2048), (127, 96), (129, 160), (300, 2048), (4, 16384)])
def test_four_bits(qsm, T, H):
    x = draw((T, H), 6, torch.bfloat16)
    npre, rpre = side(qsm, "rms", H, 60)
    n = qsm.ResidualNorm(H, pre=npre)
    out = qsm.Mx4Tensor.empty(T, H)
    out.scales.fill_(77)                      # the padding is written too
    xo, h = n(x, h=out)
    assert xo is x and h is out
    _, (wh, eh) = ref.residual(x, None, None, 1.0, None, rpre)
    check_codes(h, None, wh, eh)


@pytest.mark.parametrize("post,pre,gate", [("rms", "rms", "none"), (None, "layer", "full"), ("layer", None, "channel"), (None, "rms", "token")])
@pytest.mark.parametrize("T,H", [(4096, 1024), (1700, 2048), (3400, 1000), (800, 5120), (200, 16384), (1, 16384)])
def test_many_rows(qsm, T, H, post, pre, gate):
    """Rows that follow one another through the same threads; in place, too."""
    for xt, yt, gt in ((torch.bfloat16, torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32, torch.float32)):
        x, y = draw((T, H), T + H, xt), draw((T, H), T + H + 1, yt)
        g = gate_of(gate, T, H, 5, gt)
        npost, rpost = side(qsm, post, H, 10)
        npre, rpre = side(qsm, pre, H, 20, bias=pre == "layer")
        n = qsm.ResidualNorm(H, pre=npre, post=npost, scale=0.22)
        (wx, ex), wh = ref.residual(x, y, g, n.scale, rpost, rpre)
        xo, h = n(x, y, g)
        assert ref.lies_between(xo, wx, ex) and (h is None or ref.lies_between(h, *wh))
        n(x, y, g, x_out=x, h=None if h is None else y)
        assert torch.equal(x, xo) and (h is None or torch.equal(y, h))


@pytest.mark.parametrize("T,H", [(1700, 2048), (3401, 1024), (200, 16384)])
def test_four_bits_of_many_rows(qsm, T, H):
    x = draw((T, H), 6, torch.bfloat16)
    npre, rpre = side(qsm, "rms", H, 60)
    out = qsm.Mx4Tensor.empty(T, H)
    out.scales.fill_(77)
    _, h = qsm.ResidualNorm(H, pre=npre)(x, h=out)
    _, (wh, eh) = ref.residual(x, None, None, 1.0, None, rpre)
    check_codes(h, None, wh, eh)


def test_large_values_sum_in_range(qsm):
    # squares of 1e4 over 4096 columns, an offset a thousand times the spread: the centred sum keeps it
    H = 4096
    x = (1e4 + draw((4, H), 7)).float()
    npre, rpre = side(qsm, "layer", H, 70)
    _, h = qsm.ResidualNorm(H, pre=npre)(x)
    _, wh = ref.residual(x, None, None, 1.0, None, rpre)
    assert ref.lies_between(h, *wh)
    zero = torch.zeros(2, H, device="cuda")   # eps alone
    _, h = qsm.ResidualNorm(H, pre=qsm.Norm(kind="rms"))(zero)
    assert not h.any()


def test_values_that_are_not_finite_stay_in_their_rows(qsm):
    T, H = 6, 256
    x = draw((T, H), 8, torch.bfloat16)
    clean = x.clone()
    x[1, 3], x[4, 5] = float("nan"), float("inf")
    n = qsm.ResidualNorm(H, pre=qsm.Norm(kind="rms"))
    _, want = n(clean)
    _, h = n(x)
    good = [0, 2, 3, 5]
    assert torch.equal(h[good], want[good])
    assert h[1].isnan().all()
    assert h[4, 5].isnan() and not h[4, :5].any()       # x / inf, and inf / inf
    st = status()
    _, q = n(x, h="mx4", dev_status=st)
    v = qsm.mx4_dequantize(q)
    assert st.item() == 2
    assert torch.equal(v[good], qsm.mx4_dequantize(n(clean, h="mx4")[1])[good])
    assert v[1].isnan().all() and v[4, :32].isnan().all() and not v[4, 32:].any()


def test_layouts(qsm):
    """In place, side by side in one matrix, strided rows; what lies between stays."""
    T, H = 37, 264
    x, y = draw((T, H), 9, torch.bfloat16), draw((T, H), 10, torch.bfloat16)
    npre, _ = side(qsm, "rms", H, 80)
    n = qsm.ResidualNorm(H, pre=npre, scale=0.5)
    wx, wh = n(x, y)
    a, b = x.clone(), y.clone()
    assert n(a, b, x_out=a, h=b) == (a, b) and torch.equal(a, wx) and torch.equal(b, wh)
    a, b = x.clone(), y.clone()
    n(a, b, x_out=b, h=a)
    assert torch.equal(b, wx) and torch.equal(a, wh)
    m = torch.full((T, 4 * H + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    m[:, :H], m[:, H:2 * H] = x, y
    n(m[:, :H], m[:, H:2 * H], x_out=m[:, 2 * H:3 * H], h=m[:, 3 * H + 8:])
    assert torch.equal(m[:, :H], x) and torch.equal(m[:, H:2 * H], y)
    assert torch.equal(m[:, 2 * H:3 * H], wx) and torch.equal(m[:, 3 * H + 8:], wh)
    assert (m[:, 3 * H:3 * H + 8] == 7).all()
    big = torch.full((T + 2, H), 7.0, dtype=torch.bfloat16, device="cuda")
    n(x, y, x_out=big[:T], h=wh.clone())
    assert torch.equal(big[:T], wx) and (big[T:] == 7).all()
    empty = torch.empty(0, H, dtype=torch.bfloat16, device="cuda")
    xo, h = n(empty, empty)
    assert xo.shape == h.shape == (0, H)


def test_refusals(qsm):
    T, H = 4, 64
    x = draw((T, H), 11, torch.bfloat16)
    n = qsm.ResidualNorm(H, pre=qsm.Norm())
    bad = [lambda: n(x[:, :32]), lambda: n(x.double()), lambda: n(x, x[:2]), lambda: n(x.t().contiguous().t()),
           lambda: n(x, gate=x), lambda: n(x, x.clone(), x[:, :8]), lambda: n(x, x_out=x[:2]),
           lambda: n(x, x_out=x.float()), lambda: n(x, h=x[:2]), lambda: n(x, h=torch.int32), lambda: n(x, h="fp4"),
           lambda: n(x, h=qsm.Mx4Tensor.empty(T + 1, H)), lambda: n(x.cpu()), lambda: n(x, x.cpu()),
           lambda: n(x.expand(2, T, H)), lambda: n(x[:1].expand(T, H)),
           lambda: n(x, dev_status=torch.zeros(1, device="cuda")),
           lambda: qsm.ResidualNorm(H)(x), lambda: qsm.ResidualNorm(H)(x, x, h=torch.bfloat16),
           lambda: qsm.ResidualNorm(H, pre=qsm.Norm(torch.ones(32, device="cuda"))),
           lambda: qsm.ResidualNorm(H, pre=qsm.Norm(torch.ones(H, device="cuda").half())),
           lambda: n(x, x.clone(), x_out=x, h=x)]
    for f in bad:
        with pytest.raises(qsm.QSMError):
            f()
    m = draw((T, 72), 12, torch.bfloat16)
    with pytest.raises(qsm.QSMError):
        n(m[:, 4:68])                          # rows not 16-byte aligned


def test_another_stream_and_a_graph(qsm):
    T, H = 64, 2048
    n = qsm.ResidualNorm(H, pre=side(qsm, "rms", H, 90)[0], post=side(qsm, "rms", H, 91)[0])
    x, y = draw((T, H), 13, torch.bfloat16), draw((T, H), 14, torch.bfloat16)
    wx, wh = n(x, y)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = n(x, y, stream=s)
    s.synchronize()
    assert torch.equal(got[0], wx) and torch.equal(got[1], wh)
    xo, h = torch.empty_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        n(x, y, x_out=xo, h=h)
    for seed in (15, 16):
        x.copy_(draw((T, H), seed, torch.bfloat16))
        wx, wh = n(x, y)
        g.replay()
        assert torch.equal(xo, wx) and torch.equal(h, wh)


@pytest.mark.parametrize("T,H", [(5, 96), (3401, 992)])
def test_padding_scales_are_zeros_beside_rows_that_are_not_finite(qsm, T, H):
    """Few rows and many; a row with a NaN, one of zeros under eps = 0 (0 / 0)."""
    x = draw((T, H), 17, torch.bfloat16)
    x[1, 3] = float("nan")
    x[T - 1] = 0
    out = qsm.Mx4Tensor.empty(T, H)
    out.scales.fill_(77)
    st = status()
    qsm.ResidualNorm(H, pre=qsm.Norm(kind="rms", eps=0.0))(x, h=out, dev_status=st)
    there = qsm.mx4_tile_scales(torch.ones((T, H // 32), dtype=torch.uint8)).cuda().bool()
    s = out.scales.view(torch.uint8).reshape(-1)
    assert st.item() == 2 and not s[~there].any()
    assert s[there].eq(255).sum().item() == 2 * (H // 32)


@pytest.mark.parametrize("T", [1, 9])
def test_a_gate_for_all_tokens_beside_what_is_written(qsm, T):
    """The gate in a row of the matrix whose other columns are written."""
    H = 128
    x, y, g = draw((T, H), 18, torch.bfloat16), draw((T, H), 19, torch.bfloat16), draw((H,), 20, torch.bfloat16)
    n = qsm.ResidualNorm(H, pre=qsm.Norm())
    wx, wh = n(x, y, g)
    m = torch.full((T, 3 * H), 7.0, dtype=torch.bfloat16, device="cuda")
    m[T // 2, H:2 * H] = g
    n(x, y, m[T // 2, H:2 * H], x_out=m[:, :H], h=m[:, 2 * H:])
    assert torch.equal(m[:, :H], wx) and torch.equal(m[:, 2 * H:], wh) and torch.equal(m[T // 2, H:2 * H], g)
    with pytest.raises(qsm.QSMError):
        n(x, y, m[T // 2, H - 8:2 * H - 8], x_out=m[:, :H])


def test_offsets_that_pass_32_bits(qsm):
    """2^32 elements and more, in rows and in scales; the last rows as a call of their own."""
    T, H = (1 << 18) + 37, 16384
    n = qsm.ResidualNorm(H, pre=qsm.Norm())
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    x[-40:] = draw((40, H), 21, torch.bfloat16)
    want, want4 = n(x[-40:].clone())[1], n(x[-40:].clone(), h="mx4")[1]
    _, h = n(x)
    assert torch.equal(h[-40:], want) and not h[:1000].any()
    del h
    _, q = n(x, h="mx4")
    codes = q.codes.view(torch.uint8).reshape(T, H // 2)
    assert torch.equal(codes[-40:], want4.codes.view(torch.uint8).reshape(40, H // 2))
    last = x[-40:].clone()
    n(x, x, x_out=x)
    assert torch.equal(x[-40:], 2 * last) and not x[:1000].any()   # x + x: exact
