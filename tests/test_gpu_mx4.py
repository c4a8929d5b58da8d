"""The MXFP4 calls on the GPU against their definitions in 64 bits.

Tolerances (fixed before the first run):
  quantization, dequantization and routing are exact;
  products of MXFP4 operands: every product is exact, so only the fp32 sums
    round, each of the at most K partial sums by at most 2^-23 of the largest
    of them (the tensor cores may truncate): |y - ref| <= b = K 2^-23 sum |a w|;
    a bf16 y is the rounding of something that close, so it lies between the
    roundings of ref - b and ref + b;
  few-row products: besides, each input is kept to 2^-16 of the largest
    magnitude in its block of 32;
  the MoE layer: the repository's bound of 2e-3 of the largest output with
    16-bit activations; with 4-bit activations h is rounded to 4 bits, and an
    h within about 2^-20 of a rounding boundary may fall on the other side (by
    a quarter of its value, 2^-17 of them): relative 2-norm 3e-3."""
import math

import numpy as np
import pytest
import torch

import _mx4_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def mx4(qsm, x, experts=1):
    """(Mx4Tensor, float64 values) of the quantized x [experts * rows, cols]."""
    t = qsm.mx4_quantize(x)
    v = qsm.mx4_dequantize(t, torch.float32).double()
    if experts == 1:
        return t, v
    rows = x.shape[0] // experts
    return (qsm.Mx4Tensor(t.codes, t.scales, rows, x.shape[1], experts),
            v.reshape(experts, rows, x.shape[1]))


# --------------------------------------------------------------- quantization

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 2048), (3, 96), (128, 128), (129, 160), (300, 4064)])
def test_quantize_is_the_definition(qsm, dtype, rows, cols):
    x = ref.draw(rows, cols, rows + cols).to(DTYPES[dtype])
    st = status()
    t = qsm.mx4_quantize(x, dev_status=st)
    codes, scales = ref.quantize(x)
    assert torch.equal(t.codes.cpu(), codes)
    tiles = t.scales.cpu()
    assert torch.equal(ref.untile(tiles, rows, cols), scales)
    assert torch.equal(tiles, qsm.mx4_tile_scales(scales))      # padding included
    for name, dt in DTYPES.items():
        want = ref.values(codes, scales)
        assert torch.equal(qsm.mx4_dequantize(t, dt).cpu().double(), want.to(dt).double())
    assert st.item() == 0


def test_quantize_edges(qsm):
    f32max, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    x = torch.zeros(8, 64, device="cuda")
    x[0, :9] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -6.5, 7.99])  # ties, over 6
    x[1, 0] = f32max                                    # the largest exponent
    x[2, 0], x[2, 1] = tiny, -tiny                      # subnormals: the smallest scale
    x[3, 0], x[3, 1] = 2.0 ** -126, 2.0 ** -127
    x[4, :] = -0.0
    x[5, 0], x[5, 33] = 1e-30, 3e20                     # blocks far apart
    x[6, :] = 6.0
    x[7, :] = torch.tensor([1.0, -1.0] * 32)
    st = status()
    t = qsm.mx4_quantize(x, dev_status=st)
    codes, scales = ref.quantize(x)
    assert torch.equal(t.codes.cpu(), codes)
    assert torch.equal(ref.untile(t.scales.cpu(), 8, 64), scales)
    assert st.item() == 0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
def test_quantize_marks_blocks_that_are_not_finite(qsm, dtype, what):
    x = ref.draw(130, 128, 3).to(DTYPES[dtype])
    good = qsm.mx4_quantize(x)
    x[129, 70] = what
    st = status()
    t = qsm.mx4_quantize(x, dev_status=st)
    assert st.item() == qsm.DEV_NONFINITE
    v, w = qsm.mx4_dequantize(t), qsm.mx4_dequantize(good)
    assert torch.isnan(v[129, 64:96]).all()
    v[129, 64:96] = w[129, 64:96]
    assert torch.equal(v, w)                            # no other block is touched


def test_quantize_reads_strided_rows(qsm):
    big = ref.draw(70, 512, 9).to(torch.bfloat16)
    x = big[:, 64:256]
    assert x.stride(0) == 512
    a, b = qsm.mx4_quantize(x), qsm.mx4_quantize(x.contiguous())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    with pytest.raises(qsm.QSMError):                   # columns apart
        qsm.mx4_quantize(big[:, ::2])
    with pytest.raises(qsm.QSMError):                   # rows not 16-byte aligned
        qsm.mx4_quantize(big[:, 4:100])


def test_dequantize_every_code_and_scale(qsm):
    codes = torch.arange(256, dtype=torch.uint8).repeat(16)[: 256 * 16].reshape(256, 16)
    codes = (codes.int() * 7 + torch.arange(16)[None].int() * 16).to(torch.uint8)
    scales = torch.arange(256, dtype=torch.uint8)[:, None]
    t = qsm.Mx4Tensor(codes.cuda(), qsm.mx4_tile_scales(scales).cuda(), 256, 32)
    v = qsm.mx4_dequantize(t, torch.float32).cpu()
    want = ref.values(codes, scales).float()
    assert torch.isnan(v[255]).all() and torch.equal(v[:255], want[:255])
    b = qsm.mx4_dequantize(t).cpu()
    assert torch.equal(b[:255], want[:255].to(torch.bfloat16))


def test_no_rows(qsm):
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    t = qsm.mx4_quantize(x)
    w, _ = mx4(qsm, ref.draw(40, 64, 1))
    assert qsm.mx4_dequantize(t).shape == (0, 64)
    assert qsm.mx4_gemm(t, w).shape == (0, 40) and qsm.mx4_gemm(w, t).shape == (40, 0)
    assert qsm.mx4_gemv(x, w).shape == (0, 40)


# ------------------------------------------------------------------- products

def product_bound(a, w):
    return a.shape[1] * 2.0 ** -23 * (a.abs() @ w.abs().T)


def near(y, want, b):
    """Where y is within b of want, before its own rounding."""
    if y.dtype == torch.float32:
        return (y.double() - want).abs() <= b
    # float64 -> bf16 by way of fp32 rounds twice: one fp32 ulp more of room
    b = b + want.abs() * 2.0 ** -23
    return (y >= (want - b).to(torch.bfloat16)) & (y <= (want + b).to(torch.bfloat16))


# one tile and less; two CTAs on one scale tile (64 columns); the wider tiles;
# K below, at and past a stage, and an odd number of blocks; pairs of SMs
GEMM = [(1, 1, 32), (5, 70, 64), (128, 64, 96), (130, 200, 256), (33, 257, 288), (200, 640, 1056),
        (1000, 2600, 352), (128 * 19, 4096, 64), (2401, 4200, 96), (700, 15001, 544), (500, 4100, 288),
        (2100, 4096, 96), (2177, 4090, 544),
        # long sums on pairs of SMs: an odd number of row tiles, a last tile of one
        # row, columns that end inside a tile, an odd number of blocks
        (2100, 4096, 4128), (2177, 4090, 4096), (130, 2000, 8192), (4000, 8001, 2080)]


@pytest.mark.parametrize("m,n,k", GEMM)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gemm(qsm, m, n, k, dtype):
    a, av = mx4(qsm, ref.draw(m, k, m + k))
    w, wv = mx4(qsm, ref.draw(n, k, n + k))
    st = status()
    y = qsm.mx4_gemm(a, w, DTYPES[dtype], dev_status=st)
    want = av @ wv.T
    assert near(y, want, product_bound(av, wv)).all()
    assert torch.equal(y, qsm.mx4_gemm(a, w, DTYPES[dtype]))
    assert st.item() == 0


@pytest.mark.parametrize("m,n,k", [(130, 200, 256), (2432, 4096, 64), (2250, 4096, 64), (2250, 4096, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gemm_writes_only_its_part_of_y(qsm, m, n, k, dtype):
    a, _ = mx4(qsm, ref.draw(m, k, 1))
    w, _ = mx4(qsm, ref.draw(n, k, 2))
    want = qsm.mx4_gemm(a, w, DTYPES[dtype])
    for pad, off in ((16, 8), (5, 3)):                  # aligned rows, and rows that are not
        big = torch.full((m + 2, n + pad), 7.0, dtype=DTYPES[dtype], device="cuda")
        qsm.mx4_gemm(a, w, DTYPES[dtype], y=big[1:m + 1, off:off + n])
        assert torch.equal(big[1:m + 1, off:off + n], want)
        big[1:m + 1, off:off + n] = 7.0
        assert (big == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(130, 200, 128), (2432, 4096, 128), (2250, 4096, 128), (2250, 4096, 4096)])
def test_gemm_keeps_what_is_not_a_number_apart(qsm, m, n, k):
    x, z = ref.draw(m, k, 5), ref.draw(n, k, 6)
    want = qsm.mx4_gemm(mx4(qsm, x)[0], mx4(qsm, z)[0])
    x[7, 40], z[150, 100] = math.nan, math.inf
    y = qsm.mx4_gemm(qsm.mx4_quantize(x), qsm.mx4_quantize(z))
    assert torch.isnan(y[7]).all() and torch.isnan(y[:, 150]).all()
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[7], keep[:, 150] = False, False
    assert torch.equal(y[keep], want[keep])


def test_gemm_refuses(qsm):
    a, _ = mx4(qsm, ref.draw(4, 64, 1))
    w, _ = mx4(qsm, ref.draw(4, 96, 1))
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemm(a, w)
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemm(a, a, torch.float16)
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemm(a, a, y=torch.empty(4, 5, dtype=torch.bfloat16, device="cuda"))


def block_max(x):
    b = x.abs().reshape(x.shape[0], -1, 32)
    return b.amax(dim=2, keepdim=True).expand_as(b).reshape(x.shape)


def rows_bound(x, w):
    return 2.0 ** -16 * (block_max(x) @ w.abs().T) + product_bound(x, w)


# one stage and less, splits of K over 2, 4 and 8 CTAs, a ragged last stage,
# more rows than fit at once
GEMV = [(1, 1, 32), (1, 512, 2048), (2, 130, 96), (3, 200, 512), (7, 300, 1056), (8, 2048, 2048),
        (9, 129, 4064), (17, 1000, 288), (32, 640, 2048), (31, 257, 8192), (32, 200, 16384), (5, 40000, 256),
        (29, 19500, 2048), (32, 19456, 2560)]   # in halves


@pytest.mark.parametrize("t,n,k", GEMV)
def test_gemv(qsm, t, n, k):
    x = ref.draw(t, k, t + k, spread=6).to(torch.bfloat16)
    w, wv = mx4(qsm, ref.draw(n, k, n))
    st = status()
    y = qsm.mx4_gemv(x, w, dev_status=st)
    xv = x.double()
    want = xv @ wv.T
    assert near(y, want, rows_bound(xv, wv)).all()
    assert torch.equal(y, qsm.mx4_gemv(x, w))
    assert st.item() == 0


def test_gemv_is_exact_where_it_can_be(qsm):
    """One-hot rows give the weights themselves; so do rows whose blocks span
    at most eight binades, up to the bf16 result (K one block: no sums)."""
    w, wv = mx4(qsm, ref.draw(300, 256, 4))
    x = torch.zeros(32, 256, dtype=torch.bfloat16, device="cuda")
    cols = torch.arange(32) * 8 + 3
    x[torch.arange(32), cols] = torch.tensor([(-1.0) ** i * (1 + i / 128) * 2.0 ** (i - 16) for i in range(32)],
                                             dtype=torch.bfloat16, device="cuda")
    want = x.double()[torch.arange(32), cols][:, None] * wv[:, cols].T
    assert torch.equal(qsm.mx4_gemv(x, w), want.to(torch.bfloat16))


def test_gemv_edges(qsm):
    w, wv = mx4(qsm, ref.draw(130, 128, 4))
    x = ref.draw(4, 128, 8).to(torch.bfloat16)
    x[0] = 0
    x[1, 5] = 2.0 ** 126                                # the largest exponent that is taken
    x[2, :] = 2.0 ** -133                               # a subnormal row
    st = status()
    y = qsm.mx4_gemv(x, w, dev_status=st)
    want = x.double() @ wv.T
    assert (y[0] == 0).all() and st.item() == 0
    big = rows_bound(x.double(), wv)
    # inputs under 2^-111 are kept to 2^-127
    big[2] += 128 * 2.0 ** -127 * wv.abs().amax()
    assert near(y, want, big)[:3].all()
    for what in (math.inf, math.nan, 2.0 ** 127):
        z = x.clone()
        z[1, 5] = what
        st = status()
        v = qsm.mx4_gemv(z, w, dev_status=st)
        assert st.item() == qsm.DEV_NONFINITE and torch.isnan(v[1]).all()
        assert torch.equal(v[[0, 2, 3]], y[[0, 2, 3]])


def test_gemv_strided_rows_and_refusals(qsm):
    w, _ = mx4(qsm, ref.draw(130, 128, 4))
    big = ref.draw(9, 512, 8).to(torch.bfloat16)
    x = big[::2, 128:256]
    assert torch.equal(qsm.mx4_gemv(x, w), qsm.mx4_gemv(x.contiguous(), w))
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemv(torch.zeros(33, 128, dtype=torch.bfloat16, device="cuda"), w)
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemv(big[:, :160], w)
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemv(big[:, :128].float(), w)
    with pytest.raises(qsm.QSMError):
        qsm.mx4_gemv(big[:, 4:132], w)                  # not 16-byte aligned


# ------------------------------------------------------------------ MoE layer

def layer(qsm, H, I, E, k, seed, bias=False, gate=False):
    def weights(e, rows, cols, s):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed * 16 + s)
        w = torch.randn((e * rows, cols), generator=g, device="cuda") * cols ** -0.5
        t, v = mx4(qsm, w, e)
        return t, v.reshape(e, rows, cols)
    q, v = zip(*(weights(e, r, c, s) for s, (e, r, c) in
                 enumerate([(E, 2 * I, H), (E, H, I), (1, 2 * I, H), (1, H, I)])))
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + 9)
    router = torch.randn((E, H), generator=g, device="cuda") * 0.05
    b = torch.randn(E, generator=g, device="cuda") * 2 if bias else None
    sg = torch.randn(H, generator=g, device="cuda") * 0.05 if gate else None
    return qsm.Mx4Layer(H, I, E, k, *q, router, b, sg), v


def hidden(T, H, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)


def check_layer(qsm, L, v, x, acts, renormalize=True, bias_select_only=False, f=None):
    f = f or qsm.Mx4Forward(L, x.shape[0], acts, renormalize=renormalize, want_f32=True,
                            bias_select_only=bias_select_only)
    y = f(x)
    torch.cuda.synchronize()
    assert f.dev_status.item() == 0
    idx, w = qsm.moe_route(x, L.w_router, L.k, L.logit_bias, renormalize, bias_select_only=bias_select_only)
    assert torch.equal(f.topk_idx, idx) and torch.equal(f.topk_w, w)   # the router's bits
    want = ref.moe(x, idx.long(), w, *v, gate=L.shared_gate, four=acts == "mx4")
    d = f.y_f32.double() - want
    if acts == "mx4":
        assert (d.norm() / want.norm()).item() <= 3e-3
    else:
        assert (d.abs().max() / want.abs().max()).item() <= 2e-3
    assert torch.equal(y, f.y_f32.to(torch.bfloat16))
    return f, want


# one token and slots of fewer than eight; slots cut at eight tokens; every
# expert for every token; one expert; E past a warp's and a block's width;
# H of one column tile and of an odd number of them
MOE16 = [(1, 128, 128, 4, 1), (1, 2048, 512, 256, 8), (2, 256, 128, 8, 8), (5, 384, 256, 16, 2),
         (8, 2048, 512, 64, 8), (9, 640, 384, 8, 3), (33, 256, 128, 1, 1), (40, 2048, 512, 256, 8),
         (64, 512, 128, 300, 9), (17, 4096, 256, 8, 2),
         # one launch: ragged quarters of H, experts that do not fill a warp, most
         # experts per token, one expert, an odd number of stages of I
         (1, 896, 256, 8, 8), (2, 2048, 512, 256, 8), (2, 1024, 128, 64, 32), (1, 4096, 384, 33, 5),
         (2, 1152, 640, 1, 1), (1, 2048, 128, 256, 1)]


@pytest.mark.parametrize("t,h,i,e,k", MOE16)
def test_moe_16_bit_activations(qsm, t, h, i, e, k):
    L, v = layer(qsm, h, i, e, k, seed=t)
    check_layer(qsm, L, v, hidden(t, h, t + 1), "bf16")


MOE4 = [(1, 128, 128, 4, 1), (3, 256, 128, 8, 8), (64, 640, 384, 16, 2), (65, 2048, 512, 256, 8),
        (129, 256, 128, 1, 1), (300, 384, 256, 24, 5), (260, 512, 128, 300, 9), (1000, 2048, 512, 64, 8)]


@pytest.mark.parametrize("t,h,i,e,k", MOE4)
def test_moe_4_bit_activations(qsm, t, h, i, e, k):
    L, v = layer(qsm, h, i, e, k, seed=t)
    check_layer(qsm, L, v, hidden(t, h, t + 1), "mx4")


@pytest.mark.parametrize("acts", ["bf16", "mx4"])
@pytest.mark.parametrize("renormalize,select_only", [(False, False), (True, True), (False, True)])
def test_moe_routing_variants_and_gate(qsm, acts, renormalize, select_only):
    L, v = layer(qsm, 256, 128, 16, 4, seed=3, bias=True, gate=True)
    check_layer(qsm, L, v, hidden(37, 256, 4), acts, renormalize, select_only)


@pytest.mark.parametrize("acts", ["bf16", "mx4"])
def test_moe_uneven_and_empty_experts(qsm, acts):
    """A bias that sends every token to the same experts: long groups (cut into
    slots and blocks) beside empty ones."""
    L, v = layer(qsm, 256, 128, 32, 3, seed=5)
    L.logit_bias = torch.zeros(32, device="cuda")
    L.logit_bias[[0, 7, 31]] = 100.0
    T = 64 if acts == "bf16" else 400
    f, _ = check_layer(qsm, L, v, hidden(T, 256, 6), acts)
    assert set(f.topk_idx.unique().tolist()) == {0, 7, 31}


@pytest.mark.parametrize("acts", ["bf16", "mx4"])
def test_moe_calls_do_not_depend_on_one_another(qsm, acts):
    L, v = layer(qsm, 512, 256, 16, 4, seed=7)
    T = 24
    xs = [hidden(T, 512, s) for s in range(3)]
    f = qsm.Mx4Forward(L, T, acts, want_f32=True)
    outs = []
    for x in xs + xs:
        outs.append(f(x).clone())
    for a, b in zip(outs[:3], outs[3:]):
        assert torch.equal(a, b)                         # the same bits, whatever ran between
    check_layer(qsm, L, v, xs[1], acts, f=f)
    # a token's routing and (16-bit activations) result do not need the others
    y1 = qsm.Mx4Forward(L, 1, acts)(xs[0][5:6].contiguous())
    assert (y1.double() - outs[0][5:6].double()).norm() <= 1e-2 * y1.double().norm()


def test_moe_one_launch_routing_variants(qsm):
    """The one-launch form, many calls on one workspace: other inputs each
    time, the same bits for the same ones."""
    L, v = layer(qsm, 1024, 256, 48, 6, seed=11, bias=True, gate=True)
    for t in (1, 2):
        for renorm, only in ((True, False), (False, True)):
            f = qsm.Mx4Forward(L, t, renormalize=renorm, bias_select_only=only, want_f32=True)
            first = None
            for s in (1, 2, 3, 1):
                f, _ = check_layer(qsm, L, v, hidden(t, 1024, s), "bf16", renorm, only, f=f)
                first = f.y_f32.clone() if first is None else first
            assert torch.equal(f.y_f32, first)


def test_moe_one_launch_timeout_is_reported(qsm):
    """A wait that nothing ends runs out, the call reports it and returns, and
    the context and (zeroed) workspace go on working."""
    L, v = layer(qsm, 1024, 128, 16, 2, seed=12)
    f = qsm.Mx4Forward(L, 1, want_f32=True)
    x = hidden(1, 1024, 3)
    want = f(x).clone()
    torch.cuda.synchronize()
    qsm.debug_barrier_skew(1)
    try:
        f(x)
        torch.cuda.synchronize()
    finally:
        qsm.debug_barrier_skew(0)
    assert f.dev_status.item() & qsm.DEV_TIMEOUT
    f.dev_status.zero_()
    f.workspace.zero_()
    assert torch.equal(f(x), want)
    check_layer(qsm, L, v, x, "bf16", f=f)


@pytest.mark.parametrize("acts,t,h", [("bf16", 1, 1024), ("bf16", 3, 256), ("bf16", 20, 256), ("mx4", 100, 256)])
def test_moe_on_another_stream_and_in_a_graph(qsm, acts, t, h):
    L, v = layer(qsm, h, 128, 16, 2, seed=8)
    f = qsm.Mx4Forward(L, t, acts, want_f32=True)
    x = hidden(t, h, 1)
    want = f(x).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(want)
    f(x, stream=s, out=out)
    s.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f(x)
        with torch.cuda.graph(g, stream=s):
            f(x)
            y = qsm.mx4_gemv(x[:2], L.shared_gate_up)
    xn = hidden(t, h, 2)
    x.copy_(xn)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(f.y, f(xn)) and torch.equal(y, qsm.mx4_gemv(xn[:2], L.shared_gate_up))


def test_moe_not_finite_tokens_stay_apart(qsm):
    """A token that holds an infinity sets the status and spoils its own row."""
    L, v = layer(qsm, 256, 128, 16, 2, seed=9)
    for acts, T in (("bf16", 12), ("mx4", 90)):
        x = hidden(T, 256, 3)
        f = qsm.Mx4Forward(L, T, acts)
        want = f(x).clone()
        x[4, 9] = math.inf
        y = f(x)
        torch.cuda.synchronize()
        assert f.dev_status.item() & qsm.DEV_NONFINITE
        keep = torch.arange(T, device="cuda") != 4
        assert not torch.isfinite(y[4]).any()
        assert torch.equal(y[keep], want[keep])


def test_moe_outputs_out_of_fp16_range_are_reported(qsm):
    L, _ = layer(qsm, 256, 128, 4, 1, seed=2)
    x = hidden(70, 256, 3)
    x *= 2.0 ** 20
    f = qsm.Mx4Forward(L, 70, "mx4")
    f(x)
    torch.cuda.synchronize()
    assert f.dev_status.item() & qsm.DEV_FP16_RANGE


def test_moe_refuses(qsm):
    L, _ = layer(qsm, 256, 128, 8, 2, seed=1)
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Forward(L, 65, "bf16")
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Forward(L, 4, "fp8")
    f = qsm.Mx4Forward(L, 4)
    for bad in (hidden(5, 256, 1), hidden(4, 256, 1).float(), hidden(4, 512, 1)[:, ::2]):
        with pytest.raises(qsm.QSMError):
            f(bad)
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Layer.quantize(200, 128, 8, 2, *(torch.zeros(1, 4, 64, device="cuda"),) * 4, None)
    assert f(hidden(4, 256, 1)).shape == (4, 256)
    assert qsm.Mx4Forward(L, 0)(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")).shape == (0, 256)


def test_refuses_what_is_on_the_host_or_of_another_type(qsm):
    """No launch may ever see a host address or a short array."""
    L, _ = layer(qsm, 256, 128, 8, 2, seed=1)
    f = qsm.Mx4Forward(L, 4)
    x = hidden(4, 256, 1)
    for call in (lambda: f(x.cpu()), lambda: f(x, out=torch.empty(4, 256, dtype=torch.bfloat16)),
                 lambda: qsm.mx4_quantize(x.cpu()), lambda: qsm.mx4_gemv(x.cpu(), L.shared_gate_up),
                 lambda: qsm.mx4_gemv(x, L.shared_gate_up, dev_status=torch.zeros(1, dtype=torch.int32)),
                 lambda: qsm.mx4_quantize(x, dev_status=torch.zeros(1, device="cuda"))):
        with pytest.raises(qsm.QSMError):
            call()
    good = L.w_router
    for bad in (good.cpu(), good.double(), good[:7], good.t(), None):
        L.w_router = bad
        with pytest.raises(qsm.QSMError):
            qsm.Mx4Forward(L, 4)
    L.w_router, L.logit_bias = good, torch.zeros(7, device="cuda")
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Forward(L, 4)
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Layer(256, 128, 8, 2, L.gate_up, L.down, L.shared_gate_up, L.shared_down, good,
                     shared_gate=torch.zeros(256, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Forward(L, -1)
    assert qsm.moe_mx4_workspace_bytes(L, 4, "fp8") == 0


def test_layer_from_dense_weights(qsm):
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    def r(*s):
        return torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16) * 0.05
    w = (r(6, 256, 384), r(6, 384, 128), r(1, 256, 384), r(1, 384, 128))
    L = qsm.Mx4Layer.quantize(384, 128, 6, 2, *w, torch.randn((6, 384), generator=g, device="cuda") * 0.05)
    v = [ref.rounded(t) for t in w]
    check_layer(qsm, L, v, hidden(7, 384, 5), "bf16")


def test_example_runs(qsm):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "mx4_generate.py"), "--steps", "3"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens" in r.stdout
