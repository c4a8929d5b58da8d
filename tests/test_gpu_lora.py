"""Low-rank adapters on the GPU against the formula in 64 bits.

Tolerance (fixed before the first run).  v = A x: products are exact, a sum is at most K / 128 fp32
additions in a warp and 40 more (inside an MMA, over the warps, over the cluster), each off by at
most 2^-23 (the tensor cores may truncate) of sum |a x|.  c v is rounded to fp32 and split: 2^-17 of
|c v| for bf16 outputs, 2^-23 for fp32 ones.  The second product has at most rank / 4 + 40 additions
of 2^-23 of sum |c v b|, and y is added with one more rounding; out is the rounding of that."""
import pytest
import torch

import _block_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def randn(*shape, seed):
    return torch.randn(shape, generator=gen(seed), device="cuda")


def adapters(qsm, n, rank, K, N, seed, mixed=True, scale=True):
    """Ranks that do not count hold NaN."""
    a = (randn(n, rank, K, seed=seed) * K ** -0.5).bfloat16()
    b = (randn(n, N, rank, seed=seed + 1) * rank ** -0.5).bfloat16()
    s = randn(n, seed=seed + 2) if scale else None
    r = None
    if mixed:
        r = torch.randint(0, rank + 1, (n,), generator=gen(seed + 3), device="cuda").int()
        for i, m in enumerate(r.tolist()):
            a[i, m:], b[i, :, m:] = float("nan"), float("nan")
    return qsm.LoraAdapters(a, b, s, r)


def definition(x, L, ids, y, dtype):
    """(out, bound) in 64 bits."""
    T = x.shape[0]
    out = torch.zeros(T, L.N, dtype=torch.float64, device="cuda") if y is None else y.double()
    err = torch.zeros_like(out)
    split = 2.0 ** -17 if dtype is torch.bfloat16 else 2.0 ** -23
    for i in range(L.n):
        t = torch.nonzero(ids == i)[:, 0]
        r = L.rank if L.ranks is None else L.ranks[i].item()
        if not len(t) or not r:
            continue
        a, b = L.a[i, :r].double(), L.b[i, :, :r].double()
        c = 1.0 if L.scale is None else L.scale[i].double()
        xv = x[t].double()
        v, dv = xv @ a.T * c, (L.K / 128 + 40) * 2 * U * (xv.abs() @ a.abs().T) * abs(c)
        dv = dv + (split + 2 * U) * v.abs()
        out[t] += v @ b.T
        err[t] = dv @ b.abs().T + (r / 4 + 40) * 2 * U * ((v.abs() + dv) @ b.abs().T)
    return out.cpu(), (err + 2 * U * (out.abs() + err)).cpu()


def check(qsm, T, L, seed, dtype=torch.bfloat16, none=0.2, ids=None, y=True):
    x = randn(T, L.K, seed=seed).bfloat16()
    if ids is None:
        ids = torch.randint(0, L.n, (T,), generator=gen(seed + 1), device="cuda").int()
        ids[torch.rand(T, generator=gen(seed + 2), device="cuda") < none] = -1
    base = randn(T, L.N, seed=seed + 3).to(dtype) if y else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qsm.lora_add(x, L, ids, base, dtype=dtype, dev_status=st)
    want, err = definition(x, L, ids, base, dtype)
    assert out.dtype == dtype and ref.lies_between(out, want, err)
    if base is not None and bool((ids < 0).any()):
        assert torch.equal(out[ids < 0], base[ids < 0])
    assert st.item() == 0
    return x, ids, base, out


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 33, 63, 64, 65, 130, 400])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tokens(qsm, T, dtype):
    check(qsm, T, adapters(qsm, 5, 64, 512, 320, 1), 2, dtype)


@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("K,N", [(8, 1), (40, 7), (264, 33), (2048, 2050), (1000, 96), (8192, 264)])
def test_shapes(qsm, rank, K, N):
    for T, dtype in ((1, torch.float32), (20, torch.bfloat16), (100, torch.float32)):
        check(qsm, T, adapters(qsm, 3, rank, K, N, T, mixed=rank % 16 == 8, scale=N % 2 == 0), 5, dtype)


def test_one_adapter_each_and_all_the_same(qsm):
    L = adapters(qsm, 64, 32, 2048, 512, 7, mixed=False)
    for T in (64, 200):
        check(qsm, T, L, 8, ids=(torch.arange(T, device="cuda") % 64).int())
        check(qsm, T, L, 9, ids=torch.full((T,), 63, device="cuda").int())
        check(qsm, T, L, 10, ids=torch.full((T,), -1, device="cuda").int())
        check(qsm, T, L, 11, y=False)
        check(qsm, T, L, 11, torch.float32, y=False)


def test_packed_prompts(qsm):
    L = adapters(qsm, 4, 64, 1024, 1032, 12)
    ids = torch.repeat_interleave(torch.tensor([2, 0, -1, 3, 2, 1]), torch.tensor([100, 1, 63, 300, 64, 72])).int().cuda()
    check(qsm, 600, L, 13, ids=ids)
    check(qsm, 600, L, 13, torch.float32, ids=ids)


def test_values_of_more_than_sixteen_bits_pass(qsm):
    """fp32 outputs: A x up to 2^22 in whole numbers, B a unit matrix: exact."""
    K, R = 1024, 32
    a = torch.randint(-64, 65, (2, R, K), generator=gen(1), device="cuda").bfloat16()
    x = torch.randint(-64, 65, (9, K), generator=gen(2), device="cuda").bfloat16()
    L = qsm.LoraAdapters(a, torch.eye(R, device="cuda").bfloat16().repeat(2, 1, 1))
    ids = (torch.arange(9, device="cuda") % 2).int()
    out = qsm.lora_add(x, L, ids, dtype=torch.float32)
    want = torch.einsum("tk,trk->tr", x.double(), a[ids.long()].double())
    assert want.abs().max() > 1 << 16 and torch.equal(out.double(), want)


def test_ids_out_of_range_count_as_none(qsm):
    L = adapters(qsm, 3, 16, 64, 40, 14, mixed=False)
    x, y = randn(70, 64, seed=15).bfloat16(), randn(70, 40, seed=16).bfloat16()
    ids = torch.zeros(70, dtype=torch.int32, device="cuda")
    good = qsm.lora_add(x, L, ids, y)
    ids[3], ids[66], ids[10], ids[11] = 3, 2 ** 31 - 1, -5, -2 ** 31
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qsm.lora_add(x, L, ids, y, dev_status=st)
    odd = [3, 66, 10, 11]
    rest = [t for t in range(70) if t not in odd]
    assert st.item() == 16 and torch.equal(out[odd], y[odd]) and torch.equal(out[rest], good[rest])


def test_ranks_out_of_range_are_taken_into_it(qsm):
    L = adapters(qsm, 2, 16, 64, 40, 17, mixed=False)
    x, ids = randn(6, 64, seed=18).bfloat16(), torch.tensor([0, 1, 0, 1, 0, 1], device="cuda").int()
    y = randn(6, 40, seed=19).bfloat16()
    M = qsm.LoraAdapters(L.a, L.b, L.scale, torch.tensor([99, -3], device="cuda").int())
    out, full = qsm.lora_add(x, M, ids, y), qsm.lora_add(x, L, ids, y)
    assert torch.equal(out[ids == 0], full[ids == 0]) and torch.equal(out[ids == 1], y[ids == 1])


def test_values_that_are_not_finite_stay_with_their_tokens(qsm):
    L = adapters(qsm, 2, 16, 128, 64, 20, mixed=False)
    x, ids = randn(12, 128, seed=21).bfloat16(), (torch.arange(12, device="cuda") % 2).int()
    y = randn(12, 64, seed=22).bfloat16()
    want = qsm.lora_add(x, L, ids, y)
    bad = x.clone()
    bad[4, 7], bad[5, 9] = float("nan"), float("inf")
    out = qsm.lora_add(bad, L, ids, y)
    keep = [t for t in range(12) if t not in (4, 5)]
    assert torch.equal(out[keep], want[keep]) and out[4].isnan().all() and not out[5].isfinite().any()
    # an infinite A x times a single column of B: the infinity comes through as one
    one = qsm.LoraAdapters(torch.ones(1, 8, 8, device="cuda").bfloat16(), torch.ones(1, 8, 8, device="cuda").bfloat16(),
                           None, torch.ones(1, device="cuda").int())
    v = torch.zeros(1, 8, device="cuda").bfloat16()
    v[0, 0] = float("inf")
    for dt in (torch.bfloat16, torch.float32):
        assert (qsm.lora_add(v, one, torch.zeros(1, device="cuda").int(), dtype=dt) == float("inf")).all()


def test_a_token_does_not_depend_on_the_others(qsm):
    L = adapters(qsm, 4, 32, 512, 256, 23, mixed=False)
    T = 50
    x, y = randn(T, 512, seed=24).bfloat16(), randn(T, 256, seed=25).float()
    ids = torch.randint(0, 4, (T,), generator=gen(26), device="cuda").int()
    out = qsm.lora_add(x, L, ids, y)
    z, other = randn(T, 512, seed=27).bfloat16(), torch.randint(-1, 4, (T,), generator=gen(28), device="cuda").int()
    z[17], other[17] = x[17], ids[17]
    assert torch.equal(qsm.lora_add(z, L, other, y)[17], out[17])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N", [256, 131])
def test_layouts(qsm, dtype, N):
    L = adapters(qsm, 3, 16, 128, N, 29, mixed=False)
    T = 37
    x, ids, y, want = check(qsm, T, L, 30, dtype)
    z = y.clone()
    assert qsm.lora_add(x, L, ids, z, out=z) is z and torch.equal(z, want)
    m = torch.full((T, 3 * N + 5), 7.0, dtype=dtype, device="cuda")
    m[:, :N] = y
    qsm.lora_add(x, L, ids, m[:, :N], out=m[:, N + 1:2 * N + 1])
    assert torch.equal(m[:, N + 1:2 * N + 1], want) and torch.equal(m[:, :N], y)
    assert (m[:, N] == 7).all() and (m[:, 2 * N + 1:] == 7).all()
    w = torch.full((T, 128 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    w[:, 8:136] = x
    assert torch.equal(qsm.lora_add(w[:, 8:136], L, ids, y), want)
    big = torch.full((T + 2, N), 7.0, dtype=dtype, device="cuda")
    qsm.lora_add(x, L, ids, y, out=big[:T])
    assert torch.equal(big[:T], want) and (big[T:] == 7).all()
    e = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    assert qsm.lora_add(e, L, ids[:0], y[:0]).shape == (0, N)


def test_streams_and_a_graph(qsm):
    L = adapters(qsm, 3, 16, 256, 512, 31, mixed=False)
    x, ids, y, want = check(qsm, 20, L, 32)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = qsm.lora_add(x, L, ids, y, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = qsm.lora_add(x, L, ids, y)
    x.copy_(randn(20, 256, seed=33).bfloat16())
    ids.copy_(torch.randint(-1, 3, (20,), generator=gen(34), device="cuda").int())
    L.a[1] *= 2                                # an adapter that is loaded anew
    want = qsm.lora_add(x, L, ids, y)
    g.replay()
    assert torch.equal(out, want)


def test_refusals(qsm):
    L = adapters(qsm, 3, 16, 64, 40, 35, mixed=False)
    x, y, ids = randn(4, 64, seed=36).bfloat16(), randn(4, 40, seed=37).bfloat16(), torch.zeros(4, device="cuda").int()
    f = qsm.lora_add
    for bad in (lambda: f(x.float(), L, ids, y), lambda: f(x[:, :32], L, ids, y), lambda: f(x.cpu(), L, ids, y),
                lambda: f(x, L, ids.long(), y), lambda: f(x, L, ids[:3], y), lambda: f(x, L, ids.cpu(), y),
                lambda: f(x, L, ids, y.half()), lambda: f(x, L, ids, y[:, :32]), lambda: f(x, L, ids, y, dtype=torch.float32),
                lambda: f(x, L, ids, y, out=y.float()), lambda: f(x, L, ids, y, out=y[:3]), lambda: f(x, L, ids, dtype=torch.float16),
                lambda: f(x, L, ids, y.t().contiguous().t()), lambda: f(x, L, ids, y, dev_status=ids.long())):
        with pytest.raises(qsm.QSMError):
            bad()
    a, b = L.a, L.b
    for bad in (dict(a=a[:, :, :63], b=b), dict(a=a.float(), b=b), dict(a=a, b=b[:, :, :8]), dict(a=a[:, :, ::2], b=b),
                dict(a=a, b=b, scale=torch.ones(2, device="cuda")), dict(a=a, b=b, ranks=torch.ones(3, device="cuda")),
                dict(a=a, b=b, ranks=torch.ones(3).int())):
        with pytest.raises(qsm.QSMError):
            qsm.LoraAdapters(**bad)
    with pytest.raises(AttributeError):
        L.a = a.clone()


@pytest.mark.parametrize("off", [0, 8, 16])
@pytest.mark.parametrize("K,N", [(4096, 2048), (4104, 2056), (8192, 96)])
def test_rows_on_every_16_bytes(qsm, off, K, N):
    """a, x, y and out at addresses and strides that are or are not multiples of 32 bytes."""
    n, R = 2, 16
    def view(shape, seed, dtype=torch.bfloat16, pad=off):
        t = torch.empty(shape[0], shape[1] + pad, dtype=dtype, device="cuda").fill_(float("nan"))
        t[:, pad:] = randn(*shape, seed=seed).to(dtype) * shape[1] ** -0.5
        return t[:, pad:]
    buf = torch.empty(n * R * K + 16, dtype=torch.bfloat16, device="cuda")
    a = buf[off:off + n * R * K].view(n, R, K)
    a.copy_(randn(n, R, K, seed=1) * K ** -0.5)
    L = qsm.LoraAdapters(a, (randn(n, N, R, seed=2) / 4).bfloat16())
    for T in (5, 40):
        x, y = view((T, K), 3), view((T, N), 4)
        out = torch.full((T, N + off), 7.0, dtype=torch.bfloat16, device="cuda")
        ids = (torch.arange(T, device="cuda") % 3 - 1).int()
        qsm.lora_add(x, L, ids, y, out=out[:, off:])
        want, err = definition(x, L, ids, y, torch.bfloat16)
        assert ref.lies_between(out[:, off:], want, err) and (out[:, :off] == 7).all()


def test_offsets_that_pass_32_bits(qsm):
    """Adapters, x and y past 2^32 elements; the last ones as a call of their own."""
    n, R, K, N = 70, 128, 1 << 19, 24
    a = torch.zeros((n, R, K), dtype=torch.bfloat16, device="cuda")
    a[-1] = 1
    b = torch.ones((n, N, R), dtype=torch.bfloat16, device="cuda")
    x = torch.zeros((3, K), dtype=torch.bfloat16, device="cuda")
    x[:, ::1024] = 1
    ids = torch.tensor([n - 1, 0, -1], device="cuda").int()
    out = qsm.lora_add(x, qsm.LoraAdapters(a, b), ids, dtype=torch.float32)
    assert (out[0] == K // 1024 * R).all() and not out[1:].any()    # whole numbers: exact
    del a, x
    T, N = (1 << 18) + 37, (1 << 14) + 8
    L = adapters(qsm, 2, 8, 64, N, 50, mixed=False)
    x = randn(T, 64, seed=51).bfloat16()
    y = torch.zeros((T, N), dtype=torch.bfloat16, device="cuda")
    y[-40:] = randn(40, N, seed=52).bfloat16()
    ids = torch.full((T,), -1, device="cuda").int()
    ids[-40:] = (torch.arange(40, device="cuda") % 3 - 1).int()
    tail = x[-40:].clone(), ids[-40:].clone(), y[-40:].clone()
    want, err = definition(tail[0], L, tail[1], tail[2], torch.bfloat16)
    qsm.lora_add(x, L, ids, y, out=y)
    assert ref.lies_between(y[-40:], want, err) and not y[:-40].any()


@pytest.mark.parametrize("T,n", [(65, 1), (300, 40), (600, 500), (1000, 1023), (100, 1100), (700, 2000), (16500, 9)])
def test_adapters_in_any_order(qsm, T, n):
    """More items than run at once, tokens of an adapter anywhere, more adapters than a CTA counts
    (1100, 2000), more tokens than it looks through (16500); out over y, ids out of range."""
    L = adapters(qsm, n, 8, 64, 40, 60, mixed=False)
    x, y = randn(T, 64, seed=61).bfloat16(), randn(T, 40, seed=62).bfloat16()
    ids = torch.randint(-1, n, (T,), generator=gen(63), device="cuda").int()
    if T > 2000:
        ids[:9000] = 3
    used = {i: torch.nonzero(ids == i)[:, 0] for i in set(ids.tolist()) if i >= 0}
    want, err = y.double(), torch.zeros(T, 40, dtype=torch.float64, device="cuda")
    for i, t in used.items():   # the bound of definition(), adapter by adapter
        a, b, c, xv = L.a[i].double(), L.b[i].double(), L.scale[i].double(), x[t].double()
        v, dv = xv @ a.T * c, (64 / 128 + 40) * 2 * U * (xv.abs() @ a.abs().T) * abs(c)
        dv = dv + (2.0 ** -17 + 2 * U) * v.abs()
        want[t] += v @ b.T
        err[t] = dv @ b.abs().T + 42 * 2 * U * ((v.abs() + dv) @ b.abs().T)
    err = err + 2 * U * (want.abs() + err)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qsm.lora_add(x, L, ids, y, dev_status=st)
    assert ref.lies_between(out, want.cpu(), err.cpu()) and st.item() == 0
    assert torch.equal(out[ids < 0], y[ids < 0])
    bad = torch.where(ids < 0, n + 5, ids)
    z = y.clone()
    qsm.lora_add(x, L, bad, z, out=z, dev_status=st)
    assert torch.equal(z, out) and st.item() == (16 if (ids < 0).any() else 0)


@pytest.mark.parametrize("rank", [8, 40, 64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,n,N", [(100, 1100, 40), (700, 2000, 41), (130, 1030, 72), (16500, 9, 40), (16500, 3, 33)])
def test_tiles_one_after_another(qsm, rank, dtype, T, n, N):
    """More than 64 tokens that are not grouped by adapter (too many adapters, or tokens): several tiles, and
    clusters that take many slots in turn, at every number of ranks."""
    L = adapters(qsm, n, rank, 72, N, 70, scale=N % 2 == 0)
    x = randn(T, 72, seed=75).bfloat16()
    ids = torch.randint(-1, n, (T,), generator=gen(76), device="cuda").int()
    if T > 2000:
        ids[:9000] = 2
    y = randn(T, N, seed=77).to(dtype)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = qsm.lora_add(x, L, ids, y, dev_status=st)
    # the bound of definition(), all tokens at once
    a, b = L.a.double().nan_to_num(0), L.b.double().nan_to_num(0)
    i = ids.long().clamp_min(0)
    c = (ids >= 0).double()[:, None] * (1.0 if L.scale is None else L.scale.double()[i][:, None])
    split = 2.0 ** -17 if dtype is torch.bfloat16 else 2.0 ** -23
    want, err = y.double(), torch.zeros(T, N, dtype=torch.float64, device="cuda")
    for t in torch.arange(T, device="cuda").split(500):
        at, bt, xt = a[i[t]], b[i[t]], x[t].double()
        v = torch.einsum("tk,trk->tr", xt, at) * c[t]
        dv = (72 / 128 + 40) * 2 * U * torch.einsum("tk,trk->tr", xt.abs(), at.abs()) * c[t].abs() + (split + 2 * U) * v.abs()
        want[t] += torch.einsum("tr,tnr->tn", v, bt)
        err[t] = torch.einsum("tr,tnr->tn", dv, bt.abs()) + (rank / 4 + 40) * 2 * U * torch.einsum("tr,tnr->tn", v.abs() + dv, bt.abs())
    err = err + 2 * U * (want.abs() + err)
    assert ref.lies_between(out, want.cpu(), err.cpu()) and st.item() == 0
    assert torch.equal(out[ids < 0], y[ids < 0])


@pytest.mark.parametrize("R", [24, 32, 64, 128])
@pytest.mark.parametrize("T,n", [(5, 2), (40, 3), (64, 2), (200, 3), (200, 1100), (16500, 5)])
def test_whole_numbers_are_exact(qsm, R, T, n):
    """fp32 outputs: A x up to 2^22 in whole numbers, a row of B with a single one of 1, -2 or 4: exact,
    whichever way the second product takes (slots, items or tiles; rows of whole 16-byte units or not)."""
    K = 1024
    a = torch.randint(-64, 65, (n, R, K), generator=gen(1), device="cuda").bfloat16()
    x = torch.randint(-64, 65, (T, K), generator=gen(2), device="cuda").bfloat16()
    ids = torch.randint(0, n, (T,), generator=gen(3), device="cuda").int()
    v = torch.cat([torch.einsum("tk,trk->tr", x[t].float(), a[ids[t].long()].float()).double()   # whole: exact in fp32
                   for t in torch.arange(T, device="cuda").split(256)])
    assert v.abs().max() > 1 << 16 and v.abs().max() < 1 << 22
    for N in (R, R + 5, 2 * R + 8):
        row = torch.arange(N, device="cuda")
        b = torch.zeros(n, N, R, device="cuda")
        factor = torch.tensor([1.0, -2.0, 4.0], device="cuda")[row % 3]
        b[:, row, (row * 7 + 3) % R] = factor
        L = qsm.LoraAdapters(a, b.bfloat16())
        want = v[:, (row * 7 + 3) % R] * factor.double()
        assert torch.equal(qsm.lora_add(x, L, ids, dtype=torch.float32).double(), want)
        y = torch.randint(-64, 65, (T, N), generator=gen(4), device="cuda").float()
        assert torch.equal(qsm.lora_add(x, L, ids, y).double(), want + y.double())


@pytest.mark.parametrize("T,n", [(50, 4), (500, 4), (500, 1100)])
@pytest.mark.parametrize("rank", [16, 64])
def test_a_token_does_not_depend_on_the_others_values(qsm, T, n, rank):
    """The others' x and y change, the ids stay: the same bits, at a K of many blocks for each warp."""
    L = adapters(qsm, n, rank, 8192, 264, 90, mixed=False)
    ids = torch.randint(-1, 4, (T,), generator=gen(91), device="cuda").int()
    x, y = randn(T, 8192, seed=92).bfloat16(), randn(T, 264, seed=93)
    out = qsm.lora_add(x, L, ids, y)
    keep = torch.rand(T, generator=gen(94), device="cuda") < 0.1
    z = torch.where(keep[:, None], x, randn(T, 8192, seed=95).bfloat16())
    z[~keep, 5] = float("nan")
    w = torch.where(keep[:, None], y, randn(T, 264, seed=96))
    assert torch.equal(qsm.lora_add(z, L, ids, w)[keep], out[keep])
