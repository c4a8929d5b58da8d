"""The operators around the products with the layers and projections they stand beside: routed
by scores, both layers; and a decoding step through all of them, eager and captured.

Tolerances: the layers' own (tests/_gpu_cases.py, tests/test_gpu_mx4.py), for the routing that
the scores gave; norms, adapters and 4-bit products as in their tests, each on the values that the
call before it left."""
import pytest
import torch

import _block_ref as ref
import _gpu_cases as cases
import _mx4_ref
import synth

pytestmark = pytest.mark.gpu


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def mx4_layer(qsm, H, I, E, k, seed, router=True):
    def weights(e, rows, cols, s):
        w = torch.randn((e * rows, cols), generator=gen(seed * 16 + s), device="cuda") * cols ** -0.5
        t = qsm.mx4_quantize(w)
        v = qsm.mx4_dequantize(t, torch.float32).double().reshape(e, rows, cols)
        return qsm.Mx4Tensor(t.codes, t.scales, rows, cols, e), v
    q, v = zip(*(weights(e, r, c, s) for s, (e, r, c) in
                 enumerate([(E, 2 * I, H), (E, H, I), (1, 2 * I, H), (1, H, I)])))
    w = torch.randn((E, H), generator=gen(seed * 16 + 9), device="cuda") * 0.05
    return qsm.Mx4Layer(H, I, E, k, *q, w if router else None), v, w


@pytest.mark.parametrize("T", [1, 2, 3, 40, 65, 300])
def test_q8_layer_routed_by_scores(qsm, T):
    shape = synth.TINY
    Lg, q, wr, _ = cases.layer(shape)
    x = cases.x_for(shape, T, 3, Lg, wr, None).cuda()
    r = qsm.MoERouter(Lg.w_router, shape.k, "sigmoid", 0.1 * torch.randn(shape.E, generator=gen(1), device="cuda"),
                      groups=4, groups_kept=2, group_best=2, scale=2.5)
    L = qsm.Layer(shape.H, shape.I, shape.E, shape.k, Lg.gate_up, Lg.down, Lg.shared_gate_up, Lg.shared_down, None)
    f = qsm.MoEForward(L, T, want_f32=True, router=r)
    y = f(x)
    torch.cuda.synchronize()
    ids, w = qsm.moe_route_scores(x, r)
    assert torch.equal(f.topk_idx, ids) and torch.equal(f.topk_w, w) and f.dev_status.item() == 0
    err, _ = cases.check_layer_output(y, f.y_f32, x.cpu(), ids.cpu().numpy(), w.double().cpu().numpy(), q)
    assert err <= cases.TOL


@pytest.mark.parametrize("T,acts", [(1, "bf16"), (2, "bf16"), (9, "bf16"), (64, "bf16"), (1, "mx4"), (100, "mx4"), (300, "mx4")])
def test_mx4_layer_routed_by_scores(qsm, T, acts):
    H, I, E, k = 512, 256, 32, 4
    L, v, wr = mx4_layer(qsm, H, I, E, k, T, router=False)
    x = torch.randn((T, H), generator=gen(T), device="cuda").bfloat16()
    r = qsm.MoERouter(wr, k, "sigmoid", groups=8, groups_kept=3, group_best=2, scale=2.5)
    f = qsm.Mx4Forward(L, T, acts, want_f32=True, router=r)
    y = f(x)
    ids, w = qsm.moe_route_scores(x, r)
    assert torch.equal(f.topk_idx, ids) and torch.equal(f.topk_w, w) and f.dev_status.item() == 0
    want = _mx4_ref.moe(x, ids.long(), w, *v, four=acts == "mx4")
    d = f.y_f32.double() - want
    assert (d.norm() / want.norm()).item() <= 3e-3 if acts == "mx4" else (d.abs().max() / want.abs().max()).item() <= 2e-3
    assert torch.equal(y, f.y_f32.to(torch.bfloat16))
    out = x.clone()
    assert torch.equal(f(out, out=out), y)                # onto x itself


def test_a_softmax_router_gives_the_layers_own_result(qsm):
    T, H, I, E, k = 40, 512, 256, 32, 4
    L, _, wr = mx4_layer(qsm, H, I, E, k, 3)
    x = torch.randn((T, H), generator=gen(5), device="cuda").bfloat16()
    own, by = qsm.Mx4Forward(L, T, want_f32=True), qsm.Mx4Forward(L, T, want_f32=True, router=qsm.MoERouter(wr, k))
    own(x), by(x)
    assert torch.equal(own.topk_idx, by.topk_idx)
    # weights within 2e-5 of one another: so are the outputs, of terms up to ten times as large
    assert (own.y_f32 - by.y_f32).abs().max() <= 2e-5 * 10 * own.y_f32.abs().max()


def test_layers_refuse_other_routers(qsm):
    L, _, wr = mx4_layer(qsm, 512, 256, 32, 4, 3, router=False)
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Forward(L, 4)                              # no router at all
    for other in (qsm.MoERouter(wr, 3), qsm.MoERouter(wr[:16].contiguous(), 4), qsm.MoERouter(wr[:, :256].contiguous(), 4)):
        with pytest.raises(qsm.QSMError):
            qsm.Mx4Forward(L, 4, router=other)
        with pytest.raises(qsm.QSMError):
            qsm.MoEForward(type("L", (), dict(H=512, E=32, k=4))(), 4, router=other)
    f = qsm.Mx4Forward(L, 4, router=qsm.MoERouter(wr, 4))
    with pytest.raises(qsm.QSMError):
        f(torch.zeros(5, 512, dtype=torch.bfloat16, device="cuda"))


def test_q8_layer_routed_by_scores_refuses_strided_tokens(qsm):
    """The router takes rows at any stride, the expert products do not: nothing is launched."""
    shape = synth.TINY
    Lg, _, wr, _ = cases.layer(shape)
    r = qsm.MoERouter(Lg.w_router, shape.k)
    L = qsm.Layer(shape.H, shape.I, shape.E, shape.k, Lg.gate_up, Lg.down, Lg.shared_gate_up, Lg.shared_down, None)
    f = qsm.MoEForward(L, 4, router=r)
    f.topk_idx.fill_(-7)
    with pytest.raises(qsm.QSMError):
        f(torch.zeros(4, 2 * shape.H, dtype=torch.bfloat16, device="cuda")[:, :shape.H])
    assert (f.topk_idx == -7).all() and f.route_ws is None


def test_ids_out_of_range_leave_their_assignment_out(qsm):
    """moe_mx4_experts itself."""
    import ctypes
    from quantized_sparse_moe_gb300 import mx4
    T, H, I, E, k = 6, 256, 128, 8, 2
    L, v, wr = mx4_layer(qsm, H, I, E, k, 4, router=False)
    x = torch.randn((T, H), generator=gen(6), device="cuda").bfloat16()
    ids, w = qsm.moe_route_scores(x, qsm.MoERouter(wr, k))
    for acts, code in (("bf16", 16), ("mx4", 1)):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad = ids.clone()
        bad[2, 1], bad[4, 0] = E, -1
        ws = torch.zeros(qsm.moe_mx4_workspace_bytes(L, T, acts, False), dtype=torch.uint8, device="cuda")
        y, y32 = torch.empty_like(x), torch.empty(T, H, device="cuda")
        assert mx4.lib().moe_mx4_experts(ctypes.byref(L.c), x.data_ptr(), T, code, bad.data_ptr(), w.data_ptr(), y.data_ptr(),
                                         y32.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(),
                                         torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert st.item() == (1 if acts == "mx4" else 0)
        kept = w.clone()
        kept[2, 1], kept[4, 0] = 0, 0
        want = _mx4_ref.moe(x, ids.long(), kept, *v, four=acts == "mx4")
        d = y32.double() - want
        assert (d.norm() / want.norm()).item() <= 3e-3


class Step:
    """Two blocks and the vocabulary's projection, as a decoding program holds them."""

    def __init__(self, qsm, T, acts):
        H, I, E, k, N, n = 512, 256, 32, 4, 1000, 5
        self.qsm, self.H, self.T = qsm, H, T
        self.layers = [mx4_layer(qsm, H, I, E, k, 7 + s, router=False) for s in range(2)]
        self.routers = [qsm.MoERouter(w, k, "sigmoid", groups=8, groups_kept=4, group_best=2, scale=2.0)
                        for _, _, w in self.layers]
        self.forward = [qsm.Mx4Forward(L, T, acts, router=r) for (L, _, _), r in zip(self.layers, self.routers)]
        self.w = [1 + 0.1 * torch.randn(H, generator=gen(20 + i), device="cuda") for i in range(5)]
        norm = lambda i: qsm.Norm(self.w[i])  # noqa: E731
        self.enter = qsm.ResidualNorm(H, pre=norm(0))
        self.between = [qsm.ResidualNorm(H, pre=norm(1), post=norm(2), scale=0.5),
                        qsm.ResidualNorm(H, pre=norm(3), post=norm(4), scale=0.5)]
        self.head = qsm.mx4_quantize(torch.randn((N, H), generator=gen(30), device="cuda") * H ** -0.5)
        self.lora = qsm.LoraAdapters((torch.randn((n, 16, H), generator=gen(31), device="cuda") * H ** -0.5).bfloat16(),
                                     (torch.randn((n, N, 16), generator=gen(32), device="cuda") * 0.25).bfloat16())
        self.ids = (torch.arange(T, device="cuda") % (n + 1) - 1).int()
        self.four = acts == "mx4"

    def __call__(self, x):
        qsm, seen = self.qsm, []
        _, h = self.enter(x)
        for f, n in zip(self.forward, self.between):
            y = f(h).clone()
            seen.append((x, y, h))
            x, h = n(x, y)
        if self.four:
            _, h4 = n(seen[-1][0], seen[-1][1], h="mx4")
            logits = qsm.mx4_gemm(h4, self.head)
        else:
            logits = qsm.mx4_gemv(h, self.head)
        return seen, x, h, logits, qsm.lora_add(h, self.lora, self.ids, logits)


@pytest.mark.parametrize("T,acts", [(1, "bf16"), (7, "bf16"), (70, "mx4")])
def test_a_step_through_all_of_them(qsm, T, acts):
    s = Step(qsm, T, acts)
    x = torch.randn((T, s.H), generator=gen(40 + T), device="cuda").bfloat16()
    seen, last, h, logits, out = s(x)
    no = (None, None, None, 0.0)
    _, (wh, eh) = ref.residual(x, None, None, 1.0, no, (s.w[0].cpu(), None, "rms", 1e-6))
    assert ref.lies_between(seen[0][2], wh, eh)
    nexts = [(seen[1][0], seen[1][2]), (last, h)]
    for i, ((xi, yi, hi), (xn, hn)) in enumerate(zip(seen, nexts)):
        ids, w = qsm.moe_route_scores(hi, s.routers[i])
        want = _mx4_ref.moe(hi, ids.long(), w, *s.layers[i][1], four=s.four)
        assert ((yi.double() - want).norm() / want.norm()).item() <= 3e-3 + 2 ** -9
        (wx, ex), (wh, eh) = ref.residual(xi, yi, None, 0.5, (s.w[2 + 2 * i].cpu(), None, "rms", 1e-6),
                                          (s.w[1 + 2 * i].cpu(), None, "rms", 1e-6))
        assert ref.lies_between(xn, wx, ex) and ref.lies_between(hn, wh, eh)
    a, b = s.lora.a.double(), s.lora.b.double()
    want = logits.double()
    for t, i in enumerate(s.ids.tolist()):
        if i >= 0:
            want[t] += b[i] @ (a[i] @ h[t].double())
    assert ((out.double() - want).abs() <= 2 ** -8 * want.abs() + 1e-4).all()
    assert torch.equal(out[s.ids < 0], logits[s.ids < 0])
    for f in s.forward:
        assert f.dev_status.item() == 0


def test_a_step_captured_and_replayed(qsm):
    s = Step(qsm, 5, "bf16")
    x = torch.randn((5, s.H), generator=gen(50), device="cuda").bfloat16()
    s(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = s(x)
    for seed in (51, 52):
        x.copy_(torch.randn((5, s.H), generator=gen(seed), device="cuda").bfloat16())
        want = s(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[4], want[4]) and torch.equal(got[1], want[1])


def test_two_threads_at_once(qsm):
    """The same plans from two threads, each on a stream of its own."""
    import threading
    s = Step(qsm, 3, "bf16")
    plans = s.routers[0], qsm.ResidualNorm(s.H, pre=qsm.Norm()), s.lora
    ids = torch.tensor([0, -1, 1], device="cuda").int()
    y = torch.randn((3, s.lora.N), generator=gen(60), device="cuda").bfloat16()

    def calls(x):
        _, h = plans[1](x, x)
        return (h, *qsm.moe_route_scores(h, plans[0]), qsm.lora_add(h, plans[2], ids, y))

    xs = [torch.randn((3, s.H), generator=gen(61 + i), device="cuda").bfloat16() for i in range(2)]
    want = [calls(x) for x in xs]
    torch.cuda.synchronize()
    good = [False, False]

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [calls(xs[i]) for _ in range(200)]
            torch.cuda.current_stream().synchronize()
            good[i] = all(torch.equal(a, b) for g in got for a, b in zip(g, want[i]))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert good == [True, True]


def test_first_calls_inside_a_capture(qsm):
    """Sizes that no call had before, captured at once; two graphs replayed on two streams."""
    s = Step(qsm, 6, "bf16")
    H, T = s.H, 11
    n = qsm.ResidualNorm(H, pre=qsm.Norm())
    y = torch.randn((T, s.lora.N), generator=gen(70), device="cuda").bfloat16()
    ids = (torch.arange(T, device="cuda") % 3 - 1).int()
    xs = [torch.randn((T, H), generator=gen(71 + i), device="cuda").bfloat16() for i in range(2)]
    kept = dict(qsm._mx4._words)
    qsm._mx4._words.clear()

    def calls(x):
        _, h = n(x, x)
        _, q = n(x, x, h="mx4")
        return (h, q.codes, *s.routers[0].route(h), qsm.lora_add(h, s.lora, ids, y))

    torch.cuda.synchronize()
    graphs, got = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(calls(x))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for x, g in zip(xs, got):
        assert all(torch.equal(a, b) for a, b in zip(calls(x), g))
    qsm._mx4._words.update(kept)


def test_the_example_runs_with_all_of_them():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "mx4_generate.py"), "--steps", "3", "--scores", "--adapter"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens" in r.stdout


@pytest.mark.parametrize("T,acts", [(1, "bf16"), (5, "bf16"), (17, "bf16"), (64, "bf16"), (5, "mx4"), (130, "mx4")])
@pytest.mark.parametrize("k", [2, 4, 32])
def test_an_expert_named_more_than_once(qsm, T, acts, k):
    """moe_mx4_experts: with 4-bit activations its weights add up, with 16-bit ones such tokens are
    refused on the device, the others as ever.  The workspace holds zeros, which would pass for an output."""
    import ctypes
    from quantized_sparse_moe_gb300 import mx4
    H, I, E = 256, 128, 40
    L, v, _ = mx4_layer(qsm, H, I, E, k, 5, router=False)
    x = torch.randn((T, H), generator=gen(80 + T), device="cuda").bfloat16()
    w = torch.rand((T, k), generator=gen(81), device="cuda") / k
    ids = torch.stack([torch.randperm(E, generator=gen(82 + t), device="cuda")[:k] for t in range(T)]).int()
    ids[0] = E - 1                                                      # all the same
    ids[T // 2, 0] = ids[T // 2, k - 1]                                 # the first and the last one
    if T > 2:
        w[2], ids[2] = 0, 0                                             # padding
        ids[1] = torch.arange(k, device="cuda").int()
        ids[1, :2], w[1, :2] = E, 0                                     # out of range, twice: left out
    twice = torch.tensor([len(set(row)) < len(row) for row in ids.tolist()], device="cuda")
    twice[1:2] = False
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.zeros(qsm.moe_mx4_workspace_bytes(L, T, acts, False), dtype=torch.uint8, device="cuda")
    y, y32 = torch.empty_like(x), torch.empty(T, H, device="cuda")
    assert mx4.lib().moe_mx4_experts(ctypes.byref(L.c), x.data_ptr(), T, 16 if acts == "bf16" else 1, ids.data_ptr(), w.data_ptr(),
                                     y.data_ptr(), y32.data_ptr(), ws.data_ptr(), ws.numel(), st.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    one = lambda j, w: _mx4_ref.moe(x, ids[:, j:j + 1].long().clamp_max(E - 1), w[:, j:j + 1], *v, four=acts == "mx4")  # noqa: E731
    shared = one(0, torch.zeros_like(w))
    want = shared + sum(one(j, w) - shared for j in range(k))
    if acts == "bf16":
        assert y32[twice].isnan().all() and y[twice].isnan().all() and st.item() & 1
        y, y32, want = y[~twice], y32[~twice], want[~twice]
    d = y32.double() - want
    if len(d):
        assert (d.norm() / want.norm()).item() <= 3e-3 if acts == "mx4" else (d.abs().max() / want.abs().max()).item() <= 2e-3
    assert torch.equal(y, y32.to(torch.bfloat16))
