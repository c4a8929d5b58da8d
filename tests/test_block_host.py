"""The calls around the products on the host: the argument checks of the C
entry points (they answer before anything is enqueued, so they need no GPU) and
of the binding."""
import ctypes
import os
import shutil

import pytest
import torch

nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and
                          not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="nvcc missing")
OK, BAD, UNSUP, SMALL = 0, 1, 2, 3
P = 1 << 20            # never dereferenced: every call below is refused, or has no rows
FAR = 1 << 30          # between the operands


def at(n):
    return P + n * FAR


@nvcc
def test_residual_norm_refuses_bad_arguments():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import block
    f = qsm.lib().residual_norm
    none, rms = block.NormC(0, 0.0, None, None), block.NormC(1, 1e-6, at(20), None)

    def call(T=4, H=64, xt=0, yt=0, gt=0, ht=0, gate=0, sig=0, scale=1.0, post=none, pre=rms,
             x=at(0), ldx=64, y=at(1), ldy=64, g=None, ldg=0, o=at(2), ldo=64, h=at(3), ldh=64,
             hs=at(4), st=at(5)):
        c = block.ResidualNormC(H, xt, yt, gt, ht, gate, sig, scale, post, pre)
        return f(ctypes.byref(c), T, x, ldx, y, ldy, g, ldg, o, ldo, h, ldh, hs, st, None)

    assert call(T=0) == OK
    assert f(None, 4, P, 64, P, 64, None, 0, P, 64, P, 64, None, None, None) == BAD
    assert call(T=-1) == BAD and call(H=60) == BAD and call(H=0) == BAD
    assert call(H=16392, ldx=16392, ldy=16392, ldo=16392, ldh=16392) == UNSUP
    assert call(T=(1 << 30) + 1) == UNSUP
    assert call(x=None) == BAD and call(h=None, o=None) == BAD
    for odd in ("x", "y", "o", "h"):
        assert call(**{odd: at(7) + 8}) == BAD
    for ld in ("ldx", "ldy", "ldo", "ldh"):
        assert call(**{ld: 56}) == BAD and call(**{ld: 68}) == BAD
    for t in ("xt", "yt", "ht"):
        assert call(**{t: 4}) == BAD and call(**{t: -1}) == BAD
    assert call(xt=3) == BAD
    assert call(scale=float("nan")) == BAD and call(scale=float("inf")) == BAD
    assert call(sig=2) == BAD and call(gate=3, g=at(6)) == BAD
    # norms
    assert call(pre=none) == BAD                                       # h without a pre
    assert call(pre=block.NormC(3, 1e-6, None, None)) == BAD
    assert call(pre=block.NormC(1, -1.0, None, None)) == BAD
    assert call(pre=block.NormC(1, float("nan"), None, None)) == BAD
    assert call(pre=block.NormC(1, 1e-6, at(20) + 4, None)) == BAD
    assert call(post=block.NormC(0, 0.0, at(20), None)) == BAD
    # gates
    assert call(gate=1) == BAD and call(g=at(6)) == BAD                # kind without values, and the reverse
    assert call(gate=1, g=at(6), ldg=8) == BAD and call(gate=1, g=at(6) + 8) == BAD
    assert call(gate=2, g=at(6) + 1) == BAD and call(gate=2, g=at(6), ldg=-1) == BAD
    assert call(gate=1, g=at(6), gt=3) == BAD
    assert call(gate=1, g=at(6), y=None) == BAD
    # MXFP4
    assert call(ht=3, H=72, ldx=72, ldy=72, ldo=72) == BAD             # H % 32
    assert call(ht=3, hs=None) == BAD and call(ht=3, st=None) == BAD and call(ht=3, hs=at(4) + 8) == BAD


@nvcc
def test_residual_norm_refuses_overlaps():
    """What is written may be x or y, lie beside them in one matrix, and nothing else.  The
    accepted layouts run on the GPU (test_gpu_residual_norm)."""
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import block
    f = qsm.lib().residual_norm
    none, rms = block.NormC(0, 0.0, None, None), block.NormC(1, 1e-6, at(20), None)

    def call(o=at(2), ldo=64, h=at(3), ldh=64, ht=0, g=None, gate=0, hs=at(4), T=4, ldx=64):
        c = block.ResidualNormC(64, 0, 0, 0, ht, gate, 0, 1.0, none, rms)
        return f(ctypes.byref(c), T, at(0), ldx, at(1), 64, g, 0, o, ldo, h, ldh, hs, at(5), None)

    assert call(o=at(0) + 128) == BAD and call(h=at(0) + 128) == BAD      # a row further on
    assert call(o=at(1) + 16) == BAD and call(h=at(1) + 16) == BAD
    assert call(h=at(2)) == BAD and call(o=at(3) + 3 * 128) == BAD        # each other
    assert call(h=at(0), ht=2) == BAD and call(h=at(0), ht=3) == BAD      # x, with another size
    assert call(o=at(20)) == BAD and call(h=at(20)) == BAD                # a weight
    assert call(o=at(6), g=at(6), gate=1) == BAD
    assert call(o=at(0), ldo=128) == BAD                                  # x, with another stride
    assert call(ht=3, hs=at(0)) == BAD and call(ht=3, hs=at(2)) == BAD and call(ht=3, hs=at(3)) == BAD
    assert call(o=at(0) + 64, ldo=128, ldx=128) == BAD                    # half of it beside x


def test_binding_refuses_bad_norms():
    import quantized_sparse_moe_gb300 as qsm
    for kw in (dict(kind="max"), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(qsm.QSMError):
            qsm.Norm(**kw)
    with pytest.raises(qsm.QSMError):
        qsm.Norm(torch.ones(1, 64))
    with pytest.raises(qsm.QSMError):
        qsm.ResidualNorm(64, device="cpu")
    n = qsm.Norm(torch.ones(64))
    with pytest.raises(AttributeError):
        n.weight = torch.ones(64)
    with pytest.raises(qsm.QSMError):
        qsm.ResidualNorm(64, pre=n, device="cuda:0")                      # weight not on the GPU


@nvcc
def test_route_scores_refuses_bad_arguments():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import block
    L = qsm.lib()
    assert L.moe_router_split_bytes(8, 64) == 3 * 128 * 64 * 2 and L.moe_router_split_bytes(0, 64) == 0
    assert L.moe_router_split_bytes(300, 128) == 3 * 512 * 128 * 2 and L.moe_router_split_bytes(8, 96) == 0
    for a in ((None, 8, 64, P, None), (P, 8, 96, P, None), (P, 0, 64, P, None), (P, 8, 64, None, None),
              (P + 4, 8, 64, P, None), (P, 8, 64, P + 8, None)):
        assert L.moe_router_split(*a) == BAD

    def call(T=4, x=at(0), ldx=128, idx=at(1), w=at(2), st=at(3), **over):
        f = dict(H=128, E=16, k=4, score=0, groups=1, groups_kept=1, group_best=1, renormalize=1, scale=1.0,
                 w_split=at(4), bias=None)
        f.update(over)
        return L.moe_route_scores(ctypes.byref(block.RouterC(*f.values())), x, ldx, T, idx, w, st, None)
    assert call(T=0) == OK
    assert L.moe_route_scores(None, P, 128, 4, P, P, P, None) == BAD
    assert call(T=-1) == BAD and call(H=96) == BAD and call(H=0) == BAD and call(E=0) == BAD
    assert call(k=0) == BAD and call(k=17) == BAD and call(score=2) == BAD and call(renormalize=2) == BAD
    assert call(groups=3) == BAD and call(groups=4, groups_kept=0) == BAD and call(groups=4, groups_kept=5) == BAD
    assert call(groups=0) == BAD and call(groups=8, groups_kept=1) == BAD    # two experts for k = 4
    assert call(group_best=0) == BAD and call(group_best=3) == BAD
    assert call(groups=16, groups_kept=8, group_best=2) == BAD               # a group of one
    assert call(scale=float("nan")) == BAD and call(scale=float("inf")) == BAD
    assert call(E=513, k=4) == UNSUP and call(E=512, k=33) == UNSUP and call(E=128, groups=64, groups_kept=8) == UNSUP
    for none in ("x", "idx", "w", "st", "w_split"):
        assert call(**{none: None}) == BAD
    assert call(x=at(0) + 8) == BAD and call(idx=at(1) + 2) == BAD and call(bias=at(5) + 2) == BAD
    assert call(ldx=120) == BAD and call(ldx=132) == BAD


@nvcc
def test_route_scores_refuses_overlaps():
    """The ids and weights are written while other tokens' x, the weights and the bias are read."""
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import block
    L = qsm.lib()

    def call(idx=at(1), w=at(2), T=4, ldx=128):
        r = block.RouterC(128, 16, 4, 0, 1, 1, 1, 1, 1.0, at(4), at(5))
        return L.moe_route_scores(ctypes.byref(r), at(0), ldx, T, idx, w, at(3), None)
    for there in (at(0), at(0) + 3 * 256 + 240, at(4), at(4) + 2 * 3 * 128 * 64 * 2 - 4, at(5) + 60):
        assert call(idx=there) == BAD and call(w=there) == BAD
    assert call(w=at(1)) == BAD and call(w=at(1) + 60) == BAD and call(idx=at(2) - 60) == BAD
    assert call(idx=at(0) + 256, ldx=256, T=100) == BAD  # 1600 bytes from the gap of 256 behind a row on
    assert L.moe_router_split(P, 16, 128, P, None) == BAD and L.moe_router_split(P, 16, 128, P + 16 * 128 * 4 - 16, None) == BAD


@nvcc
def test_lora_refuses_bad_arguments():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import block
    f = qsm.lib().lora_add

    def call(n=3, rank=16, K=64, N=48, a=at(10), b=at(11), scale=None, ranks=None, T=4, x=at(0), ldx=64,
             ids=at(1), dt=0, y=at(2), ldy=48, o=at(3), ldo=48, st=at(4)):
        c = block.LoraC(n, rank, K, N, a, b, scale, ranks)
        return f(ctypes.byref(c), x, ldx, T, ids, dt, y, ldy, o, ldo, st, None)
    assert call(T=0) == OK
    assert f(None, P, 64, 4, P, 0, P, 48, P, 48, P, None) == BAD
    for kw in (dict(n=0), dict(rank=0), dict(rank=12), dict(K=60), dict(K=0), dict(N=0), dict(T=-1), dict(dt=1), dict(dt=3)):
        assert call(**kw) == BAD
    assert call(rank=136) == UNSUP and call(K=(1 << 28) + 8, ldx=1 << 29) == UNSUP and call(N=(1 << 28) + 1) == UNSUP
    for none in ("a", "b", "x", "ids", "o", "st"):
        assert call(**{none: None}) == BAD
    for odd in (dict(a=at(10) + 8), dict(b=at(11) + 8), dict(x=at(0) + 8), dict(ids=at(1) + 2), dict(y=at(2) + 1),
                dict(o=at(3) + 1), dict(o=at(3) + 2, dt=2, y=None), dict(scale=at(12) + 2), dict(ranks=at(12) + 2), dict(st=at(4) + 1)):
        assert call(**odd) == BAD
    for ld in (dict(ldx=56), dict(ldx=68), dict(ldy=47), dict(ldo=47)):
        assert call(**ld) == BAD
    # overlaps: out may be y, or lie beside it in one matrix
    assert call(o=at(0)) == BAD and call(o=at(2) + 96) == BAD and call(o=at(2), ldo=64) == BAD
    assert call(o=at(1)) == BAD and call(o=at(10)) == BAD and call(o=at(11)) == BAD
    assert call(o=at(12), scale=at(12)) == BAD and call(o=at(12), ranks=at(12)) == BAD
    assert call(o=at(2) + 32, ldy=96, ldo=96) == BAD


def test_binding_refuses_bad_adapters():
    import quantized_sparse_moe_gb300 as qsm
    a, b = torch.zeros(2, 8, 64).bfloat16(), torch.zeros(2, 32, 8).bfloat16()
    for bad in ((a, b), (a[0], b), (a, b[:1]), (a, b[:, :, :4]), (a[:, :4], b[:, :, :4]), (a.float(), b.float())):
        with pytest.raises(qsm.QSMError):
            qsm.LoraAdapters(*bad)                                         # not on a GPU, or misshapen


@nvcc
def test_experts_refuse_bad_arguments():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import mx4
    lib = qsm.lib()

    def layer(H=256, I=128, E=8, k=2, **over):
        f = dict(gate_up=mx4.Mx4C(E, 2 * I, H, P, P), down=mx4.Mx4C(E, H, I, P, P),
                 shared_gate_up=mx4.Mx4C(1, 2 * I, H, P, P), shared_down=mx4.Mx4C(1, H, I, P, P),
                 shared_gate=None)
        f.update(over)
        return mx4.Mx4LayerC(H, I, E, k, *f.values())

    def call(L, T=4, acts=0, x=P, idx=P, w=P, y=P, ws=1 << 40):
        return lib.moe_mx4_experts(ctypes.byref(L), x, T, acts, idx, w, y, None, P, ws, P, None)
    assert call(layer(), T=0) == OK
    assert call(layer(), T=-1) == BAD and call(layer(), acts=2) == BAD and call(layer(), acts=17) == BAD
    assert call(layer(H=192)) == UNSUP and call(layer(k=9)) == UNSUP and call(layer(), T=65) == UNSUP
    assert call(layer(), x=None) == BAD and call(layer(), idx=None) == BAD and call(layer(), w=None) == BAD
    assert call(layer(), idx=P + 2) == BAD and call(layer(), w=P + 1) == BAD and call(layer(), y=P + 4) == BAD
    assert call(layer(down=mx4.Mx4C(8, 256, 160, P, P))) == BAD
    ws = lib.moe_mx4_workspace_bytes
    for T, acts, sized in ((1, 0, 16), (2, 16, 16), (40, 0, 16), (65, 1, 1)):
        need = ws(ctypes.byref(layer()), T, sized)
        assert need > 0 and call(layer(), T=T, acts=acts, ws=need - 1) == SMALL
    with pytest.raises(qsm.QSMError):
        qsm.MoEForward(type("L", (), dict(H=256, E=8, k=2))(), 4, router=type("R", (), dict(H=256, E=8, k=3))())


@nvcc
def test_experts_refuse_outputs_over_the_choice():
    """One token's y is written while another's ids and weights are read."""
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import mx4
    lib = qsm.lib()
    H, I, E, k, T = 256, 128, 8, 2, 4
    L = mx4.Mx4LayerC(H, I, E, k, mx4.Mx4C(E, 2 * I, H, at(1), at(2)), mx4.Mx4C(E, H, I, at(3), at(4)),
                      mx4.Mx4C(1, 2 * I, H, at(5), at(6)), mx4.Mx4C(1, H, I, at(7), at(8)), None)

    def call(y=at(10), y32=at(11), idx=at(12), w=at(13), acts=0):
        return lib.moe_mx4_experts(ctypes.byref(L), at(0), T, acts, idx, w, y, y32, at(14), 1 << 40, at(15), None)
    n = T * H * 2
    for acts in (0, 1):
        assert call(idx=at(10), acts=acts) == BAD and call(w=at(10), acts=acts) == BAD
        assert call(idx=at(10) + n - 4, acts=acts) == BAD and call(w=at(10) - 4, acts=acts) == BAD
        assert call(idx=at(11) + 2 * n - 4, acts=acts) == BAD and call(w=at(11) - 28, acts=acts) == BAD


def test_layer_refuses_a_router_of_another_device():
    import quantized_sparse_moe_gb300 as qsm
    layer, router = (type(n, (), dict(H=256, E=8, k=2, device=1)) for n in "LR")
    for device in ("cuda:0", "cpu"):
        with pytest.raises(qsm.QSMError):
            qsm.MoEForward(layer(), 4, device, router=router())
