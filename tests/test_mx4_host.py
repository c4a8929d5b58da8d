"""MXFP4 on the host: the scale layout, the reference the GPU tests compare
against, and the argument checks of the C entry points (they answer before
anything is enqueued, so they need no GPU)."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

import _mx4_ref as ref

nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and
                          not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="nvcc missing")


@pytest.mark.parametrize("rows,cols", [(1, 32), (128, 128), (129, 160), (300, 1056)])
def test_scale_tiles_follow_the_stated_layout(rows, cols):
    import quantized_sparse_moe_gb300 as qsm
    s = torch.randint(0, 255, (rows, cols // 32), dtype=torch.uint8)
    t = qsm.mx4_tile_scales(s)
    assert t.numel() == qsm.mx4_scale_bytes(rows, cols)
    cts = -(-cols // 128)
    seen = np.zeros(t.numel(), bool)
    for r in range(rows):
        for b in range(cols // 32):
            at = ((r // 128) * cts + b // 4) * 512 + 16 * (r % 32) + 4 * (r % 128 // 32) + b % 4
            assert t[at] == s[r, b]
            seen[at] = True
    assert not t.numpy()[~seen].any()          # the padding holds 0
    assert torch.equal(ref.untile(t, rows, cols), s)


def test_expert_tiles_follow_one_another():
    import quantized_sparse_moe_gb300 as qsm
    s = torch.randint(0, 255, (3, 130, 5), dtype=torch.uint8)
    each = torch.cat([qsm.mx4_tile_scales(s[e]) for e in range(3)])
    assert torch.equal(qsm.mx4_tile_scales(s), each)


def test_reference_quantization_by_hand():
    # largest 6.5: scale 2^(2 - 2) = 1; ties 0.25 -> 0, 0.75 -> 1, 1.25 -> 1,
    # 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4, and 6.5 becomes 6
    x = torch.zeros(1, 64)
    x[0, :8] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -6.5])
    c, s = ref.quantize(x)
    assert s.tolist() == [[127, 0]]
    assert c[0, :4].tolist() == [0 | 2 << 4, 2 | 4 << 4, 4 | 6 << 4, 6 | 15 << 4]
    assert ref.values(c, s)[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, -6]


def test_reference_values_are_the_format():
    codes = torch.tensor([[c | (15 - c) << 4 for c in range(16)]], dtype=torch.uint8)
    v = ref.values(codes, torch.tensor([[130]], dtype=torch.uint8))[0].reshape(16, 2)
    for c in range(16):
        sign, e, m = c >> 3, c >> 1 & 3, c & 1
        one = (m * 0.5 if e == 0 else (1 + m / 2) * 2.0 ** (e - 1)) * (-1) ** sign * 8
        assert v[c, 0] == one and v[15 - c, 1] == one


@nvcc
def test_entry_points_refuse_bad_arguments():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import mx4
    lib = qsm.lib()
    ok, bad, unsup = 0, 1, 2
    p, odd = 1 << 20, (1 << 20) + 4        # never dereferenced: every call below is refused
    assert lib.mx4_scale_bytes(129, 160) == 4 * 512 and lib.mx4_scale_bytes(-1, 32) == 0
    q = lib.mx4_quantize
    assert q(p, 0, 64, 0, 64, p, p, p, None) == ok                    # no rows
    assert q(p, 3, 64, 1, 64, p, p, p, None) == bad                   # type
    assert q(p, 0, 64, 1, 48, p, p, p, None) == bad                   # cols % 32
    assert q(p, 0, 32, 1, 64, p, p, p, None) == bad                   # stride < cols
    assert q(p, 0, 68, 1, 64, p, p, p, None) == bad                   # stride % 8
    assert q(odd, 0, 64, 1, 64, p, p, p, None) == bad                 # alignment
    assert q(None, 0, 64, 1, 64, p, p, p, None) == bad
    assert q(p, 0, 64, 1, 64, p, p, None, None) == bad
    assert q(p, 0, 64, -1, 64, p, p, p, None) == bad

    def m(e, r, c, codes=p, scales=p):
        return ctypes.byref(mx4.Mx4C(e, r, c, codes, scales))
    d = lib.mx4_dequantize
    assert d(m(1, 0, 64), 0, p, None) == ok
    assert d(m(1, 4, 40), 0, p, None) == bad and d(m(1, 4, 64), 5, p, None) == bad
    assert d(m(1, 4, 64, codes=odd), 0, p, None) == bad and d(m(1, 4, 64), 0, None, None) == bad
    g = lib.mx4_gemm
    assert g(m(1, 0, 64), m(1, 8, 64), 0, p, 8, p, None) == ok
    assert g(m(1, 4, 64), m(1, 8, 96), 0, p, 8, p, None) == bad       # K differs
    assert g(m(2, 4, 64), m(1, 8, 64), 0, p, 8, p, None) == bad       # experts
    assert g(m(1, 4, 64), m(1, 8, 64), 1, p, 8, p, None) == bad       # fp16 output
    assert g(m(1, 4, 64), m(1, 8, 64), 0, p, 7, p, None) == bad       # ldy < N
    assert g(m(1, 4, 64), m(1, 8, 64), 2, (1 << 20) + 2, 8, p, None) == bad
    assert g(m(1, 4, 64), m(1, 8, 64), 0, p, 8, None, None) == bad
    v = lib.mx4_gemv
    assert v(p, 64, 0, m(1, 8, 64), p, p, None) == ok
    assert v(p, 64, 33, m(1, 8, 64), p, p, None) == unsup             # too many rows
    assert v(p, 65568, 1, m(1, 8, 65568), p, p, None) == unsup        # K
    assert v(p, 64, -1, m(1, 8, 64), p, p, None) == bad
    assert v(p, 63, 1, m(1, 8, 64), p, p, None) == bad and v(odd, 64, 1, m(1, 8, 64), p, p, None) == bad

    def layer(H=256, I=128, E=8, k=2, **over):
        f = dict(gate_up=mx4.Mx4C(E, 2 * I, H, p, p), down=mx4.Mx4C(E, H, I, p, p),
                 shared_gate_up=mx4.Mx4C(1, 2 * I, H, p, p), shared_down=mx4.Mx4C(1, H, I, p, p),
                 shared_gate=None)
        f.update(over)
        return mx4.Mx4LayerC(H, I, E, k, *f.values())

    def fwd(L, T=4, acts=0, flags=1, x=p, ws=1 << 40, y=p):
        return lib.moe_mx4_forward(ctypes.byref(L), x, T, acts, p, None, flags, p, p, y, None, p, ws, p, None)
    assert fwd(layer(), T=0) == ok
    assert fwd(layer(), T=-1) == bad and fwd(layer(), acts=2) == bad and fwd(layer(), flags=4) == bad
    assert fwd(layer(H=192)) == unsup and fwd(layer(I=64)) == unsup and fwd(layer(k=9)) == unsup
    assert fwd(layer(), T=65) == unsup                                # acts="bf16": 64 tokens
    assert fwd(layer(), x=None) == bad and fwd(layer(), y=odd) == bad
    assert fwd(layer(down=mx4.Mx4C(8, 256, 160, p, p))) == bad        # a plane of another shape
    assert fwd(layer(gate_up=mx4.Mx4C(8, 256, 256, p, None))) == bad
    assert fwd(layer(), acts=1, ws=16) == 3                           # workspace too small
    ws = lib.moe_mx4_workspace_bytes
    assert ws(ctypes.byref(layer()), 65, 0) == 0 and ws(ctypes.byref(layer()), 65, 1) > 0
    assert ws(ctypes.byref(layer(H=200)), 4, 1) == 0 and ws(None, 4, 1) == 0


def test_binding_refuses_bad_tensors():
    import quantized_sparse_moe_gb300 as qsm
    u8 = dict(dtype=torch.uint8)
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Tensor(torch.zeros(1, 24, **u8), torch.zeros(512, **u8), 1, 48)   # cols % 32
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Tensor(torch.zeros(1, 32, **u8), torch.zeros(500, **u8), 1, 64)   # scale bytes
    with pytest.raises(qsm.QSMError):
        qsm.Mx4Tensor(torch.zeros(1, 32, **u8), torch.zeros(512, **u8), 1, 64)   # not on a GPU
    with pytest.raises(qsm.QSMError):
        qsm.mx4_quantize(torch.zeros(4, 64))                                     # not on a GPU
    with pytest.raises(qsm.QSMError):
        qsm.mx4_quantize(torch.zeros(4, 64, dtype=torch.float64))


@nvcc
def test_layer_refuses_outputs_that_overlap_its_input():
    """With a gated shared expert x is read until y is written: y is x, or apart
    from it (refused before anything is enqueued)."""
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import mx4
    H, I, E, p = 256, 128, 8, 1 << 20
    L = mx4.Mx4LayerC(H, I, E, 2, mx4.Mx4C(E, 2 * I, H, p, p), mx4.Mx4C(E, H, I, p, p),
                      mx4.Mx4C(1, 2 * I, H, p, p), mx4.Mx4C(1, H, I, p, p), p)

    def fwd(y, y32=None, acts=0, ws=0):   # no workspace: what is not refused before stops there
        return qsm.lib().moe_mx4_forward(ctypes.byref(L), p, 4, acts, p, None, 1, p, p, y, y32, p, ws, p, None)
    for acts in (0, 1):
        for off in (16, 4 * H * 2 - 16, -16, 16 - 4 * H * 2):
            assert fwd(p + off, acts=acts) == 1
        for off in (0, 4 * H * 2, -4 * H * 2):
            assert fwd(p + off, acts=acts) == 3
        assert fwd(p, p + 16, acts=acts) == 1 and fwd(p, p, acts=acts) == 1
        assert fwd(p, p + 4 * H * 2, acts=acts) == 3 and fwd(p, p - 4 * H * 4, acts=acts) == 3
        L.shared_gate = None
        assert fwd(p + 16, acts=acts) == 3
        L.shared_gate = p


@nvcc
def test_separate_launches_are_a_value_of_acts():
    import quantized_sparse_moe_gb300 as qsm
    from quantized_sparse_moe_gb300 import mx4
    H, I, E, p = 256, 128, 8, 1 << 20
    L = mx4.Mx4LayerC(H, I, E, 2, mx4.Mx4C(E, 2 * I, H, p, p), mx4.Mx4C(E, H, I, p, p),
                      mx4.Mx4C(1, 2 * I, H, p, p), mx4.Mx4C(1, H, I, p, p), None)
    lib, ref = qsm.lib(), ctypes.byref(L)
    for acts, want in ((16, 3), (17, 1), (32, 1), (-1, 1), (18, 1)):
        assert lib.moe_mx4_forward(ref, p, 4, acts, p, None, 1, p, p, p, None, p, 0, p, None) == want
        assert (lib.moe_mx4_workspace_bytes(ref, 4, acts) > 0) == (want == 3)


@nvcc
def test_scale_bytes_of_the_largest_sizes():
    import quantized_sparse_moe_gb300 as qsm
    n = 2 ** 31 - 1
    for rows, cols in ((n, 32), (n - 126, 160), (1, n - 31), (300, n)):
        assert qsm.lib().mx4_scale_bytes(rows, cols) == qsm.mx4_scale_bytes(rows, cols)
