"""The MoE layer with MXFP4 weights on its own input, and the gated shared
expert at widths where several threads' columns make up a token."""
import pytest
import torch

from test_gpu_mx4 import check_layer, hidden, layer

pytestmark = pytest.mark.gpu
CASES = [("bf16", 1, 2048), ("bf16", 2, 1152), ("bf16", 3, 128), ("bf16", 3, 2048), ("bf16", 40, 1152),
         ("bf16", 17, 4224), ("mx4", 1, 128), ("mx4", 70, 2048), ("mx4", 65, 1152), ("mx4", 300, 4224)]


@pytest.mark.parametrize("acts,t,h", CASES)
def test_gated_shared_expert(qsm, acts, t, h):
    L, v = layer(qsm, h, 128, 16, 3, seed=t, gate=True)
    check_layer(qsm, L, v, hidden(t, h, t + 1), acts)


@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("acts,t,h", CASES)
def test_in_place_gives_the_same_bits(qsm, acts, t, h, gate):
    L, _ = layer(qsm, h, 128, 16, 3, seed=t, gate=gate)
    f = qsm.Mx4Forward(L, t, acts)
    x = hidden(t, h, 2)
    want = f(x).clone()
    for _ in range(3):
        z = x.clone()
        assert f(z, out=z) is z
        assert torch.equal(z, want)


def test_refuses_a_shifted_output(qsm):
    L, _ = layer(qsm, 256, 128, 8, 2, seed=1, gate=True)
    f = qsm.Mx4Forward(L, 4)
    big = hidden(8, 256, 1)
    with pytest.raises(qsm.QSMError):
        f(big[:4], out=big[1:5])
    assert f(big[:4], out=big[4:]) is not None
