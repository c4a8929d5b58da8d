"""The MoE layer with MXFP4 activations at small magnitudes: every step of it
but the upper limit of the held outputs is free of scale, so the bounds of
test_gpu_mx4.py hold at every scale, and powers of two in the down weights come
out in y exactly."""
import pytest
import torch

from test_gpu_mx4 import check_layer, hidden, layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,h,i,e,k", [(3, 256, 128, 8, 8), (70, 384, 256, 24, 5), (300, 2048, 512, 32, 4)])
@pytest.mark.parametrize("power", [-7, -12, -16, -20])
def test_small_activations(qsm, t, h, i, e, k, power):
    L, v = layer(qsm, h, i, e, k, seed=t, gate=True)
    check_layer(qsm, L, v, hidden(t, h, t + 1) * 2.0 ** power, "mx4")


@pytest.mark.parametrize("power", [1, 14, 60])
def test_powers_of_two_in_the_down_weights_are_exact(qsm, power):
    L, _ = layer(qsm, 640, 256, 16, 3, seed=4)
    x = hidden(150, 640, 5)
    f = qsm.Mx4Forward(L, 150, "mx4", want_f32=True)
    f(x)
    want = f.y_f32.clone()
    for m in (L.down, L.shared_down):
        assert int(m.scales.min()) > power
        m.scales -= power
    f(x)
    assert torch.equal(f.y_f32 * 2.0 ** power, want)
    assert f.dev_status.item() == 0


def test_rows_of_very_different_size(qsm):
    """A token 2^20 times smaller than its neighbours keeps its bits."""
    L, v = layer(qsm, 256, 128, 8, 2, seed=6)
    x = hidden(90, 256, 7)
    x[::3] *= 2.0 ** -20
    f, want = check_layer(qsm, L, v, x, "mx4")
    d = (f.y_f32.double() - want)[::3]
    assert (d.norm() / want[::3].norm()).item() <= 3e-3
