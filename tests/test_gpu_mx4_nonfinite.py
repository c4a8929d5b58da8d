"""The one-launch form of the MXFP4 layer on what is not finite: as the other
forms, a token's row shows it and the status word reports it, and the other
token is left alone."""
import math

import pytest
import torch

from test_gpu_mx4 import hidden, layer

pytestmark = pytest.mark.gpu


def overflowing(qsm, t):
    """Two experts a token, the second with a weight that underflows to 0 and
    weights so large that its h overflows."""
    L, _ = layer(qsm, 1024, 128, 16, 2, seed=3, bias=True)
    L.logit_bias = torch.zeros(16, device="cuda")
    L.logit_bias[3], L.logit_bias[5] = 1000.0, 500.0
    L.gate_up.scales.reshape(16, -1)[5] = 250
    return L, hidden(t, 1024, 2)


def check(qsm, L, x, **kw):
    f = qsm.Mx4Forward(L, x.shape[0], **kw)
    y = f(x)
    torch.cuda.synchronize()
    assert f.topk_idx.tolist() == [[3, 5]] * x.shape[0] and (f.topk_w == torch.tensor([1.0, 0.0], device="cuda")).all()
    assert f.dev_status.item() & qsm.DEV_NONFINITE
    assert torch.isnan(y).all()            # 0 x infinity


@pytest.mark.parametrize("t", [1, 2])
def test_weight_of_zero_does_not_hide_an_overflow(qsm, t):
    check(qsm, *overflowing(qsm, t))


@pytest.mark.parametrize("t", [1, 2, 5])
def test_weight_of_zero_in_separate_launches(qsm, t):
    check(qsm, *overflowing(qsm, t), one_launch=False)


@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("bad", [0, 1])
def test_a_token_that_is_not_finite_stays_apart(qsm, what, bad):
    L, _ = layer(qsm, 1024, 128, 16, 2, seed=9, gate=True)
    x = hidden(2, 1024, 3)
    f = qsm.Mx4Forward(L, 2, want_f32=True)
    f(x)
    good = 1 - bad
    idx, w, y = f.topk_idx[good].clone(), f.topk_w[good].clone(), f.y_f32[good].clone()
    x[bad, 700] = what
    f(x)
    torch.cuda.synchronize()
    assert f.dev_status.item() & qsm.DEV_NONFINITE
    assert not torch.isfinite(f.y[bad]).any()
    assert torch.equal(f.topk_idx[good], idx) and torch.equal(f.topk_w[good], w)
    # the other experts change the order of fp32 sums at most
    assert (f.y_f32[good] - y).abs().max() <= 2.0 ** -14 * y.abs().max()
    one = qsm.Mx4Forward(L, 1)
    z = one(x[bad:bad + 1].contiguous())
    torch.cuda.synchronize()
    assert one.dev_status.item() & qsm.DEV_NONFINITE and not torch.isfinite(z).any()
