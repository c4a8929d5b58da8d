"""What the one-launch form's order of sums means for a token of two: the other
token changes which experts' products share an accumulator, and nothing else.

Bound: every product is exact, so two orders differ by the rounding of fp32
sums alone.  A digit plane's sum has (k + 1) I terms, and six planes and four
CTAs are added, each addition off by at most 2^-23 (the tensor cores may
truncate) of the sum of magnitudes; the digits' magnitudes add up to at most
three times the value's; two results."""
import pytest
import torch

from test_gpu_mx4 import check_layer, hidden, layer

pytestmark = pytest.mark.gpu


def magnitudes(x, idx, w, v):
    """sum over slots of weight |h| |W_down| of one token, [H]."""
    gu, dn, sgu, sdn = v
    half = gu.shape[1] // 2

    def one(up, down):
        g = up @ x
        return down.abs() @ (g[:half] * torch.sigmoid(g[:half]) * g[half:]).abs()
    s = one(sgu[0], sdn[0])
    for e, z in zip(idx.tolist(), w.tolist()):
        s = s + z * one(gu[e], dn[e])
    return s


@pytest.mark.parametrize("h,i,e,k", [(2048, 512, 256, 8), (1024, 128, 64, 32), (1152, 640, 16, 3)])
def test_the_other_token_changes_the_order_of_sums_only(qsm, h, i, e, k):
    L, v = layer(qsm, h, i, e, k, seed=h + k)
    f = qsm.Mx4Forward(L, 2, want_f32=True)
    x = hidden(2, h, 1)
    runs = []
    for s in (1, 2, 3, 4):
        x[1] = hidden(1, h, 10 + s)[0]
        check_layer(qsm, L, v, x, "bf16", f=f)
        runs.append((f.y_f32[0].clone(), f.topk_idx[0].clone(), f.topk_w[0].clone()))
    x[1] = hidden(1, h, 11)[0]
    f(x)
    assert torch.equal(f.y_f32[0], runs[0][0])                   # the same two tokens: the same bits
    b = 2 * ((k + 1) * i + 10) * 2.0 ** -23 * 3 * magnitudes(x[0].double(), runs[0][1], runs[0][2], v)
    for y, idx, w in runs[1:]:
        assert torch.equal(idx, runs[0][1]) and torch.equal(w, runs[0][2])
        assert ((y - runs[0][0]).double().abs() <= b).all()


@pytest.mark.parametrize("t", [3, 9, 40])
def test_in_separate_launches_a_token_does_not_see_the_others(qsm, t):
    L, _ = layer(qsm, 512, 256, 32, 4, seed=t)
    f = qsm.Mx4Forward(L, t, want_f32=True)
    x = hidden(t, 512, 1)
    f(x)
    want = f.y_f32[0].clone()
    for s in (2, 3):
        x[1:] = hidden(t - 1, 512, s)
        f(x)
        assert torch.equal(f.y_f32[0], want)


@pytest.mark.parametrize("t,h,i,e,k", [(1, 2048, 512, 256, 8), (2, 2048, 512, 256, 8), (1, 1024, 128, 64, 32)])
def test_the_one_launch_form_can_be_left_out(qsm, t, h, i, e, k):
    L, v = layer(qsm, h, i, e, k, seed=t + 20, gate=True)
    x = hidden(t, h, 3)
    one = qsm.Mx4Forward(L, t, want_f32=True)
    n = qsm.launch_count()
    check_layer(qsm, L, v, x, "bf16", f=one)
    few = qsm.launch_count() - n
    many = qsm.Mx4Forward(L, t, want_f32=True, one_launch=False)
    n = qsm.launch_count()
    check_layer(qsm, L, v, x, "bf16", f=many)
    assert qsm.launch_count() - n == few + 3          # route, gate_up, down, combine
    assert many.workspace.numel() >= qsm.moe_mx4_workspace_bytes(L, t, one_launch=False) > 0
    assert torch.equal(one.topk_idx, many.topk_idx) and torch.equal(one.topk_w, many.topk_w)
