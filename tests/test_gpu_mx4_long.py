"""The MXFP4 layer beyond the sizes of test_gpu_mx4.py: more work items on a CTA
than its table of tiles holds, and long prompts."""
import pytest

from test_gpu_mx4 import check_layer, hidden, layer

pytestmark = pytest.mark.gpu


def test_more_items_than_a_cta_tabulates(qsm):
    """160 experts, nearly all with tokens, and 64 column tiles of down each: over
    10000 items, 67 for some of 152 CTAs."""
    L, v = layer(qsm, 16384, 128, 160, 8, seed=1)
    f, _ = check_layer(qsm, L, v, hidden(100, 16384, 2), "mx4")
    assert (f.topk_idx.unique().numel() + 1) * 64 > 64 * 152


@pytest.mark.parametrize("t,h,i,e,k", [(4096, 256, 128, 64, 8), (4111, 640, 128, 16, 3), (3000, 2048, 512, 8, 2)])
def test_long_prompts(qsm, t, h, i, e, k):
    L, v = layer(qsm, h, i, e, k, seed=t % 100, gate=True)
    check_layer(qsm, L, v, hidden(t, h, 3), "mx4")


@pytest.mark.parametrize("t,k", [(200, 12), (1500, 20)])
def test_more_than_eight_experts_a_token(qsm, t, k):
    """The CUDA-core router on many tokens."""
    L, v = layer(qsm, 256, 128, 64, k, seed=k)
    check_layer(qsm, L, v, hidden(t, 256, 4), "mx4")
