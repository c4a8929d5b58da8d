"""The router's workspace with more than eight experts a token: its size and
the refusal of less on the host (which answers before anything is enqueued, so
needs no GPU), and the call on a workspace of exactly that size."""
import os
import shutil

import pytest
import torch

nvcc = pytest.mark.skipif(shutil.which("nvcc") is None and
                          not os.path.exists("/usr/local/cuda/bin/nvcc"), reason="nvcc missing")


def plain_need(T, E):
    """Counters (4 bytes per 8 tokens) and fp32 logits of the CUDA-core router."""
    up = lambda v: (v + 255) // 256 * 256  # noqa: E731
    return up((T + 7) // 8 * 4) + up(T * E * 4)


@nvcc
@pytest.mark.parametrize("T,H,E", [(65, 128, 16), (190, 128, 256), (4096, 128, 64), (4096, 2048, 256)])
def test_workspace_holds_the_logits_of_every_k(T, H, E):
    """More than eight experts a token take the CUDA-core router at any T: the
    size that is stated covers its logits, and less is refused."""
    import quantized_sparse_moe_gb300 as qsm
    need = qsm.route_workspace_bytes(T, H, E)
    assert need >= plain_need(T, E)
    p = 1 << 20                             # never dereferenced: the call is refused
    assert qsm.lib().moe_route(p, p, None, T, H, E, 9, 1, p, p, p, plain_need(T, E) - 1, p, None) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k", [(1000, 128, 64, 12), (3100, 256, 256, 9)])
def test_many_experts_a_token_stay_inside_the_workspace(qsm, T, H, E, k):
    """Ids and weights against 64 bits, and the bytes after the workspace."""
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn((E, H), generator=g, device="cuda") * 0.05
    n = qsm.route_workspace_bytes(T, H, E)
    space = torch.zeros(n + (1 << 20), dtype=torch.uint8, device="cuda")
    space[n:] = 77
    for _ in range(2):
        idx, wt = qsm.moe_route(x, w, k, workspace=space[:n])
        assert (space[n:] == 77).all()
    l = x.double() @ w.double().T
    # fp32 sums of H products: each rounding at most 2^-24 of the magnitudes so far
    b = H * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T)
    got = l.gather(1, idx.long())
    assert all(len(set(r)) == k for r in idx.tolist())
    kth = l.topk(k, dim=1).values[:, -1:]
    assert (got >= kth - 2 * b.amax(dim=1, keepdim=True)).all()
    # a relative error of the weights of at most twice the largest logit's absolute one, and
    # what the exponential and the division round (2^-20 covers both)
    want = torch.softmax(got, dim=1)
    assert ((wt.double() - want).abs() <= want * (4 * b.amax(dim=1, keepdim=True) + 2.0 ** -20)).all()


@pytest.mark.gpu
def test_one_workspace_serves_calls_of_other_sizes(qsm):
    """Calls of few and many tokens, and of both routers, one after the other on
    one workspace that was zeroed once."""
    H, E = 128, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    w = torch.randn((E, H), generator=g, device="cuda") * 0.05
    space = torch.zeros(qsm.route_workspace_bytes(4100, H, E), dtype=torch.uint8, device="cuda")
    for T, k in ((1000, 9), (4100, 9), (700, 12), (2000, 8), (4100, 10), (8, 4), (3000, 9), (64, 9), (513, 9)):
        x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
        want = qsm.moe_route(x, w, k)                    # on a fresh workspace
        idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
        wt = torch.full((T, k), -7.0, device="cuda")
        qsm.moe_route(x, w, k, topk_idx=idx, topk_w=wt, workspace=space)
        assert torch.equal(idx, want[0]) and torch.equal(wt, want[1])
