"""Few-row products and the few-token layer where their result is exact, so that
every digit plane of the activations shows by itself.

A block of 32 activations holds one large value, which meets a weight of 0, and
one small one, m 8^d of the 2^15 units that the large one's exponent makes: all
of it lies in plane d (m under 4, or a carry into d + 1).  The product of the
small value and a 4-bit weight has at most five bits, and every other product
is 0: y has to be that product's bits, whatever the sums' order.  The blocks
walk through all of K, and with it all stages, CTAs of a cluster and buffers."""
import pytest
import torch

from test_gpu_mx4 import mx4

pytestmark = pytest.mark.gpu

# one CTA for all of K, and clusters of 2, 4 and 8; ragged last stages; rows cut
# into slots; rows in halves
ROWS = [(10, 19456, 2048), (3, 8192, 8192), (16, 8192, 2048), (8, 4096, 4064), (1, 512, 2048), (5, 2048, 8192),
        (32, 640, 16384), (7, 300, 4064), (18, 19456, 3584), (26, 19456, 3584), (32, 19456, 2560), (2, 129, 96)]


@pytest.mark.parametrize("t,n,k", ROWS)
def test_every_plane_in_every_block(qsm, t, n, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(n + k)
    w = torch.randn((n, k), generator=g, device="cuda")
    w[:, ::32] = 0
    w, wv = mx4(qsm, w)
    blocks, row, done = k // 32, torch.arange(t, device="cuda"), set()
    sign = torch.where(row % 2 == 0, 1.0, -1.0).double()
    scale = torch.exp2((row % 7).double() - 3)
    for step in range(-(-blocks // t)):
        # neighbouring rows lie far apart in K
        b = (row * (-(-blocks // t)) + step) % blocks
        done.update(b.tolist())
        for d in range(6):
            m = torch.tensor([1.0, 1.0, 1.0] if d == 5 else [1.0, 3.0, 5.0], device="cuda").double()[(row + step) % 3]
            col = 32 * b + 1 + (7 * row + 5 * step + d) % 31
            x = torch.zeros((t, k), dtype=torch.float64, device="cuda")
            x[row, 32 * b] = 1.5 * scale
            x[row, col] = sign * scale * m * 8.0 ** d * 2.0 ** -15
            want = x[row, col][:, None] * wv[:, col].T
            assert torch.equal(x.to(torch.bfloat16).double(), x)
            y = qsm.mx4_gemv(x.to(torch.bfloat16), w)
            assert torch.equal(y.double(), want), (step, d)
    assert done == set(range(blocks))


def exact_layer(qsm, H, I, E):
    """A layer whose expert e takes the tokens with their one value in column
    7 + 31 e.  Its h is 96 at the first of every 32 intermediates, where down is
    0, and at one other m 8^d 2^-9: the value and the place go through all."""
    col = 7 + 31 * torch.arange(E, device="cuda") % (H - 7)
    gate_up = torch.zeros((E, 2 * I, H), device="cuda")
    gate_up[:, :I] = 4                                  # x = 16: 64, and silu(64) = 64 (to a few 2^-24)
    gate_up[:, I::32] = 1.5 / 16                        # times 16
    g = torch.Generator(device="cuda")
    g.manual_seed(I)
    e = torch.arange(E, device="cuda")
    at = 32 * (e % (I // 32)) + 1 + (5 * e) % 31
    d = e % 6
    small = torch.where((d < 5) & (e % 4 >= 2), 3.0, 1.0).double() * 8.0 ** d * 2.0 ** -15
    gate_up[e, I + at] = (small / 16).float()[:, None]
    down = torch.randn((E, H, I), generator=g, device="cuda")
    down[:, :, ::32] = 0
    parts = [mx4(qsm, w.reshape(-1, w.shape[-1]), w.shape[0]) for w in (gate_up, down)]
    assert torch.equal(parts[0][1].float(), gate_up)    # the format holds them
    shared = [mx4(qsm, torch.randn((r, c), generator=g, device="cuda") * 0)[0] for r, c in ((2 * I, H), (H, I))]
    router = torch.zeros((E, H), device="cuda")
    router[e, col] = 1
    L = qsm.Mx4Layer(H, I, E, 1, parts[0][0], parts[1][0], *shared, router)
    return L, col, (64 * small)[:, None] * parts[1][1][e, :, at]


@pytest.mark.parametrize("one_launch", [True, False])
@pytest.mark.parametrize("h,i,e", [(1024, 640, 60), (2048, 512, 96), (896, 128, 24), (384, 256, 48)])
@pytest.mark.parametrize("t", [1, 2, 3, 11, 40])
def test_every_plane_of_h(qsm, t, h, i, e, one_launch):
    L, col, want = exact_layer(qsm, h, i, e)
    f = qsm.Mx4Forward(L, t, want_f32=True, one_launch=one_launch)
    for first in range(0, e, t):
        ids = (first + 5 * torch.arange(t, device="cuda")) % e
        x = torch.zeros((t, h), dtype=torch.bfloat16, device="cuda")
        x[torch.arange(t, device="cuda"), col[ids]] = 16
        f(x)
        assert torch.equal(f.topk_idx[:, 0].long(), ids) and (f.topk_w == 1).all()
        assert torch.equal(f.y_f32.double(), want[ids])
    assert f.dev_status.item() == 0
