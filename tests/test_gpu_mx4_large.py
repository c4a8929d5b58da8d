"""The MXFP4 calls where byte offsets, element offsets and products of sizes
pass 2^31 and 2^32."""
import pytest
import torch

import _mx4_ref as ref
from test_gpu_mx4 import mx4

pytestmark = pytest.mark.gpu


def test_gemm_of_more_columns_than_31_bits_of_scale_bytes(qsm):
    """2^29 columns have 2^31 bytes of scales before the last ones.  Two values a
    row, at both ends: exact."""
    k = 2 ** 29 + 2 ** 16 + 32
    x = torch.zeros((3, k), dtype=torch.bfloat16, device="cuda")
    x[:, 5] = torch.tensor([1.0, -3.0, 0.5], device="cuda")
    x[:, k - 7] = torch.tensor([2.0, 64.0, -6.0], device="cuda")
    t = qsm.mx4_quantize(x)
    z = torch.stack((x[:, 5], x[:, k - 7]), dim=1).double()
    del x
    for dtype in (torch.bfloat16, torch.float32):
        assert torch.equal(qsm.mx4_gemm(t, t, dtype).double(), (z @ z.T).to(dtype).double())


def test_gemm_of_more_outputs_than_31_bits(qsm):
    m, n, k = 70001, 40008, 64
    a, av = mx4(qsm, torch.randn((m, k), device="cuda"))
    w, wv = mx4(qsm, torch.randn((n, k), device="cuda"))
    y = qsm.mx4_gemm(a, w)
    for rows in (slice(0, 300), slice(2 ** 31 // n - 100, 2 ** 31 // n + 100), slice(m - 300, m)):
        want = av[rows] @ wv.T
        b = k * 2.0 ** -23 * (av[rows].abs() @ wv.abs().T) + want.abs() * 2.0 ** -23
        assert ((y[rows] >= (want - b).to(y.dtype)) & (y[rows] <= (want + b).to(y.dtype))).all()


def test_gemv_of_more_outputs_than_31_bits(qsm):
    t, n, k = 32, 2 ** 26 + 77, 32
    w, wv = mx4(qsm, torch.randn((n, k), device="cuda"))
    x = torch.zeros((t, k), dtype=torch.bfloat16, device="cuda")
    x[torch.arange(t), torch.arange(t)] = 2.0            # twice the columns of w: exact
    y = qsm.mx4_gemv(x, w)
    for i in range(0, t, 5):
        assert torch.equal(y[i].double(), 2 * wv[:, i])
    assert torch.equal(y[t - 1].double(), 2 * wv[:, t - 1])


def test_quantize_more_values_than_32_bits(qsm):
    rows, cols = 2 ** 21 + 5, 2080
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    t = qsm.mx4_quantize(x)
    y = qsm.mx4_dequantize(t)
    for at in (0, 2 ** 31 // cols - 3, 2 ** 32 // cols - 3, rows - 6):
        codes, scales = ref.quantize(x[at:at + 6])
        assert torch.equal(t.codes[at:at + 6].cpu(), codes)
        assert torch.equal(y[at:at + 6].cpu().double(), ref.values(codes, scales).to(y.dtype).double())
