"""The MXFP4 calls on a stream other than the current one, with nothing between
the two streams but what a caller knows of."""
import pytest
import torch

import _mx4_ref as ref
from test_gpu_mx4 import mx4

pytestmark = pytest.mark.gpu
HOLD = 200_000_000      # cycles: about a tenth of a second


def outputs(r):
    return (r.codes, r.scales) if hasattr(r, "codes") else (r,)


@pytest.mark.parametrize("call", ["quantize", "dequantize", "gemm", "gemv"])
def test_outputs_are_not_memory_that_the_current_stream_still_uses(qsm, call):
    """A tensor is freed while the current stream has not written it yet: an
    output of another stream's call must not get its memory."""
    x = ref.draw(24, 4096, 1).to(torch.bfloat16)
    a, w = mx4(qsm, ref.draw(40, 4096, 2))[0], mx4(qsm, ref.draw(512, 4096, 3))[0]
    run = {"quantize": lambda **s: qsm.mx4_quantize(x, **s), "dequantize": lambda **s: qsm.mx4_dequantize(a, **s),
           "gemm": lambda **s: qsm.mx4_gemm(a, w, **s), "gemv": lambda **s: qsm.mx4_gemv(x, w, **s)}[call]
    want = [t.clone() for t in outputs(run())]
    side = torch.cuda.Stream()
    run(stream=side)
    torch.cuda.synchronize()
    torch.cuda._sleep(HOLD)
    late = [torch.full_like(t, 7) for t in want]
    del late
    got = outputs(run(stream=side))
    torch.cuda.synchronize()
    for g, t in zip(got, want):
        assert torch.equal(g, t)
