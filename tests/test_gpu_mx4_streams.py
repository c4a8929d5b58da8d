"""The MXFP4 calls on a stream other than the current one, with nothing between
the two streams but what a caller knows of."""
import pytest
import torch

import _mx4_ref as ref
from test_gpu_mx4 import hidden, layer, mx4

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


@pytest.mark.parametrize("acts,t", [("bf16", 1), ("bf16", 5), ("mx4", 70)])
def test_first_call_waits_for_the_zeroed_buffers(qsm, acts, t):
    """The buffers are zeroed behind much other work of the current stream; the
    first call comes at once on another."""
    L, _ = layer(qsm, 1024, 128, 16, 2, seed=t)
    x = hidden(t, 1024, 1)
    want = qsm.Mx4Forward(L, t, acts, want_f32=True)(x).clone()
    side = torch.cuda.Stream()
    dirty = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del dirty                              # what the buffers are likely made of
    torch.cuda._sleep(HOLD)
    f = qsm.Mx4Forward(L, t, acts, want_f32=True)
    y = f(x, stream=side)
    torch.cuda.synchronize()
    assert f.dev_status.item() == 0 and torch.equal(y, want)
    with torch.cuda.stream(side):          # and with the stream as the current one
        f = qsm.Mx4Forward(L, t, acts)
        y = f(x)
    y = f(x)
    torch.cuda.synchronize()
    assert f.dev_status.item() == 0 and torch.equal(y, want)
