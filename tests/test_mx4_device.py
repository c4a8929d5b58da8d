"""The MXFP4 binding with operands that are not on the current device: the
library launches on the current one, so such a call is refused before it.
Checked on the host with stand-ins for the tensors and the library."""
import pytest
import torch

HERE, THERE = 0, 1


class Fake:
    """As much of a CUDA tensor as the binding looks at."""

    def __init__(self, shape, dtype, dev):
        self.shape, self.dtype, self.dev = torch.Size(shape), dtype, dev
        self.device = torch.device("cuda", dev)

    def stride(self):
        return (self.shape[-1], 1)[-len(self.shape):]

    def get_device(self):
        return self.dev

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 20


class Library:
    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        if name.startswith("_"):
            raise AttributeError(name)

        def call(*a):
            self.called.append(name)
            return 4096 if name.endswith("_bytes") else 0
        return call


class Stream:
    def __init__(self, dev):
        self.cuda_stream, self.device_index, self.waited = 7, dev, 0

    def wait_event(self, event):
        self.waited += 1


class Event:
    def record(self):
        pass


@pytest.fixture
def mx4(monkeypatch):
    from quantized_sparse_moe_gb300 import mx4
    fake = Library()
    monkeypatch.setattr(mx4, "_lib", fake)
    monkeypatch.setattr(mx4, "lib", lambda: fake)
    monkeypatch.setattr(mx4, "_stream_of", lambda dev: 0)
    monkeypatch.setattr(mx4, "_current_device", lambda: HERE)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    mx4.fake = fake
    yield mx4
    del mx4.fake


def tensor(mx4, rows, cols, dev, experts=1):
    u8 = torch.uint8
    return mx4.Mx4Tensor(Fake((experts * rows, cols // 2), u8, dev),
                         Fake((experts * mx4.mx4_scale_bytes(rows, cols),), u8, dev), rows, cols, experts)


def layer(mx4, dev):
    H, I, E = 256, 128, 8
    return mx4.Mx4Layer(H, I, E, 2, tensor(mx4, 2 * I, H, dev, E), tensor(mx4, H, I, dev, E),
                        tensor(mx4, 2 * I, H, dev), tensor(mx4, H, I, dev), Fake((E, H), torch.float32, dev))


def calls(mx4, dev, stream=None):
    bf16 = torch.bfloat16
    a, w = tensor(mx4, 4, 64, dev), tensor(mx4, 8, 64, dev)
    x, y, st = Fake((4, 64), bf16, dev), Fake((4, 8), bf16, dev), Fake((1,), torch.int32, dev)
    return {"mx4_quantize": lambda: mx4.mx4_quantize(x, out=a, dev_status=st, stream=stream),
            "mx4_dequantize": lambda: mx4.mx4_dequantize(a, y=Fake((4, 64), bf16, dev), stream=stream),
            "mx4_gemm": lambda: mx4.mx4_gemm(a, w, y=y, dev_status=st, stream=stream),
            "mx4_gemv": lambda: mx4.mx4_gemv(x, w, y=y, dev_status=st, stream=stream)}


NAMES = ["mx4_quantize", "mx4_dequantize", "mx4_gemm", "mx4_gemv"]


@pytest.mark.parametrize("name", NAMES)
def test_operands_on_another_device_are_refused(mx4, name):
    with pytest.raises(mx4.QSMError):
        calls(mx4, THERE)[name]()
    assert not mx4.fake.called
    calls(mx4, HERE)[name]()
    assert mx4.fake.called == [name]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(mx4, name):
    with pytest.raises(mx4.QSMError):
        calls(mx4, HERE, Stream(THERE))[name]()
    assert not mx4.fake.called
    calls(mx4, HERE, Stream(HERE))[name]()
    assert mx4.fake.called == [name]


def forward(mx4, monkeypatch, dev):
    """An Mx4Forward of stand-ins, built while `dev` is the current device."""
    make = lambda shape, dtype=None, device=None: Fake(shape if isinstance(shape, tuple) else (shape,), dtype, dev)  # noqa: E731
    with monkeypatch.context() as m:
        m.setattr(mx4, "_current_device", lambda: dev)
        m.setattr(torch, "empty", make)
        m.setattr(torch, "zeros", make)
        m.setattr(torch.cuda, "Event", Event)
        f = mx4.Mx4Forward(layer(mx4, dev), 4)
    mx4.fake.called.clear()
    return f


def test_a_layer_on_another_device_is_refused(mx4, monkeypatch):
    with pytest.raises(mx4.QSMError):     # the sizes depend on the current device
        mx4.moe_mx4_workspace_bytes(layer(mx4, THERE), 4)
    with pytest.raises(mx4.QSMError):
        mx4.Mx4Forward(layer(mx4, THERE), 4)
    assert not mx4.fake.called
    for dev, stream, ok in ((THERE, None, False), (HERE, Stream(THERE), False), (HERE, Stream(HERE), True),
                            (HERE, None, True)):
        f = forward(mx4, monkeypatch, dev)
        x = Fake((4, 256), torch.bfloat16, dev)
        if ok:
            f(x, stream=stream)
            assert mx4.fake.called == ["moe_mx4_forward"]
        else:
            with pytest.raises(mx4.QSMError):
                f(x, stream=stream)
            assert not mx4.fake.called


def test_another_stream_waits_for_the_zeroed_buffers(mx4, monkeypatch):
    """Once for each stream, and not inside a capture."""
    f = forward(mx4, monkeypatch, HERE)
    x, s = Fake((4, 256), torch.bfloat16, HERE), Stream(HERE)
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    f(x, stream=s)
    assert s.waited == 0
    capturing[0] = False
    f(x, stream=s)
    f(x, stream=s)
    assert s.waited == 1
    f(x)                                   # the stream that the buffers were made on
    assert mx4.fake.called == ["moe_mx4_forward"] * 4


def test_what_the_calls_point_to_cannot_be_replaced(mx4):
    """The C structures hold addresses that were taken once: another tensor in
    an attribute would not be seen, and the old one's memory be given back."""
    t, L = tensor(mx4, 8, 64, HERE), layer(mx4, HERE)
    for what, names in ((t, ("codes", "scales", "rows", "cols", "experts")),
                        (L, ("gate_up", "down", "shared_gate_up", "shared_down", "shared_gate", "H", "k"))):
        for name in names:
            old = getattr(what, name)
            with pytest.raises(AttributeError):
                setattr(what, name, Fake((1,), torch.uint8, HERE))
            assert getattr(what, name) is old
            setattr(what, name, old)       # as an update in place (a.x -= 1) does
    router = Fake((8, 256), torch.float32, HERE)
    L.w_router, L.logit_bias = router, None    # taken when an Mx4Forward is made
    assert L.w_router is router
