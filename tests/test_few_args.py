"""The binding of the few-token calls, on the CPU: device tensors without memory and a stand-in for the
library show what a call would launch, on which stream, and what it refuses before that."""
import contextlib
import warnings

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import combine_moe_route_softmax_gb300 as moe

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Library:
    """Counts launches and says on which stream each was; sizes are made up."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 4096
        def call(*a):
            self.log.append((name, a[-1]))          # the stream is the last argument
            return 0
        return call


@pytest.fixture
def here(monkeypatch):
    """(log of launches and zeroed workspaces, tensor maker); the current stream is 1 unless changed."""
    log, current = [], [1]

    @contextlib.contextmanager
    def on(stream):
        current.append(stream.cuda_stream)
        yield
        current.pop()
    zeros = torch.zeros

    def logged_zeros(*a, **k):
        log.append(("zeros", current[-1]))
        return zeros(*a, **k)
    lib = Library(log)
    monkeypatch.setattr(moe, "_lib", lib)
    monkeypatch.setattr(moe, "lib", lambda: lib)
    monkeypatch.setattr(moe, "_ptr", lambda t: 4096 if isinstance(t, torch.Tensor) else t)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: current[-1], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with FakeTensorMode(), warnings.catch_warnings():
        warnings.simplefilter("ignore")
        monkeypatch.setattr(torch, "zeros", logged_zeros)
        make = lambda *shape, dtype=BF: torch.empty(*shape, dtype=dtype, device="cuda")
        yield log, make


def packed(make, N=64, K=256, group=64, mats=1):
    return moe.W4Packed(make(mats, 4096, dtype=U8), mats, N, K, group, False)


@pytest.mark.parametrize("stream", [None, 7])
def test_calls_make_what_they_need_on_their_stream(here, stream):
    """A workspace is zeroed, and the kernel launched, on the call's stream."""
    log, make = here
    s = None if stream is None else Stream(stream)
    want = stream or 1
    x = make(4, 256)
    moe.moe_linear_w4(x, packed(make), stream=s)
    moe.moe_route_hidden(x, make(8, 256), 2, stream=s)
    moe.moe_pack_w4(make(64, 128, dtype=U8), make(4, 64), stream=s)
    moe.moe_quantize_weight_w4(make(64, 256), 64, stream=s)
    layer = moe.MoeLayerFew(4, 256, 128, 8, 2, w13=make(8, 256, 256), w2=make(8, 256, 128), w_router=make(8, 256))
    assert log.pop() == ("zeros", 1)
    layer.forward(x, stream=s)
    assert len(log) == 7
    assert all(at == want for _, at in log), log
