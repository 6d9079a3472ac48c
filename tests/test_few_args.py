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


# -------------------------------------------------------------------------- what is refused, and what is not
def refused(here, f, *a, **k):
    log = here[0]
    before = len(log)
    with pytest.raises((ValueError, AssertionError, moe.MoeError)):
        f(*a, **k)
    assert not [name for name, _ in log[before:] if name != "zeros"], "it was launched"


def test_linear_arguments(here):
    log, make = here
    x, w = make(4, 256), packed(make)
    cpu = torch.empty(64, dtype=F32)
    for bad in (dict(bias=make(64)), dict(bias=make(63, dtype=F32)), dict(bias=cpu),
                dict(bias=make(128, dtype=F32)[::2]), dict(out=torch.empty(4, 64, dtype=BF)), dict(out=make(4, 64, dtype=I32)),
                dict(out=make(3, 64)), dict(ws=torch.empty(4096, dtype=U8)), dict(ws=make(8192, dtype=U8)[::2]),
                dict(dev_status=make(1, dtype=torch.int64)), dict(dev_status=torch.zeros(1, dtype=I32)),
                dict(out_dtype=torch.float16)):
        refused(here, moe.moe_linear_w4, x, w, **bad)
    for bad in (make(4, 256, dtype=torch.float16), torch.empty(4, 256, dtype=BF), make(4, 128), make(256, 4).T, make(256)):
        refused(here, moe.moe_linear_w4, bad, w)
    refused(here, moe.moe_linear_w4, x, packed(make, mats=2))
    moe.moe_linear_w4(x, w, bias=make(1, 64, dtype=F32), out=make(4, 80, dtype=F32)[:, :64], ws=make(4096, dtype=U8),
                      dev_status=make(1, dtype=I32))
    moe.moe_linear_w4(make(4, 300)[:, 8:264], w)
    assert [n for n, _ in log].count("moe_linear_w4") == 2


def test_packed_weights(here):
    log, make = here
    for bad in (make(1, 4095, dtype=U8), make(2, 4096, dtype=U8), make(1, 4096, dtype=torch.int8), torch.empty(1, 4096, dtype=U8),
                make(4096, dtype=U8)):
        refused(here, moe.W4Packed, bad, 1, 64, 256, 64, False)
    assert moe.W4Packed(make(3, 4096, dtype=U8), 3, 64, 256, 64, False)[2].mats == 1


def test_weight_preparation_arguments(here):
    log, make = here
    for bad in (dict(w=make(64, 256, dtype=F32)), dict(w=make(64, 256, dtype=torch.float16)), dict(group=0), dict(group=48),
                dict(group=16), dict(w=make(64, 0)), dict(w=make(0, 256)), dict(w=torch.empty(64, 256, dtype=BF)),
                dict(w=make(256, 64).T), dict(w=make(64, 160), group=64)):
        refused(here, moe.moe_quantize_weight_w4, **{**dict(w=make(64, 256), group=64), **bad})
    q, s, z = make(64, 128, dtype=U8), make(4, 64), make(4, 64, dtype=U8)
    for bad in (dict(q=make(64, 128, dtype=I32)), dict(q=make(64, 128)), dict(scales=make(4, 64, dtype=F32)),
                dict(scales=make(4, 63)), dict(scales=make(0, 64)), dict(scales=make(3, 64)), dict(zeros=make(4, 64)),
                dict(zeros=make(3, 64, dtype=U8)), dict(zeros=torch.empty(4, 64, dtype=U8)), dict(q=make(0, 128, dtype=U8)),
                dict(q=make(128, 64, dtype=U8).T)):
        refused(here, moe.moe_pack_w4, **{**dict(q=q, scales=s, zeros=z), **bad})
    moe.moe_pack_w4(q, s, z)
    moe.moe_quantize_weight_w4(make(2, 64, 256), 32, True)


def test_route_hidden_arguments(here):
    log, make = here
    x, w = make(4, 256), make(8, 256)
    for bad in (dict(w_router=make(8, 128)), dict(w_router=make(8, 512)), dict(w_router=make(8, 256, dtype=F32)),
                dict(w_router=torch.empty(8, 256, dtype=BF)), dict(w_router=make(256, 8).T), dict(w_router=make(2048)),
                dict(bias=make(8)), dict(bias=make(7, dtype=F32)), dict(bias=torch.empty(8, dtype=F32)),
                dict(num_tokens=make(1, dtype=torch.int64)), dict(num_tokens=torch.tensor([4], dtype=I32)),
                dict(logits=make(4, 8)), dict(logits=make(4, 9, dtype=F32)), dict(logits=make(8, 4, dtype=F32).T),
                dict(topk_idx=make(4, 2, dtype=torch.int64)), dict(topk_idx=make(4, 3, dtype=I32)),
                dict(topk_w=make(4, 2)), dict(topk_w=make(2, 4, dtype=F32).T), dict(ws=torch.empty(256, dtype=U8))):
        refused(here, moe.moe_route_hidden, **{**dict(x=x, w_router=w, K=2), **bad})
    moe.moe_route_hidden(x, w, 2, bias=make(8, dtype=F32), num_tokens=make(1, dtype=I32), logits=make(4, 8, dtype=F32),
                         topk_idx=make(4, 2, dtype=I32), topk_w=make(4, 2, dtype=F32), ws=make(256, dtype=U8))
    assert log[-1][0] == "moe_route_hidden"


def layer_weights(make, dtype, E=8, H=256, I=128, shared=True):
    kw = {}
    for name, e, n, k in (("w13", E, 2 * I, H), ("w2", E, H, I), ("shared_w13", 1, 2 * I, H), ("shared_w2", 1, H, I)):
        if name.startswith("shared") and not shared:
            continue
        lead = () if name.startswith("shared") else (e,)
        if dtype == moe.MOE_W4:
            kw[name] = packed(make, n, k, 64, e)
        elif dtype == moe.MOE_E4M3:
            kw[name] = make(*lead, n, k, dtype=U8)
            kw[name + "_scales"] = make(*lead, n // 128, k // 128, dtype=F32)
        else:
            kw[name] = make(*lead, n, k)
    return kw


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_E4M3, moe.MOE_W4])
def test_layer_weights(here, dtype):
    log, make = here
    good = layer_weights(make, dtype)
    new = lambda **k: moe.MoeLayerFew(4, 256, 128, 8, 2, dtype, **{**good, **k})
    one = U8 if dtype == moe.MOE_E4M3 else BF
    for bad in (dict(w13=make(8, 256, 128, dtype=one)), dict(w13=make(7, 256, 256, dtype=one)), dict(w2=make(8, 128, 256, dtype=one)),
                dict(w2=make(8, 256, 128, dtype=F32)), dict(w2=torch.empty(8, 256, 128, dtype=one)),
                dict(w13=make(256, 256, 8, dtype=one).permute(2, 0, 1)), dict(shared_w2=None), dict(shared_w13=None),
                dict(shared_w13=make(2, 256, 256, dtype=one)), dict(w_router=make(8, 128)), dict(w_router=make(8, 256, dtype=F32)),
                dict(w_router=torch.empty(8, 256, dtype=BF)), dict(w_router=make(8, 256), router_bias=make(8)),
                dict(w_router=make(8, 256), router_bias=make(7, dtype=F32))):
        refused(here, new, **bad)
    if dtype == moe.MOE_E4M3:
        for bad in (make(8, 1, 2, dtype=F32), make(8, 2, 2), make(7, 2, 2, dtype=F32), torch.empty(8, 2, 2, dtype=F32)):
            refused(here, new, w13_scales=bad)
        new(w13=make(8, 256, 256, dtype=torch.float8_e4m3fn), shared_w2=make(1, 256, 128, dtype=U8))
    else:
        refused(here, new, w13=make(8, 256, 256, dtype=U8))
    new(w_router=make(8, 256), router_bias=make(8, dtype=F32))


@pytest.mark.parametrize("dtype", [moe.MOE_BF16, moe.MOE_E4M3, moe.MOE_W4])
def test_layer_forward_arguments(here, dtype):
    log, make = here
    layer = moe.MoeLayerFew(4, 256, 128, 8, 2, dtype, **layer_weights(make, dtype, shared=False))
    x = make(3, 256)
    i, w = make(3, 2, dtype=I32), make(3, 2, dtype=F32)
    for bad in (dict(topk_idx=make(3, 2, dtype=torch.int64)),         # as torch.topk returns them
                dict(topk_idx=None), dict(topk_w=None), dict(topk_idx=None, topk_w=None), dict(topk_w=make(3, 2)),
                dict(topk_idx=make(2, 3, dtype=I32).T), dict(topk_idx=make(2, 2, dtype=I32)), dict(topk_idx=make(3, 3, dtype=I32)),
                dict(topk_idx=torch.empty(3, 2, dtype=I32)), dict(topk_w=make(3, 4, dtype=F32)[:, ::2]),
                dict(out=make(3, 256, dtype=F32)), dict(out=make(3, 512)[:, ::2]), dict(out=make(2, 256)), dict(out=torch.empty(3, 256, dtype=BF)),
                dict(logits=make(3, 8)), dict(logits=make(3, 7, dtype=F32)), dict(logits=make(8, 3, dtype=F32).T),
                dict(num_tokens=make(1, dtype=torch.int64)), dict(num_tokens=torch.zeros(1, dtype=I32)),
                dict(dev_status=make(1, dtype=torch.int64))):
        refused(here, layer.forward, x, **{**dict(topk_idx=i, topk_w=w), **bad})
    for bad in (make(5, 256), make(3, 128), make(3, 256, dtype=F32), make(256, 3).T, torch.empty(3, 256, dtype=BF)):
        refused(here, layer.forward, bad, topk_idx=i, topk_w=w)
    # rows past the call's in a buffer are left alone
    layer.forward(x, out=make(4, 256), topk_idx=make(4, 2, dtype=I32), topk_w=make(4, 2, dtype=F32), logits=make(4, 8, dtype=F32),
                  num_tokens=make(1, dtype=I32), dev_status=make(1, dtype=I32))
    layer.forward(x, logits=make(3, 8, dtype=F32))
    layer.forward(x, logits=make(3, 8, dtype=F32), topk_w=make(3, 2, dtype=F32))
    assert [n for n, _ in log].count("moe_layer_few") == 3
