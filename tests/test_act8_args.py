"""The binding of the 8-bit activation path, on the CPU: device tensors without memory and a stand-in for the library
show what a call would launch, on which stream, and what it refuses before that."""
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from test_few_args import Stream, here, refused  # noqa: F401

BF, F32, I32, U8, I64 = torch.bfloat16, torch.float32, torch.int32, torch.uint8, torch.int64


def names(log):
    return [n for n, _ in log if n != "zeros"]


def test_norm_arguments(here):  # noqa: F811
    log, make = here
    x, w = make(4, 256), make(256)
    f = lambda **k: dict(dict(x=x, weight=w, eps=1e-6), **k)  # noqa: E731
    for bad in (f(x=make(4, 256, dtype=F32)), f(x=torch.empty(4, 256, dtype=BF)), f(x=make(256, 4).T), f(x=make(256)),
                f(weight=make(255)), f(weight=make(256, dtype=torch.float16)), f(weight=torch.empty(256)),
                f(residual=make(4, 128)), f(residual=make(4, 256, dtype=torch.float16)), f(residual=make(8, 256)[::2]),
                f(residual=x, residual_out=make(4, 256, dtype=F32)), f(residual_out=make(4, 256)), f(bf16=False),
                f(out=make(4, 256, dtype=F32)), f(out=make(3, 256)), f(q=make(4, 256, dtype=U8)),
                f(q_scales=make(4, 2, dtype=F32)), f(q=make(4, 256, dtype=U8), q_scales=make(4, 2)),
                f(q=make(4, 256), q_scales=make(4, 2, dtype=F32)), f(num_tokens=make(1, dtype=I64)),
                f(num_tokens=torch.zeros(1, dtype=I32))):
        refused(here, moe.moe_rmsnorm, **bad)
    out, q, s, r = moe.moe_rmsnorm(x, w, 1e-6)
    assert out.shape == (4, 256) and q is s is r is None
    out, q, s, r = moe.moe_rmsnorm(make(4, 300)[:, 8:264], make(256, dtype=F32), 1e-6, residual=make(4, 256, dtype=F32),
                                   bf16=False, e4m3=True, num_tokens=make(1, dtype=I32))
    assert out is None and q.shape == (4, 256) and s.shape == (4, 2) and r.dtype is F32
    res = make(4, 256)
    out, q, s, r = moe.moe_rmsnorm(x, w, 1e-6, residual=res, residual_out=res, q=make(4, 256, dtype=torch.float8_e4m3fn),
                                   q_scales=make(4, 2, dtype=F32))
    assert out is None and r is res
    assert names(log) == ["moe_rmsnorm"] * 3


def test_linear_arguments(here):  # noqa: F811
    log, make = here
    a = dict(x=make(4, 256, dtype=U8), x_scales=make(4, 2, dtype=F32), w=make(130, 256, dtype=U8),
             w_scales=make(2, 2, dtype=F32))
    for bad in (dict(x=make(4, 256)), dict(x=make(256, dtype=U8)), dict(x=make(4, 512, dtype=U8)[:, ::2]),
                dict(x=torch.empty(4, 256, dtype=U8)), dict(x_scales=make(4, 2)), dict(x_scales=make(4, 1, dtype=F32)),
                dict(x_scales=make(2, 4, dtype=F32).T), dict(w=make(130, 128, dtype=U8)), dict(w=make(130, 256, dtype=torch.int8)),
                dict(w_scales=make(1, 2, dtype=F32)), dict(w_scales=make(2, 2, dtype=BF)), dict(bias=make(130)),
                dict(bias=make(128, dtype=F32)), dict(out=make(4, 128)), dict(out=make(4, 130, dtype=I32)),
                dict(out=make(130, 4).T), dict(out_dtype=torch.float16), dict(ws=make(4096)), dict(ws=torch.empty(4096, dtype=U8)),
                dict(dev_status=make(1, dtype=I64))):
        refused(here, moe.moe_linear_e4m3, **{**a, **bad})
    moe.moe_linear_e4m3(**a, bias=make(130, dtype=F32), out=make(4, 160, dtype=F32)[:, 5:135], ws=make(4096, dtype=U8))
    f8 = {k: v if v.dtype is F32 else make(*v.shape, dtype=torch.float8_e4m3fn) for k, v in a.items()}
    assert moe.moe_linear_e4m3(**f8).dtype is BF
    assert names(log) == ["moe_linear_e4m3"] * 2


def test_dispatch_arguments(here):  # noqa: F811
    log, make = here
    a = dict(topk_idx=make(4, 2, dtype=I32), E=8, x=make(4, 256, dtype=U8), x_scales=make(4, 2, dtype=F32))
    for bad in (dict(topk_idx=make(4, 2, dtype=I64)), dict(topk_idx=make(8, dtype=I32)), dict(topk_idx=make(3, 2, dtype=I32)),
                dict(x=make(4, 256)), dict(x=torch.empty(4, 256, dtype=U8)), dict(x_scales=make(4, 3, dtype=F32)),
                dict(xp=make(8, 128, dtype=U8)), dict(xp=make(9, 256, dtype=U8)), dict(xp_scales=make(8, 2)),
                dict(topk_w=make(4, 2)), dict(dev_status=torch.zeros(1, dtype=I32)), dict(ws=torch.empty(9, dtype=U8))):
        refused(here, moe.moe_permute_e4m3, **{**a, **bad})
    p = moe.moe_permute_e4m3(**a, with_shared=True)
    assert p["xp"].shape == (12, 256) and p["cu_seqlens"].shape == (10,) and p["shared_map"].shape == (4,)
    p = moe.moe_permute_e4m3(**a, with_shared=True, max_tokens=5, topk_w=make(4, 2, dtype=F32))
    assert p["xb"].shape == (9, 5, 256) and p["masked_m"].shape == (9,) and p["row_weights"].shape == (45,)
    assert names(log) == ["moe_permute_e4m3"] * 2


def test_layer_arguments(here):  # noqa: F811
    log, make = here
    layer = object.__new__(moe.MoeLayer)
    layer.desc, layer.weights = moe.LayerDesc(4, 256, 128, 8, 2, moe.MOE_E4M3, 0), moe.LayerWeights()
    layer.ws = make(4096, dtype=U8)
    a = dict(x=make(4, 256, dtype=U8), x_scales=make(4, 2, dtype=F32), out=make(4, 256), topk_idx=make(4, 2, dtype=I32),
             topk_w=make(4, 2, dtype=F32))
    for bad in (dict(x=make(4, 256)), dict(x=make(3, 256, dtype=U8)), dict(x_scales=make(4, 1, dtype=F32)),
                dict(out=make(4, 256, dtype=F32)), dict(topk_idx=make(4, 2, dtype=I64)), dict(topk_w=make(4, 2)),
                dict(logits=make(4, 8)), dict(num_tokens=make(1, dtype=I64)), dict(dispatch_scale=make(1, dtype=F32))):
        refused(here, layer.forward, **{**a, **bad})
    layer.forward(**a, logits=make(4, 8, dtype=F32), num_tokens=make(1, dtype=I32))
    assert names(log) == ["moe_layer_forward_e4m3"]
    layer.desc.dtype = moe.MOE_BF16
    refused(here, layer.forward, **a)


@pytest.mark.parametrize("stream", [None, 7])
def test_calls_make_what_they_need_on_their_stream(here, stream):  # noqa: F811
    log, make = here
    s, want = (None, 1) if stream is None else (Stream(stream), stream)
    codes, sc = make(4, 256, dtype=U8), make(4, 2, dtype=F32)
    moe.moe_rmsnorm(make(4, 256), make(256), 1e-6, e4m3=True, stream=s)
    moe.moe_linear_e4m3(codes, sc, make(130, 256, dtype=U8), make(2, 2, dtype=F32), stream=s)
    moe.moe_permute_e4m3(make(4, 2, dtype=I32), 8, codes, sc, stream=s)
    assert names(log) == ["moe_rmsnorm", "moe_linear_e4m3", "moe_permute_e4m3"]
    assert all(at == want for _, at in log), log
