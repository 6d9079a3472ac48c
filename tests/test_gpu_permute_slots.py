"""The permute with as many slots per token as it takes, and a shared expert."""
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(out_dtype=moe.MOE_E4M3), dict(scale="e4m3"), dict(scale="nvfp4")])
def test_permute_of_32_slots_keeps_the_shared_row(kw):
    """Top-32 with a shared expert: a token has 33 destination rows, one more than a warp has lanes."""
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(7)
    T, H, E, K = 40, 512, 40, 32
    idx = torch.topk(torch.randn(T, E, generator=g, device="cuda"), K, 1)[1].to(torch.int32)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    more = dict(kw)
    if "scale" in kw:
        more = dict(dispatch_format=more["scale"], dispatch_scale=torch.full((1,), 16.0, device="cuda"))
    p = moe.moe_permute(idx, E, x, with_shared=True, **more)
    rows = p["xp"][p["shared_map"].long()]
    if "out_dtype" in kw:
        q, s = moe.moe_quantize_act_fp8(x)
        assert torch.equal(rows, q) and torch.equal(p["xp_scales"][p["shared_map"].long()], s)
    else:
        assert torch.equal(rows, x)
