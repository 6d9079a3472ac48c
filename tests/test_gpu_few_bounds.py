"""The few-token layer and product on the GPU against 64-bit forms within the average bounds of
few_bounds, at the sizes of test_gpu_few."""
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
import few_bounds as bounds
import few_ref as ref
from test_gpu_few import LAYER, LINEAR, Weights, gen, normal, random_routing, w4_random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H,I,E,K,dtype,shared,pad,group,zeros,tiled", LAYER)
def test_layer_few_average(T, H, I, E, K, dtype, shared, pad, group, zeros, tiled):
    g = gen(T + H * E)
    w = Weights(g, dtype, H, I, E, shared, group, zeros, tiled)
    x = normal(g, T, H)
    idx, wt = random_routing(g, T, K, E, pad)
    out, _, _ = moe.MoeLayerFew(T, H, I, E, K, **w.kw).forward(x, topk_idx=idx, topk_w=wt)
    want, _ = w.want(x, idx, wt)
    assert bounds.layer_ratio(out, want, w.half) <= 1


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("e4m3", 0), ("w4", 32), ("w4", 128)])
@pytest.mark.parametrize("columns", [1, 4, 6, 8, 13, 16, 32])
def test_layer_few_h_terms(dtype, group, columns):
    """h in two terms, whatever the number of columns an expert has: 1-4 share a tensor instruction,
    5-8 and 9-16 have two, more have two passes."""
    g = gen(columns)
    T, H, I, E = 32, 2048, 640, 32 // columns
    w = Weights(g, dtype, H, I, E, False, group)
    x = normal(g, T, H)
    idx = torch.arange(T, dtype=torch.int32, device="cuda")[:, None] // columns
    idx[idx >= E] = -1
    wt = torch.rand(T, 1, generator=g, device="cuda") + 0.5
    out, _, _ = moe.MoeLayerFew(T, H, I, E, 1, **w.kw).forward(x, topk_idx=idx.contiguous(), topk_w=wt)
    want, _ = w.want(x, idx, wt)
    assert bounds.layer_ratio(out, want, w.half) <= 1
