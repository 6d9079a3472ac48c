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


# sizes that share K out in other ways: with the most slots of the joins, with fewer, not at all
SHARED = [(17, 512, 7168, 128, False, False, True), (20, 2048, 4096, 32, True, False, True), (24, 1056, 2048, 64, True, True, False),
          (25, 2048, 4096, 128, False, False, True), (28, 7168, 1408, 32, False, True, True), (32, 7168, 7168, 32, True, False, True),
          (40, 512, 11008, 64, False, False, True), (64, 2048, 4096, 32, True, True, True), (9, 7168, 14336, 32, True, False, False)]


@pytest.mark.parametrize("T,N,K,group,zeros,bias,f32", LINEAR + SHARED)
def test_linear_w4_average(T, N, K, group, zeros, bias, f32):
    g = gen(T + N * K)
    if N > 5:
        q, s, z = w4_random(g, 1, N, K, group, zeros)
    else:
        q = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = normal(g, 1, K // group, N)
        z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    x = normal(g, T, K)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.moe_linear_w4(x, moe.moe_pack_w4(q, s, z), bias=b, out_dtype=torch.float32 if f32 else torch.bfloat16,
                          dev_status=status)
    want, _ = ref.linear(x, ref.w4_values(q[0], s[0], None if z is None else z[0]), b)
    assert status.item() == 0 and bounds.linear_ratio(y, want, K) <= 1
