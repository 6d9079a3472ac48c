"""The few-token operators at sizes whose weights pass 32-bit offsets: 256 experts at H = 7168, I = 2048, and a
head of 300,032 rows at K = 16384."""
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
import few_bounds as bounds
import few_ref as ref
from test_gpu_few import Weights, gen, normal, w4_random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,group,zeros,tiled,T", [("bf16", 0, False, False, 3), ("bf16", 0, False, True, 1),
                                                       ("e4m3", 0, False, False, 1), ("e4m3", 0, False, True, 6),
                                                       ("w4", 32, True, False, 2), ("w4", 128, False, False, 9)])
def test_layer_few_all_experts(dtype, group, zeros, tiled, T):
    g = gen(T + group)
    H, I, E, K = 7168, 2048, 256, 4
    w = Weights(g, dtype, H, I, E, False, group, zeros, tiled)
    x = normal(g, T, H)
    idx = torch.tensor([[255, 0, 254, 128], [127, 255, 3, 200], [254, 255, 129, -1]], dtype=torch.int32, device="cuda")
    idx = idx[torch.arange(T, device="cuda") % 3].contiguous()
    wt = torch.rand(T, K, generator=g, device="cuda") + 0.2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _, _ = moe.MoeLayerFew(T, H, I, E, K, **w.kw).forward(x, topk_idx=idx, topk_w=wt, dev_status=status)
    want, err = w.want(x, idx, wt)
    assert status.item() == 0 and ref.close(out, want, err) <= 1 and bounds.layer_ratio(out, want, w.half) <= 1


@pytest.mark.parametrize("T", [1, 11])
def test_linear_w4_long_head(T):
    g = gen(T)
    N, K, group = 300032, 16384, 128
    q, s, z = w4_random(g, 1, N, K, group, True)
    x = normal(g, T, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = moe.moe_pack_w4(q, s, z)
    y = moe.moe_linear_w4(x, p, out_dtype=torch.float32, dev_status=status)
    assert status.item() == 0
    for rows in (slice(0, 512), slice(149984, 150496), slice(N - 1024, N)):
        want, err = ref.linear(x, ref.w4_values(q[0, rows], s[0][:, rows], z[0][:, rows]))
        assert ref.close(y[:, rows], want, err) <= 1 and bounds.linear_ratio(y[:, rows], want, K) <= 1
