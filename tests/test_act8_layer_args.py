"""What MoeLayer.forward on E4M3 rows refuses beside shapes and types: tensors of another device than the current one (the
kernels would be launched here with addresses of there), and a combine scale of another type."""
import torch

import combine_moe_route_softmax_gb300 as moe
from test_few_args import here, refused  # noqa: F401

F32, I32, U8 = torch.float32, torch.int32, torch.uint8


def test_layer_tensors_are_on_the_current_device(here):  # noqa: F811
    log, make = here
    layer = object.__new__(moe.MoeLayer)
    layer.desc, layer.weights = moe.LayerDesc(4, 256, 128, 8, 2, moe.MOE_E4M3, 0), moe.LayerWeights()
    layer.ws = make(4096, dtype=U8)
    kinds = dict(x=((4, 256), U8), x_scales=((4, 2), F32), out=((4, 256), torch.bfloat16), topk_idx=((4, 2), I32),
                 topk_w=((4, 2), F32), logits=((4, 8), F32), num_tokens=((1,), I32), dev_status=((1,), I32), fq_scale=((1,), F32))
    a = {k: make(*shape, dtype=t) for k, (shape, t) in kinds.items()}
    for k, (shape, t) in kinds.items():
        refused(here, layer.forward, **{**a, k: torch.empty(shape, dtype=t, device="cuda:1")})
    refused(here, layer.forward, **{**a, "fq_scale": make(1, dtype=torch.float64)})
    refused(here, layer.forward, **{**a, "fq_scale": torch.ones(1)})
    layer.forward(**a)
    assert [n for n, _ in log if n != "zeros"] == ["moe_layer_forward_e4m3"]
    layer.ws = torch.empty(4096, dtype=U8, device="cuda:1")
    refused(here, layer.forward, **a)
