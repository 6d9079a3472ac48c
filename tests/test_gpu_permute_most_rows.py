"""The batched permute with the most rows that it takes, 2^31 - 1, of which one is real: src_row is written to its end and
not past it.  Rows that are not real are neither read nor written, so the one row is all there is of xb here."""
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
MOST, H = 2 ** 31 - 1, 128


@pytest.mark.parametrize("codes", [True, False])       # one launch, four launches
def test_src_row_of_the_most_rows(codes):
    need_gpu()
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    guard = 1 << 20
    src = torch.full((guard + MOST + guard,), 7, dtype=torch.int32, device="cuda")
    idx = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    x = torch.arange(H, device="cuda").to(torch.uint8 if codes else torch.bfloat16)
    xb, xs = torch.zeros_like(x), torch.ones(1, device="cuda")
    scales, mm, inv = torch.zeros(1, device="cuda"), torch.zeros_like(idx), torch.zeros_like(idx) - 9
    ws = torch.empty(moe.moe_permute_batched_workspace_bytes(1, 1, 1, False), dtype=torch.uint8, device="cuda")
    p, stream = lambda t: t.data_ptr(), torch.cuda.current_stream().cuda_stream
    rows = src[guard:guard + MOST]
    if codes:
        code = moe.lib().moe_permute_e4m3(p(idx), 1, 1, 1, 0, MOST, p(x), p(xs), H, p(xb), p(scales), None, p(mm), p(rows), p(inv),
                                          None, p(ws), ws.numel(), None, None, None, stream)
    else:
        code = moe.lib().moe_permute_batched(p(idx), 1, 1, 1, 0, MOST, p(x), H, moe.MOE_BF16, p(xb), None, p(mm), p(rows), p(inv),
                                             None, p(ws), ws.numel(), None, None, 0, None, None, stream)
    torch.cuda.synchronize()
    assert code == 0 and mm.item() == 1 and inv.item() == 0 and torch.equal(xb, x)
    assert rows[0].item() == 0 and (not codes or scales.item() == 1)
    for i in range(1, MOST, 1 << 28):
        assert (rows[i:i + (1 << 28)] == -1).all()
    assert (src[:guard] == 7).all() and (src[-guard:] == 7).all()
