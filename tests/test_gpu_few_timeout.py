"""The few-token kernels' failure detection, exercised without faulting or hanging anything: every wait is
bounded, the first of a CTA that runs out sets MOE_DEV_PIPELINE_TIMEOUT and ends the others, the copies in flight are
waited for, and the call returns.  Test-only exports of the library run a call with another limit than 2 s."""
import ctypes
import time

import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from test_gpu_few import Weights, gen, normal, random_routing, w4_random

pytestmark = pytest.mark.gpu

MS = 1_000_000


def hook(name):
    """The test-only form of a call: the limit in nanoseconds before the stream."""
    f = getattr(moe.lib(), f"moe_testing_{name}_wait_limit")
    args, f.restype = moe._SIGS["moe_" + name]
    f.argtypes = args[:-1] + [ctypes.c_ulonglong] + args[-1:]
    return f


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("T,N,K,group", [(1, 512, 4096, 128), (5, 4096, 2048, 64), (24, 640, 7168, 32), (70, 320, 7168, 128),
                                         (24, 40960, 4096, 128)])
def test_linear_wait_that_runs_out(T, N, K, group):
    g = gen(T)
    f = hook("linear_w4")
    q, s, z = w4_random(g, 1, N, K, group, True)
    p, x = moe.moe_pack_w4(q, s, z), normal(g, T, K)
    ws = moe.moe_linear_w4_workspace(T, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = moe.moe_linear_w4(x, p, ws=ws)
    out = torch.empty_like(want)

    def call(limit):
        torch.cuda.synchronize()
        t0 = time.monotonic()
        assert f(x.data_ptr(), T, K, K, p.data.data_ptr(), N, group, 1, None, out.data_ptr(), 0, N, ws.data_ptr(), ws.numel(),
                 status.data_ptr(), limit, stream()) == 0
        torch.cuda.synchronize()
        return time.monotonic() - t0
    call(2000 * MS)
    assert status.item() == 0 and torch.equal(out, want)
    # a few nanoseconds: the first wait that does not end at its first look runs out.  With one or two items
    # to a warp that look may be long enough for all of them: the product is whole then.
    assert call(4) < 1.0
    assert status.item() in (0, moe.MOE_DEV_PIPELINE_TIMEOUT)
    if status.item() == 0:
        assert T * N < 1 << 19 and torch.equal(out, want)
    ws.zero_()
    status.zero_()
    assert torch.equal(moe.moe_linear_w4(x, p, ws=ws, dev_status=status), want) and status.item() == 0


LAYERS = [("bf16", 0, False), ("bf16", 0, True), ("e4m3", 0, False), ("e4m3", 0, True), ("w4", 64, False), ("w4", 32, True)]


class Layer:
    def __init__(self, dtype, group, router, T=6, H=2048, I=1408, E=12, K=4):
        g = gen(T + group)
        self.f = hook("layer_few")
        kw = dict(w_router=normal(g, E, H, std=H ** -0.5)) if router else {}
        self.layer = moe.MoeLayerFew(T, H, I, E, K, **Weights(g, dtype, H, I, E, True, group).kw, **kw)
        self.x = normal(g, T, H)
        self.idx, self.wt = random_routing(g, T, K, E, 0.0)
        self.idx2, self.wt2 = self.idx.clone(), self.wt.clone()        # written where the layer routes
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.want = self.forward()
        self.out = torch.empty_like(self.want)
        assert self.status.item() == 0

    def forward(self):
        return self.layer.forward(self.x, topk_idx=self.idx2, topk_w=self.wt2, dev_status=self.status)[0]

    def call(self, limit):
        """Seconds of a call with that limit of each wait."""
        n = self.layer
        torch.cuda.synchronize()
        t0 = time.monotonic()
        d = n._descs[self.x.shape[0]]
        assert self.f(ctypes.byref(d), n._w, self.x.data_ptr(), None, None, self.idx2.data_ptr(),
                      self.wt2.data_ptr(), self.out.data_ptr(), *n._ws, self.status.data_ptr(), limit, stream()) == 0
        torch.cuda.synchronize()
        return time.monotonic() - t0

    def works_again(self):
        self.layer.ws.zero_()
        self.status.zero_()
        return torch.equal(self.forward(), self.want) and self.status.item() == 0


@pytest.mark.parametrize("dtype,group,router", LAYERS)
def test_layer_wait_that_runs_out(dtype, group, router):
    """A limit of a few nanoseconds: grid barrier, copies, h of other CTAs, whichever comes first."""
    n = Layer(dtype, group, router)
    n.call(2000 * MS)
    assert n.status.item() == 0 and torch.equal(n.out, n.want)
    assert n.call(4) < 1.0
    assert n.status.item() == moe.MOE_DEV_PIPELINE_TIMEOUT
    assert n.works_again()


@pytest.mark.parametrize("dtype,group,router", LAYERS)
def test_layer_waits_end_together(dtype, group, router):
    """Counters that are not zero at the start: no expert's h is ever reported ready, and hundreds of units wait for
    it.  The call is over a few limits later, not a limit per unit."""
    n = Layer(dtype, group, router)
    at = 256 + -(-4 * (2048 // 32) // 256) * 256          # behind the barrier and the row tiles' counters
    n.layer.ws[at:at + 4 * 1024].view(torch.int32).fill_(1 << 20)
    assert n.call(100 * MS) < 0.8
    assert n.status.item() == moe.MOE_DEV_PIPELINE_TIMEOUT
    assert n.works_again()
