"""Every variant of the product of E4M3 operands at sizes that the library would give to another one, and the waits inside
them: one that runs out sets the status word, and the context and the workspace go on."""
import ctypes
import time

import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import need_gpu
from test_gpu_act8 import check_linear, operands

pytestmark = pytest.mark.gpu
FEW, TILES_64, TILES_128, TILES_256, SWAP = -1, 0, 1, 2, 3
_P, _I, _L, _Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def call(o, variant, parts=1, dtype=torch.float32, limit_ns=2_000_000_000, ws=None, status=None, out=None, mute=0):
    x, xs, w, wsc, bias = o
    (T, K), N = x.shape, w.shape[0]
    f = moe.lib().moe_testing_linear_e4m3
    f.argtypes, f.restype = [_P, _P, _I, _I, _P, _P, _I, _P, _P, _I, _L, _P, _Z, _P, _I, _I, ctypes.c_ulonglong, _I, _P], _I
    if out is None:
        out = torch.full((T, N), torch.nan, dtype=dtype, device="cuda")
    if ws is None:
        ws = moe.moe_linear_e4m3_workspace(1000, 128, 128)
    code = f(x.data_ptr(), xs.data_ptr(), T, K, w.data_ptr(), wsc.data_ptr(), N, None if bias is None else bias.data_ptr(),
             out.data_ptr(), int(out.dtype is torch.float32), out.stride(0), ws.data_ptr(), ws.numel(),
             None if status is None else status.data_ptr(), variant, parts, limit_ns, mute, torch.cuda.current_stream().cuda_stream)
    assert code == 0
    return out


@pytest.mark.parametrize("variant,T", [(FEW, 1), (FEW, 8), (FEW, 9), (FEW, 16), (SWAP, 1), (SWAP, 16), (SWAP, 32), (TILES_64, 1),
                                       (TILES_64, 130), (TILES_64, 1500), (TILES_128, 1), (TILES_128, 300),
                                       (TILES_128, 1100), (TILES_256, 1), (TILES_256, 100), (TILES_256, 385)])
@pytest.mark.parametrize("N,K", [(1, 128), (127, 256), (300, 640), (1029, 2048), (5000, 384), (20000, 128)])
def test_variants(variant, T, N, K):
    o = operands(T, N, K, bias=N % 2 == 0)
    for dtype in (torch.float32, torch.bfloat16):
        check_linear(call(o, variant, dtype=dtype), *o)


@pytest.mark.parametrize("variant,T,N", [(SWAP, 20, 300), (SWAP, 32, 4096), (SWAP, 3, 1), (TILES_64, 20, 300), (TILES_64, 200, 900),
                                         (TILES_64, 128, 1), (TILES_64, 700, 576), (TILES_64, 1100, 1200),
                                         (TILES_128, 20, 300), (TILES_128, 400, 1000), (TILES_128, 2000, 1300),
                                         (SWAP, 32, 20000)])
@pytest.mark.parametrize("K", [128, 384, 2176])
@pytest.mark.parametrize("parts", [2, 3, 5, 8])
def test_shared_k(variant, T, N, K, parts):
    """Parts of unequal length, more parts than K blocks; the sums do not depend on which part comes last."""
    o = operands(T, N, K, bias=True)
    ws = moe.moe_linear_e4m3_workspace(1000, 128, 128)
    first = call(o, variant, parts, ws=ws)
    check_linear(first, *o)
    for _ in range(5):
        assert torch.equal(call(o, variant, parts, ws=ws), first)
    assert not ws[:4096].any()          # the counters are left zero


@pytest.mark.parametrize("variant", [FEW, SWAP, TILES_64, TILES_128, TILES_256])
def test_strided_unaligned_out(variant):
    """An out that starts on an odd element, rows an odd number of elements apart."""
    o = operands(16, 300, 256, bias=True)
    for dtype in (torch.float32, torch.bfloat16):
        buf = torch.full((18, 333), 5.0, dtype=dtype, device="cuda")
        out = call(o, variant, out=buf[1:17, 7:307])
        check_linear(out, *o)
        buf[1:17, 7:307] = 5
        assert (buf == 5).all()


@pytest.mark.parametrize("variant,T,parts", [(FEW, 8, 1), (FEW, 16, 1), (SWAP, 32, 1), (SWAP, 32, 4), (TILES_64, 300, 1),
                                             (TILES_64, 100, 4), (TILES_128, 300, 1), (TILES_128, 200, 3),
                                             (TILES_256, 600, 1)])
@pytest.mark.parametrize("N,K", [(1000, 7168), (300, 128)])
def test_wait_that_runs_out(variant, T, parts, N, K):
    """Copies or MMAs that are never issued, and a limit of 20 ms: the call comes back soon with the status set, and the
    next one is right."""
    o = operands(T, N, K)
    ws = moe.moe_linear_e4m3_workspace(1000, 128, 128)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    begin = time.monotonic()
    call(o, variant, parts, limit_ns=20_000_000, ws=ws, status=status, mute=1)
    torch.cuda.synchronize()
    assert time.monotonic() - begin < 1
    assert status.item() == moe.MOE_DEV_PIPELINE_TIMEOUT
    status.zero_()
    ws.zero_()
    check_linear(call(o, variant, parts, ws=ws, status=status), *o[:4])
    assert status.item() == 0


def test_library_chooses_among_them():
    """Sizes on both sides of each border of the choice give results within the same bounds."""
    for T in (8, 9, 16, 17, 32, 33, 128, 129):
        for N, K in ((576, 1024), (9728, 4096), (9729, 3456)):
            o = operands(T, N, K)
            check_linear(moe.moe_linear_e4m3(*o[:4], out_dtype=torch.float32), *o[:4])
