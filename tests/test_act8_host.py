"""Host side of the 8-bit activation path, on the CPU: sizes, refusals of the C calls (nothing is launched), and the
plain forms of its tests against other ones."""
import ctypes

import pytest
import torch

import act8_ref as ref
import combine_moe_route_softmax_gb300 as moe

A = 1 << 30      # a device-looking address, never dereferenced
ERR_ARG, ERR_WS, ERR_UNSUPPORTED = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from combine_moe_route_softmax_gb300 import build
        build.build()
    return moe.lib()


def test_norm_refusals(lib):
    names = ("x", "T", "H", "xs", "w", "w32", "eps", "r", "r32", "ro", "out", "q", "qs", "n")
    d = dict(x=A, T=4, H=256, xs=256, w=A, w32=0, eps=1e-6, r=A, r32=0, ro=A, out=A, q=A, qs=A, n=None)
    f = lambda **k: lib.moe_rmsnorm(*[{**d, **k}[n] for n in names], None)  # noqa: E731
    for bad in (dict(T=-1), dict(H=0), dict(H=-8), dict(H=260), dict(H=65544), dict(H=264, xs=264), dict(xs=255), dict(xs=248),
                dict(xs=260), dict(w32=2), dict(r32=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None), dict(w=None),
                dict(out=None, q=None, qs=None), dict(q=None), dict(qs=None), dict(r=None), dict(ro=None), dict(x=A + 8),
                dict(w=A + 4), dict(r=A + 8), dict(ro=A + 2), dict(out=A + 8), dict(q=A + 4), dict(qs=A + 2), dict(n=A + 1)):
        assert f(**bad) == ERR_ARG, bad
    assert f(T=0, x=None, w=None) == 0


def test_linear_refusals(lib):
    size = lib.moe_linear_e4m3_workspace_bytes
    assert size(4, 64, 256) > 0 and size(0, 64, 256) > 0
    for t, n, k in ((-1, 64, 256), (4, 0, 256), (4, 64, 0), (4, 64, 200), (4, (1 << 24) + 1, 256), (4, 64, (1 << 22) + 128)):
        assert size(t, n, k) == 0
    names = ("x", "xs", "T", "K", "w", "ws", "N", "b", "out", "f32", "os", "wk", "nwk")
    d = dict(x=A, xs=A, T=4, K=256, w=A, ws=A, N=64, b=None, out=A, f32=0, os=64, wk=A, nwk=size(4, 64, 256))
    f = lambda **k: lib.moe_linear_e4m3(*[{**d, **k}[n] for n in names], None, None)  # noqa: E731
    for bad in (dict(T=-1), dict(K=100), dict(N=0), dict(os=63), dict(f32=2), dict(x=None), dict(xs=None), dict(w=None),
                dict(ws=None), dict(out=None), dict(x=A + 8), dict(w=A + 8), dict(xs=A + 2), dict(ws=A + 1), dict(b=A + 2),
                dict(out=A + 1), dict(out=A + 2, f32=1), dict(wk=A + 64)):
        assert f(**bad) == ERR_ARG, bad
    assert f(wk=None) == ERR_WS and f(nwk=255) == ERR_WS
    assert f(T=0, x=None, xs=None, out=None) == 0


def test_rows_past_32_bits_are_refused(lib):
    """Rows and the steps between them are counted in 32 bits: 2^30 rows are the most."""
    most = 1 << 30
    assert lib.moe_rmsnorm(A, most + 1, 8, 8, A, 0, 1e-6, None, 0, None, A, None, None, None, None) == ERR_ARG
    assert lib.moe_rmsnorm(A, (1 << 31) - 1, 8, 8, A, 0, 1e-6, None, 0, None, A, None, None, None, None) == ERR_ARG
    assert lib.moe_linear_e4m3_workspace_bytes(most, 1, 128) > 0
    for T in (most + 1, (1 << 31) - 1):
        assert lib.moe_linear_e4m3_workspace_bytes(T, 1, 128) == 0
        assert lib.moe_linear_e4m3(A, A, T, 128, A, A, 1, None, A, 0, 1, A, 1 << 30, None, None) == ERR_ARG


@pytest.mark.parametrize("N,K", [(64, 256), (576, 7168), (4096, 7168), (40960, 4096), (7168, 16384), (1, 128)])
def test_linear_workspace_serves_fewer_rows(lib, N, K):
    """The size never falls with the rows: a workspace made for T rows serves any number up to T."""
    last = 0
    for T in list(range(1, 700)) + [1000, 2000, 4096, 8192, 16384]:
        n = lib.moe_linear_e4m3_workspace_bytes(T, N, K)
        assert n >= last and n % 256 == 0, T
        last = n


def test_dispatch_and_layer_refusals(lib):
    names = ("idx", "T", "K", "E", "sh", "mt", "x", "xs", "H", "xp", "xps", "cu", "mm", "src", "inv", "smap", "ws", "nws")
    need = lib.moe_permute_workspace_bytes(4, 2, 8, 1)
    d = dict(idx=A, T=4, K=2, E=8, sh=1, mt=0, x=A, xs=A, H=256, xp=A, xps=A, cu=A, mm=None, src=A, inv=A, smap=A, ws=A, nws=need)
    f = lambda **k: lib.moe_permute_e4m3(*[{**d, **k}[n] for n in names], None, None, None, None)  # noqa: E731
    for bad in (dict(T=-1), dict(K=0), dict(E=0), dict(sh=2), dict(mt=-1), dict(H=100), dict(x=None), dict(xs=None),
                dict(xp=None), dict(xps=None), dict(cu=None), dict(src=None), dict(inv=None), dict(smap=None), dict(x=A + 8),
                dict(xp=A + 4), dict(xs=A + 2), dict(mt=4), dict(idx=None)):
        assert f(**bad) == ERR_ARG, bad
    assert f(nws=need - 1) == ERR_WS and f(ws=None) == ERR_WS
    assert f(H=116224) == ERR_UNSUPPORTED
    desc = moe.LayerDesc(4, 256, 128, 8, 2, moe.MOE_E4M3, 0)
    n = lib.moe_layer_workspace_bytes(ctypes.byref(desc))
    w = moe.LayerWeights(A, A, A, A, None, None, None, None)
    g = lambda desc=desc, xs=A, nws=n, x=A: lib.moe_layer_forward_e4m3(  # noqa: E731
        ctypes.byref(desc), ctypes.byref(w), None, None, A, A, x, xs, None, A, A, nws, None, None)
    assert g(xs=None) == ERR_ARG and g(x=None) == ERR_ARG and g(xs=A + 1) == ERR_ARG and g(nws=n - 1) == ERR_WS
    assert g(desc=moe.LayerDesc(4, 256, 128, 8, 2, moe.MOE_BF16, 0)) == ERR_ARG


# -------------------------------------------------------------------------------------- plain forms
def test_plain_e4m3_values_are_torchs():
    q = torch.arange(256, dtype=torch.uint8)
    a, b = ref.e4m3_values(q), q.view(torch.float8_e4m3fn).double()
    assert torch.equal(a.nan_to_num(1e9), b.nan_to_num(1e9)) and a.isnan().sum() == 2


def test_plain_norm_and_code_bounds():
    g = torch.Generator().manual_seed(0)
    x, w = torch.randn(5, 256, generator=g), torch.rand(256, generator=g)
    y, h = ref.norm(x, w, 1e-5, x * 0.5)
    want = torch.nn.functional.rms_norm(1.5 * x.double(), (256,), w.double(), 1e-5)
    assert torch.allclose(y, want, rtol=1e-7) and torch.allclose(h, 1.5 * x.double())
    lo, hi = ref.code_bounds(y, 0.0)
    assert torch.equal(lo, hi) and lo.max() == 448
    s = ref.block_scales(y).repeat_interleave(128, 1)
    assert ((lo * s - y.abs()).abs() <= torch.maximum(y.abs() * 2.0 ** -4, s * 2.0 ** -10) * 1.0001).all()
    wrong = ref.code_bounds(y * 1.02, 0.0)[0]      # a scale per block hides a common factor,
    assert torch.equal(wrong, lo)
    wrong = ref.code_bounds(y.roll(1, 1), 0.0)[0]  # not another column
    assert not torch.equal(wrong, lo)


def test_plain_linear():
    """By scalar loops, and what its bound turns away."""
    g = torch.Generator().manual_seed(1)
    T, N, K = 3, 130, 256
    x = (torch.randn(T, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    w = (torch.randn(N, K, generator=g) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    xs, ws = torch.rand(T, 2, generator=g), torch.rand(2, 2, generator=g)
    y, err = ref.linear(x, xs, w, ws)
    xv, wv = x.double(), w.double()
    for t, n in ((0, 0), (2, 127), (1, 128), (2, 129)):
        s = sum(float(xv[t, k]) * float(wv[n, k]) * float(xs[t, k // 128]) * float(ws[n // 128, k // 128]) for k in range(K))
        assert abs(s - float(y[t, n])) < 1e-9 * abs(s) + 1e-6
    short, _ = ref.linear(x[:, :128], xs[:, :1], w[:, :128], ws[:, :1])
    swapped, _ = ref.linear(x, xs.flip(1), w, ws)
    for other in (short, swapped):
        assert ((other - y).abs() > err).float().mean() > 0.9


def test_plain_permute_against_the_oracle():
    from oracle import moe_ref
    g = torch.Generator().manual_seed(2)
    idx = torch.topk(torch.randn(20, 6, generator=g), 3, 1)[1].to(torch.int32)
    idx[torch.rand(20, 3, generator=g) < 0.2] = -1
    a = ref.permute(idx, 6, True)
    for k, want in zip(("cu", "src", "inv", "smap"), moe_ref.permute(idx.numpy(), 6, with_shared=True)):
        assert a[k].tolist() == want.tolist(), k
