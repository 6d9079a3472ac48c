"""Host side of the few-token calls, on the CPU: sizes, refusals (nothing is launched), and the
plain forms of their tests against one another."""
import ctypes

import numpy as np
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
import few_ref as ref

A = 1 << 30      # a device-looking address, never dereferenced
ERR_ARG, ERR_WS = 1, 2


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(moe.LIB_PATH):
        from combine_moe_route_softmax_gb300 import build
        build.build()
    return moe.lib()


def test_packed_sizes(lib):
    block = 2048 + 8 * 8 * 4      # group 32: codes and scales of 16 rows x 256 columns
    assert lib.moe_w4_packed_bytes(32, 256, 32, 0) == 2 * block
    assert lib.moe_w4_packed_bytes(1, 128, 32, 1) == 2 * (block + 128)      # padded to 32 rows x 256 columns
    assert lib.moe_w4_packed_bytes(4096, 7168, 128, 0) == 4096 // 16 * 28 * (2048 + 64)
    for n, k, g, z in ((0, 256, 32, 0), (32, 0, 32, 0), (32, 200, 32, 0), (-1, 256, 32, 0), (1 << 25, 256, 32, 0),
                       (32, 1 << 23, 32, 0), (32, 256, 48, 0), (32, 256, 32, 2)):
        assert lib.moe_w4_packed_bytes(n, k, g, z) == 0


def test_quantize_and_pack_refusals(lib):
    q = lambda **k: lib.moe_quantize_weight_w4(*[{**dict(w=A, mats=1, rows=16, cols=128, group=32, q=A, s=A, z=None),
                                                  **k}[n] for n in ("w", "mats", "rows", "cols", "group", "q", "s", "z")],
                                               None)
    for bad in (dict(group=16), dict(group=96), dict(cols=96), dict(rows=0), dict(mats=-1), dict(w=None), dict(q=None),
                dict(s=None)):
        assert q(**bad) == ERR_ARG, bad
    assert q(mats=0, w=None) == 0
    names = ("q", "s", "z", "mats", "N", "K", "group", "out")
    d = dict(q=A, s=A, z=A, mats=1, N=32, K=256, group=64, out=2 * A)
    p = lambda **k: lib.moe_pack_w4(*[{**d, **k}[n] for n in names], None)
    for bad in (dict(q=None), dict(s=None), dict(out=None), dict(out=2 * A + 8), dict(s=A + 1), dict(q=A + 2),
                dict(out=A + 1024), dict(group=8), dict(mats=2, N=48), dict(K=192)):
        assert p(**bad) == ERR_ARG, bad
    assert p(mats=0) == 0


def test_linear_refusals(lib):
    ws = lib.moe_linear_w4_workspace_bytes(4, 64, 256)
    assert ws > 0 and lib.moe_linear_w4_workspace_bytes(-1, 64, 256) == 0
    names = ("x", "T", "K", "xs", "w", "N", "group", "z", "b", "out", "f32", "os", "ws", "nws")
    d = dict(x=A, T=4, K=256, xs=256, w=A, z=0, N=64, group=64, b=None, out=A, f32=0, os=64, ws=A, nws=ws)
    f = lambda **k: lib.moe_linear_w4(*[{**d, **k}[n] for n in names], None, None)
    for bad in (dict(T=-1), dict(K=100), dict(xs=248), dict(xs=260), dict(os=63), dict(group=48), dict(N=0), dict(f32=2),
                dict(z=2), dict(x=None), dict(w=None), dict(out=None), dict(x=A + 8), dict(w=A + 8), dict(out=A + 1),
                dict(b=A + 2), dict(ws=A + 64)):
        assert f(**bad) == ERR_ARG, bad
    assert f(ws=None) == ERR_WS and f(nws=ws - 1) == ERR_WS
    assert f(T=0, x=None) == 0


def test_route_hidden_refusals(lib):
    n = lib.moe_route_hidden_workspace_bytes()
    names = ("x", "T", "H", "w", "b", "E", "K", "n", "l", "i", "v", "ws", "nws")
    d = dict(x=A, T=4, H=256, w=A, b=None, E=8, K=2, n=None, l=A, i=A, v=A, ws=A, nws=n)
    f = lambda **k: lib.moe_route_hidden(*[{**d, **k}[m] for m in names], None)
    for bad in (dict(T=33), dict(T=-1), dict(H=200), dict(E=0), dict(E=1025), dict(K=0), dict(K=9), dict(E=64, K=33),
                dict(x=None), dict(w=None), dict(l=None), dict(i=None), dict(v=None), dict(x=A + 2), dict(w=A + 8),
                dict(ws=A + 16)):
        assert f(**bad) == ERR_ARG, bad
    assert f(ws=None) == ERR_WS and f(nws=n - 1) == ERR_WS
    assert f(T=0, x=None) == 0


def desc(**k):
    v = dict(T=4, H=256, I=128, E=8, K=2, dtype=moe.MOE_BF16, has_shared=0, weight_tiles=0, group=0, zeros=0)
    v.update(k)
    return moe.FewDesc(*[v[f] for f, _ in moe.FewDesc._fields_])


def test_layer_few_descriptor(lib):
    size = lambda **k: lib.moe_layer_few_workspace_bytes(ctypes.byref(desc(**k)))
    assert size() > 0 and size(T=0) > 0 and size(T=32) > size()
    assert size(dtype=moe.MOE_W4, group=32) > 0 and size(dtype=moe.MOE_E4M3, weight_tiles=1) > 0
    for bad in (dict(T=33), dict(T=-1), dict(H=192), dict(I=0), dict(E=0), dict(E=1025), dict(K=9), dict(K=0),
                dict(dtype=3), dict(has_shared=2), dict(weight_tiles=2), dict(group=64), dict(dtype=moe.MOE_W4),
                dict(dtype=moe.MOE_W4, group=48), dict(dtype=moe.MOE_W4, group=64, weight_tiles=1), dict(zeros=1),
                dict(dtype=moe.MOE_W4, group=64, zeros=2), dict(H=1 << 18)):
        assert size(**bad) == 0, bad


def test_layer_few_refusals(lib):
    def call(d=None, w=None, **k):
        d = d or desc()
        v = dict(x=A, l=None, n=None, i=A, v=A, out=A, ws=A, nws=lib.moe_layer_few_workspace_bytes(ctypes.byref(d)))
        v.update(k)
        f = dict(w13=A, w2=A)
        f.update(w or {})
        wts = moe.FewWeights(**f)
        return lib.moe_layer_few(ctypes.byref(d), ctypes.byref(wts), *[v[m] for m in ("x", "l", "n", "i", "v", "out", "ws",
                                                                                      "nws")], None, None)
    for bad in (dict(x=None), dict(i=None), dict(v=None), dict(out=None), dict(x=A + 8), dict(ws=A + 16),
                dict(w=dict(w13=None)), dict(w=dict(w2=None)), dict(w=dict(w13=A + 8)), dict(w=dict(w2=A + 8)),
                dict(w=dict(w_router=A), l=A), dict(w=dict(w_router=A + 2)),
                dict(d=desc(has_shared=1)), dict(d=desc(has_shared=1), w=dict(shared_w13=A)),
                dict(d=desc(dtype=moe.MOE_E4M3)), dict(d=desc(dtype=moe.MOE_E4M3), w=dict(w13_scales=A)),
                dict(d=desc(dtype=moe.MOE_E4M3, has_shared=1),
                     w=dict(w13_scales=A, w2_scales=A, shared_w13=A, shared_w2=A)),
                dict(d=desc(E=1024, H=1 << 17, I=1 << 17, weight_tiles=1))):     # coordinates past int32
        assert call(**bad) == ERR_ARG, bad
    assert call(ws=None) == ERR_WS
    assert call(nws=lib.moe_layer_few_workspace_bytes(ctypes.byref(desc())) - 1) == ERR_WS
    bad = desc(H=100)
    assert call(d=bad, nws=1 << 30) == ERR_ARG
    assert call(d=desc(T=0), x=None) == 0


def test_binding_refusals():
    p = moe.W4Packed(None, 1, 256, 256, 32, False)
    with pytest.raises(ValueError):     # a packed matrix of another shape
        moe.MoeLayerFew(1, 256, 256, 2, 1, moe.MOE_W4, w13=p, w2=p, device="cpu")
    with pytest.raises(IndexError):
        p[1]


@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
def test_reference_pack_keeps_values(group, zeros):
    """few_ref.pack_w4 read back by the kernels' rule (lane, word, nibble) gives every value."""
    rng = np.random.default_rng(group)
    N, K = 40, 384
    q = rng.integers(0, 256, (N, K // 2), dtype=np.uint8)
    s = rng.integers(0, 1 << 16, (K // group, N), dtype=np.uint16)
    z = rng.integers(0, 16, (K // group, N), dtype=np.uint8) if zeros else None
    ng, nsl = 256 // group, 2
    data = ref.pack_w4(q, s, z)
    blocks = data.reshape(-1, nsl, 2048 + 8 * ng * (6 if zeros else 4))
    code = ref.unpack_codes(torch.from_numpy(q)).numpy()
    for n, k in [(0, 0), (7, 5), (8, 129), (17, 255), (31, 256), (39, 383), (24, 301)]:
        b = blocks[n // 16, k // 256]
        r, kk = n % 16, k % 256
        j, t, i = kk // 32, kk % 32 // 8, kk % 8
        at = r // 8 * 1024 + j // 4 * 512 + ((r % 8) * 4 + t) * 16 + j % 4 * 4
        w = int(b[at:at + 4].view(np.uint32)[0])
        assert (w >> (4 * (i // 2 + 4 * (i % 2)))) & 15 == code[n, k]
        o = ((r % 8) * ng + kk // group) * 2 + r // 8
        assert b[2048:2048 + 32 * ng].view(np.uint16)[o] == s[k // group, n]
        assert z is None or b[2048 + 32 * ng + o] == z[k // group, n]


@pytest.mark.parametrize("N,K", [(16, 128), (320, 7168), (4096, 2048), (40960, 4096), (1000, 16384)])
def test_linear_workspace_serves_fewer_rows(lib, N, K):
    """A workspace made for T rows is enough for any fewer."""
    sizes = [lib.moe_linear_w4_workspace_bytes(t, N, K) for t in range(130)]
    assert all(b and b % 256 == 0 for b in sizes)
    assert all(b >= a for a, b in zip(sizes, sizes[1:]))
