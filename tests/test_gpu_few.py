"""The few-token operators on the GPU: 4-bit weights (quantise, pack, product), the router from
hidden states and the whole layer in one launch, against 64-bit forms (few_ref) within the
rounding counted there."""
import numpy as np
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
import few_ref as ref
from gpu_helpers import bits, need_gpu
from oracle.formats import bf16_bits_to_f32

pytestmark = pytest.mark.gpu


def gen(seed):
    need_gpu()
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def w4_random(g, mats, n, k, group, zeros):
    """Codes, scales (k**-0.5 over the codes' spread, a few negative and zero), zero points."""
    q = torch.randint(0, 256, (mats, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (torch.rand(mats, k // group, n, generator=g, device="cuda") + 0.25) / (4.6 * k ** 0.5)
    s[:, :, ::7] *= -1
    s[:, :, 5] = 0
    z = torch.randint(0, 16, (mats, k // group, n), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return q, s.to(torch.bfloat16), z


# ------------------------------------------------------------------------ weight preparation
@pytest.mark.parametrize("rows,cols,group,zeros", [(48, 256, 32, False), (33, 384, 64, True), (16, 128, 128, True),
                                                   (130, 640, 128, False)])
def test_quantize_w4_bit_exact(rows, cols, group, zeros):
    g = gen(rows)
    w = normal(g, 2, rows, cols, std=0.05)
    w[0, 1] = 0                 # an empty group: scale 1
    w[1, 2] = w[1, 2].abs()     # one-sided
    w[1, 3, 0] = 300.0
    q, s, z = moe.moe_quantize_weight_w4(w, group, zeros)
    for m in range(2):
        oq, os_, oz = ref.quantize_w4(bf16_bits_to_f32(bits(w[m])), group, zeros)
        assert np.array_equal(bits(s[m]), os_)
        assert (z is None) == (oz is None) and (z is None or np.array_equal(z[m].cpu().numpy(), oz))
        assert np.array_equal(q[m].cpu().numpy(), oq)


@pytest.mark.parametrize("mats,N,K,group,zeros", [(1, 1, 128, 32, True), (1, 50, 384, 64, False), (2, 64, 256, 128, True),
                                                  (3, 32, 640, 32, True)])
def test_pack_w4_layout(mats, N, K, group, zeros):
    g = gen(N)
    q, s, z = w4_random(g, mats, N, K, group, zeros) if N > 5 else (
        torch.randint(0, 256, (mats, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
        normal(g, mats, K // group, N), torch.randint(0, 16, (mats, K // group, N), generator=g, device="cuda", dtype=torch.uint8))
    p = moe.moe_pack_w4(q, s, z)
    for m in range(mats):
        want = ref.pack_w4(q[m].cpu().numpy(), bits(s[m]), None if z is None else z[m].cpu().numpy())
        assert np.array_equal(p.data[m].cpu().numpy(), want)


# ----------------------------------------------------------------------------------- linear
LINEAR = [(1, 512, 256, 32, False, False, False), (1, 32, 128, 128, False, False, True), (2, 1, 128, 64, True, True, True),
          (3, 50, 384, 32, True, True, False), (8, 272, 1408, 128, False, False, True),
          (9, 4096, 640, 64, True, False, False), (17, 1000, 2048, 128, True, True, True),
          (32, 2048, 896, 32, False, True, False), (33, 96, 512, 64, True, False, True),
          (100, 160, 256, 128, False, False, True), (5, 7168, 4096, 128, False, False, False),
          (2, 40960, 2048, 64, True, True, True), (24, 1600, 4096, 128, False, True, True),
          (32, 96, 7168, 32, True, False, False), (70, 64, 7040, 64, True, True, False), (8, 33, 32768, 128, False, False, True)]


@pytest.mark.parametrize("T,N,K,group,zeros,bias,f32", LINEAR)
def test_linear_w4(T, N, K, group, zeros, bias, f32):
    g = gen(T * N)
    if N > 5:
        q, s, z = w4_random(g, 1, N, K, group, zeros)
    else:
        q = torch.randint(0, 256, (1, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = normal(g, 1, K // group, N)
        z = torch.randint(0, 16, s.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    x = normal(g, T, K)
    b = torch.randn(N, generator=g, device="cuda") if bias else None
    p = moe.moe_pack_w4(q, s, z)
    ws = moe.moe_linear_w4_workspace(T, N, K)
    dt = torch.float32 if f32 else torch.bfloat16
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = moe.moe_linear_w4(x, p, bias=b, out_dtype=dt, ws=ws, dev_status=status)
    assert status.item() == 0
    want, err = ref.linear(x, ref.w4_values(q[0], s[0], None if z is None else z[0]), b)
    assert y.dtype == dt and ref.close(y, want, err) <= 1
    again = moe.moe_linear_w4(x, p, bias=b, out_dtype=dt, ws=ws)
    assert torch.equal(again, y)
    assert not ws[:4 * -(-N // 32) * -(-T // 32)].any()          # the counters are zero again


def test_linear_w4_strides_and_out():
    """Rows of x and out inside wider buffers; what lies between the rows stays."""
    g = gen(5)
    T, N, K = 6, 96, 384
    q, s, z = w4_random(g, 1, N, K, 64, True)
    p = moe.moe_pack_w4(q, s, z)
    wide = normal(g, T, K + 72)
    out = torch.full((T, N + 10), 7.0, device="cuda", dtype=torch.bfloat16)
    moe.moe_linear_w4(wide[:, 8:8 + K], p, out=out[:, :N])
    assert torch.equal(out[:, :N], moe.moe_linear_w4(wide[:, 8:8 + K].contiguous(), p))
    assert (out[:, N:] == 7).all()


def test_linear_w4_workspace_for_fewer_rows():
    """One workspace, row counts up and down: what one call leaves is not where another counts."""
    g = gen(41)
    N, K = 320, 7168           # K shared between CTAs at every T
    q, s, _ = w4_random(g, 1, N, K, 32, False)
    p = moe.moe_pack_w4(q, s)
    ws = moe.moe_linear_w4_workspace(100, N, K)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for T in (100, 24, 100, 8, 33, 1, 64, 31, 100):
        x = normal(g, T, K)
        out = moe.moe_linear_w4(x, p, out_dtype=torch.float32, ws=ws, dev_status=status)
        assert torch.equal(out, moe.moe_linear_w4(x, p, out_dtype=torch.float32)) and status.item() == 0


def test_linear_w4_rows_are_apart():
    """A row of x with NaN or infinity leaves the other rows as they are."""
    g = gen(6)
    q, s, z = w4_random(g, 1, 64, 256, 32, True)
    p = moe.moe_pack_w4(q, s, z)
    x = normal(g, 12, 256)
    y = moe.moe_linear_w4(x, p)
    x[3, 7] = float("nan")
    x[9, 0] = float("inf")
    z2 = moe.moe_linear_w4(x, p)
    keep = [i for i in range(12) if i not in (3, 9)]
    assert torch.equal(z2[keep], y[keep]) and z2[3].isnan().all() and not z2[9].isfinite().any()


# ------------------------------------------------------------------------------------ route
@pytest.mark.parametrize("T,H,E,K,bias", [(1, 2048, 64, 8, False), (1, 128, 1, 1, True), (2, 256, 60, 3, True),
                                          (5, 7168, 256, 8, False), (32, 640, 1000, 32, True), (31, 1024, 8, 8, False)])
def test_route_hidden(T, H, E, K, bias):
    g = gen(T + H)
    x, w = normal(g, T, H), normal(g, E, H, std=H ** -0.5)
    b = torch.randn(E, generator=g, device="cuda") * 0.1 if bias else None
    ws = moe.moe_route_hidden_workspace()
    idx, wt, logits = moe.moe_route_hidden(x, w, K, bias=b, ws=ws)
    oi, ow, oz = ref.route(x, w, b, K)
    # one float32 rounding; the 8-term partial sums add at most a few steps of their own size
    size = (x.double().abs() @ w.double().abs().T) / 8
    assert ((logits.double() - oz).abs() <= 2.0 ** -24 * oz.abs() + 2.0 ** -24 * size).all()
    i2, w2 = moe.moe_route_topk(logits, K)
    assert torch.equal(idx, i2) and torch.equal(wt, w2)          # the selection is moe_route_topk's
    assert torch.equal(idx, oi)
    assert ((wt.double() - ow).abs() <= 2.0 ** -20 * ow).all()
    assert not ws.any()


def test_route_hidden_ties_and_padding():
    """Equal experts: the lower id; rows past num_tokens: -1 and 0."""
    g = gen(3)
    T, H, E, K = 7, 256, 40, 6
    x, w = normal(g, T, H), normal(g, E, H)
    w[20:] = w[:20]
    n = torch.tensor([4], dtype=torch.int32, device="cuda")
    idx, wt, _ = moe.moe_route_hidden(x, w, K, num_tokens=n)
    assert (idx[4:] == -1).all() and (wt[4:] == 0).all()
    assert torch.equal(idx[:4, 1::2], idx[:4, 0::2] + 20)
    assert torch.equal(idx[:4], ref.route(x, w, None, K)[0][:4])


# ------------------------------------------------------------------------------------ layer
class Weights:
    """One layer's weights in a format, for the library and as float64 matrices."""

    def __init__(self, g, dtype, H, I, E, shared, group=0, zeros=False, tiled=False):
        self.kw = dict(dtype={"bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3, "w4": moe.MOE_W4}[dtype])
        self.val = {}
        self.half = dtype != "bf16"
        for name, mats, n, k in (("w13", E, 2 * I, H), ("w2", E, H, I)) + (
                (("shared_w13", 1, 2 * I, H), ("shared_w2", 1, H, I)) if shared else ()):
            one = name.startswith("shared")
            if dtype == "bf16":
                w = normal(g, mats, n, k, std=k ** -0.5)
                self.val[name] = lambda e, w=w: w[e].double()
            elif dtype == "e4m3":
                # every finite code, subnormals among them
                w = torch.randint(0, 256, (mats, n, k), generator=g, device="cuda", dtype=torch.uint8)
                w[w % 128 == 127] = 3
                s = (torch.rand(mats, n // 128, k // 128, generator=g, device="cuda") + 0.5) / (100 * k ** 0.5)
                self.val[name] = lambda e, w=w, s=s: ref.e4m3_values(w[e], s[e])
                self.kw[name + "_scales"] = s[0] if one else s
            else:
                q, s, z = w4_random(g, mats, n, k, group, zeros)
                self.val[name] = lambda e, q=q, s=s, z=z: ref.w4_values(q[e], s[e], None if z is None else z[e])
                w = moe.moe_pack_w4(q, s, z)
            if dtype != "w4":
                w = w[0] if one else w
                if tiled:
                    w = moe.moe_pack_weights(w)
            self.kw[name] = w
        if tiled:
            self.kw["weight_tiles"] = True

    def want(self, x, idx, wt):
        v = self.val
        sh = (v["shared_w13"](0), v["shared_w2"](0)) if "shared_w13" in v else None
        return ref.layer(x, idx, wt, v["w13"], v["w2"], sh, self.half)


def random_routing(g, T, K, E, pad):
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32)
    idx[torch.rand(T, K, generator=g, device="cuda") < pad] = -1
    return idx.contiguous(), torch.rand(T, K, generator=g, device="cuda")


LAYER = [
    # T, H, I, E, K, dtype, shared, pad, group, zeros, tiled
    (1, 128, 128, 1, 1, "bf16", False, 0.0, 0, False, False),
    (1, 256, 512, 8, 2, "bf16", False, 0.0, 0, False, False),
    (1, 256, 512, 8, 2, "bf16", True, 0.0, 0, False, True),
    (5, 384, 640, 12, 4, "bf16", True, 0.2, 0, False, False),
    (32, 256, 384, 4, 4, "bf16", True, 0.1, 0, False, False),     # 32 rows per expert: two passes each
    (32, 512, 256, 1, 1, "bf16", False, 0.0, 0, False, True),
    (7, 2048, 1408, 16, 8, "bf16", False, 0.1, 0, False, True),
    (1, 128, 256, 3, 2, "e4m3", True, 0.0, 0, False, False),
    (3, 1024, 384, 16, 8, "e4m3", True, 0.0, 0, False, True),
    (13, 640, 256, 6, 3, "e4m3", False, 0.3, 0, False, False),
    (32, 384, 512, 40, 8, "e4m3", True, 0.0, 0, False, True),
    (1, 256, 128, 5, 2, "w4", False, 0.0, 32, False, False),
    (2, 384, 1408, 7, 3, "w4", True, 0.0, 64, True, False),
    (6, 1152, 384, 9, 4, "w4", True, 0.2, 128, True, False),
    (20, 512, 640, 3, 2, "w4", True, 0.1, 32, True, False),
    (32, 256, 256, 64, 8, "w4", False, 0.0, 128, False, False),
    # many units per SM: the sequence of units goes round its ring many times
    (1, 7168, 2048, 4, 3, "e4m3", True, 0.0, 0, False, False),
    (3, 4096, 2048, 8, 4, "w4", True, 0.0, 32, True, False),
    (2, 2048, 4096, 6, 3, "bf16", False, 0.0, 0, False, True),
]


@pytest.mark.parametrize("T,H,I,E,K,dtype,shared,pad,group,zeros,tiled", LAYER)
def test_layer_few(T, H, I, E, K, dtype, shared, pad, group, zeros, tiled):
    g = gen(T * H + E)
    w = Weights(g, dtype, H, I, E, shared, group, zeros, tiled)
    x = normal(g, T, H)
    idx, wt = random_routing(g, T, K, E, pad)
    layer = moe.MoeLayerFew(T, H, I, E, K, **w.kw)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, _, _ = layer.forward(x, topk_idx=idx, topk_w=wt, dev_status=status)
    want, err = w.want(x, idx, wt)
    assert status.item() == 0
    assert ref.close(out, want, err) <= 1
    again, _, _ = layer.forward(x, topk_idx=idx, topk_w=wt)
    assert torch.equal(again, out)


@pytest.mark.parametrize("dtype,group", [("bf16", 0), ("e4m3", 0), ("w4", 64)])
@pytest.mark.parametrize("T", [1, 4, 11])
def test_layer_few_routes(dtype, group, T):
    """The router inside, or logits given: moe_route_hidden's choice, the same output bits as
    with that choice as input."""
    g = gen(T + group)
    H, I, E, K = 512, 256, 24, 4
    w = Weights(g, dtype, H, I, E, True, group)
    x, wr = normal(g, T, H), normal(g, E, H, std=H ** -0.5)
    b = torch.randn(E, generator=g, device="cuda") * 0.1
    idx, wt, logits = moe.moe_route_hidden(x, wr, K, bias=b)
    given = moe.MoeLayerFew(T, H, I, E, K, **w.kw)
    out, _, _ = given.forward(x, topk_idx=idx, topk_w=wt)
    o2, i2, w2 = given.forward(x, logits=logits)
    o3, i3, w3 = moe.MoeLayerFew(T, H, I, E, K, w_router=wr, router_bias=b, **w.kw).forward(x)
    for i, v, o in ((i2, w2, o2), (i3, w3, o3)):
        assert torch.equal(i, idx) and torch.equal(v, wt) and torch.equal(o, out)
    want, err = w.want(x, idx, wt)
    assert ref.close(out, want, err) <= 1


def test_layer_few_fewer_tokens_and_num_tokens():
    """One layer object serves smaller batches; rows past num_tokens are padding: +0."""
    g = gen(9)
    H, I, E, K = 256, 384, 10, 3
    w = Weights(g, "bf16", H, I, E, True)
    wr = normal(g, E, H, std=H ** -0.5)
    layer = moe.MoeLayerFew(16, H, I, E, K, w_router=wr, **w.kw)
    x = normal(g, 16, H)
    full, fi, fw = layer.forward(x)
    for t in (1, 3, 9):
        n = torch.tensor([t], dtype=torch.int32, device="cuda")
        out, idx, wt = layer.forward(x, num_tokens=n)
        assert torch.equal(idx[:t], fi[:t]) and (idx[t:] == -1).all() and (wt[t:] == 0).all()
        want, err = w.want(x, idx, wt)
        assert ref.close(out, want, err) <= 1
        assert (bits(out[t:]) == 0).all()
        small, si, _ = layer.forward(x[:t])
        assert torch.equal(si, fi[:t])
        want, err = w.want(x[:t], si, fw[:t])
        assert ref.close(small, want, err) <= 1


def test_layer_few_padding_rows_and_bad_ids():
    g = gen(10)
    T, H, I, E, K = 6, 256, 128, 5, 3
    w = Weights(g, "bf16", H, I, E, True)
    x = normal(g, T, H)
    x[2] = float("nan")              # a token without slots is not read
    idx, wt = random_routing(g, T, K, E, 0.0)
    idx[2] = -1
    idx[4, 1] = -1
    wt[4, 1] = float("nan")          # nor is a padding slot's weight
    layer = moe.MoeLayerFew(T, H, I, E, K, **w.kw)
    out, _, _ = layer.forward(x, topk_idx=idx, topk_w=wt)
    assert (bits(out[2]) == 0).all()
    keep = [0, 1, 3, 4, 5]
    clean = torch.where(idx >= 0, wt, 0.0)
    want, err = w.want(x[keep], idx[keep], clean[keep])
    assert ref.close(out[keep], want, err) <= 1
    # ids outside [-1, E): padding, and a status bit
    bad = idx.clone()
    bad[4, 1] = E
    bad[2, 0] = -7
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o2, _, _ = layer.forward(x, topk_idx=bad, topk_w=wt, dev_status=status)
    assert status.item() == moe.MOE_DEV_BAD_EXPERT and torch.equal(bits_t(o2), bits_t(out))
    # nothing valid at all
    none = torch.full_like(idx, -1)
    o3 = torch.full_like(out, 5.0)
    layer.forward(x, out=o3, topk_idx=none, topk_w=wt)
    assert (bits(o3) == 0).all()
    # and the workspace serves the next call
    o4, _, _ = layer.forward(x, topk_idx=idx, topk_w=wt)
    assert torch.equal(bits_t(o4), bits_t(out))


def bits_t(t):
    return t.view(torch.int16)


def test_layer_few_repeated_ids():
    """The same expert in several slots of a token counts once per slot (more than 32 rows)."""
    g = gen(11)
    T, H, I, E, K = 15, 128, 128, 4, 4
    w = Weights(g, "bf16", H, I, E, False)
    x = normal(g, T, H)
    idx = torch.full((T, K), 2, dtype=torch.int32, device="cuda")
    idx[::2, 1] = 0
    wt = torch.rand(T, K, generator=g, device="cuda")
    out, _, _ = moe.MoeLayerFew(T, H, I, E, K, **w.kw).forward(x, topk_idx=idx, topk_w=wt)
    want, err = w.want(x, idx, wt)
    assert ref.close(out, want, err) <= 1


def test_layer_few_infinite_intermediate():
    """h past BF16's range becomes infinite once, not NaN from its second term."""
    T, H, I, E, K = 1, 128, 128, 1, 1
    g = gen(12)
    w13 = torch.zeros(1, 2 * I, H, device="cuda", dtype=torch.bfloat16)
    w13[0, 0, 0] = w13[0, I, 0] = 2.0 ** 70
    w2 = torch.zeros(1, H, I, device="cuda", dtype=torch.bfloat16)
    w2[0, :, 0] = 1.0
    x = torch.ones(T, H, device="cuda", dtype=torch.bfloat16)
    idx = torch.zeros(T, K, dtype=torch.int32, device="cuda")
    wt = torch.ones(T, K, device="cuda")
    out, _, _ = moe.MoeLayerFew(T, H, I, E, K, w13=w13, w2=w2).forward(x, topk_idx=idx, topk_w=wt)
    assert torch.isposinf(out).all()


def test_few_streams_and_graph():
    """On a side stream, and captured into a graph that is replayed with new inputs."""
    g = gen(13)
    T, H, I, E, K = 4, 256, 256, 8, 2
    w = Weights(g, "e4m3", H, I, E, True)
    wr = normal(g, E, H, std=H ** -0.5)
    q, s, z = w4_random(g, 1, 128, H, 64, True)
    p = moe.moe_pack_w4(q, s, z)
    ws = moe.moe_linear_w4_workspace(T, 128, H)
    layer = moe.MoeLayerFew(T, H, I, E, K, w_router=wr, **w.kw)
    xs = [normal(g, T, H) for _ in range(3)]

    def step(x):
        o, i, v = layer.forward(x)
        return o, i, v, moe.moe_linear_w4(o, p, ws=ws)
    want = [[t.clone() for t in step(x)] for x in xs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step(xs[1])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(x)
    for i in (2, 0, 1):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i]))


def test_few_two_streams_at_once():
    """Two layers and two products on two streams, each with a workspace of its own: the bits of calls
    one after the other."""
    g = gen(23)
    T, H, I, E, K = 6, 512, 384, 16, 4
    streams = [torch.cuda.Stream() for _ in range(2)]
    sides = []
    for dtype, group in (("e4m3", 0), ("w4", 64)):
        w = Weights(g, dtype, H, I, E, True, group)
        q, sc, z = w4_random(g, 1, 416, H, 64, True)
        sides.append((moe.MoeLayerFew(T, H, I, E, K, w_router=normal(g, E, H, std=H ** -0.5), **w.kw),
                      moe.moe_pack_w4(q, sc, z), moe.moe_linear_w4_workspace(T, 416, H),
                      [normal(g, T, H) for _ in range(12)], torch.zeros(1, dtype=torch.int32, device="cuda")))

    def one(side, i):
        layer, p, ws, xs, status = side
        out, idx, w = layer.forward(xs[i], dev_status=status)
        return out, idx, w, moe.moe_linear_w4(out, p, ws=ws, dev_status=status)
    want = [[one(side, i) for i in range(12)] for side in sides]
    torch.cuda.synchronize()
    got = [[], []]
    for i in range(12):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                got[k].append(one(sides[k], i))
    torch.cuda.synchronize()
    for k in range(2):
        assert sides[k][4].item() == 0
        assert all(torch.equal(a, b) for x, y in zip(got[k], want[k]) for a, b in zip(x, y))


def test_layer_few_near_layer_forward():
    """The same layer through moe_layer_forward (BF16 h and rows): equal to its extra roundings."""
    g = gen(14)
    T, H, I, E, K = 16, 512, 384, 8, 2
    w = Weights(g, "bf16", H, I, E, True)
    x = normal(g, T, H)
    idx, wt = random_routing(g, T, K, E, 0.1)
    out, _, _ = moe.MoeLayerFew(T, H, I, E, K, **w.kw).forward(x, topk_idx=idx, topk_w=wt)
    kw = {k: v for k, v in w.kw.items() if k != "dtype"}
    old = torch.empty_like(out)
    moe.MoeLayer(T, H, I, E, K, moe.MOE_BF16, **kw).forward(x, old, idx, wt)
    # three more BF16 roundings (h, the rows): within 2e-2 of the largest output, as its own tests hold it
    assert (out.float() - old.float()).abs().max() <= 2e-2 * old.float().abs().max()


@pytest.mark.parametrize("dtype,H,I,E,K,T,group", [("bf16", 2048, 1408, 64, 8, 5, 0), ("e4m3", 2048, 1408, 64, 8, 5, 0),
                                                   ("w4", 2048, 1408, 64, 8, 5, 32), ("e4m3", 1024, 2048, 32, 4, 20, 0)])
def test_layer_few_behind_other_work(dtype, H, I, E, K, T, group):
    """Right behind kernels that wrote the weights some SMs run far behind others.  Tiles of phase 2
    have other numbers of parts than those of phase 1: the joins of a late one stay its own.  Every
    call has other inputs than the one before, and gives the bits of a quiet call, with no wait
    run out."""
    g = gen(31)
    w = Weights(g, dtype, H, I, E, False, group)
    layer, quiet = (moe.MoeLayerFew(T, H, I, E, K, **w.kw) for _ in range(2))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    big = [t for t in layer.tensors if t is not None]
    for i in range(16):
        x = normal(g, T, H)
        idx, wt = random_routing(g, T, K, E, 0.1)
        torch.cuda.synchronize()
        want, _, _ = quiet.forward(x, topk_idx=idx, topk_w=wt)
        torch.cuda.synchronize()
        for t in big if i % 2 else big[::-1]:
            t.view(torch.uint8).bitwise_or_(0)
        got, _, _ = layer.forward(x, topk_idx=idx, topk_w=wt, dev_status=status)
        assert torch.equal(got, want) and status.item() == 0


@pytest.mark.parametrize("weights", ["bf16", "e4m3", "w4"])
def test_decode_few_example(weights):
    """The operators together: 12 greedy steps, routed inside the layers and ahead of them."""
    need_gpu()
    from combine_moe_route_softmax_gb300 import decode_few
    ms, same = decode_few.run(tokens=5, layers=2, H=512, I=256, E=16, K=4, vocab=1024, weights=weights, group=64, steps=12)
    assert same and all(t > 0 for t in ms.values())


def test_decode_few_step_values():
    """One BF16 layer and the head against the 64-bit forms of each, fed each other's outputs."""
    need_gpu()
    from combine_moe_route_softmax_gb300 import decode_few
    step = decode_few.DecodeStep(3, 1, 512, 256, 16, 4, 640, "bf16", 32, shared=False)
    x = step.table[:3].contiguous()
    logits, ids = step(x)
    layer = step.inside[0]
    y, idx, w = layer.forward(x)
    assert torch.equal(idx, ids[0])
    val = lambda t: (lambda e: t[e].double())
    want, err = ref.layer(x, idx, w, val(layer.tensors[0]), val(layer.tensors[2]), None, False)
    assert ref.close(y, want, err) <= 1
    again = moe.moe_linear_w4(x + y, step.head, out_dtype=torch.float32)
    assert torch.equal(again, logits)
