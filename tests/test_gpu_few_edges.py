"""The few-token operators on the GPU at values and calls where they can go wrong: infinities, masked
experts, NaN, zero points of a whole byte, streams, waits that run out."""
import numpy as np
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
import few_ref as ref
from gpu_helpers import bits
from test_gpu_few import Weights, gen, normal, random_routing, w4_random

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- infinite intermediate values
def infinite_h_layer(dtype):
    """An E4M3 or 4-bit layer whose h is infinite in row 0 for tokens with x[0] = 1 and 1 in row 16 for those
    with x[128] = 1 (silu(40) * 0.025 to within BF16); the other rows of h are 0."""
    H, I = 256, 128
    up, down = 40.0, 0.025
    if dtype == "e4m3":
        code = lambda v: torch.tensor(v, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
        w13 = torch.zeros(1, 2 * I, H, dtype=torch.uint8, device="cuda")
        w13[0, 0, 0] = w13[0, I, 0] = w13[0, 16, 128] = w13[0, I + 16, 128] = code(1.0)
        s13 = torch.tensor([[[2.0 ** 70, up], [2.0 ** 70, down]]], device="cuda")
        w2 = torch.zeros(1, H, I, dtype=torch.uint8, device="cuda")
        w2[0, :, 0] = w2[0, :, 16] = code(1.0)
        kw = dict(w13=w13, w13_scales=s13, w2=w2, w2_scales=torch.ones(1, 2, 1, device="cuda"))
        return moe.MoeLayerFew(4, H, I, 1, 1, moe.MOE_E4M3, **kw), H
    def packed(n, k, entries):
        q = torch.full((1, n, k // 2), 0x88, dtype=torch.uint8, device="cuda")
        s = torch.ones(1, k // 128, n, dtype=torch.bfloat16, device="cuda")
        for r, c, v in entries:
            q[0, r, c // 2] = 0x89                  # 1 in the even column
            s[0, c // 128, r] = v
        return moe.moe_pack_w4(q, s)
    w13 = packed(2 * I, H, [(0, 0, 2.0 ** 70), (I, 0, 2.0 ** 70), (16, 128, up), (I + 16, 128, down)])
    w2 = packed(H, I, [(r, c, 1.0) for r in range(H) for c in (0, 16)])
    return moe.MoeLayerFew(4, H, I, 1, 1, moe.MOE_W4, w13=w13, w2=w2), H


@pytest.mark.parametrize("dtype", ["e4m3", "w4"])
def test_layer_few_infinite_beside_finite(dtype):
    """h infinite in a block of small values, beside a block of larger ones: infinity, not NaN; tokens without
    it have their values."""
    gen(0)
    layer, H = infinite_h_layer(dtype)
    x = torch.zeros(4, H, dtype=torch.bfloat16, device="cuda")
    x[0, 0] = x[1, 128] = 1.0
    x[2, 0] = x[2, 128] = 1.0
    idx = torch.zeros(4, 1, dtype=torch.int32, device="cuda")
    out, _, _ = layer.forward(x, topk_idx=idx, topk_w=torch.ones(4, 1, device="cuda"))
    assert torch.isposinf(out[0]).all() and torch.isposinf(out[2]).all()
    assert ((out[1].float() - 1).abs() <= 2.0 ** -6).all() and (out[3] == 0).all()



# ------------------------------------------------------------------------ zero points of a whole byte
@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_zero_points_above_15(group):
    """A zero point is any byte (formats that store z - 1 have 16): kept by the packing, used by the product
    and the layer."""
    g = gen(group)
    N, K = 96, 384
    q, s, _ = w4_random(g, 1, N, K, group, False)
    z = torch.randint(0, 256, s.shape, generator=g, device="cuda", dtype=torch.uint8)
    z[:, :, ::3] = 16
    p = moe.moe_pack_w4(q, s, z)
    assert np.array_equal(p.data[0].cpu().numpy(), ref.pack_w4(q[0].cpu().numpy(), bits(s[0]), z[0].cpu().numpy()))
    for T in (1, 5, 20):
        x = normal(g, T, K)
        y = moe.moe_linear_w4(x, p, out_dtype=torch.float32)
        want, err = ref.linear(x, ref.w4_values(q[0], s[0], z[0]))
        assert ref.close(y, want, err) <= 1
    H, I, E = 256, 128, 3
    val, kw = {}, {}
    for name, n, k in (("w13", 2 * I, H), ("w2", H, I)):
        q, s, _ = w4_random(g, E, n, k, group, False)
        z = torch.randint(0, 40, s.shape, generator=g, device="cuda", dtype=torch.uint8)
        kw[name] = moe.moe_pack_w4(q, s, z)
        val[name] = lambda e, q=q, s=s, z=z: ref.w4_values(q[e], s[e], z[e])
    x = normal(g, 6, H)
    idx, wt = random_routing(g, 6, 2, E, 0.0)
    out, _, _ = moe.MoeLayerFew(6, H, I, E, 2, moe.MOE_W4, **kw).forward(x, topk_idx=idx, topk_w=wt)
    want, err = ref.layer(x, idx, wt, val["w13"], val["w2"], None, True)
    assert ref.close(out, want, err) <= 1


# ----------------------------------------------------------------------------- masked experts, NaN
@pytest.mark.parametrize("T,H,E,K", [(1, 256, 12, 4), (4, 2048, 64, 8), (5, 640, 40, 3), (32, 1024, 300, 8)])
def test_route_hidden_masked_experts(T, H, E, K):
    """A bias of -infinity takes an expert out, one of +infinity puts it first; the logits are what a plain sum
    gives, and the other experts' bits do not change."""
    g = gen(T + E)
    x, w = normal(g, T, H), normal(g, E, H, std=H ** -0.5)
    b = torch.randn(E, generator=g, device="cuda") * 0.1
    _, _, plain = moe.moe_route_hidden(x, w, K, bias=b)
    masked = torch.arange(E, device="cuda") % 3 == 1
    b2 = torch.where(masked, float("-inf"), b)
    idx, wt, logits = moe.moe_route_hidden(x, w, K, bias=b2)
    assert torch.equal(logits, torch.where(masked, float("-inf"), plain))
    oi, ow, _ = ref.route(x, w, b2, K)
    assert torch.equal(idx, oi) and not masked[idx.long()].any()
    assert ((wt.double() - ow).abs() <= 2.0 ** -20 * ow).all()
    b3 = b.clone()
    b3[E - 1] = float("inf")
    idx, _, logits = moe.moe_route_hidden(x, w, K, bias=b3)
    assert torch.isposinf(logits[:, E - 1]).all() and (idx[:, 0] == E - 1).all()
    assert torch.equal(logits[:, :E - 1], plain[:, :E - 1])


@pytest.mark.parametrize("T", [1, 3, 9])
def test_route_hidden_infinite_and_nan_inputs(T):
    """An infinite or NaN element of x: what a plain sum of the products gives, in that token alone."""
    g = gen(T)
    H, E, K = 512, 24, 4
    x, w = normal(g, T, H), normal(g, E, H, std=H ** -0.5)
    w[w == 0] = 0.01
    _, _, plain = moe.moe_route_hidden(x, w, K)
    for v in (float("inf"), float("-inf"), float("nan")):
        y = x.clone()
        y[T - 1, 77] = v
        _, _, logits = moe.moe_route_hidden(y, w, K)
        want = y.double() @ w.double().T
        assert torch.equal(logits[:T - 1], plain[:T - 1])
        assert torch.equal(logits[T - 1].isnan(), want[T - 1].isnan())
        if v == v:
            assert torch.equal(logits[T - 1], want[T - 1].float())


def test_layer_few_masked_experts():
    """The same mask inside the layer: the masked experts' weights are not read."""
    g = gen(21)
    T, H, I, E, K = 6, 256, 128, 9, 3
    w = Weights(g, "bf16", H, I, E, True)
    wr = normal(g, E, H, std=H ** -0.5)
    b = torch.zeros(E, device="cuda")
    b[::2] = float("-inf")
    w.kw["w13"][::2] = float("nan")
    x = normal(g, T, H)
    out, idx, wt = moe.MoeLayerFew(T, H, I, E, K, w_router=wr, router_bias=b, **w.kw).forward(x)
    oi, ow, _ = ref.route(x, wr, b, K)
    assert torch.equal(idx, oi) and ((wt.double() - ow).abs() <= 2.0 ** -20 * ow).all()
    want, err = w.want(x, idx, wt)
    assert ref.close(out, want, err) <= 1


@pytest.mark.parametrize("E,K", [(6, 6), (40, 5), (300, 32)])
def test_layer_few_selects_as_route_topk_does(E, K):
    """Given logits with infinities, zeros of both signs and every kind of NaN, the layer's choice is
    moe_route_topk's: ids, and weights bit for bit (NaN or not)."""
    g = gen(E)
    T, H, I = 8, 128, 128
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[1, ::2] = float("-inf")
    logits[2] = float("-inf")
    logits[3, 1::2] = 0.0
    logits[3, ::2] = -0.0
    nan = torch.tensor([0x7fc00000, 0x7f800001, -1, -2, -0x400000], dtype=torch.int32, device="cuda").view(torch.float32)
    logits[4, :5] = nan
    logits[5] = nan[2]                     # all bits set: the lowest place in the order
    logits[6, ::3] = nan[2]
    logits[6, 1::3] = nan[3]
    logits[7, ::2] = nan[4]
    w13 = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device="cuda")
    w2 = torch.zeros(E, H, I, dtype=torch.bfloat16, device="cuda")
    _, idx, wt = moe.MoeLayerFew(T, H, I, E, K, w13=w13, w2=w2).forward(normal(g, T, H), logits=logits)
    oi, ow = moe.moe_route_topk(logits, K)
    assert torch.equal(idx, oi)
    assert torch.equal(wt.isnan(), ow.isnan()) and torch.equal(wt[~wt.isnan()], ow[~ow.isnan()])


# ------------------------------------------------------------------------------------------- streams
@pytest.mark.parametrize("raw", [False, True], ids=["object", "handle"])
def test_few_calls_on_another_stream_than_the_current(raw):
    """stream=s while the current stream is busy: nothing of the call waits for it, and the workspace that the call
    makes is zero when its kernel starts."""
    g = gen(17)
    T, H, E, K, N, KL = 20, 1024, 64, 8, 160, 7168       # the product's K is shared between CTAs
    x, w = normal(g, T, H), normal(g, E, H, std=H ** -0.5)
    q, s, z = w4_random(g, 1, N, KL, 32, True)
    p, xl = moe.moe_pack_w4(q, s, z), normal(g, T, KL)
    lw = Weights(g, "e4m3", 256, 128, 6, True)
    layer = moe.MoeLayerFew(T, 256, 128, 6, 2, w_router=normal(g, 6, 256), **lw.kw)
    xs = normal(g, T, 256)

    def calls(**k):
        return (*moe.moe_route_hidden(x, w, K, **k), moe.moe_linear_w4(xl, p, **k), *layer.forward(xs, **k),
                *[t for t in moe.moe_quantize_weight_w4(w, 32, True, **k)])
    want = calls()
    side = torch.cuda.Stream()
    for stream in (side, torch.cuda.current_stream()):
        with torch.cuda.stream(stream):                    # memory that a workspace is likely to get
            junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (256, 4096, 1 << 20, 1 << 22) * 3]
            del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    got = calls(stream=side.cuda_stream if raw else side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------------------- logits by row
@pytest.mark.parametrize("H,E,K", [(7168, 256, 8), (640, 60, 4), (2048, 1000, 32)])
def test_route_hidden_rows_by_themselves(H, E, K):
    """A token's logits are the same bits in any call of up to 4 tokens, and in any of more, at any place; the two
    differ by the errors that moe.h states; both keep near ties that are further apart than that in order."""
    g = gen(H)
    x, w = normal(g, 32, H), normal(g, E, H, std=H ** -0.5)
    w[1::2] = w[::2][:E // 2]
    w[1::2, 5] += 2.0 ** -9 * w[1::2, 5].abs() + 2.0 ** -12      # near ties: one weight a little larger
    z = x.double() @ w.double().T
    size = x.double().abs() @ w.double().abs().T
    few = torch.cat([moe.moe_route_hidden(x[i:i + n], w, K)[2] for i, n in ((0, 1), (1, 2), (3, 3), (6, 4), (10, 1))])
    assert torch.equal(few, torch.cat([moe.moe_route_hidden(x[i:i + 1], w, K)[2] for i in range(11)]))
    idx, _, many = moe.moe_route_hidden(x, w, K)
    assert torch.equal(many[3:9], moe.moe_route_hidden(x[3:9].contiguous(), w, K)[2])
    assert torch.equal(many[11:], moe.moe_route_hidden(x[11:].contiguous(), w, K)[2])
    for logits, rows, eps in ((few, slice(0, 11), 2.0 ** -21), (many, slice(0, 32), 2.0 ** -19)):
        err = eps * size[rows] + 2.0 ** -24 * z[rows].abs()
        assert ((logits.double() - z[rows]).abs() <= err).all()
        far = (z[rows, 1::2] - z[rows, ::2][:, :E // 2]).abs() > err[:, 1::2] + err[:, ::2][:, :E // 2]
        up = logits[:, 1::2] > logits[:, ::2][:, :E // 2]
        assert torch.equal(up[far], (z[rows, 1::2] > z[rows, ::2][:, :E // 2])[far])
    # the layers' own router: 12 warps with 4-bit weights, 16 with the others
    for dtype, group in (("w4", 128), ("e4m3", 0), ("bf16", 0)):
        lw = Weights(g, dtype, H, 128, K, False, group)
        n = moe.MoeLayerFew(32, H, 128, K, K, w_router=w[:K].contiguous(), **lw.kw)
        _, i2, w2 = n.forward(x)
        i1, w1, _ = moe.moe_route_hidden(x, w[:K].contiguous(), K)
        assert torch.equal(i1, i2) and torch.equal(w1, w2)
