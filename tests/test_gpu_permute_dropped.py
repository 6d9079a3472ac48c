"""The batched permute where an expert is named in several slots of a token and its block overflows: ranks in that expert's
block then grow faster than shared ranks, so that a token may have lost every slot and still have its shared row."""
import numpy as np
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import bits, host, need_gpu
from oracle import moe_ref as ref
from oracle.formats import bf16_bits_to_f32

pytestmark = pytest.mark.gpu
POISON = 0x77


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def repeated_ids(T, E, K, seed, pad=0.1):
    """Most tokens name the first expert in most of their slots; some slots and some tokens are padding."""
    rng = np.random.default_rng(seed)
    idx = rng.integers(0, E, (T, K))
    idx[rng.random((T, K)) < 0.7] = 0
    idx[rng.random((T, K)) < pad] = -1
    idx[rng.random(T) < pad] = -1
    return idx.astype(np.int32)


def permute(form, idx, E, max_tokens, H, seed):
    """The call of `form` into buffers full of POISON -> (its maps, xb bytes [rows, ..], xb_scales or None, what a routed
    and what a shared row of each token hold, and their scales)."""
    T, K = idx.shape
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    nseg, rows = E + 1, (E + 1) * max_tokens
    codes = form in ("e4m3", "codes")
    q, s = ref.act_quant_1x128(bf16_bits_to_f32(bits(x)))
    xb = torch.full((rows, H * (1 if codes else 2)), POISON, dtype=torch.uint8, device="cuda")
    xs = torch.full((rows, H // 128), -3.0, device="cuda") if codes else None
    maps = [torch.full((n,), -99, dtype=torch.int32, device="cuda") for n in (nseg, rows, T * K, T)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_permute_batched_workspace_bytes(T, K, E, True), dtype=torch.uint8, device="cuda")
    ids, p = torch.from_numpy(idx).cuda(), lambda t: None if t is None else t.data_ptr()
    stream = torch.cuda.current_stream().cuda_stream
    routed = shared = q if codes else bits(x).view(np.uint8)
    if form == "codes":
        xc, sc = torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()
        code = moe.lib().moe_permute_e4m3(p(ids), T, K, E, 1, max_tokens, p(xc), p(sc), H, p(xb), p(xs), None, p(maps[0]),
                                          p(maps[1]), p(maps[2]), p(maps[3]), p(ws), ws.numel(), p(status), None, None, stream)
    else:
        fmt = form if form in ("fq e4m3", "fq nvfp4") else None
        scale = torch.full((1,), 16.0, device="cuda") if fmt else None
        if fmt:
            routed = ref.dispatch_qdq_bits(bits(x), np.float32(16.0), fmt.split()[1]).view(np.uint8)
        code = moe.lib().moe_permute_batched(p(ids), T, K, E, 1, max_tokens, p(x), H, moe.MOE_E4M3 if codes else moe.MOE_BF16,
                                             p(xb), p(xs), p(maps[0]), p(maps[1]), p(maps[2]), p(maps[3]), p(ws), ws.numel(),
                                             p(status), p(scale), int(fmt == "fq nvfp4"), None, None, stream)
    torch.cuda.synchronize()
    assert code == 0 and status.item() == moe.MOE_DEV_OVERFLOW
    return maps, host(xb), None if xs is None else host(xs), routed, shared, s


FORMS = ["bf16", "e4m3", "fq e4m3", "fq nvfp4", "codes"]


@pytest.mark.parametrize("form,T,E,K,H,max_tokens",
                         [(f, 4, 2, 2, 256, 4) for f in FORMS] +             # the first two tokens fill the expert's block
                         [(f, 300, 8, 4, 384, 200) for f in FORMS] +
                         [(f, 8193, 8, 4, 128, 5000) for f in FORMS] +       # more than 32768 slots: codes in four launches
                         [(f, 1200, 2, 32, 128, 900) for f in FORMS] +       # no lane left for the shared row
                         [("codes", 8192, 8, 4, 128, 5000), ("codes", 4800, 8, 4, 128, 3000),
                          ("bf16", 40, 4, 3, 58240, 25)])                    # BF16 rows too long to stand in shared memory
def test_shared_rows_of_tokens_that_lost_every_slot(form, T, E, K, H, max_tokens):
    idx = np.zeros((T, K), dtype=np.int32) if T == 4 else repeated_ids(T, E, K, seed=T + K)
    m, src, inv, smap, st = ref.permute_batched(idx, E, max_tokens, with_shared=True)
    lost = (inv < 0).all(1) & (smap >= 0)
    assert st == ref.STATUS_OVERFLOW and lost.any(), "the case that this test is for"
    maps, xb, xs, routed, shared, scales = permute(form, idx, E, max_tokens, H, seed=T)
    for got, want in zip(maps, (m, src, inv.ravel(), smap)):
        assert np.array_equal(host(got), want)
    live = np.nonzero(src >= 0)[0]
    tok = ref.row_tokens(src[live], T, K)
    want = np.where((src[live] < T * K)[:, None], routed[tok], shared[tok])
    assert np.array_equal(xb[live], want)
    assert (xb[src < 0] == POISON).all()
    if xs is not None:
        assert np.array_equal(xs[live], scales[tok]) and (xs[src < 0] == -3.0).all()


@pytest.mark.parametrize("kw", [{}, dict(fuse_combine=True), dict(dtype="e4m3"), dict(dtype="e4m3", rows="codes"),
                                dict(dtype="e4m3", fuse_combine=True)])
def test_layer_with_a_callers_repeated_ids(kw):
    """The layer on ids of the caller's own, its workspace full of NaN: what the ragged layout gives where the dropped slots
    have weight 0 (each adds +-0 to a sum that starts at +0), and +0 for a token that lost every slot: the combine adds the
    shared row to tokens that have a slot with a row, as the oracle's does."""
    kw = dict(kw)
    fp8, codes = kw.pop("dtype", "bf16") == "e4m3", kw.pop("rows", "") == "codes"
    T, H, I, E, K, mt = 60, 512, 256, 6, 3, 60
    g = torch.Generator(device="cuda").manual_seed(5)
    mats = [(torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).to(torch.bfloat16)
            for s in ((E, 2 * I, H), (E, H, I), (2 * I, H), (H, I))]
    names = ("w13", "w2", "shared_w13", "shared_w2")
    w = dict(zip(names, mats))
    if fp8:
        for n, t in zip(names, mats):
            w[n], w[n + "_scales"] = moe.moe_quantize_weight_fp8(t)
    dtype = moe.MOE_E4M3 if fp8 else moe.MOE_BF16
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    x, xs = moe.moe_quantize_act_fp8(x) if codes else (x, None)
    idx = repeated_ids(T, E, K, seed=9)
    m, src, inv, smap, st = ref.permute_batched(idx, E, mt, with_shared=True)
    lost = (inv < 0).all(1)
    assert (lost & (smap >= 0)).any() and (smap >= 0).sum() == (idx >= 0).any(1).sum()
    ids, wt = torch.from_numpy(idx).cuda(), torch.rand(T, K, generator=g, device="cuda")
    outs = []
    for max_tokens, weights in ((mt, wt), (0, wt * torch.from_numpy(inv >= 0).cuda())):
        layer = moe.MoeLayer(T, H, I, E, K, dtype, max_tokens=max_tokens, **(kw if max_tokens else {}), **w)
        layer.ws.fill_(255)
        out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        layer.forward(x, out, ids, weights, x_scales=xs)
        outs.append(out)
    outs[1][torch.from_numpy(lost).cuda()] = 0
    assert not outs[0].isnan().any() and np.array_equal(*map(bits, outs))
