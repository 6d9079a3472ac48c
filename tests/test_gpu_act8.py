"""The 8-bit activation path on the GPU: the norm, the product of E4M3 operands and the dispatch of E4M3 rows against
64-bit forms, their options, and a block that uses them together."""
import pytest
import torch

import act8_ref as ref
import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
EPS = 1e-6


@pytest.fixture(autouse=True)
def gpu():
    need_gpu()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def codes(g, rows, cols):
    return (randn(g, rows, cols) * 130).clamp(-448, 448).to(torch.float8_e4m3fn).view(U8)


def scales(g, rows, cols, unit):
    return (torch.rand(rows, cols, generator=g, device="cuda") + 0.5) * unit


# -------------------------------------------------------------------------------------------- norm
def check_norm(got, x, weight, eps, residual, n):
    """got: (out, q, q_scales, residual_out) of the first n rows against the 64-bit form."""
    out, q, s, r = got
    y, h = ref.norm(x[:n], weight, eps, None if residual is None else residual[:n])
    if out is not None:
        assert ((out[:n].double() - y).abs() <= (ref.half_step(BF) + 2 * ref.NORM_ERR) * y.abs() + 1e-40).all()
    if q is not None:
        want = ref.block_scales(y)
        assert ((s[:n].double() - want).abs() <= (ref.NORM_ERR + 2 * ref.F32) * want).all()
        lo, hi = ref.code_bounds(y, 2 * ref.NORM_ERR + 4 * ref.F32)
        v = ref.e4m3_values(q[:n])
        assert ((v.abs() >= lo) & (v.abs() <= hi)).all()
        assert ((v * y >= 0) | (v == 0)).all()
    if residual is not None:
        assert ((r[:n].double() - h).abs() <= (ref.half_step(r.dtype) * 1.01 + ref.F32) * h.abs()).all()


@pytest.mark.parametrize("T,H", [(1, 128), (1, 7168), (3, 8192), (153, 256), (200, 7168), (5, 8320), (2, 16384),
                                 (3, 65536), (1027, 2048), (400, 4352)])
@pytest.mark.parametrize("residual", [None, BF, F32])
@pytest.mark.parametrize("weight", [BF, F32])
def test_norm(T, H, residual, weight):
    g = gen(T + H)
    x = (randn(g, T, H) * (torch.rand(T, 1, generator=g, device="cuda") * 3 + 0.01)).to(BF)
    w = (randn(g, H) * 0.3 + 1).to(weight)
    r = None if residual is None else (randn(g, T, H) * 4).to(residual)
    check_norm(moe.moe_rmsnorm(x, w, EPS, residual=r, e4m3=True), x, w, EPS, r, T)


@pytest.mark.parametrize("T,H", [(1, 8), (7, 264), (300, 1000), (2, 40), (160, 8200)])
def test_norm_bf16_only_odd_widths(T, H):
    g = gen(H)
    x, w, r = randn(g, T, H).to(BF), randn(g, H), randn(g, T, H)
    got = moe.moe_rmsnorm(x, w, 1e-5, residual=r)
    assert got[1] is None and got[2] is None
    check_norm(got, x, w, 1e-5, r, T)


def test_norm_outputs_alone_are_the_same():
    g = gen(1)
    x, w, r = randn(g, 37, 640).to(BF), randn(g, 640).to(BF), randn(g, 37, 640).to(BF)
    both = moe.moe_rmsnorm(x, w, EPS, residual=r, e4m3=True)
    assert torch.equal(moe.moe_rmsnorm(x, w, EPS, residual=r)[0], both[0])
    only = moe.moe_rmsnorm(x, w, EPS, residual=r, bf16=False, e4m3=True)
    assert only[0] is None and all(torch.equal(a, b) for a, b in zip(only[1:], both[1:]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_in_place(dtype):
    """The residual is added to in place, and out may be x."""
    g = gen(2)
    x, w, r = randn(g, 301, 7168).to(BF), randn(g, 7168).to(BF), randn(g, 301, 7168).to(dtype)
    want = moe.moe_rmsnorm(x, w, EPS, residual=r, e4m3=True)
    x2, r2 = x.clone(), r.clone()
    q, s = torch.empty_like(want[1]), torch.empty_like(want[2])
    moe.moe_rmsnorm(x2, w, EPS, residual=r2, residual_out=r2, out=x2, q=q, q_scales=s)
    for a, b in zip((x2, q, s, r2), want):
        assert torch.equal(a, b)


def test_norm_strided_rows():
    g = gen(3)
    wide = randn(g, 50, 1024).to(BF)
    x, w = wide[:, 128:640], randn(g, 512)
    a, b = moe.moe_rmsnorm(x, w, EPS, e4m3=True), moe.moe_rmsnorm(x.contiguous(), w, EPS, e4m3=True)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


@pytest.mark.parametrize("n", [0, 1, 99, 200, 300, -5])
def test_norm_num_tokens_leaves_the_rest(n):
    """Rows past num_tokens are neither read (they hold NaN) nor written."""
    g = gen(4)
    T, H = 200, 384
    live = min(max(n, 0), T)
    x, w, r = randn(g, T, H).to(BF), randn(g, H).to(BF), randn(g, T, H)
    x[live:], r[live:] = torch.nan, torch.nan
    bufs = (torch.full((T, H), 7.0, dtype=BF, device="cuda"), torch.full((T, H), 99, dtype=U8, device="cuda"),
            torch.full((T, H // 128), 5.0, device="cuda"), torch.full((T, H), 3.0, device="cuda"))
    moe.moe_rmsnorm(x, w, EPS, residual=r, out=bufs[0], q=bufs[1], q_scales=bufs[2], residual_out=bufs[3],
                    num_tokens=torch.tensor([n], dtype=I32, device="cuda"))
    check_norm(bufs, x, w, EPS, r, live)
    for b, v in zip(bufs, (7.0, 99, 5.0, 3.0)):
        assert (b[live:] == v).all()


def test_norm_special_values():
    """A row of zeros (scale 1), values near the ends of the range, NaN and infinity kept to their own row."""
    g = gen(5)
    x = randn(g, 8, 256).to(BF)
    w = torch.ones(256, device="cuda")
    x[1] = 0
    x[2] *= 1e15
    x[3] *= 1e-18
    x[4, 7] = torch.nan
    x[5, 9] = torch.inf
    x[6, :128] = 0
    out, q, s, _ = moe.moe_rmsnorm(x, w, EPS, e4m3=True)
    rows = [0, 1, 2, 3, 6, 7]
    check_norm((out[rows], q[rows], s[rows], None), x[rows], w, EPS, None, len(rows))
    assert (out[1] == 0).all() and (q[1] == 0).all() and (s[1] == 1).all() and (s[6, 0] == 1).all()
    assert out[4].isnan().all()
    assert out[5, 9].isnan() and (out[5, :9] == 0).all()
    assert moe.moe_rmsnorm(x[1:2], w, 0.0)[0].isnan().all()      # 0 * (1 / 0), as the formula has it


def test_norm_no_rows():
    x = torch.empty(0, 256, dtype=BF, device="cuda")
    out, q, s, r = moe.moe_rmsnorm(x, torch.ones(256, device="cuda"), EPS, residual=x.float(), e4m3=True)
    assert out.shape == q.shape == r.shape == (0, 256) and s.shape == (0, 2)


# ------------------------------------------------------------------------------------------ linear
def check_linear(out, x, xs, w, ws, bias=None):
    y, err = ref.linear(x, xs, w, ws, bias)
    assert ((out.double() - y).abs() <= err + ref.half_step(out.dtype) * (y.abs() + err)).all()
    # on the average far closer: the roundings of a few hundred float32 additions do not line up, and the output's
    # own is at most 2^-8 / sqrt(3) in the mean
    n = y.norm()
    assert (out.double() - y).norm() <= (1e-5 if out.dtype is F32 else 1e-5 + 2.0 ** -8 / 3 ** 0.5) * n


def operands(T, N, K, seed=0, bias=False):
    g = gen(seed + 7 * T + 3 * N + K)
    return (codes(g, T, K), scales(g, T, K // 128, 1 / 130), codes(g, N, K),
            scales(g, -(-N // 128), K // 128, 1 / (130 * K ** 0.5)), randn(g, N) if bias else None)


SHAPES = [(1, 1, 128), (1, 512, 256), (1, 4096, 7168), (1, 130, 16384), (2, 576, 384), (7, 129, 1152), (8, 128, 2048),
          (9, 1000, 512), (13, 4096, 7168), (16, 7168, 2048), (17, 300, 640), (31, 256, 7168), (32, 4096, 896),
          (33, 640, 1024), (48, 2048, 2048), (63, 1030, 512), (64, 512, 7168), (65, 128, 128), (100, 7168, 2048),
          (127, 576, 7168), (128, 8200, 1024), (129, 256, 256), (255, 1536, 1536), (256, 4096, 7168), (257, 999, 384),
          (300, 576, 7168), (511, 127, 2048), (700, 576, 7168), (1000, 2048, 512), (2049, 4096, 1024), (4100, 700, 384)]


@pytest.mark.parametrize("T,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear(T, N, K, dtype):
    x, xs, w, ws, b = operands(T, N, K, bias=(T + N) % 2 == 1)
    check_linear(moe.moe_linear_e4m3(x, xs, w, ws, bias=b, out_dtype=dtype), x, xs, w, ws, b)


def test_linear_blocks_meet_their_own_scales():
    """Scales that differ by powers of two from block to block, and codes that are exact sums: the result is exact,
    so a scale of another block, row or column shows in full."""
    g = gen(11)
    for T, N, K in ((3, 300, 640), (40, 520, 1280), (300, 1100, 2048)):
        x = torch.randint(0, 2, (T, K), generator=g, device="cuda").to(torch.float8_e4m3fn).view(U8)
        w = torch.randint(0, 2, (N, K), generator=g, device="cuda").to(torch.float8_e4m3fn).view(U8)
        xs = torch.exp2(torch.randint(0, 5, (T, K // 128), generator=g, device="cuda").float())
        ws = torch.exp2(torch.randint(0, 5, (-(-N // 128), K // 128), generator=g, device="cuda").float())
        y, _ = ref.linear(x, xs, w, ws)
        assert torch.equal(moe.moe_linear_e4m3(x, xs, w, ws, out_dtype=F32).double(), y)


@pytest.mark.parametrize("T", [1, 20, 200])
def test_linear_strided_out_and_neighbours(T):
    """Rows of out may be strided, and nothing beside them is touched."""
    N, K = 333, 512
    x, xs, w, ws, b = operands(T, N, K, bias=True)
    for dtype in (BF, F32):
        buf = torch.full((T + 2, N + 60), 5.0, dtype=dtype, device="cuda")
        out = moe.moe_linear_e4m3(x, xs, w, ws, bias=b, out=buf[1:T + 1, 7:7 + N])
        check_linear(out, x, xs, w, ws, b)
        assert torch.equal(out, moe.moe_linear_e4m3(x, xs, w, ws, bias=b, out_dtype=dtype))
        assert (buf[0] == 5).all() and (buf[-1] == 5).all() and (buf[:, :7] == 5).all() and (buf[:, 7 + N:] == 5).all()


def test_linear_nothing_and_float8_tensors():
    x, xs, w, ws, _ = operands(4, 256, 384)
    assert moe.moe_linear_e4m3(x[:0], xs[:0], w, ws).shape == (0, 256)
    a = moe.moe_linear_e4m3(x.view(torch.float8_e4m3fn), xs, w.view(torch.float8_e4m3fn), ws)
    assert torch.equal(a, moe.moe_linear_e4m3(x, xs, w, ws))


@pytest.mark.parametrize("T", [5, 40, 160])
def test_linear_nan_stays_in_its_row_and_column(T):
    x, xs, w, ws, _ = operands(T, 260, 512)
    x[2, 300] = 0x7f
    w[77, 5] = 0xff
    out = moe.moe_linear_e4m3(x, xs, w, ws, out_dtype=F32)
    bad = torch.zeros(T, 260, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 77] = True, True
    assert torch.equal(out.isnan(), bad)


def test_linear_repeats_bit_for_bit_and_shares_a_workspace_over_rows():
    N, K = 1000, 7168
    ws_ = moe.moe_linear_e4m3_workspace(300, N, K)
    for T in (300, 1, 129, 33, 16, 300, 64, 8, 200):
        x, xs, w, ws, _ = operands(T, N, K)
        first = moe.moe_linear_e4m3(x, xs, w, ws, out_dtype=F32, ws=ws_)
        check_linear(first, x, xs, w, ws)
        for _ in range(5):
            assert torch.equal(moe.moe_linear_e4m3(x, xs, w, ws, out_dtype=F32, ws=ws_), first)
        assert torch.equal(moe.moe_linear_e4m3(x, xs, w, ws, out_dtype=F32), first)


def test_linear_two_streams_at_once():
    cases = [operands(T, N, K) for T, N, K in ((4, 4096, 7168), (150, 4096, 2048), (24, 576, 7168), (600, 1000, 1024))]
    want = [moe.moe_linear_e4m3(*c[:4], out_dtype=F32) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[] for _ in cases]
    for _ in range(20):
        for i, (s, c) in enumerate(zip(streams, cases)):
            got[i].append(moe.moe_linear_e4m3(*c[:4], out_dtype=F32, stream=s))
    torch.cuda.synchronize()
    for a, w in zip(got, want):
        assert all(torch.equal(b, w) for b in a)


def test_linear_large_offsets():
    """Weights of more than 2^32 bytes, and outputs of more than 2^31 elements: the last rows and columns are met."""
    K, N = 16384, 270000
    free = torch.cuda.mem_get_info()[0]
    if free < 30 << 30:
        pytest.skip("needs 30 GB")
    g = gen(21)
    w = torch.empty(N, K, dtype=U8, device="cuda")
    for i in range(0, N, 30000):
        w[i:i + 30000] = codes(g, min(30000, N - i), K)
    ws = scales(g, -(-N // 128), K // 128, 1 / (130 * K ** 0.5))
    pick = torch.tensor([0, 1, 127, 128, 131072, 262143, 262144, 262145, N - 129, N - 1], device="cuda")
    for T in (3, 60, 8000):
        x, xs = codes(g, T, K), scales(g, T, K // 128, 1 / 130)
        out = moe.moe_linear_e4m3(x, xs, w, ws)
        rows = torch.tensor([0, T // 2, T - 1], device="cuda")
        up = ws[pick // 128]
        a = ref.e4m3_values(x[rows]) * xs[rows].double().repeat_interleave(128, 1)
        b = ref.e4m3_values(w[pick]) * up.double().repeat_interleave(128, 1)
        y, size = a @ b.T, a.abs() @ b.abs().T
        err = size * (128 * 2.0 ** -23 + (K // 128 + 65) * ref.F32)
        assert ((out[rows][:, pick].double() - y).abs() <= err + ref.half_step(BF) * (y.abs() + err)).all()
        del out


# ---------------------------------------------------------------------------------------- dispatch
def ids(g, T, E, K, pad=0.0):
    i = torch.topk(torch.randn(T, E, generator=g, device="cuda"), K, dim=1)[1].to(I32)
    i[torch.rand(T, K, generator=g, device="cuda") < pad] = -1
    return i


def check_dispatch(p, idx, E, x, xs, shared, max_tokens=0, fill=None):
    want = ref.permute(idx.cpu(), E, shared, max_tokens)
    live = want["token"] >= 0
    at, tok = live.nonzero()[:, 0].cuda(), want["token"][live].cuda()
    xp = (p["xb"] if max_tokens else p["xp"]).view(-1, x.shape[1])
    sc = (p["xb_scales"] if max_tokens else p["xp_scales"]).view(-1, xs.shape[1])
    assert torch.equal(xp[at], x.view(U8)[tok]) and torch.equal(sc[at], xs[tok])
    if fill is not None:
        rest = (~live).nonzero()[:, 0].cuda()
        assert (xp[rest] == fill[0]).all() and (sc[rest] == fill[1]).all()
    assert torch.equal(p["src_row"].cpu().long(), want["src"]) and torch.equal(p["inv_map"].cpu().long(), want["inv"])
    if shared:
        assert torch.equal(p["shared_map"].cpu().long(), want["smap"])
    if max_tokens:
        assert torch.equal(p["masked_m"].cpu().long(), want["counts"])
    else:
        assert torch.equal(p["cu_seqlens"].cpu().long(), want["cu"])


@pytest.mark.parametrize("T,H,E,K", [(1, 128, 1, 1), (1, 7168, 256, 8), (3, 256, 8, 2), (64, 640, 60, 6), (65, 2048, 64, 8),
                                     (128, 7168, 256, 8), (333, 384, 1024, 3), (700, 8320, 16, 4), (2500, 512, 256, 8),
                                     (40, 16384, 40, 32), (512, 128, 16, 8), (513, 128, 16, 8), (1216, 256, 8, 1),
                                     (1217, 256, 8, 3), (3, 116096, 8, 2), (4097, 128, 4, 1), (2432, 128, 8, 1), (2433, 128, 8, 1),
                                     (1024, 128, 64, 32), (1025, 128, 64, 32), (4864, 128, 8, 6), (4865, 128, 8, 6),
                                     (3000, 256, 1, 1), (2048, 7168, 256, 8), (4256, 7168, 8, 2), (4300, 7168, 8, 2)])
@pytest.mark.parametrize("shared", [False, True])
def test_dispatch(T, H, E, K, shared):
    g = gen(T + H + E)
    x, xs, idx = codes(g, T, H), scales(g, T, H // 128, 1.0), ids(g, T, E, K, 0.15)
    rows = T * K + (T if shared else 0)
    xp, sc = torch.full((rows, H), 77, dtype=U8, device="cuda"), torch.full((rows, H // 128), -3.0, device="cuda")
    p = moe.moe_permute_e4m3(idx, E, x, xs, with_shared=shared, xp=xp, xp_scales=sc)
    check_dispatch(p, idx, E, x, xs, shared, fill=(77, -3.0))


@pytest.mark.parametrize("max_tokens", [1, 20, 64])
def test_dispatch_batched(max_tokens):
    g = gen(max_tokens)
    T, H, E, K = 64, 512, 8, 3
    x, xs, idx = codes(g, T, H), scales(g, T, H // 128, 1.0), ids(g, T, E, K, 0.1)
    rows = (E + 1) * max_tokens
    xp, sc = torch.full((rows, H), 77, dtype=U8, device="cuda"), torch.full((rows, H // 128), -3.0, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    p = moe.moe_permute_e4m3(idx, E, x, xs, with_shared=True, max_tokens=max_tokens, xp=xp, xp_scales=sc, dev_status=status)
    check_dispatch(p, idx, E, x, xs, True, max_tokens, fill=(77, -3.0))
    assert status.item() == (0 if max_tokens == 64 else moe.MOE_DEV_OVERFLOW)


@pytest.mark.parametrize("max_tokens", [300, 900])
def test_dispatch_batched_many(max_tokens):
    g = gen(max_tokens)
    T, H, E, K = 2000, 256, 8, 3
    x, xs, idx = codes(g, T, H), scales(g, T, H // 128, 1.0), ids(g, T, E, K, 0.1)
    rows = (E + 1) * max_tokens
    xp, sc = torch.full((rows, H), 77, dtype=U8, device="cuda"), torch.full((rows, H // 128), -3.0, device="cuda")
    status = torch.zeros(1, dtype=I32, device="cuda")
    p = moe.moe_permute_e4m3(idx, E, x, xs, with_shared=True, max_tokens=max_tokens, xp=xp, xp_scales=sc, dev_status=status)
    check_dispatch(p, idx, E, x, xs, True, max_tokens, fill=(77, -3.0))
    assert status.item() == moe.MOE_DEV_OVERFLOW      # the shared expert's 1998 or so tokens


@pytest.mark.parametrize("T,E,K", [(50, 8, 4), (900, 60, 6), (9000, 60, 6)])
def test_dispatch_one_expert_in_several_slots(T, E, K):
    """A token that names an expert twice has two rows there; one expert may take nearly all rows."""
    g = gen(T)
    x, xs = codes(g, T, 256), scales(g, T, 2, 1.0)
    idx = torch.randint(-1, E, (T, K), generator=g, device="cuda").to(I32)
    idx[torch.rand(T, K, generator=g, device="cuda") < 0.8] = E - 1
    check_dispatch(moe.moe_permute_e4m3(idx, E, x, xs, with_shared=True), idx, E, x, xs, True)


def test_dispatch_no_tokens():
    x, xs, idx = torch.empty(0, 256, dtype=U8, device="cuda"), torch.empty(0, 2, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda")
    p = moe.moe_permute_e4m3(idx, 4, x, xs, with_shared=True)
    assert p["cu_seqlens"].tolist() == [0] * 6 and p["xp"].shape == (0, 256)
    p = moe.moe_permute_e4m3(idx, 4, x, xs, max_tokens=3)
    assert p["masked_m"].tolist() == [0] * 4 and (p["src_row"] == -1).all()


def test_dispatch_large_offsets():
    """Rows past 2^31 bytes."""
    g = gen(5)
    T, H, E, K = 34000, 8192, 128, 8
    x, xs, idx = codes(g, T, H), scales(g, T, H // 128, 1.0), ids(g, T, E, K)
    p = moe.moe_permute_e4m3(idx, E, x, xs)
    inv = p["inv_map"].long()
    assert torch.equal(inv.flatten().sort()[0], torch.arange(T * K, device="cuda"))
    for k in range(K):
        assert torch.equal(p["xp_scales"][inv[:, k]], xs)
        for i in range(0, T, 8500):
            assert torch.equal(p["xp"][inv[i:i + 8500, k]], x[i:i + 8500])


def test_dispatch_all_padding_bad_ids_and_weights():
    g = gen(31)
    T, H, E, K = 70, 256, 8, 4
    x, xs = codes(g, T, H), scales(g, T, H // 128, 1.0)
    idx = torch.full((T, K), -1, dtype=I32, device="cuda")
    p = moe.moe_permute_e4m3(idx, E, x, xs, with_shared=True)
    check_dispatch(p, idx, E, x, xs, True)
    idx = ids(g, T, E, K, 0.2)
    idx[3, 1], idx[69, 0] = E, -7
    status = torch.zeros(1, dtype=I32, device="cuda")
    w = torch.rand(T, K, device="cuda")
    p = moe.moe_permute_e4m3(idx, E, x, xs, with_shared=True, dev_status=status, topk_w=w)
    check_dispatch(p, idx, E, x, xs, True)
    assert status.item() == moe.MOE_DEV_BAD_EXPERT
    n = int(p["cu_seqlens"][-1])
    src = p["src_row"][:n].long()
    want = torch.cat((w.flatten(), torch.ones(T, device="cuda")))[src]
    assert torch.equal(p["row_weights"][:n], want)
    idx[5] = idx[5, 0].clamp(min=0)       # one expert in every slot of a token
    check_dispatch(moe.moe_permute_e4m3(idx, E, x, xs), idx, E, x, xs, False)


def test_dispatch_matches_the_quantising_permute():
    """Rows quantised first and dispatched are those that moe_permute quantises on the way."""
    g = gen(41)
    x, idx = randn(g, 300, 1024).to(BF), ids(g, 300, 16, 4, 0.1)
    a = moe.moe_permute(idx, 16, x, with_shared=True, out_dtype=moe.MOE_E4M3)
    b = moe.moe_permute_e4m3(idx, 16, *moe.moe_quantize_act_fp8(x), with_shared=True)
    n = int(a["cu_seqlens"][-1])
    for k in ("cu_seqlens", "src_row", "inv_map", "shared_map"):
        assert torch.equal(a[k], b[k])
    assert torch.equal(a["xp"][:n], b["xp"][:n]) and torch.equal(a["xp_scales"][:n], b["xp_scales"][:n])


# ------------------------------------------------------------------------------------------- layer
def e4m3_layer(g, T, H, I, E, K, **kw):
    def weights(*shape):
        return moe.moe_quantize_weight_fp8((randn(g, *shape) * shape[-1] ** -0.5).to(BF))
    (a, ca), (b, cb) = weights(E, 2 * I, H), weights(E, H, I)
    (c, cc), (d, cd) = weights(2 * I, H), weights(H, I)
    return moe.MoeLayer(T, H, I, E, K, moe.MOE_E4M3, w13=a, w2=b, w13_scales=ca, w2_scales=cb, shared_w13=c,
                        shared_w2=d, shared_w13_scales=cc, shared_w2_scales=cd, **kw)


@pytest.mark.parametrize("kw", [{}, dict(max_tokens=40), dict(weight_in_down=True), dict(fuse_combine=True),
                                dict(weight_tiles=True)])
def test_layer_on_e4m3_rows_is_the_layer_on_bf16_rows(kw):
    g = gen(51)
    T, H, I, E, K = 90, 512, 256, 8, 3
    layer = e4m3_layer(g, T, H, I, E, K, **kw)
    x, logits = randn(g, T, H).to(BF), randn(g, T, E)
    n = torch.tensor([77], dtype=I32, device="cuda")
    outs = []
    for x_, s_ in ((x, None), moe.moe_quantize_act_fp8(x)):
        idx, w = torch.empty(T, K, dtype=I32, device="cuda"), torch.empty(T, K, device="cuda")
        out = torch.empty(T, H, dtype=BF, device="cuda")
        outs.append((layer.forward(x_, out, idx, w, logits=logits, num_tokens=n, x_scales=s_), idx, w))
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_block_of_the_path_in_a_graph():
    """A block as a model runs it -- norm, router, layer on the norm's E4M3 rows, norm, head -- eager, then
    captured and replayed on new inputs and another number of tokens."""
    g = gen(61)
    T, H, I, E, K, V = 48, 512, 256, 8, 2, 1000
    layer = e4m3_layer(g, T, H, I, E, K)
    router = randn(g, E, H) * H ** -0.5
    w1, w2 = randn(g, H) * 0.1 + 1, (randn(g, H) * 0.1 + 1).to(BF)
    head, head_s = codes(g, V, H), scales(g, -(-V // 128), H // 128, 1 / (130 * H ** 0.5))
    ws = moe.moe_linear_e4m3_workspace(T, V, H)
    status = torch.zeros(1, dtype=I32, device="cuda")
    x, res, n = randn(g, T, H).to(BF), randn(g, T, H), torch.tensor([T], dtype=I32, device="cuda")
    idx, wt, y = torch.empty(T, K, dtype=I32, device="cuda"), torch.empty(T, K, device="cuda"), torch.empty_like(x)

    def block():
        a, q, s, r = moe.moe_rmsnorm(x, w1, EPS, residual=res, e4m3=True, num_tokens=n)
        layer.forward(q, y, idx, wt, logits=a.float() @ router.T, num_tokens=n, dev_status=status, x_scales=s)
        _, q2, s2, r2 = moe.moe_rmsnorm(y, w2, EPS, residual=r, bf16=False, e4m3=True, num_tokens=n)
        out = moe.moe_linear_e4m3(q2, s2, head, head_s, out_dtype=F32, ws=ws, dev_status=status)
        return a, q, s, r, q2, s2, r2, out

    def check(got, live):
        a, q, s, r, q2, s2, r2, out = got
        check_norm((a, q, s, r), x, w1, EPS, res, live)
        check_norm((None, q2, s2, r2), y, w2, EPS, r, live)
        check_linear(out[:live], q2[:live], s2[:live], head, head_s)
        assert status.item() == 0

    check(block(), T)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        block()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block()
    for live in (T, 31, 1):
        x.copy_(randn(g, T, H))
        res.copy_(randn(g, T, H))
        n.fill_(live)
        graph.replay()
        torch.cuda.synchronize()
        check(got, live)


@pytest.mark.parametrize("weights", ["e4m3", "w4"])
def test_decode_step_with_norms_and_an_e4m3_head(weights):
    """The decode step's own path: the router inside the layers and ahead of them give the same bits, and each step of the
    stack is the sum of its parts."""
    from combine_moe_route_softmax_gb300 import decode_few
    size = dict(layers=2, H=256, I=128, E=8, K=2, vocab=512, weights=weights, act8=True)
    ms, same = decode_few.run(tokens=5, steps=3, **size)
    assert same and all(t > 0 for t in ms.values())
    step = decode_few.DecodeStep(5, **size)
    x = step.table[:5].clone()
    logits, ids = step(x)
    d = stream = None
    for i, layer in enumerate(step.inside):
        a, _, _, r = moe.moe_rmsnorm(x if i == 0 else d, step.norms[i], EPS, residual=None if i == 0 else stream)
        stream = x if i == 0 else r
        d, idx, _ = layer.forward(a)
        assert torch.equal(idx, ids[i])
    _, q, s, _ = moe.moe_rmsnorm(d, step.norms[-1], EPS, residual=stream, bf16=False, e4m3=True)
    check_linear(logits, q, s, *step.head)
