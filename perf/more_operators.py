"""The 8-bit activation path as measured work: what each case stands for, its inputs, and one pass of it.

Three operators around a Mixture-of-Experts layer whose weights are E4M3 with 128 x 128 block scales:

* ``norm``      the residual's addition and root-mean-square norm ahead of the layer, leaving the new
  residual, BF16 rows (for the router) and E4M3 rows with a scale per 1 x 128 block: ``moe_rmsnorm``.
* ``linear``    y = x W^T (+ bias) with both operands in E4M3, scales per 1 x 128 block of x and per
  128 x 128 block of W (a dense projection, a shared expert's matrix, a head): ``moe_linear_e4m3``.
* ``dispatch``  rows that are E4M3 already, gathered into the expert-major layout with their scales:
  ``moe_permute_e4m3``.

``run`` computes a case in elementary torch operations, or calls the library when ``own`` is set.
"""
import math

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def _norm(name, T, H, residual="bf16", weight="bf16", bf16=True, e4m3=True, valid=0):
    """residual: "bf16", "f32" or "" (none); valid > 0: rows of the bucket that are tokens."""
    return {"name": name, "op": "norm", "T": T, "H": H, "residual": residual, "weight": weight, "bf16": bf16,
            "e4m3": e4m3, "valid": valid}


def _linear(name, T, N, K, bias=False, f32=False):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "bias": bias, "f32": f32}


def _dispatch(name, T, H, E, K, shared, pad=0.0):
    return {"name": name, "op": "dispatch", "T": T, "H": H, "E": E, "K": K, "shared": shared, "pad": pad}


def listed():
    return [
        # one token ahead of a "decode" layer: latency counts
        _norm("norm 1x7168", 1, 7168),
        # a decode batch of 128 at "decode", the residual kept in float32
        _norm("norm 128x7168 f32 residual", 128, 7168, residual="f32", weight="f32"),
        # the first norm of a stack (no residual yet) on an odd number of "mid" rows, BF16 rows only
        _norm("norm 1027x2048 bf16 only", 1027, 2048, residual="", e4m3=False),
        # the "prefill" bucket of 16384 rows, 12000 of them tokens
        _norm("norm 16384x7168 12000 valid", 16384, 7168, valid=12000),
        # the smallest product, one token at the "tiny" workload's sizes: latency counts
        _linear("e4m3 1x512x256", 1, 512, 256),
        # one token through a wide dense projection: its weights are read once from memory
        _linear("e4m3 1x7168x16384", 1, 7168, 16384),
        # thirteen tokens in flight through the gate/up matrix of the "decode" workload's shared expert
        _linear("e4m3 13x4096x7168", 13, 4096, 7168),
        # the "decode" batch through a head over a vocabulary, float32 results
        _linear("e4m3 128x40960x4096 f32", 128, 40960, 4096, f32=True),
        # an odd batch through a narrow projection that is no multiple of 128 wide, with a bias
        _linear("e4m3 700x576x7168 bias", 700, 576, 7168, bias=True),
        # the "prefill" batch through the gate/up matrix of its shared expert
        _linear("e4m3 8192x4096x7168", 8192, 4096, 7168),
        # the "decode" batch into 256 experts and the shared one
        _dispatch("dispatch 128 of decode", 128, 7168, 256, 8, True),
        # the "prefill" batch, a tenth of the slots padding
        _dispatch("dispatch 8192 of prefill", 8192, 7168, 256, 8, True, pad=0.1),
    ]


def _size(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(("norm", "linear", "linear", "linear", "dispatch"))
    if op == "norm":
        e4m3 = rng.random() < 0.7
        T = _size(rng, 1, 16384, 1)
        H = _size(rng, 256, 7168, 128) if e4m3 else _size(rng, 256, 7168, 8)
        c = _norm("", T, H, rng.choice(("bf16", "bf16", "f32", "")), rng.choice(("bf16", "f32")),
                  not e4m3 or rng.random() < 0.6, e4m3, rng.randint(1, T) if rng.random() < 0.3 else 0)
        if c["residual"] == "f32" and c["T"] * c["H"] > 8192 * 7168:
            c["residual"] = "bf16"
    elif op == "linear":
        while True:
            N = _size(rng, 64, 40960, 1) if rng.random() < 0.3 else _size(rng, 64, 40960, 64)
            c = _linear("", _size(rng, 1, 8192, 1), N, _size(rng, 128, 16384, 128), rng.random() < 0.4,
                        rng.random() < 0.3)
            if c["T"] * c["N"] * c["K"] <= 8192 * 4096 * 7168 and c["N"] * c["K"] <= 40960 * 4096:
                break
    else:
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 256))
        while True:
            c = _dispatch("", _size(rng, 1, 8192, 1), _size(rng, 256, 7168, 128), E, rng.randint(1, min(8, E)),
                          rng.random() < 0.5, rng.choice((0.0, 0.1, 0.3)))
            if work(c)["bytes"] <= 6e8:
                break
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _codes(g, rows, cols):
    """E4M3 codes as a quantiser leaves them: normal values, the block's largest near 448."""
    v = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.bfloat16) * 130
    return v.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _scales(g, rows, cols, unit):
    return (torch.rand(rows, cols, generator=g, device="cuda") + 0.5) * unit


def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        # rows of different sizes, and a residual that has grown past the layer's output
        s = {"x": (torch.randn(T, H, generator=g, device="cuda") *
                   (torch.rand(T, 1, generator=g, device="cuda") * 2 + 0.1)).to(torch.bfloat16)}
        if c["residual"]:
            r = torch.randn(T, H, generator=g, device="cuda") * 4
            s["residual"] = r if c["residual"] == "f32" else r.to(torch.bfloat16)
        else:
            s["residual"] = None
        w = torch.randn(H, generator=g, device="cuda") * 0.3 + 1
        s["weight"] = w if c["weight"] == "f32" else w.to(torch.bfloat16)
        s["n"] = torch.tensor([c["valid"]], dtype=torch.int32, device="cuda") if c["valid"] else None
        return s
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        return {"x": _codes(g, T, K), "x_scales": _scales(g, T, K // 128, 1 / 130),
                "w": _codes(g, N, K), "w_scales": _scales(g, -(-N // 128), K // 128, 1 / (130 * math.sqrt(K))),
                "bias": torch.randn(N, generator=g, device="cuda") if c["bias"] else None}
    # distinct experts per token, padding slots -1, some tokens without any
    E, K = c["E"], c["K"]
    idx = torch.topk(torch.randn(T, E, generator=g, device="cuda"), K, dim=1)[1].to(torch.int32)
    idx[torch.rand(T, K, generator=g, device="cuda") < c["pad"]] = -1
    return {"x": _codes(g, T, c["H"]), "x_scales": _scales(g, T, c["H"] // 128, 1 / 130), "idx": idx}


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    # the buffers that a serving program keeps: rows that a pass leaves alone keep what they held
    T = c["T"]
    if c["op"] == "norm":
        H = c["H"]
        s["out"] = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") if c["bf16"] else None
        s["q"] = torch.zeros(T, H, dtype=torch.uint8, device="cuda") if c["e4m3"] else None
        s["q_scales"] = torch.zeros(T, H // 128, device="cuda") if c["e4m3"] else None
        s["residual_out"] = None if s["residual"] is None else torch.zeros_like(s["residual"])
    elif c["op"] == "dispatch":
        rows = T * c["K"] + (T if c["shared"] else 0)
        s["xp"] = torch.zeros(rows, c["H"], dtype=torch.uint8, device="cuda")
        s["xp_scales"] = torch.zeros(rows, c["H"] // 128, device="cuda")
    if own:
        import combine_moe_route_softmax_gb300 as moe
        if c["op"] == "linear":
            s["ws"] = moe.moe_linear_e4m3_workspace(T, c["N"], c["K"])
        elif c["op"] == "dispatch":
            s["ws"] = torch.empty(moe.moe_permute_workspace_bytes(T, c["K"], c["E"], c["shared"]), dtype=torch.uint8,
                                  device="cuda")
    return s


# ------------------------------------------------------------------------------- plain form
def _fp8(t):
    return t.view(torch.float8_e4m3fn)


def _plain_norm(c, s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    y = h * (1 / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)) * s["weight"].float()
    live = None if s["n"] is None else (torch.arange(c["T"], device=h.device) < s["n"]).unsqueeze(1)
    keep = lambda new, old: new if live is None else torch.where(live, new, old)  # noqa: E731
    got = {}
    if c["bf16"]:
        got["out"] = keep(y.to(torch.bfloat16), s["out"])
    if c["e4m3"]:
        b = y.view(c["T"], -1, 128)
        sc = b.abs().amax(2) / 448
        sc = torch.where(sc > 0, sc, 1.0)
        q = (b / sc.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).view(y.shape)
        got["q"] = _fp8(keep(q, s["q"]))
        got["q_scales"] = keep(sc, s["q_scales"])
    if s["residual"] is not None:
        got["residual"] = keep(h.to(s["residual"].dtype), s["residual_out"])
    return got


def _plain_linear(c, s):
    K, N = c["K"], c["N"]
    x = (_fp8(s["x"]).float().view(c["T"], K // 128, 128) * s["x_scales"].unsqueeze(2)).view(c["T"], K)
    up = s["w_scales"].repeat_interleave(128, 0)[:N]
    w = (_fp8(s["w"]).float().view(N, K // 128, 128) * up.unsqueeze(2)).view(N, K)
    y = x @ w.T
    if s["bias"] is not None:
        y = y + s["bias"]
    return y if c["f32"] else y.to(torch.bfloat16)


def _plain_dispatch(c, s):
    T, K, E, idx = c["T"], c["K"], c["E"], s["idx"]
    flat = idx.flatten().long()
    if c["shared"]:   # the shared expert is one more segment: every token with a valid slot
        flat = torch.cat((flat, torch.where((idx >= 0).any(1), E, -1)))
    nseg = E + int(c["shared"])
    order = torch.argsort(torch.where(flat < 0, nseg, flat), stable=True)       # padding goes last
    row = torch.arange(order.numel(), device=flat.device)
    cu = (flat.unsqueeze(1) < torch.arange(nseg + 1, device=flat.device)).logical_and(flat.unsqueeze(1) >= 0).sum(0)
    live = row < cu[-1]
    src = torch.where(live, order, -1)
    inv = torch.empty_like(order)
    inv[order] = torch.where(live, row, -1)
    token = torch.where(order < T * K, order // K, order - T * K)
    xp = torch.where(live.unsqueeze(1), s["x"][token], s["xp"])
    sc = torch.where(live.unsqueeze(1), s["x_scales"][token], s["xp_scales"])
    got = {"xp": _fp8(xp), "xp_scales": sc, "cu_seqlens": cu.int(), "src_row": src.int(),
           "inv_map": inv[:T * K].view(T, K).int()}
    if c["shared"]:
        got["shared_map"] = inv[T * K:].int()
    return got


def run(state):
    s, c = state, state["case"]
    if own:
        import combine_moe_route_softmax_gb300 as moe
        if c["op"] == "linear":
            return moe.moe_linear_e4m3(s["x"], s["x_scales"], s["w"], s["w_scales"], bias=s["bias"],
                                       out_dtype=torch.float32 if c["f32"] else torch.bfloat16, ws=s["ws"])
        if c["op"] == "norm":
            out, q, sc, r = moe.moe_rmsnorm(s["x"], s["weight"], EPS, residual=s["residual"], out=s["out"], q=s["q"],
                                            q_scales=s["q_scales"], residual_out=s["residual_out"], num_tokens=s["n"])
            got = {"out": out, "q": None if q is None else _fp8(q), "q_scales": sc, "residual": r}
            return {k: v for k, v in got.items() if v is not None}
        p = moe.moe_permute_e4m3(s["idx"], c["E"], s["x"], s["x_scales"], with_shared=c["shared"], xp=s["xp"],
                                 xp_scales=s["xp_scales"], ws=s["ws"])
        got = {k: p[k] for k in ("xp_scales", "cu_seqlens", "src_row", "inv_map")}
        got["xp"] = _fp8(p["xp"])
        if c["shared"]:
            got["shared_map"] = p["shared_map"]
        return got
    return {"norm": _plain_norm, "linear": _plain_linear, "dispatch": _plain_dispatch}[c["op"]](c, s)


# -------------------------------------------------------------------------------------- work
def work(case):
    c = case
    T = c["T"]
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        b = T * K + T * K // 32 + N * K + 4 * -(-N // 128) * (K // 128) + T * N * (4 if c["f32"] else 2)
        return {"bytes": b + (4 * N if c["bias"] else 0), "flops": 2 * T * N * K}
    H = c["H"]
    if c["op"] == "norm":
        n = c["valid"] or T
        res = {"": 0, "bf16": 4, "f32": 8}[c["residual"]]
        b = n * H * (2 + res + (2 if c["bf16"] else 0)) + (n * (H + H // 32) if c["e4m3"] else 0)
        return {"bytes": b + H * (2 if c["weight"] == "bf16" else 4), "flops": 8 * n * H}
    # rows written: the valid slots, and a shared row for each token with one
    K = c["K"]
    rows = T * K * (1 - c["pad"]) + (T * (1 - c["pad"] ** K) if c["shared"] else 0)
    index = 8 * T * K + 4 * rows + 4 * c["E"] + (4 * T if c["shared"] else 0)
    return {"bytes": int((T * (1 - c["pad"] ** K) + rows) * (H + H // 32) + index), "flops": 0}


# ------------------------------------------------------------------------- exact (64 bits)
def _e4m3_64(code):
    """The value of E4M3 codes from the format's definition: sign, 4 exponent bits (bias 7), 3 of mantissa."""
    i = torch.arange(256, device=code.device)
    e, m = ((i >> 3) & 15).double(), (i & 7).double()
    v = torch.where(e > 0, (1 + m / 8) * torch.exp2(e - 7), m / 8 * 2.0 ** -6) * torch.where(i < 128, 1.0, -1.0)
    return torch.where((i & 127) == 127, math.nan, v)[code.long()]


def exact(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    T = c["T"]
    if c["op"] == "linear":
        N, K = c["N"], c["K"]
        y = torch.zeros(T, N, dtype=torch.float64, device="cuda")
        row_block = torch.arange(N, device="cuda") // 128
        step = 2048   # columns at a time: E4M3 products, each block's sum times its two scales
        for k0 in range(0, K, step):
            k1 = min(K, k0 + step)
            block = torch.arange(k0, k1, device="cuda") // 128
            y += (_e4m3_64(s["x"][:, k0:k1]) * s["x_scales"].double()[:, block]) @ \
                (_e4m3_64(s["w"][:, k0:k1]) * s["w_scales"].double()[row_block][:, block]).T
        return y if s["bias"] is None else y + s["bias"].double()
    if c["op"] == "norm":
        n = c["valid"] or T
        h = s["x"][:n].double() + (0 if s["residual"] is None else s["residual"][:n].double())
        y = h / torch.sqrt(h.square().sum(1, keepdim=True) / c["H"] + EPS) * s["weight"].double()
        whole = lambda v: torch.cat((v, v.new_zeros(T - n, v.shape[1])))  # noqa: E731
        got = {}
        if c["bf16"]:
            got["out"] = whole(y)
        if c["e4m3"]:
            sc = torch.stack([blk.abs().max(1)[0] for blk in y.split(128, 1)], 1) / 448
            got["q"] = whole(y / sc.repeat_interleave(128, 1))
            got["q_scales"] = whole(sc)
        if s["residual"] is not None:
            got["residual"] = whole(h)
        return got
    # a copy: nothing is computed but the order, here by filling the segments one after the other
    idx = s["idx"]
    token, slot = [], []
    for e in range(c["E"]):
        t, k = (idx == e).nonzero(as_tuple=True)
        token.append(t)
        slot.append(t * c["K"] + k)
    if c["shared"]:
        t = (idx >= 0).any(1).nonzero()[:, 0]
        token.append(t)
        slot.append(T * c["K"] + t)
    cu = torch.tensor([0] + [len(t) for t in token], device=idx.device).cumsum(0)
    token, slot = torch.cat(token), torch.cat(slot)
    total = T * c["K"] + (T if c["shared"] else 0)
    src = torch.full((total,), -1, device=idx.device)
    src[:len(slot)] = slot
    inv = torch.full((total,), -1, device=idx.device)
    inv[slot] = torch.arange(len(slot), device=idx.device)
    sc = torch.zeros(total, c["H"] // 128, dtype=torch.float64, device=idx.device)
    sc[:len(slot)] = s["x_scales"].double()[token]
    got = {"xp": None, "xp_scales": sc, "cu_seqlens": cu.int(), "src_row": src.int(),
           "inv_map": inv[:T * c["K"]].view(T, -1).int()}
    if c["shared"]:
        got["shared_map"] = inv[T * c["K"]:].int()
    return got
