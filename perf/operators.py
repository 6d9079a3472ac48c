"""The few-token MoE operators as measured work: what each case stands for, its inputs, and one pass of it.

Three operators that a decode step of a Mixture-of-Experts model needs next to the prefill path:

* ``linear``  y = x W^T (+ bias) for a few rows of BF16 x, with W in 4-bit codes with a BF16 scale (and
  optionally a zero point) per group of 32, 64 or 128 columns: ``moe_linear_w4``.
* ``route``   the router from hidden states: logits = x Wr^T + bias, then the top K of them and their
  renormalised softmax weights: ``moe_route_hidden``.
* ``layer``   the whole layer for 1 to 32 tokens in one kernel: (router ->) gate/up with SwiGLU -> down ->
  the sum over a token's experts, with BF16, E4M3 (128 x 128 block scales) or 4-bit weights:
  ``MoeLayerFew``.

``run`` computes a case in elementary torch operations, or calls the library when ``own`` is set.
"""
import math

import torch

own = False

CHUNK = 1 << 31     # float32 weights that the plain form of a layer holds at a time (8 GB)


# ------------------------------------------------------------------------------------- cases
def _linear(name, T, N, K, group, zeros=False, bias=False, f32=False):
    return {"name": name, "op": "linear", "T": T, "N": N, "K": K, "group": group, "zeros": zeros, "bias": bias,
            "f32": f32}


def _route(name, T, H, E, K, bias=False):
    return {"name": name, "op": "route", "T": T, "H": H, "E": E, "K": K, "bias": bias}


def _layer(name, T, H, I, E, K, dtype, shared, router, pad=0.0, group=0, zeros=False):
    return {"name": name, "op": "layer", "T": T, "H": H, "I": I, "E": E, "K": K, "dtype": dtype, "shared": shared,
            "router": router, "pad": pad, "group": group, "zeros": zeros}


def listed():
    return [
        # the smallest product, one token at the "tiny" workload's sizes: latency counts
        _linear("w4 1x512x256 g32", 1, 512, 256, 32),
        # one token through a 4-bit gate/up matrix of the "decode" workload's shared expert
        _linear("w4 1x4096x7168 g128", 1, 4096, 7168, 128),
        # seven tokens in flight, down projection's shape, with zero points and a bias
        _linear("w4 7x7168x2048 g64 zp", 7, 7168, 2048, 64, zeros=True, bias=True),
        # a wide output (a head over a vocabulary) for a small decode batch, float32 results
        _linear("w4 24x40960x4096 g128 f32", 24, 40960, 4096, 128, f32=True),
        # one token of the "mid" workload's router
        _route("route 1x2048 64/8", 1, 2048, 64, 8),
        # the largest few-token batch of the "decode" workload's router
        _route("route 32x7168 256/8 bias", 32, 7168, 256, 8, bias=True),
        # the smallest layer, one token at "tiny": latency counts
        _layer("layer bf16 tiny T1", 1, 256, 512, 8, 2, "bf16", False, True),
        # a few tokens at "mid", routed elsewhere, a tenth of the slots padding
        _layer("layer bf16 mid T5", 5, 2048, 1408, 64, 8, "bf16", False, False, pad=0.1),
        # one token at "decode": E4M3 weights, a shared expert, the router inside
        _layer("layer e4m3 decode T1", 1, 7168, 2048, 256, 8, "e4m3", True, True),
        # a decode batch of sixteen at "decode"
        _layer("layer e4m3 decode T16", 16, 7168, 2048, 256, 8, "e4m3", True, True),
        # one token at "decode" with 4-bit weights
        _layer("layer w4 decode T1", 1, 7168, 2048, 256, 8, "w4", True, True, group=128),
        # the largest few-token batch at "mid", 4-bit weights with zero points, small groups
        _layer("layer w4 mid T32 g32 zp", 32, 2048, 1408, 64, 8, "w4", True, False, group=32, zeros=True),
    ]


def _size(rng, lo, hi, step):
    """A multiple of step in [lo, hi], spread over its logarithm (no 3072, nor its half or double)."""
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
        if lo <= v <= hi and v not in (1536, 3072, 6144):
            return v


def draw(rng):
    op = rng.choice(("linear", "layer", "layer", "route"))
    if op == "linear":
        while True:
            c = _linear("", _size(rng, 1, 32, 1), _size(rng, 256, 40960, 16), _size(rng, 256, 7168, 128),
                        rng.choice((32, 64, 128)), rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.3)
            if c["N"] * c["K"] <= 40960 * 4096:
                break
    elif op == "route":
        E = rng.choice((8, 16, 60, 64, 96, 128, 160, 256))
        c = _route("", _size(rng, 1, 32, 1), _size(rng, 256, 7168, 128), E, rng.randint(1, min(8, E)), rng.random() < 0.5)
    else:
        dtype = rng.choice(("bf16", "e4m3", "w4"))
        while True:
            E = rng.choice((8, 16, 60, 64, 96, 128))
            c = _layer("", _size(rng, 1, 32, 1), _size(rng, 256, 7168, 128), _size(rng, 256, 2048, 128), E,
                       rng.randint(1, min(8, E)), dtype, rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice((0.0, 0.2)), rng.choice((32, 64, 128)) if dtype == "w4" else 0,
                       dtype == "w4" and rng.random() < 0.5)
            if c["router"]:
                c["pad"] = 0.0
            if _weight_bytes(c) * c["E"] <= 6e9 and work(c)["bytes"] <= 4e9:
                break
    del c["name"]
    return c


# ------------------------------------------------------------------------------------ inputs
def _normal(g, shape, std):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)


def _w4(g, mats, n, k, group, zeros):
    """Codes as a quantiser leaves them (a bell around the zero point), scales for a weight of
    standard deviation 1/sqrt(k): q [mats, n, k/2] (even column in the low nibble), scales and zeros
    [mats, k/group, n]."""
    q = torch.empty(mats, n, k // 2, dtype=torch.uint8, device="cuda")
    for m in range(mats):
        c = (torch.randn(n, k, generator=g, device="cuda", dtype=torch.bfloat16) * 2.5 + 8).round_().clamp_(0, 15)
        c = c.to(torch.uint8).view(n, k // 2, 2)
        torch.bitwise_or(c[..., 0], c[..., 1] << 4, out=q[m])
    s = (torch.rand(mats, k // group, n, generator=g, device="cuda") + 0.5) / (2.5 * math.sqrt(k))
    z = torch.randint(6, 11, (mats, k // group, n), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return {"w": q, "scales": s.to(torch.bfloat16), "zeros": z}


def _weights(g, c, mats, n, k):
    if c["dtype"] == "w4":
        return _w4(g, mats, n, k, c["group"], c["zeros"])
    if c["dtype"] == "e4m3":
        q = torch.empty(mats, n, k, dtype=torch.uint8, device="cuda")
        for m in range(mats):
            v = torch.randn(n, k, generator=g, device="cuda", dtype=torch.bfloat16) * 100
            q[m] = v.clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        s = (torch.rand(mats, n // 128, k // 128, generator=g, device="cuda") + 0.5) / (100 * math.sqrt(k))
        return {"w": q, "scales": s, "zeros": None}
    w = torch.empty(mats, n, k, dtype=torch.bfloat16, device="cuda")
    for m in range(mats):
        w[m] = _normal(g, (n, k), 1 / math.sqrt(k))
    return {"w": w, "scales": None, "zeros": None}


def _inputs(c, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    T = c["T"]
    if c["op"] == "linear":
        w = _w4(g, 1, c["N"], c["K"], c["group"], c["zeros"])
        return {"x": _normal(g, (T, c["K"]), 1.0), "q": w["w"][0], "scales": w["scales"][0],
                "zeros": w["zeros"][0] if c["zeros"] else None,
                "bias": torch.randn(c["N"], generator=g, device="cuda") if c["bias"] else None}
    H, E, K = c["H"], c["E"], c["K"]
    s = {"x": _normal(g, (T, H), 1.0)}
    if c["op"] == "route" or c["router"]:
        s["w_router"] = _normal(g, (E, H), 1 / math.sqrt(H))
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.1 if c.get("bias") else None
    else:
        # routed elsewhere: distinct experts, padding slots -1, weights that sum to one
        l = torch.randn(T, E, generator=g, device="cuda")
        v, idx = torch.topk(l, K, dim=1)
        s["topk_idx"] = idx.to(torch.int32)
        s["topk_idx"][torch.rand(T, K, generator=g, device="cuda") < c["pad"]] = -1
        s["topk_w"] = torch.softmax(v, 1)
    if c["op"] == "layer":
        I = c["I"]
        s["w13"], s["w2"] = _weights(g, c, E, 2 * I, H), _weights(g, c, E, H, I)
        s["s13"], s["s2"] = (_weights(g, c, 1, 2 * I, H), _weights(g, c, 1, H, I)) if c["shared"] else (None, None)
    return s


def prepare(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    s["case"] = c
    if own:
        # what a serving program does once per model and holds for its life: 4-bit weights in the
        # kernels' order, the workspace of a call, a layer's descriptor with its weights' addresses
        import combine_moe_route_softmax_gb300 as moe
        if c["op"] == "linear":
            s["packed"] = moe.moe_pack_w4(s["q"], s["scales"], s["zeros"])
            s["ws"] = moe.moe_linear_w4_workspace(c["T"], c["N"], c["K"])
        elif c["op"] == "route":
            s["ws"] = moe.moe_route_hidden_workspace()
        else:
            def form(w, one):
                if w is None:
                    return None, None
                if c["dtype"] == "w4":
                    return moe.moe_pack_w4(w["w"], w["scales"], w["zeros"]), None
                pick = (lambda t: None if t is None else t[0]) if one else (lambda t: t)
                return pick(w["w"]), pick(w["scales"])

            (w13, c13), (w2, c2) = form(s["w13"], False), form(s["w2"], False)
            (s13, d13), (s2, d2) = form(s["s13"], True), form(s["s2"], True)
            s["layer"] = moe.MoeLayerFew(
                c["T"], c["H"], c["I"], c["E"], c["K"],
                {"bf16": moe.MOE_BF16, "e4m3": moe.MOE_E4M3, "w4": moe.MOE_W4}[c["dtype"]],
                w13=w13, w2=w2, shared_w13=s13, shared_w2=s2, w13_scales=c13, w2_scales=c2,
                shared_w13_scales=d13, shared_w2_scales=d2, w_router=s.get("w_router"))
    return s


# ------------------------------------------------------------------------------- plain form
def _codes(q):
    """[..., k/2] bytes -> [..., k] code values in float32."""
    return torch.stack((q & 15, q >> 4), -1).flatten(-2).float()


def _dequant(c, w, pick=None):
    """Weights [m, n, k] in float32 (those of the matrices in pick)."""
    take = (lambda t: t) if pick is None else (lambda t: t.index_select(0, pick))
    v = take(w["w"])
    if c["dtype"] == "bf16":
        return v.float()
    if c["dtype"] == "e4m3":
        m, n, k = v.shape
        v = v.view(torch.float8_e4m3fn).float().view(m, n // 128, 128, k // 128, 128)
        return (v * take(w["scales"])[:, :, None, :, None]).view(m, n, k)
    m, n, kh = v.shape
    s = take(w["scales"]).float().transpose(1, 2).unsqueeze(-1)
    z = take(w["zeros"]).float().transpose(1, 2).unsqueeze(-1) if w["zeros"] is not None else 8.0
    return ((_codes(v).view(m, n, s.shape[2], -1) - z) * s).view(m, n, 2 * kh)


def _plain_linear(c, s):
    w = _dequant({"dtype": "w4"}, {"w": s["q"][None], "scales": s["scales"][None],
                                   "zeros": None if s["zeros"] is None else s["zeros"][None]})[0]
    y = s["x"].float() @ w.T
    if s["bias"] is not None:
        y = y + s["bias"]
    return y if c["f32"] else y.to(torch.bfloat16)


def _plain_route(c, s):
    # in 64 bits: which expert a near tie falls to must not hang on the order of the sum
    logits = s["x"].double() @ s["w_router"].double().T
    if s.get("bias") is not None:
        logits = logits + s["bias"].double()
    logits = logits.float()
    v, idx = torch.sort(logits, dim=1, descending=True, stable=True)   # equal logits: the lower id first
    v, idx = v[:, :c["K"]], idx[:, :c["K"]]
    e = torch.exp(v - v[:, :1])
    return idx.to(torch.int32), e / e.sum(1, keepdim=True), logits


def _expert(x, w13, w2):
    """SwiGLU experts: x [b, h], w13 [b, 2i, h], w2 [b, h, i] -> [b, h]."""
    g, u = torch.bmm(w13, x.unsqueeze(2)).squeeze(2).chunk(2, 1)
    h = g / (1 + torch.exp(-g)) * u
    return torch.bmm(w2, h.unsqueeze(2)).squeeze(2)


def _plain_layer(c, s):
    x, K = s["x"].float(), c["K"]
    if c["router"]:
        idx, wt, _ = _plain_route(c, s)
    else:
        idx, wt = s["topk_idx"], s["topk_w"]
    outs = []
    # the chosen experts' weights in 32 bits, as many tokens at a time as CHUNK holds
    n = max(1, CHUNK // (K * 3 * c["I"] * c["H"]))
    for xc, ic, wc in zip(x.split(n), idx.split(n), wt.split(n)):
        pick = ic.clamp(min=0).flatten()
        y = _expert(xc.repeat_interleave(K, 0), _dequant(c, s["w13"], pick), _dequant(c, s["w2"], pick))
        y = y.view(-1, K, c["H"]) * wc.unsqueeze(2)
        outs.append(torch.where((ic >= 0).unsqueeze(2), y, 0.0).sum(1))
    out = torch.cat(outs)
    if c["shared"]:
        g, u = (x @ _dequant(c, s["s13"])[0].T).chunk(2, 1)
        y = (g / (1 + torch.exp(-g)) * u) @ _dequant(c, s["s2"])[0].T
        out = out + torch.where((idx >= 0).any(1, keepdim=True), y, 0.0)
    out = out.to(torch.bfloat16)
    return (out, idx, wt) if c["router"] else out


def run(state):
    s, c = state, state["case"]
    if own:
        import combine_moe_route_softmax_gb300 as moe
        if c["op"] == "linear":
            return moe.moe_linear_w4(s["x"], s["packed"], bias=s["bias"],
                                     out_dtype=torch.float32 if c["f32"] else torch.bfloat16, ws=s["ws"])
        if c["op"] == "route":
            return moe.moe_route_hidden(s["x"], s["w_router"], c["K"], bias=s["bias"], ws=s["ws"])
        if c["router"]:
            return s["layer"].forward(s["x"])
        return s["layer"].forward(s["x"], topk_idx=s["topk_idx"], topk_w=s["topk_w"])[0]
    return {"linear": _plain_linear, "route": _plain_route, "layer": _plain_layer}[c["op"]](c, s)


# -------------------------------------------------------------------------------------- work
def _matrix_bytes(c, n, k):
    if c["dtype"] == "w4":
        return n * k // 2 + n * (k // c["group"]) * (3 if c["zeros"] else 2)
    return n * k + n * k // 4096 if c["dtype"] == "e4m3" else 2 * n * k


def _weight_bytes(c):
    return _matrix_bytes(c, 2 * c["I"], c["H"]) + _matrix_bytes(c, c["H"], c["I"])


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "linear":
        b = _matrix_bytes({"dtype": "w4", **c}, c["N"], c["K"]) + T * c["K"] * 2 + T * c["N"] * (4 if c["f32"] else 2)
        return {"bytes": b + (4 * c["N"] if c["bias"] else 0), "flops": 2 * T * c["N"] * c["K"]}
    H, E, K = c["H"], c["E"], c["K"]
    route = {"bytes": 2 * E * H + 2 * T * H + 4 * T * E + 8 * T * K, "flops": 2 * T * E * H}
    if c["op"] == "route":
        return route
    # the experts that T tokens with K valid distinct choices of E meet, on average
    met = E * (1 - (1 - K * (1 - c["pad"]) / E) ** T) + (1 if c["shared"] else 0)
    rows = T * K * (1 - c["pad"]) + (T if c["shared"] else 0)
    b = met * _weight_bytes(c) + 4 * T * H + (2 * E * H if c["router"] else 0) + 8 * T * K
    return {"bytes": int(b), "flops": int(6 * rows * H * c["I"] + (2 * T * E * H if c["router"] else 0))}


# ------------------------------------------------------------------------- exact (64 bits)
def _matrix64(c, w, e):
    """Matrix e of a weight set in float64, from the definition of its format."""
    v = w["w"][e]
    if c["dtype"] == "bf16":
        return v.double()
    if c["dtype"] == "e4m3":
        sign = torch.where(v >= 128, -1.0, 1.0).double()
        ex, man = ((v >> 3) & 15).double(), (v & 7).double()
        val = sign * torch.where(ex > 0, torch.exp2(ex - 7) * (1 + man / 8), man * 2.0 ** -9)
        up = w["scales"][e].double()
        return val * up.repeat_interleave(128, 0).repeat_interleave(128, 1)
    n, kh = v.shape
    code = torch.empty(n, 2 * kh, dtype=torch.float64, device=v.device)
    code[:, 0::2] = (v % 16).double()
    code[:, 1::2] = (v // 16).double()
    s = w["scales"][e].double().T
    rep = 2 * kh // s.shape[1]
    z = 8.0 if w["zeros"] is None else w["zeros"][e].double().T.repeat_interleave(rep, 1)
    return (code - z) * s.repeat_interleave(rep, 1)


def _swiglu64(x, a, b):
    z = x @ a.T
    half = z.shape[1] // 2
    return (z[:, half:] * z[:, :half] * torch.sigmoid(z[:, :half])) @ b.T


def exact(case, seed):
    c = dict(case)
    s = _inputs(c, seed)
    if c["op"] == "linear":
        w = {k: None if s[j] is None else s[j][None] for k, j in (("w", "q"), ("scales", "scales"), ("zeros", "zeros"))}
        y = s["x"].double() @ _matrix64({"dtype": "w4"}, w, 0).T
        return y if s["bias"] is None else y + s["bias"].double()
    x = s["x"].double()
    T, K = c["T"], c["K"]
    if "w_router" in s:
        z = (x[:, None, :] * s["w_router"].double()[None]).sum(2)
        if s.get("bias") is not None:
            z = z + s["bias"].double()
        order = torch.argsort(-z, dim=1, stable=True)[:, :K]
        wt = torch.softmax(torch.gather(z, 1, order), 1)
        if c["op"] == "route":
            return order.to(torch.int32), wt, z
    else:
        order, wt = s["topk_idx"].long(), s["topk_w"].double()
    out = torch.zeros(T, c["H"], dtype=torch.float64, device=x.device)
    for e in sorted(set(order.flatten().tolist()) - {-1}):
        t, k = (order == e).nonzero(as_tuple=True)
        y = _swiglu64(x[t], _matrix64(c, s["w13"], e), _matrix64(c, s["w2"], e))
        out.index_add_(0, t, y * wt[t, k].unsqueeze(1))
    if c["shared"]:
        some = (order >= 0).any(1)
        out[some] += _swiglu64(x[some], _matrix64(c, s["s13"], 0), _matrix64(c, s["s2"], 0))
    return (out, order.to(torch.int32), wt) if c["router"] else out
