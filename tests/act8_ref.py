"""Plain 64-bit forms of the 8-bit activation path's operators, with the error that a correct kernel may make
on each output.  No code shared with the library.

Roundings counted, each half a step (finfo.eps / 2 of the value: float32 2^-24, BF16 2^-8, E4M3 2^-4 or half of
its smallest step 2^-9):
* norm: h is one sum; a sum of H squares in any order in which a value takes part in at most 64 + 16 additions
  (64 columns in a thread, then a tree) is off by 80 of them, and r by half of that and 4 of its own; y has two
  products more.  Together at most 48 of |y|.
* linear: products of E4M3 values are exact in float32; a block of 128 is at most 128 additions, counted as a whole
  step (2^-23) each because a tensor core cuts instead of rounding; then one product of the scales, one fused
  addition per block, at most 64 additions where shares are joined, and the bias."""
import torch

F32 = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def e4m3_values(q):
    """uint8 codes -> float64, from the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    q = q.view(torch.uint8).long()
    sign = torch.where(q >= 128, -1.0, 1.0).double()
    e, m = (q // 8 % 16).double(), (q % 8).double()
    v = sign * torch.where(e > 0, torch.exp2(e - 7) * (1 + m / 8), m * 2.0 ** -9)
    return torch.where(q % 128 == 127, torch.nan, v)


def norm(x, weight, eps, residual=None):
    """(y, h) in float64."""
    h = x.double() + (0.0 if residual is None else residual.double())
    r = 1.0 / torch.sqrt(h.square().mean(1, keepdim=True) + eps)
    return h * r * weight.double(), h


NORM_ERR = 48 * F32      # of |y|


def block_scales(y):
    s = y.abs().view(y.shape[0], y.shape[1] // 128, 128).amax(2) / 448
    return torch.where(s > 0, s, 1.0)


def code_bounds(y, slack):
    """The smallest and largest E4M3 magnitude that |y| / scale may have become, each within `slack` of it."""
    v = (y.view(y.shape[0], y.shape[1] // 128, 128).abs() / block_scales(y).unsqueeze(2)).view(y.shape)
    near = lambda u: u.clamp(max=448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
    return near(v * (1 - slack)), near(v * (1 + slack))


def linear(x, xs, w, ws, bias=None):
    """(out, allowed error before the output's rounding) of E4M3 codes with their scales."""
    T, K = x.shape
    N = w.shape[0]
    up = ws.double().repeat_interleave(128, 0)[:N]
    a, b = e4m3_values(x).view(T, K // 128, 128), e4m3_values(w).view(N, K // 128, 128)
    a, b = (a * xs.double().unsqueeze(2)).view(T, K), (b * up.unsqueeze(2)).view(N, K)
    y, size = a @ b.T, a.abs() @ b.abs().T
    err = size * (128 * 2.0 ** -23 + (K // 128 + 64 + 1) * F32)
    if bias is not None:
        y = y + bias.double()
        err = err + F32 * (y.abs() + size)
    return y, err


def permute(idx, E, shared, max_tokens=0):
    """Rows of the expert-major layout, filled segment by segment: dict(token [rows] (-1: no row), src, inv, smap,
    and cu, or counts for the batched layout, with what was dropped)."""
    T, K = idx.shape
    idx = idx.tolist()
    segs = [[] for _ in range(E + int(shared))]
    for t in range(T):
        for k in range(K):
            if 0 <= idx[t][k] < E:
                segs[idx[t][k]].append((t, t * K + k))
    if shared:
        for t in range(T):
            if any(0 <= e < E for e in idx[t]):
                segs[E].append((t, T * K + t))
    rows = len(segs) * max_tokens if max_tokens else T * K + (T if shared else 0)
    token, src, inv = [-1] * rows, [-1] * rows, [-1] * (T * K + T)
    cu, at = [0], 0
    for i, s in enumerate(segs):
        kept = s[:max_tokens] if max_tokens else s
        p = i * max_tokens if max_tokens else at
        for j, (t, slot) in enumerate(kept):
            token[p + j], src[p + j], inv[slot] = t, slot, p + j
        at += len(kept)
        cu.append(at)
    return dict(token=torch.tensor(token), src=torch.tensor(src), inv=torch.tensor(inv[:T * K]).view(T, K),
                smap=torch.tensor(inv[T * K:]), cu=torch.tensor(cu), counts=torch.tensor([b - a for a, b in zip(cu, cu[1:])]))
