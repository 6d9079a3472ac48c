"""The average bounds of few_bounds on the CPU: a plain float32 layer or product passes them at every
size that the GPU tests run, and one with a mistake planted in it does not."""
import pytest
import torch

import few_bounds as bounds
from test_gpu_few import LAYER, LINEAR


def matrix(g, n, k):
    return (torch.randn(n, k, generator=g) * k ** -0.5).to(torch.bfloat16).float()


def two_terms(h, half):
    """h as the kernels keep it: BF16 hi + lo, or FP16 of 16 values scaled to their largest."""
    if not half:
        hi = h.to(torch.bfloat16).float()
        return hi + (h - hi).to(torch.bfloat16).float()
    b = h.view(h.shape[0], -1, 16)
    sc = torch.exp2(14 - torch.floor(torch.log2(b.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100))))
    hi = (b * sc).half().float()
    return ((hi + (b * sc - hi).half().float()) / sc).view(h.shape)


def one_term(h, half):
    if not half:
        return h.to(torch.bfloat16).float()
    b = h.view(h.shape[0], -1, 16)
    sc = torch.exp2(14 - torch.floor(torch.log2(b.abs().amax(2, keepdim=True).clamp(min=2.0 ** -100))))
    return ((b * sc).half().float() / sc).view(h.shape)


def fp8(w):
    s = w.abs().amax() / 448
    return (w / s).to(torch.float8_e4m3fn).float() * s


class Plain:
    """The layer in float32; each planted mistake is one of its methods' replacements."""

    def __init__(self, half):
        self.half = half
        self.terms = two_terms

    def w13(self, w):
        return w

    def w2(self, w):
        return w

    def expert(self, x, w13, w2):
        z = x @ self.w13(w13).T
        i = z.shape[1] // 2
        h = z[:, :i] / (1 + torch.exp(-z[:, :i])) * z[:, i:]
        return self.terms(h, self.half) @ self.w2(w2).T


def without(lo, n):
    def cut(w):
        w = w.clone()
        w[:, lo:lo + n] = 0
        return w
    return cut


MISTAKES = {
    "w13_32_columns": ("w13", without(32, 32)),
    "w2_32_columns": ("w2", without(0, 32)),
    "w13_item": ("w13", lambda w: without(w.shape[1] - 64, 64)(w)),
    "w13_fp8": ("w13", fp8),
    "w2_fp8": ("w2", fp8),
}


@pytest.mark.parametrize("case", LAYER, ids=lambda c: "x".join(str(v) for v in c[:6]))
def test_layer_bound(case):
    T, H, I, E, K, dtype, shared = case[:7]
    half = dtype != "bf16"
    g = torch.Generator().manual_seed(T + H + E)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).float()
    # one expert per slot of a token is enough for the sums; every row goes through each
    ex = [(matrix(g, 2 * I, H), matrix(g, H, I)) for _ in range(min(K, 2) + shared)]
    wt = torch.rand(T, len(ex), generator=g)

    def out(layer, dt):
        y = sum(wt[:, k, None].to(dt) * layer.expert(x.to(dt), a.to(dt), b.to(dt)) for k, (a, b) in enumerate(ex))
        return y if dt == torch.float64 else y.to(torch.bfloat16)
    exact = Plain(half)
    exact.terms = lambda h, half: h
    want = out(exact, torch.float64)
    assert bounds.layer_ratio(out(Plain(half), torch.float32), want, half) <= 1
    for name, (at, mistake) in MISTAKES.items():
        bad = Plain(half)
        setattr(bad, at, mistake)
        assert bounds.layer_ratio(out(bad, torch.float32), want, half) > 2, name
    if T * H >= 4096 or not half:
        bad = Plain(half)
        bad.terms = one_term
        assert bounds.layer_ratio(out(bad, torch.float32), want, half) > 1.2, "h in one term"


@pytest.mark.parametrize("case", LINEAR, ids=lambda c: "x".join(str(v) for v in c[:4]))
def test_linear_bound(case):
    T, N, K, group, _, _, f32 = case
    g = torch.Generator().manual_seed(T * N)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).float()
    w = matrix(g, N, K)
    want = x.double() @ w.double().T
    dt = torch.float32 if f32 else torch.bfloat16
    ratio = lambda y: bounds.linear_ratio(y.to(dt), want, K)
    assert ratio(x @ w.T) <= 1
    assert ratio(x @ without(8, 8)(w).T) > 2
    assert ratio(x @ without(0, min(group, K // 2))(w).T) > 2
    assert ratio(x @ fp8(w).T) > 2
    if f32:
        assert ratio((x @ w.T).to(torch.bfloat16)) > 2
        assert ratio((x @ w.T).half()) > 2
