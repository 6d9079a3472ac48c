"""The norm's codes bit for bit.  With eps = 2^40 and a mean square below 2^15, less than half a step of eps, the root is 2^20
and r = 2^-20 exactly whatever the order of the sum, so that the float32 y = (h r) w is known, and with it the scales and codes:
IEEE divisions and the E4M3 rounding of the oracle."""
import numpy as np
import pytest
import torch

import combine_moe_route_softmax_gb300 as moe
from gpu_helpers import host, need_gpu
from oracle import moe_ref as ref

pytestmark = pytest.mark.gpu
EPS = 2.0 ** 40


def check(x, w):
    q, s = moe.moe_rmsnorm(x, w, EPS, bf16=False, e4m3=True)[1:3]
    h = host(x.float())
    with np.errstate(all="ignore"):
        y = (h * np.float32(2.0 ** -20)) * host(w)
        want_q, want_s = ref.act_quant_1x128(y)
    assert np.array_equal(host(s), want_s)
    assert np.array_equal(host(q), want_q)
    return y, want_q, want_s


# weights that put a block's scale on both sides of 8e-25 and 1e24, and into the subnormals
@pytest.mark.parametrize("unit", [1.0, 0.77, 1e-9, 2.1e-16, 1.9e-17, 1.3e-18, 1e-25, 1e-31, 1e-33, 1e9, 3e28, 4e30, 1.7e31, 1e33])
@pytest.mark.parametrize("T,H", [(3, 512), (700, 1024), (5, 8320)])
def test_codes_are_the_rounded_quotients(unit, T, H):
    need_gpu()
    g = torch.Generator(device="cuda").manual_seed(H)
    x = torch.randn(T, H, generator=g, device="cuda") * torch.exp2(torch.randint(-12, 7, (T, H), generator=g, device="cuda").float())
    x[torch.rand(T, H, generator=g, device="cuda") < 0.05] = 0.0
    x[torch.rand(T, H, generator=g, device="cuda") < 0.05] = -0.0
    x[:, 128:256] = -0.0                       # a block of nothing but zeros: scale 1
    w = (torch.rand(H, generator=g, device="cuda") + 0.5) * unit
    w[torch.rand(H, generator=g, device="cuda") < 0.3] *= -1
    w[5], w[9] = 0.0, -0.0
    y, q, s = check(x.to(torch.bfloat16), w)
    assert (q == 0x80).any() and (s[:, 1] == 1).all() and np.isfinite(s).all()


def test_quotients_on_the_codes_borders():
    """Values within a step of the middle between two codes, where a quotient that is off by a unit in its last place shows."""
    need_gpu()
    codes = np.arange(0, 0x7f, dtype=np.uint8)
    from oracle.formats import e4m3_decode64
    v = e4m3_decode64(codes)
    mid = ((v[1:] + v[:-1]) / 2)[:126]
    for amax in (448.0, 447.0, 300.0, 257.0, 1.0 + 2.0 ** -7, 1.3359375):
        s = np.float32(np.float32(amax) / np.float32(448))
        y = (mid * np.float64(s)).astype(np.float32)
        w = np.concatenate([np.nextafter(y, np.float32(d)) for d in (-1, 1e9)] + [y] + [-y])
        w = np.concatenate([np.append(b, np.full(128 - len(b), amax, np.float32)) for b in np.split(w, 4)]).astype(np.float32)
        assert w.size == 512
        check(torch.ones(2, 512, dtype=torch.bfloat16, device="cuda"), torch.from_numpy(w * np.float32(2.0 ** 20)).cuda())
