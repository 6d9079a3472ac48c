"""Plain 64-bit forms of the few-token operators, with the error that a correct kernel may
make on each output.  No code shared with the library.

Rounding counted: one rounding to the output's type (half a step, finfo.eps / 2 of the value);
float32 sums on the tensor cores, at most one step (2^-23) of the largest partial sum per
tensor instruction and per scale group -- a partial sum is at most |row| * |column|
(Cauchy-Schwarz) and a row of k columns takes at most k/8 of them; silu and the
product, 2^-20 of h; h as two BF16 terms, 2^-16 of h, or as one FP16 term whose block of 16
is scaled to its largest value, half a step (2^-11) of h and 2^-25 of the slot's largest; the
combine, one float32 step per slot."""
import torch

STEP = 2.0 ** -23


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def unpack_codes(q):
    """uint8 [..., k/2] -> float64 codes [..., k]: the even column in the low nibble."""
    out = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    out[..., 0::2] = (q % 16).double()
    out[..., 1::2] = (q // 16).double()
    return out


def w4_values(q, scales, zeros=None):
    """[n, k] float64 of one matrix from codes [n, k/2], scales (and zeros) [k/group, n]."""
    c = unpack_codes(q)
    g = c.shape[-1] // scales.shape[0]
    s = scales.double().T.repeat_interleave(g, 1)
    z = 8.0 if zeros is None else zeros.double().T.repeat_interleave(g, 1)
    return (c - z) * s


def e4m3_values(q, scales):
    sign = torch.where(q >= 128, -1.0, 1.0).double()
    ex, man = (q // 8 % 16).double(), (q % 8).double()
    v = sign * torch.where(ex > 0, torch.exp2(ex - 7) * (1 + man / 8), man * 2.0 ** -9)
    return v * scales.double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def linear(x, w, bias=None):
    """(y, allowed error before the output rounding) of y = x w^T + bias."""
    x = x.double()
    y = x @ w.T
    err = w.shape[1] / 8 * STEP * x.norm(dim=1)[:, None] * w.norm(dim=1)[None]
    if bias is not None:
        y = y + bias.double()
        err = err + STEP * (y.abs() + bias.double().abs())
    return y, err


def swiglu(x, w13, w2, half=False):
    """(y, allowed error) of one expert for rows x; half: h as one FP16 term."""
    x = x.double()
    i = w13.shape[0] // 2
    z, dz = linear(x, w13)
    g, u = z[:, :i], z[:, i:]
    silu = g * torch.sigmoid(g)
    h = silu * u
    dh = 1.1 * u.abs() * dz[:, :i] + silu.abs() * dz[:, i:] + 1.1 * dz[:, :i] * dz[:, i:] + h.abs() * ((2.0 ** -11 if half else 2.0 ** -16) + 2.0 ** -20)
    if half:
        dh = dh + 2.0 ** -25 * h.abs().amax(1, keepdim=True)
    y, dy = linear(h, w2)
    return y, dy + dh @ w2.abs().T


def layer(x, idx, wt, w13, w2, shared=None, half=False):
    """(out, allowed error) [T, H]; w13(e), w2(e) give an expert's float64 matrices, shared is a pair."""
    T, K = idx.shape
    H = x.shape[1]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    size = torch.zeros_like(out)
    for e in sorted(set(idx.flatten().tolist()) - {-1}):
        t, k = (idx == e).nonzero(as_tuple=True)
        y, d = swiglu(x[t], w13(e), w2(e), half)
        w = wt[t, k].double().unsqueeze(1)
        out.index_add_(0, t, w * y)
        err.index_add_(0, t, w.abs() * d)
        size.index_add_(0, t, (w * y).abs())
    if shared is not None:
        some = (idx >= 0).any(1)
        y, d = swiglu(x[some], *shared, half)
        out[some] += y
        err[some] += d
        size[some] += y.abs()
    return out, err + (K + 2) * STEP * size


def close(got, want, err):
    """Worst ratio of |got - want| to the allowed error (at most 1 for a correct kernel)."""
    tol = err + half_step(got.dtype) * want.abs() * (1 + 2.0 ** -6) + half_step(got.dtype) * err
    return ((got.double() - want).abs() / tol.clamp(min=1e-300)).max().item()


def route(x, w_router, bias, K):
    """(ids int32, weights float64, logits float64): float32-rounded logits decide, ties to the lower id."""
    z = x.double() @ w_router.double().T
    if bias is not None:
        z = z + bias.double()
    order = torch.sort(z.float(), dim=1, descending=True, stable=True)[1][:, :K]
    return order.to(torch.int32), torch.softmax(torch.gather(z, 1, order), 1), z


def pack_w4(q, scales, zeros=None):
    """moe_pack_w4 of one matrix, from the layout's definition: numpy uint8 bytes."""
    import numpy as np
    N, K = q.shape[0], 2 * q.shape[1]
    group = K // scales.shape[0]
    N32, K256, ng = (N + 31) // 32 * 32, (K + 255) // 256 * 256, 256 // group
    code = np.zeros((N32, K256), np.uint32)
    code[:N, 0:K:2] = q & 15
    code[:N, 1:K:2] = q >> 4
    nsl, nrb = K256 // 256, N32 // 16
    oq = np.zeros((nrb, nsl, 2, 2, 8, 4, 4), np.uint32)      # [row block][slice][half][J][g][t][word]
    for h in range(2):
        for j in range(8):
            for g in range(8):
                for t in range(4):
                    for i in range(8):
                        nib = i // 2 + 4 * (i % 2)
                        oq[:, :, h, j // 4, g, t, j % 4] |= code[h * 8 + g::16, j * 32 + t * 8 + i::256] << (4 * nib)

    def params(p, dt):
        full = np.zeros((K256 // group, N32), dt)
        full[:K // group, :N] = p
        # [slice][group][row block][half][g] -> [row block][slice][g][group][half]
        v = np.ascontiguousarray(full.reshape(nsl, ng, nrb, 2, 8).transpose(2, 0, 4, 1, 3))
        return v.reshape(nrb, nsl, -1).view(np.uint8)
    parts = [oq.reshape(nrb, nsl, -1).view(np.uint8), params(scales, np.uint16)]
    if zeros is not None:
        parts.append(params(zeros, np.uint8))
    return np.concatenate(parts, axis=2).reshape(-1)


def quantize_w4(w, group, with_zeros):
    """moe_quantize_weight_w4 of one BF16 matrix given as float32 numpy [rows, cols]: (codes,
    scales as uint16 BF16 bits, zeros or None), float32 steps as documented."""
    import numpy as np
    from oracle.formats import bf16_bits_to_f32, f32_to_bf16_bits
    f = np.float32
    R, C = w.shape
    b = w.reshape(R, C // group, group)
    lo, hi = np.minimum(b.min(2), f(0)), np.maximum(b.max(2), f(0))
    raw = (hi - lo) / f(15) if with_zeros else np.maximum(hi, -lo) / f(7)
    sb = f32_to_bf16_bits(raw.astype(f))
    s = bf16_bits_to_f32(sb)
    sb = np.where(s > 0, sb, np.uint16(0x3F80)).astype(np.uint16)
    s = bf16_bits_to_f32(sb)
    z = np.clip(np.rint(-lo / s), 0, 15).astype(f) if with_zeros else np.full_like(s, 8)
    c = np.clip(np.rint(b / s[..., None]) + z[..., None], 0, 15).astype(np.uint8).reshape(R, C)
    return (c[:, 0::2] | c[:, 1::2] << 4).astype(np.uint8), sb.T.copy(), z.astype(np.uint8).T.copy() if with_zeros else None
