"""How far the few-token operators' outputs may be off on average, as fractions of the outputs' own
size: bounds that fail when a term, a column or a unit of a sum is missing, beside the worst-case
ones of few_ref.

An output is the correctly rounded 64-bit value unless the error before its rounding carries it over
a midpoint, so over many outputs the mean of |output - correctly rounded value| is the mean of that
error.  The error counted, for rows of random signs (a partial sum is no larger than the sum's
own typical size):
  sums      a float32 accumulator takes at most 64 tensor instructions (8 items of 4, two terms) before
            it is joined, each off by at most one step (2^-23) of the running sum; scale groups and
            joins round to nearest, off by the root of their number;
  h         silu(g) u: at most three times the sums' error, silu and the product 2^-20, and what
            its two terms leave: 2^-17 (BF16) or 2^-22 (FP16)."""
import torch

STEP = 2.0 ** -23


def spacing(v):
    """Distance from the BF16 values v to the next larger magnitude."""
    return torch.nextafter(v.abs(), torch.full_like(v, float("inf"))).double() - v.abs().double()


def mean_moved(got, want):
    """(mean |got - correctly rounded want| over the size of want, what one output in doubt adds)."""
    rn = want.to(got.dtype)
    size = want.square().mean().sqrt().clamp(min=1e-300)
    d = (got.double() - rn.double()).abs().mean() / size
    return d.item(), (spacing(rn).mean() / size).item()


def sampled(bound, one, n):
    """The bound on a mean of n outputs whose true mean is `bound`: four deviations, and four outputs."""
    return bound + 4 * (bound * one / n) ** 0.5 + 4 * one / n


def layer_bound(half):
    return 4 * 64 * STEP + 2.0 ** -20 + (2.0 ** -22 if half else 2.0 ** -17)


def linear_bound(K):
    return (8 + 2 * (K / 32) ** 0.5) * STEP


def layer_ratio(got, want, half):
    """At most 1 for a correct layer output (BF16) of random inputs; rows of padding (0) left out."""
    rows = want.abs().amax(1) > 0
    got, want = got[rows], want[rows]
    d, one = mean_moved(got, want)
    return d / sampled(layer_bound(half), one, want.numel())


def linear_ratio(got, want, K):
    if got.dtype == torch.float32:
        return ((got.double() - want).square().mean() / want.square().mean()).sqrt().item() / (linear_bound(K) + 2.0 ** -24)
    d, one = mean_moved(got, want)
    return d / sampled(linear_bound(K), one, want.numel())
