"""How far moe_gate's logits are off, over many of them: what its sums over 512 columns are for."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H, COLUMNS, STEP = 7168, 512, 16


def bounds():
    """(rms, mean towards zero) of the error of a logit of N(0, 1), by arithmetic.

    A sum over 512 columns is 32 steps of 16 products, and after j of them it has a standard deviation of
    sqrt(16 j / H).  A step that cuts to 24 bits loses less than 2^-23 of the sum's size, whose mean is sqrt(2 / pi) of
    that deviation: in all less than `run`, towards the sum's zero.  The 14 sums of a logit have the signs of independent
    numbers: their losses add up by their squares (a loss's mean square is at most pi / 2 times its squared mean), and in
    the direction of the logit itself by the 2 / pi * asin(14^-1/2) that a part's sign has in common with the whole's.
    To these come the fp32 additions of the 14 sums (half a unit of 2^-23 each, of a sum of at most 1 on average).
    Summed over all columns at once, the same arithmetic loses 448 steps' worth, 16 times a run's at a loss of half a unit
    a step: 1e-5, all of it towards zero."""
    n = H // COLUMNS
    run = sum(math.sqrt(2 / math.pi) * math.sqrt(STEP * j / H) * 2.0 ** -23 for j in range(1, COLUMNS // STEP + 1))
    added = math.sqrt(n) * 2.0 ** -24
    return math.sqrt(n * math.pi / 2) * run + added, n * 2 / math.pi * math.asin(n ** -0.5) * run + added


def test_the_bounds_lie_between_the_two_ways_to_sum():
    rms, towards_zero = bounds()
    whole = sum(0.36 * math.sqrt(2 / math.pi) * math.sqrt(STEP * j / H) * 2.0 ** -23 for j in range(1, H // STEP + 1))
    assert 2 * rms < whole and 4 * towards_zero < whole


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E", [(1, 1024), (16, 1024), (17, 1024), (64, 512), (256, 256), (1024, 256), (1024, 64), (16384, 256)])
def test_errors_of_many_logits(lib, T, E, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    w = (torch.randn((E, H), generator=g, device="cuda") * H ** -0.5).to(dtype)
    got = lib.moe_gate(x, w, torch.empty((T, E), device="cuda")).double()
    want = torch.cat([part.double() @ w.double().T for part in x.split(2048)])
    off, size = got - want, want.square().mean().sqrt().item()
    rms, towards_zero = bounds()
    # a thousand logits at the least: the figures of a sample are within 5 / sqrt(n) of their own
    spread = 1 + 5 / math.sqrt(T * E)
    assert off.square().mean().sqrt().item() <= rms * size * spread
    assert abs((off * want.sign()).mean().item()) <= towards_zero * size + 5 * rms * size / math.sqrt(T * E)
