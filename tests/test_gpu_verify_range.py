"""moe_verify_drafts of rows whose weights sum to far more or less than 1: they count relative to their sum."""
import pytest
import torch

from tests.test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V", [300, 33001, 140001])
@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** -95, 2.0 ** -110, 2.0 ** -118, 2.0 ** 100, 2.0 ** 126])
def test_rows_whose_sum_is_far_from_one(lib, V, with_q, factor):
    """Weights are relative to their sum, at the ends of fp32 too; sums of finite entries may pass fp32's largest."""
    b = Batch([1, 0, 1, 1, 0, 2], V, with_q=with_q, seed=V)
    b.p = b.p * 2.0 ** 7 if factor > 1 else (b.p * 2.0 ** 24).round() * 2.0 ** -24      # multiples of what fp32 has left
    if with_q:
        b.q = b.q * 2.0 ** 7 if factor > 1 else (b.q * 2.0 ** 24).round() * 2.0 ** -24
        b.q *= factor
    b.p *= factor
    b.p.clamp_(max=3e38)
    if with_q:
        b.q.clamp_(max=3e38)
    if factor == 2.0 ** 126:
        b.p[:, 10:30] = 3e38                               # their sum is not a finite fp32
    b.ua[::2] = 1e30
    b.check(lib)


def test_sums_past_the_largest_number_with_infinities_among_them(lib):
    b = Batch([0, 1, 0], 5000, seed=5)
    b.p[:, ::7] = 2e38
    b.p[:, 100] = float("inf")
    b.q[:, ::7] = 1e38
    b.ua[:] = 1e30
    b.check(lib)


@pytest.mark.parametrize("V", [40, 9000, 128000])
@pytest.mark.parametrize("unit", [2.0 ** -149, 2.0 ** -140, 2.0 ** -127, 2.0 ** -100])
def test_rows_of_few_units(lib, V, unit):
    """Three entries of a unit, down to fp32's smallest: a third of the random numbers each."""
    n = 24
    b = Batch([0] * n, V, seed=1)
    b.p.zero_()
    b.p[:, [3, V // 2, V - 1]] = unit
    b.us = (torch.arange(n, device="cuda") + 0.5) / n
    _, out = b.check(lib)
    assert [o[0] for o in out] == [3] * 8 + [V // 2] * 8 + [V - 1] * 8


def test_residuals_of_small_numbers(lib):
    b = Batch([1] * 12, 5000, seed=2)
    b.ua[:] = 1e30
    b.tokens[:] = 7
    b.p = (b.p * 2.0 ** 20).round() * 2.0 ** -20 + 2.0 ** -20
    b.q = b.p.clone()
    b.p *= 2.0 ** -126
    b.q *= 2.0 ** -126
    b.q[:, 100::500] -= 2.0 ** -146                         # the residual: 2^-146 at ten places
    b.us = (torch.arange(12, device="cuda") + 0.5) / 12
    b.check(lib)
