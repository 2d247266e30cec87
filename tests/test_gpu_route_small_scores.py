"""moe_route's renormalised sigmoids where fp32 has few bits of the scores, or none."""
import numpy as np
import pytest
import torch

from tests.test_gpu_route import TYPES, bias_of, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [5, 8197])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("level", [-30.0, -41.0, -45.0, -80.0, -95.0, -102.0, -104.0, -150.0, -400.0, -700.0])
def test_shares_of_small_scores(lib, T, dtype, bias, level):
    E, k, n = 64, 6, 23
    g = torch.Generator(device="cuda").manual_seed(int(-level))
    z = (level - 6.0 * torch.rand((n, E), generator=g, device="cuda")).to(TYPES[dtype])
    z[1, 10:] = -float("inf")
    z[2, 3:] = -float("inf")                          # fewer than k
    z[3] = -float("inf")
    z[4] = torch.finfo(TYPES[dtype]).min              # scores that are 0 in 64 bits: weights 0
    z[5, 5:] = torch.finfo(TYPES[dtype]).min
    z[6, 7] = 1.0                                     # one that takes all
    z[7] = z[7, 0]
    if dtype == "f16":
        z[4], z[5, 5:] = -60000.0, -60000.0
    b = bias_of(E) if bias else None
    big = z.repeat(-(-T // n), 1)[:T].contiguous()
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    lib.moe_route(big, ids, w, bias=b, scale=2.5, flags=lib.MOE_ROUTE_RENORM)
    ids, w = ids.cpu().numpy(), w.double().cpu().numpy()
    rows, b = z.double().cpu().numpy(), None if b is None else b.double().cpu().numpy()
    for t in range(T):
        if t >= n:
            assert (ids[t] == ids[t - n]).all() and (w[t] == w[t - n]).all()
            continue
        # 64-bit scores: subnormal below -708, of which -706 at the lowest here has all bits
        want, weight = plain(rows[t], k, b, scale=2.5, renorm=True)
        assert (ids[t] == want).all(), (t, ids[t], want)
        # exp within 2 units of 2^-24, its argument (a difference of at most 8) rounded to 2^-22, a sum of k
        # terms, a division and the scale of half a unit each: under 32 units.  Weights of a term beside a much
        # larger one (row 6) are at most e^-30, off by their whole size at most where they are subnormal.
        assert (np.abs(w[t] - weight) <= 32 * 2.0 ** -24 * np.abs(weight) + 2.0 ** -120).all(), (t, w[t], weight)


@pytest.mark.parametrize("T", [5, 8197])
@pytest.mark.parametrize("level", [-15.0, -18.0, -22.0, -30.0, -40.0, -60.0, -200.0])
def test_small_scores_beside_much_smaller_ones(lib, T, level):
    E, k, n = 128, 8, 29
    g = torch.Generator(device="cuda").manual_seed(int(-level))
    z = level - 75.0 * torch.rand((n, E), generator=g, device="cuda") ** 0.1        # most of them far below
    z[:, ::16] = level - 9.0 * torch.rand((n, E // 16), generator=g, device="cuda")
    z[:, 1::32] = -float("inf")
    b = torch.zeros(E, device="cuda")
    b[5:9] = 1.0                                      # chosen for their biases, whatever their scores
    big = z.repeat(-(-T // n), 1)[:T].contiguous()
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    lib.moe_route(big, ids, w, bias=b, flags=lib.MOE_ROUTE_RENORM)
    rows, b = z.double().cpu().numpy(), b.double().cpu().numpy()
    for t in range(min(n, T)):
        want, weight = plain(rows[t], k, b, renorm=True)
        assert (ids[t].cpu().numpy() == want).all()
        # as above, with arguments of up to 75 that are rounded to half of 2^-17; beside scores of 2^-30 and
        # above the smallest ones are subnormal, to 2^-149 / 2^-30
        tol = (32 + 64) * 2.0 ** -24 * np.abs(weight) + 2.0 ** -118
        assert (np.abs(w[t].double().cpu().numpy() - weight) <= tol).all(), (t, w[t], weight)
