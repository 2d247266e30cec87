"""moe_route of many tokens, which a warp routes several at a time, against a plain 64-bit routing."""
import numpy as np
import pytest
import torch

from tests.test_gpu_route import TYPES, bias_of, logits_of, plain

pytestmark = pytest.mark.gpu

MANY = 8195          # an odd number, more than a warp a token is for


def check(lib, logits, k, bias=None, n_group=1, topk_group=1, scale=1.0, flags=0, n_tokens=None, T=MANY):
    """The rows of `logits` over and over, T in all, as they lie (strides, alignment)."""
    n, E = logits.shape
    ld = logits.stride(0)
    big = torch.full((T, ld), 5.0, dtype=logits.dtype, device="cuda")[:, :E]
    big.copy_(logits.repeat(-(-T // n), 1)[:T])
    ids = torch.full((T, k + 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k + 1), 77.0, device="cuda")
    count = None if n_tokens is None else torch.tensor([n_tokens], dtype=torch.int32, device="cuda")
    lib.moe_route(big, ids[:, :k], w[:, :k], bias=bias, n_group=n_group, topk_group=topk_group, scale=scale, flags=flags, n_tokens=count)
    assert (ids[:, k:] == 77).all() and (w[:, k:] == 77.0).all()
    ids, w = ids[:, :k].cpu().numpy(), w[:, :k].double().cpu().numpy()
    live = T if n_tokens is None else max(0, min(n_tokens, T))
    assert (ids[live:] == -1).all() and (w[live:] == 0).all()
    # the same row gives the same answer wherever it stands
    for a in (ids, w):
        assert (a[n:live] == a[: max(0, live - n)]).all()
    softmax, renorm, pair = (bool(flags & f) for f in (lib.MOE_ROUTE_SOFTMAX, lib.MOE_ROUTE_RENORM, lib.MOE_ROUTE_GROUP_PAIR))
    z, b = logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy()
    for t in range(min(n, live)):
        want, weight = plain(z[t], k, b, n_group, topk_group, scale, softmax, renorm, pair)
        assert (ids[t] == want).all(), (t, ids[t], want)
        # as for few tokens: exp within 2 units of 2^-24 (and its argument z - max rounded), sums of E and k
        # terms and divisions of half a unit each; what fp32 has as subnormals, to 2^-140
        fin = z[t][np.isfinite(z[t])]
        spread = float(fin.max() - fin.min()) if softmax and len(fin) else 0.0
        tol = 2.0 ** -24 * (24 + min(spread, 200.0))
        assert (np.abs(w[t] - weight) <= tol * np.abs(weight) + 2.0 ** -120 * max(1.0, abs(scale))).all(), (t, w[t], weight)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,k,n_group,topk_group", [
    (8, 1, 1, 1), (8, 8, 1, 1), (32, 4, 1, 1), (40, 8, 1, 1), (64, 6, 1, 1), (64, 8, 8, 7), (64, 2, 4, 1), (64, 5, 2, 1), (72, 7, 1, 1),
    (96, 8, 3, 2), (128, 8, 4, 2), (128, 8, 8, 5), (128, 1, 8, 1), (160, 6, 1, 1), (160, 6, 5, 4), (224, 8, 7, 3), (256, 8, 8, 4),
    (256, 8, 1, 1), (256, 3, 4, 1), (256, 7, 2, 1), (264, 8, 1, 1), (288, 8, 9, 4), (384, 8, 6, 4), (504, 5, 1, 1), (512, 8, 16, 3),
    (512, 8, 8, 8), (512, 8, 2, 1)])
def test_shapes(lib, dtype, E, k, n_group, topk_group):
    for i, (bias, flags) in enumerate([(None, lib.MOE_ROUTE_SOFTMAX | lib.MOE_ROUTE_RENORM), (bias_of(E), lib.MOE_ROUTE_GROUP_PAIR),
                                       (bias_of(E), lib.MOE_ROUTE_SOFTMAX), (None, lib.MOE_ROUTE_RENORM),
                                       (bias_of(E), lib.MOE_ROUTE_RENORM | lib.MOE_ROUTE_GROUP_PAIR), (None, lib.MOE_ROUTE_SOFTMAX)]):
        check(lib, logits_of(37, E, dtype, seed=i), k, bias, n_group, topk_group, scale=2.5, flags=flags)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("flags", [0, 1, 2, 3, 4, 6, 7])
def test_masked_experts_and_odd_values(lib, dtype, bias, flags):
    E = 128
    z = logits_of(41, E, dtype, seed=3)
    inf, nan = float("inf"), float("nan")
    z[0] = -inf                                    # nothing open
    z[1] = nan
    z[2, 5:] = -inf                                # fewer open than k
    z[3, ::2], z[3, 1::4] = nan, -inf
    z[4, 7] = z[4, 40] = inf                       # count as the largest number
    z[5] = inf
    z[6] = 0.0                                     # all alike: the first ones
    z[7, 10:20] = 3.0
    z[8] = -88.0 if dtype != "f16" else -60.0      # scores next to nothing
    z[8, 33] = -89.0
    z[9] = torch.where(torch.arange(E, device="cuda") % 16 == 0, z[9], -inf)   # one open expert a group
    z[10, :112] = -inf                             # one group left
    z[11] = 300.0                                  # sigmoids that are 1 in 64 bits too
    z[11, 9] = 400.0
    z[12, 8:] = -inf                               # as many open as k
    z[13, 9:] = -inf
    z[14, :40] = 2.0                               # more of the same than the list holds
    z[15, 31] = nan
    b = bias_of(E) if bias else None
    if bias:
        b[17], b[18], b[19], b[3], b[44] = -inf, nan, inf, 1e6, -1e6
    check(lib, z, 8, b, n_group=8, topk_group=5, flags=flags)
    check(lib, z, 8, b, flags=flags)
    check(lib, z, 3, b, flags=flags, n_tokens=8193)


def test_values_that_fp32_cannot_tell_apart(lib):
    """Logits an ulp apart, and biases that all but cancel the difference: 64 bits decide."""
    T, E = 32, 256
    z = torch.empty((T, E), device="cuda").uniform_(0.9, 0.9000002, generator=torch.Generator(device="cuda").manual_seed(5))
    check(lib, z, 8)
    check(lib, z, 8, torch.zeros(E, device="cuda"))
    wide = logits_of(T, E, seed=9)
    wide[:] = wide[:1] + 1e-6 * logits_of(T, E, seed=10)
    level = (0.7 - torch.sigmoid(wide[0].double())).float()    # score + bias is 0.7 to some 2^-24 for every expert
    some = torch.where(torch.arange(E, device="cuda") % 19 == 3, level, level - 0.5)     # for 13 of them: the list settles it
    groups = torch.where(torch.arange(E, device="cuda") % 32 < 2, level, level - 0.5)    # for two of each group
    for bias in (level, some, groups):
        for flags in (0, lib.MOE_ROUTE_GROUP_PAIR, lib.MOE_ROUTE_RENORM):
            check(lib, wide, 8, bias, flags=flags)
            check(lib, wide, 8, bias, n_group=8, topk_group=4, flags=flags)
    soft = (0.5 - torch.softmax(wide[0].double(), 0)).float()
    check(lib, wide, 8, soft, flags=lib.MOE_ROUTE_SOFTMAX)
    check(lib, wide, 8, soft, n_group=8, topk_group=4, flags=lib.MOE_ROUTE_SOFTMAX | lib.MOE_ROUTE_GROUP_PAIR)


def test_near_values_of_a_softmax(lib):
    """Shares and biases that come to nearly the same for a few experts, or two of each group: few and many tokens."""
    T, E = 32, 256
    wide = logits_of(T, E, seed=9)
    wide[:] = wide[:1] + 1e-6 * logits_of(T, E, seed=10)
    level = (0.5 - torch.softmax(wide[0].double(), 0)).float()
    e = torch.arange(E, device="cuda")
    for at in (e % 19 == 3, e % 32 < 2, e % 32 < 5, e < 20):
        bias = torch.where(at, level, level - 0.25)
        for flags in (lib.MOE_ROUTE_SOFTMAX, lib.MOE_ROUTE_SOFTMAX | lib.MOE_ROUTE_GROUP_PAIR | lib.MOE_ROUTE_RENORM):
            for n in (T, MANY):
                check(lib, wide, 8, bias, flags=flags, T=n)
                check(lib, wide, 5, bias, n_group=8, topk_group=4, flags=flags, T=n)


def test_infinite_biases(lib):
    """Groups whose experts are +inf rank before all others, in the order of their numbers."""
    z, inf = logits_of(20, 256, seed=6), float("inf")
    for at in ([70, 75, 170, 180], [70, 75, 170, 180, 230, 231], [3, 70, 170], list(range(256)), [255]):
        b = bias_of(256)
        b[at] = inf
        for topk_group in (1, 2, 3):
            for flags in (0, lib.MOE_ROUTE_GROUP_PAIR):
                for T in (8195, 20):
                    check(lib, z, 2, b, n_group=8, topk_group=topk_group, flags=flags, T=T)


def test_ties_go_to_the_lowest_number(lib):
    z = logits_of(100, 256, seed=2).mul(2).round().div(2).to(torch.bfloat16)      # many equal logits
    for bias in (None, torch.zeros(256, device="cuda"), torch.full((256,), 0.25, device="cuda")):
        check(lib, z, 8, bias, n_group=8, topk_group=4, flags=lib.MOE_ROUTE_GROUP_PAIR if bias is not None else 0)
        check(lib, z, 8, bias, flags=lib.MOE_ROUTE_SOFTMAX)


@pytest.mark.parametrize("T", [8191, 8192, 8193, 12159, 12161, 30011])
@pytest.mark.parametrize("E,pad,shift", [(256, 0, 0), (256, 8, 0), (256, 3, 1), (64, 16, 8), (60, 4, 0)])
def test_lengths_strides_and_alignment(lib, T, E, pad, shift):
    for dtype in TYPES:
        base = logits_of(50, E + pad + shift, dtype, seed=T)
        check(lib, base[:, shift: shift + E], 6, bias_of(E), flags=lib.MOE_ROUTE_RENORM, T=T)


@pytest.mark.parametrize("n", [-5, 0, 1, 3, 4095, 8194, 10 ** 6])
def test_rows_behind_a_padded_batch(lib, n):
    z = logits_of(61, 64)
    check(lib, z, 4, n_tokens=n, flags=lib.MOE_ROUTE_SOFTMAX)
    check(lib, z, 4, bias_of(64), n_tokens=n)


def test_offsets_past_32_bits(lib):
    T, ld = 8200, 1 << 19                            # rows 1 MiB apart
    z = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")[:, :64]
    z.copy_(logits_of(T, 64, "bf16"))
    out = [(torch.empty((T, 4), dtype=torch.int32, device="cuda"), torch.empty((T, 4), device="cuda")) for _ in range(2)]
    lib.moe_route(z, *out[0])
    lib.moe_route(z.contiguous(), *out[1])
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    check(lib, z[-50:].contiguous(), 4)


def test_as_for_few_tokens(lib):
    """The tokens of a large call one part after another: the same experts, the weights to their rounding."""
    T = 8192
    for dtype in TYPES:
        z, b = logits_of(T, 256, dtype, seed=4), bias_of(256)
        z[torch.rand((T, 256), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) < 0.3] = -float("inf")
        for flags in (0, 1, 2, 4, 6, 7):
            kw = dict(bias=b, n_group=8, topk_group=4, scale=2.5, flags=flags)
            ids, w = torch.empty((T, 8), dtype=torch.int32, device="cuda"), torch.empty((T, 8), device="cuda")
            lib.moe_route(z, ids, w, **kw)
            few, fw = torch.empty_like(ids), torch.empty_like(w)
            for i in range(0, T, 1024):
                lib.moe_route(z[i: i + 1024], few[i: i + 1024], fw[i: i + 1024], **kw)
            assert torch.equal(ids, few)
            # softmax: the arguments of exp span some 15, rounded to 2^-24 of it on either side
            assert ((w - fw).abs() <= 2.0 ** -23 * 40 * fw.abs()).all()
