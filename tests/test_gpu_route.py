"""moe_route against a plain 64-bit routing, token by token."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def plain(z, k, bias=None, n_group=1, topk_group=1, scale=1.0, softmax=False, renorm=False, pair=False):
    """ids and 64-bit weights of one token; z: 64-bit logits."""
    z = np.where(np.isnan(z), -np.inf, np.minimum(z, np.finfo(np.float32).max))
    is_open = z > -np.inf
    if softmax:
        top = z.max() if is_open.any() else 0.0
        e = np.where(is_open, np.exp(z - top), 0.0)
        score = e / e.sum() if is_open.any() else e
    else:
        with np.errstate(over="ignore"):
            score = 1.0 / (1.0 + np.exp(-z))
    if bias is None:
        value = z.copy()
    else:
        value = score + bias
        is_open &= bias > -np.inf
    if n_group > 1:
        size, marks = len(z) // n_group, []
        for g in range(n_group):
            at = range(g * size, (g + 1) * size)
            v = sorted((float(score[e] if pair and bias is None else value[e]) for e in at if is_open[e]), reverse=True)
            marks.append(-np.inf if not v else sum(v[:2]) if pair else v[0])
        kept = sorted(range(n_group), key=lambda g: (-marks[g], g))[:topk_group]
        is_open &= np.isin(np.arange(len(z)) // size, kept)
    order = sorted(np.flatnonzero(is_open), key=lambda e: (-value[e], e))[:k]
    w = score[order]
    if renorm:
        w = w / w.sum() if w.sum() > 0 else w
    ids = np.full(k, -1)
    weights = np.zeros(k)
    ids[: len(order)], weights[: len(order)] = order, scale * w
    return ids, weights


def check(lib, logits, k, bias=None, n_group=1, topk_group=1, scale=1.0, flags=0, n_tokens=None):
    T, E = logits.shape
    ids = torch.full((T, k + 3), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, k + 1), 77.0, device="cuda")
    count = None if n_tokens is None else torch.tensor([n_tokens], dtype=torch.int32, device="cuda")
    lib.moe_route(logits, ids[:, :k], w[:, :k], bias=bias, n_group=n_group, topk_group=topk_group, scale=scale, flags=flags, n_tokens=count)
    assert (ids[:, k:] == 77).all() and (w[:, k:] == 77.0).all()
    softmax, renorm, pair = (bool(flags & f) for f in (lib.MOE_ROUTE_SOFTMAX, lib.MOE_ROUTE_RENORM, lib.MOE_ROUTE_GROUP_PAIR))
    z, b = logits.double().cpu().numpy(), None if bias is None else bias.double().cpu().numpy()
    ids, w = ids[:, :k].cpu().numpy(), w[:, :k].double().cpu().numpy()
    for t in range(T):
        if n_tokens is not None and t >= n_tokens:
            assert (ids[t] == -1).all() and (w[t] == 0).all()
            continue
        want, weight = plain(z[t], k, b, n_group, topk_group, scale, softmax, renorm, pair)
        assert (ids[t] == want).all(), (t, ids[t], want)
        # exp within 2 units of 2^-24 (and its argument z - max rounded: 2^-24 of it), sums of E and k
        # terms and divisions of half a unit each; what fp32 has as subnormals, to 2^-140
        fin = z[t][np.isfinite(z[t])]
        spread = float(fin.max() - fin.min()) if softmax and len(fin) else 0.0
        tol = 2.0 ** -24 * (24 + min(spread, 200.0))
        assert (np.abs(w[t] - weight) <= tol * np.abs(weight) + 2.0 ** -120 * max(1.0, abs(scale))).all(), (t, w[t], weight)
    return ids


def logits_of(T, E, dtype="f32", seed=0, gain=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn((T, E), generator=g, device="cuda")).to(TYPES[dtype])


def bias_of(E, seed=1, gain=0.1):
    return gain * torch.randn(E, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("E,k,n_group,topk_group", [
    (1, 1, 1, 1), (2, 2, 1, 1), (8, 2, 1, 1), (31, 7, 1, 1), (32, 32, 1, 1), (33, 3, 1, 1), (60, 4, 1, 1), (64, 6, 1, 1), (64, 6, 8, 3),
    (128, 8, 4, 2), (160, 6, 8, 3), (256, 8, 8, 4), (256, 8, 1, 1), (257, 9, 1, 1), (288, 8, 32, 7), (384, 16, 2, 1), (512, 22, 16, 5),
    (96, 12, 3, 2), (1000, 31, 8, 8), (1024, 32, 32, 1), (21, 3, 7, 2)])
def test_shapes(lib, dtype, E, k, n_group, topk_group):
    for i, (bias, flags) in enumerate([(None, lib.MOE_ROUTE_SOFTMAX | lib.MOE_ROUTE_RENORM), (bias_of(E), lib.MOE_ROUTE_GROUP_PAIR),
                                       (bias_of(E), lib.MOE_ROUTE_SOFTMAX), (None, lib.MOE_ROUTE_RENORM | lib.MOE_ROUTE_GROUP_PAIR),
                                       (bias_of(E), lib.MOE_ROUTE_RENORM | lib.MOE_ROUTE_GROUP_PAIR), (None, 0)]):
        check(lib, logits_of(37, E, dtype, seed=i), k, bias, n_group, topk_group, scale=2.5, flags=flags)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("flags", [0, 1, 2, 3, 4, 6, 7])
def test_masked_experts_and_odd_values(lib, dtype, bias, flags):
    z = logits_of(40, 64, dtype, seed=3)
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
    z[9] = torch.where(torch.arange(64, device="cuda") % 8 == 0, z[9], -inf)   # one open expert a group
    z[10, :56] = -inf                              # one group left
    z[11] = 300.0                                  # sigmoids that are 1 in 64 bits too
    z[11, 9] = 400.0
    b = bias_of(64) if bias else None
    if bias:
        b[17], b[18], b[19], b[3], b[44] = -inf, nan, inf, 1e6, -1e6
    check(lib, z, 8, b, n_group=8, topk_group=3, flags=flags)
    check(lib, z, 20, b, flags=flags)
    check(lib, z, 3, b, flags=flags, n_tokens=23)


def test_values_that_fp32_cannot_tell_apart(lib):
    """Logits an ulp apart, and biases that all but cancel the difference: 64 bits decide."""
    T, E = 64, 128
    z = torch.empty((T, E), device="cuda").uniform_(0.9, 0.9000002, generator=torch.Generator(device="cuda").manual_seed(5))
    check(lib, z, 8)
    check(lib, z, 8, torch.zeros(E, device="cuda"))
    check(lib, z, 8, flags=lib.MOE_ROUTE_GROUP_PAIR, n_group=16, topk_group=5)
    wide = logits_of(T, E, seed=9)
    wide[:] = wide[:1] + 1e-6 * logits_of(T, E, seed=10)
    level = (0.7 - torch.sigmoid(wide[0].double())).float()    # score + bias is 0.7 to some 2^-24 for every expert
    for flags in (0, lib.MOE_ROUTE_GROUP_PAIR, lib.MOE_ROUTE_RENORM):
        check(lib, wide, 8, level, flags=flags)
        check(lib, wide, 8, level, n_group=8, topk_group=4, flags=flags)
    soft = (0.5 - torch.softmax(wide[0].double(), 0)).float()
    check(lib, wide, 8, soft, flags=lib.MOE_ROUTE_SOFTMAX)
    check(lib, wide, 8, soft, n_group=8, topk_group=4, flags=lib.MOE_ROUTE_SOFTMAX | lib.MOE_ROUTE_GROUP_PAIR)


def test_ties_go_to_the_lowest_number(lib):
    z = logits_of(200, 256, seed=2).mul(2).round().div(2).to(torch.bfloat16)      # many equal logits
    for bias in (None, torch.zeros(256, device="cuda"), torch.full((256,), 0.25, device="cuda")):
        check(lib, z, 8, bias, n_group=8, topk_group=4, flags=lib.MOE_ROUTE_GROUP_PAIR)
        check(lib, z, 32, bias, flags=lib.MOE_ROUTE_SOFTMAX)


@pytest.mark.parametrize("T", [1, 2, 3, 5, 700])
@pytest.mark.parametrize("E,pad,shift", [(256, 0, 0), (256, 3, 1), (60, 1, 0), (10, 6, 3)])
def test_strides_and_alignment(lib, T, E, pad, shift):
    for dtype in TYPES:
        base = logits_of(T, E + pad + shift, dtype, seed=T)
        z = base[:, shift: shift + E]
        check(lib, z if T < 100 else z[::7][:50], 6, bias_of(E), flags=lib.MOE_ROUTE_RENORM)


@pytest.mark.parametrize("n", [-5, 0, 1, 99, 100, 1000])
def test_rows_behind_a_padded_batch(lib, n):
    check(lib, logits_of(100, 64), 4, n_tokens=n, flags=lib.MOE_ROUTE_SOFTMAX)


def test_large_batch_repeats_and_in_a_graph(lib):
    z, b = logits_of(9001, 256, seed=8), bias_of(256)
    out = [(torch.empty((9001, 8), dtype=torch.int32, device="cuda"), torch.empty((9001, 8), device="cuda")) for _ in range(2)]
    kw = dict(bias=b, n_group=8, topk_group=4, scale=2.5, flags=lib.MOE_ROUTE_RENORM | lib.MOE_ROUTE_GROUP_PAIR)
    lib.moe_route(z, *out[0], **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_route(z, *out[1], **kw)
    for _ in range(2):
        out[1][0].fill_(-7)
        graph.replay()
        assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    at = torch.randperm(9001, generator=torch.Generator().manual_seed(0))[:300]
    ids = check(lib, z[at.cuda()].contiguous(), 8, b, 8, 4, 2.5, kw["flags"])
    assert (ids == out[0][0][at.cuda()].cpu().numpy()).all()


def test_offsets_past_32_bits(lib):
    T, ld = 300, 1 << 23                            # rows 32 MiB apart
    z = torch.empty((T, ld), device="cuda")[:, :64]
    z.copy_(logits_of(T, 64))
    check(lib, z, 4)


def test_refusals(lib):
    z, ids, w = logits_of(4, 16), torch.full((4, 2), 9, dtype=torch.int32, device="cuda"), torch.full((4, 2), 9.0, device="cuda")
    n = torch.zeros(1, dtype=torch.int32, device="cuda")
    for args, kw in (((z.double(), ids, w), {}), ((z, ids.long(), w), {}), ((z, ids, w[:, :1]), {}), ((z, ids, w.half()), {}),
                     ((z.t(), ids, w), {}), ((z, ids, w), dict(bias=torch.zeros(15, device="cuda"))),
                     ((z, ids, w), dict(bias=torch.zeros(16))), ((z, ids, w), dict(n_tokens=n.long())),
                     ((z.cpu(), ids, w), {}), ((z, ids[:2], w), {})):
        with pytest.raises(ValueError):
            lib.moe_route(*args, **kw)
    for kw in (dict(n_group=3), dict(n_group=16, topk_group=1), dict(topk_group=2), dict(flags=64), dict(scale=float("nan"))):
        with pytest.raises(lib.MoeError):
            lib.moe_route(z, ids, w, **kw)
    assert (ids == 9).all() and (w == 9.0).all()
