"""moe_verify_drafts of vocabularies that a warp needs several rounds of loads for."""
import pytest
import torch

from tests.test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,V,dtype,with_q", [
    ([3], 160003, "f32", True), ([2, 0, 3], 301007, "bf16", True), ([1, 2, 1, 0, 3, 2, 1, 1], 131073, "f32", False),
    ([1] * 40 + [0, 2], 33001, "f16", True), ([0, 1] * 90, 17003, "f32", True), ([0, 1, 0] * 210, 9001, "f32", True),
    ([0] * 620, 17011, "bf16", False)])
def test_batches(lib, counts, V, dtype, with_q):
    Batch(counts, V, dtype, with_q, seed=V).check(lib)


@pytest.mark.parametrize("ld,shift", [(70013, 0), (70016, 3), (70024, 8)])
def test_strides_and_alignment(lib, ld, shift):
    for dtype in ("f32", "bf16"):
        Batch([1] * 39, 70001, dtype, ld=ld, shift=shift, seed=ld).check(lib)


@pytest.mark.parametrize("V,B", [(1 << 20, 64), (1 << 18, 512), (1 << 22, 4)])
def test_borders_that_are_hit_exactly(lib, V, B):
    """Sums of equal powers of two: u on a border takes the entry behind it, marks or not."""
    i32 = dict(dtype=torch.int32, device="cuda")
    p = torch.full((1, V), 1.0 / V, device="cuda").expand(B, V).contiguous()
    want = torch.arange(B, device="cuda") * (V // B) + torch.randint(0, 3, (B,), device="cuda") * (V // B // 4)
    accepted, out = torch.empty(B, **i32), torch.empty((B, 1), **i32)

    def draw(u):
        lib.moe_verify_drafts(p, torch.zeros(B, **i32), torch.arange(B + 1, **i32), torch.rand(B, device="cuda"), u, accepted, out)
        return out[:, 0].long()

    assert torch.equal(draw(want / V), want)
    p[:, ::2] = 0.0                                       # entries without weight are never drawn
    want = want // 2 * 2
    assert torch.equal(draw(want / V), want + 1)


def test_extreme_random_numbers_and_empty_stretches(lib):
    b = Batch([1] * 9, 140001, seed=4)
    b.us = torch.tensor([0.0, 1.0, 2.0, float("inf"), float("nan"), -1.0, 1 - 2.0 ** -24, 2.0 ** -126, 0.5], device="cuda")
    b.p[:, :3] = 0.0
    b.p[:, -70000:] = 0.0
    b.check(lib)
    b.p[:, 10: 60000] = 0.0
    b.check(lib)
    b.p[:] = 0.0
    b.p[:, 99999] = 1e-30                                 # one entry has it all
    b.check(lib)


@pytest.mark.parametrize("with_q", [True, False])
def test_odd_probabilities(lib, with_q):
    b = Batch([1] * 8, 140001, with_q=with_q, seed=6)
    r = b.cu
    nan, inf = float("nan"), float("inf")
    b.p[r[1], 5:9] = nan
    b.p[r[2]] = 0.0                                         # nothing to draw from
    b.p[r[3]] = nan
    b.p[r[4], 7], b.p[r[4] + 1, 100008] = inf, -inf         # looked for entry by entry
    if with_q:
        b.q[r[5]] = b.p[r[5]] * 1.5                         # q above p everywhere: the residual is empty
        b.ua[r[5]] = 0.9999
        b.q[r[6], 100:200] = nan
        b.ua[r[6]] = 1e30
        b.q[r[7], 70003], b.q[r[7], 4] = inf, -inf
        b.ua[r[7]] = 1e30
    b.check(lib)
