"""moe_verify_drafts where the drawn token lies at an end: u_sample of 1 and above, and weights that are tiny beside the others."""
import pytest
import torch

from tests.test_gpu_verify import Batch, TYPES

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


def drawn(lib, p, u, dtype="f32"):
    """The token that each row of p gives for its u."""
    B = p.shape[0]
    accepted, out = torch.full((B,), -7, **I32), torch.full((B, 1), -7, **I32)
    lib.moe_verify_drafts(p, torch.zeros(B, **I32), torch.arange(B + 1, **I32), torch.zeros(B, device="cuda"), u, accepted, out)
    return out[:, 0].tolist()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("V,B", [(1, 3), (40, 8), (1000, 5), (33001, 40), (128000, 16), (160003, 2), (9001, 630), (1 << 20, 1)])
def test_the_last_entry_with_weight(lib, V, B, dtype):
    """For a u of 1 or more it is the last j with w_j > 0, however small that weight is."""
    tail = {"f32": 1e-30, "bf16": 1e-30, "f16": 2.0 ** -24}[dtype]
    g = torch.Generator(device="cuda").manual_seed(V)
    p = torch.softmax(torch.randn((B, V), generator=g, device="cuda"), 1).to(TYPES[dtype])
    p[:, V // 2 + 1:] = 0.0                               # nothing in the second half
    p[:, 0] = 1.0
    last = torch.randint(V // 2, V, (B,), generator=g, device="cuda")
    p.scatter_(1, last[:, None], torch.full((B, 1), tail, device="cuda").to(TYPES[dtype]))     # but one small entry
    want = last.tolist()
    for u in (1.0, 2.0, float("inf")):
        assert drawn(lib, p, torch.full((B,), u, device="cuda")) == want, u


@pytest.mark.parametrize("V,B", [(500, 4), (70001, 6), (160003, 3)])
def test_the_last_entry_of_a_residual(lib, V, B):
    """The same for what a refused draft leaves: p above q by an ulp of a small entry at the end."""
    b = Batch([1] * B, V, seed=V)
    b.ua[:] = 1e30
    b.us[:] = 1.0
    b.q.copy_(b.p)
    b.p[:, 1] = 0.5
    b.p[:, V - 3] = 1e-30
    b.q[:, V - 3] = 0.0
    b.tokens[:] = 7
    _, out = b.check(lib)
    assert [o[0] for o in out] == [V - 3] * B
