"""moe_kv_pages whose lengths and counts lie in one cache line, before and after: steps that follow one another at once."""
import pytest
import torch

pytestmark = pytest.mark.gpu

I32 = dict(dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("B,new,page", [(20, 3, 16), (200, 7, 16), (1600, 1, 16), (1600, 9, 32), (64, 300, 16)])
def test_a_chain_of_steps(lib, B, new, page):
    """40 steps as a graph give what they give with a wait behind each."""
    steps, max_pages = 40, -(-41 * new // page) + 2
    pool = B * max_pages
    g = torch.Generator(device="cuda").manual_seed(B)
    gain = torch.randint(0, new + 1, (steps, B), generator=g, device="cuda").int()
    cut = torch.randint(0, 3, (steps, B), generator=g, device="cuda").int()

    def made():
        lengths, counts = torch.zeros(2 * B, **I32), torch.tensor([pool, 0], **I32)       # neighbours in memory
        return dict(lengths=(lengths[:B], lengths[B:]), counts=(counts[:1], counts[1:]), table=torch.full((B, max_pages), -9, **I32),
                    free=torch.randperm(pool, generator=torch.Generator().manual_seed(1)).to(**I32), keep=torch.zeros((steps, B), **I32),
                    cu=torch.full((steps, B + 1), -7, **I32), slots=torch.full((steps, B * new), -7, dtype=torch.int64, device="cuda"),
                    err=lib.new_error_word())

    def step(s, i):
        old, out = s["lengths"][i % 2], s["lengths"][1 - i % 2]
        lib.moe_kv_pages(old, gain[i], s["table"], s["free"], s["counts"][i % 2], page, out, s["cu"][i], s["counts"][1 - i % 2],
                         kv_keep=None if i % 4 else s["keep"][i], slots=s["slots"][i], err=s["err"])

    def keeps(s, i):
        if i % 4 == 0:
            s["keep"][i] = (s["lengths"][i % 2] - cut[i]).clamp_(min=0)

    slow = made()
    for i in range(steps):
        keeps(slow, i)
        torch.cuda.synchronize()
        step(slow, i)
        torch.cuda.synchronize()
    names = ("table", "cu", "slots", "err")
    quick = made()
    first = {n: quick[n].clone() for n in ("table", "free")}
    quick["keep"].copy_(slow["keep"])
    step(made(), 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            step(quick, i)
    for _ in range(20):
        for n, t in first.items():
            quick[n].copy_(t)
        quick["lengths"][0].zero_()
        quick["counts"][0].fill_(pool)
        graph.replay()
        for n in names:
            assert torch.equal(quick[n], slow[n]), n
        for i in range(2):
            assert torch.equal(quick["lengths"][i], slow["lengths"][i]) and torch.equal(quick["counts"][i], slow["counts"][i])
        left = slow["counts"][steps % 2].item()
        assert torch.equal(quick["free"][:left], slow["free"][:left])
