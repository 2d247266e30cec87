"""moe_gate beside the products that hold an SM's tensor memory, on two streams and one behind the other."""
import pytest
import torch

pytestmark = pytest.mark.gpu

HIDDEN, INNER, EXPERTS, TOP_K = 512, 256, 8, 2


class Products:
    """A routed-expert FFN of a few tokens: its weight-stationary GEMMs take all of an SM's tensor memory."""

    def __init__(self, lib, T, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=g, device="cuda").bfloat16()  # noqa: E731
        w13, w2 = normal(EXPERTS, 2 * INNER, HIDDEN) * HIDDEN ** -0.5, normal(EXPERTS, HIDDEN, INNER) * INNER ** -0.5
        w13_q, w13_s = torch.empty_like(w13, dtype=torch.uint8), torch.empty((EXPERTS, 2 * INNER // 128, HIDDEN // 128), device="cuda")
        w2_q, w2_s = torch.empty_like(w2, dtype=torch.uint8), torch.empty((EXPERTS, HIDDEN // 128, INNER // 128), device="cuda")
        lib.moe_quant_weight_fp8(w13, w13_q, w13_s)
        lib.moe_quant_weight_fp8(w2, w2_q, w2_s)
        x = normal(T, HIDDEN)
        ids = torch.stack([torch.randperm(EXPERTS, generator=torch.Generator().manual_seed(t))[:TOP_K] for t in range(T)]).int().cuda()
        self.out = torch.empty((T, HIDDEN), dtype=torch.bfloat16, device="cuda")
        self.held = x, ids, torch.full((T, TOP_K), 0.5, device="cuda"), w13_q, w13_s, w2_q, w2_s
        self.desc = lib.make_ffn_desc(*self.held[:3], w13_q, w13_s, w2_q, w2_s, self.out, 0, EXPERTS, lib.MOE_LAYOUT_MASKED,
                                      max_m=-(-T // 128) * 128)
        self.ws = lib.alloc_workspace(self.desc)
        self.run = lambda stream: lib.moe_ffn(self.desc, self.ws, stream=stream)


class Gates:
    """Calls that split the hidden dimension over clusters of small CTAs, and larger ones."""

    def __init__(self, lib, seed=1):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lib, self.calls, self.err = lib, [], lib.new_error_word()
        for T, E, H in ((17, 16, 1024), (24, 8, 1024), (17, 32, 1024), (20, 16, 512), (64, 256, 7168), (300, 60, 2040), (24, 16, 128),
                        (1500, 256, 1024)):
            x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
            w = (torch.randn((E, H), generator=g, device="cuda") * H ** -0.5).bfloat16()
            self.calls.append((x, w, torch.empty((T, E), device="cuda")))

    def run(self, stream):
        for c in self.calls:
            self.lib.moe_gate(*c, err=self.err, stream=stream)


def test_on_two_streams(lib):
    products, gates = Products(lib, 48), Gates(lib)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    products.run(one)
    gates.run(two)
    torch.cuda.synchronize()
    want = [products.out.clone()] + [c[2].clone() for c in gates.calls]
    for _ in range(100):
        products.out.zero_()
        for c in gates.calls:
            c[2].zero_()
        torch.cuda.synchronize()
        for _ in range(5):
            products.run(one)
            gates.run(two)
            products.run(one)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [products.out] + [c[2] for c in gates.calls]))
    assert lib.moe_read_device_status(gates.err) == (lib.MOE_OK, 0)


def test_one_behind_the_other(lib):
    """No wait of the host between a product, a gate, a product: as calls and as a graph."""
    products, gates = Products(lib, 20, seed=3), Gates(lib, seed=4)
    stream = torch.cuda.Stream()
    products.run(stream)
    gates.run(stream)
    stream.synchronize()
    want = [products.out.clone()] + [c[2].clone() for c in gates.calls]

    def chain():
        for c in gates.calls:
            products.run(stream)
            lib.moe_gate(*c, err=gates.err, stream=stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        chain()
    for i in range(40):
        products.out.zero_()
        for c in gates.calls:
            c[2].zero_()
        torch.cuda.synchronize()
        if i % 2:
            with torch.cuda.stream(stream):
                graph.replay()
        else:
            chain()
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, [products.out] + [c[2] for c in gates.calls]))
    assert lib.moe_read_device_status(gates.err) == (lib.MOE_OK, 0)
