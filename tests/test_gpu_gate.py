"""moe_gate against 64-bit sums."""
import pytest
import torch

from tests.gpu_common import Guarded, SENTINEL_F32, f32_bits

pytestmark = pytest.mark.gpu


def made(T, E, H, dtype, seed=0, x_ld=None, w_ld=None, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.zeros((T, x_ld or H), device="cuda", dtype=dtype)[:, :H]
    w = torch.zeros((E, w_ld or H), device="cuda", dtype=dtype)[:, :H]
    x.copy_(torch.randn((T, H), generator=g, device="cuda") * gain)
    w.copy_(torch.randn((E, H), generator=g, device="cuda") * H ** -0.5)
    return x, w


def bound(x, w):
    """Products are exact in fp32's range; sums of 512 columns on the tensor cores lose at most
    a bit of 2^-23 of the running magnitude at each of their 32 steps of 16 (and within a step),
    the fp32 sums of these at most 2^-24 each of theirs.  All of it relative to sum |x w|."""
    n = -(-x.shape[1] // 512) + 8
    return ((64 * 2.0 ** -23) + n * 2.0 ** -24) * (x.double().abs() @ w.double().abs().T) + 1e-37


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,E,H", [(1, 1, 8), (1, 256, 7168), (2, 16, 64), (3, 17, 72), (31, 60, 2040), (64, 256, 512), (128, 128, 128),
                                   (129, 257, 136), (130, 1024, 264), (200, 300, 1000), (257, 8, 4096), (333, 60, 2040), (1000, 512, 192),
                                   (5000, 64, 256), (4097, 255, 520), (7, 31, 8200), (20000, 33, 128), (16461, 256, 264),
                                   (3000, 512, 7168), (8193, 200, 2048), (900, 129, 1032), (9, 300, 72), (16, 1024, 7168),
                                   (13, 5, 8), (12, 200, 2056), (16, 153, 4104), (8, 305, 520), (17, 256, 7168), (700, 512, 4096)])
def test_logits(lib, T, E, H, dtype):
    x, w = made(T, E, H, dtype, seed=T + E)
    out = Guarded((T, E), torch.float32, f32_bits(SENTINEL_F32))
    lib.moe_gate(x, w, out.t)
    assert ((out.t.double() - x.double() @ w.double().T).abs() <= bound(x, w)).all()
    assert out.intact()


@pytest.mark.parametrize("T,E,H", [(5, 20, 96), (150, 256, 640)])
def test_strides_and_what_lies_between_rows(lib, T, E, H):
    x, w = made(T, E, H, torch.bfloat16, x_ld=H + 24, w_ld=H + 8)
    x._base[:, H:] = float("nan")                 # never read as part of a row
    w._base[:, H:] = float("nan")
    room = torch.full((T, E + 5), SENTINEL_F32, device="cuda")
    lib.moe_gate(x, w, room[:, :E])
    assert ((room[:, :E].double() - x.double() @ w.double().T).abs() <= bound(x, w)).all()
    assert (room[:, E:] == SENTINEL_F32).all()


def test_nan_and_inf_stay_in_their_rows(lib):
    x, w = made(70, 40, 256, torch.bfloat16)
    x[3, 100], x[4, 7], w[11, 9] = float("nan"), float("inf"), float("nan")
    out = lib.moe_gate(x, w, torch.empty((70, 40), device="cuda"))
    clean = torch.ones((70, 40), dtype=torch.bool, device="cuda")
    clean[3:5] = clean[:, 11] = False
    assert out[3].isnan().all() and not out[4].isfinite().any() and out[:, 11].isnan().all()
    assert out[clean].isfinite().all()


def test_large_and_small_magnitudes(lib):
    x, w = made(40, 24, 384, torch.bfloat16, gain=2.0 ** 60)
    out = lib.moe_gate(x, w, torch.empty((40, 24), device="cuda"))
    assert ((out.double() - x.double() @ w.double().T).abs() <= bound(x, w)).all()
    x, w = made(40, 24, 384, torch.bfloat16, gain=2.0 ** -60)
    out = lib.moe_gate(x, w, torch.empty((40, 24), device="cuda"))
    assert ((out.double() - x.double() @ w.double().T).abs() <= bound(x, w)).all()


@pytest.mark.parametrize("T", [1, 8, 64, 700, 9000])
def test_repeats_bit_for_bit_and_in_a_graph(lib, T):
    x, w = made(T, 256, 1024, torch.bfloat16)
    first = lib.moe_gate(x, w, torch.empty((T, 256), device="cuda")).clone()
    out = torch.empty((T, 256), device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_gate(x, w, out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, first)


def test_on_another_stream(lib):
    x, w = made(300, 128, 512, torch.float16)
    out, ref = torch.empty((300, 128), device="cuda"), lib.moe_gate(x, w, torch.empty((300, 128), device="cuda"))
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    lib.moe_gate(x, w, out, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)


def test_offsets_past_32_bits(lib):
    T, H, ld = 600, 128, 1 << 23                   # rows 16 MiB apart: 10 GB of address space
    x = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")[:, :H]
    y, w = made(T, 32, H, torch.bfloat16)
    x.copy_(y)
    out = lib.moe_gate(x, w, torch.empty((T, 32), device="cuda"))
    assert torch.equal(out, lib.moe_gate(y, w, torch.empty((T, 32), device="cuda")))


def test_refusals(lib):
    x, w = made(4, 8, 64, torch.bfloat16)
    out = torch.full((4, 8), SENTINEL_F32, device="cuda")
    for args in ((x.float(), w, out), (x, w.half(), out), (x, w, out.half()), (x, w[:, :56], out), (x.t(), w, out),
                 (x, w, out[:, :4]), (x.cpu(), w, out)):
        with pytest.raises(ValueError):
            lib.moe_gate(*args)
    with pytest.raises(lib.MoeError):               # an x that starts between 16-byte boundaries
        lib.moe_gate(torch.zeros((4, 65), dtype=torch.bfloat16, device="cuda")[:, 1:], w, out)
    assert (out == SENTINEL_F32).all()
    assert lib.moe_gate(x[:0], w, out[:0]).shape == (0, 8)
