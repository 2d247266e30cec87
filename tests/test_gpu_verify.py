"""moe_verify_drafts against a plain 64-bit verification, sequence by sequence."""
import math
import random

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def next_token(w, u):
    w = np.where((w > 0) & np.isfinite(w), w, 0.0)
    sums = np.cumsum(w)
    if not sums[-1] > 0:
        return None
    over = np.flatnonzero(sums > u * sums[-1])
    return int(over[0]) if len(over) else int(np.flatnonzero(w)[-1])


def plain(p, q, tokens, rows, n, u_accept, u_sample):
    """(accepted, next token or -1, whether something was bad) of one sequence with rows (r0, r1)."""
    clean = lambda x: np.where(np.isfinite(x), x, np.nan)  # noqa: E731
    s, V, a, bad = rows[1] - 1 - n, p.shape[1], 0, False
    u = u_sample if u_sample > 0 else 0.0
    for a in range(n + 1):
        if a == n:
            w = p[s + a].copy()
            break
        d, v = tokens[s + a + 1], u_accept[s + a]
        v = v if v > 0 else 0.0
        if 0 <= d < V and v * (1.0 if q is None else q[s + a, d]) < p[s + a, d]:
            continue
        bad = not 0 <= d < V
        w = p[s + a].copy()
        if q is not None:
            with np.errstate(invalid="ignore"):
                w = (w - q[s + a]).astype(np.float64)
        elif 0 <= d < V:
            w[d] = 0.0
        break
    t = next_token(w, u)
    if t is None and a < n:
        t = next_token(p[s + a], u)
    return a, -1 if t is None else t, bad or t is None


class Batch:
    def __init__(self, counts, V, dtype="f32", with_q=True, prompt=None, seed=0, ld=None, shift=0, gain=2.0, apart=0.7):
        """counts: drafts of each sequence, None: a sequence without rows; prompt: rows in front of the last standing token."""
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.n = [0 if c is None else c for c in counts]
        prompt = prompt or [0] * len(counts)
        rows = [0 if c is None else c + 1 + m for c, m in zip(counts, prompt)]
        T = sum(rows)
        self.cu = [sum(rows[:i]) for i in range(len(rows) + 1)]
        z = gain * torch.randn((T, V), generator=g, device="cuda")
        wide = torch.full((T, (ld or V) + shift), float("nan"), device="cuda", dtype=TYPES[dtype])
        self.p = wide[:, shift: shift + V]
        self.p.copy_(torch.softmax(z, 1))
        q = torch.softmax(z + apart * torch.randn((T, V), generator=g, device="cuda"), 1) if T else z
        self.tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
        if T > 1:
            self.tokens[1:] = torch.multinomial(q, 1, generator=g).flatten()[:-1].int()
        self.q = q.to(TYPES[dtype]) if with_q else None
        self.ua, self.us = torch.rand(T, generator=g, device="cuda"), torch.rand(len(rows), generator=g, device="cuda")
        self.given = bool(prompt and any(prompt)) or None in counts
        self.max_out = max(self.n) + 1

    def check(self, lib, max_out=None, bits=None, lens=True):
        B, width = len(self.n), max_out or self.max_out
        i32 = dict(dtype=torch.int32, device="cuda")
        accepted, out = torch.full((B,), -7, **i32), torch.full((B, width + 2), -7, **i32)
        length = torch.arange(1000, 1000 + B, **i32) if lens else None
        keep = torch.full((B,), -7, **i32) if lens else None
        err = lib.new_error_word()
        lib.moe_verify_drafts(self.p, self.tokens, torch.tensor(self.cu, **i32), self.ua, self.us, accepted, out[:, :width], draft_probs=self.q,
                              n_draft=torch.tensor(self.n, **i32) if self.given else None, kv_len=length, kv_keep=keep, err=err)
        assert (out[:, width:] == -7).all()
        p, q = self.p.double().cpu().numpy(), None if self.q is None else self.q.double().cpu().numpy()
        tokens, ua, us, want_bits = self.tokens.tolist(), self.ua.double().tolist(), self.us.double().tolist(), 0
        accepted, out, keep = accepted.tolist(), out[:, :width].tolist(), keep.tolist() if lens else None
        for b, n in enumerate(self.n):
            r = self.cu[b], self.cu[b + 1]
            if r[0] == r[1] or n > width - 1:
                want_bits |= 0 if r[0] == r[1] else 1
                assert accepted[b] == 0 and out[b] == [-1] * width
                assert not lens or keep[b] == 1000 + b
                continue
            a, t, bad = plain(p, q, tokens, r, n, ua, us[b])
            want_bits |= 4 if bad else 0
            s = r[1] - 1 - n
            assert accepted[b] == a, (b, accepted[b], a)
            assert out[b] == tokens[s + 1: s + 1 + a] + [t] + [-1] * (width - a - 1), (b, out[b], a, t)
            assert not lens or keep[b] == 1000 + b - (n - a)
        assert lib.moe_read_device_status(err)[1] == (want_bits if bits is None else bits)
        return accepted, out


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("with_q", [True, False])
@pytest.mark.parametrize("V", [1, 2, 7, 31, 33, 100, 257, 1000, 4099, 32003])
def test_vocabularies(lib, dtype, with_q, V):
    Batch([3, 0, 1, 5, 2, 4, 3, 3], V, dtype, with_q, seed=V).check(lib)


@pytest.mark.parametrize("counts", [[0], [3], [8] * 40, [1, 0, 7] * 100, [40], [70, 3], [33, 32, 31]])
def test_batches(lib, counts):
    Batch(counts, 1500, seed=len(counts), apart=0.2).check(lib)
    Batch(counts, 501, "bf16", with_q=False, seed=1, gain=6.0).check(lib, lens=False)


def test_prompts_and_sequences_without_rows(lib):
    Batch([2, None, 0, 3, None, 0], 777, prompt=[0, 0, 9, 4, 0, 100]).check(lib)
    Batch([None], 777).check(lib)
    Batch([None, 2], 777, with_q=False).check(lib)


def test_too_many_drafts_for_the_output(lib):
    Batch([2, 5, 1, 3], 300).check(lib, max_out=3)


@pytest.mark.parametrize("ld,shift", [(1003, 0), (1000, 0), (1000, 1), (1010, 3), (1024, 4)])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_strides_and_alignment(lib, ld, shift, dtype):
    Batch([2, 3, 0, 4], 999, dtype, ld=ld, shift=shift).check(lib)
    b = Batch([2, 3, 0, 4], 999, dtype)
    wide = torch.full((b.p.shape[0], ld + shift), 3.0, device="cuda", dtype=TYPES[dtype])
    b.q = wide[:, shift: shift + 999].copy_(b.q)            # q laid out in another way than p
    b.check(lib)


def test_borders_that_are_hit_exactly(lib):
    """Sums of multiples of 2^-12: u on a border takes the entry behind it."""
    V = 4096
    b = Batch([0] * 64, V)
    b.p.fill_(2.0 ** -12)
    b.us = torch.arange(64, device="cuda") * 2.0 ** -6
    _, out = b.check(lib)
    assert [o[0] for o in out] == [64 * i for i in range(64)]
    b.p[:, ::2] = 0.0                                       # entries without weight are never drawn
    _, out = b.check(lib)
    assert [o[0] for o in out] == [64 * i + 1 for i in range(64)]


def test_extreme_random_numbers(lib):
    b = Batch([2] * 8, 1000, seed=4)
    b.us = torch.tensor([0.0, 1.0, 2.0, float("inf"), float("nan"), -1.0, 1 - 2.0 ** -24, 2.0 ** -126], device="cuda")
    b.p[:, :3] = 0.0
    b.p[:, -5:] = 0.0
    b.check(lib)
    b.ua[:] = torch.tensor([float("nan"), -1.0, 0.0, 1.0, 2.0, float("inf")] * 4, device="cuda")
    b.check(lib)


@pytest.mark.parametrize("with_q", [True, False])
def test_odd_probabilities(lib, with_q):
    b = Batch([2] * 10, 600, with_q=with_q, seed=6)
    r = b.cu
    nan, inf = float("nan"), float("inf")
    b.ua[r[1]] = 1e30                                       # turned down
    b.p[r[1], 5:9] = nan
    b.p[r[2]] = 0.0                                         # nothing to draw from
    b.p[r[3]] = nan
    b.p[r[4], 7], b.p[r[4] + 1, 8] = inf, -inf
    if with_q:
        b.q[r[5]] = b.p[r[5]] * 1.5                         # q above p everywhere: the residual is empty
        b.ua[r[5]] = 0.9999
        b.q[r[6], 100:200] = nan
        b.ua[r[6]] = 1e30
        b.q[r[7], 3], b.q[r[7], 4] = inf, -inf
        b.ua[r[7]] = 1e30
    b.tokens[r[8] + 1] = 600                                # drafts outside the vocabulary
    b.tokens[r[9] + 1] = -3
    b.p[r[0]: r[0] + 3] *= 1e-30                            # rows that do not sum to 1
    if with_q:
        b.q[r[0]: r[0] + 3] *= 1e-30
    b.check(lib)


def test_flat_and_spiked_distributions(lib):
    """Borders 1e-6 apart, and one entry that has almost all of it."""
    V = 150001
    b = Batch([0] * 16, V)
    b.p.copy_(torch.rand((16, V), device="cuda", generator=torch.Generator(device="cuda").manual_seed(2)) / V)
    b.check(lib)
    b.p *= 1e-6
    b.p[:, 70000] = 1.0
    b.us = torch.linspace(0, 1, 16, device="cuda")
    b.check(lib)
    b = Batch([1] * 16, V, seed=3, gain=0.05, apart=0.05)   # residuals that are differences of near values
    b.ua[:] = 0.999999
    b.check(lib)


def test_row_faults(lib):
    """Offsets that leave the rows, decrease, or drafts that take them all: told, nothing else touched."""
    b = Batch([2, 2, 2, 2], 100)
    b.given = True
    i32 = dict(dtype=torch.int32, device="cuda")
    for cu, n in (([0, 3, 6, 9, 13], [2, 2, 2, 2]), ([-1, 3, 6, 9, 12], [2] * 4), ([0, 3, 2, 9, 12], [2, 0, 2, 2]), ([0, 3, 6, 9, 12], [2, 3, 2, 2]),
                  ([0, 3, 6, 9, 12], [2, -1, 2, 2]), ([0, 3, 6, 9, 12], [1 << 30, 2, 2, 2])):
        accepted, out, err = torch.full((4,), -7, **i32), torch.full((4, 3), -7, **i32), lib.new_error_word()
        lib.moe_verify_drafts(b.p, b.tokens, torch.tensor(cu, **i32), b.ua, b.us, accepted, out, draft_probs=b.q,
                              n_draft=torch.tensor(n, **i32), err=err)
        assert lib.moe_read_device_status(err)[0] == lib.MOE_ERR_BAD_INDEX
        p, q = b.p.double().cpu().numpy(), b.q.double().cpu().numpy()
        for s in range(4):
            if not 0 <= cu[s] < cu[s + 1] <= 12 or not 0 <= n[s] < cu[s + 1] - cu[s]:
                assert accepted[s] == 0 and out[s].tolist() == [-1] * 3
            else:
                a, t, _ = plain(p, q, b.tokens.tolist(), (cu[s], cu[s + 1]), n[s], b.ua.double().tolist(), b.us.double().tolist()[s])
                assert accepted[s] == a and out[s, a] == t


def test_distribution_of_tokens(lib):
    """What comes out is distributed as the target has it, whatever the drafts: the frequencies of
    the first new token over 20000 sequences lie within 5 standard deviations of its distribution."""
    V, B = 12, 20000
    g = torch.Generator(device="cuda").manual_seed(11)
    p = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
    q = torch.softmax(torch.randn(V, generator=g, device="cuda"), 0)
    tokens = torch.zeros(2 * B, dtype=torch.int32, device="cuda")
    tokens[1::2] = torch.multinomial(q, B, replacement=True, generator=g).int()
    i32 = dict(dtype=torch.int32, device="cuda")
    out, accepted = torch.empty((B, 2), **i32), torch.empty(B, **i32)
    lib.moe_verify_drafts(p.expand(2 * B, V).contiguous(), tokens, torch.arange(0, 2 * B + 1, 2, **i32),
                          torch.rand(2 * B, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda"), accepted, out,
                          draft_probs=q.expand(2 * B, V).contiguous())
    seen = torch.bincount(out[:, 0].long(), minlength=V).double() / B
    assert ((seen - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / B).sqrt()).all()
    rate = torch.minimum(p, q).sum().item()
    assert abs(accepted.double().mean().item() - rate) <= 5 * math.sqrt(rate * (1 - rate) / B)


def test_large_batch_of_sequences(lib):
    r = random.Random(3)
    Batch([r.randint(0, 2) for _ in range(3000)], 200, seed=12).check(lib)
    B = 70000                                               # more than a grid's second dimension holds
    i32 = dict(dtype=torch.int32, device="cuda")
    p = torch.zeros((B, 8), device="cuda")
    want = torch.arange(B, **i32) % 8
    p.scatter_(1, want.long()[:, None], 1.0)
    accepted, out = torch.empty(B, **i32), torch.empty((B, 1), **i32)
    lib.moe_verify_drafts(p, torch.zeros(B, **i32), torch.arange(B + 1, **i32), torch.rand(B, device="cuda"), torch.rand(B, device="cuda"),
                          accepted, out)
    assert torch.equal(out[:, 0], want) and (accepted == 0).all()


def test_offsets_past_32_bits(lib):
    b = Batch([2, 2], 100)
    far = torch.empty((6, 1 << 30), dtype=torch.float16, device="cuda")
    b.p, b.q = far[:, 5:105].copy_(b.p), b.q.half()
    b.check(lib)


@pytest.mark.parametrize("V,B", [(50021, 1), (128, 64), (9000, 300)])
def test_repeats_and_in_a_graph(lib, V, B):
    b = Batch([3] * B, V, seed=9)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, outs = torch.tensor(b.cu, **i32), [(torch.empty(B, **i32), torch.empty((B, 4), **i32)) for _ in range(2)]
    lib.moe_verify_drafts(b.p, b.tokens, cu, b.ua, b.us, *outs[0], draft_probs=b.q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_verify_drafts(b.p, b.tokens, cu, b.ua, b.us, *outs[1], draft_probs=b.q)
    for _ in range(3):
        outs[1][1].fill_(-5)
        graph.replay()
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


def test_lengths_in_place(lib):
    b = Batch([3, 1, 2], 500, seed=2)
    i32 = dict(dtype=torch.int32, device="cuda")
    accepted, out, length = torch.empty(3, **i32), torch.empty((3, 4), **i32), torch.full((3,), 50, **i32)
    lib.moe_verify_drafts(b.p, b.tokens, torch.tensor(b.cu, **i32), b.ua, b.us, accepted, out, draft_probs=b.q, kv_len=length, kv_keep=length)
    assert torch.equal(length, 50 - torch.tensor(b.n, **i32) + accepted)


def test_refusals(lib):
    b = Batch([1, 1], 50)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu, acc, out = torch.tensor(b.cu, **i32), torch.full((2,), 9, **i32), torch.full((2, 2), 9, **i32)
    good = dict(probs=b.p, tokens=b.tokens, cu_new=cu, u_accept=b.ua, u_sample=b.us, accepted=acc, out_tokens=out)
    for kw in (dict(probs=b.p.double()), dict(draft_probs=b.q.half()), dict(draft_probs=b.q[:, :49]), dict(tokens=b.tokens.long()),
               dict(cu_new=cu[:2]), dict(u_accept=b.ua[:3]), dict(u_sample=b.us.cpu()), dict(accepted=acc.long()),
               dict(kv_len=acc, kv_keep=acc[:1]), dict(probs=b.p.t())):
        with pytest.raises(ValueError):
            lib.moe_verify_drafts(**{**good, **kw})
    for kw in (dict(kv_len=acc.clone()), dict(kv_keep=acc.clone())):
        with pytest.raises(lib.MoeError):
            lib.moe_verify_drafts(**{**good, **kw})
    assert (acc == 9).all() and (out == 9).all()
