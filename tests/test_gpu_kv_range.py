"""The cache operators at the ends of their ranges.

The tolerance of attention is that of test_gpu_kv (a softmax weight off by at most 2^-11
+ 2^-14, the output's rounding, 1e-7)."""
import math
import random

import pytest
import torch

from tests.test_gpu_kv import Cache, angles, check_append, check_attention, plain_attention, rotated

pytestmark = pytest.mark.gpu

U = 2.0 ** -11 + 2.0 ** -14


@pytest.mark.parametrize("new", [1, 40, 150])
@pytest.mark.parametrize("power", [70, -70])
def test_attention_key_scales_far_from_one(lib, new, power):
    # queries as large as the keys are small, or the other way round: scores of a few units
    t = new + 300
    c = Cache([t], [new], 2, 64, 16)
    c.ks.mul_(2.0 ** -power)
    T, q_heads = new, 4
    q = (torch.randn((T, q_heads, 64), generator=torch.Generator().manual_seed(5)) * 2.0 ** power).bfloat16().cuda()
    out, lse = torch.zeros_like(q), torch.zeros((T, q_heads), device="cuda")
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 0.125, new))
    lib.moe_kv_attention(q, *c.args(), out, ws, 0.125, max_q=new, lse=lse)
    ref, mag, ref_lse = plain_attention(c, q, 0.125, 0, 0.0, False)
    assert ((out.double() - ref).abs() <= U * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-7).all()
    assert ((lse.double() - ref_lse).abs() <= 2.0 ** -16 * (ref_lse.abs() + 16)).all()


@pytest.mark.parametrize("new", [1, 3, 40])
@pytest.mark.parametrize("softcap", [63.0, 65.0, 300.0, 1e4, 1e6, 1e9, 1e30])
def test_attention_large_caps(lib, new, softcap):
    # tanh(s / cap) is nearly s / cap: what is lost must be small beside s, not beside the cap
    check_attention(lib, [new + 80, 300], [new, new], 2, 4, 128, 32, softcap=softcap, q_gain=3.0)
    check_attention(lib, [new + 500], [new], 1, 2, 64, 16, "f16", softcap=softcap, window=100, q_gain=10.0)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("softcap", [1e-3, 1e-20, 1e-42])
@pytest.mark.parametrize("q_gain", [0.0, 1.0])
def test_attention_small_caps(lib, new, softcap, q_gain):
    # all scores are next to nothing: the mean of the values
    check_attention(lib, [new + 80, 300], [new, new], 2, 4, 128, 32, softcap=softcap, q_gain=q_gain)


def one_long_row_beside_many(lib, new, dim, dtype, page=16):
    """Sequences whose first keys take nearly all of the weight but hold zeros: the output
    is what a thousand others bring, each at 78.5 * 2^-24 of the largest weight."""
    heads, batch, t = 8, 20 if new > 32 else 64, 1024
    c = Cache([t] * batch, [new] * batch, heads, dim, page, scale=1.0)
    c.k.zero_()
    c.v.copy_(torch.randint(0x30, 0x38, c.v.shape, device="cuda", dtype=torch.uint8))     # 0.5 .. 0.9375, all of one sign
    for b in range(batch):
        for j in range(0, 64, 16):                # keys 0, 16, 32, 48: one for each warp of a decode CTA
            p = int(c.table[b, j // page])
            c.k[p, :, j % page, 0] = 0x38         # 1.0
            c.v[p, :, j % page] = 0
    c.ks.fill_(1.0)
    c.vs.fill_(1.0)
    q = torch.zeros((batch * new, heads, dim))
    q[..., 0] = math.log(2.0) * (24 - math.log2(78.5))
    q = q.to(dtype).cuda()
    out = torch.zeros_like(q)
    err = lib.new_error_word()
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 1.0, new))
    lib.moe_kv_attention(q, *c.args(), out, ws, 1.0, max_q=new, flags=lib.MOE_KV_FULL, err=err)
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)
    ref, mag, _ = plain_attention(c, q, 1.0, 0, 0.0, True)
    bound = U * (mag + ref.abs()) + (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -11) * ref.abs() + 1e-7
    return ((out.double() - ref).abs() / bound).max().item()


@pytest.mark.parametrize("new", [1, 33])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_one_dominant_key(lib, new, dim):
    assert one_long_row_beside_many(lib, new, dim, torch.float16) <= 1.0


@pytest.mark.parametrize("new", [1, 5, 40, 200])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 16), (128, 64)])
@pytest.mark.parametrize("low,high", [(-22, 9), (9, -22), (-20, -7), (0, -13)])
def test_attention_small_pages_under_large_ones(lib, new, dim, page, low, high):
    # runs of 64 keys have one V scale and the other by turns; those with the larger one
    # hold zeros in half of the dimensions, where the output is the others' alone
    heads, batch, t = (8, 64, 1024) if new <= 5 else (2, 1, new + 700)      # several runs for every warp
    c = Cache([t] * batch, [new] * batch, heads, dim, page, scale=2.0 ** -7)
    table = c.table[:, : c.pages_of[0]].long()
    turn = (torch.arange(table.shape[1], device="cuda") * page // 64) % 2 == 1
    one, other = table[:, ~turn].flatten(), table[:, turn].flatten()
    c.vs[one], c.vs[other] = 1.25 * 2.0 ** low, 1.5 * 2.0 ** high
    c.v[other if high > low else one, :, :, : dim // 2] = 0
    check_attention(lib, c.total, c.new, heads, 2 * heads, dim, page, q_gain=0.5, cache=c)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_scales_of_neighbouring_pages(lib, new):
    # each 16 keys another scale, within one step of the kernel for prompts
    c = Cache([new + 500], [new], 2, 128, 16, scale=2.0 ** -7)
    c.vs.copy_(torch.exp2(torch.randint(-11, 12, c.vs.shape, generator=torch.Generator().manual_seed(2)).float()))
    c.v[(c.vs > 1)[:, 0], :, :, :64] = 0
    check_attention(lib, [new + 500], [new], 2, 4, 128, 16, q_gain=0.5, cache=c)


@pytest.mark.parametrize("new", [1, 40])
def test_attention_smallest_scales_over_many_keys(lib, new):
    # a million keys of equal weight under V scales below the smallest that count: the sum of
    # weights over scales stays in range
    t, page, dim = 1 << 20, 128, 64
    pages = t // page
    k = torch.zeros((pages, 1, page, dim), dtype=torch.uint8, device="cuda")
    v = torch.randint(0x30, 0x40, k.shape, dtype=torch.uint8, device="cuda")
    ks, vs = torch.ones((pages, 1), device="cuda"), torch.full((pages, 1), 2.0 ** -100, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    cu, kv_len = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, new], [t]))
    q = torch.ones((new, 2, dim), dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    args = (q, k, v, ks, vs, table, cu, kv_len, out)
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(*args, 0.125, new))
    lib.moe_kv_attention(*args, ws, 0.125, max_q=new, flags=lib.MOE_KV_FULL)
    ref = v.view(torch.float8_e4m3fn).float().mean((0, 1, 2)).double() * 2.0 ** -80
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref).all()


@pytest.mark.parametrize("heads,q_heads,new", [(1, 64, 1), (1, 128, 2), (1, 64, 9), (2, 96, 7), (1, 20, 13), (1, 17, 1)])
def test_attention_wide_groups(lib, heads, q_heads, new):
    # units and groups of rows that end inside a token
    check_attention(lib, [new + 300, 77], [new, min(new, 3)], heads, q_heads, 128, 32)
    check_attention(lib, [new + 300, 77], [new, min(new, 3)], heads, q_heads, 64, 64, "f16", window=40)


def test_sliced_page_table(lib):
    c = Cache([200, 90, 33], [5, 40, 1], 2, 64, 16)
    wide = torch.full((3, 40), -5, dtype=torch.int32, device="cuda")
    wide[:, 7:7 + c.table.shape[1]] = c.table
    c.table = wide[:, 7:7 + c.table.shape[1]]
    x = torch.randn((46, 2, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    err = lib.new_error_word()
    lib.moe_kv_append(x, x, *c.args(), err=err)
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)
    check_attention(lib, c.total, c.new, 2, 4, 64, 16, cache=c)


@pytest.mark.parametrize("new,window", [(1, 1), (1, 50), (3, 17), (9, 64)])
def test_attention_many_sequences_under_a_window(lib, new, window):
    total = [new + (37 * i) % 191 for i in range(150)]
    check_attention(lib, total, [new if i % 7 else 0 for i in range(150)], 2, 8, 64, 16, window=window)


def test_attention_as_many_sequences_as_the_limits_allow(lib):
    # 2^20 sequences of 64 kv heads, nearly all without new tokens
    batch, heads, dim, page = 1 << 20, 64, 64, 16
    n, t = 34, 40
    c = Cache([t], [n], heads, dim, page)
    at = batch - 7                                       # the one that has some
    table = torch.full((batch, 3), -1, dtype=torch.int32, device="cuda")
    table[at] = c.table[0, :3]
    cu, kv_len = torch.zeros(batch + 1, dtype=torch.int32, device="cuda"), torch.zeros(batch, dtype=torch.int32, device="cuda")
    cu[at + 1:], kv_len[at] = n, t
    q = torch.randn((n, heads, dim), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    args = (q, c.k, c.v, c.ks, c.vs, table, cu, kv_len, out)
    err = lib.new_error_word()
    lib.moe_kv_attention(*args, lib.alloc_kv_workspace(lib.make_kv_attention_desc(*args, 0.125)), 0.125, err=err)
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)
    ref, mag, _ = plain_attention(c, q, 0.125, 0, 0.0, False)
    assert ((out.double() - ref).abs() <= U * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-7).all()


@pytest.mark.parametrize("heads,q_heads", [(1, 1), (2, 10), (1, 16)])
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_attention_mixed_batches(lib, heads, q_heads, seed):
    # steps, drafts, chunks and idle sequences in any order: every sequence's rows are found
    r = random.Random(seed)
    new = [r.choice([0, 1, 1, 1, 2, 5, r.randint(6, 40), r.randint(30, 300)]) for _ in range(r.choice([3, 40, 90]))]
    check_attention(lib, [n + r.randint(0, 90) for n in new], new, heads, q_heads, 64, 16, max_q=r.choice([0, None, 5000]))


def test_attention_max_q_far_above_the_rows(lib):
    check_attention(lib, [50, 7, 3], [1, 1, 0], 1, 4, 64, 16, max_q=1000)


def test_append_wide_groups(lib):
    check_append(lib, [300, 40], [40, 3], 1, 33, 128, 32, 128, False, "bf16")
    check_append(lib, [300, 40, 9], [1, 1, 1], 1, 64, 64, 16, 64, True, "f16")


# ---------------------------------------------------------------- sequences that are skipped
def appended(lib, c, cs, q_heads=2, seed=3):
    """One append; what was there before, the rows, the queries' output and the status bits."""
    T = int(c.cu.max())
    x = torch.randn((T, 2 * c.heads + q_heads, c.dim), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
    q = x[:, :q_heads]
    out = torch.full((T, q_heads, c.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    err = lib.new_error_word()
    lib.moe_kv_append(x[:, q_heads:q_heads + c.heads], x[:, q_heads + c.heads:], *c.args(), cos_sin=cs, q=q, q_out=out, err=err)
    return before, x, out, lib.moe_read_device_status(err)[1]


@pytest.mark.parametrize("batch", [2, 40])          # the kernel for prompts, the one for few tokens
@pytest.mark.parametrize("what,bit", [("long", 1), ("short", 4)])
def test_append_skips_a_bad_sequence_whole(lib, batch, what, bit):
    # 20 new tokens that fall on a page inside the table and on one past it; or more new tokens than tokens
    c = Cache([40] + [17] * (batch - 1), [20] + [1] * (batch - 1), 2, 64, 16, scale=2.0 ** -9)
    if what == "long":
        c.table = c.table[:, :2].contiguous()
    else:
        c.kv_len[0] = 19
    cs = angles(64, 64)
    before, x, out, status = appended(lib, c, cs)
    assert status == bit
    own = c.table[0, : min(c.table.shape[1], 3)].long()
    for now, was in zip((c.k, c.v, c.ks, c.vs), before):
        assert torch.equal(now[own], was[own])
    assert (out[:20] == 7).all()
    # the others are served
    ref = rotated(x[20:, :2], cs, torch.full((batch - 1,), 16, device="cuda"), 64, False)
    assert ((out[20:].double() - ref).abs() <= 2.0 ** -8 * 1.001 * ref.abs() + 1e-6).all()
    page = c.table[1:, 1].long()
    assert (c.vs[page] == torch.exp2(torch.ceil(torch.log2(x[20:, 4:].double().abs().amax(2) / 448)))).all()


@pytest.mark.parametrize("cu", [[0, 100, 50, 150], [0, 30, -3, 150], [-5, 20, 30, 150], [60, 60, 59, 150], [0, 150, 0, 150]])
def test_offsets_that_decrease_are_told(lib, cu):
    # whatever the units' search lands on; nothing outside the rows and pages is touched
    T = 150
    c = Cache([160, 160, 160], [1, 1, 1], 2, 64, 16)
    c.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    spare = [p for p in range(c.k.shape[0]) if p not in set(c.table.flatten().tolist())]
    assert spare
    for batch_of_units in (1, 60):
        if batch_of_units > 1:                      # a batch with few tokens a sequence: the other kernel
            c.cu = torch.cat([c.cu, torch.full((57,), 150, dtype=torch.int32, device="cuda")])
            c.kv_len = torch.cat([c.kv_len, c.kv_len.new_zeros(57)])
            c.table = torch.cat([c.table, c.table.new_full((57, c.table.shape[1]), -1)])
        x = torch.randn((T, 2, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
        before = c.k[spare].clone(), c.ks[spare].clone()
        q = torch.zeros_like(x)
        err = lib.new_error_word()
        lib.moe_kv_append(x, x, *c.args(), cos_sin=angles(160, 64), q=x, q_out=q, err=err)
        assert lib.moe_read_device_status(err)[1] & 4
        assert torch.equal(c.k[spare], before[0]) and torch.equal(c.ks[spare], before[1])
        out = torch.zeros_like(x)
        err = lib.new_error_word()
        ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(x, *c.args(), out, 0.125))
        lib.moe_kv_attention(x, *c.args(), out, ws, 0.125, err=err)
        assert lib.moe_read_device_status(err)[1] & 4


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what,bit", [("long", 1), ("short", 4), ("max_q", 1)])
def test_attention_skips_a_bad_sequence_alone(lib, new, what, bit):
    total, news = [90, 45 + new, 300], [new, new + 2, new]
    c = Cache(total, news, 2, 64, 16)
    max_q = new + 2
    if what == "long":
        c.table[1] = -1
        c.kv_len[1] = 16 * c.table.shape[1] + 1
    elif what == "short":
        c.kv_len[1] = new + 1
    else:
        max_q = new + 1
    T = sum(news)
    q = torch.randn((T, 4, 64), generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full((T, 4), 7.0, device="cuda")
    err = lib.new_error_word()
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 0.125, max_q))
    lib.moe_kv_attention(q, *c.args(), out, ws, 0.125, max_q=max_q, lse=lse, err=err)
    assert lib.moe_read_device_status(err)[1] == bit
    mine = torch.zeros(T, dtype=torch.bool, device="cuda")
    mine[new:2 * new + 2] = True
    assert (out[mine] == 7).all() and (lse[mine] == 7).all()
    good = Cache(total, news, 2, 64, 16)               # the same codes, as they were
    good.total, good.new = [total[0], 0, total[2]], [new, 0, new]
    ref, mag, _ = plain_attention(good, q, 0.125, 0, 0.0, False)
    ok = (out.double() - ref).abs() <= U * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-7
    assert ok[~mine].all()
