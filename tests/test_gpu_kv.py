"""The paged 8-bit key/value cache on the GPU against plain 64-bit
implementations written here: appending (bit for bit) and attention.

Tolerances.  Appending: the scale is compared exactly; a code may differ by one
step where the fp32 rotation moves a value across a rounding midpoint, so for
rotated keys codes are compared through |q s - x| <= half a step + 2^-20 |x|
against the 64-bit x, and for values (no arithmetic before the rounding) bit for
bit.  Attention, with u = 2^-11 (f16 rounding of a softmax weight): out = sum_j p_j
v_j / sum_j p_j, each p_j off by at most u + 2^-20 * |scores| (fp32 scores of |s| <=
64 and exp2), so |err| <= (u + 2^-14) * (sum_j p_j |v_j| + |out|) + the output
type's rounding 2^-8 |out| (bf16) or 2^-11 |out| (f16) + 1e-7."""
import math

import numpy as np
import pytest
import torch

from tests.gpu_common import Guarded

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def table_of_codes():
    """The 256 E4M3 values in float64."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, (b & 7).astype(np.float64)
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * np.exp2(e.astype(np.float64) - 10))
    v[(b & 127) == 127] = np.nan
    return torch.from_numpy(np.where(b >= 128, -v, v)).cuda()


def to_codes(x):
    """float64 -> the nearest E4M3 value, ties to even, saturating; NaN stays."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 1).clamp(min=-6).double() - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def pow2_scale(amax):
    a = amax.double().clamp(min=float(np.float32(1e-4)))
    return torch.exp2(torch.ceil(torch.log2(a / 448.0)))


class Cache:
    """A paged cache for sequences of the given total and new lengths, with
    random codes, and pages in shuffled order."""

    def __init__(self, total, new, heads, dim, page, layout="hnd", seed=0, poison=False, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.total, self.new, self.heads, self.dim, self.page = total, new, heads, dim, page
        self.pages_of = [-(-t // page) for t in total]
        pool = sum(self.pages_of) + 2
        order = torch.randperm(pool, generator=g)
        self.table = torch.full((len(total), max(self.pages_of + [1]) + 1), 1 << 30, dtype=torch.int32)
        at = 0
        for b, n in enumerate(self.pages_of):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.cu = torch.tensor([sum(new[:i]) for i in range(len(new) + 1)], dtype=torch.int32)
        self.kv_len = torch.tensor(total, dtype=torch.int32)
        self.k, self.v = (self._codes(pool, layout, g) for _ in range(2))
        self.ks, self.vs = (torch.exp2(torch.randint(-8, -5, (pool, heads), generator=g).float()) if scale is None
                            else torch.full((pool, heads), scale) for _ in range(2))
        if poison:     # what no row may see: slots past the lengths and pages of nobody
            for c in (self.k, self.v):
                flat = torch.full_like(c, 0x7F)
                for b, t in enumerate(total):
                    for j in range(t):
                        p = int(self.table[b, j // page])
                        flat[p, :, j % page] = c[p, :, j % page]
                c.copy_(flat)
            for s in (self.ks, self.vs):
                used = set(self.table[self.table < pool].tolist())
                for p in range(pool):
                    if p not in used:
                        s[p] = math.nan
        for name in ("table", "cu", "kv_len", "ks", "vs"):
            setattr(self, name, getattr(self, name).cuda())

    def _codes(self, pool, layout, g):
        shape = (pool, self.heads, self.page, self.dim)
        x = torch.randn(shape, generator=g) * 60
        c = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        if layout == "hnd":
            return c.cuda()
        if layout == "nhd":
            return c.transpose(1, 2).contiguous().cuda().transpose(1, 2)
        buf = torch.zeros((pool, self.heads + 1, self.page, self.dim + 16), dtype=torch.uint8, device="cuda")   # "sliced"
        view = buf[:, 1:, :, 16:]
        view.copy_(c)
        return view

    def args(self):
        return self.k, self.v, self.ks, self.vs, self.table, self.cu, self.kv_len

    def values(self, b, which, upto):
        """float64 [heads, upto, dim] of sequence b."""
        codes, scale = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        ids = self.table[b, : -(-upto // self.page)].long()
        x = table_of_codes()[codes[ids].long()] * scale[ids].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(self.heads, -1, self.dim)[:, :upto]


def angles(n, rot, seed=3):
    th = torch.arange(n)[:, None] * 10000.0 ** (-torch.arange(rot // 2) / max(1, rot // 2))
    return torch.cat([th.cos(), th.sin()], 1).float().cuda()


def rotated(x, cs, pos, rot, interleaved):
    x = x.double().clone()
    if rot:
        c, s = (t.double()[pos][:, None] for t in (cs[:, : rot // 2], cs[:, rot // 2:]))
        ia = torch.arange(rot // 2, device=x.device) * (2 if interleaved else 1)
        ib = ia + (1 if interleaved else rot // 2)
        a, b = x[..., ia].clone(), x[..., ib].clone()
        x[..., ia], x[..., ib] = a * c - b * s, b * c + a * s
    return x


def check_append(lib, total, new, heads, q_heads, dim, page, rot, interleaved, dtype, layout="hnd", seed=1, gain=1.0, scale=None):
    dt = TYPES[dtype]
    c = Cache(total, new, heads, dim, page, layout, seed, scale=scale)
    g = torch.Generator().manual_seed(seed + 50)
    T = sum(new)
    rows = (torch.randn((T, q_heads + 2 * heads, dim), generator=g) * gain).to(dt).cuda()
    q, k, v = rows[:, :q_heads], rows[:, q_heads:q_heads + heads], rows[:, q_heads + heads:]
    cs = angles(max(total) + 1, rot) if rot else None
    before = {n: t.clone() for n, t in (("k", c.k), ("v", c.v), ("ks", c.ks), ("vs", c.vs))}
    qo = Guarded((T, max(q_heads, 1), dim), dt, 0x7E57)
    err = lib.new_error_word()
    lib.moe_kv_append(k, v, *c.args(), cos_sin=cs, flags=lib.MOE_KV_INTERLEAVED if interleaved else 0,
                      q=q if q_heads else None, q_out=qo.t if q_heads else None, err=err)
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)
    assert qo.intact()
    dec = table_of_codes()
    want = {n: t.clone() for n, t in before.items()}
    for b, (t, n) in enumerate(zip(total, new)):
        if n == 0:
            continue
        t0, pos = int(c.cu[b]), torch.arange(t - n, t, device="cuda")
        if q_heads:
            ref = rotated(q[t0:t0 + n], cs, pos, rot, interleaved)
            got = qo.t[t0:t0 + n].double()
            unit = 2.0 ** (-8 if dtype == "bf16" else -11)
            assert ((got - ref).abs() <= unit * 1.001 * ref.abs() + 1e-6 * gain).all()
        for name, x in (("k", rotated(k[t0:t0 + n], cs, pos, rot, interleaved)), ("v", v[t0:t0 + n].double())):
            codes, scales = want[name], want[name + "s"]
            got_c, got_s = getattr(c, name), getattr(c, name + "s")
            for pi in range((t - n) // page, (t - 1) // page + 1):
                p, lo, hi = int(c.table[b, pi]), max(pi * page, t - n), min(pi * page + page, t)
                xs = x[lo - (t - n):hi - (t - n)]                          # [m, heads, dim]
                s = pow2_scale(xs.abs().amax((0, 2)))
                if lo % page:
                    s = torch.maximum(s, before[name + "s"][p].double())
                assert torch.equal(got_s[p].double(), s), (b, pi, name)
                old = dec[before[name][p, :, : lo % page].long()] * (before[name + "s"][p].double() / s)[:, None, None]
                assert torch.equal(dec[got_c[p, :, : lo % page].long()], to_codes(old))
                got = dec[got_c[p, :, lo - pi * page:hi - pi * page].long()]
                y = xs.transpose(0, 1) / s[:, None, None]
                if name == "v" or not rot:
                    assert torch.equal(got, to_codes(y))
                else:
                    _, e = torch.frexp(y)
                    half = torch.exp2((e - 1).clamp(min=-6).double() - 4)
                    assert ((got - y).abs() <= half + 2.0 ** -20 * y.abs().amax()).all()
                codes[p, :, lo - pi * page:hi - pi * page] = got_c[p, :, lo - pi * page:hi - pi * page]
                codes[p, :, : lo % page] = got_c[p, :, : lo % page]
                scales[p] = got_s[p]
    for name in ("k", "v", "ks", "vs"):      # nothing else changed
        assert torch.equal(getattr(c, name), want[name]), name


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page,rot,interleaved,layout", [
    (128, 16, 128, False, "hnd"), (128, 32, 64, True, "nhd"), (128, 64, 96, False, "sliced"), (128, 128, 128, True, "hnd"),
    (64, 16, 32, True, "hnd"), (64, 32, 64, False, "nhd"), (64, 64, 16, False, "hnd"), (64, 128, 48, True, "sliced"),
    (64, 16, 0, False, "hnd")])
def test_append(lib, dtype, dim, page, rot, interleaved, layout):
    check_append(lib, [1, 5, page, page + 1, 300, 77, 40, 3 * page], [1, 0, page, 1, 131, 77, 3, page + 5], 3, 6, dim, page, rot,
                 interleaved, dtype, layout)


@pytest.mark.parametrize("scale", [2.0 ** -22, 2.0 ** -7, 0.013, 64.0])
def test_append_joins_a_page_under_old_scales(lib, scale):
    # far smaller than the new tokens need (the old codes shrink, to zero too), about right, not a power of two, far larger
    check_append(lib, [70, 71, 95, 129], [1, 30, 2, 1], 2, 0, 128, 64, 64, False, "bf16", scale=scale)


def test_append_no_queries_one_head_large_values(lib):
    check_append(lib, [1000], [1], 1, 0, 64, 32, 64, False, "bf16", gain=1e30)
    check_append(lib, [33], [33], 1, 1, 128, 16, 0, False, "f16", gain=1e-4)


def test_append_in_place_queries(lib):
    c = Cache([9], [4], 2, 128, 16)
    cs = angles(16, 128)
    x = torch.randn((4, 6, 128), device="cuda").bfloat16()
    k = torch.randn((4, 2, 128), device="cuda").bfloat16()
    ref = rotated(x, cs, torch.arange(5, 9, device="cuda"), 128, False).bfloat16()
    lib.moe_kv_append(k, k, *c.args(), cos_sin=cs, q=x, q_out=x)
    assert (x.double() - ref.double()).abs().max() <= 2.0 ** -7 * ref.abs().max().double()


@pytest.mark.parametrize("n", [3, 16])
def test_append_non_finite_values(lib, n):
    # infinities saturate and take no part in the page's maximum, NaN is kept
    c = Cache([n], [n], 1, 64, 16)
    v = torch.ones((n, 1, 64), device="cuda").bfloat16()
    v[1, 0, 3], v[1, 0, 4], v[2, 0, 5] = math.inf, -math.inf, math.nan
    lib.moe_kv_append(v, v, *c.args())
    p = int(c.table[0, 0])
    for codes, s in ((c.k, c.ks), (c.v, c.vs)):
        assert float(s[p, 0]) == 2.0 ** -8
        row = codes[p, 0, :3].cpu()
        assert int(row[1, 3]) == 0x7E and int(row[1, 4]) == 0xFE and int(row[2, 5]) == 0x7F
        assert (row[0] == 0x78).all()          # 1 / 2^-8 = 256


@pytest.mark.parametrize("what,bits", [("page", 4), ("negative page", 4), ("long", 1), ("short", 4), ("rows", 4), ("angles", 4)])
def test_append_flags_bad_descriptors(lib, what, bits):
    c = Cache([40, 20], [5, 4], 2, 64, 16)
    cs = angles(64, 64)
    if what == "page":
        c.table[0, 2] = c.k.shape[0]
    elif what == "negative page":
        c.table[0, 2] = -1
    elif what == "long":
        c.table = c.table[:, :2].contiguous()
    elif what == "short":
        c.kv_len[0] = 4
    elif what == "rows":
        c.cu[0] = -3
    else:
        cs = cs[:38].contiguous()
    x = torch.randn((9, 2, 64), device="cuda").bfloat16()
    q = torch.zeros_like(x)
    before = c.k.clone(), c.ks.clone()
    err = lib.new_error_word()
    lib.moe_kv_append(x, x, *c.args(), cos_sin=cs, q=x, q_out=q, err=err)
    assert lib.moe_read_device_status(err)[1] & bits
    own = c.table[0, : c.table.shape[1]].long()
    own = own[(own >= 0) & (own < c.k.shape[0])]
    assert torch.equal(c.k[own], before[0][own]) and torch.equal(c.ks[own], before[1][own])


# ---------------------------------------------------------------- attention
def plain_attention(c, q, sm_scale, window, softcap, full):
    """float64 out, sum_j p_j |v_j| and lse, row by row of a sequence."""
    T, Hq, D = q.shape
    G = Hq // c.heads
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device="cuda")
    mag, lse = torch.zeros_like(out), torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b, (t, n) in enumerate(zip(c.total, c.new)):
        if not n or not t:
            continue
        t0 = int(c.cu[b])
        k, v = c.values(b, "k", t), c.values(b, "v", t)
        qs = q[t0:t0 + n].double().view(n, c.heads, G, D)
        s = torch.einsum("ihgd,hjd->hgij", qs, k) * sm_scale
        if softcap:
            s = softcap * torch.tanh(s / softcap)
        j, pos = torch.arange(t, device="cuda"), torch.arange(t - n, t, device="cuda")[:, None]
        seen = torch.ones((n, t), dtype=torch.bool, device="cuda")
        if not full:
            seen = j <= pos
        if window:
            seen &= j > pos - window
        s = torch.where(seen, s, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, 0.0, m))
        l = p.sum(-1, keepdim=True)
        safe = torch.where(l > 0, l, 1.0)
        # a weight of an unseen token is no number: keep its value out of the product
        for i in range(n):
            cols = seen[i]
            pi = (p / safe)[:, :, i, cols]
            out[t0 + i] = torch.einsum("hgj,hjd->hgd", pi, v[:, cols]).reshape(Hq, D)
            mag[t0 + i] = torch.einsum("hgj,hjd->hgd", pi, v[:, cols].abs()).reshape(Hq, D)
        lse[t0:t0 + n] = (m + torch.log(l))[..., 0].permute(2, 0, 1).reshape(n, Hq)
    return out, mag, lse


def check_attention(lib, total, new, heads, q_heads, dim, page, dtype="bf16", layout="hnd", window=0, softcap=0.0, full=False,
                    seed=1, q_gain=1.0, max_q=None, cache=None, workspace=None):
    dt = TYPES[dtype]
    c = cache or Cache(total, new, heads, dim, page, layout, seed, poison=True)
    T = sum(new)
    rows = (torch.randn((T, q_heads + 2, dim), generator=torch.Generator().manual_seed(seed + 9)) * q_gain).to(dt).cuda()
    q = rows[:, 1:-1]
    sm_scale = 1.0 / math.sqrt(dim)
    out = Guarded((T, q_heads, dim), dt, 0x7E57)
    lse = Guarded((T, q_heads), torch.float32, 0x7FC12345)
    err = lib.new_error_word()
    flags = lib.MOE_KV_FULL if full else 0
    d = lib.make_kv_attention_desc(q, *c.args(), out.t, sm_scale, max(new) if max_q is None else max_q, window, softcap, flags)
    ws = lib.alloc_kv_workspace(d) if workspace is None else workspace
    for _ in range(2):                               # a workspace serves call after call
        lib.moe_kv_attention(q, *c.args(), out.t, ws, sm_scale, max_q=max(new) if max_q is None else max_q, window=window,
                             softcap=softcap, flags=flags, lse=lse.t, err=err)
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)
    assert out.intact() and lse.intact()
    ref, mag, ref_lse = plain_attention(c, q, sm_scale, window, softcap, full)
    got = out.t.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    u = 2.0 ** -11 + 2.0 ** -14
    bound = u * (mag + ref.abs()) + 2.0 ** (-8 if dtype == "bf16" else -11) * ref.abs() + 1e-7
    worst = ((got - ref).abs() / bound).nan_to_num(0).max().item() if T else 0.0
    assert worst <= 1.0, worst
    same = (lse.t.double() - ref_lse).abs() <= 2.0 ** -16 * (ref_lse.abs() + 16) * max(1.0, q_gain)
    assert (same | (lse.t.double() == ref_lse) | (torch.isnan(ref_lse) & torch.isnan(lse.t.double()))).all()
    return got


DECODE = [1, 2, 15, 16, 17, 63, 64, 65, 100, 129, 1000, 0]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("dim,page", [(128, 16), (128, 64), (128, 128), (64, 16), (64, 32), (64, 128)])
@pytest.mark.parametrize("heads,q_heads", [(2, 2), (1, 5), (2, 16)])
def test_attention_decode(lib, dtype, dim, page, heads, q_heads):
    total = DECODE[:-1]
    check_attention(lib, total, [1] * len(total), heads, q_heads, dim, page, dtype)


@pytest.mark.parametrize("layout", ["nhd", "sliced"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_strides(lib, dim, layout):
    check_attention(lib, [200, 77, 33], [1, 1, 1], 3, 6, dim, 32, layout=layout)
    check_attention(lib, [200, 177, 33], [40, 111, 7], 3, 6, dim, 32, layout=layout)


@pytest.mark.parametrize("new", [2, 3, 4, 7, 8, 16, 17, 33])
@pytest.mark.parametrize("heads,q_heads", [(2, 2), (1, 7), (2, 8)])
def test_attention_draft(lib, new, heads, q_heads):
    check_attention(lib, [new, new + 1, 64 + new, 131, 500], [new, 1, new, new, 0], heads, q_heads, 128, 64, "f16")


@pytest.mark.parametrize("dim,page,dtype", [(128, 16, "bf16"), (128, 128, "f16"), (64, 64, "bf16"), (64, 32, "f16")])
@pytest.mark.parametrize("heads,q_heads", [(2, 2), (1, 4), (1, 12)])
def test_attention_prompts(lib, dim, page, dtype, heads, q_heads):
    check_attention(lib, [1, 127, 128, 129, 300, 700], [1, 127, 100, 129, 300, 257], heads, q_heads, dim, page, dtype)


@pytest.mark.parametrize("new", [1, 3, 150])
@pytest.mark.parametrize("window,softcap", [(1, 0.0), (16, 0.0), (100, 5.0), (5000, 0.0), (0, 30.0), (0, 0.5)])
def test_attention_window_and_cap(lib, new, window, softcap):
    check_attention(lib, [new, new + 63, new + 64, 700], [new] * 4, 2, 6, 128, 32, window=window, softcap=softcap, q_gain=3.0)
    check_attention(lib, [new, 333], [new] * 2, 1, 1, 64, 64, "f16", window=window, softcap=softcap)


@pytest.mark.parametrize("new", [1, 4, 200])
def test_attention_full(lib, new):
    check_attention(lib, [new, 65, 300][: 2 if new > 65 else 3] if new < 65 else [new, 300], [new] * (3 if new < 65 else 2), 2, 8,
                    128, 32, full=True)


def test_attention_unknown_and_mixed_lengths(lib):
    # decode steps, drafts and chunks in one call; max_q unknown
    check_attention(lib, [900, 20, 64, 500, 31, 129], [1, 5, 0, 200, 31, 2], 2, 8, 128, 16, max_q=0)
    check_attention(lib, [900, 20, 64, 500, 31, 129], [1, 5, 0, 200, 31, 2], 4, 4, 64, 64, "f16")


def test_attention_many_sequences(lib):
    total = [1 + (37 * i) % 91 for i in range(700)]
    check_attention(lib, total, [1] * 700, 1, 2, 64, 16)


def test_attention_long_sequence_splits(lib):
    check_attention(lib, [20011, 3], [1, 1], 1, 8, 128, 64)
    check_attention(lib, [20011, 5000], [4, 2], 1, 4, 64, 128, "f16")
    check_attention(lib, [9000, 5000], [20, 12], 1, 8, 128, 128, "f16")


@pytest.mark.parametrize("dim,window,softcap", [(128, 600, 50.0), (128, 600, 0.0), (64, 600, 0.0), (128, 0, 0.0), (64, 130, 20.0)])
def test_attention_prompts_fill_the_gpu(lib, dim, window, softcap):
    # more CTAs than SMs, the two tiles of each with different keys: a tile's work does
    # not disturb the other's, whichever is ahead; again and again the same bits
    new = [1380, 777, 300]
    c = Cache([n + 300 for n in new], new, 4, dim, 64)
    q = (torch.randn((sum(new), 32, dim), generator=torch.Generator().manual_seed(3)) * 2).bfloat16().cuda()
    out = torch.empty_like(q)
    sm_scale = dim ** -0.5
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, sm_scale, max(new)))
    first = None
    for _ in range(10):
        out.fill_(math.nan)
        lib.moe_kv_attention(q, *c.args(), out, ws, sm_scale, max_q=max(new), window=window, softcap=softcap)
        first = out.clone() if first is None else first
        assert torch.equal(out, first)
    # against the plain form in 32 bits, row block by row block (the 64-bit one above is for small cases)
    for b, n in enumerate(new):
        t0, t = int(c.cu[b]), c.total[b]
        j, pos = torch.arange(t, device="cuda"), torch.arange(t - n, t, device="cuda")[:, None]
        seen = (j <= pos) & ((j > pos - window) if window else (j >= 0))
        for h in range(4):
            k, v = (c.values(b, w, t)[h].float() for w in ("k", "v"))
            s = torch.einsum("igd,jd->gij", q[t0:t0 + n, 8 * h:8 * h + 8].float(), k) * sm_scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            p = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            ref, mag = torch.einsum("gij,jd->igd", p, v), torch.einsum("gij,jd->igd", p, v.abs())
            err = (first[t0:t0 + n, 8 * h:8 * h + 8].float() - ref).abs()
            assert (err <= (2.0 ** -11 + 2.0 ** -14) * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-5).all()


@pytest.mark.parametrize("dim,dtype,window,softcap,full", [
    (128, "bf16", 0, 0.0, False), (64, "f16", 3000, 0.0, False), (128, "f16", 0, 20.0, False), (64, "bf16", 0, 0.0, True),
    (128, "bf16", 700, 0.0, False)])
def test_attention_many_rows_split_over_keys(lib, dim, dtype, window, softcap, full):
    # more rows than the decode kernel takes, too few for all SMs; runs of keys that some rows or a whole tile do not see
    check_attention(lib, [7013, 40, 900, 2500], [40, 40, 33, 9], 1, 4, dim, 64, dtype, window=window, softcap=softcap, full=full)
    check_attention(lib, [5000], [300], 1, 1, dim, 32, dtype, window=window, softcap=softcap, full=full)


def test_attention_nan_in_a_split(lib):
    c = Cache([6000], [50], 1, 64, 16)
    for j, d in ((5990, 5), (3000, 9), (20, 63)):
        c.v[int(c.table[0, j // 16]), 0, j % 16, d] = 0x7F
    got = check_attention(lib, [6000], [50], 1, 2, 64, 16, cache=c)
    assert torch.isnan(got[:, :, 9]).all() and torch.isnan(got[:, :, 63]).all()
    assert torch.isnan(got[40:, :, 5]).all() and not torch.isnan(got[:40, :, 5]).any()


def test_attention_sharp_and_large_scores(lib):
    # one token takes all the weight; scores of some hundreds
    check_attention(lib, [300, 70], [1, 40], 2, 4, 128, 32, q_gain=8.0)


@pytest.mark.parametrize("new", [1, 30])
def test_attention_zero_and_tiny_queries(lib, new):
    check_attention(lib, [77], [new], 1, 2, 64, 16, q_gain=0.0)
    check_attention(lib, [77], [new], 1, 2, 64, 16, q_gain=1e-20)


@pytest.mark.parametrize("new", [1, 20])
def test_attention_scales_far_apart(lib, new):
    c = Cache([200], [new], 2, 64, 16)
    c.vs.copy_(torch.exp2(torch.randint(-22, 10, c.vs.shape, generator=torch.Generator().manual_seed(1)).float()))
    c.ks.mul_(torch.rand(c.ks.shape, generator=torch.Generator().manual_seed(2)).cuda() + 0.5)
    check_attention(lib, [200], [new], 2, 4, 64, 16, cache=c)


@pytest.mark.parametrize("new,q_heads,window", [(3, 4, 0), (40, 4, 0), (3, 4, 9), (40, 4, 9), (200, 2, 0), (200, 2, 50)])
def test_attention_nan_reaches_only_rows_that_see_it(lib, new, q_heads, window):
    c = Cache([new + 60], [new], 2, 64, 16)
    for j, h, d in ((new + 59, 0, 5), (60 + new // 2, 1, 9), (59, 1, 63), (10, 0, 0)):
        c.v[int(c.table[0, j // 16]), h, j % 16, d] = 0x7F
    got = check_attention(lib, [new + 60], [new], 2, q_heads, 64, 16, window=window, cache=c)
    assert torch.isnan(got).any() and not torch.isnan(got).all()


def test_attention_nan_keys_and_queries(lib):
    c = Cache([90, 90], [30, 1], 1, 64, 16)
    c.k[int(c.table[0, 5]), 0, 3, 7] = 0xFF          # token 83 of sequence 0: rows 23 .. 29
    q = torch.randn((31, 2, 64), device="cuda").bfloat16()
    q[30, 1, 0] = math.nan
    out = torch.zeros_like(q)
    d = lib.make_kv_attention_desc(q, *c.args(), out, 0.125, 30)
    lib.moe_kv_attention(q, *c.args(), out, lib.alloc_kv_workspace(d), 0.125, max_q=30)
    bad = torch.isnan(out).all(-1)
    assert bad[23:30].all() and not torch.isnan(out[:23]).any()
    assert bad[30, 1] and not torch.isnan(out[30, 0]).any()


def test_attention_repeats_bit_for_bit(lib):
    a = check_attention(lib, [5000, 700, 64], [1, 1, 1], 2, 8, 128, 32)
    b = check_attention(lib, [5000, 700, 64], [1, 1, 1], 2, 8, 128, 32)
    assert torch.equal(a, b)


def test_attention_other_stream_and_graph(lib):
    c = Cache([600, 40], [1, 1], 2, 128, 32, poison=True)
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    out, ref = torch.zeros_like(q), torch.zeros_like(q)
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 0.1, 1))
    lib.moe_kv_attention(q, *c.args(), ref, ws, 0.1, max_q=1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    lib.moe_kv_attention(q, *c.args(), out, ws, 0.1, max_q=1, stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    k = torch.randn((2, 2, 128), device="cuda").bfloat16()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.moe_kv_append(k, k, *c.args())
        lib.moe_kv_attention(q, *c.args(), out, ws, 0.1, max_q=1)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    first = out.clone()
    lib.moe_kv_attention(q, *c.args(), ref, ws, 0.1, max_q=1)
    torch.cuda.synchronize()
    assert torch.equal(first, ref)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("what,bits", [("page", 4), ("negative page", 4), ("long", 1), ("short", 4), ("rows", 4), ("max_q", 1)])
def test_attention_flags_bad_descriptors(lib, what, bits, new):
    c = Cache([90, 45], [new, new], 2, 64, 16)
    max_q = new
    if what == "page":
        c.table[0, 4] = c.k.shape[0]
    elif what == "negative page":
        c.table[0, 4] = -7
    elif what == "long":
        c.table = c.table[:, :5].contiguous()
    elif what == "short":
        c.kv_len[0] = new - 1
    elif what == "rows":
        c.cu[0] = -3
    else:
        if new == 1:
            pytest.skip("a sequence with new tokens has at least one")
        max_q = new - 1
    q = torch.randn((2 * new, 4, 64), device="cuda").bfloat16()
    out = torch.zeros_like(q)
    err = lib.new_error_word()
    ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 0.1, max_q))
    lib.moe_kv_attention(q, *c.args(), out, ws, 0.1, max_q=max_q, err=err)
    assert lib.moe_read_device_status(err)[1] & bits
    # the workspace is fit for the next call
    good = Cache([90, 45], [new, new], 2, 64, 16)
    check_attention(lib, [90, 45], [new, new], 2, 4, 64, 16, cache=good, workspace=ws)


@pytest.mark.parametrize("new", [1, 40])
def test_offsets_past_32_bits(lib, new):
    # pages a gigabyte apart: the last one's bytes lie past 2^32
    c = Cache([64], [new], 2, 64, 16, scale=1.0)
    assert c.pages_of == [4]
    far = [torch.zeros((5 << 30) + (1 << 20), dtype=torch.uint8, device="cuda").as_strided((6, 2, 16, 64), (1 << 30, 1024, 64, 1))
           for _ in range(2)]
    c.table[0, :4] = torch.tensor([1, 3, 4, 5], dtype=torch.int32)
    c.k, c.v = far
    c.ks, c.vs = (torch.ones((6, 2), device="cuda") for _ in range(2))
    x = torch.randn((64, 2, 64), generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    whole = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    lib.moe_kv_append(x, x, c.k, c.v, c.ks, c.vs, c.table, whole, c.kv_len)
    ref = to_codes(x.double().transpose(0, 1) / c.ks[c.table[0, :4].long()].double().repeat_interleave(16, 0).t()[:, :, None])
    got = table_of_codes()[c.k[c.table[0, :4].long()].long()].transpose(0, 1).reshape(2, 64, 64)
    assert torch.equal(got, ref)
    check_attention(lib, [64], [new], 2, 4, 64, 16, cache=c)


def test_append_many_new_tokens_in_a_batch_of_single_ones(lib):
    # few new tokens on average: the kernel for single tokens meets whole pages
    check_append(lib, [200] + [50 + i for i in range(60)], [131] + [1] * 60, 2, 4, 128, 64, 128, False, "bf16")
    check_append(lib, [200] + [50 + i for i in range(60)], [131] + [2] * 60, 3, 0, 64, 16, 32, True, "f16")


def test_append_then_attend_matches_plain_layer(lib):
    # a decode loop of a few steps: what was appended is what attention reads
    heads, q_heads, dim, page = 2, 6, 64, 16
    c = Cache([40, 17], [7, 17], heads, dim, page)
    cs = angles(64, 64)
    kv_len = c.kv_len.clone()
    new = [7, 17]
    for step in range(3):
        T = sum(new)
        x = torch.randn((T, q_heads + 2 * heads, dim), generator=torch.Generator().manual_seed(step)).bfloat16().cuda()
        q = torch.empty((T, q_heads, dim), dtype=torch.bfloat16, device="cuda")
        c.cu = torch.tensor([0, new[0], T], dtype=torch.int32, device="cuda")
        c.kv_len, c.new, c.total = kv_len, new, kv_len.tolist()
        lib.moe_kv_append(x[:, q_heads:q_heads + heads], x[:, q_heads + heads:], *c.args(), cos_sin=cs, q=x[:, :q_heads], q_out=q)
        out = torch.empty_like(q)
        ws = lib.alloc_kv_workspace(lib.make_kv_attention_desc(q, *c.args(), out, 0.125, max(new)))
        lib.moe_kv_attention(q, *c.args(), out, ws, 0.125, max_q=max(new))
        ref, mag, _ = plain_attention(c, q, 0.125, 0, 0.0, False)
        assert ((out.double() - ref).abs() <= (2.0 ** -11 + 2.0 ** -14) * (mag + ref.abs()) + 2.0 ** -8 * ref.abs() + 1e-7).all()
        new = [1, 1]
        kv_len = kv_len + 1
