"""The two ways from a Python call to the library (csrc/binding.cpp and the Python binding) make the
same call: same results, same refusals."""
import pytest
import torch

from tests.test_gpu_kv_pages import State
from tests.test_gpu_verify import Batch

pytestmark = pytest.mark.gpu


@pytest.fixture
def long_way(lib, monkeypatch):
    """Calls `f` the quick way, and then without it."""
    assert lib._native is not None

    def both(f):
        quick = f()
        with monkeypatch.context() as m:
            m.setattr(lib, "_native", None)
            return quick, f()
    return both


def outcome(f):
    try:
        r = f()
        return [t.clone() if torch.is_tensor(t) else t for t in (r if isinstance(r, tuple) else (r,))]
    except (ValueError, RuntimeError) as e:
        return type(e), str(e)


def same(a, b):
    if isinstance(a, tuple):
        return a == b
    return len(a) == len(b) and all(torch.equal(x, y) if torch.is_tensor(x) else x == y for x, y in zip(a, b))


def test_gate(lib, long_way):
    x, w = torch.randn((5, 96), device="cuda").bfloat16(), torch.randn((20, 96), device="cuda").bfloat16()
    out = torch.empty((5, 20), device="cuda")
    err = lib.new_error_word()
    for args in ((x, w, out), (x[:1], w, out[:1]), (x[:, :64], w[:, :64], out), (x[:0], w, out[:0]), (x, w[:1], out[:, :1]),
                 (x.half(), w.half(), out), (x.float(), w, out), (x, w.half(), out), (x.t(), w, out), (x.cpu(), w, out),
                 (x, w, out.cpu()), (x, w, out[:4]), (x[:, :60], w[:, :60], out), (x[:, 1:89], w[:, :88], out)):
        assert same(*long_way(lambda: outcome(lambda: lib.moe_gate(*args, err=err)))), [a.shape for a in args]


def test_route(lib, long_way):
    z, b = torch.randn((6, 16), device="cuda"), torch.randn(16, device="cuda")
    ids, w = torch.empty((6, 3), dtype=torch.int32, device="cuda"), torch.empty((6, 3), device="cuda")
    n = torch.tensor([4], dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(bias=b), dict(bias=b, n_group=4, topk_group=2, flags=7), dict(n_tokens=n, scale=2), dict(flags=99), dict(bias=b[:3]),
               dict(n_tokens=n.long()), dict(n_group=3), dict(scale=float("inf")), dict(bias=b.cpu())):
        assert same(*long_way(lambda: outcome(lambda: lib.moe_route(z, ids, w, **kw)))), kw
    for args in ((z.half(), ids, w), (z[:, ::2], ids, w), (z, ids[:, :2], w), (z[:1], ids[:1], w[:1]), (z.double(), ids, w)):
        assert same(*long_way(lambda: outcome(lambda: lib.moe_route(*args))))


def test_pages(lib, long_way):
    s = State([10, 20, 0], [10, 18, 0], [4, 1, 30], 16, spare=9, max_pages=5)

    def call(**kw):
        d, stack = s.tensors()
        d.update(kw)
        r = outcome(lambda: lib.moe_kv_pages(**d))
        return r if isinstance(r, tuple) else [d[n] for n in ("kv_len", "cu_new", "page_table", "free_list", "free_count_out")] + \
            [d[n] for n in ("seqs", "positions", "slots") if d[n] is not None]

    i32 = dict(dtype=torch.int32, device="cuda")
    for kw in (dict(), dict(kv_keep=None), dict(seqs=None), dict(seqs=None, positions=None, slots=None), dict(page_size=24),
               dict(kv_len=torch.zeros(2, **i32)), dict(slots=torch.zeros(35, **i32)), dict(n_new=torch.zeros(3, dtype=torch.int64, device="cuda")),
               dict(free_count=torch.zeros(1, dtype=torch.int32)), dict(page_size=1 << 40)):
        if kw.get("page_size") == 1 << 40:
            with pytest.raises(Exception):
                lib.moe_kv_pages(**{**s.tensors()[0], **kw})
            continue
        assert same(*long_way(lambda: call(**kw))), list(kw)


def test_verify(lib, long_way):
    b = Batch([2, 0, 3], 50)
    i32 = dict(dtype=torch.int32, device="cuda")
    cu = torch.tensor(b.cu, **i32)

    def call(**kw):
        acc, out, keep = torch.full((3,), -7, **i32), torch.full((3, 4), -7, **i32), torch.full((3,), -7, **i32)
        d = dict(probs=b.p, tokens=b.tokens, cu_new=cu, u_accept=b.ua, u_sample=b.us, accepted=acc, out_tokens=out, draft_probs=b.q,
                 kv_len=torch.full((3,), 9, **i32), kv_keep=keep)
        d.update(kw)
        r = outcome(lambda: lib.moe_verify_drafts(**d))
        return r if isinstance(r, tuple) else [acc, out, keep]

    for kw in (dict(), dict(draft_probs=None), dict(kv_len=None, kv_keep=None), dict(kv_len=None), dict(n_draft=torch.tensor([1, 0, 2], **i32)),
               dict(probs=b.p.half(), draft_probs=b.q.half()), dict(draft_probs=b.q.half()), dict(probs=b.p[:, ::2]), dict(u_sample=b.us[:2]),
               dict(tokens=b.tokens.cpu()), dict(probs=b.p.double())):
        assert same(*long_way(lambda: call(**kw))), list(kw)


def test_the_current_stream_is_taken(lib):
    """On a side stream that waits behind a long copy, the call's output comes after it."""
    x, w = torch.ones((4, 64), device="cuda").bfloat16(), torch.ones((8, 64), device="cuda").bfloat16()
    out, big = torch.zeros((4, 8), device="cuda"), torch.empty(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(8):
            big.add_(1.0)
        x.mul_(2.0)
        lib.moe_gate(x, w, out)
    side.synchronize()
    assert (out == 128.0).all()
