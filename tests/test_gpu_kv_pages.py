"""moe_kv_pages against a plain allocator."""
import random

import pytest
import torch

from tests.gpu_common import Guarded

pytestmark = pytest.mark.gpu


class State:
    """A paged cache's host copy: sequences with pages, and a free list."""

    def __init__(self, old, keep, new, P, spare, max_pages, seed=0, rows=None, capacity=None):
        r = random.Random(seed)
        held = [-(-o // P) if 0 <= o <= max_pages * P else 0 for o in old]
        ids = list(range(sum(held) + spare))
        r.shuffle(ids)
        self.P, self.max_pages, self.old, self.keep, self.new = P, max_pages, old, keep, new
        self.table = []
        for h in held:
            self.table.append([ids.pop() for _ in range(h)])
        self.free = ids
        self.capacity = sum(held) + spare if capacity is None else capacity
        self.rows = sum(n for n in new if n > 0) if rows is None else rows

    def plain(self, count=None):
        """(kv_len, cu_new, tables, free list, seqs, positions, slots, bits) after the call."""
        P, most, bits = self.P, self.max_pages * self.P, 0
        up = lambda x: -(-x // P)  # noqa: E731
        f = len(self.free) if count is None else count
        list_ok = 0 <= f <= self.capacity
        bad = [not list_ok or o < 0 or n < 0 or o > most or k < 0 or k > o for o, k, n in zip(self.old, self.keep, self.new)]
        B = len(self.old)
        want = [k + n for k, n in zip(self.keep, self.new)]
        wide = [not x and w > most for x, w in zip(bad, want)]
        room = f + sum(max(0, up(self.old[b]) - up(want[b])) for b in range(B) if not bad[b] and not wide[b])
        rows = pages = 0
        total = []
        for b in range(B):
            if bad[b]:
                total.append(None)
                bits |= 4
                continue
            ok = not wide[b]
            if ok:
                rows += self.new[b]
                ok = self.new[b] == 0 or rows <= self.rows
            if ok:
                need = max(0, up(want[b]) - up(self.old[b]))
                pages += need
                ok = need == 0 or pages <= room
            if not ok:
                bits |= 1
            total.append(want[b] if ok else self.keep[b])
        back = sum(max(0, up(self.old[b]) - up(t)) for b, t in enumerate(total) if t is not None)
        if not list_ok or f + back > self.capacity:
            return list(self.old), [0] * (B + 1), self.table, None, [-1] * self.rows, [-1] * self.rows, [-1] * self.rows, bits | 4
        table, free = [list(t) for t in self.table], list(self.free)
        for b, t in enumerate(total):
            if t is not None and up(t) < len(table[b]):
                free += table[b][up(t):]
                table[b] = table[b][:up(t)]
        for b, t in enumerate(total):
            if t is not None:
                while len(table[b]) < up(t):
                    table[b].append(free.pop())
        cu, seqs, pos, slots = [0], [], [], []
        for b, t in enumerate(total):
            n = 0 if t is None else t - self.keep[b]
            cu.append(cu[-1] + n)
            for p in range(self.keep[b], self.keep[b] + n):
                seqs.append(b)
                pos.append(p)
                slots.append(table[b][p // P] * P + p % P)
        tail = [-1] * (self.rows - len(seqs))
        length = [self.old[b] if t is None else t for b, t in enumerate(total)]
        return length, cu, table, free, seqs + tail, pos + tail, slots + tail, bits

    def tensors(self, pad=0):
        i32 = dict(dtype=torch.int32, device="cuda")
        B = len(self.old)
        table = torch.full((B, self.max_pages + pad), -9, **i32)
        for b, t in enumerate(self.table):
            table[b, : len(t)] = torch.tensor(t, **i32)
        stack = Guarded((self.capacity,), torch.int32, -8)
        stack.t[: len(self.free)] = torch.tensor(self.free, **i32)
        d = dict(kv_old=torch.tensor(self.old, **i32), n_new=torch.tensor(self.new, **i32), page_table=table[:, : self.max_pages],
                 free_list=stack.t, free_count=torch.tensor([len(self.free)], **i32), page_size=self.P,
                 kv_len=Guarded((B,), torch.int32, -7).t, cu_new=Guarded((B + 1,), torch.int32, -7).t,
                 free_count_out=torch.full((1,), -7, **i32), kv_keep=torch.tensor(self.keep, **i32),
                 seqs=torch.full((self.rows,), -7, **i32), positions=torch.full((self.rows,), -7, **i32),
                 slots=torch.full((self.rows,), -7, dtype=torch.int64, device="cuda"))
        return d, stack

    def check(self, lib, pad=0, count=None, status=None, **kw):
        d, stack = self.tensors(pad)
        if count is not None:
            d["free_count"].fill_(count)
        d.update(kw)
        err = lib.new_error_word()
        lib.moe_kv_pages(**d, err=err)
        length, cu, table, free, seqs, pos, slots, bits = self.plain(count)
        assert d["kv_len"].tolist() == length
        assert d["cu_new"].tolist() == cu
        for name, want in (("seqs", seqs), ("positions", pos), ("slots", slots)):
            if d[name] is not None:
                assert d[name].tolist() == want, name
        before = self.tensors(pad)[0]["page_table"].tolist()
        for b, row in enumerate(d["page_table"].tolist()):
            assert row[: len(table[b])] == table[b], b
            assert row[len(table[b]):] == before[b][len(table[b]):]           # entries past the pages: untouched
        if free is None:
            assert d["free_count_out"].item() == d["free_count"].item()
            assert stack.t.tolist() == self.tensors()[1].t.tolist()
        else:
            assert d["free_count_out"].item() == len(free)
            assert stack.t.tolist()[: len(free)] == free
            everything = sorted(sum(table, []) + free)
            assert everything == sorted(set(everything))                      # no page twice
        assert stack.intact()
        assert lib.moe_read_device_status(err)[1] == (bits if status is None else status)
        return d


def drawn(seed, batch, P, longest, new, faults=False):
    r = random.Random(seed)
    old, keep, gain = [], [], []
    for _ in range(batch):
        o = r.choice([0, P, r.randint(0, longest), r.randint(0, longest)])
        k = r.choice([o, o, max(0, o - r.randint(0, 6)), 0, r.randint(0, o)])
        n = r.choice([0, 1, 1, r.randint(0, new)])
        if faults and r.random() < 0.15:
            o, k, n = r.choice([(-1, 0, 1), (5, 6, 1), (5, -1, 1), (5, 5, -1), (1 << 30, 5, 1), (5, 5, (1 << 31) - 1), (-(1 << 31), 0, 0)])
        old.append(o)
        keep.append(k)
        gain.append(n)
    return old, keep, gain


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("batch,longest,new", [(1, 100, 1), (3, 200, 40), (33, 500, 9), (300, 300, 5), (513, 64, 3), (7, 3000, 5000), (2000, 40, 40)])
def test_steps(lib, P, batch, longest, new):
    for seed in range(3):
        old, keep, gain = drawn(seed * 1000 + batch, batch, P, longest, new)
        most = -(-(longest + new + P) // P)
        State(old, keep, gain, P, spare=batch * (new // P + 2), max_pages=most, seed=seed).check(lib, pad=seed)
        State(old, keep, gain, P, spare=sum(gain) // P // 3, max_pages=most, seed=seed, rows=sum(gain) + 11).check(lib)   # pages run out
        State(old, keep, gain, P, spare=batch * (new // P + 2), max_pages=most, seed=seed, rows=sum(gain) // 2).check(lib)  # rows run out


@pytest.mark.parametrize("batch", [4, 70, 600])
def test_faults_leave_their_sequences_alone(lib, batch):
    for seed in range(6):
        old, keep, gain = drawn(seed, batch, 16, 200, 30, faults=True)
        gain = [g if g < 1 << 20 else (1 << 31) - 1 for g in gain]
        rows = sum(g for g in gain if 0 < g < 1 << 20)
        State(old, keep, gain, 16, spare=batch * 3, max_pages=15, seed=seed, rows=rows).check(lib)


def test_everything_at_once(lib):
    """No sequences, no rows, empty sequences, a cache that fills and empties whole."""
    State([], [], [], 16, spare=5, max_pages=4, rows=0).check(lib)
    State([], [], [], 16, spare=5, max_pages=4, rows=7).check(lib)
    State([], [], [], 16, spare=5, max_pages=4, rows=5000).check(lib)
    State([3], [3], [1], 16, spare=5, max_pages=4, rows=200001).check(lib)
    State([0, 0, 0], [0, 0, 0], [0, 0, 0], 16, spare=0, max_pages=4).check(lib)
    State([64] * 50, [0] * 50, [0] * 50, 16, spare=0, max_pages=4).check(lib)             # all end
    State([0] * 50, [0] * 50, [64] * 50, 16, spare=200, max_pages=4).check(lib)           # all begin, to the last page
    State([0] * 50, [0] * 50, [64] * 50, 16, spare=199, max_pages=4).check(lib)           # one page short
    State([64] * 50, [0] * 50, [64] * 50, 16, spare=0, max_pages=4).check(lib)            # all replaced
    State([64] * 25 + [0] * 25, [0] * 25 + [0] * 25, [0] * 25 + [64] * 25, 16, spare=0, max_pages=4).check(lib)   # pages change hands
    State([64, 0], [64, 0], [1, 1], 16, spare=9, max_pages=4).check(lib)                  # a full table row


@pytest.mark.parametrize("count", [-1, 41, 1 << 30, -(1 << 31)])
def test_a_broken_free_count_moves_nothing(lib, count):
    State([64, 10, 0], [20, 10, 0], [3, 30, 64], 16, spare=36, max_pages=5).check(lib, count=count)


def test_a_list_without_room_moves_nothing(lib):
    State([64, 10], [0, 10], [0, 3], 16, spare=8, max_pages=5, capacity=9).check(lib)


@pytest.mark.parametrize("given", [(), ("seqs",), ("positions",), ("slots",), ("seqs", "slots")])
def test_row_tensors_are_optional(lib, given):
    s = State([10, 20, 0], [10, 18, 0], [4, 1, 30], 16, spare=9, max_pages=5)
    s.check(lib, **{n: None for n in ("seqs", "positions", "slots") if n not in given})


def test_without_kv_keep(lib):
    s = State([10, 16, 31], [10, 16, 31], [4, 1, 2], 16, spare=9, max_pages=5)
    s.check(lib, kv_keep=None)


def test_largest_batch_and_long_sequences(lib):
    r = random.Random(1)
    B = 8192
    old = [r.randint(0, 60) for _ in range(B)]
    State(old, [max(0, o - r.randint(0, 30)) for o in old], [r.randint(0, 20) for _ in range(B)], 16, spare=B, max_pages=6).check(lib)
    State([1 << 20, 3], [(1 << 20) - 5, 3], [200000, 1], 16, spare=13000, max_pages=80000).check(lib)
    State([1 << 20, 3], [0, 3], [0, 1], 16, spare=3, max_pages=80000).check(lib)


def test_slots_past_32_bits(lib):
    s = State([0], [0], [40], 128, spare=1, max_pages=3)
    d, _ = s.tensors()
    d["free_list"][0] = 2 ** 31 - 1
    lib.moe_kv_pages(**d)
    assert d["slots"].tolist() == [(2 ** 31 - 1) * 128 + i for i in range(40)]


def test_steps_in_a_replayed_graph(lib):
    """Two captured steps that hand lengths and counts back and forth, twenty times."""
    P, B = 16, 9
    old = [5 * b for b in range(B)]
    s = State(old, old, [3] * B, P, spare=B * 12, max_pages=14)
    d, stack = s.tensors()
    other = dict(d, kv_old=d["kv_len"], kv_len=d["kv_old"], free_count=d["free_count_out"], free_count_out=d["free_count"], kv_keep=None)
    d["kv_keep"] = None
    err = lib.new_error_word()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.moe_kv_pages(**d, err=err)
        lib.moe_kv_pages(**other, err=err)
    length = torch.tensor(old)
    for i in range(20):
        graph.replay()
        length += 6
        assert d["kv_old"].cpu().tolist() == length.tolist()
    held = [t[: -(-n // P)] for t, n in zip(d["page_table"].tolist(), length.tolist())]
    used = sum(held, []) + stack.t.tolist()[: d["free_count"].item()]
    assert sorted(used) == list(range(len(used)))
    assert lib.moe_read_device_status(err) == (lib.MOE_OK, 0)


def test_refusals(lib):
    d, _ = State([10, 20], [10, 20], [4, 1], 16, spare=9, max_pages=5).tensors()
    for kw in (dict(kv_old=d["kv_old"].long()), dict(n_new=d["n_new"][:1]), dict(kv_len=d["kv_len"].cpu()), dict(slots=d["slots"].int()),
               dict(page_table=d["page_table"].t().contiguous().t()), dict(seqs=d["seqs"][:-1]), dict(cu_new=d["cu_new"][:-1]),
               dict(free_count=torch.zeros(2, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            lib.moe_kv_pages(**{**d, **kw})
    for kw in (dict(kv_len=d["kv_old"]), dict(free_count_out=d["free_count"]), dict(page_size=24), dict(positions=d["seqs"])):
        with pytest.raises(lib.MoeError):
            lib.moe_kv_pages(**{**d, **kw})
    assert (d["kv_len"] == -7).all()
