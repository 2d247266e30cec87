"""Refusals of the calls that decide what a serving step works on, which need no GPU:
descriptors are checked on the host before any CUDA call."""
import ctypes
import math
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import fp8_grouped_expert_x128_gb300 as lib
    return lib


def gate(moe, **kw):
    d = dict(x=256, w=1 << 20, logits=1 << 24, T=5, x_ld=64, w_ld=64, logits_ld=10, E=10, H=64, dtype=0)
    return moe._lib.moe_gate(ctypes.byref(moe.moe_gate_desc(**{**d, **kw})), None)


def route(moe, **kw):
    d = dict(logits=256, topk_ids=1 << 20, topk_w=1 << 24, T=5, logits_ld=16, ids_ld=4, w_ld=4, scale=1.0, E=16, k=4, n_group=4,
             topk_group=2, dtype=2)
    return moe._lib.moe_route(ctypes.byref(moe.moe_route_desc(**{**d, **kw})), None)


def pages(moe, **kw):
    names = ("kv_old", "kv_keep", "n_new", "page_table", "free_list", "free_count", "kv_len", "cu_new", "free_count_out", "seqs",
             "positions", "slots")
    d = {n: (i + 1) << 20 for i, n in enumerate(names)}
    d.update(table_ld=8, free_capacity=100, rows=64, batch=4, max_pages=8, page_size=16)
    return moe._lib.moe_kv_pages(ctypes.byref(moe.moe_kv_pages_desc(**{**d, **kw})), None)


def verify(moe, **kw):
    names = ("probs", "draft_probs", "tokens", "cu_new", "n_draft", "u_accept", "u_sample", "kv_len", "accepted", "out_tokens", "kv_keep")
    d = {n: (i + 1) << 20 for i, n in enumerate(names)}
    d.update(T=9, vocab=100, p_ld=100, q_ld=100, out_ld=4, batch=3, max_out=4, dtype=2)
    return moe._lib.moe_verify_drafts(ctypes.byref(moe.moe_verify_desc(**{**d, **kw})), None)


@pytest.mark.parametrize("bad,rc", [
    (dict(x=None), -1), (dict(w=None), -1), (dict(logits=None), -1), (dict(x=264), -1), (dict(w=(1 << 20) + 2), -1),
    (dict(logits=(1 << 24) + 2), -1), (dict(T=-1), -1), (dict(E=0), -1), (dict(H=0), -1), (dict(H=60), -1), (dict(x_ld=56), -1),
    (dict(x_ld=68), -1), (dict(w_ld=60), -1), (dict(logits_ld=9), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1), (dict(flags=1), -1),
    (dict(E=1025, logits_ld=2000), -2), (dict(H=1 << 21, x_ld=1 << 21, w_ld=1 << 21), -2), (dict(T=(1 << 24) + 1), -2),
    (dict(x_ld=1 << 31), -2), (dict(logits_ld=1 << 31), -2),
    (dict(logits=256 + 512), -1), (dict(logits=(1 << 20) - 4 * 49), -1)])      # on x, into w
def test_gate_refusals(moe, bad, rc):
    assert gate(moe, **bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(logits=None), -1), (dict(topk_ids=None), -1), (dict(topk_w=None), -1), (dict(logits=258), -1), (dict(logits=257, dtype=0), -1),
    (dict(topk_ids=2), -1), (dict(topk_w=2), -1), (dict(bias=2), -1), (dict(n_tokens=2), -1), (dict(T=-1), -1), (dict(E=0), -1),
    (dict(E=1025), -1), (dict(k=0), -1), (dict(k=33), -1), (dict(k=9), -1), (dict(n_group=0), -1), (dict(n_group=3), -1),
    (dict(topk_group=0), -1), (dict(topk_group=5), -1), (dict(logits_ld=15), -1), (dict(ids_ld=3), -1), (dict(w_ld=3), -1),
    (dict(dtype=3), -1), (dict(flags=8), -1), (dict(scale=math.inf), -1), (dict(scale=math.nan), -1),
    (dict(E=128, logits_ld=128, n_group=64), -2), (dict(T=(1 << 24) + 1), -2), (dict(logits_ld=1 << 31), -2)])
def test_route_refusals(moe, bad, rc):
    assert route(moe, **bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(kv_old=None), -1), (dict(n_new=None), -1), (dict(page_table=None), -1), (dict(free_list=None), -1), (dict(free_count=None), -1),
    (dict(kv_len=None), -1), (dict(cu_new=None), -1), (dict(free_count_out=None), -1), (dict(kv_old=(1 << 20) + 2), -1),
    (dict(slots=(12 << 20) + 4), -1), (dict(seqs=(10 << 20) + 2), -1), (dict(batch=-1), -1), (dict(max_pages=-1), -1), (dict(rows=-1), -1),
    (dict(free_capacity=-1), -1), (dict(table_ld=7), -1), (dict(flags=1), -1), (dict(page_size=8), -2), (dict(page_size=48), -2),
    (dict(batch=8193), -2), (dict(max_pages=1 << 28, table_ld=1 << 28), -2), (dict(rows=(1 << 30) + 1), -2),
    (dict(free_capacity=(1 << 30) + 1), -2), (dict(table_ld=1 << 31), -2),
    # outputs on inputs and on each other: lengths and counts need two buffers
    (dict(kv_len=1 << 20), -1), (dict(kv_len=(1 << 20) + 12), -1), (dict(free_count_out=6 << 20), -1), (dict(cu_new=(3 << 20) - 4), -1),
    (dict(positions=10 << 20), -1), (dict(kv_len=(2 << 20)), -1), (dict(free_list=(4 << 20) + 4 * 31), -1)])
def test_pages_refusals(moe, bad, rc):
    assert pages(moe, **bad) == rc


@pytest.mark.parametrize("bad,rc", [
    (dict(probs=None), -1), (dict(tokens=None), -1), (dict(cu_new=None), -1), (dict(u_accept=None), -1), (dict(u_sample=None), -1),
    (dict(accepted=None), -1), (dict(out_tokens=None), -1), (dict(kv_len=None), -1), (dict(kv_keep=None), -1),
    (dict(probs=(1 << 20) + 2), -1), (dict(draft_probs=1, dtype=0), -1), (dict(tokens=2), -1), (dict(n_draft=2), -1), (dict(T=-1), -1),
    (dict(batch=-1), -1), (dict(vocab=0), -1), (dict(max_out=0), -1), (dict(max_out=1025, out_ld=2000), -1), (dict(p_ld=99), -1),
    (dict(q_ld=99), -1), (dict(out_ld=3), -1), (dict(dtype=3), -1), (dict(flags=1), -1),
    (dict(vocab=(1 << 24) + 1, p_ld=1 << 25, q_ld=1 << 25), -2), (dict(batch=(1 << 20) + 1), -2), (dict(T=(1 << 24) + 1), -2),
    (dict(p_ld=1 << 31), -2)])
def test_verify_refusals(moe, bad, rc):
    assert verify(moe, **bad) == rc


def test_null_descriptors(moe):
    for name in ("moe_gate", "moe_route", "moe_kv_pages", "moe_verify_drafts"):
        assert getattr(moe._lib, name)(None, None) == -1


def test_no_tokens_launch_nothing(moe):
    assert gate(moe, T=0, x=None, logits=None) == 0
    assert route(moe, T=0, logits=None, topk_ids=None, topk_w=None) == 0
    assert verify(moe, batch=0, cu_new=None, u_sample=None, accepted=None, out_tokens=None) == 0


def test_binding_refuses_cpu_tensors(moe):
    x, f, i = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_gate(x, x, f)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_route(f, i, f[:, :2])
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_kv_pages(n, n, i, n, n[:1], 16, n, n, n[:1])
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_verify_drafts(f, n, n, f[:, 0], f[:, 0], n, i)


def test_descriptors_match_the_header(moe):
    """Field names and order of the binding's structures are the header's."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "moe_fp8.h")).read(), flags=re.S)
    for name in ("moe_gate_desc", "moe_route_desc", "moe_kv_pages_desc", "moe_verify_desc"):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
        skip = {"const", "float", "int32_t", "int64_t", "void"}
        fields = [w for decl in body.split(";") for w in re.findall(r"\w+", decl) if w not in skip]
        assert fields == [f[0] for f in getattr(moe, name)._fields_], name


def test_packed_descriptors_have_the_structures_layout(moe):
    """The bytes that the calls pack are the structures' own."""
    for pack, cls in ((moe._gate_pack, moe.moe_gate_desc), (moe._route_pack, moe.moe_route_desc),
                      (moe._kv_pages_pack, moe.moe_kv_pages_desc), (moe._verify_pack, moe.moe_verify_desc)):
        values = tuple(range(1, 1 + len(cls._fields_)))
        assert pack(*values) == bytes(cls(*values)), cls


def test_quick_way_is_there_and_leaves_the_telling_to_python(moe):
    """_binding.so is built beside the library; it answers 1 for whatever it would not take as it is."""
    assert moe._native is not None
    x, f, i = torch.zeros((2, 64), dtype=torch.bfloat16), torch.zeros((2, 8)), torch.zeros((2, 2), dtype=torch.int32)
    n = torch.zeros(2, dtype=torch.int32)
    assert moe._native.gate(x, x, f, None) == 1                                # tensors of the CPU
    assert moe._native.gate(None, 3, "x", ()) == 1
    assert moe._native.gate() == 1
    assert moe._native.route(f, i, f, None, None, 1, 1, 1.0, 0) == 1
    assert moe._native.route(f, i, f, None, None, "1", 1 << 40, None, 0) == 1
    assert moe._native.kv_pages(n, n, i, n, n, 16, n, n, n, None, None, None, None, None) == 1
    assert moe._native.verify(f, n, n, f, f, n, i, None, None, None, None, None) == 1


@pytest.mark.parametrize("bad", [
    dict(topk_ids=256), dict(topk_ids=256 + 4 * 79), dict(topk_w=256 + 64), dict(topk_w=(1 << 20) + 76), dict(topk_ids=(1 << 24) - 76),
    dict(bias=(1 << 20) - 60), dict(n_tokens=1 << 24), dict(topk_w=(1 << 20) + 4, ids_ld=8, w_ld=8)])
def test_route_outputs_on_inputs_and_each_other(moe, bad):
    assert route(moe, **bad) == -1


@pytest.mark.parametrize("bad", [
    dict(accepted=3 << 20), dict(out_tokens=1 << 20), dict(out_tokens=(2 << 20) + 4 * 899), dict(kv_keep=9 << 20), dict(accepted=(4 << 20) + 12),
    dict(kv_keep=(8 << 20) + 4), dict(accepted=8 << 20), dict(out_tokens=(11 << 20) - 44), dict(accepted=(10 << 20) + 44),
    dict(kv_keep=(6 << 20) + 32), dict(accepted=(7 << 20) - 8)])
def test_verify_outputs_on_inputs_and_each_other(moe, bad):
    assert verify(moe, **bad) == -1
