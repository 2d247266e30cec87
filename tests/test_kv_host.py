"""Refusals of the key/value cache calls that need no GPU: descriptors are
checked on the host before any CUDA call."""
import ctypes
import math

import pytest
import torch


@pytest.fixture(scope="module")
def moe():
    import __graft_entry__
    __graft_entry__._builder().build()
    import fp8_grouped_expert_x128_gb300 as lib
    return lib


def cache(moe, **kw):
    d = dict(k=256, v=256, k_scale=256, v_scale=256, page_table=256, cu_new=256, kv_len=256, k_page_ld=4096, k_head_ld=1024,
             k_slot_ld=64, v_page_ld=4096, v_head_ld=1024, v_slot_ld=64, table_ld=8, pages=10, batch=2, max_pages=8,
             page_size=16, kv_heads=4, dim=64, dtype=0)
    return moe.moe_kv_cache(**{**d, **kw})


def append(moe, c=None, **kw):
    d = dict(cache=c or cache(moe), T=5, k=256, v=256, q=256, q_out=256, cos_sin=256, k_token_ld=256, k_head_ld=64,
             v_token_ld=256, v_head_ld=64, q_token_ld=512, q_head_ld=64, qo_token_ld=512, qo_head_ld=64, q_heads=8,
             rot_dim=64, max_pos=100)
    return moe._lib.moe_kv_append(ctypes.byref(moe.moe_kv_append_desc(**{**d, **kw})), None)


def attention(moe, c=None, ws=256, nbytes=1 << 30, **kw):
    d = dict(cache=c or cache(moe), T=5, q=256, out=256, q_token_ld=512, q_head_ld=64, o_token_ld=512, o_head_ld=64,
             sm_scale=0.125, q_heads=8, max_q=4)
    desc = moe.moe_kv_attention_desc(**{**d, **kw})
    return (moe._lib.moe_kv_attention(ctypes.byref(desc), ws, nbytes, None), moe.moe_kv_attention_workspace_size(desc))


@pytest.mark.parametrize("bad,rc", [
    (dict(dim=80), -2), (dict(dim=256), -2), (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=256), -2),
    (dict(dtype=2), -1), (dict(kv_heads=0), -1), (dict(batch=-1), -1), (dict(pages=-1), -1), (dict(k_page_ld=4100), -1),
    (dict(k_slot_ld=-64), -1), (dict(v_head_ld=8), -1), (dict(k=None), -1), (dict(v=264), -1), (dict(k_scale=None), -1),
    (dict(page_table=None), -1), (dict(kv_len=None), -1), (dict(cu_new=None), -1), (dict(table_ld=-1), -1),
    (dict(max_pages=(1 << 31) - 1), -2), (dict(batch=1 << 21), -2)])
def test_cache_descriptor_refusals(moe, bad, rc):
    assert append(moe, cache(moe, **bad)) == rc
    assert attention(moe, cache(moe, **bad))[0] == rc


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(k=None), dict(v=264), dict(rot_dim=8), dict(rot_dim=80), dict(rot_dim=-16), dict(cos_sin=None),
    dict(cos_sin=260), dict(flags=2), dict(q_out=None), dict(q=None), dict(q_heads=0), dict(k_token_ld=100), dict(q_head_ld=4),
    dict(qo_token_ld=-8), dict(max_pos=-1)])
def test_append_refusals(moe, bad):
    assert append(moe, **bad) == -1


@pytest.mark.parametrize("bad", [
    dict(T=-1), dict(q=None), dict(out=None), dict(out=264), dict(q_heads=6), dict(q_heads=0), dict(max_q=-1), dict(window=-1),
    dict(window=4, flags=1), dict(flags=2), dict(softcap=-1.0), dict(softcap=math.inf), dict(sm_scale=math.nan),
    dict(q_token_ld=4), dict(o_head_ld=-8), dict(ws=None), dict(ws=128), dict(nbytes=0)])
def test_attention_refusals(moe, bad):
    assert attention(moe, **bad)[0] == -1


def test_null_descriptors_and_sizes(moe):
    assert moe._lib.moe_kv_append(None, None) == -1
    assert moe._lib.moe_kv_attention(None, 256, 256, None) == -1
    assert moe._lib.moe_kv_attention_workspace_size(None) == 0
    assert attention(moe, q_heads=6)[1] == 0
    assert attention(moe, T=1 << 25)[1] == 0


def test_no_tokens_launch_nothing(moe):
    assert append(moe, T=0, k=None, v=None, q=None, q_out=None, q_heads=0, cos_sin=None) == 0
    assert attention(moe, T=0, q=None, out=None, ws=None)[0] == 0
    empty = cache(moe, batch=0, k=None, page_table=None, cu_new=None, kv_len=None)
    assert append(moe, empty) == 0
    assert attention(moe, empty)[0] == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(moe):
    kc = torch.zeros((4, 2, 16, 64), dtype=torch.uint8)
    sc = torch.ones((4, 2))
    table, cu, ln = torch.zeros((1, 2), dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_kv_append(q, q, kc, kc, sc, sc, table, cu, ln)
    with pytest.raises(ValueError, match="CUDA"):
        moe.moe_kv_attention(q, kc, kc, sc, sc, table, cu, ln, q, torch.zeros(1024, dtype=torch.uint8), 1.0)


def test_descriptors_match_the_header(moe):
    """Field names and order of the binding's structures are the header's."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_fp8.h")).read(), flags=re.S)
    for name in ("moe_kv_cache", "moe_kv_append_desc", "moe_kv_attention_desc"):
        body = re.search(r"typedef struct %s \{(.*?)\} %s;" % (name, name), text, flags=re.S).group(1)
        fields = []
        for decl in body.split(";"):
            words = re.findall(r"\w+", decl)
            skip = {"const", "uint8_t", "float", "int32_t", "int64_t", "void", "moe_kv_cache"}
            fields += [w for w in words if w not in skip]
        assert fields == [f[0] for f in getattr(moe, name)._fields_], name


def test_packed_descriptors_have_the_structures_layout(moe):
    """The bytes that the calls pack are the structures' own."""
    c = tuple(range(1, 22))
    for pack, cls, n in ((moe._kv_append_pack, moe.moe_kv_append_desc, 19), (moe._kv_attention_pack, moe.moe_kv_attention_desc, 15)):
        rest = tuple(range(30, 30 + n))
        assert pack(*c, *rest) == bytes(cls(c, *rest))


def test_prefill_kernel_compiles_to_its_register_split(moe, tmp_path):
    """The kernel hands registers between warpgroups with setmaxnreg: the split counts
    on a launch allocation of exactly 96 registers for its 640 threads (the launch
    refuses anything else), and its loops on next to no spills."""
    import os
    import re
    import shutil
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    src = os.path.join(root, "fp8_grouped_expert_x128_gb300", "csrc", "kv_prefill.cu")
    r = subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17", "--expt-relaxed-constexpr",
                        "-I", os.path.join(root, "include"), "-Xptxas", "-v", "-c", src, "-o", str(tmp_path / "p.o")],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    current, seen = "", 0
    for line in r.stderr.splitlines():
        m = re.search(r"Compiling entry function '(\S+)'", line)
        current = m.group(1) if m else current
        if "kv_prefill_kernel" not in current:
            continue
        m = re.search(r"(\d+) bytes spill stores", line)
        assert m is None or int(m.group(1)) <= 64, line
        m = re.search(r"Used (\d+) registers", line)
        if m:
            assert int(m.group(1)) == 96, current
            seen += 1
    assert seen == 8            # two types x two dimensions x with and without the cap
