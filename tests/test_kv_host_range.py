"""Limits of the key/value cache calls, checked on the host before any CUDA call."""
import types

import pytest
import torch

from tests.test_kv_host import append, attention, cache, moe  # noqa: F401


@pytest.mark.parametrize("page_size", [16, 32, 64, 128])
def test_positions_do_not_wrap_around(moe, page_size):  # noqa: F811
    """The kernels look pages up ahead of a sequence's end: up to 32 tiles of 64 keys and a
    step in the one for few rows, 64 groups of 16 keys and a block in the one for many.  A
    length next to 2^31 would turn such a position negative, and the lookup, which only
    compares it with the length, would read in front of the page table."""
    longest = ((1 << 31) - (1 << 16)) // page_size
    ahead = max(32 * 64 + 64, (64 + 8) * 16 + 128)
    assert longest * page_size + ahead < 1 << 31
    for pages in (longest + 1, ((1 << 31) - 1) // page_size):
        assert append(moe, cache(moe, page_size=page_size, max_pages=pages)) == -2
        assert attention(moe, cache(moe, page_size=page_size, max_pages=pages))[0] == -2


class OnGpu:
    """As much of a tensor on some GPU as the binding looks at; there is no memory behind it."""

    def __init__(self, shape, dtype, device):
        self.meta, self.device_number = torch.empty(shape, dtype=dtype, device="meta"), device

    def get_device(self):
        return self.device_number

    def data_ptr(self):
        return 4096

    def __getattr__(self, name):
        return getattr(self.meta, name)


def calls(moe, device, workspace=None):  # noqa: F811
    def t(*shape, dtype):
        return OnGpu(shape, dtype, device)

    cache = [t(4, 2, 16, 64, dtype=torch.uint8) for _ in range(2)] + [t(4, 2, dtype=torch.float32) for _ in range(2)]
    cache += [t(1, 2, dtype=torch.int32), t(2, dtype=torch.int32), t(1, dtype=torch.int32)]
    q, ws = t(1, 2, 64, dtype=torch.bfloat16), workspace or t(1 << 20, dtype=torch.uint8)
    return [lambda **kw: moe.moe_kv_append(q, q, *cache, **kw),
            lambda **kw: moe.moe_kv_attention(q, *cache, q, ws, 1.0, **kw),
            lambda **kw: moe.make_kv_attention_desc(q, *cache, q, 1.0, **kw)]


class Library:
    """In the library's place: counts the calls that get through."""

    def __init__(self):
        self.through = 0

    def __getattr__(self, name):
        def call(*args):
            self.through += 1
            return 0
        return call


def test_tensors_of_another_gpu_than_the_current_one_are_refused(moe, monkeypatch):  # noqa: F811
    """The library launches on the current GPU: with the handle of another one's stream (0 for
    every GPU's default stream) it would use foreign pointers there."""
    library = Library()
    monkeypatch.setattr(moe, "_lib", library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    for call in calls(moe, 1):
        with pytest.raises(ValueError, match="GPU 1, but GPU 0 is current"):
            call()
    append_call, attention_call, describe = calls(moe, 0)
    other, own = (types.SimpleNamespace(device_index=d, cuda_stream=77) for d in (1, 0))
    for call in (append_call, attention_call):
        with pytest.raises(ValueError, match="stream: on GPU 1"):
            call(stream=other)
    assert library.through == 0
    append_call()
    append_call(stream=own)
    attention_call()
    attention_call(stream=own)
    describe()
    assert library.through == 4


def test_a_workspace_that_only_looks_large_is_refused(moe, monkeypatch):  # noqa: F811
    """An expanded tensor counts bytes that it does not have."""
    library = Library()
    monkeypatch.setattr(moe, "_lib", library)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    one = OnGpu((1,), torch.uint8, 0)
    one.meta = one.meta.expand(1 << 20)
    assert one.nbytes == 1 << 20
    with pytest.raises(ValueError, match="workspace"):
        calls(moe, 0, one)[1]()
    assert library.through == 0


def test_kernels_for_large_caps_keep_the_register_split(moe, tmp_path):  # noqa: F811
    """They hand registers between warpgroups like those without: 96 a thread at launch (the
    launch refuses anything else), next to no spills."""
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
        if "kv_prefill_bend_kernel" not in current:
            continue
        m = re.search(r"(\d+) bytes spill stores", line)
        assert m is None or int(m.group(1)) <= 64, line
        m = re.search(r"Used (\d+) registers", line)
        if m:
            assert int(m.group(1)) == 96, current
            seen += 1
    assert seen == 4            # two types x two dimensions
