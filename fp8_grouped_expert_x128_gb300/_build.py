"""Builds libmoe_fp8.so in-tree for sm_103a with nvcc (no cmake, no torch
extension machinery): every .cu under csrc/ is compiled in parallel, then
linked into one shared library next to this file.  Beside it, with g++ and the
headers of Python and torch, _binding.so: the quick way from Python to some of the
calls (csrc/binding.cpp).  Where that does not build, the calls go the longer way.

    python fp8_grouped_expert_x128_gb300/_build.py [--force] [--verbose] [--ptxas-info]
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import importlib.metadata
import importlib.util
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe_fp8.so")
BINDING = os.path.join(PKG, "_binding.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe_fp8.so")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return hdrs + [os.path.abspath(__file__)]


def _stale(out: str, ins: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(i) > t for i in ins)


def _installed(name: str) -> str:
    try:
        return importlib.metadata.version(name)
    except importlib.metadata.PackageNotFoundError:
        return ""


def _build_binding(cuda: str, force: bool) -> None:
    """_binding.so, if its headers are there.  It holds torch's and Python's layouts beside the library's, so one of
    other versions, or of an older source, is taken away before it is built again."""
    src, stamp = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.txt")
    spec = importlib.util.find_spec("torch")
    gxx = os.environ.get("CXX") or shutil.which("g++")
    cmd, tmp = [], BINDING + ".tmp"
    if spec is not None and gxx is not None:
        torch_dir = list(spec.submodule_search_locations)[0]
        cmd = [gxx, "-O2", "-std=c++17", "-fPIC", "-shared", src, "-o", tmp, "-I", os.path.join(torch_dir, "include"),
               "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
               "-I", os.path.join(cuda, "include"), "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python",
               "-Wl,-rpath," + os.path.join(torch_dir, "lib")]
    made_with = "\n".join([" ".join(cmd), "torch " + _installed("torch"), "python " + sys.version, ""])
    was = ""
    if os.path.exists(stamp):
        with open(stamp) as f:
            was = f.read()
    if not force and was == made_with and not _stale(BINDING, [src, os.path.join(INCLUDE, "moe_fp8.h"), os.path.abspath(__file__)]):
        return
    if os.path.exists(BINDING):
        os.remove(BINDING)
    if not cmd:
        print("_binding.so is not built: it takes torch and g++", file=sys.stderr)
        return
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(f"_binding.so is not built:\n{' '.join(cmd)}\n{r.stderr[-2000:]}", file=sys.stderr)
        return
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(made_with)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile (if stale) and return the path of libmoe_fp8.so."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])
    deps = _deps()
    jobs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or _stale(obj, [src] + deps):
            jobs.append((src, obj))

    def run(job):
        src, obj = job
        cmd = [nvcc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, file=sys.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(_build_binding, os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), force)
        list(ex.map(run, jobs))
        binding.result()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in sources()]
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-lpthread", "-ldl", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true", help="print registers/spills per kernel")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.ptxas_info else None
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose or a.ptxas_info, extra_flags=extra))
