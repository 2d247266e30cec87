"""Python's other threads run while a call is in the library."""
import ctypes
import shutil
import subprocess
import threading
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

SOURCE = """
#include <time.h>
volatile int flag = 0;
/* Stands for a launch that has to wait: returns 0 once another thread has set the flag, -3 after two seconds. */
int waits(const void *desc, void *stream) {
  struct timespec t = {0, 1000000};
  (void)desc; (void)stream;
  for (int i = 0; i < 2000; ++i) {
    if (flag) return 0;
    nanosleep(&t, 0);
  }
  return -3;
}
"""

NAMES = ("moe_gate", "moe_route", "moe_kv_pages", "moe_verify_drafts")


@pytest.mark.parametrize("which", range(4))
def test_a_call_that_waits_for_another_thread(lib, tmp_path, which):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    (tmp_path / "waits.c").write_text(SOURCE)
    subprocess.run([cc, "-O1", "-shared", "-fPIC", "-o", str(tmp_path / "waits.so"), str(tmp_path / "waits.c")], check=True)
    helper = ctypes.CDLL(str(tmp_path / "waits.so"))
    flag = ctypes.c_int.in_dll(helper, "flag")
    real = [ctypes.cast(getattr(lib._lib, n), ctypes.c_void_p).value for n in NAMES]
    fake = list(real)
    fake[which] = ctypes.cast(helper.waits, ctypes.c_void_p).value
    i32 = dict(dtype=torch.int32, device="cuda")
    f, i, n, one = torch.zeros((2, 8), device="cuda"), torch.zeros((2, 2), **i32), torch.zeros(2, **i32), torch.zeros(1, **i32)
    x = torch.zeros((2, 8), dtype=torch.bfloat16, device="cuda")
    calls = (lambda: lib._native.gate(x, x, f[:, :2], None), lambda: lib._native.route(f, i, f[:, :2], None, None, 1, 1, 1.0, 0),
             lambda: lib._native.kv_pages(n, n, i, n, one, 16, n, torch.zeros(3, **i32), one, None, None, None, None, None),
             lambda: lib._native.verify(f, n, torch.zeros(3, **i32), f[0, :2], f[0, :2], n, i, None, None, None, None, None))

    def other():
        time.sleep(0.05)
        flag.value = 1

    thread = threading.Thread(target=other)
    try:
        lib._native.connect(*fake)
        thread.start()
        assert calls[which]() == 0
    finally:
        lib._native.connect(*real)
        thread.join()
