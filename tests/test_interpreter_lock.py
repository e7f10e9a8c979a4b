"""The compiled calls leave the interpreter to other threads while an entry point runs: one
that returns only once another Python thread has set its flag."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

from test_current_device import compiled_calls

pytestmark = pytest.mark.gpu

SOURCE = """
#include <time.h>
volatile int waiting, flag;
int entry(void) {
  struct timespec ms = {0, 1000000};
  waiting = 1;
  for (int i = 0; i < 2000; ++i) {
    if (flag) return 0;
    nanosleep(&ms, 0);
  }
  return 1;
}
"""


@pytest.mark.parametrize("which", ["append", "decode", "prompt"])
def test_other_threads_run(tmp_path, which):
    (tmp_path / "entry.c").write_text(SOURCE)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(tmp_path / "entry.so"),
                    str(tmp_path / "entry.c")], check=True)
    lib = ctypes.CDLL(str(tmp_path / "entry.so"))
    waiting, flag = ctypes.c_int.in_dll(lib, "waiting"), ctypes.c_int.in_dll(lib, "flag")
    calls = compiled_calls(tmp_path, lib.entry, 0)

    def set_flag():
        end = time.monotonic() + 5
        while not waiting.value and time.monotonic() < end:
            time.sleep(0.001)
        flag.value = 1

    q, kv = (torch.zeros(2, h, 64, device="cuda").bfloat16() for h in (4, 2))
    cache = torch.zeros(3, 16, 2, 64, device="cuda").bfloat16()
    n = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    thread = threading.Thread(target=set_flag)
    thread.start()
    try:
        if which == "append":
            calls.append(kv, kv, cache, cache, slots, None, None, q, None, None, None, False)
        elif which == "decode":
            calls.decode(q, cache, cache, table, n[:2], None, 0, None, None, None, False, None, ws)
        else:
            calls.prompt(q, kv, kv, n, None, None, True, 0, None, False, None, ws)
    finally:
        thread.join()
