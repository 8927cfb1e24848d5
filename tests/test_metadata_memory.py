"""The host metadata checks when host memory runs out: a status, not an exception through the C ABI (no GPU)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# A child process, limited to little more memory than it has: an exception that leaves a C entry ends it.
PROGRAM = """
import ctypes, resource, sys
import numpy as np
lib = ctypes.CDLL(sys.argv[1])
lib.msgl_last_error.restype = ctypes.c_char_p
n = 20_000_000
ids = np.arange(n, dtype=np.int32)
p = ids.ctypes.data_as(ctypes.c_void_p)
one, free = np.array([n], dtype=np.int32), np.array([n], dtype=np.int32)
pages = int([x for x in open("/proc/self/statm").read().split()][0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (pages + (64 << 20),) * 2)
if sys.argv[2] == "store":
    rc = lib.msgl_check_store_meta(ctypes.c_int64(n), p, n)
else:
    rc = lib.msgl_check_step_meta(ctypes.c_int64(n + 1), 1, p, 1, n, n, None, one.ctypes.data_as(ctypes.c_void_p),
                                  np.zeros(1, np.int32).ctypes.data_as(ctypes.c_void_p), 1,
                                  free.ctypes.data_as(ctypes.c_void_p), 1, 0)
print("rc", rc, lib.msgl_last_error().decode())
"""


@pytest.mark.parametrize("which", ["store", "step"])
def test_out_of_host_memory(which):
    from paged_kv_attention_24_gb300 import build
    lib = build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM, lib, which], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
    assert r.stdout.startswith("rc 2 ") and "host memory" in r.stdout, r.stdout
