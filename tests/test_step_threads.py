"""The step's Python calls beside other Python threads: a call that waits for room in the launch queue does not
hold them up."""
import ctypes
import threading
import time

import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import shared_batch

pytestmark = pytest.mark.gpu

BUSY_S = 0.7


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls():
    w = shared_batch.make(16, 8, 16, [(32, [1, 2])], seed=1).cuda()
    pool = ops.KVPool(w.k, w.v, 16)
    out = ops.step_tables(w.table, i32(0, 0), i32(0, 0), i32(1, 2), 256, 16, total_tokens=2)
    ws = torch.empty(ops.decode_shared_workspace_size(2, 16, 8, w.max_seq), dtype=torch.uint8, device="cuda")
    o, lse, first, shared = torch.empty_like(w.q), torch.empty(2, 16, device="cuda"), i32(0, 0), i32(0, 0)
    c, f = i32(0, 0), i32(1, 2)
    torch.cuda.synchronize()
    return {
        "tables": lambda s: ops.step_tables(w.table, c, c, f, 256, 16, out=out, stream=s),
        "groups": lambda s: ops.shared_prefixes(w.table, w.seq, 16, w.max_seq, 16, first, shared, stream=s),
        "decode": lambda s: ops.attn_decode_shared(pool, w.q, w.table, w.seq, w.first, w.shared, w.max_seq, w.scale,
                                                   out=o, lse=lse, workspace=ws, stream=s),
    }


@pytest.mark.parametrize("name", ["tables", "groups", "decode"])
def test_other_threads_run_while_a_call_waits(name):
    call = calls()[name]
    s = torch.cuda.Stream()
    call(s)
    s.synchronize()
    stop, gap = threading.Event(), [0.0]

    def tick():
        last = time.perf_counter()
        while not stop.is_set():
            time.sleep(0.001)
            now = time.perf_counter()
            gap[0], last = max(gap[0], now - last), now
    t = threading.Thread(target=tick)
    t.start()
    try:
        # the stream is busy on the host's side for a while (usleep in C, without Python), so that the queue fills
        usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p)
        launch = ctypes.CDLL("libcuda.so.1").cuLaunchHostFunc
        launch.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
        gap[0] = 0.0
        assert launch(s.cuda_stream, usleep, int(BUSY_S * 1e6)) == 0
        longest, began = 0.0, time.perf_counter()
        while longest < 0.1 and time.perf_counter() - began < BUSY_S:
            t0 = time.perf_counter()
            call(s)
            longest = max(longest, time.perf_counter() - t0)
    finally:
        s.synchronize()
        stop.set()
        t.join()
    if longest < 0.1:
        pytest.skip("the launch queue did not fill")
    assert gap[0] < BUSY_S / 3, (gap[0], longest)
