"""The rotary store, the draft verification and the page calls beside other Python threads, on streams of their own and
from several threads at once."""
import ctypes
import threading
import time

import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import i32

pytestmark = pytest.mark.gpu

BUSY_S = 0.7


def calls(seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    z = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    pool = ops.KVPool(normal(256, 2, 128), normal(256, 2, 128), 16)
    q, kv, out, rope = normal(4, 4, 128), normal(4, 2, 128), torch.zeros(4, 4, 128, dtype=torch.bfloat16, device="cuda"), ops.Rope([0.5] * 8)
    pos, loc = i32([1, 2, 3, 4 + seed], "cuda"), i32([7, 9, 100, 3], "cuda")
    p = torch.rand(4, 99, generator=g, device="cuda")
    tok, cu, u = i32([5, 6, 7, 8], "cuda"), i32([0, 2, 4], "cuda"), torch.rand(4, generator=g, device="cuda")
    ver = ops.Verified(z(2), z(4), z(2))
    table, lens = torch.arange(16, dtype=torch.int32, device="cuda").reshape(4, 4).contiguous(), i32([40, 20 + seed], "cuda")
    free, forked = ops.FreePages(z(16), z(1)), ops.Forked(z(1), z(1), z(1), z(1))
    ws = torch.zeros(ops.page_map_workspace_size(256, 16), dtype=torch.uint8, device="cuda")
    com = ops.Compaction(z(4, 4), z(16), z(8), z(8), z(1), z(1))
    a, b, n, f = i32([0], "cuda"), i32([3], "cuda"), i32([20], "cuda"), i32([15], "cuda")
    torch.cuda.synchronize()
    return {
        "rope": lambda s: ops.rope_store_kv(pool, q, kv, kv, pos, loc, rope, q_out=out, stream=s),
        "verify": lambda s: ops.verify_drafts(p, None, tok, cu, u, u[:2], out=ver, stream=s),
        "fork": lambda s: ops.fork_requests(table, a, b, n, f, 256, 16, out=forked, stream=s),
        "copy": lambda s: ops.copy_pages(pool, a, f, stream=s),
        "free": lambda s: ops.free_pages(table, lens, 256, 16, out=free, workspace=ws, stream=s),
        "compact": lambda s: ops.compact_pages(table, lens, 256, 16, out=com, workspace=ws, stream=s),
    }, (out, pool.k, pool.v, *ver, table, *free, *forked, *com)


@pytest.mark.parametrize("name", ["rope", "verify", "fork", "copy", "free", "compact"])
def test_other_threads_run_while_a_call_waits(name):
    call = calls()[0][name]
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


def test_calls_of_several_threads_at_once():
    """Four threads with streams and buffers of their own: each gets what it gets alone."""
    alone = []
    for seed in range(4):
        fs, outs = calls(seed)
        for f in fs.values():
            f(None)
        torch.cuda.synchronize()
        alone.append([x.clone() for x in outs])
    both, errors = [calls(seed) for seed in range(4)], []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            for _ in range(200):
                for f in both[seed][0].values():
                    f(s)
            s.synchronize()
        except Exception as e:      # noqa: BLE001 (shown by the assertion below)
            errors.append(e)
    ts = [threading.Thread(target=work, args=(seed,)) for seed in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors
    for want, (_, got) in zip(alone, both):
        for a, b in zip(want, got):
            assert torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a, b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


def test_scratch_of_a_call_is_in_its_streams_order():
    """Without a workspace the scratch comes from the allocator; two streams with calls in flight do not share it."""
    n = 60000                                      # (too many for the one launch that needs no scratch)
    streams = [torch.cuda.Stream() for _ in range(3)]
    rows = [torch.randperm(n, device="cuda").int()[:5000 + 100 * i].reshape(1, -1).contiguous() for i in range(3)]
    lens = [i32([r.shape[1]], "cuda") for r in rows]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        for s, r, m in zip(streams, rows, lens):
            with torch.cuda.stream(s):
                got.append((ops.free_pages(r, m, n, 1), r))
    torch.cuda.synchronize()
    for out, r in got:
        free = torch.ones(n, dtype=torch.bool)
        free[r[0].long().cpu()] = False
        want = torch.nonzero(free)[:, 0].int()
        assert out.num_free.item() == len(want) and torch.equal(out.pages[:len(want)].cpu(), want)
