"""The step calls with tables whose rows are further apart than their columns (the C ABI's strides), and
two batches at once on streams of their own."""
import ctypes
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import shared_batch
from tests.test_decode_shared import VARIANTS, run, varied
from tests.test_step_tables import dev, resident, tables

pytestmark = pytest.mark.gpu


def pitched(x, pitch, fill):
    """x [rows, width] in rows of `pitch` entries."""
    y = np.full((x.shape[0], pitch), fill, dtype=np.int32)
    y[:, :x.shape[1]] = x
    return y


def stream():
    return torch.cuda.current_stream().cuda_stream


def test_tables_and_groups():
    ps, pages, cached = 16, 200, np.array([0, 33, 160, 16, 255, 200])
    new = np.array([5, 100, 1, 16, 1, 0])
    rng = np.random.default_rng(1)
    table, free = resident(rng, 8, 20, cached, [7, 1, 0, 3, 5, 2], ps, pages)
    rows = np.array([7, 1, 0, 3, 5, 2])
    start = np.full((6, 18), -5, dtype=np.int32)
    want, bits = tables(table, rows, cached, new, free, pages * ps, ps, 130, start)
    assert bits == 0
    rt, ids = dev(pitched(table, 41, 77)), dev(pitched(start, 33, 78))
    seq, cu, pos, loc, taken = (dev(np.zeros(n)) for n in (6, 7, 130, 130, 1))
    inputs = [dev(x) for x in (rows, cached, new, free)]
    status = ops.new_status()
    out = ops._StepOut(ids.data_ptr(), 33, 18, seq.data_ptr(), cu.data_ptr(), pos.data_ptr(), loc.data_ptr(),
                       taken.data_ptr(), 130)
    r, c, n, f = (x.data_ptr() for x in inputs)
    rc = ops.load().msgl_step_tables(pages * ps, ps, rt.data_ptr(), 8, 41, 20, r, c, n, 6, f, len(free),
                                     ctypes.byref(out), status.data_ptr(), stream())
    assert rc == 0 and ops.read_status(status) == 0
    assert np.array_equal(ids.cpu().numpy(), pitched(want[0], 33, 78))
    assert np.array_equal(rt.cpu().numpy(), pitched(want[6], 41, 77))
    for got, w in zip((seq, cu, pos, loc, taken), want[1:6]):
        assert np.array_equal(got.cpu().numpy(), w)

    # groups of a table with such rows: equal up to the width, the entries behind it differ
    for width in (9, 300):   # (one launch, and two)
        x = np.tile(np.arange(width, dtype=np.int32), (4, 1))
        x[2, 5:] += 1
        y = pitched(x, width + 6, 0)
        y[:, width:] = np.arange(24).reshape(4, 6)
        t, lens = dev(y), dev([140] * 4)
        first, shared = dev([9] * 4), dev([9] * 4)
        pt = ops._Pages(t.data_ptr(), width + 6, width)
        rc = ops.load().msgl_shared_prefixes(ctypes.byref(pt), lens.data_ptr(), 4, ps, width * ps, 16, first.data_ptr(),
                                             shared.data_ptr(), status.data_ptr(), stream())
        assert rc == 0 and ops.read_status(status) == 0
        assert first.tolist() == [0] * 4 and shared.tolist() == [80] * 4


@pytest.mark.parametrize("variant", list(VARIANTS))
@pytest.mark.parametrize("ps", [1, 16])
def test_shared_decode(variant, ps):
    w, kw = varied(shared_batch.make(40, 8, ps, [(320, [1, 50, 3]), (0, [70]), (160, [20, 7])], seed=31), variant)
    g = w.cuda()
    want = run(g, **kw)
    W = g.table.shape[1]
    t = torch.full((6, W + 5), 10 ** 8, dtype=torch.int32, device="cuda")
    t[:, :W] = g.table
    pool = ops.KVPool(g.k, g.v, ps)
    pt = ops._Pages(t.data_ptr(), W + 5, W)
    n = ops.decode_shared_workspace_size(6, 40, 8, g.max_seq)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(g.q), torch.empty(6, 40, device="cuda")
    status = ops.new_status()
    rc = ops.load().msgl_attn_decode_shared(
        ctypes.byref(pool.c()), ctypes.byref(pt), g.q.data_ptr(), 40, g.first.data_ptr(), g.shared.data_ptr(),
        g.seq.data_ptr(), 6, g.max_seq, ops.SHARING[kw["sharing"]], g.scale, o.data_ptr(), lse.data_ptr(), ws.data_ptr(),
        n, status.data_ptr(), stream())
    assert rc == 0 and ops.read_status(status) == 0
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_two_streams_at_once(variant):
    batches = [varied(shared_batch.make(64, 8, ps, groups, seed=40 + ps), variant)
               for ps, groups in ((1, [(700, [1, 90, 3, 20]), (0, [300])]), (16, [(2000, list(range(1, 40)))]))]
    kw = batches[0][1]
    gs = [b.cuda() for b, _ in batches]
    want = [run(g, **kw) for g in gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in gs]
    got = [[], []]
    for _ in range(8):
        for i, g in enumerate(gs):
            got[i].append(run(dataclasses.replace(g), stream=streams[i], **kw))
    torch.cuda.synchronize()
    for i in range(2):
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])
