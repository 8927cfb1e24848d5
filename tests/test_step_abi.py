"""Host-side behaviour of the step tables, the prefix groups and the shared decode (no GPU).

Every call below fails a host check, or is a size query or a metadata check on host copies,
before anything is launched.
"""
import ctypes

import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import shared_batch

INVALID, UNSUPPORTED, OUT_OF_RANGE, WORKSPACE = 1, 2, 4, 6


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_24_gb300 import build
    build.build()
    return ops.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_step_out_layout_matches_the_header(tmp_path):
    import os
    import subprocess
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "msgl_attn.h"', "int main(void) {",
             'printf("%zu\\n", sizeof(msgl_step_out));']
    lines += [f'printf("%zu\\n", offsetof(msgl_step_out, {name}));' for name, _ in ops._StepOut._fields_]
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(root, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(ops._StepOut)] + [getattr(ops._StepOut, n).offset for n, _ in ops._StepOut._fields_]


def test_step_tables_refusals(lib):
    def call(slots=256, ps=16, table=16, rows=4, stride=8, width=8, cached=16, reqs=2, free=16, num_free=3, out="good",
             **over):
        o = ops._StepOut(16, 8, 8, 16, 16, 16, 16, 16, 5)
        for k, v in over.items():
            setattr(o, k, v)
        return lib.msgl_step_tables(slots, ps, table, rows, stride, width, None, cached, None, reqs, free, num_free,
                                    ctypes.byref(o) if out else None, None, None)

    for want, kw in [(INVALID, dict(out=None)), (UNSUPPORTED, dict(ps=3)), (UNSUPPORTED, dict(ps=512)),
                     (INVALID, dict(slots=250)), (INVALID, dict(slots=-16)), (UNSUPPORTED, dict(slots=2 ** 31 + 16)),
                     (INVALID, dict(rows=-1)), (INVALID, dict(reqs=-1)), (INVALID, dict(num_free=-1)),
                     (INVALID, dict(stride=7)), (INVALID, dict(width=-1)), (INVALID, dict(table=None)),
                     (INVALID, dict(cached=None)), (INVALID, dict(free=None)), (INVALID, dict(total_tokens=-1)),
                     (INVALID, dict(stride=8, width=8, page_ids=None)), (INVALID, dict(seq_lens=None)),
                     (INVALID, dict(cu_ext=None)), (INVALID, dict(positions=None)), (INVALID, dict(out_loc=None)),
                     (INVALID, dict(pages_taken=None)), (UNSUPPORTED, dict(total_tokens=2 ** 31 - 1))]:
        assert call(**kw) == want, kw
        assert lib.msgl_last_error(), kw


def test_shared_prefixes_refusals(lib):
    def call(pages=ops._Pages(16, 8, 8), seq=16, reqs=2, ps=16, max_seq=100, least=16, first=16, shared=16):
        return lib.msgl_shared_prefixes(ctypes.byref(pages) if pages else None, seq, reqs, ps, max_seq, least, first,
                                        shared, None, None)

    for want, kw in [(INVALID, dict(pages=None)), (INVALID, dict(pages=ops._Pages(16, 4, 8))),
                     (INVALID, dict(pages=ops._Pages(None, 8, 8))), (INVALID, dict(seq=None)), (INVALID, dict(reqs=-1)),
                     (UNSUPPORTED, dict(ps=24)), (INVALID, dict(max_seq=0)), (INVALID, dict(least=0)),
                     (UNSUPPORTED, dict(max_seq=2 ** 30 + 1)),
                     (INVALID, dict(first=None)), (INVALID, dict(shared=None))]:
        assert call(**kw) == want, kw
    assert call(reqs=0) == 0


def test_decode_shared_refusals(lib):
    size = lib.msgl_decode_shared_workspace_size(4, 64, 8, 128, 100)
    assert size > lib.msgl_decode_workspace_size(4, 64, 8, 128, 100) and size % 256 == 0
    assert lib.msgl_decode_shared_workspace_size(0, 64, 8, 128, 100) == 0
    assert lib.msgl_decode_shared_workspace_size(4, 64, 8, 64, 100) == 0

    def call(pool=(16, 16, 256, 16, 8, 128), hq=64, first=16, shared=16, seq=16, reqs=4, max_seq=100, sharing=0,
             scale=0.1, ws=256, ws_bytes=size, q=16, o=16, lse=16):
        p, t = ops._Pool(*pool), ops._Pages(16, 8, 8)
        return lib.msgl_attn_decode_shared(ctypes.byref(p), ctypes.byref(t), q, hq, first, shared, seq, reqs, max_seq,
                                           sharing, scale, o, lse, ws, ws_bytes, None, None)

    for want, kw in [(UNSUPPORTED, dict(pool=(16, 16, 256, 16, 8, 64))), (INVALID, dict(pool=(18, 16, 256, 16, 8, 128))),
                     (INVALID, dict(hq=12)), (UNSUPPORTED, dict(hq=8 * 72)), (INVALID, dict(first=None)),
                     (INVALID, dict(shared=None)), (INVALID, dict(seq=None)), (INVALID, dict(sharing=3)),
                     (INVALID, dict(sharing=-1)), (INVALID, dict(scale=0.0)), (INVALID, dict(scale=float("nan"))),
                     (INVALID, dict(max_seq=0)), (UNSUPPORTED, dict(max_seq=2 ** 30 + 1)), (INVALID, dict(reqs=-1)),
                     (UNSUPPORTED, dict(reqs=70000)), (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=size - 1)),
                     (WORKSPACE, dict(ws_bytes=100)), (INVALID, dict(ws=128)), (INVALID, dict(q=8)),
                     (INVALID, dict(o=None)), (INVALID, dict(lse=None))]:
        assert call(**kw) == want, (kw, lib.msgl_last_error())
    assert lib.msgl_attn_decode_shared(None, None, None, 64, 16, 16, 16, 1, 10, 0, 0.1, 16, 16, 256, size, None, None) == 1
    assert call(reqs=0, first=None, shared=None, seq=None, q=None, o=None, lse=None, ws=None) == 0


def test_tensors_must_be_on_the_gpu():
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.step_tables(t, i32(1, 2), None, i32(1, 2), 64, 16, total_tokens=2)
    with pytest.raises(ValueError, match="CUDA"):
        ops.shared_prefixes(t, i32(1, 2), 16, 64, 1)
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)

    class Pool:
        k = v = torch.zeros(64, 8, 128, dtype=torch.bfloat16)
        page_size = 16
    with pytest.raises(ValueError, match="CUDA"):
        ops.attn_decode_shared(Pool, q, t, i32(1, 2), i32(0, 0), i32(0, 0), 64, 0.1)


def expect(status, fragment, fn, *args, **kw):
    with pytest.raises(ops.MsglError) as e:
        fn(*args, **kw)
    assert e.value.status == status and fragment in str(e.value), str(e.value)


def test_step_meta():
    good = dict(num_slots=160, page_size=16, req_table=torch.tensor([[3, -1, -1], [0, 7, -1]], dtype=torch.int32),
                req_rows=i32(1, 0), cached_lens=i32(20, 16), new_lens=i32(12, 17), free_pages=i32(5, 9, 1),
                total_tokens=29)
    ops.check_step_meta(**good)
    ops.check_step_meta(**dict(good, new_lens=None))
    for status, fragment, change in [
            (OUT_OF_RANGE, "request 1: row 2", dict(req_rows=i32(1, 2))),
            (INVALID, "row 1 belongs to an earlier", dict(req_rows=i32(1, 1))),
            (INVALID, "request 0: cached_len -1", dict(cached_lens=i32(-1, 16))),
            (INVALID, "new_len -2", dict(new_lens=i32(12, -2))),
            (OUT_OF_RANGE, "need 4 pages", dict(new_lens=i32(40, 1))),
            (OUT_OF_RANGE, "page_ids[1] = -1", dict(cached_lens=i32(20, 17))),
            (INVALID, "total_tokens = 28", dict(total_tokens=28)),
            (OUT_OF_RANGE, "num_free = 1", dict(free_pages=i32(5))),
            (OUT_OF_RANGE, "free_pages[0] = 10", dict(free_pages=i32(10, 2, 1))),
            (INVALID, "free_pages[1] = 3 is in use", dict(free_pages=i32(5, 3, 1))),
            (INVALID, "free_pages[1] = 5 is in use", dict(free_pages=i32(5, 5, 1))),
            (INVALID, "page_size 3", dict(page_size=3))]:
        expect(status, fragment, ops.check_step_meta, **dict(good, **change))


def test_groups_meta():
    w = shared_batch.make(8, 8, 16, [(40, [1, 20]), (0, [30]), (64, [2, 3, 4])], seed=1)
    good = dict(num_slots=w.k.shape[0], page_size=16, page_table=w.table, seq_lens=w.seq, group_start=w.first,
                shared_lens=w.shared, max_seq_len=w.max_seq)
    ops.check_groups_meta(**good)
    # shared whole pages are read through the first row only
    t = w.table.clone()
    t[1, :2] = -1
    ops.check_groups_meta(**dict(good, page_table=t))

    def changed(t, at, value):
        t = t.clone()
        t[at] = value
        return t
    for status, fragment, change in [
            (INVALID, "request 2: seq_len 0", dict(seq_lens=changed(w.seq, 2, 0))),
            (INVALID, "request 3: seq_len 66 is outside", dict(max_seq_len=60)),
            (INVALID, "request 4: group_start 0", dict(group_start=changed(w.first, 4, 0))),
            (INVALID, "request 0: group_start 1", dict(group_start=changed(w.first, 0, 1))),
            (INVALID, "request 1: shared_len 70", dict(shared_lens=changed(w.shared, 1, 70))),
            (INVALID, "request 5: shared_len 63 but", dict(shared_lens=changed(w.shared, 5, 63))),
            (OUT_OF_RANGE, "request 0: page_ids[1] = 999", dict(page_table=changed(w.table, (0, 1), 999))),
            (OUT_OF_RANGE, "request 1: page_ids[2] = -4", dict(page_table=changed(w.table, (1, 2), -4))),
            (OUT_OF_RANGE, "table width", dict(page_table=w.table[:, :4].contiguous()))]:
        expect(status, fragment, ops.check_groups_meta, **dict(good, **change))
