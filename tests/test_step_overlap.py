"""Which arrays of a step may share memory: msgl_step_tables and msgl_shared_prefixes refuse an output over
an input."""
import ctypes

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.test_step_tables import dev, resident, tables

B, W, ROWS, T, FREE = 4, 8, 6, 10, 5


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_24_gb300 import build
    build.build()
    return ops.load()


# entries of each array, laid out with space between them
SIZES = dict(req_table=ROWS * W, req_rows=B, cached_lens=B, new_lens=B, free_pages=FREE, page_ids=B * W, seq_lens=B,
             cu_ext=B + 1, positions=T, out_loc=T, pages_taken=1)
INPUTS = ("req_rows", "cached_lens", "new_lens", "free_pages")


def addresses():
    at, x = {}, 1 << 20
    for name, n in SIZES.items():
        at[name] = x
        x += 4 * n
    return at


def call(lib, at, stride=W, table_stride=W):
    out = ops._StepOut(at["page_ids"], stride, W, at["seq_lens"], at["cu_ext"], at["positions"], at["out_loc"],
                       at["pages_taken"], T)
    rc = lib.msgl_step_tables(1024, 16, at["req_table"], ROWS, table_stride, W, at["req_rows"], at["cached_lens"],
                              at["new_lens"], B, at["free_pages"], FREE, ctypes.byref(out), None, None)
    return rc, lib.msgl_last_error().decode()


@pytest.mark.parametrize("out", [n for n in SIZES if n not in INPUTS])
@pytest.mark.parametrize("other", list(SIZES))
def test_an_output_over_another_array_is_refused(lib, out, other):
    if out == other:
        return
    for shift in (0, SIZES[other] - 1, 1 - SIZES[out]):   # the same start; one entry in common at either end
        at = addresses()
        at[out] = at[other] + 4 * shift
        rc, text = call(lib, at)
        assert rc == 1 and "overlaps" in text, (out, other, shift, text)


def test_rows_with_a_pitch(lib):
    """Columns of one allocation: refused where the columns meet, by any row."""
    for first in (W - 1, -(W - 1), 40 + W - 1, 3 * 40, 5 * 40 - (W - 1)):
        at = addresses()
        at["req_table"] = 1 << 24
        at["page_ids"] = (1 << 24) + 4 * first
        rc, text = call(lib, at, stride=40, table_stride=40)
        assert rc == 1 and "page_ids overlaps req_table" in text, (first, text)
    at["page_ids"] = (1 << 24) + 4 * W
    at["cached_lens"] = (1 << 24) + 4 * (40 * 3 + 2 * W - 1)   # inside the last row's columns
    rc, text = call(lib, at, stride=40, table_stride=40)
    assert rc == 1 and "page_ids overlaps cached_lens" in text, text


@pytest.mark.parametrize("out", ["group_start", "shared_lens"])
@pytest.mark.parametrize("other", ["page_ids", "seq_lens", "group_start", "shared_lens"])
def test_prefix_groups_over_another_array_are_refused(lib, out, other):
    if out == other:
        return
    for shift in (0, B - 1, 1 - B):
        at = dict(page_ids=1 << 20, seq_lens=2 << 20, group_start=3 << 20, shared_lens=4 << 20)
        at[out] = at[other] + 4 * shift
        pages = ops._Pages(at["page_ids"], 40, W)
        rc = lib.msgl_shared_prefixes(ctypes.byref(pages), at["seq_lens"], B, 16, 128, 16, at["group_start"],
                                      at["shared_lens"], None, None)
        text = lib.msgl_last_error().decode()
        assert rc == 1 and "overlaps" in text, (out, other, shift, text)


@pytest.mark.gpu
def test_the_lengths_of_the_step_before_as_its_own_output():
    """A decode loop that passes the last step's seq_lens on needs two sets of outputs."""
    rt, free = dev(np.full((3, 8), -1)), dev(np.arange(40))
    a = ops.step_tables(rt, dev([0, 0, 0]), dev([20, 30, 40]), free, 1024, 16, total_tokens=90)
    b = ops.step_tables(rt, a.seq_lens, None, free[a.pages_taken.item():], 1024, 16, total_tokens=3)
    torch.cuda.synchronize()
    with pytest.raises(ops.MsglError, match="seq_lens overlaps cached_lens") as e:
        ops.step_tables(rt, b.seq_lens, None, free, 1024, 16, out=b)
    assert e.value.status == 1
    assert b.seq_lens.tolist() == [21, 31, 41]
    with pytest.raises(ops.MsglError, match="overlaps free_pages"):
        ops.step_tables(rt, a.seq_lens, None, free, 1024, 16, out=b._replace(out_loc=free[:3]))


@pytest.mark.gpu
def test_tables_that_are_columns_of_one_allocation():
    ps, pages, cached, new = 16, 100, np.array([0, 33, 100, 16]), np.array([5, 60, 1, 16])
    rng = np.random.default_rng(3)
    table, free = resident(rng, 6, 9, cached, [5, 1, 0, 3], ps, pages)
    rows, start = np.array([5, 1, 0, 3]), np.full((4, 9), -5, dtype=np.int32)
    want, bits = tables(table, rows, cached, new, free, pages * ps, ps, 82, start)
    assert bits == 0
    both = np.full((6, 20), 77, dtype=np.int32)
    both[:, :9], both[:4, 9:18] = table, start
    both = dev(both)
    seq, cu, pos, loc, taken = (dev(np.zeros(n)) for n in (4, 5, 82, 82, 1))
    r, c, n, f = (dev(x) for x in (rows, cached, new, free))
    status = ops.new_status()
    out = ops._StepOut(both.data_ptr() + 4 * 9, 20, 9, seq.data_ptr(), cu.data_ptr(), pos.data_ptr(), loc.data_ptr(),
                       taken.data_ptr(), 82)
    rc = ops.load().msgl_step_tables(pages * ps, ps, both.data_ptr(), 6, 20, 9, r.data_ptr(), c.data_ptr(),
                                     n.data_ptr(), 4, f.data_ptr(), len(free), ctypes.byref(out), status.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and ops.read_status(status) == 0
    got = both.cpu().numpy()
    assert np.array_equal(got[:, :9], want[6]) and np.array_equal(got[:4, 9:18], want[0])
    assert np.all(got[:, 18:] == 77) and np.all(got[4:, 9:] == 77)
    for x, w in zip((seq, cu, pos, loc, taken), want[1:6]):
        assert np.array_equal(x.cpu().numpy(), w)


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [1, 16])
def test_page_table_in_place(ps):
    """The resident table as the step's own page table: the same rows at the same pitch, no req_rows."""
    cached, new = np.array([0, 33, 100, 16]), np.array([5, 60, 1, 16])
    rng = np.random.default_rng(4)
    table, free = resident(rng, 4, 160, cached, range(4), ps, 400)
    want, bits = tables(table, None, cached, new, free, 400 * ps, ps, 82, table)
    assert bits == 0
    rt = dev(table)
    out = ops.StepTables(rt, *(dev(np.zeros(n)) for n in (4, 5, 82, 82, 1)))
    ops.step_tables(rt, dev(cached), dev(new), dev(free), 400 * ps, ps, out=out)
    for x, w in zip(out, want):
        assert np.array_equal(x.cpu().numpy(), w)
    assert np.array_equal(rt.cpu().numpy(), want[6])
    with pytest.raises(ops.MsglError, match="page_ids overlaps req_table"):
        ops.step_tables(rt, dev(cached), dev(new), dev(free), 400 * ps, ps, out=out, req_rows=dev([3, 2, 1, 0]))
