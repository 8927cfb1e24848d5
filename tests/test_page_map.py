"""Free pages and compaction against their definitions; every entry has to be equal, and a compacted pool has to hold
what it held."""
import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.step_reference import i32

pytestmark = pytest.mark.gpu


def requests(batch, ps, longest, num_pages, seed, share=0, rows=None, width=None):
    """(table, rows, lens): distinct pages but for the first `share` of each row, which the rows have in common."""
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, batch)
    width = width or ref.pages_of(longest, ps) + 2
    rows = rows or batch + 3
    table = rng.integers(-3, num_pages + 3, (rows, width)).astype(np.int32)      # what stands behind a length counts nothing
    where = rng.permutation(rows)[:batch]
    order = rng.permutation(num_pages).tolist()
    common = [order.pop() for _ in range(share)]
    for r, n in zip(where, lens):
        k = ref.pages_of(n, ps)
        for c in range(k):
            table[r, c] = common[c] if c < share else order.pop()
    return table, where.tolist(), lens.tolist(), rng


def some_held(rng, num_pages, share):
    return (rng.random(num_pages) < share).astype(np.uint8) * rng.integers(1, 256, num_pages).astype(np.uint8)


def run_free(table, rows, lens, num_pages, ps, held=None, flags=0, own=False, shift=0):
    status = ops.new_status()
    out = None if own else ops.FreePages(*[torch.full((n,), -9, dtype=torch.int32, device="cuda") for n in (num_pages, 1)])
    h = None
    if held is not None:
        h = torch.zeros(num_pages + shift, dtype=torch.uint8, device="cuda")[shift:]
        h.copy_(torch.from_numpy(held))
    got = ops.free_pages(i32(table, "cuda"), i32(lens, "cuda"), num_pages * ps, ps, None if rows is None else i32(rows, "cuda"),
                         h, out, status=status)
    used = ref.held_by(table, rows, lens, num_pages, ps) | (False if held is None else held != 0)
    want = np.nonzero(~used)[0].tolist()
    assert got.num_free.tolist() == [len(want)]
    assert got.pages.tolist() == want + [-1] * (num_pages - len(want))
    assert ops.read_status(status) == flags


@pytest.mark.parametrize("ps", [1, 16, 256])
@pytest.mark.parametrize("batch,longest,num_pages", [(1, 1, 1), (1, 40, 50), (3, 70, 255), (40, 60, 3000), (9, 2000, 20011),
                                                     (1500, 12, 33000)])
def test_free(ps, batch, longest, num_pages):
    table, rows, lens, rng = requests(batch, ps, longest * (1 if ps == 1 else ps // 8), num_pages, batch + ps)
    run_free(table, rows, lens, num_pages, ps)
    run_free(table, rows, lens, num_pages, ps, some_held(rng, num_pages, 0.3), own=True)
    run_free(table, rows, lens, num_pages, ps, some_held(rng, num_pages, 0.9), shift=5)


@pytest.mark.parametrize("pages", [700, 40000])
def test_free_without_rows_and_with_shared_pages(pages):
    table, rows, lens, rng = requests(12, 4, 90, pages, 3, share=5)
    run_free(table, rows, lens, pages, 4)
    lens3 = [0, 3, 8] + [4 * table.shape[1]] * 2              # (whole rows, whatever stands in them)
    run_free(table, None, lens3, pages, 4, flags=ops.DEVERR_PAGE_RANGE if ref.names_no_page(table, None, lens3, pages, 4) else 0)
    run_free(table, [rows[0], rows[0], -1], [lens[0], lens[0], 5], pages, 4)


@pytest.mark.parametrize("first", [0, 5, 31, 1000])
@pytest.mark.parametrize("pages", [1500, 40000])
def test_free_of_pages_in_a_row(pages, first):
    """Neighbouring pages share words of the bitmap: whole rows of them, broken runs, one page many times."""
    table = np.tile(np.arange(first, first + 300, dtype=np.int32), (40, 1))
    table[1::2] = table[1::2, ::-1]
    table[3, 10:200] = first + 7
    table[5, ::3] = -1
    lens = [300] * 40
    run_free(table, None, lens, pages, 1, flags=ops.DEVERR_PAGE_RANGE)
    run_free(table[:3], None, [300, 299, 33], pages, 1)
    run_compact(table[:3], None, [300, 299, 33], pages, 1)
    run_compact(table, None, lens, pages, 1, flags=ops.DEVERR_PAGE_RANGE)


@pytest.mark.parametrize("batch", [70, 601])
def test_tables_much_wider_than_what_is_in_them(batch):
    """The rows' units are counted and dealt out, in one batch of requests and in two."""
    table, rows, lens, rng = requests(batch, 1, 900, 300000, batch, width=60000)
    lens[5], lens[-1], rows[9] = 0, -4, -1
    table[rows[-1]] = rng.integers(0, 300000, 60000)
    run_free(table, rows, lens, 300000, 1, flags=ops.DEVERR_LENGTH)
    run_compact(table, rows, lens, 300000, 1, some_held(rng, 300000, 0.2), flags=ops.DEVERR_LENGTH)


def test_held_as_bools():
    held = torch.zeros(64, dtype=torch.bool, device="cuda")
    held[[3, 40]] = True
    out = ops.free_pages(i32([[5, 6]], "cuda"), i32([2], "cuda"), 64, 1, held=held)
    assert out.pages[:out.num_free.item()].tolist() == [p for p in range(64) if p not in (3, 5, 6, 40)]


def test_free_at_the_ends():
    empty = np.zeros((0, 0), np.int32)
    run_free(empty, None, [], 0, 16)
    run_free(empty, None, [], 1, 16)
    run_free(np.zeros((2, 0), np.int32), None, [0, 0], 70, 1)
    for n in (320, 40960):
        full = np.arange(n, dtype=np.int32).reshape(2, n // 2)
        run_free(full, None, [n // 2, n // 2], n, 1)
        run_free(full, None, [n // 2, n // 2 - 1], n, 1)
        run_free(full, None, [0, 0], n, 1, np.ones(n, np.uint8))
    run_free(empty, None, [], 40000, 1)


@pytest.mark.parametrize("pages", [300, 40001])
def test_free_of_what_is_wrong(pages):
    table, rows, lens, rng = requests(6, 8, 100, pages, 5)
    ids = np.clip(table, 0, pages - 1)
    for bad, flag in ((-1, ops.DEVERR_LENGTH), (8 * table.shape[1] + 1, ops.DEVERR_LENGTH), (2 ** 31 - 1, ops.DEVERR_LENGTH)):
        run_free(ids, rows, [bad] + lens[1:], pages, 8, flags=flag)      # all that its row names is kept
    run_free(ids, [table.shape[0], -2] + rows[2:], lens, pages, 8, flags=ops.DEVERR_ROW)
    ids[rows[0], 0] = pages
    run_free(ids, rows, [8] + lens[1:], pages, 8, flags=ops.DEVERR_PAGE_RANGE)


def test_free_of_millions_of_pages():
    num_pages = 2633785
    rng = np.random.default_rng(7)
    table = rng.permutation(num_pages)[:30 * 5000].astype(np.int32).reshape(30, 5000)
    lens = rng.integers(0, 5001, 30).tolist()
    held = some_held(rng, num_pages, 0.01)
    table[3, 0], table[4, 0], lens[3], lens[4] = num_pages - 1, 0, 5000, 5000
    run_free(table, None, lens, num_pages, 1, held)
    run_free(table, None, [5001] + lens[1:], num_pages, 1, held, flags=ops.DEVERR_LENGTH)


# ------------------------------------------------------------------- compact

def run_compact(table, rows, lens, num_pages, ps, held=None, flags=0, out=None):
    """out: None (in place, buffers of its own), "new" or "same" (a table of its own, or in place, in given buffers)"""
    status, t = ops.new_status(), i32(table, "cuda")
    n = num_pages
    blank = np.full(table.shape, -9, np.int32)
    o = None
    if out:
        o = ops.Compaction(i32(blank, "cuda") if out == "new" else t,
                           *[torch.full((k,), -9, dtype=torch.int32, device="cuda") for k in (n, n // 2, n // 2, 1, 1)])
    h = None if held is None else torch.from_numpy(held).cuda()
    got = ops.compact_pages(t, i32(lens, "cuda"), n * ps, ps, None if rows is None else i32(rows, "cuda"), h, o, status=status)
    want = ref.compact(table, rows, lens, held, n, ps, blank if out == "new" else None)
    assert np.array_equal(got.page_table.cpu().numpy(), want[0])
    if out == "new":
        assert np.array_equal(t.cpu().numpy(), table)
    for name, a, b in zip(got._fields[1:], got[1:], want[1:4] + ([want[4]], [want[5]])):
        assert a.tolist() == list(b), name
    assert ops.read_status(status) == flags
    return got


@pytest.mark.parametrize("out", [None, "new", "same"])
@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("batch,longest,num_pages", [(1, 1, 1), (1, 1, 2), (1, 40, 50), (3, 70, 255), (40, 60, 3000),
                                                     (9, 2000, 20011), (1500, 12, 33000)])
def test_compact(ps, batch, longest, num_pages, out):
    table, rows, lens, rng = requests(batch, ps, longest * (1 if ps == 1 else 2), num_pages, batch + ps)
    run_compact(table, rows, lens, num_pages, ps, out=out)
    run_compact(table, rows, lens, num_pages, ps, some_held(rng, num_pages, 0.3), out=out)


@pytest.mark.parametrize("pages", [2000, 40000])
def test_compact_shared_pages_and_rows_named_twice(pages):
    table, rows, lens, rng = requests(12, 4, 90, pages, 3, share=9)
    got = run_compact(table, rows, lens, pages, 4)
    again = got.page_table.cpu().numpy()
    got = run_compact(again, rows, lens, pages, 4)             # nothing is left to move
    assert got.num_moves.item() == 0
    run_compact(table, rows + rows[:5] + [-1], lens + lens[:5] + [7], pages, 4)
    run_compact(table, rows + rows[:5], lens + lens[:5], pages, 4, out="new")


def test_compact_wide_rows_named_many_times():
    """More units than warps: rows are read again after another warp has renamed them."""
    table = np.random.default_rng(4).permutation(300000)[:2 * 60000].astype(np.int32).reshape(2, 60000)
    run_compact(table, [0, 1] * 12, [60000, 59999, 60000, 31] * 6, 300000, 1)


def test_compact_at_the_ends():
    empty = np.zeros((0, 0), np.int32)
    run_compact(empty, None, [], 0, 16)
    run_compact(empty, None, [], 5, 16)
    run_compact(empty, None, [], 40000, 1)
    for n in (320, 40960):
        m = n // 2
        full = np.random.default_rng(1).permutation(n).astype(np.int32).reshape(2, m)
        run_compact(full, None, [m, m], n, 1)
        run_compact(full, None, [m, 1], n, 1)
        run_compact(full, None, [m, 20], n, 1, np.ones(n, np.uint8))
        run_compact(full, None, [m, 0], n, 1, (np.arange(n) >= n - 20).astype(np.uint8))


@pytest.mark.parametrize("pages", [300, 40001])
def test_compact_what_is_wrong(pages):
    table, rows, lens, rng = requests(6, 8, 100, pages, 5)
    ids = np.clip(table, 0, pages - 1)
    run_compact(ids, rows, [-1] + lens[1:], pages, 8, flags=ops.DEVERR_LENGTH)
    run_compact(ids, [table.shape[0]] + rows[1:], lens, pages, 8, flags=ops.DEVERR_ROW)
    ids[rows[0], 0] = pages
    ids[rows[0], 1] = -1
    run_compact(ids, rows, [16] + lens[1:], pages, 8, flags=ops.DEVERR_PAGE_RANGE, out="new")


def test_large_compaction():
    n = 1310723
    rng = np.random.default_rng(9)
    table = rng.permutation(n)[:40 * 9000].astype(np.int32).reshape(40, 9000)
    lens = rng.integers(0, 9001, 40).tolist()
    run_compact(table, None, lens, n, 1, some_held(rng, n, 0.05))


@pytest.mark.parametrize("share", [0.0, 0.6])
def test_a_pool_whose_shares_take_several_rounds(share):
    n = 4600011
    rng = np.random.default_rng(10)
    table = rng.integers(0, n, (30, 9000)).astype(np.int32)
    table[7, 0], table[8, 0] = n - 1, 0
    lens = rng.integers(1, 9001, 30).tolist()
    held = some_held(rng, n, share) if share else None
    run_free(table, None, lens, n, 1, held)
    run_compact(table, None, lens, n, 1, held)


def test_a_compacted_pool_reads_as_before():
    ps, n = 16, 400
    table, rows, lens, rng = requests(20, ps, 300, n, 11, share=3)
    pool = ops.KVPool(torch.randn(n * ps, 2, 128, device="cuda").bfloat16(), torch.randn(n * ps, 2, 128, device="cuda").bfloat16(), ps)

    def tokens(t):
        return [x[torch.tensor([int(t[r, j // ps]) * ps + j % ps for j in range(m)], dtype=torch.long, device="cuda")]
                for r, m in zip(rows, lens) for x in (pool.k, pool.v)]
    before = tokens(table)
    c = ops.compact_pages(i32(table, "cuda"), i32(lens, "cuda"), n * ps, ps, i32(rows, "cuda"))
    ops.check_copy_meta(n * ps, ps, c.src, c.dst)
    ops.copy_pages(pool, c.src, c.dst, count=c.num_moves)
    now = c.page_table.cpu().numpy()
    assert all(torch.equal(a, b) for a, b in zip(before, tokens(now)))
    used = ref.held_by(now, rows, lens, n, ps)
    assert used[:c.num_used.item()].all() and not used[c.num_used.item():].any() and c.num_moves.item() > 0


@pytest.mark.parametrize("pages", [4000, 70000])                # one launch, several
def test_graph_and_stream(pages):
    table, rows, lens, rng = requests(30, 4, 200, pages, 13)
    t, r, n = i32(table, "cuda"), i32(rows, "cuda"), i32(lens, "cuda")
    free = ops.FreePages(torch.zeros(pages, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    first = ops.free_pages(t, n, 4 * pages, 4, r, stream=side)
    side.synchronize()
    assert first.num_free.item() == pages - ref.held_by(table, rows, lens, pages, 4).sum()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.free_pages(t, n, 4 * pages, 4, r, out=free)
        c = ops.compact_pages(t, n, 4 * pages, 4, r)
    for seed in range(14, 20):
        table, rows, lens, rng = requests(30, 4, 200, pages, seed)
        t.copy_(i32(table)), r.copy_(i32(rows)), n.copy_(i32(lens))
        graph.replay()
        want = np.nonzero(~ref.held_by(table, rows, lens, pages, 4))[0].tolist()
        assert free.pages.tolist() == want + [-1] * (pages - len(want))
        assert np.array_equal(t.cpu().numpy(), ref.compact(table, rows, lens, None, pages, 4)[0])
        assert c.num_used.item() == pages - len(want)


def test_refusals():
    t, n = torch.zeros(3, 4, dtype=torch.int32, device="cuda"), i32([1, 2], "cuda")
    for f in (ops.free_pages, ops.compact_pages):
        for args in ((t.long(), n, 64, 16), (t, n, 60, 16), (t, n, -16, 16), (t, n, 64, 0), (t[0], n, 64, 16), (t.t(), n, 64, 16),
                     (t, n, 64, 16, i32([1], "cuda")), (t, n, 64, 16, None, n), (t, n, 64, 16, None, torch.zeros(3, dtype=torch.uint8, device="cuda")),
                     (t, n.cpu(), 64, 16)):
            with pytest.raises(ValueError):
                f(*args)
        with pytest.raises(ops.MsglError):
            f(t, n, 66, 3)
    four = torch.zeros(4, dtype=torch.int32, device="cuda")
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.free_pages(t, n, 64, 16, out=ops.FreePages(t[0], one))
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.free_pages(t, n, 64, 16, out=ops.FreePages(four, four[3:]))
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.compact_pages(t, n, 64, 16, out=ops.Compaction(t, four, four[:2], torch.zeros_like(four[:2]), one, one.clone()))
    held = torch.zeros(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.free_pages(t, n, 64, 16, held=held[:4], out=ops.FreePages(held.view(torch.int32), one))
