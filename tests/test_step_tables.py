"""msgl_step_tables and msgl_shared_prefixes against plain Python loops (whole numbers: equal)."""
import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops

pytestmark = pytest.mark.gpu


def tables(req_table, rows, cached, new, free, num_slots, ps, total, page_table):
    """The step written out request by request; returns the outputs and the status bits."""
    req_table, page_table = req_table.copy(), page_table.copy()
    B = len(cached)
    new = [1] * B if new is None else list(new)
    rows = list(range(B)) if rows is None else list(rows)
    P = lambda x: -(-x // ps)
    most = min(req_table.shape[1], page_table.shape[1])
    seq, cu, pos, loc = [0] * B, [0] * (B + 1), [0] * total, [-1] * total
    bits, tok, off, taken = 0, 0, 0, 0
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        ok = c >= 0 and n >= 0 and c + n < 2 ** 31 and P(c + n) <= most and 0 <= rows[b] < req_table.shape[0]
        t, need = max(n, 0), P(c + n) - P(c) if ok else 0
        fits, paged = tok + t <= total, need == 0 or off + need <= len(free)
        cu[b] = min(tok, total)
        if not ok or not fits:
            bits |= ops.DEVERR_LENGTH
        if not paged:
            bits |= ops.DEVERR_NO_PAGES
        if ok and fits and paged:
            seq[b] = c + n
            for p in range(P(c + n)):
                if p >= P(c):
                    req_table[rows[b], p] = free[off + p - P(c)]
                page_table[b, p] = req_table[rows[b], p]
            for i in range(n):
                page = int(page_table[b, (c + i) // ps])
                pos[tok + i] = c + i
                if 0 <= page < num_slots // ps:
                    loc[tok + i] = page * ps + (c + i) % ps
                else:
                    bits |= ops.DEVERR_PAGE_RANGE
            if need:
                taken = off + need
        tok += t
        off += need
    cu[B] = min(tok, total)
    return [page_table, np.array(seq), np.array(cu), np.array(pos), np.array(loc), np.array([taken]), req_table], bits


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def check(req_table, rows, cached, new, free, num_slots, ps, total, width, stream=None):
    B = len(cached)
    start = np.full((B, width), -5, dtype=np.int32)
    want, bits = tables(req_table, rows, cached, new, free, num_slots, ps, total, start)
    out = ops.StepTables(dev(start), dev(np.full(B, -9)), dev(np.full(B + 1, -9)), dev(np.full(total, -9)),
                         dev(np.full(total, -9)), dev([-9]))
    rt = dev(req_table)
    status = ops.new_status()
    got = ops.step_tables(rt, dev(cached), None if new is None else dev(new), dev(free), num_slots, ps,
                          req_rows=None if rows is None else dev(rows), out=out, status=status, stream=stream)
    assert ops.read_status(status, stream) == bits
    for name, x, y in zip(list(ops.StepTables._fields) + ["req_table"], list(got) + [rt], want):
        assert np.array_equal(x.cpu().numpy(), y), name
    return want


def resident(rng, rows, width, cached, row_of, ps, pages):
    """A table whose rows hold the cached tokens' pages, and the ids left over."""
    order = rng.permutation(pages).astype(np.int32)
    t = np.full((rows, width), -1, dtype=np.int32)
    k = 0
    for b, c in enumerate(cached):
        n = -(-c // ps)
        t[row_of[b], :n] = order[k:k + n]
        k += n
    return t, order[k:]


@pytest.mark.parametrize("ps", [1, 2, 16, 64, 256])
@pytest.mark.parametrize("B,chi,nhi", [(1, 0, 1), (1, 40, 700), (4, 200, 1), (33, 300, 1), (7, 90, 129), (70, 64, 64),
                                       (300, 20, 5), (3, 5000, 3000)])
def test_matches_the_loops(ps, B, chi, nhi):
    rng = np.random.default_rng(ps * 1000 + B)
    cached = rng.integers(0, chi, B, endpoint=True)
    new = rng.integers(0, nhi, B, endpoint=True)
    rows = rng.permutation(B + 5)[:B]
    width = -(-int((cached + new).max()) // ps) + int(rng.integers(0, 4))
    pages = sum(-(-int(c) // ps) for c in cached) + sum(-(-int(n) // ps) + 1 for n in new)
    table, free = resident(rng, B + 5, max(width + 3, 1), cached, rows, ps, pages)
    check(table, rows, cached, new, free, pages * ps, ps, int(new.sum()), max(width, 1))
    check(table, rows, cached, new, free, pages * ps, ps, int(new.sum()) + 37, max(width, 1))


@pytest.mark.parametrize("ps", [1, 16])
def test_decode_step_without_new_lens_or_rows(ps):
    cached = np.array([0, 15, 16, 17, 31, 100])
    rng = np.random.default_rng(3)
    table, free = resident(rng, 6, 128, cached, range(6), ps, 300)
    check(table, None, cached, None, free, 300 * ps, ps, 6, 128)


def test_empty_steps():
    check(np.zeros((2, 4), np.int32), None, np.zeros(0, int), np.zeros(0, int), np.arange(3), 64, 16, 0, 4)
    check(np.zeros((2, 4), np.int32), None, np.zeros(0, int), np.zeros(0, int), np.arange(3), 64, 16, 9, 4)
    check(np.zeros((2, 4), np.int32), None, np.array([0, 32]), np.array([0, 0]), np.zeros(0, int), 64, 16, 0, 4)


def test_refused_requests():
    rng = np.random.default_rng(5)
    cached = np.array([10, 30, -1, 16, 5, 40, 0])
    rows = np.array([0, 1, 2, 3, 4, 5, 6])
    table, free = resident(rng, 8, 6, np.maximum(cached, 0), rows, 16, 64)
    new = np.array([7, 3, 4, 16, 2, 30, 1])
    ok = dict(num_slots=1024, ps=16)

    def go(total=None, free=free, rows=rows, new=new, cached=cached, width=6, **kw):
        total = int(np.maximum(new, 0).sum()) if total is None else total
        return check(table, rows, cached, new, free, ok["num_slots"], 16, total, width)

    go()                                                     # a negative cached length
    go(new=np.array([7, 3, 4, -2, 2, 30, 1]))                # a negative new length
    go(rows=np.array([0, 1, 2, 8, 4, -1, 6]))                # rows outside the table
    go(width=4)                                              # 70 tokens need 5 columns
    go(total=28)                                             # tokens past the buffer: the last requests are refused
    go(free=free[:2])                                        # too few pages
    go(free=free[:0])
    go(new=np.array([7, 3, 4, 16, 2, 2 ** 31 - 1, 1]), total=100)
    bad = free.copy()
    bad[1] = 64                                              # a page id past the pool
    bad[0] = -3
    go(free=bad)


def test_rows_and_tables_far_apart():
    """Offsets that pass 32 bits: entries of a resident table of more than 2^31 ids."""
    rows, width = 70000, 32768
    t = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    t[69999, :3] = torch.tensor([5, 9, 2], dtype=torch.int32)
    out = ops.step_tables(t, dev([40]), dev([20]), dev([11, 12]), 1024, 16, total_tokens=20, width=8,
                          req_rows=dev([69999]))
    assert out.page_table.tolist() == [[5, 9, 2, 11, -1, -1, -1, -1]]
    assert t[69999, :5].tolist() == [5, 9, 2, 11, -1]
    assert out.out_loc.tolist() == [2 * 16 + 8 + i for i in range(8)] + [11 * 16 + i for i in range(12)]
    assert out.pages_taken.item() == 1


def test_captured_step():
    rng = np.random.default_rng(6)
    ps = 16
    c = [rng.integers(0, 200, 20) for _ in range(3)]
    n = [rng.integers(0, 50, 20) for _ in range(3)]
    total = max(int(x.sum()) for x in n) + 5
    made = [resident(rng, 20, 40, x, range(20), ps, 700) for x in c]
    rt, cached, new = dev(made[0][0]), dev(c[0]), dev(n[0])
    free = dev(np.full(120, -1))
    out = ops.StepTables(dev(np.full((20, 40), -1)), dev(np.zeros(20)), dev(np.zeros(21)), dev(np.zeros(total)),
                         dev(np.zeros(total)), dev([0]))
    free.copy_(dev(made[0][1][:120]))
    ops.step_tables(rt, cached, new, free, 700 * ps, ps, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.step_tables(rt, cached, new, free, 700 * ps, ps, out=out)
    for i in (1, 2, 0):
        table, left = made[i]
        rt.copy_(dev(table)), cached.copy_(dev(c[i])), new.copy_(dev(n[i])), free.copy_(dev(left[:120]))
        out.page_table.fill_(-1)
        graph.replay()
        want, bits = tables(table, None, c[i], n[i], left[:120], 700 * ps, ps, total, np.full((20, 40), -1, np.int32))
        assert bits == 0
        for x, y in zip(list(out) + [rt], want):
            assert np.array_equal(x.cpu().numpy(), y)


def test_on_another_stream():
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        check(np.zeros((2, 4), np.int32), None, np.array([3, 17]), np.array([40, 2]), np.arange(1, 9), 1024, 16, 42, 4,
              stream=s)


def test_tables_binding_refusals():
    rt, c, n, f = dev(np.zeros((4, 8))), dev([1, 2]), dev([3, 4]), dev(np.arange(8))
    good = dict(req_table=rt, cached_lens=c, new_lens=n, free_pages=f, num_slots=256, page_size=16, total_tokens=7)
    ops.step_tables(**good)
    for name, wrong in [("req_table", rt.long()), ("cached_lens", c.cpu()), ("new_lens", dev([1])),
                        ("free_pages", f.float()), ("req_rows", dev([0])), ("total_tokens", None),
                        ("req_table", dev(np.zeros((4, 16)))[:, ::2])]:
        with pytest.raises(ValueError):
            ops.step_tables(**dict(good, **{name: wrong}))
    for name, wrong, code in [("page_size", 3, 2), ("page_size", 512, 2), ("num_slots", 255, 1),
                              ("num_slots", 2 ** 31 + 16, 2), ("num_slots", -16, 1)]:
        with pytest.raises(ops.MsglError) as e:
            ops.step_tables(**dict(good, **{name: wrong}))
        assert e.value.status == code, (name, wrong)
    out = ops.step_tables(**good)
    for i, field in enumerate(out):
        with pytest.raises(ValueError):
            ops.step_tables(**dict(good, total_tokens=None),
                            out=ops.StepTables(*[dev(np.zeros((1, 1)) if j == 0 else np.zeros(2 + j)) if j == i else x
                                                 for j, x in enumerate(out)]))


# ---------------------------------------------------------------- shared prefixes

def groups(table, seq, ps, max_seq, min_shared):
    B, W = table.shape
    first, m, bits = list(range(B)), [0] * B, 0
    ok = [1 <= s <= max_seq and -(-s // ps) <= W for s in seq]
    for b in range(B):
        if not 1 <= seq[b] <= max_seq:
            bits |= ops.DEVERR_LENGTH
        elif not ok[b]:
            bits |= ops.DEVERR_PAGE_RANGE
        if b and ok[b] and ok[b - 1]:
            both = min(int(seq[b]), int(seq[b - 1]))
            d = 0
            while d < -(-both // ps) and table[b, d] == table[b - 1, d]:
                d += 1
            m[b] = min(d * ps, both)
            if m[b] >= min_shared:
                first[b] = first[b - 1]
    shared = [min([m[i] for i in range(B) if first[i] == first[b] and i != first[b]], default=0) for b in range(B)]
    return first, shared, bits


def check_groups(table, seq, ps, max_seq, min_shared):
    want = groups(np.asarray(table), seq, ps, max_seq, min_shared)
    status = ops.new_status()
    first, shared = ops.shared_prefixes(dev(table), dev(seq), ps, max_seq, min_shared, status=status)
    assert ops.read_status(status) == want[2]
    assert first.tolist() == want[0] and shared.tolist() == want[1]
    return want


@pytest.mark.parametrize("ps", [1, 16, 256])
@pytest.mark.parametrize("B,width", [(1, 1), (2, 3), (9, 40), (100, 70), (128, 256), (129, 256), (128, 257), (12, 9000),
                                     (1024, 5), (1025, 5), (1500, 9), (2100, 33)])
def test_groups_match_the_loops(ps, B, width):
    rng = np.random.default_rng(B + width + ps)
    table = np.zeros((B, width), np.int32)
    row = rng.integers(0, 1000, width)
    for b in range(B):
        # keep a random part of the row before (all of it now and then)
        keep = int(rng.integers(0, width + 1)) if rng.random() < 0.7 else width
        row = np.concatenate([row[:keep], rng.integers(0, 1000, width - keep)])
        table[b] = row
    seq = rng.integers(1, width * ps, B, endpoint=True)
    for min_shared in (1, ps, max(1, width * ps // 3), width * ps):
        check_groups(table, seq, ps, width * ps, min_shared)


def test_groups_of_equal_rows_and_odd_lengths():
    table = np.tile(np.arange(20, dtype=np.int32), (5, 1))
    assert check_groups(table, [320, 33, 320, 5, 100], 16, 320, 1)[1] == [5] * 5
    assert check_groups(table, [320, 33, 320, 5, 100], 16, 320, 6)[0] == [0, 0, 0, 3, 4]


def test_groups_with_bad_lengths():
    table = np.tile(np.arange(20, dtype=np.int32), (6, 1))
    check_groups(table, [100, 0, 100, 100, 400, 100], 16, 1000, 16)
    check_groups(table, [100, -5, 100, 101, 100, 2 ** 31 - 1], 16, 100, 16)


def test_groups_capture_and_refusals():
    table, seq = dev(np.tile(np.arange(8), (4, 1))), dev([100, 100, 100, 100])
    first, shared = dev([0] * 4), dev([0] * 4)
    ops.shared_prefixes(table, seq, 16, 128, 16, first, shared)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.shared_prefixes(table, seq, 16, 128, 16, first, shared)
    table[2, 3] = 77
    graph.replay()
    assert first.tolist() == [0, 0, 0, 0] and shared.tolist() == [48] * 4
    table[2, 0] = 77
    graph.replay()
    assert first.tolist() == [0, 0, 2, 3] and shared.tolist() == [100, 100, 0, 0]
    for bad in [dict(page_size=3), dict(min_shared=0), dict(max_seq_len=0)]:
        with pytest.raises(ops.MsglError):
            ops.shared_prefixes(**dict(dict(page_table=table, seq_lens=seq, page_size=16, max_seq_len=128,
                                            min_shared=16), **bad))
    for bad in [dict(page_table=table[0]), dict(seq_lens=seq[:2]), dict(seq_lens=seq.long()),
                dict(group_start=first[:2])]:
        with pytest.raises(ValueError):
            ops.shared_prefixes(**dict(dict(page_table=table, seq_lens=seq, page_size=16, max_seq_len=128,
                                            min_shared=16), **bad))
