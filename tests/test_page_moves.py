"""Forks and page copies against their definitions: every table entry and every pool byte has to be equal."""
import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.step_reference import i32

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------- fork

def run_fork(table, parents, children, lens, free, num_pages, ps, flags=0, own=False):
    t, status = i32(table, "cuda"), ops.new_status()
    n = len(lens)
    out = None if own else ops.Forked(*[torch.full((k,), -9, dtype=torch.int32, device="cuda") for k in (n, n, n, 1)])
    args = [i32(x, "cuda") for x in (parents, children, lens, free)]
    got = ops.fork_requests(t, *args, num_pages * ps, ps, out=out, status=status)
    want = ref.fork(table, parents, children, lens, free, num_pages, ps)
    assert np.array_equal(t.cpu().numpy(), want[0])
    for name, a, b in zip(got._fields, got, want[1:4] + ([want[4]],)):
        assert a.tolist() == b, name
    assert ops.read_status(status) == flags
    return t, got


def tables(rows, width, num_pages, seed):
    rng = np.random.default_rng(seed)
    return rng.integers(0, num_pages, (rows, width)).astype(np.int32), rng


@pytest.mark.parametrize("ps", [1, 2, 16, 256])
@pytest.mark.parametrize("width,n", [(1, 3), (7, 5), (300, 40), (5000, 6)])
def test_forks(ps, width, n):
    table, rng = tables(2 * n + 3, width, 9000, width + ps)
    rows = rng.permutation(2 * n + 3)
    parents, children = rng.choice(rows[:3], n), rows[3:3 + n]
    lens = rng.integers(0, width * ps + 1, n)
    lens[0], lens[-1] = 0, width * ps
    run_fork(table, parents.tolist(), children.tolist(), lens.tolist(), rng.permutation(9000)[:n].tolist(), 9000, ps)
    run_fork(table, parents.tolist(), children.tolist(), lens.tolist(), rng.permutation(9000)[:n].tolist(), 9000, ps, own=True)


def test_one_token_and_the_borders_of_a_page():
    table, rng = tables(9, 4, 50, 1)
    run_fork(table, [0] * 8, list(range(1, 9)), [1, 15, 16, 17, 31, 32, 63, 64], [40, 41, 42, 43, 44], 50, 16)


def test_many_forks():
    n = 3000
    table, rng = tables(2 * n, 3, 10 ** 6, 2)
    rows = rng.permutation(2 * n)
    run_fork(table, rows[:n].tolist(), rows[n:].tolist(), rng.integers(0, 25, n).tolist(), rng.permutation(10 ** 6)[:n].tolist(),
             10 ** 6, 8)


def test_padding():
    table, rng = tables(6, 5, 99, 3)
    run_fork(table, [0, -1, 1, -1], [2, -1, 3, -1], [17, 5, 33, 99], [90, 91], 99, 16)


def test_refused_forks_leave_everything():
    table, rng = tables(8, 4, 60, 4)
    table[2] = [70, 1, -5, 3]
    f = ops.DEVERR_ROW
    run_fork(table, [0, 0], [8, 3], [17, 18], [50, 51], 60, 16, f)          # row outside
    run_fork(table, [-1, 0], [4, 3], [17, 18], [50, 51], 60, 16, f)
    run_fork(table, [0, -1], [-1, 3], [17, 18], [50, 51], 60, 16, f)
    run_fork(table, [0, 1], [3, 3], [17, 18], [50, 51], 60, 16, f)          # one child twice
    run_fork(table, [0, 3], [3, 4], [17, 18], [50, 51], 60, 16, f)          # a child that is a parent
    run_fork(table, [0], [0], [17], [50], 60, 16, f)
    run_fork(table, [0, 1], [3, 4], [-1, 18], [50, 51], 60, 16, ops.DEVERR_LENGTH)
    run_fork(table, [0, 1], [3, 4], [65, 18], [50, 51], 60, 16, ops.DEVERR_LENGTH)
    run_fork(table, [0, 1], [3, 4], [2 ** 31 - 1, 18], [50, 51], 60, 16, ops.DEVERR_LENGTH)
    run_fork(table, [0, 1, 0], [3, 4, 5], [17, 18, 32], [50], 60, 16, ops.DEVERR_NO_PAGES)
    run_fork(table, [0, 1], [3, 4], [17, 18], [], 60, 16, ops.DEVERR_NO_PAGES)
    run_fork(table, [0, 1], [3, 4], [17, 18], [60, 51], 60, 16, ops.DEVERR_PAGE_RANGE)
    run_fork(table, [0, 1], [3, 4], [17, 18], [-1, 51], 60, 16, ops.DEVERR_PAGE_RANGE)
    run_fork(table, [2, 2, 2], [3, 4, 5], [40, 5, 17], [50, 51, 52], 60, 16, ops.DEVERR_PAGE_RANGE)


def test_no_forks_and_no_columns():
    t = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    e = i32([], "cuda")
    out = ops.fork_requests(t, e, e, e, e, 64, 16)
    assert out.pages_taken.tolist() == [0]
    status = ops.new_status()
    out = ops.fork_requests(t, i32([0, 1], "cuda"), i32([2, -5], "cuda"), i32([0, 0], "cuda"), e, 64, 16, status=status)
    assert out.src.tolist() == [-1, -1] and ops.read_status(status) == ops.DEVERR_ROW


def test_fork_refusals():
    t = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    a, b, c = (i32(x, "cuda") for x in ([0], [1], [5]))
    for args in ((t, a, i32([1, 2], "cuda"), c, a), (t, a, b, None, a), (t, a.long(), b, c, a), (t[0], a, b, c, a),
                 (t.t(), a, b, c, a), (t, a, b.cpu(), c, a)):
        with pytest.raises(ValueError):
            ops.fork_requests(*args, 64, 16)
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.fork_requests(t, a, b, c, t.flatten()[8:], 64, 16)
    with pytest.raises(ops.MsglError, match="overlaps"):
        ops.fork_requests(t, a, b, c, a, 64, 16, out=ops.Forked(a, torch.zeros_like(a), torch.zeros_like(a), torch.zeros_like(a)))
    with pytest.raises(ops.MsglError):
        ops.fork_requests(t, a, b, c, a, 64, 24)


# ---------------------------------------------------------------------- copy

def pools(n, slots, hkv, ps, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    make = lambda: torch.randint(-2 ** 15, 2 ** 15, (slots, hkv, 128), generator=g, device="cuda").to(torch.int16).view(torch.bfloat16)
    return [ops.KVPool(make(), make(), ps) for _ in range(n)]


def run_copy(ps_pools, src, dst, tokens=None, count=None, flags=0, expect=None):
    ps = ps_pools[0].page_size
    want = []
    num_pages = ps_pools[0].k.shape[0] // ps
    pairs = list(zip(src, dst))[:len(src) if count is None else max(count, 0)]
    for p in ps_pools:
        for x in (p.k, p.v):
            y = x.view(torch.int16).cpu().clone()
            old = y.clone()
            for i, (s, d) in enumerate(pairs):
                n = ps if tokens is None else tokens[i]
                if 0 <= s < num_pages and 0 <= d < num_pages and 0 <= n <= ps:
                    y[d * ps:d * ps + n] = old[s * ps:s * ps + n]
            want.append(y)
    status = ops.new_status()
    ops.copy_pages(ps_pools, i32(src, "cuda"), i32(dst, "cuda"), None if tokens is None else i32(tokens, "cuda"),
                   None if count is None else i32([count], "cuda"), status=status)
    got = [x.view(torch.int16).cpu() for p in ps_pools for x in (p.k, p.v)]
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.read_status(status) == flags


@pytest.mark.parametrize("ps", [1, 2, 8, 16, 64, 256])
@pytest.mark.parametrize("hkv", [1, 3, 8])
@pytest.mark.parametrize("layers", [1, 3])
def test_copies(ps, hkv, layers):
    rng = np.random.default_rng(ps + hkv)
    pages = max(12, 600 // ps)
    p = pools(layers, pages * ps, hkv, ps)
    order = rng.permutation(pages)
    n = pages // 2 - 1
    src, dst = order[:n].tolist(), order[n:2 * n].tolist()
    run_copy(p, src, dst)
    run_copy(p, src, dst, rng.integers(0, ps + 1, n).tolist())
    run_copy(p, src[:1], dst[:1])


def test_one_page_to_many():
    p = pools(2, 64 * 16, 8, 16)
    run_copy(p, [5] * 40, list(range(10, 50)), [i % 17 for i in range(40)])


def test_padding_and_counts():
    p = pools(1, 40 * 16, 2, 16)
    run_copy(p, [1, -1, 3, 4, -1], [11, -1, 13, 14, -1], [3, 99, 16, 1, -4])
    for count in (-3, 0, 2, 5, 9):
        run_copy(p, [1, 2, 3, 4, -1], [21, 22, 23, 24, -1], count=count)


def test_long_lists_are_taken_in_groups():
    """Enough pairs that a warp looks at 32 of them; most are padding, some are wrong, the last group is not full."""
    ps, pages = 64, 300
    p = pools(3, pages * ps, 8, ps)
    n = 200001
    src, dst, tokens = np.full(n, -1), np.full(n, -1), np.full(n, -7)
    at = np.random.default_rng(3).permutation(n)[:100]
    at[:3] = 0, n - 1, n - 33
    src[at], dst[at], tokens[at] = np.arange(100), np.arange(150, 250), np.arange(100) % (ps + 1)
    bad = [i for i in range(40, 2000, 97) if src[i] == -1]
    src[bad[::2]] = 5
    dst[bad[1::2]] = pages
    run_copy(p, src.tolist(), dst.tolist(), tokens.tolist(), flags=ops.DEVERR_PAGE_RANGE)
    src[bad], dst[bad] = -1, -1
    run_copy(p, src.tolist(), dst.tolist())


def test_a_page_onto_itself_and_a_pool_named_twice():
    p = pools(2, 20 * 16, 8, 16)
    run_copy([p[0], p[1], p[0]], [5, 6], [5, 9])


def test_bad_pairs_are_passed_over():
    p = pools(2, 20 * 16, 8, 16)
    run_copy(p, [1, 20, 3], [11, 12, 13], flags=ops.DEVERR_PAGE_RANGE)
    run_copy(p, [1, 2, -1], [11, -2, 13], flags=ops.DEVERR_PAGE_RANGE)
    run_copy(p, [1, 2, 3], [11, 12, 13], [17, 16, -1], flags=ops.DEVERR_LENGTH)


def test_many_layers_in_several_launches():
    p = pools(150, 6 * 2, 1, 2)
    run_copy(p, [0, 1], [4, 5], [2, 1])


def test_single_pool_and_nothing_to_do():
    p = pools(1, 64, 1, 16)
    before = p[0].k.clone()
    ops.copy_pages(p[0], i32([0], "cuda"), i32([3], "cuda"))
    assert torch.equal(p[0].k[48:].view(torch.int16), before[:16].view(torch.int16))
    ops.copy_pages(p, i32([], "cuda"), i32([], "cuda"))
    ops.copy_pages([], i32([0], "cuda"), i32([1], "cuda"))


def test_pages_whose_offsets_pass_32_bits():
    hkv, ps = 64, 16
    slots = (2 ** 31 // (hkv * 128) // ps + 40) * ps
    k, v = (torch.zeros(slots, hkv, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    last = slots // ps - 1
    k[3 * ps:4 * ps].normal_(), v[3 * ps:4 * ps].normal_()
    ops.copy_pages(ops.KVPool(k, v, ps), i32([3], "cuda"), i32([last], "cuda"))
    assert torch.equal(k[last * ps:], k[3 * ps:4 * ps]) and torch.equal(v[last * ps:], v[3 * ps:4 * ps])
    k[:64 * ps], v[:64 * ps] = 0, 0
    ops.copy_pages(ops.KVPool(k, v, ps), i32([last], "cuda"), i32([7], "cuda"), i32([5], "cuda"))
    assert torch.equal(k[7 * ps:7 * ps + 5], k[last * ps:last * ps + 5]) and k[7 * ps + 5:8 * ps].count_nonzero() == 0
    assert v[8 * ps:64 * ps].count_nonzero() == 0


def test_copy_refusals():
    p = pools(2, 64, 1, 16)
    a, b = i32([0], "cuda"), i32([1], "cuda")
    for args in ((p, a, i32([1, 2], "cuda")), (p, a.long(), b), (p, a, b, i32([1, 2], "cuda")), (p, a, b, None, i32([1, 2], "cuda")),
                 (p, a.cpu(), b)):
        with pytest.raises(ValueError):
            ops.copy_pages(*args)
    with pytest.raises(ops.MsglError):
        ops.copy_pages([p[0], ops.KVPool(p[1].k, p[1].v, 8)], a, b)
    with pytest.raises(ops.MsglError):
        ops.copy_pages([p[0], ops.KVPool(p[1].k[:32], p[1].v[:32], 16)], a, b)
    with pytest.raises(AttributeError):
        ops.copy_pages([p[0], 5], a, b)
