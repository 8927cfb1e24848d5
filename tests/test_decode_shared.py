"""msgl_attn_decode_shared against the fp64 oracle run on every request's full page table.

The tolerances are those of every other parity test (tests/parity.py): P is
rounded to bf16 before the PV product (2^-8 of |v| under the softmax) and o
once at the end; a joined prefix adds fp32 arithmetic only.

Every case runs in each of the call's variants: the group's rows together
against its shared keys ("always"), shared keys read once a request by the
split kernel, or, for short requests, in a single launch ("never"; max_seq_len
is only a bound, and a larger one takes a short batch to the split kernel).
"""
import dataclasses

import pytest
import torch

import oracle
from paged_kv_attention_24_gb300 import ops
from tests import shared_batch
from tests.parity import assert_lse_close, assert_o_close

pytestmark = pytest.mark.gpu


def run(g, **kw):
    return ops.attn_decode_shared(ops.KVPool(g.k, g.v, g.ps), g.q, g.table, g.seq, g.first, g.shared, g.max_seq,
                                  g.scale, **kw)


# sharing, and the least max_seq_len: "auto" by a bound that leaves the choice to the device
VARIANTS = {"always": ("always", 0), "short": ("never", 0), "split": ("never", 2000), "auto": ("auto", 40000)}


def varied(w, variant):
    """The batch with the variant's bound, and the keyword that asks for the variant."""
    return dataclasses.replace(w, max_seq=max(w.max_seq, VARIANTS[variant][1])), dict(sharing=VARIANTS[variant][0])


def check(w, what=""):
    ref_o, ref_l, a = w.reference()
    for variant in VARIANTS:
        g, kw = varied(w, variant)
        status = ops.new_status()
        o, lse = run(g.cuda(), status=status, **kw)
        assert ops.read_status(status) == 0
        assert_o_close(o, ref_o, f"{what} {variant}", abs_ref=a)
        assert_lse_close(lse, ref_l, f"{what} {variant}")


def rising(n, lo, step):
    return [lo + step * i for i in range(n)]


CASES = {
    # (shared keys, own keys of each request), ...
    "alone": [(0, [1])],
    "alone-with-shared-len": [(40, [9])],
    "two": [(64, [1, 2])],
    "short-prefix": [(1, [1, 5, 17])],
    "no-prefix": [(0, [3, 130, 64])],
    "tile-minus-one": [(127, [1, 16])],
    "tile": [(128, [15, 1])],
    "tile-plus-one": [(129, [1, 16, 33])],
    "two-tiles": [(256, rising(9, 1, 7))],
    "nothing-of-its-own": [(300, [0, 4, 0])],
    "mixed": [(0, [50]), (513, [1, 100, 3]), (0, [700]), (64, [2, 2]), (1000, rising(5, 1, 31))],
    "long": [(5000, rising(6, 1, 90))],
}


@pytest.mark.parametrize("ps", [1, 16, 64, 256])
@pytest.mark.parametrize("case", list(CASES))
def test_matches_oracle(case, ps):
    check(shared_batch.make(16, 8, ps, CASES[case], seed=100 + ps), f"{case} ps {ps}")


# q heads, kv heads, and group sizes around the number of query rows a tile holds (128 / G) and
# around two tiles of them
@pytest.mark.parametrize("hq,hkv,n", [(8, 8, 130), (8, 8, 257), (16, 8, 63), (16, 8, 64), (16, 8, 65), (32, 16, 129),
                                      (40, 8, 25), (40, 8, 26), (40, 8, 51), (64, 8, 15), (64, 8, 16), (64, 8, 17),
                                      (64, 8, 33), (28, 4, 37), (48, 3, 20), (16, 1, 9), (64, 1, 2), (64, 1, 5),
                                      (5, 5, 140)])
def test_head_layouts_and_tile_edges(hq, hkv, n):
    check(shared_batch.make(hq, hkv, 16, [(0, [33]), (272, [1 + i % 40 for i in range(n)]), (48, [3, 9])],
                            seed=hq + n), f"{hq}/{hkv} x {n}")


@pytest.mark.parametrize("ps", [2, 4, 8, 32, 128])
def test_other_page_sizes(ps):
    check(shared_batch.make(40, 8, ps, [(333, [1, 20, 150]), (77, [5, 5])], seed=ps), f"ps {ps}")


@pytest.mark.parametrize("hq,hkv,ps", [(8, 1, 1), (16, 8, 1), (5, 5, 2), (64, 1, 4), (64, 32, 8)])
def test_many_short_requests_of_small_pages(hq, hkv, ps):
    """Requests of a few keys each, so most 16-key tiles of a range are nearly empty."""
    groups = [(20 + 3 * i, [1 + (7 * i + j) % (3 + i % 8) for j in range(30)]) for i in range(9)]
    check(shared_batch.make(hq, hkv, ps, groups + [(700, [1, 33, 250])], seed=60 + hkv), f"{hq}/{hkv} ps {ps}")


def test_many_groups_split_over_the_grid():
    groups = [(200 + 37 * i, [1 + (5 * i + j) % 23 for j in range(1 + i % 6)]) for i in range(60)]
    check(shared_batch.make(16, 8, 16, groups, seed=7))


@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("variant", list(VARIANTS))
def test_prefix_is_read_through_the_first_row(variant, ps):
    """The rows behind a group's first may hold anything in the shared columns."""
    w = shared_batch.make(40, 8, ps, [(320, [1, 50, 3]), (160, [20, 7])], seed=8)
    ref_o, ref_l, a = w.reference()
    for b in (1, 2, 4):
        w.table[b, :int(w.shared[b]) // ps] = -1
    w, kw = varied(w, variant)
    o, lse = run(w.cuda(), **kw)
    assert_o_close(o, ref_o, abs_ref=a)
    assert_lse_close(lse, ref_l)


def test_large_scores_and_scales():
    """Scores of a few hundred, growing along the sequence and then falling (the running
    maximum moves in every tile), and rows of which one side holds all the weight."""
    w = shared_batch.make(16, 8, 16, [(700, [1, 40, 300])], seed=9, scale=1.0)
    up = torch.linspace(0.05, 3.0, w.k.shape[0])[:, None, None]
    w.k = (w.k.float() * up).to(torch.bfloat16)
    w.recopy()
    check(w)
    w.k = (w.k.float().flip(0).nan_to_num(1.0)).to(torch.bfloat16)
    w.recopy()
    check(w)


@pytest.mark.parametrize("ps", [1, 16, 64])
def test_slots_whose_offsets_pass_32_bits(ps):
    """Pages at both ends of pools of 9 GB: the same results as side by side in a small one."""
    w = shared_batch.make(40, 8, ps, [(320, [1, 50, 3]), (0, [70, 200]), (700, [20, 7])], seed=9)
    slots = 4400000 // ps * ps
    assert slots * 8 * 128 > 2 ** 32
    pages, n = slots // ps, w.k.shape[0] // ps
    at = torch.arange(n)
    at = torch.where(at % 2 == 0, at, pages - 1 - at)
    free = torch.cuda.mem_get_info()[0]
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    k = torch.empty(slots, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    k.view(pages, -1)[at.cuda()] = w.k.view(n, -1).cuda()
    v.view(pages, -1)[at.cuda()] = w.v.view(n, -1).cuda()
    table = torch.where(w.table >= 0, at[w.table.clamp(min=0).long()].int(), w.table)
    for variant in VARIANTS:
        x, kw = varied(w, variant)
        want = run(x.cuda(), **kw)
        got = run(dataclasses.replace(x.cuda(), k=k, v=v, table=table.cuda()), **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), variant


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_repeats_are_bit_identical(variant):
    w = shared_batch.make(64, 8, 64, [(1600, rising(20, 1, 13)), (640, [5, 6])], seed=11)
    w, kw = varied(w, variant)
    g = w.cuda()
    a, b = run(g, **kw), run(g, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_dirty_workspace_and_outputs(variant):
    w = shared_batch.make(40, 8, 16, [(600, [1, 90, 3]), (0, [7])], seed=12)
    w, kw = varied(w, variant)
    g = w.cuda()
    clean = run(g, **kw)
    n = ops.decode_shared_workspace_size(4, 40, 8, g.max_seq)
    ws = torch.full((n // 4,), float("nan"), device="cuda").view(torch.uint8)
    out, lse = torch.full_like(g.q, float("nan")), torch.full((4, 40), float("nan"), device="cuda")
    run(g, workspace=ws, out=out, lse=lse, **kw)
    assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_rows_in_error_leave_the_others_alone(variant):
    w = shared_batch.make(16, 8, 16, [(160, [1, 40, 9]), (0, [20]), (320, [3, 4, 5, 6])], seed=13)
    w, kw = varied(w, variant)
    g = w.cuda()
    good = run(g, **kw)

    def expect(bits, rows, maybe=(), **changed):
        status = ops.new_status()
        o, lse = run(dataclasses.replace(g, **changed), status=status, **kw)
        assert ops.read_status(status) == bits
        for b in range(8):
            if b in rows or (b in maybe and torch.all(lse[b] == float("-inf"))):
                assert torch.all(o[b] == 0) and torch.all(lse[b] == float("-inf")), b
            else:
                # (a row in error may move the others' key ranges: equal up to the join's rounding)
                assert torch.allclose(o[b].float(), good[0][b].float(), atol=1e-2, rtol=2 ** -7), b
                assert torch.allclose(lse[b], good[1][b], atol=1e-4), b

    def edit(t, *changes):
        t = t.clone()
        for at, value in changes:
            t[at] = value
        return t

    expect(ops.DEVERR_PAGE_RANGE, {0, 1, 2}, table=edit(g.table, ((0, 4), 100000)))   # a shared page
    expect(ops.DEVERR_PAGE_RANGE, {5}, table=edit(g.table, ((5, 20), -7)))            # an own page
    expect(ops.DEVERR_PAGE_RANGE, {3}, table=edit(g.table, ((3, 1), -1)))
    expect(ops.DEVERR_LENGTH, {1}, seq=edit(g.seq, (1, 0)))
    expect(ops.DEVERR_LENGTH, {3, 7}, seq=edit(g.seq, (3, -4), (7, g.max_seq + 1)))
    expect(ops.DEVERR_LENGTH, {0}, seq=edit(g.seq, (0, 0)))                           # the first row of a group
    expect(ops.DEVERR_GROUP, {2}, seq=edit(g.seq, (2, 100)))                          # shorter than the prefix
    expect(ops.DEVERR_GROUP, {6}, shared=edit(g.shared, (6, 304)))
    # (group_start[b] is b or group_start[b - 1]: the row behind a wrong entry breaks the rule too)
    expect(ops.DEVERR_GROUP, {1, 2}, first=edit(g.first, (1, -1)))
    # (and the rows of its group behind that one may fall with it)
    expect(ops.DEVERR_GROUP, {5, 6}, {7}, first=edit(g.first, (5, 0)), shared=edit(g.shared, (5, 160)))
    expect(ops.DEVERR_GROUP, {3}, first=edit(g.first, (3, 7)))


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_every_row_in_error(variant):
    w = shared_batch.make(16, 8, 16, [(160, [1, 40, 9])], seed=19)
    w, kw = varied(w, variant)
    g = w.cuda()
    good = run(g, **kw)
    status = ops.new_status()
    bad = dataclasses.replace(g, seq=torch.tensor([0, 200, 169], dtype=torch.int32, device="cuda"),
                              shared=torch.tensor([160, 150, 140], dtype=torch.int32, device="cuda"))
    o, lse = run(bad, status=status, **kw)
    again = run(g, **kw)
    assert ops.read_status(status) == ops.DEVERR_LENGTH | ops.DEVERR_GROUP
    assert torch.all(o == 0) and torch.all(lse == float("-inf"))
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_narrow_table_is_a_page_error(variant):
    w = shared_batch.make(16, 8, 16, [(160, [1, 40]), (0, [20])], seed=14)
    w, kw = varied(w, variant)
    g = w.cuda()
    g.table = g.table[:, :9].contiguous()      # the prefix needs 10
    status = ops.new_status()
    o, lse = run(g, status=status, **kw)
    assert ops.read_status(status) == ops.DEVERR_PAGE_RANGE
    assert torch.all(o[:2] == 0) and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_nan_query_rows_stay_their_own(variant):
    w = shared_batch.make(64, 8, 64, [(500, rising(18, 1, 3))], seed=15)
    w, kw = varied(w, variant)
    g = w.cuda()
    good = run(g, **kw)
    g.q[3] = float("nan")
    g.q[9, 5] = float("inf")
    o, lse = run(g, **kw)
    keep = [b for b in range(18) if b not in (3, 9)]
    assert torch.equal(o[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_captured_replays_with_new_lengths_and_groups(variant):
    """One captured call serves steps with other groups and lengths."""
    a = shared_batch.make(40, 8, 16, [(320, [1, 50, 3, 9]), (160, [20, 7])], seed=16, width=64)
    b = shared_batch.make(40, 8, 16, [(0, [100]), (600, [1, 2]), (48, [30, 31, 32])], seed=17, width=64)
    slots = max(a.k.shape[0], b.k.shape[0])
    max_seq = max(a.max_seq, b.max_seq, VARIANTS[variant][1])
    k = torch.zeros(slots, 8, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    live = a.cuda()
    ws = torch.empty(ops.decode_shared_workspace_size(6, 40, 8, max_seq), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(live.q), torch.empty(6, 40, device="cuda")
    status = ops.new_status()

    def call():
        ops.attn_decode_shared(ops.KVPool(k, v, 16), live.q, live.table, live.seq, live.first, live.shared, max_seq,
                               a.scale, out=out, lse=lse, workspace=ws, status=status,
                               sharing=VARIANTS[variant][0])

    k[:a.k.shape[0]], v[:a.k.shape[0]] = live.k, live.v
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for w in (a, b, a):
        k[:w.k.shape[0]], v[:w.k.shape[0]] = w.k.cuda(), w.v.cuda()
        for name in ("q", "table", "seq", "first", "shared"):
            getattr(live, name).copy_(getattr(w, name))
        graph.replay()
        assert ops.read_status(status) == 0
        ref_o, ref_l, abs_ref = w.reference()
        assert_o_close(out, ref_o, abs_ref=abs_ref)
        assert_lse_close(lse, ref_l)


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_captured_with_its_own_scratch(variant):
    """A capture without a workspace takes its scratch from the graph's memory."""
    w, kw = varied(shared_batch.make(40, 8, 16, [(320, [1, 50, 3, 9]), (160, [20, 7])], seed=20), variant)
    ref_o, ref_l, abs_ref = w.reference()
    g = w.cuda()
    run(g, **kw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = run(g, **kw)
    for _ in range(3):
        o.fill_(float("nan")), lse.fill_(float("nan"))
        graph.replay()
        run(g, **kw)
        assert_o_close(o, ref_o, abs_ref=abs_ref)
        assert_lse_close(lse, ref_l)


@pytest.mark.parametrize("variant", list(VARIANTS))
def test_on_another_stream(variant):
    w = shared_batch.make(16, 8, 1, [(900, rising(8, 1, 11))], seed=18)
    ref_o, ref_l, a = w.reference()
    w, kw = varied(w, variant)
    g = w.cuda()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o, lse = run(g, stream=s, **kw)
    s.synchronize()
    assert_o_close(o, ref_o, abs_ref=a)
    assert_lse_close(lse, ref_l)


@pytest.mark.parametrize("ps", [1, 64])
@pytest.mark.parametrize("own", [3, 500])
def test_auto_takes_either_way(ps, own):
    """Batches large enough for the choice to be made on the device, from their lengths: with little of
    their own the shared keys are worth a pass of their own, with much they are not."""
    w = shared_batch.make(16, 8, ps, [(1200, [own + i % 7 for i in range(40)]), (0, [own]),
                                      (900, [own + i % 5 for i in range(30)])], seed=21)
    ref_o, ref_l, a = w.reference()
    g = w.cuda()
    status = ops.new_status()
    o, lse = run(g, status=status)
    assert ops.read_status(status) == 0
    assert_o_close(o, ref_o, abs_ref=a)
    assert_lse_close(lse, ref_l)


def test_binding_refusals():
    w = shared_batch.make(16, 8, 16, [(32, [1, 2])], seed=19)
    g = w.cuda()
    pool = ops.KVPool(g.k, g.v, 16)
    args = [g.q, g.table, g.seq, g.first, g.shared, g.max_seq, g.scale]
    for at, wrong in [(0, g.q.float()), (1, g.table.long()), (1, g.table[0]), (2, g.seq[:1]), (3, g.first.cpu()),
                      (4, g.shared.float()), (3, torch.zeros(4, dtype=torch.int32, device="cuda")[::2])]:
        bad = list(args)
        bad[at] = wrong
        with pytest.raises(ValueError):
            ops.attn_decode_shared(pool, *bad)
    with pytest.raises(ValueError):
        ops.attn_decode_shared(pool, *args, lse=torch.empty(2, 8, device="cuda"))
    with pytest.raises(ops.MsglError) as e:
        ops.attn_decode_shared(pool, *args, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 6
    with pytest.raises(KeyError):
        ops.attn_decode_shared(pool, *args, sharing="maybe")
