"""msgl_attn_decode_shared where its kernels take their longer ways: many (pair of Q tiles, kv head) items for
one CTA of the shared keys' kernel, more rows than that kernel has threads, the largest batch of the contract,
and the choice that the device makes.

What a call did is read from the plan it leaves in the workspace: units of work per CTA, and for each row its
status bits, first own key, place in its pair of Q tiles (-1: no shared keys taken together) and pieces.
"""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.parity import assert_lse_close, assert_o_close
from tests.test_decode_shared import run
from tests.test_decode_shared_batch import recycled

pytestmark = pytest.mark.gpu

ROW_PLAN = 40   # bytes of a row's plan


def call(w, **kw):
    """Runs the batch on the GPU; returns (o, lse, status bits, units per CTA, rows' plans [B, 4])."""
    g = w.cuda()
    B, hq = g.q.shape[:2]
    n = ops.decode_shared_workspace_size(B, hq, g.k.shape[1], g.max_seq)
    ws, status = torch.empty(n, dtype=torch.uint8, device="cuda"), ops.new_status()
    o, lse = run(g, workspace=ws, status=status, **kw)
    at = n - -(-(256 + B * ROW_PLAN) // 256) * 256
    per = int(ws[at:at + 8].view(torch.int64).item())
    rows = ws[at + 256:at + 256 + B * ROW_PLAN].view(torch.int32).view(B, ROW_PLAN // 4)[:, :4].cpu()
    return o, lse, ops.read_status(status), per, rows


def check(w, o, lse, what="", rows=slice(None)):
    ref_o, ref_l, a = w.reference()
    assert_o_close(o[rows], ref_o[rows], what, abs_ref=a[rows])
    assert_lse_close(lse[rows], ref_l[rows], what)


# One key tile a group, so that an item is a unit, and long requests, which leave the shared keys to few CTAs.
# (hq, hkv, page size, groups, requests of a group, own keys): one Q tile and two, gathered rows, page boxes
# and 16-byte copies
MANY = [(1, 1, 16, 300, 2, 3000), (1, 1, 1, 300, 2, 4500), (8, 1, 64, 240, 3, 1500), (32, 1, 16, 130, 5, 1500),
        (32, 1, 2, 130, 5, 3500), (64, 2, 128, 90, 3, 3000), (16, 8, 16, 100, 4, 2000)]


@pytest.mark.parametrize("hq,hkv,ps,groups,n,own", MANY)
def test_more_items_a_cta_than_one_list_holds(hq, hkv, ps, groups, n, own):
    """A CTA's list holds 32 items; the refills carry the counters of every role over."""
    rng = np.random.default_rng(hq + ps)
    shared = lambda i: ps * (1 + i % (128 // ps)) if ps < 128 else 128
    w = recycled(hq, hkv, ps, [(shared(i), rng.integers(own - 200, own + 200, n).tolist()) for i in range(groups)],
                 seed=hq * 100 + ps)
    o, lse, bits, per, plan = call(w, sharing="always")
    assert bits == 0 and torch.all(plan[:, 0] == 0) and torch.all(plan[:, 2] >= 0)
    assert per > 40, per
    check(w, o, lse)
    again = call(w, sharing="always")
    assert torch.equal(again[0], o) and torch.equal(again[1], lse)

    # a bad page among the shared keys of groups in later lists marks their rows and no others
    bad = sorted({groups // 3, groups // 2 + 1, groups - 1})
    table = w.table.clone()
    lost = []
    for i in bad:
        table[i * n, 0] = 10 ** 6 if i % 2 else -1
        lost += range(i * n, i * n + n)
    o2, lse2, bits, per2, _ = call(dataclasses.replace(w, table=table), sharing="always")
    assert bits == ops.DEVERR_PAGE_RANGE and per2 == per
    assert torch.all(o2[lost] == 0) and torch.all(lse2[lost] == float("-inf"))
    keep = [b for b in range(groups * n) if b not in set(lost)]
    assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[keep], lse[keep])


@pytest.mark.parametrize("ps", [1, 16])
def test_more_rows_than_threads(ps):
    """Several rows for each thread of the count, the walk over them and the plan: 1300 requests in groups of 1 to 9
    that begin inside a thread's rows, with two and three key tiles."""
    sizes = [1 + (7 * i) % 9 for i in range(260)]
    groups = [(0 if n == 1 else 32 * (1 + (5 * i) % 11), [1 + (13 * i + 3 * j) % 40 for j in range(n)])
              for i, n in enumerate(sizes)]
    w = recycled(16, 2, ps, groups, seed=ps)
    assert len(w.seq) > 3 * 384
    for sharing in ("always", "auto", "never"):
        for max_seq in (w.max_seq, 40000):
            o, lse, bits, _, plan = call(dataclasses.replace(w, max_seq=max_seq), sharing=sharing)
            assert bits == 0
            if sharing == "always":
                assert torch.all((plan[:, 2] >= 0) == (w.shared > 0))
            check(w, o, lse, f"{sharing} {max_seq}")


def test_largest_batch():
    """65535 requests of a few keys each."""
    groups, left, i = [], 65535, 0
    while left:
        n = min(left, 1 + (11 * i) % 60)
        groups.append((16 * (i % 4), [1 + (i + j) % 5 for j in range(n)]))
        left -= n
        i += 1
    w = recycled(2, 1, 16, groups, seed=3)
    ref_o, ref_l, a = w.reference()
    for sharing, max_seq in (("always", 100), ("never", 100), ("never", 2000)):
        o, lse, bits, _, _ = call(dataclasses.replace(w, max_seq=max_seq), sharing=sharing)
        assert bits == 0
        assert_o_close(o, ref_o, sharing, abs_ref=a)
        assert_lse_close(lse, ref_l, sharing)


def test_auto_goes_both_ways():
    """Which way the device took stands in the plan: with little of their own the rows go through their shared
    keys together, and the result is that of "always" bit for bit; where the requests' own keys keep HBM busy for
    longer than it takes to read the shared ones once a request, they do not."""
    little = recycled(16, 8, 16, [(1280, [3 + i % 7 for i in range(40)]), (0, [5]), (960, [3] * 30)], seed=21,
                      pages=1000)
    o, lse, bits, _, plan = call(little)
    assert bits == 0 and torch.all((plan[:, 2] >= 0) == (little.shared > 0))
    check(little, o, lse)
    always = call(little, sharing="always")
    assert torch.equal(always[0], o) and torch.equal(always[1], lse)

    much = recycled(16, 8, 16, [(288, [3000 + i % 7 for i in range(40)]), (0, [2900])], seed=22, pages=1000)
    o, lse, bits, _, plan = call(much)
    assert bits == 0 and torch.all(plan[:, 2] == -1)
    check(much, o, lse)
    assert torch.any(call(much, sharing="always")[4][:, 2] >= 0)
