"""msgl_attn_decode_shared: what a row's result has to do with the rest of its batch, and large batches.

Requests take their pages at random from a small pool, so that many long requests stay cheap;
the fp64 oracle and the tolerances are those of the other tests of this call.
"""
import dataclasses

import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import shared_batch
from tests.parity import assert_lse_close, assert_o_close
from tests.test_decode_shared import VARIANTS, run, varied

pytestmark = pytest.mark.gpu


def recycled(hq, hkv, ps, groups, seed, pages=300):
    """groups: a list of (shared keys, a whole number of pages; [own keys of each request])."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    seq, first, shared = [], [], []
    for s, own in groups:
        assert s % ps == 0
        lead = len(seq)
        seq += [s + o for o in own]
        first += [lead] * len(own)
        shared += [s] * len(own)
    table = rng.integers(0, pages, (len(seq), -(-max(seq) // ps))).astype(np.int32)
    for b, (lead, s) in enumerate(zip(first, shared)):
        table[b, :s // ps] = table[lead, :s // ps]
    normal = lambda *shape: torch.randn(*shape, generator=gen).to(torch.bfloat16)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    return shared_batch.SharedBatch(ps=ps, scale=128 ** -0.5, k=normal(pages * ps, hkv, 128),
                                    v=normal(pages * ps, hkv, 128), q=normal(len(seq), hq, 128), seq=i32(seq),
                                    table=torch.from_numpy(table), first=i32(first), shared=i32(shared),
                                    max_seq=max(seq))


def rows_of(w, a, b):
    """Requests a..b-1 (whole groups) as a batch of their own."""
    cut = {n: getattr(w, n)[a:b].contiguous() for n in ("q", "seq", "table", "first", "shared")}
    cut["first"] = cut["first"] - a
    return dataclasses.replace(w, **cut)


@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("variant", list(VARIANTS))
def test_a_group_alone_and_in_a_batch(variant, ps):
    """The mode says how shared keys are read; the pieces of a row follow from the whole batch.  So a group
    gives the same result alone and among others up to the roundings, each within the bounds of exact
    arithmetic, and the same arguments give the same bits."""
    w = recycled(40, 8, ps, [(640, [1, 300, 77, 5]), (0, [900]), (160, [20, 7, 2000]), (1280, [9] * 11)], seed=ps)
    ref = w.reference()
    g, kw = varied(w, variant)
    whole = run(g.cuda(), **kw)
    for a, b in ((0, 4), (4, 5), (5, 8), (8, 19)):
        alone = run(rows_of(g, a, b).cuda(), **kw)
        for o, lse in (alone, (whole[0][a:b], whole[1][a:b])):
            assert_o_close(o, ref[0][a:b], f"{variant} {a}", abs_ref=ref[2][a:b])
            assert_lse_close(lse, ref[1][a:b], f"{variant} {a}")
    again = run(g.cuda(), **kw)
    assert torch.equal(again[0], whole[0]) and torch.equal(again[1], whole[1])
