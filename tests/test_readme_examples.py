"""The README's examples of a step over drafted tokens, and of forks and a compaction behind it, run as they stand there."""
import os
import re

import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.step_reference import i32
from tests.test_speculative_step import D, FREQ, HKV, HQ, PAGES, SCALE, WIDTH, Engine, probabilities, speculative_step

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example(call):
    """The one example that makes this call."""
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if call in b]
    assert len(blocks) == 1
    return blocks[0]


@pytest.mark.parametrize("call", ["ops.verify_drafts", "ops.fork_requests"])
def test_examples_are_python(call):
    compile(example(call), "README.md", "exec")


@pytest.mark.gpu
@pytest.mark.parametrize("ps", [1, 16])
def test_forks_and_compaction(ps):
    e = Engine(ps, 12, 90 + ps)
    rows, lens = [9, 2, 11, 5], torch.zeros(4, dtype=torch.int32, device="cuda")   # (no request in row 0 or 1)
    for most in (30, 4):
        speculative_step(e, rows, lens, most)
    live, n = rows[1:], lens.tolist()[1:]              # the first request finishes
    parents, children, upto = [2, 2, 5, 11, 2], [0, 7, 10, 4, 9], [n[0], n[0] - 1, n[2], 0, n[0]]
    names = dict(ops=ops, torch=torch, req_table=e.table, rows=i32(live, "cuda"), lens=lens[1:].clone(), k_pool=e.pools[0].k,
                 page_size=ps, pools=e.pools, parents=i32(parents, "cuda"), children=i32(children, "cuda"),
                 fork_lens=i32(upto, "cuda"))
    exec(example("ops.fork_requests"), names)
    for a, b, m in zip(parents, children, upto):
        e.stored[b] = [[x[:m] for x in layer] for layer in e.stored[a]]
    rows, seq = names["rows"].tolist(), names["lens"].tolist()
    assert rows == live + children and seq == n + upto
    e.check_stored(rows, seq)
    used = ref.held_by(e.table.cpu().numpy(), rows, seq, PAGES, ps)
    assert used.sum() == names["c"].num_used.item() and used[:used.sum()].all()
    lens = names["lens"].clone()
    speculative_step(e, rows, lens, 3)                 # and they go on, each on pages of its own


@pytest.mark.gpu
def test_a_step_over_drafts():
    ps, rows = 16, [3, 1, 4]
    e = Engine(ps, 6, 91)
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    speculative_step(e, rows, lens, 20)
    cached, new = lens.tolist(), [1, 4, 3]
    T = sum(new)
    qkv = e.normal(T, HQ + 2 * HKV, D)
    p, d = probabilities(e, T)
    drawn = torch.multinomial(d, 1, generator=e.gen)[:, 0].int()
    names = dict(ops=ops, inv_freq=FREQ, req_table=e.table, lens=lens, k_pool=e.pools[0].k, page_size=ps, rows=i32(rows, "cuda"),
                 new_lens=i32(new, "cuda"), T=T, pool=e.pools[0], q=qkv[:, :HQ], k=qkv[:, HQ:HQ + HKV], v=qkv[:, HQ + HKV:],
                 max_new_len=max(new), max_seq_len=WIDTH * ps, scale=SCALE, target_probs=p, draft_probs=d,
                 tokens=torch.cat([drawn[:1], drawn[:-1]]), accept_u=torch.rand(T, generator=e.gen, device="cuda"),
                 sample_u=torch.rand(3, generator=e.gen, device="cuda"))
    exec(example("ops.verify_drafts"), names)
    t, out = names["t"], names["out"]
    want = ref.verify(p.cpu(), d.cpu(), names["tokens"].tolist(), t.cu_ext.tolist(), names["accept_u"].tolist(),
                      names["sample_u"].tolist(), cached, [-1] * T)
    for a, b in zip(out, want):
        assert a.tolist() == b.tolist()
    assert names["lens"] is out.kv_lens and names["o"].shape == (T, HQ, D) and names["o"].isfinite().all()
    # the table holds the new tokens' pages, and the pool their values
    for r, c, m, at in zip(rows, cached, new, (0, 1, 5)):
        slots = e.slots(r, c + m)[c:]
        assert t.out_loc[at:at + m].tolist() == slots.tolist()
        assert torch.equal(e.pools[0].v[slots], names["v"][at:at + m])
