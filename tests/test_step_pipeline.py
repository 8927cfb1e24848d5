"""A serving step's calls together: radix cache -> step tables -> store -> extend, then decode steps with
prefix groups and the shared decode, eager and as one captured graph; every result against the fp64 oracle."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_24_gb300 import ops
from paged_kv_attention_24_gb300.radix import RadixCache
from tests.parity import assert_lse_close, assert_o_close

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGES, WIDTH = 40, 8, 128, 400, 64


class Engine:
    """The device state of a small engine: a pool, a resident page table, the free pages."""

    def __init__(self, ps, seed):
        self.ps, self.gen = ps, torch.Generator(device="cuda").manual_seed(seed)
        self.pool = ops.KVPool(*[torch.full((PAGES * ps, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                                 for _ in range(2)], ps)
        self.table = torch.full((12, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.status = ops.new_status()

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def ok(self):
        assert ops.read_status(self.status) == 0

    def check(self, q, o, lse, table, seq):
        args = (q.cpu(), self.pool.k.cpu(), self.pool.v.cpu(), self.ps, table.cpu(), seq.cpu(), D ** -0.5)
        ref_o, ref_l = oracle.decode(*args)
        a, _ = oracle.decode(args[0], args[1], args[2].abs(), *args[3:])
        assert_o_close(o, ref_o, abs_ref=a)
        assert_lse_close(lse, ref_l)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def admitted(e, seed):
    """Requests that share parts of a cached prompt, prefilled through the step tables."""
    rng = np.random.default_rng(seed)
    cache = RadixCache(e.ps, PAGES)
    words = lambda n: rng.integers(0, 1000, size=n).tolist()
    base = words(40 * e.ps)
    tokens = [base + words(3)] + [base[:int(n * e.ps)] + words(m) for n, m in
                                  ((40, 5), (40, 2 * e.ps + 1), (40, 1), (25, 7), (25, 3 * e.ps), (0, e.ps), (0, 9))]
    n0, pages0, lease0 = cache.admit(tokens[0])
    rows = rng.permutation(12)[:len(tokens)]
    # the first request alone, then the others over what it left in the cache
    prompt = dict(row=rows[:1], cached=[0], toks=tokens[:1])
    free_order = [int(p) for p in pages0]
    for step, batch in enumerate((prompt, dict(row=rows[1:], cached=None, toks=tokens[1:]))):
        if step == 1:
            cache.insert(tokens[0][:40 * e.ps], np.asarray(pages0[:40]), lease0)
            got = [cache.admit(t) for t in batch["toks"]]
            batch["cached"] = [g[0] for g in got]
            free_order = []
            for r, (n, pages, _) in zip(batch["row"], got):
                keep = n // e.ps
                e.table[int(r), :keep] = i32(pages[:keep])
                free_order += [int(p) for p in pages[keep:]]
        new = [len(t) - c for t, c in zip(batch["toks"], batch["cached"])]
        T = sum(new)
        cached = i32(batch["cached"])
        out = ops.step_tables(e.table, cached, i32(new), i32(free_order + [-1, -1]), PAGES * e.ps, e.ps,
                              total_tokens=T, width=WIDTH, req_rows=i32(batch["row"]), status=e.status)
        assert out.pages_taken.item() == len(free_order)
        ops.store_kv(e.pool, e.normal(T, HKV, D), e.normal(T, HKV, D), out.out_loc, status=e.status)
        q = e.normal(T, HQ, D)
        longest = max(len(t) for t in batch["toks"])
        o, lse = ops.attn_extend(e.pool, q, out.page_table, cached, i32(new), out.cu_ext, max(new), longest, D ** -0.5,
                                 positions=out.positions, status=e.status)
        e.ok()
        last = (out.cu_ext[1:] - 1).long()
        e.check(q[last], o[last], lse[last], out.page_table, out.seq_lens)
        ops.check_extend_meta(PAGES * e.ps, e.ps, out.page_table, cached, i32(new), out.cu_ext, out.positions,
                              max(new), longest)
    used = set(int(p) for r in rows for p in e.table[int(r)].tolist() if p >= 0)
    left = [p for p in range(PAGES) if p not in used]
    return rows, [len(t) for t in tokens], left


@pytest.mark.parametrize("ps", [1, 16])
@pytest.mark.parametrize("sharing", ["auto", "always", "never"])
def test_decode_steps_over_radix_prefixes(ps, sharing):
    e = Engine(ps, 70 + ps)
    rows, seq, left = admitted(e, 5)
    # six requests share 25 pages, four of them 40: the threshold chooses
    for least, groups in ((16, ([0] * 6 + [6, 7], [25 * ps] * 6 + [0, 0])),
                          (30 * ps, ([0] * 4 + [4, 5, 6, 7], [40 * ps] * 4 + [0] * 4)),
                          (16, ([0] * 6 + [6, 7], [25 * ps] * 6 + [0, 0]))):
        B = len(seq)
        cached = i32(seq)
        out = ops.step_tables(e.table, cached, None, i32(left), PAGES * ps, ps, total_tokens=B, width=WIDTH,
                              req_rows=i32(rows), status=e.status)
        left = left[out.pages_taken.item():]
        ops.store_kv(e.pool, e.normal(B, HKV, D), e.normal(B, HKV, D), out.out_loc, status=e.status)
        first, shared = ops.shared_prefixes(out.page_table, out.seq_lens, ps, WIDTH * ps, least, status=e.status)
        assert (first.tolist(), shared.tolist()) == groups
        q = e.normal(B, HQ, D)
        o, lse = ops.attn_decode_shared(e.pool, q, out.page_table, out.seq_lens, first, shared, WIDTH * ps, D ** -0.5,
                                        status=e.status, sharing=sharing)
        e.ok()
        ops.check_groups_meta(PAGES * ps, ps, out.page_table, out.seq_lens, first, shared, WIDTH * ps)
        e.check(q, o, lse, out.page_table, out.seq_lens)
        seq = [s + 1 for s in seq]


@pytest.mark.parametrize("sharing", ["auto", "always"])
def test_one_captured_decode_step(sharing):
    """The four calls of a decode step in one graph; lengths and free pages change between replays, and the
    batch is padded with requests that the step refuses."""
    ps = 16
    e = Engine(ps, 90)
    rows, seq, left = admitted(e, 6)
    B = len(seq) + 2
    cached, req_rows = i32(list(seq) + [0, 0]), i32(list(rows) + [-1, -1])      # two rows of padding
    free = i32(left[:B])
    out = ops.step_tables(e.table, cached, None, free, PAGES * ps, ps, total_tokens=B, width=WIDTH, req_rows=req_rows)
    k, v, q = e.normal(B, HKV, D), e.normal(B, HKV, D), e.normal(B, HQ, D)
    first, shared, status = i32([0] * B), i32([0] * B), ops.new_status()
    ws = torch.empty(ops.decode_shared_workspace_size(B, HQ, HKV, WIDTH * ps), dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(q), torch.empty(B, HQ, device="cuda")

    def step():
        ops.step_tables(e.table, cached, None, free, PAGES * ps, ps, req_rows=req_rows, out=out, status=status)
        ops.store_kv(e.pool, k, v, out.out_loc, status=status)
        ops.shared_prefixes(out.page_table, out.seq_lens, ps, WIDTH * ps, 16, first, shared, status=status)
        ops.attn_decode_shared(e.pool, q, out.page_table, out.seq_lens, first, shared, WIDTH * ps, D ** -0.5, out=o,
                               lse=lse, workspace=ws, status=status, sharing=sharing)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        k.copy_(e.normal(B, HKV, D)), v.copy_(e.normal(B, HKV, D)), q.copy_(e.normal(B, HQ, D))
        status.zero_()
        graph.replay()
        # the padding is refused by the tables, skipped by the store and written as zero by the decode
        assert ops.read_status(status) == ops.DEVERR_LENGTH | ops.DEVERR_SLOT_RANGE
        assert out.out_loc[-2:].tolist() == [-1, -1] and out.seq_lens[-2:].tolist() == [0, 0]
        assert torch.all(o[-2:] == 0) and torch.all(lse[-2:] == float("-inf"))
        n = B - 2
        e.check(q[:n], o[:n], lse[:n], out.page_table[:n], out.seq_lens[:n])
        taken = out.pages_taken.item()
        left = left[taken:]
        free.copy_(i32(left[:B]))
        cached[:n] += 1
