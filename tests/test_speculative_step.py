"""A speculative serving loop on the device: free pages -> step tables -> rotary store -> extend over the drafts ->
verification, whose lengths are the next step's; then forks with their page copies, shared decode steps over them and a
compaction in between.  The pool is checked against what every request stored, the attention against the fp64 oracle;
eager, and as one captured graph with padded requests."""
import numpy as np
import pytest
import torch

import oracle
from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.parity import assert_lse_close, assert_o_close
from tests.step_reference import assert_rounded, i32, rope_rows

pytestmark = pytest.mark.gpu

HQ, HKV, D, PAGES, WIDTH, V = 16, 4, 128, 500, 90, 300
SCALE = D ** -0.5
FREQ = [1e4 ** (-j / 64) for j in range(64)]


class Engine:
    """Two layers' pools, a resident table, and per row what its tokens stored (read back once, when they were stored)."""

    def __init__(self, ps, rows, seed):
        self.ps, self.rng = ps, np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        nan = lambda: torch.full((PAGES * ps, HKV, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.pools = [ops.KVPool(nan(), nan(), ps) for _ in range(2)]
        self.table = torch.full((rows, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.rope, self.status = ops.Rope(FREQ), ops.new_status()
        self.stored = {}                       # row -> per layer (k, v) of its tokens

    def normal(self, *shape):
        return torch.randn(*shape, generator=self.gen, device="cuda").to(torch.bfloat16)

    def slots(self, row, n):
        t = self.table[row].tolist()
        return torch.tensor([t[j // self.ps] * self.ps + j % self.ps for j in range(n)], dtype=torch.long, device="cuda")

    def check_stored(self, rows, lens):
        for r, n in zip(rows, lens):
            at = self.slots(r, n)
            for pool, (k, v) in zip(self.pools, self.stored[r]):
                assert torch.equal(pool.k[at], k[:n]) and torch.equal(pool.v[at], v[:n]), r

    def store(self, t, rows, cached, new):
        """The step's tokens through the rotary store, in both layers; returns the turned q of each."""
        T = t.positions.shape[0]
        out = []
        for i, pool in enumerate(self.pools):
            qkv = self.normal(T, HQ + 2 * HKV, D)
            q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
            turned = ops.rope_store_kv(pool, q, k, v, t.positions, t.out_loc, self.rope, status=self.status)
            n = sum(new)
            pos = [t.positions[:n].tolist()]
            assert_rounded(turned[:n], *rope_rows(q[:n].cpu(), pos, FREQ, [0] * 64, False, 1.0, None, 0))
            loc = t.out_loc[:n].long()
            assert_rounded(pool.k[loc], *rope_rows(k[:n].cpu(), pos, FREQ, [0] * 64, False, 1.0, None, 0))
            assert torch.equal(pool.v[loc], v[:n])
            out.append(turned)
            for r, c, m, at in zip(rows, cached, new, np.concatenate([[0], np.cumsum(new)])):
                layers = self.stored.setdefault(r, [[torch.zeros(0, HKV, D, dtype=torch.bfloat16, device="cuda")] * 2 for _ in self.pools])
                layers[i] = [torch.cat([old[:c], x[loc[at:at + m]]]) for old, x in zip(layers[i], (pool.k, pool.v))]
        return out

    def ok(self):
        assert ops.read_status(self.status) == 0


def probabilities(e, T):
    z = 3 * torch.randn(T, V, generator=e.gen, device="cuda")
    return torch.softmax(z, -1), torch.softmax(z + 0.4 * torch.randn(T, V, generator=e.gen, device="cuda"), -1)


def speculative_step(e, rows, lens, most):
    """One step of the loop with up to `most` drafts a request; lens: the device's lengths, updated in place."""
    cached = lens.tolist()
    new = (1 + e.rng.integers(0, most + 1, len(rows))).tolist()
    T = sum(new)
    r = i32(rows, "cuda")
    ops.check_held_meta(PAGES * e.ps, e.ps, e.table, lens, r)
    free = ops.free_pages(e.table, lens, PAGES * e.ps, e.ps, r, status=e.status)
    used = ref.held_by(e.table.cpu().numpy(), rows, cached, PAGES, e.ps)
    assert free.pages[:free.num_free.item()].tolist() == np.nonzero(~used)[0].tolist()
    ops.check_step_meta(PAGES * e.ps, e.ps, e.table, r, lens, i32(new), free.pages[:free.num_free.item()], T)
    t = ops.step_tables(e.table, lens, i32(new, "cuda"), free.pages, PAGES * e.ps, e.ps, total_tokens=T, width=WIDTH, req_rows=r,
                        status=e.status)
    qs = e.store(t, rows, cached, new)
    for q, pool in zip(qs, e.pools):
        o, lse = ops.attn_extend(pool, q, t.page_table, lens, i32(new, "cuda"), t.cu_ext, max(new), WIDTH * e.ps, SCALE,
                                 positions=t.positions, status=e.status)
        args = (q.cpu(), pool.k.cpu(), pool.v.cpu(), e.ps, t.page_table.cpu(), i32(cached), i32(new), SCALE)
        want, want_lse = oracle.extend(*args)
        size, _ = oracle.extend(args[0], args[1], args[2].abs(), *args[3:])
        assert_o_close(o, want, abs_ref=size)
        assert_lse_close(lse, want_lse)
    p, q = probabilities(e, T)
    drawn = torch.multinomial(q, 1, generator=e.gen)[:, 0].int()
    tokens = torch.cat([drawn[:1], drawn[:-1]])
    au, su = torch.rand(T, generator=e.gen, device="cuda"), torch.rand(len(rows), generator=e.gen, device="cuda")
    ops.check_draft_meta(V, tokens, t.cu_ext, au, su)
    buf = torch.zeros(len(rows), dtype=torch.int32, device="cuda"), torch.zeros(T, dtype=torch.int32, device="cuda")
    got = ops.verify_drafts(p, q, tokens, t.cu_ext, au, su, cached_lens=lens, out=ops.Verified(*buf, lens), status=e.status)
    want = ref.verify(p.cpu(), q.cpu(), tokens.tolist(), t.cu_ext.tolist(), au.tolist(), su.tolist(), cached, [0] * T)
    for a, b in zip(got, want):
        assert a.tolist() == b.tolist()
    e.ok()
    e.check_stored(rows, lens.tolist())


@pytest.mark.parametrize("ps", [1, 16])
def test_loop_forks_decodes_and_compaction(ps):
    e = Engine(ps, 40, 30 + ps)
    order = e.rng.permutation(40).tolist()
    rows, lens = order[:6], torch.zeros(6, dtype=torch.int32, device="cuda")
    for most in (0, 30, 4, 4, 0, 6):
        speculative_step(e, rows, lens, most)
    # the first and the fourth request finish; the others get two more samples each, one of a shorter prefix
    live = [rows[i] for i in (1, 2, 4, 5)]
    n = lens[[1, 2, 4, 5]].tolist()
    parents, children = live + live, order[6:14]
    upto = n + [max(0, x - 3) for x in n]
    r = i32(live, "cuda")
    free = ops.free_pages(e.table, i32(n, "cuda"), PAGES * ps, ps, r, status=e.status)
    ops.check_fork_meta(PAGES * ps, ps, e.table, i32(parents), i32(children), i32(upto), free.pages[:free.num_free.item()])
    f = ops.fork_requests(e.table, i32(parents, "cuda"), i32(children, "cuda"), i32(upto, "cuda"), free.pages, PAGES * ps, ps,
                          status=e.status)
    ops.check_copy_meta(PAGES * ps, ps, f.src, f.dst, f.tokens)
    ops.copy_pages(e.pools, f.src, f.dst, f.tokens, status=e.status)
    e.ok()
    for a, b, m in zip(parents, children, upto):
        e.stored[b] = [[x[:m] for x in layer] for layer in e.stored[a]]
    # families next to each other, so that the decode reads a prefix once
    rows = [x for i in range(4) for x in (live[i], children[i], children[4 + i])]
    seq = [x for i in range(4) for x in (n[i], upto[i], upto[4 + i])]
    e.check_stored(rows, seq)
    lens = i32(seq, "cuda")
    for step in range(3):
        r = i32(rows, "cuda")
        free = ops.free_pages(e.table, lens, PAGES * ps, ps, r, status=e.status)
        t = ops.step_tables(e.table, lens, None, free.pages, PAGES * ps, ps, total_tokens=len(rows), width=WIDTH, req_rows=r,
                            status=e.status)
        qs = e.store(t, rows, lens.tolist(), [1] * len(rows))
        first, shared = ops.shared_prefixes(t.page_table, t.seq_lens, ps, WIDTH * ps, ps, status=e.status)
        if ps == 1:                            # (every family shares a page of one token)
            assert first.tolist()[::3] == [0, 3, 6, 9]
        for q, pool in zip(qs, e.pools):
            o, lse = ops.attn_decode_shared(pool, q, t.page_table, t.seq_lens, first, shared, WIDTH * ps, SCALE, status=e.status)
            args = (q.cpu(), pool.k.cpu(), pool.v.cpu(), ps, t.page_table.cpu(), t.seq_lens.cpu(), SCALE)
            want, want_lse = oracle.decode(*args)
            size, _ = oracle.decode(args[0], args[1], args[2].abs(), *args[3:])
            assert_o_close(o, want, abs_ref=size)
            assert_lse_close(lse, want_lse)
        lens = t.seq_lens
        e.ok()
        e.check_stored(rows, lens.tolist())
        if step == 1:
            c = ops.compact_pages(e.table, lens, PAGES * ps, ps, r, status=e.status)
            ops.copy_pages(e.pools, c.src, c.dst, count=c.num_moves, status=e.status)
            e.ok()
            used = ref.held_by(e.table.cpu().numpy(), rows, lens.tolist(), PAGES, ps)
            assert used[:c.num_used.item()].all() and used.sum() == c.num_used.item()
            e.check_stored(rows, lens.tolist())
    lens = lens.clone()
    speculative_step(e, rows, lens, 3)


def test_one_captured_speculative_step():
    """The five calls of a step in one graph: lengths stay on the device from replay to replay, drafts change, and
    two of the batch's places are padding."""
    ps, B, most = 16, 7, 4
    e = Engine(ps, 20, 77)
    rows = e.rng.permutation(20)[:5].tolist()
    r = i32(rows + [-1, -1], "cuda")
    T = B * (most + 1)
    lens, new = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")
    qkv = e.normal(T, HQ + 2 * HKV, D)
    q, k, v = qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]
    p, d = probabilities(e, T)
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    au, su = torch.zeros(T, device="cuda"), torch.zeros(B, device="cuda")
    zeros = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")
    pool, status = e.pools[0], ops.new_status()
    turned = torch.zeros(T, HQ, D, dtype=torch.bfloat16, device="cuda")
    tables = ops.StepTables(zeros(B, WIDTH), zeros(B), zeros(B + 1), zeros(T), zeros(T), zeros(1))
    free = ops.FreePages(zeros(PAGES), zeros(1))
    ws = torch.zeros(ops.page_map_workspace_size(PAGES * ps, ps), dtype=torch.uint8, device="cuda")
    verified = ops.Verified(zeros(B), zeros(T), lens)
    o, lse = torch.zeros_like(turned), torch.zeros(T, HQ, device="cuda")
    start = zeros(B)

    def step():
        ops.free_pages(e.table, lens, PAGES * ps, ps, r, out=free, workspace=ws, status=status)
        ops.step_tables(e.table, lens, new, free.pages, PAGES * ps, ps, req_rows=r, out=tables, status=status)
        ops.rope_store_kv(pool, q, k, v, tables.positions, tables.out_loc, e.rope, q_out=turned, status=status)
        ops.attn_extend(pool, turned, tables.page_table, lens, new, tables.cu_ext, most + 1, WIDTH * ps, SCALE, out=o, lse=lse,
                        status=status)
        start.copy_(lens)
        ops.verify_drafts(p, d, tokens, tables.cu_ext, au, su, cached_lens=lens, out=verified, status=status)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                 # (no request has a token yet)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(12):
        count = (1 + e.rng.integers(0, most + 1, 5)).tolist()
        new.copy_(i32(count + [0, 0]))
        n = sum(count)
        qkv.copy_(e.normal(T, HQ + 2 * HKV, D))
        for x, y in zip((p, d), probabilities(e, T)):
            x.copy_(y)
        drawn = torch.multinomial(d, 1, generator=e.gen)[:, 0].int()
        tokens.copy_(torch.cat([drawn[:1], drawn[:-1]]))
        au.uniform_(generator=e.gen), su.uniform_(generator=e.gen)
        status.zero_(), o.fill_(3.0), turned.fill_(5.0)
        graph.replay()
        # the step tables refuse the padding; nobody else minds it
        assert ops.read_status(status) == ops.DEVERR_LENGTH
        assert torch.all(turned[n:] == 5) and torch.all(o[n:] == 3)
        cached = start.tolist()
        assert cached[5:] == [0, 0] and lens[5:].tolist() == [0, 0]
        args = (turned[:n].cpu(), pool.k.cpu(), pool.v.cpu(), ps, tables.page_table[:5].cpu(), start[:5].cpu(), new[:5].cpu(), SCALE)
        want, want_lse = oracle.extend(*args)
        size, _ = oracle.extend(args[0], args[1], args[2].abs(), *args[3:])
        assert_o_close(o[:n], want, abs_ref=size)
        assert_lse_close(lse[:n], want_lse)
        want = ref.verify(p.cpu(), d.cpu(), tokens.tolist(), tables.cu_ext.tolist(), au.tolist(), su.tolist(), cached,
                          verified.tokens.tolist())
        for a, b in zip(verified, want):
            assert a.tolist() == b.tolist()
        loc = tables.out_loc[:n].long()
        for row, c, m, at in zip(rows, cached, count, np.concatenate([[0], np.cumsum(count)])):
            layer = e.stored.setdefault(row, [[torch.zeros(0, HKV, D, dtype=torch.bfloat16, device="cuda")] * 2])
            layer[0] = [torch.cat([old[:c], x[loc[at:at + m]]]) for old, x in zip(layer[0], (pool.k, pool.v))]
        e.check_stored(rows, lens[:5].tolist())
