"""Decode batches whose groups of requests share prefix pages (seeded, on the CPU).

Unused pool slots hold NaN, page ids are handed out in a random order, and the
oracle sees the plain batch: every request's own full page table.
"""
import dataclasses

import numpy as np
import torch

import oracle


@dataclasses.dataclass
class SharedBatch:
    ps: int
    scale: float
    k: torch.Tensor
    v: torch.Tensor
    q: torch.Tensor
    seq: torch.Tensor          # int32 [B]
    table: torch.Tensor        # int32 [B, W]: every request's full table
    first: torch.Tensor        # int32 [B] group_start
    shared: torch.Tensor       # int32 [B]
    max_seq: int

    def cuda(self):
        return dataclasses.replace(self, **{f.name: getattr(self, f.name).cuda() for f in dataclasses.fields(self)
                                            if isinstance(getattr(self, f.name), torch.Tensor)})

    def recopy(self):
        """A request's copy of a partly shared page repeats the shared keys."""
        for b in range(len(self.seq)):
            s, lead = int(self.shared[b]), int(self.first[b])
            for j in range(s // self.ps * self.ps, s if lead != b else 0):
                at, src = (int(self.table[r, j // self.ps]) * self.ps + j % self.ps for r in (b, lead))
                self.k[at], self.v[at] = self.k[src], self.v[src]

    def reference(self):
        """(o, lse, o over |v|) in fp64."""
        o, lse = oracle.decode(self.q, self.k, self.v, self.ps, self.table, self.seq, self.scale)
        a, _ = oracle.decode(self.q, self.k, self.v.abs(), self.ps, self.table, self.seq, self.scale)
        return o, lse, a


def make(hq, hkv, ps, groups, seed, d=128, width=None, scale=None):
    """groups: a list of (shared keys, [own keys of each request]); a shared length that is not
    a whole number of pages is continued by each request's own keys on pages of its own, the
    last shared page repeated (the shared keys are those of the first request's)."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    pages = lambda n: -(-n // ps)
    total = sum(pages(s) + sum(pages(s % ps + o) for o in own) for s, own in groups) + 3
    order = list(rng.permutation(total))
    rows, seq, first, shared, used = [], [], [], [], set()
    for s, own in groups:
        head = [order.pop() for _ in range(pages(s))]
        lead = len(rows)
        for i, o in enumerate(own):
            whole = s // ps
            if i == 0:
                # the first request continues on the shared pages themselves
                t = head + [order.pop() for _ in range(pages(s + o) - len(head))]
            else:
                t = head[:whole] + [order.pop() for _ in range(pages(s + o) - whole)]
            rows.append(t)
            seq.append(s + o)
            first.append(lead)
            shared.append(s)
            used.update(t[j // ps] * ps + j % ps for j in range(s + o))
    slots = total * ps
    k = torch.randn(slots, hkv, d, generator=gen).to(torch.bfloat16)
    v = torch.randn(slots, hkv, d, generator=gen).to(torch.bfloat16)
    free = torch.ones(slots, dtype=torch.bool)
    free[list(used)] = False
    k[free] = float("nan")
    v[free] = float("nan")
    w = width or max(1, max(len(t) for t in rows))
    table = torch.full((len(rows), w), -1, dtype=torch.int32)
    for b, t in enumerate(rows):
        table[b, :len(t)] = torch.tensor([int(x) for x in t], dtype=torch.int32)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32)
    batch = SharedBatch(ps=ps, scale=scale or d ** -0.5, k=k, v=v,
                        q=torch.randn(len(rows), hq, d, generator=gen).to(torch.bfloat16), seq=i32(seq), table=table,
                        first=i32(first), shared=i32(shared), max_seq=max(seq))
    batch.recopy()
    return batch
