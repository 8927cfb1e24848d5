"""Cases that measure the serving-step operators around the paged decode.

Three operators, each in a plain form (elementary torch operations in 32
bits) and as the library's calls:

* ``tables``: a step's block tables and slot maps from request lengths
  (``ops.step_tables``);
* ``groups``: the requests of a batch whose page tables share a prefix
  (``ops.shared_prefixes``);
* ``decode``: one query row per request, the keys that a group of requests
  shares read once for all of them (``ops.attn_decode_shared``).

The lengths of a case are a fixed multiset, so that its work is known
without a seed; the seed deals them out to the requests and draws the page
order and the values (and, where the groups are the answer, how far each
prefix is from its length).
"""
import math

import torch

own = False

HEAD_DIM = 128
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a handful of chat requests over one short system prompt, page size 1: latency
        dict(name="decode-b4-ps1", op="decode", hq=16, hkv=8, ps=1, batch=4, glo=4, ghi=4, slo=128, shi=128,
             olo=17, ohi=72),
        # parallel samples: groups of 8 continue one prompt each, page size 1
        dict(name="decode-samples-b256-ps1", op="decode", hq=16, hkv=8, ps=1, batch=256, glo=8, ghi=8, slo=100,
             shi=1024, olo=1, ohi=1024),
        # agents over documents of several lengths, uneven groups, some requests alone
        dict(name="decode-groups-b128-ps16", op="decode", hq=40, hkv=8, ps=16, batch=128, glo=1, ghi=31, slo=512,
             shi=4096, olo=1, ohi=1023),
        # a served model with one system prompt for all, then private histories
        dict(name="decode-system-b64-ps64", op="decode", hq=64, hkv=8, ps=64, batch=64, glo=64, ghi=64, slo=2048,
             shi=2048, olo=1024, ohi=6144),
        # questions to one long document: the shared part is nearly everything
        dict(name="decode-document-b256-ps64", op="decode", hq=64, hkv=8, ps=64, batch=256, glo=256, ghi=256,
             slo=32768, shi=32768, olo=1, ohi=512),
        # the step of a small decode batch: latency
        dict(name="tables-decode-b4-ps16", op="tables", ps=16, batch=4, clo=17, chi=200, nlo=1, nhi=1, pad=0),
        # the step of a full decode batch at page size 1 (a table entry for every token)
        dict(name="tables-decode-b256-ps1", op="tables", ps=1, batch=256, clo=100, chi=2047, nlo=1, nhi=1, pad=0),
        # chunked prefill next to decode rows: ragged chunks, buffers padded to a bucket
        dict(name="tables-mixed-b72-ps16", op="tables", ps=16, batch=72, clo=0, chi=4096, nlo=1, nhi=257, pad=513),
        # long prefills at page size 1: 64 requests, half a million table entries
        dict(name="tables-prefill-b64-ps1", op="tables", ps=1, batch=64, clo=0, chi=16384, nlo=1024, nhi=1024, pad=0),
        # a few system prompts, page size 64
        dict(name="groups-b64-ps64", op="groups", ps=64, batch=64, glo=8, ghi=24, slo=2048, shi=2048, olo=1024,
             ohi=6144),
        # parallel samples at page size 1: every token is a page
        dict(name="groups-b256-ps1", op="groups", ps=1, batch=256, glo=1, ghi=31, slo=128, shi=4096, olo=1, ohi=1024),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "decode", "tables", "tables", "groups"])
    ps = rng.choice([1, 1, 2, 8, 16, 16, 32, 64, 64, 256])
    if op == "tables":
        nhi = rng.choice([1, 1, _log_int(rng, 2, 1024)])
        batch = _log_int(rng, 1, 256 if nhi <= 64 else 64)
        chi = _log_int(rng, 1, 4096 if batch > 64 else 16384)
        nlo = 1 if nhi == 1 else rng.choice([0 if batch > 1 else 1, 1, nhi])
        return dict(op=op, ps=ps, batch=batch, clo=rng.randint(0, chi), chi=chi, nlo=nlo, nhi=nhi,
                    pad=rng.choice([0, rng.randint(1, 300)]))
    if op == "groups":
        batch = _log_int(rng, 12, 256)
        ghi = rng.randint(2, batch // 4)
        shi = ps * _log_int(rng, 16, max(16, 16384 // ps))
    else:
        batch = _log_int(rng, 1, 256)
        ghi = rng.randint(1, batch)
        shi = _log_int(rng, 1, 16384)
    ohi = _log_int(rng, 1, 4096 if batch <= 64 else 700)
    slo = rng.randint(max(1, 16 * ps if op == "groups" else shi // 4), shi)
    case = dict(op=op, ps=ps, batch=batch, glo=rng.randint(1, ghi), ghi=ghi, slo=slo, shi=shi,
                olo=rng.randint(1, ohi), ohi=ohi)
    if op == "decode":
        # no more keys in memory, and no more rows, than the largest listed case has
        hq, hkv = rng.choice([(8, 8), (16, 8), (32, 8), (40, 8), (64, 8), (32, 16), (28, 4), (16, 1)])
        groups = len(_groups(case))
        while groups * case["shi"] > 65536:
            case["shi"] = max(1, case["shi"] // 2)
            case["slo"] = min(case["slo"], case["shi"])
        case.update(hq=hq, hkv=hkv)
    return case


def _spread(lo, hi, n):
    """n whole numbers that cover [lo, hi] evenly, in an order without pattern."""
    return [lo + int((hi - lo + 1) * ((k + 1) * GOLDEN % 1.0)) for k in range(n)]


def _up(x, ps):
    return -(-x // ps) * ps


def _groups(case):
    """(requests, shared keys) of each group; a group of one shares nothing."""
    sizes, left, k = [], case["batch"], 0
    while left:
        n = min(left, case["glo"] + int((case["ghi"] - case["glo"] + 1) * ((k + 1) * GOLDEN % 1.0)))
        sizes.append(n)
        left -= n
        k += 1
    shared = _spread(case["slo"], case["shi"], len(sizes))
    return [(n, _up(s, case["ps"]) if n > 1 else 0) for n, s in zip(sizes, shared)]


def work(case):
    ps, batch = case["ps"], case["batch"]
    if case["op"] == "tables":
        cached, new = _lengths(case)
        old = sum(-(-c // ps) for c in cached)
        pages = sum(-(-(c + n) // ps) for c, n in zip(cached, new))
        need = pages - old
        tokens = sum(new) + case["pad"]
        # lengths and rows in, lengths and offsets out; old pages in, all pages out; the free
        # ids in and into the resident table; positions and slots out
        return {"bytes": 4 * (3 * batch + 2 * batch + 2 + old + pages + 2 * need + 2 * tokens), "flops": 0}
    groups = _groups(case)
    if case["op"] == "groups":
        # the shared pages of every request in a group, one page more to see where they part
        pages = sum(n * (s // ps) for n, s in groups) + batch
        return {"bytes": 4 * (pages + 3 * batch), "flops": 0}
    hq, hkv = case["hq"], case["hkv"]
    own_keys = sum(_spread(case["olo"], case["ohi"], batch))
    shared_keys = sum(s for _, s in groups)
    attended = own_keys + sum(n * s for n, s in groups)
    kv = (shared_keys + own_keys) * hkv * HEAD_DIM * 2 * 2
    rows = batch * hq * (HEAD_DIM * 2 * 2 + 4)
    return {"bytes": kv + rows, "flops": 4 * HEAD_DIM * hq * attended}


# ------------------------------------------------------------------ inputs

def _lengths(case):
    return (_spread(case["clo"], case["chi"], case["batch"]),
            _spread(case["nlo"], case["nhi"], case["batch"])[::-1])


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _deal(values, g):
    """The values in an order drawn from g."""
    v = _ints(values, torch.int64)
    return v[torch.randperm(len(values), generator=g, device="cuda")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_tables(case, g) if case["op"] == "tables" else _prepare_batch(case, g)


def _prepare_tables(case, g):
    ps, batch = case["ps"], case["batch"]
    cached, new = _lengths(case)
    c, n = _deal(cached, g), _deal(new, g)
    width = -(-(case["chi"] + case["nhi"]) // ps)
    rows = 2 * batch                       # the engine's table has rows for requests not in this step
    old = -(-c // ps)
    resident = batch * (-(-case["chi"] // ps))
    num_free = batch * (-(-case["nhi"] // ps) + 1)
    num_pages = resident + num_free + 7
    order = torch.randperm(num_pages, generator=g, device="cuda").int()
    req_rows = torch.randperm(rows, generator=g, device="cuda")[:batch].int()
    req_table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
    cols = torch.arange(width, device="cuda")
    start = torch.cumsum(old, 0) - old
    ids = order[(start[:, None] + cols[None, :]).clamp(max=resident)]
    req_table[req_rows.long()] = torch.where(cols[None, :] < old[:, None], ids, -1).int()
    tokens = sum(new) + case["pad"]
    i32 = dict(dtype=torch.int32, device="cuda")
    return dict(op="tables", ps=ps, num_slots=num_pages * ps, req_table=req_table, req_rows=req_rows, cached=c.int(),
                new=n.int(), free=order[resident:resident + num_free].contiguous(),
                # the buffers of a captured step: one of each, written by every step
                out=(torch.full((batch, width), -1, **i32), torch.zeros(batch, **i32), torch.zeros(batch + 1, **i32),
                     torch.zeros(tokens, **i32), torch.zeros(tokens, **i32), torch.zeros(1, **i32)))


def _prepare_batch(case, g):
    ps, batch = case["ps"], case["batch"]
    groups = _groups(case)
    groups = [groups[i] for i in torch.randperm(len(groups), generator=g, device="cuda").tolist()]
    own_len = _deal(_spread(case["olo"], case["ohi"], batch), g)
    size, shared_g = _ints([n for n, _ in groups], torch.int64), _ints([s for _, s in groups], torch.int64)
    max_seq = max(s for _, s in groups) + case["ohi"]
    if case["op"] == "groups":
        # the answer is the groups themselves: their prefixes are up to a quarter longer or shorter
        away = torch.rand(len(groups), generator=g, device="cuda", dtype=torch.float64) / 2 - 0.25
        shared_g = shared_g + (shared_g // ps * away).round().long() * ps
        max_seq += _up(max(s for _, s in groups) // 4, ps)
    group = torch.repeat_interleave(torch.arange(len(groups), device="cuda"), size, output_size=batch)
    shared = shared_g[group]
    seq = shared + own_len
    # pages: those of the shared prefixes, group after group, then each request's own
    sp, op = shared_g // ps, -(-own_len // ps)
    most = sum(s // ps + _up(s, 4 * ps) // ps // 4 for _, s in groups)
    s_at, o_at = torch.cumsum(sp, 0) - sp, most + torch.cumsum(op, 0) - op
    num_pages = most + sum(-(-o // ps) for o in _spread(case["olo"], case["ohi"], batch)) + 5
    order = torch.randperm(num_pages, generator=g, device="cuda").int()
    width = -(-max_seq // ps)
    col, mine = torch.arange(width, device="cuda")[None, :], sp[group][:, None]
    at = torch.where(col < mine, s_at[group][:, None] + col, o_at[:, None] + col - mine)
    pages = torch.where(col < (mine + op[:, None]), order[at.clamp(0, num_pages - 1)], -1).int().contiguous()
    first = (torch.cumsum(size, 0) - size)[group]
    state = dict(op=case["op"], ps=ps, pages=pages, seq=seq.int(), max_seq=max_seq)
    if case["op"] == "groups":
        return dict(state, min_shared=max(ps, 16))
    hq, hkv = case["hq"], case["hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    slots = num_pages * ps
    return dict(state, q=normal(batch, hq, HEAD_DIM), k=normal(slots, hkv, HEAD_DIM), v=normal(slots, hkv, HEAD_DIM),
                first=first.int(), shared=shared.int(), scale=HEAD_DIM ** -0.5,
                # what the program knows on the host: its groups (first row, rows, shared keys) and lengths
                group=group, size=size, shared_g=shared_g, biggest=max(n for n, _ in groups),
                longest=max(s for _, s in groups), longest_own=case["ohi"])


# --------------------------------------------------------------- operators

def run(state):
    return {"tables": _tables, "groups": _groups_of, "decode": _decode}[state["op"]](state)


def _tables(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        out = ops.step_tables(s["req_table"], s["cached"], s["new"], s["free"], s["num_slots"], s["ps"],
                              req_rows=s["req_rows"], out=ops.StepTables(*s["out"]))
        return list(out) + [s["req_table"]]
    ps = s["ps"]
    c, n, rows = s["cached"].long(), s["new"].long(), s["req_rows"].long()
    width, tokens = s["out"][0].shape[1], s["out"][3].shape[0]
    seq = c + n
    old, pages = (c + ps - 1) // ps, (seq + ps - 1) // ps
    need = pages - old
    taken = torch.cumsum(need, 0)
    cu = torch.cumsum(n, 0)
    col = torch.arange(width, device=c.device)[None, :]
    at = ((taken - need)[:, None] + col - old[:, None]).clamp(0, s["free"].shape[0] - 1)
    here = s["req_table"][rows]
    ids = torch.where((col >= old[:, None]) & (col < pages[:, None]), s["free"][at], here)
    s["req_table"][rows] = ids
    page_table = torch.where(col < pages[:, None], ids, s["out"][0])
    t = torch.arange(tokens, device=c.device)
    b = torch.searchsorted(cu, t, right=True)
    live = b < c.shape[0]
    b = b.clamp(max=c.shape[0] - 1)
    pos = torch.where(live, c[b] + t - (cu - n)[b], 0)
    slot = torch.where(live, ids[b, (pos // ps).clamp(max=width - 1)].long() * ps + pos % ps, -1)
    cu_ext = torch.cat([torch.zeros(1, dtype=torch.int64, device=c.device), cu])
    return [page_table, seq.int(), cu_ext.int(), pos.int(), slot.int(), taken[-1:].int(), s["req_table"]]


def _groups_of(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        return ops.shared_prefixes(s["pages"], s["seq"], s["ps"], s["max_seq"], s["min_shared"])
    ps, pt, seq = s["ps"], s["pages"], s["seq"].long()
    batch = seq.shape[0]
    if batch == 1:
        return torch.zeros_like(s["seq"]), torch.zeros_like(s["seq"])
    both = torch.minimum(seq[1:], seq[:-1])
    col = torch.arange(pt.shape[1], device=pt.device)[None, :]
    same = (pt[1:] == pt[:-1]) & (col < ((both + ps - 1) // ps)[:, None])
    lead = torch.cumprod(same.int(), 1).sum(1)
    m = torch.minimum(lead * ps, both)
    joined = torch.cat([torch.zeros(1, dtype=torch.bool, device=pt.device), m >= s["min_shared"]])
    row = torch.arange(batch, device=pt.device)
    first = torch.cummax(torch.where(joined, 0, row), 0).values
    far = torch.iinfo(torch.int64).max
    m = torch.where(joined, torch.cat([m[:1], m]), far)
    least = torch.full((batch,), far, device=pt.device).scatter_reduce(0, first, m, "amin")[first]
    return first.int(), torch.where(least == far, 0, least).int()


def _decode(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        return ops.attn_decode_shared(ops.KVPool(s["k"], s["v"], s["ps"]), s["q"], s["pages"], s["seq"], s["first"],
                                      s["shared"], s["max_seq"], s["scale"])
    ps, k, v = s["ps"], s["k"], s["v"]
    batch, hq, d = s["q"].shape
    hkv = k.shape[1]
    per = hq // hkv
    q = s["q"].float().view(batch, hkv, per, d) * s["scale"]
    pt, seq, shared, group = s["pages"].long(), s["seq"].long(), s["shared"].long(), s["group"]
    row = torch.arange(batch, device=q.device)
    parts = []
    if s["longest"] > 0:
        # the shared keys: the rows of a group together against its keys, groups padded to the biggest
        rank = row - s["first"].long()
        lead = torch.cumsum(s["size"], 0) - s["size"]
        key = torch.arange(s["longest"], device=q.device)[None, :]
        held = key < s["shared_g"][:, None]
        slot = pt[lead[:, None], torch.where(held, key, 0) // ps] * ps + torch.where(held, key, 0) % ps
        kk, vv = k[slot].float(), v[slot].float()
        rows = q.new_zeros(lead.shape[0], s["biggest"], hkv, per, d)
        rows[group, rank] = q
        rows = rows.permute(0, 2, 1, 3, 4).reshape(lead.shape[0], hkv, s["biggest"] * per, d)
        x = torch.matmul(rows, kk.permute(0, 2, 3, 1)).masked_fill(~held[:, None, None, :], -math.inf)
        top = x.amax(-1, keepdim=True)
        p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        o = torch.matmul(p, vv.permute(0, 2, 1, 3)).view(lead.shape[0], hkv, s["biggest"], per, d)
        top, tot = (y.view(lead.shape[0], hkv, s["biggest"], per) for y in (top, p.sum(-1)))
        parts.append((top[group, :, rank], tot[group, :, rank], o[group, :, rank]))
    # each request's own keys
    key = torch.arange(s["longest_own"], device=q.device)[None, :] + shared[:, None]
    held = key < seq[:, None]
    at = torch.where(held, key, 0)
    slot = pt[row[:, None], at // ps] * ps + at % ps
    kk, vv = k[slot].float(), v[slot].float()
    x = torch.matmul(q, kk.permute(0, 2, 3, 1)).masked_fill(~held[:, None, None, :], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    parts.append((top[..., 0], p.sum(-1), torch.matmul(p, vv.permute(0, 2, 1, 3))))
    # joined by their maxima and sums
    top = torch.stack([m for m, _, _ in parts]).amax(0)
    w = [torch.exp(m - top) for m, _, _ in parts]
    tot = sum(a * t for a, (_, t, _) in zip(w, parts))
    o = sum(a[..., None] * y for a, (_, _, y) in zip(w, parts)) / tot[..., None]
    return o.reshape(batch, hq, d).bfloat16(), (top + torch.log(tot)).reshape(batch, hq)


def exact(case, seed):
    """Softmax attention of every request over all of its keys, one request after another, in 64 bits."""
    if case["op"] != "decode":
        return None                        # whole numbers: equal or wrong
    s = prepare(case, seed)
    ps, hkv, per = case["ps"], case["hkv"], case["hq"] // case["hkv"]
    out, lse = [], []
    for b, n in enumerate(s["seq"].tolist()):
        pages = s["pages"][b, :-(-n // ps)].long()
        slots = (pages[:, None] * ps + torch.arange(ps, device="cuda")[None, :]).reshape(-1)[:n]
        kk, vv = s["k"][slots].double(), s["v"][slots].double()
        scores = torch.einsum("hgd,nhd->hgn", s["q"][b].double().view(hkv, per, HEAD_DIM), kk) / math.sqrt(HEAD_DIM)
        out.append(torch.einsum("hgn,nhd->hgd", torch.softmax(scores, -1), vv).reshape(-1, HEAD_DIM))
        lse.append(torch.logsumexp(scores, -1).reshape(-1))
    return torch.stack(out), torch.stack(lse)
