"""Cases that measure the operators of a step around the paged cache: what is done to
the new tokens before they are stored, to drafted tokens after the attention, and to
the cache's pages between steps.

Six operators, each in a plain form (elementary torch operations in 32 bits, in 64
where angles or long sums need them) and as the library's calls:

* ``rope``: q and k normed per head and rotated by positions of one to three axes, q
  returned and k and v stored in the pool (``ops.rope_store_kv``);
* ``verify``: drafted tokens accepted or replaced by the target's probabilities
  (``ops.verify_drafts``);
* ``fork``: requests that continue other requests on the same pages
  (``ops.fork_requests``);
* ``copy``: pages copied in the pools of several layers (``ops.copy_pages``);
* ``free``: the pages that no request holds (``ops.free_pages``);
* ``compact``: the pages in use moved to the front of the pool
  (``ops.compact_pages``).

The lengths of a case are a fixed multiset, so that its work is known without a seed;
the seed deals them out to the requests and draws the page order and the values.
"""
import math

import torch

own = False

HEAD_DIM = 128
GOLDEN = 0.6180339887498949


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of a handful of chat requests, plain positions: latency
        dict(name="rope-decode-b4", op="rope", tokens=4, pad=0, hq=16, hkv=8, axes=1, pairs=64, norm=False, fused=False,
             adjacent=False, far=4096, ps=1),
        # chunked prefill beside decode rows, image positions (time, height, width), heads normed,
        # q, k and v columns of one projection, a bucket's padding behind the tokens
        dict(name="rope-mixed-t8256", op="rope", tokens=8256, pad=160, hq=64, hkv=8, axes=3, pairs=64, norm=True,
             fused=True, adjacent=False, far=40000, ps=64),
        # short drafts from looked-up text (no draft probabilities), bf16, odd vocabulary: latency
        dict(name="verify-b4-bf16", op="verify", batch=4, nlo=1, nhi=3, vocab=50001, dtype="bfloat16", given=False),
        # a full decode batch with a draft model, some requests without a draft
        dict(name="verify-b128", op="verify", batch=128, nlo=0, nhi=5, vocab=131072, dtype="float32", given=True),
        # four samples of one prompt: latency
        dict(name="fork-b4-ps16", op="fork", parents=1, kids=4, ps=16, clo=1000, chi=1000, spare=2.0),
        # groups of eight samples of long prompts, a table entry for every token
        dict(name="fork-b256-ps1", op="fork", parents=32, kids=8, ps=1, clo=512, chi=16384, spare=1.5),
        # the last pages of four forks, cut short, in eight layers: latency
        dict(name="copy-b4-l8", op="copy", pairs=4, layers=8, ps=16, hkv=8, tlo=1, thi=15, spare=16.0),
        # what a compaction moves: whole pages in four layers
        dict(name="copy-b1024-l4", op="copy", pairs=1024, layers=4, ps=16, hkv=8, tlo=16, thi=16, spare=2.5),
        # a decode batch's pool between two steps
        dict(name="free-b64-ps16", op="free", batch=64, group=1, ps=16, clo=500, chi=4096, spare=1.3, held=0.2),
        # parallel samples at page size 1, half a million pages
        dict(name="free-b256-ps1", op="free", batch=256, group=8, ps=1, clo=256, chi=3800, spare=1.4, held=0.1),
        # a pool that many finished requests left scattered
        dict(name="compact-b256-ps1", op="compact", batch=256, group=8, ps=1, clo=128, chi=2047, spare=2.0, held=0.05),
        # the same with larger pages and few requests
        dict(name="compact-b32-ps16", op="compact", batch=32, group=1, ps=16, clo=100, chi=4096, spare=3.0, held=0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "verify", "verify", "fork", "copy", "free", "compact"])
    ps = rng.choice([1, 1, 2, 8, 16, 16, 32, 64, 256])
    if op == "rope":
        hq, hkv = rng.choice([(8, 8), (16, 8), (32, 8), (40, 8), (64, 8), (32, 16), (28, 4), (16, 1)])
        return dict(op=op, tokens=_log_int(rng, 1, 8192), pad=rng.choice([0, 0, rng.randint(1, 60)]), hq=hq, hkv=hkv,
                    axes=rng.randint(1, 3), pairs=rng.choice([64, 64, 64, 48, 32, 16]), norm=rng.random() < 0.5,
                    fused=rng.random() < 0.5, adjacent=rng.random() < 0.3, far=_log_int(rng, 100, 1 << 20), ps=ps)
    if op == "verify":
        nhi = rng.randint(0, 8)
        vocab = _log_int(rng, 1000, 131072)
        return dict(op=op, batch=_log_int(rng, 1, min(128, max(1, (1 << 26) // (vocab * (nhi + 1))))),
                    nlo=rng.randint(0, nhi), nhi=nhi, vocab=vocab,
                    dtype=rng.choice(["float32", "float32", "bfloat16"]), given=rng.random() < 0.7)
    if op == "copy":
        layers, hkv = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8, 16])
        most = max(1, (1 << 28) // (4 * HEAD_DIM * ps * layers * hkv))
        thi = rng.choice([ps, rng.randint(1, ps)])
        return dict(op=op, pairs=_log_int(rng, 1, min(2048, most)), layers=layers, ps=ps, hkv=hkv,
                    tlo=rng.randint(0, thi), thi=thi, spare=rng.uniform(2.1, 3.0))
    chi = _log_int(rng, 1, 8192)
    clo = rng.randint(0, chi)
    if op == "fork":
        kids = rng.randint(1, 16)
        return dict(op=op, parents=_log_int(rng, 1, max(1, 256 // kids)), kids=kids, ps=ps, clo=clo, chi=chi,
                    spare=rng.uniform(1.1, 3.0))
    batch = _log_int(rng, 1, 256 if chi < 2048 else 96)
    return dict(op=op, batch=batch, group=rng.choice([1, rng.randint(1, batch)]), ps=ps, clo=clo, chi=chi,
                spare=rng.uniform(1.0, 3.0), held=rng.choice([0.0, rng.uniform(0.0, 0.5)]))


def _spread(lo, hi, n):
    """n whole numbers that cover [lo, hi] evenly, in an order without pattern."""
    return [lo + int((hi - lo + 1) * ((k + 1) * GOLDEN % 1.0)) for k in range(n)]


def _pages(x, ps):
    return -(-x // ps)


def _in_use(case):
    """(pages that a group shares, pages in use, pages held beside them, pages of the pool)"""
    batch = case.get("batch", case.get("parents"))
    group = case.get("group", 1)
    groups = -(-batch // group)
    shared = case["clo"] // 2 // case["ps"] if group > 1 else 0
    used = groups * shared + sum(_pages(x, case["ps"]) - shared for x in _spread(case["clo"], case["chi"], batch))
    held = int(used * case.get("held", 0.0))
    return shared, used, held, max(1, int((used + held) * case["spare"]) + case.get("kids", 0) * batch)


def work(case):
    op = case["op"]
    if op == "rope":
        # a pair takes two products and a sum for each of its two values, a normed one a square and a sum
        t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
        rotated = t * (hq + hkv)
        return {"bytes": 2 * 2 * HEAD_DIM * (rotated + t * hkv) + 4 * (t * case["axes"] + t + case["pad"]),
                "flops": rotated * (6 * case["pairs"] + (4 * HEAD_DIM if case["norm"] else 0))}
    if op == "verify":
        # the rows that a token is drawn from: the target's, and the draft's where there was one
        drafts = _spread(case["nlo"], case["nhi"], case["batch"])
        rows = case["batch"] + (sum(n > 0 for n in drafts) if case["given"] else 0)
        size = 4 if case["dtype"] == "float32" else 2
        tokens = sum(drafts) + case["batch"]
        return {"bytes": rows * case["vocab"] * size + 4 * 3 * tokens + 4 * 5 * case["batch"],
                "flops": 3 * case["batch"] * case["vocab"]}
    if op == "copy":
        tokens = sum(_spread(case["tlo"], case["thi"], case["pairs"]))
        return {"bytes": 2 * 2 * 2 * HEAD_DIM * case["hkv"] * tokens * case["layers"] + 4 * 3 * case["pairs"], "flops": 0}
    shared, used, held, num = _in_use(case)
    if op == "fork":
        n = case["parents"] * case["kids"]
        entries = sum(_pages(x, case["ps"]) for x in _spread(case["clo"], case["chi"], case["parents"]))
        return {"bytes": 4 * (entries + entries * case["kids"] + 7 * n), "flops": 0}
    entries = sum(_pages(x, case["ps"]) for x in _spread(case["clo"], case["chi"], case["batch"]))
    read = 4 * (entries + 2 * case["batch"]) + (num if case["held"] else 0)
    if op == "free":
        return {"bytes": read + 4 * num, "flops": 0}
    return {"bytes": read + 4 * (entries + num + num // 2 * 2), "flops": 0}


# ------------------------------------------------------------------ inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _deal(values, g):
    """The values in an order drawn from g."""
    v = _ints(values, torch.int64)
    return v[torch.randperm(len(values), generator=g, device="cuda")]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return {"rope": _prepare_rope, "verify": _prepare_verify, "copy": _prepare_copy}.get(case["op"], _prepare_table)(case, g)


def _prepare_rope(case, g):
    t, pad, hq, hkv, ps = case["tokens"], case["pad"], case["hq"], case["hkv"], case["ps"]
    every = t + pad

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if case["fused"]:
        qkv = normal(every, hq + 2 * hkv, HEAD_DIM)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = normal(every, hq, HEAD_DIM), normal(every, hkv, HEAD_DIM), normal(every, hkv, HEAD_DIM)
    slots = _pages(2 * every, ps) * ps
    loc = torch.randperm(slots, generator=g, device="cuda")[:every].int()
    loc[t:] = -1
    # the first axis counts on, the others are places in an image
    pos = torch.randint(0, case["far"], (case["axes"], every), generator=g, device="cuda", dtype=torch.int32)
    pos[1:] %= 1000
    pos[:, t:] = 0
    pairs = case["pairs"]
    inv_freq = 1e6 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    # pairs go to the axes in runs, the first axis the shortest one (16, 24, 24 of 64)
    first = pairs if case["axes"] == 1 else pairs // 2 if case["axes"] == 2 else pairs // 4
    rest = (pairs - first + max(1, case["axes"] - 1) - 1) // max(1, case["axes"] - 1)
    axes = [0 if j < first else 1 + (j - first) // rest for j in range(pairs)]
    weights = [1 + 0.1 * normal(HEAD_DIM) for _ in range(2)] if case["norm"] else [None, None]
    rope = dict(inv_freq=inv_freq, axes=axes, adjacent=case["adjacent"])
    return dict(op="rope", q=q, k=k, v=v, loc=loc, pos=pos, ps=ps, tokens=t, q_norm=weights[0], k_norm=weights[1],
                eps=1e-6, inv_freq=inv_freq.cuda(), axes=_ints(axes, torch.int64), adjacent=case["adjacent"], rope=rope,
                kept={}, k_pool=normal(slots, hkv, HEAD_DIM),
                v_pool=normal(slots, hkv, HEAD_DIM), out=torch.zeros(every, hq, HEAD_DIM, dtype=torch.bfloat16, device="cuda"))


def _prepare_verify(case, g):
    vocab, batch, dtype = case["vocab"], case["batch"], getattr(torch, case["dtype"])
    drafts = _deal(_spread(case["nlo"], case["nhi"], batch), g)
    cu = torch.cat([drafts.new_zeros(1), torch.cumsum(drafts + 1, 0)])
    rows = int(cu[-1])
    logits = 3 * torch.randn(rows, vocab, generator=g, device="cuda")
    p = torch.softmax(logits, -1)
    # every other row as a sampler leaves it that drops what is far below the likeliest token
    cut = torch.where(p < 0.02 * p.amax(-1, keepdim=True), 0.0, p)
    p[::2] = (cut / cut.sum(-1, keepdim=True))[::2]
    del cut
    q = torch.softmax(logits.add_(torch.randn(rows, vocab, generator=g, device="cuda"), alpha=0.7), -1)
    drawn = torch.multinomial(q, 1, generator=g)[:, 0]
    if not case["given"]:
        # text that was looked up is often what the target finds likeliest
        likely = p.argmax(-1)
        drawn = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.6, likely, drawn)
    # row r's draft is the step's token r + 1
    tokens = torch.cat([drawn[:1], drawn[:-1]]).int()
    return dict(op="verify", p=p.to(dtype), q=q.to(dtype) if case["given"] else None, tokens=tokens, cu=cu.int(),
                most=case["nhi"], accept=torch.rand(rows, generator=g, device="cuda"),
                sample=torch.rand(batch, generator=g, device="cuda"),
                cached=torch.randint(1, 4096, (batch,), generator=g, device="cuda", dtype=torch.int32),
                out=(_ints([0] * batch), _ints([0] * rows), _ints([0] * batch)))


def _prepare_copy(case, g):
    n, ps, hkv = case["pairs"], case["ps"], case["hkv"]
    num = max(2 * n, int(n * case["spare"]))
    order = torch.randperm(num, generator=g, device="cuda").int()
    tokens = _deal(_spread(case["tlo"], case["thi"], n), g).int()
    pools = [tuple(torch.randn(num * ps, hkv, HEAD_DIM, generator=g, device="cuda", dtype=torch.bfloat16)
                   for _ in range(2)) for _ in range(case["layers"])]
    return dict(op="copy", ps=ps, src=order[:n].contiguous(), dst=order[n:2 * n].contiguous(),
                tokens=None if case["tlo"] == ps else tokens, pools=pools, kept=[])


def _prepare_table(case, g):
    ps, group = case["ps"], case.get("group", 1)
    batch, kids = case.get("batch", case.get("parents")), case.get("kids", 0)
    shared, used, held, num = _in_use(case)
    lens = _deal(_spread(case["clo"], case["chi"], batch), g)
    width = max(1, _pages(case["chi"], ps) + 1)
    order = torch.randperm(num, generator=g, device="cuda").int()
    count = (lens + ps - 1) // ps
    mine = count - shared
    groups = -(-batch // group)
    at = groups * shared + torch.cumsum(mine, 0) - mine
    which = torch.arange(batch, device="cuda") // group
    col = torch.arange(width, device="cuda")[None, :]
    index = torch.where(col < shared, which[:, None] * shared + col, at[:, None] + col - shared)
    ids = torch.where(col < count[:, None], order[index.clamp(0, num - 1)], -1).int()
    rows = torch.randperm(2 * batch + kids * batch, generator=g, device="cuda")
    table = torch.full((rows.shape[0], width), -1, dtype=torch.int32, device="cuda")
    table[rows[:batch]] = ids
    state = dict(op=case["op"], ps=ps, num=num, table=table, rows=rows[:batch].int(), lens=lens.int())
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "fork":
        n = batch * kids
        who = torch.arange(batch, device="cuda").repeat_interleave(kids, output_size=n)
        return dict(state, parents=rows[:batch][who].int(), children=rows[batch:batch + n].int(), lens=lens[who].int(),
                    free=order[used:].contiguous(),
                    out=tuple(torch.zeros(k, **i32) for k in (n, n, n, 1)))
    state["held"] = None
    if held:
        state["held"] = torch.zeros(num, dtype=torch.uint8, device="cuda")
        state["held"][order[used:used + held].long()] = 1
    if case["op"] == "free":
        return dict(state, out=(torch.zeros(num, **i32), torch.zeros(1, **i32)))
    half = num // 2
    return dict(state, out=(torch.full_like(table, -1), torch.zeros(num, **i32), torch.zeros(half, **i32),
                            torch.zeros(half, **i32), torch.zeros(1, **i32), torch.zeros(1, **i32)))


# --------------------------------------------------------------- operators

def run(state):
    return {"rope": _rope, "verify": _verify, "fork": _fork, "copy": _copy, "free": _free,
            "compact": _compact}[state["op"]](state)


def _rotated(x, cos, sin, weight, eps, adjacent):
    """x [T, H, D] in the working type, normed where there is a weight; cos and sin [T, 1, pairs]."""
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight.to(x.dtype)
    n = cos.shape[-1]
    a, b, rest = (x[..., 0:2 * n:2], x[..., 1:2 * n:2], x[..., 2 * n:]) if adjacent else (
        x[..., :n], x[..., n:2 * n], x[..., 2 * n:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if adjacent else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def _rope(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        kept = s["kept"]                                    # as a program keeps its weights and its pool
        if not kept:
            kept.update(rope=ops.Rope(**s["rope"]), pool=ops.KVPool(s["k_pool"], s["v_pool"], s["ps"]))
        ops.rope_store_kv(kept["pool"], s["q"], s["k"], s["v"], s["pos"], s["loc"], kept["rope"], q_out=s["out"],
                          q_norm=s["q_norm"], k_norm=s["k_norm"], eps=s["eps"])
        return s["out"], s["k_pool"], s["v_pool"]
    t = s["tokens"]
    angle = s["pos"][s["axes"], :t].double().t() * s["inv_freq"]
    cos, sin = (f(angle).float()[:, None, :] for f in (torch.cos, torch.sin))
    s["out"][:t] = _rotated(s["q"][:t].float(), cos, sin, s["q_norm"], s["eps"], s["adjacent"]).bfloat16()
    slots = s["loc"][:t].long()
    s["k_pool"][slots] = _rotated(s["k"][:t].float(), cos, sin, s["k_norm"], s["eps"], s["adjacent"]).bfloat16()
    s["v_pool"][slots] = s["v"][:t]
    return s["out"], s["k_pool"], s["v_pool"]


def _verify(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        return tuple(ops.verify_drafts(s["p"], s["q"], s["tokens"], s["cu"], s["accept"], s["sample"],
                                       cached_lens=s["cached"], out=ops.Verified(*s["out"])))
    cu, rows, vocab = s["cu"].long(), s["p"].shape[0], s["p"].shape[1]
    first, drafts = cu[:-1], cu[1:] - cu[:-1] - 1
    i = torch.arange(max(s["most"], 1), device=cu.device)[None, :]
    live = i < drafts[:, None]
    row = torch.where(live, first[:, None] + i, 0)
    x = torch.where(live, s["tokens"].long()[(row + 1).clamp(max=rows - 1)], 0)
    px = s["p"][row, x].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"][row, x].double()
    ok = live & (s["accept"][row].double() * qx < px)
    taken = torch.cumprod(ok.int(), 1).sum(1)
    last = first + taken
    p = s["p"][last].float()
    left = taken < drafts
    if s["q"] is None:
        rejected = s["tokens"].long()[(last + 1).clamp(max=rows - 1)]
        index = torch.arange(vocab, device=cu.device)[None, :]
        w = torch.where(left[:, None] & (index == rejected[:, None]), 0.0, p)
    else:
        q = torch.where(left[:, None], s["q"][last].float(), 0.0)
        w = torch.where(p > q, p - q, 0.0)
    # nothing left over: the target's own distribution
    w = torch.where((w > 0).any(1)[:, None], w, p)
    run = torch.cumsum(w.double(), 1)
    at = (run <= s["sample"].double()[:, None] * run[:, -1:]).sum(1)
    token = torch.minimum(at, (w > 0).int().cumsum(1).argmax(1))
    accepted, out, lens = s["out"]
    accepted.copy_(taken)
    lens.copy_(s["cached"] + taken + 1)
    k = torch.arange(rows, device=cu.device)
    b = torch.searchsorted(cu, k, right=True) - 1
    place = k - first[b]
    out.copy_(torch.where(place < taken[b], s["tokens"][(k + 1).clamp(max=rows - 1)].long(),
                          torch.where(place == taken[b], token[b], -1)))
    return accepted, out, lens


def _fork(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        out = ops.fork_requests(s["table"], s["parents"], s["children"], s["lens"], s["free"], s["num"] * s["ps"], s["ps"],
                                out=ops.Forked(*s["out"]))
        return [s["table"]] + list(out)
    ps, table, lens = s["ps"], s["table"], s["lens"].long()
    parents, children = s["parents"].long(), s["children"].long()
    full, tail = lens // ps, lens % ps
    new = (tail > 0).long()
    place = torch.cumsum(new, 0) - new
    page = torch.where(tail > 0, s["free"][place.clamp(max=s["free"].shape[0] - 1)], -1)
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    theirs = table[parents]
    mine = torch.where(col < full[:, None], theirs, table[children])
    mine = torch.where((col == full[:, None]) & (tail > 0)[:, None], page[:, None], mine)
    source = torch.gather(theirs, 1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    table[children] = mine
    src, dst, tokens, taken = s["out"]
    src.copy_(torch.where(tail > 0, source, -1))
    dst.copy_(page)
    tokens.copy_(tail)
    taken.copy_(new.sum()[None])
    return [table, src, dst, tokens, taken]


def _copy(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        kept = s["kept"]
        if not kept:
            kept.extend(ops.KVPool(k, v, s["ps"]) for k, v in s["pools"])
        ops.copy_pages(kept, s["src"], s["dst"], tokens=s["tokens"])
        return [x for kv in s["pools"] for x in kv]
    ps = s["ps"]
    at = torch.arange(ps, device="cuda")[None, :]
    src, dst = ((s[k].long()[:, None] * ps + at) for k in ("src", "dst"))
    if s["tokens"] is not None:
        # the slots behind a page's copied tokens get what they hold
        src = torch.where(at < s["tokens"].long()[:, None], src, dst)
    src, dst = src.reshape(-1), dst.reshape(-1)
    return [x.index_copy_(0, dst, x[src]) for kv in s["pools"] for x in kv]


def _marked(s):
    """The pages that the requests hold, and those held beside them."""
    table = s["table"][s["rows"].long()]
    count = (s["lens"].long() + s["ps"] - 1) // s["ps"]
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    live = col < count[:, None]
    mark = torch.zeros(s["num"] + 1, dtype=torch.bool, device=table.device)
    mark[torch.where(live, table, s["num"]).long()] = True
    held = torch.zeros_like(mark[:-1]) if s["held"] is None else s["held"] != 0
    return mark[:-1], held, live, table


def _front(chosen, values, n):
    """The values where `chosen`, in order, in the front of n entries; -1 behind them."""
    place = torch.where(chosen, torch.cumsum(chosen, 0) - 1, n)
    return torch.full((n + 1,), -1, dtype=torch.int64, device=chosen.device).scatter_(0, place, values)[:n]


def _free(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        return tuple(ops.free_pages(s["table"], s["lens"], s["num"] * s["ps"], s["ps"], req_rows=s["rows"], held=s["held"],
                                    out=ops.FreePages(*s["out"])))
    mark, held, _, _ = _marked(s)
    free = ~(mark | held)
    pages, count = s["out"]
    pages.copy_(_front(free, torch.arange(s["num"], device=mark.device), s["num"]))
    count.copy_(free.sum()[None])
    return pages, count


def _compact(s):
    if own:
        from paged_kv_attention_24_gb300 import ops
        return list(ops.compact_pages(s["table"], s["lens"], s["num"] * s["ps"], s["ps"], req_rows=s["rows"],
                                      held=s["held"], out=ops.Compaction(*s["out"])))
    num = s["num"]
    mark, held, live, ids = _marked(s)
    used = mark | held
    total = used.sum()
    page = torch.arange(num, device=mark.device)
    moves = used & ~held & (page >= total)
    count = moves.sum()
    holes = ~used & (page < total)
    holes = holes & (torch.cumsum(holes, 0) <= count)
    half = num // 2
    src, dst = _front(moves, page, half), _front(holes, page, half)
    remap = torch.where(used, page, -1)
    remap = torch.cat([remap, remap[:1]]).scatter_(0, torch.where(src >= 0, src, num), dst)[:-1]
    table, new, from_, to, n_moves, n_used = s["out"]
    rows = s["rows"].long()
    table[rows] = torch.where(live, remap[ids.long().clamp(min=0)].int(), table[rows])
    new.copy_(remap)
    from_.copy_(src)
    to.copy_(dst)
    n_moves.copy_(count[None])
    n_used.copy_(total[None])
    return [table, new, from_, to, n_moves, n_used]


def exact(case, seed):
    """In 64 bits: rotation as a product with a complex number of unit length, and copies page by page.  The
    other operators' outputs are whole numbers."""
    if case["op"] == "copy":
        return _exact_copy(case, seed)
    if case["op"] != "rope":
        return None
    s = prepare(case, seed)
    t, n = s["tokens"], case["pairs"]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       s["pos"].double()[s["axes"]][:, :t].T.contiguous() * s["inv_freq"][None, :])

    def rotated(x, weight):
        x = x[:t].double()
        if weight is not None:
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / HEAD_DIM + s["eps"]) * weight.double()
        y = x.clone()
        at = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["adjacent"] else (slice(0, n), slice(n, 2 * n))
        z = torch.complex(x[..., at[0]].contiguous(), x[..., at[1]].contiguous()) * turn[:, None, :]
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        return y

    out, k_pool, v_pool = s["out"].double(), s["k_pool"].double(), s["v_pool"].double()
    out[:t] = rotated(s["q"], s["q_norm"])
    k_pool[s["loc"][:t].long()] = rotated(s["k"], s["k_norm"])
    v_pool[s["loc"][:t].long()] = s["v"][:t].double()
    return out, k_pool, v_pool


def _exact_copy(case, seed):
    s = prepare(case, seed)
    tokens = [case["ps"]] * case["pairs"] if s["tokens"] is None else s["tokens"].tolist()
    out = [x.double().view(-1, case["ps"], case["hkv"], HEAD_DIM) for kv in s["pools"] for x in kv]
    for src, dst, n in zip(s["src"].tolist(), s["dst"].tolist(), tokens):
        for x in out:
            x[dst, :n] = x[src, :n]
    return [x.view(-1, case["hkv"], HEAD_DIM) for x in out]
