"""Plain references, on the CPU and in 64 bits, of the operators around a step: the rotary store, the
verification of drafts, forks, copies, free pages and compaction (one loop per definition, nothing shared
with the kernels)."""
import math

import numpy as np
import torch


def i32(x, device="cpu"):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=device)


# -------------------------------------------------------------- rotary store

def rope_rows(x, pos, inv_freq, axes, adjacent, factor, weight, eps):
    """(turned heads, bound of what 32 bits may be off) of x [T, H, 128]; pos [A, T]."""
    x = x.double()
    if weight is not None:
        x = x * weight.double() / torch.sqrt((x ** 2).mean(-1, keepdim=True) + eps)
    y, size = x.clone(), x.abs()
    n = len(inv_freq)
    for j in range(n):
        a, b = (2 * j, 2 * j + 1) if adjacent else (j, j + n)
        # whole turns taken out in whole numbers of 2^-80 turns, so that far positions lose nothing
        step = round(float(inv_freq[j]) / (2 * math.pi) * 2 ** 80)
        angle = torch.tensor([int(p) * step % 2 ** 80 / 2 ** 80 * 2 * math.pi for p in pos[axes[j]]], dtype=torch.float64)
        c, s = torch.cos(angle)[:, None] * factor, torch.sin(angle)[:, None] * factor
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(factor)
    # The norm: 19 additions of squares, a root, a quotient and two products of 2^-24 each, halved by the root where
    # they stand under it: below 14 * 2^-24.  The angle: 2^-25 of half a turn (pi * 2^-25 at most) and 1.5 * 2^-53 of a
    # turn a position (below 2^-20.5 at 2^31 positions for frequencies up to 1), the functions 2 units of 2^-24, the
    # rotation 3 roundings: below 2^-19 of |x| + |y| together.
    return y, size * 2.0 ** -19


def assert_rounded(got, want, slack):
    """got (bf16) is want to within half a step of bf16 and the slack of its computation."""
    off = (got.double().cpu() - want).abs()
    allowed = (want.abs() + slack) * 2.0 ** -8 + slack + 2.0 ** -134
    worst = (off - allowed).max().item() if off.numel() else 0.0
    assert worst <= 0, (worst, off.max().item())


# -------------------------------------------------------------------- drafts

def verify(p, q, tokens, cu, accept_u, sample_u, cached, out):
    """(accepted, out tokens, kv lengths) as numpy arrays; out: what the tokens hold before."""
    p64 = p.double().numpy()
    q64 = None if q is None else q.double().numpy()
    p32, q32 = p.float().numpy(), None if q is None else q.float().numpy()
    V = p.shape[1]
    out = np.array(out)
    accepted, lens = [], []
    for b in range(len(sample_u)):
        first, end = int(cu[b]), int(cu[b + 1])
        start = 0 if cached is None else int(cached[b])
        if not 0 <= first < end <= len(tokens):
            accepted.append(0)
            lens.append(start)
            continue
        a = 0
        while a < end - first - 1:
            r, x = first + a, int(tokens[first + a + 1])
            if not 0 <= x < V:
                break
            if not float(accept_u[r]) * (1.0 if q is None else q64[r, x]) < p64[r, x]:
                break
            a += 1
        r = first + a
        row = np.where(p32[r] > 0, p32[r], np.float32(0)).astype(np.float64)
        w = row
        if r < end - 1:
            x = int(tokens[r + 1])
            if q is None:
                w = row.copy()
                if 0 <= x < V:
                    w[x] = 0
            else:
                with np.errstate(invalid="ignore"):
                    w = np.where(p32[r] > q32[r], p32[r] - q32[r], np.float32(0)).astype(np.float64)
            if not 0 < math.fsum(w) < math.inf:
                w = row
        total = math.fsum(w) if np.isfinite(w).all() else math.inf
        if 0 < total <= 3.4e38:
            run = np.cumsum(w.astype(np.longdouble))
            u = float(sample_u[b])
            over = np.nonzero((run > u * run[-1]) & (w > 0))[0]
            token = int(over[0]) if len(over) else int(np.nonzero(w > 0)[0][-1])
        else:
            token = -1
        for i in range(end - first):
            out[first + i] = int(tokens[first + i + 1]) if i < a else token if i == a else -1
        accepted.append(a)
        lens.append(start + a + 1)
    return np.array(accepted), out, np.array(lens)


# --------------------------------------------------------------------- pages

def pages_of(n, ps):
    return -(-n // ps)


def fork(table, parents, children, lens, free, num_pages, ps):
    """(table, src, dst, tokens, taken); the forks that break a rule change nothing."""
    old, table = np.array(table), np.array(table)
    rows, width = table.shape
    src, dst, tokens = [], [], []
    taken = 0
    for i, (a, b, n) in enumerate(zip(parents, children, lens)):
        one = (-1, -1, 0)
        fits = 0 <= a < rows and 0 <= b < rows and n >= 0 and pages_of(n, ps) <= width
        tail, full = n % ps, n // ps
        clash = any(b == x for x in parents) or any(b == x for k, x in enumerate(children) if k != i)
        place, needs = taken, fits and tail > 0
        taken += needs
        if fits and not clash and not (needs and place >= len(free)):
            page, from_ = (int(free[place]), int(old[a, full])) if needs else (-1, -1)
            if not needs or (0 <= page < num_pages and 0 <= from_ < num_pages):
                table[b, :full] = old[a, :full]
                if needs:
                    table[b, full] = page
                    one = (from_, page, tail)
        for x, y in zip((src, dst, tokens), one):
            x.append(y)
    return table, src, dst, tokens, min(taken, len(free))


def held_by(table, rows, lens, num_pages, ps):
    """The pages that the requests hold."""
    mark = np.zeros(num_pages, bool)
    for r, n in zip(range(len(lens)) if rows is None else rows, lens):
        if 0 <= r < table.shape[0]:
            k = pages_of(n, ps) if n >= 0 and pages_of(n, ps) <= table.shape[1] else table.shape[1]
            ids = table[r, :k]
            mark[ids[(ids >= 0) & (ids < num_pages)]] = True
    return mark


def names_no_page(table, rows, lens, num_pages, ps):
    """Does a request's row name an id outside the pool among those it holds?"""
    for r, n in zip(range(len(lens)) if rows is None else rows, lens):
        if 0 <= r < table.shape[0]:
            k = pages_of(n, ps) if n >= 0 and pages_of(n, ps) <= table.shape[1] else table.shape[1]
            if ((table[r, :k] < 0) | (table[r, :k] >= num_pages)).any():
                return True
    return False


def compact(table, rows, lens, held, num_pages, ps, into=None):
    """(table, remap, src, dst, moves, used)"""
    old = np.array(table)
    new = np.array(old if into is None else into)
    mine = held_by(old, rows, lens, num_pages, ps)
    other = np.zeros(num_pages, bool) if held is None else np.asarray(held) != 0
    used = mine | other
    total = int(used.sum())
    go = [p for p in range(total, num_pages) if mine[p] and not other[p]]
    to = [p for p in range(total) if not used[p]][:len(go)]
    remap = np.where(used, np.arange(num_pages), -1)
    remap[go] = to
    for r, n in zip(range(len(lens)) if rows is None else rows, lens):
        if 0 <= r < old.shape[0]:
            k = pages_of(n, ps) if n >= 0 and pages_of(n, ps) <= old.shape[1] else old.shape[1]
            for c in range(k):
                p = old[r, c]
                new[r, c] = remap[p] if 0 <= p < num_pages else p
    pad = [-1] * (num_pages // 2 - len(go))
    return new, remap, go + pad, to + pad, len(go), total
