"""The rotary store over so many tokens that a warp takes several turns of heads: heads ahead of their use, q's rotation
and then k's, rotation in place, padding in between; every token against the rotation in 64 bits."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import assert_rounded, rope_rows

pytestmark = pytest.mark.gpu

D = 128


# On 152 SMs 3040 warps run at once, 4 heads a turn.  400 tokens: 7 warps a token (3 turns each of 64/8 heads), 1100: 2
# (10 turns), from 1521 on a warp takes a token (20 turns of 64/8, 9 of 28/4, 5 of 16/1).
@pytest.mark.parametrize("T", [400, 1100, 3000, 9000])
@pytest.mark.parametrize("hq,hkv,norms,adjacent", [(64, 8, "qk", False), (28, 4, "qk", True), (16, 1, "", False),
                                                   (16, 1, "k", True)])
def test_many_turns(T, hq, hkv, norms, adjacent):
    g = torch.Generator().manual_seed(T + hq)
    qkv = torch.randn(T, hq + 2 * hkv, D, generator=g).to(torch.bfloat16)
    slots = T + 37
    loc = torch.randperm(slots, generator=g)[:T].int()
    pos = torch.randint(0, 40000, (3, T), generator=g, dtype=torch.int32)
    pads = torch.rand(T, generator=g) < 0.05
    pads[-3:] = True
    # padding is read at most: whatever stands there goes nowhere
    loc[pads], qkv[pads], pos[:, pads] = -1, float("nan"), -2 ** 31
    live = ~pads
    weight = {name + "_norm": (scale + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16) for name, scale in (("q", 1.0), ("k", -2.0))
              if name in norms}
    cuda_weight = {k: w.cuda() for k, w in weight.items()}
    f, axes = [1e6 ** (-j / 64) for j in range(64)], [0] * 16 + [1] * 24 + [2] * 24
    turn = [pos[:, live].tolist(), f, axes, adjacent, 1.0]
    q, k, v = qkv[live, :hq], qkv[live, hq:hq + hkv], qkv[live, hq + hkv:]
    want_q, want_k = (rope_rows(x, *turn, weight.get(n + "_norm"), 1e-6) for n, x in (("q", q), ("k", k)))
    rope, status = ops.Rope(f, axes, adjacent), ops.new_status()
    got = []
    for in_place in (False, True):
        rows = qkv.cuda()
        pool = ops.KVPool(*[torch.full((slots, hkv, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)], 1)
        out = rows[:, :hq] if in_place else torch.full((T, hq, D), 3.0, dtype=torch.bfloat16, device="cuda")
        ops.rope_store_kv(pool, rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], pos.cuda(), loc.cuda(), rope, q_out=out,
                          status=status, **cuda_weight)
        out, rows = out.cpu(), rows.cpu()
        assert_rounded(out[live], *want_q)
        assert_rounded(pool.k.cpu()[loc[live].long()], *want_k)
        assert torch.equal(pool.v.cpu()[loc[live].long()], v)
        assert out[pads].isnan().all() if in_place else (out[pads] == 3).all()
        rest = torch.ones(slots, dtype=torch.bool)
        rest[loc[live].long()] = False
        assert (pool.k.cpu()[rest] == 9).all() and (pool.v.cpu()[rest] == 9).all()
        assert torch.equal(rows[live, hq:], qkv[live, hq:]) and (in_place or torch.equal(rows[live, :hq], q))
        got.append((out[live], pool.k.cpu(), pool.v.cpu()))
    assert ops.read_status(status) == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T", [1, 5])
def test_what_padding_holds_does_not_matter(T, norm):
    """A batch of padding alone: rows of infinities, the farthest positions, nothing written and nothing reported."""
    q, kv = (torch.full((T, h, D), float("inf"), dtype=torch.bfloat16, device="cuda") for h in (16, 8))
    pool = ops.KVPool(*[torch.full((T, 8, D), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)], 1)
    out, status = torch.full_like(q, 3.0), ops.new_status()
    pos = torch.full((4, T), -2 ** 31, dtype=torch.int32, device="cuda")
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda") if norm else None
    ops.rope_store_kv(pool, q, kv, kv, pos, torch.full((T,), -1, dtype=torch.int32, device="cuda"),
                      ops.Rope([1e6 ** (-j / 64) for j in range(64)], [j % 4 for j in range(64)]), q_out=out, q_norm=w, k_norm=w,
                      status=status)
    assert (out == 3).all() and (pool.k == 9).all() and (pool.v == 9).all() and ops.read_status(status) == 0
