"""The rotary store against the rotation in 64 bits: pairings, axes, norms, far positions, strided and in-place
heads, padding, bad slots, streams, graphs."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import assert_rounded, i32, rope_rows

pytestmark = pytest.mark.gpu

D = 128


def freqs(pairs, base=1e6):
    return [base ** (-j / pairs) for j in range(pairs)]


def case(T, hq, hkv, axes=1, fused=False, ps=1, seed=0, slots=None):
    g = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    if fused:
        qkv = normal(T, hq + 2 * hkv, D).cuda()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        q, k, v = normal(T, hq, D).cuda(), normal(T, hkv, D).cuda(), normal(T, hkv, D).cuda()
    slots = slots or (T + 5 + ps - 1) // ps * ps
    loc = torch.randperm(slots, generator=g)[:T].int().cuda()
    pos = torch.randint(0, 5000, (axes, T), generator=g, dtype=torch.int32).cuda()
    pool = ops.KVPool(*[torch.full((slots, hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)], ps)
    return q, k, v, pos, loc, pool


def check(q, k, v, pos, loc, pool, out, inv_freq, axes=None, adjacent=False, factor=1.0, q_norm=None, k_norm=None,
          eps=1e-6):
    axes = axes or [0] * len(inv_freq)
    pos = pos.cpu().reshape(-1, q.shape[0]).tolist()
    args = (pos, inv_freq, axes, adjacent, factor)
    cpu = lambda t: None if t is None else t.cpu()
    assert_rounded(out, *rope_rows(q.cpu(), *args, cpu(q_norm), eps))
    want, slack = rope_rows(k.cpu(), *args, cpu(k_norm), eps)
    at = loc.cpu().long()
    here = (at >= 0) & (at < pool.k.shape[0])
    assert_rounded(pool.k.cpu()[at[here]], want[here], slack[here])
    assert torch.equal(pool.v.cpu()[at[here]].view(torch.int16), v.cpu()[here].view(torch.int16))
    rest = torch.ones(pool.k.shape[0], dtype=torch.bool)
    rest[at[here]] = False
    assert pool.k.cpu()[rest].isnan().all() and pool.v.cpu()[rest].isnan().all()


@pytest.mark.parametrize("T", [1, 2, 7, 131])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 8), (28, 4), (40, 8), (64, 8), (64, 1)])
def test_sizes(T, hq, hkv):
    q, k, v, pos, loc, pool = case(T, hq, hkv, seed=T)
    status = ops.new_status()
    f = freqs(64)
    out = ops.rope_store_kv(pool, q, k, v, pos[0], loc, ops.Rope(f), status=status)
    check(q, k, v, pos, loc, pool, out, f)
    assert ops.read_status(status) == 0


@pytest.mark.parametrize("pairs", [8, 16, 24, 32, 40, 48, 56, 64])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_pairings(pairs, adjacent, norm):
    q, k, v, pos, loc, pool = case(9, 12, 4, axes=3, seed=pairs)
    axes = [(j * 7) % 3 for j in range(pairs)]
    f = freqs(pairs, 1e4)
    w = [(1 + 0.3 * torch.randn(D)).to(torch.bfloat16).cuda() for _ in range(2)] if norm else [None, None]
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(f, axes, adjacent, 1.25), q_norm=w[0], k_norm=w[1], eps=1e-5)
    check(q, k, v, pos, loc, pool, out, f, axes, adjacent, 1.25, *w, eps=1e-5)


@pytest.mark.parametrize("which", ["q", "k"])
def test_one_norm_alone(which):
    q, k, v, pos, loc, pool = case(5, 8, 8, seed=3)
    w = {which + "_norm": torch.full((D,), 0.5, dtype=torch.bfloat16, device="cuda")}
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)), **w)
    check(q, k, v, pos, loc, pool, out, freqs(64), **w)


def test_zero_head_norms_to_zero():
    q, k, v, pos, loc, pool = case(3, 8, 8, seed=4)
    q[:, 2] = 0
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)), q_norm=w, k_norm=w)
    assert torch.all(out[:, 2] == 0)
    check(q, k, v, pos, loc, pool, out, freqs(64), q_norm=w, k_norm=w)


def test_far_and_negative_positions():
    q, k, v, _, loc, pool = case(8, 16, 8, axes=4, seed=5)
    far = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 2 ** 24 + 1, 2 ** 30]
    pos = i32([[far[(t + a) % 8] for t in range(8)] for a in range(4)], "cuda")
    axes = [j % 4 for j in range(64)]
    f = freqs(64)
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(f, axes))
    check(q, k, v, pos, loc, pool, out, f, axes)


@pytest.mark.parametrize("in_place", [False, True])
def test_columns_of_one_projection(in_place):
    q, k, v, pos, loc, pool = case(37, 16, 4, fused=True, seed=6)
    before = q.clone()
    wide = torch.full((37, 20, D), 7.0, dtype=torch.bfloat16, device="cuda")
    target = q if in_place else wide[:, 2:18]
    out = ops.rope_store_kv(pool, q, k, v, pos[0], loc, ops.Rope(freqs(64)), q_out=target)
    assert out.data_ptr() == target.data_ptr()
    check(before, k, v, pos, loc, pool, out, freqs(64))
    if not in_place:
        assert torch.all(wide[:, :2] == 7) and torch.all(wide[:, 18:] == 7)


@pytest.mark.parametrize("T", [1, 2, 300])
def test_output_between_the_inputs_columns(T):
    q, k, v, pos, loc, pool = case(T, 16, 4, seed=T)
    row = torch.cat([q, torch.zeros_like(q), k, v], 1)
    out = ops.rope_store_kv(pool, row[:, :16], row[:, 32:36], row[:, 36:], pos[0], loc, ops.Rope(freqs(64)), q_out=row[:, 16:32])
    check(q, k, v, pos, loc, pool, out, freqs(64))
    assert torch.equal(row[:, :16], q) and torch.equal(row[:, 32:36], k) and torch.equal(row[:, 36:], v)


def test_positions_out_of_a_larger_buffer():
    q, k, v, _, loc, pool = case(6, 8, 8, seed=7)
    buf = torch.randint(0, 900, (3, 50), dtype=torch.int32, device="cuda")
    axes = [0] * 16 + [1] * 24 + [2] * 24
    out = ops.rope_store_kv(pool, q, k, v, buf[:, :6], loc, ops.Rope(freqs(64), axes))
    check(q, k, v, buf[:, :6], loc, pool, out, freqs(64), axes)


def test_one_row_of_positions_for_all_axes():
    q, k, v, pos, loc, pool = case(5, 8, 4, seed=17)
    axes = [j % 3 for j in range(64)]
    out = ops.rope_store_kv(pool, q, k, v, pos.expand(3, 5), loc, ops.Rope(freqs(64), axes))
    check(q, k, v, pos.expand(3, 5).contiguous(), loc, pool, out, freqs(64), axes)


def test_most_heads():
    q, k, v, pos, loc, pool = case(2, 64 * 64, 64, seed=18)
    out = ops.rope_store_kv(pool, q, k, v, pos[0], loc, ops.Rope(freqs(64)))
    check(q, k, v, pos, loc, pool, out, freqs(64))


def test_padding_and_bad_slots():
    q, k, v, pos, loc, pool = case(8, 8, 8, seed=8)
    loc[3] = -1
    loc[7] = -1
    out = torch.full_like(q, 3.0)
    status = ops.new_status()
    ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)), q_out=out, status=status)
    live = torch.tensor([i for i in range(8) if i not in (3, 7)], device="cuda")
    check(q[live], k[live], v[live], pos[:, live], loc[live], pool, out[live], freqs(64))
    assert torch.all(out[[3, 7]] == 3) and ops.read_status(status) == 0
    loc[1], loc[2] = pool.k.shape[0], -2          # turned, not stored
    pool.k.fill_(float("nan")), pool.v.fill_(float("nan"))
    ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)), q_out=out, status=status)
    assert ops.read_status(status) == ops.DEVERR_SLOT_RANGE
    check(q[live], k[live], v[live], pos[:, live], loc[live], pool, out[live], freqs(64))


def test_values_that_are_no_numbers_stay_in_their_pair():
    q, k, v, pos, loc, pool = case(2, 8, 8, seed=9)
    q[0, 0, 5], k[1, 3, 70] = float("inf"), float("nan")
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)))
    fine = torch.isfinite(out)
    fine[0, 0, [5, 69]] = True
    assert fine.all()
    kept = torch.isfinite(pool.k[loc.long()])
    kept[1, 3, [6, 70]] = True
    assert kept.all()


def test_no_tokens():
    q, k, v, pos, loc, pool = case(0, 8, 8)
    assert ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64))).shape == (0, 8, D)


def test_slots_whose_offsets_pass_32_bits():
    hkv, slots = 64, (2 ** 31) // (64 * D) + 70          # elements of a pool past 2^31
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(3, hkv, D, generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    pool = ops.KVPool(*[torch.zeros(slots, hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)], 1)
    loc, pos = i32([slots - 1, 5, slots - 66], "cuda"), i32([3, 4, 5], "cuda")
    out = ops.rope_store_kv(pool, q, k, v, pos, loc, ops.Rope(freqs(64)))
    want, slack = rope_rows(k.cpu(), [pos.tolist()], freqs(64), [0] * 64, False, 1.0, None, 0)
    assert_rounded(pool.k[loc.long()], want, slack)
    assert torch.equal(pool.v[loc.long()], v)
    assert pool.k.count_nonzero() <= 3 * hkv * D
    del out


def test_own_stream_and_graph():
    q, k, v, pos, loc, pool = case(33, 16, 8, axes=2, seed=11)
    axes = [j % 2 for j in range(64)]
    rope, out, f = ops.Rope(freqs(64), axes), torch.empty_like(q), freqs(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ops.rope_store_kv(pool, q, k, v, pos, loc, rope, q_out=out, stream=side)
    side.synchronize()
    check(q, k, v, pos, loc, pool, out, f, axes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.rope_store_kv(pool, q, k, v, pos, loc, rope, q_out=out)
    for i in range(2):
        q.normal_(), k.normal_(), v.normal_(), pos.random_(0, 10 ** 6)
        pool.k.fill_(float("nan")), pool.v.fill_(float("nan"))
        graph.replay()
        check(q, k, v, pos, loc, pool, out, f, axes)


def test_refusals():
    q, k, v, pos, loc, pool = case(4, 8, 8)
    rope = ops.Rope(freqs(64))
    call = lambda **kw: ops.rope_store_kv(**{**dict(pool=pool, q=q, k=k, v=v, positions=pos, out_loc=loc, rope=rope), **kw})
    for kw in (dict(k=k[:3]), dict(out_loc=loc[:3]), dict(positions=pos[:, :3]), dict(positions=pos.long()),
               dict(q=q.float()), dict(k=k[:, :4]), dict(q=q[:, :, ::2]), dict(q=q.transpose(0, 1)), dict(q_out=q[:3]),
               dict(q_norm=k[0]), dict(v=v.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    odd = torch.zeros(4 * 8 * D + 4, dtype=torch.bfloat16, device="cuda")[4:].view(4, 8, D)
    shifted = torch.zeros(4 * 8 * D + 8 * D, dtype=torch.bfloat16, device="cuda")
    for kw in (dict(q=odd), dict(rope=ops.Rope(freqs(64), [1] * 64)), dict(q=q[:, :7]), dict(q_out=k), dict(q_out=pool.k[:4]),
               dict(q=shifted[:-8 * D].view(4, 8, D), q_out=shifted[8 * D:].view(4, 8, D)), dict(q_norm=k[0, 0], eps=-1.0),
               dict(q=q[:1].expand(4, 8, D))):
        with pytest.raises(ops.MsglError):
            call(**kw)
