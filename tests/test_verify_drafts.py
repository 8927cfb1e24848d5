"""Verification of drafts against its definition in 64 bits (longdouble sums): ragged drafts, types, strides, ties,
rows without weight, values that are no numbers, bad tokens and rows; every output has to be equal."""
import numpy as np
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests import step_reference as ref
from tests.step_reference import i32

pytestmark = pytest.mark.gpu


def batch(drafts, V, dtype=torch.float32, seed=0, near=0.7, width=3.0):
    g = torch.Generator().manual_seed(seed)
    cu = np.concatenate([[0], np.cumsum([n + 1 for n in drafts])])
    T = int(cu[-1])
    z = width * torch.randn(T, V, generator=g)
    p = torch.softmax(z, -1)
    q = torch.softmax(z + near * torch.randn(T, V, generator=g), -1)
    x = torch.multinomial(q, 1, generator=g)[:, 0]
    tokens = torch.cat([x[:1], x[:-1]]).int()
    return dict(p=p.to(dtype), q=q.to(dtype), tokens=tokens, cu=i32(cu), au=torch.rand(T, generator=g),
                su=torch.rand(len(drafts), generator=g), cached=torch.randint(0, 5000, (len(drafts),), generator=g).int())


def run(w, given=True, flags=0, **kw):
    status = ops.new_status()
    g = {k: v.cuda() for k, v in w.items()}
    T, B = len(w["tokens"]), len(w["su"])
    out = ops.Verified(*[torch.full((n,), -7, dtype=torch.int32, device="cuda") for n in (B, T, B)])
    ops.verify_drafts(g["p"], g["q"] if given else None, g["tokens"], g["cu"], g["au"], g["su"], cached_lens=g["cached"],
                      out=out, status=status, **kw)
    want = ref.verify(w["p"], w["q"] if given else None, w["tokens"].tolist(), w["cu"].tolist(), w["au"].tolist(),
                      w["su"].tolist(), w["cached"].tolist(), [-7] * T)
    for name, a, b in zip(out._fields, out, want):
        assert a.tolist() == b.tolist(), name
    assert ops.read_status(status) == flags
    return out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 127, 1000, 4097, 50001])
def test_vocabularies(V, given, dtype):
    run(batch([3, 0, 1, 7, 2], V, dtype, seed=V), given)


@pytest.mark.parametrize("drafts", [[0], [1], [5] * 40, [0] * 9, [40, 0, 70], [i % 6 for i in range(150)]])
def test_batches(drafts):
    # nearly the same distributions: long runs of accepted drafts
    run(batch(drafts, 777, seed=len(drafts), near=0.05))


@pytest.mark.parametrize("V", [131072, 151936])
@pytest.mark.parametrize("given", [True, False])
def test_large_vocabularies(V, given):
    run(batch([4, 2, 0, 3], V, seed=V), given)


def test_many_draws_of_a_flat_row():
    """Every boundary between neighbours is 1e-5 wide: 32-bit sums would miss some."""
    w = batch([0] * 300, 100003, seed=2, width=0.1)
    run(w)


@pytest.mark.parametrize("dtype,requests,V", [(torch.float32, 5, 49148), (torch.bfloat16, 5, 65528),
                                              (torch.float32, 170, 6140), (torch.bfloat16, 170, 8184)])
def test_around_the_longest_rows_that_stay_in_registers(dtype, requests, V):
    for n in (V - 5, V, V + 1, V + 13):
        w = batch([i % 3 for i in range(requests)], n, dtype, seed=n)
        w["su"][:4] = torch.tensor([0.0, 0.9999999, 1.0, 0.5])
        run(w)
        g, T = {k: v.cuda() for k, v in w.items()}, len(w["tokens"])
        want = ref.verify(w["p"], w["q"], w["tokens"].tolist(), w["cu"].tolist(), w["au"].tolist(), w["su"].tolist(), None,
                          [-1] * T)
        for shift_p, shift_q in ((1, 3), (3, 3), (0, 7)):      # rows whose first vector is not whole
            p, q = (torch.zeros(T * (n + 8) + 8, dtype=dtype, device="cuda")[s:s + T * (n + 8)].view(T, n + 8)[:, :n]
                    for s in (shift_p, shift_q))
            p.copy_(g["p"]), q.copy_(g["q"])
            for a, b in zip(ops.verify_drafts(p, q, g["tokens"], g["cu"], g["au"], g["su"]), want):
                assert a.tolist() == b.tolist(), (n, shift_p, shift_q)


def test_strided_rows_and_odd_addresses():
    w = batch([2, 3, 0], 999, seed=4)
    g = {k: v.cuda() for k, v in w.items()}
    T = len(w["tokens"])
    for dtype in (torch.float32, torch.bfloat16):
        for shift_p, shift_q, pitch in ((1, 1, 1005), (1, 2, 1001), (0, 3, 1000), (3, 0, 999)):
            p, q = (torch.zeros(T * pitch + 8, dtype=dtype, device="cuda")[s:s + T * pitch].view(T, pitch)[:, :999]
                    for s in (shift_p, shift_q))
            p.copy_(g["p"]), q.copy_(g["q"])
            got = ops.verify_drafts(p, q, g["tokens"], g["cu"], g["au"], g["su"])
            want = ref.verify(p.cpu(), q.cpu(), w["tokens"].tolist(), w["cu"].tolist(), w["au"].tolist(), w["su"].tolist(),
                              None, [-1] * T)
            for a, b in zip(got, want):
                assert a.tolist() == b.tolist(), (dtype, shift_p, shift_q, pitch)


def test_edges_of_the_draw():
    V = 8192
    w = batch([0] * 7, V, seed=5)
    w["p"][:] = 0
    w["p"][:, [3, 4000, 8000]] = 0.25              # thirds of 0.75
    w["su"] = torch.tensor([0.0, 0.25, 0.5, 0.75, 0.9999999, 1.0, float("nan")])
    out = run(w)
    # at 0 the first token with weight, never one without; 1 and what is no number the last one
    assert out.tokens.tolist() == [3, 3, 4000, 8000, 8000, 8000, 8000]
    w["p"][:, [3, 4000, 8000]] = torch.tensor([0.25, 0.25, 0.5])
    w["su"] = torch.tensor([0.25, 0.5, 0.2499999, 0.4999999, 0.75, 0.0, 0.999])
    assert run(w).tokens.tolist() == [4000, 8000, 3, 4000, 8000, 3, 8000]   # a border belongs to the token behind it


def test_accepting_at_the_border():
    """u q = p exactly does not stand, the next number below does; q = 0 stands where p > 0."""
    w = batch([1, 1, 1, 1], 64, seed=6)
    w["p"][:], w["q"][:] = 1 / 64, 1 / 32
    w["tokens"][:] = 9
    w["au"][:] = 0.5
    w["au"][2] = float(np.nextafter(np.float32(0.5), np.float32(0)))
    w["q"][4, 9] = 0
    w["p"][6, 9] = w["q"][6, 9] = 0
    assert run(w).accepted.tolist() == [0, 1, 1, 0]


def test_nothing_left_over_and_no_weight():
    w = batch([1, 1, 0, 1], 300, seed=7)
    w["q"][0] = w["p"][0]                          # p nowhere above q: the target's own row
    w["au"][:] = 0.9999
    w["p"][0, w["tokens"][1]] = 0
    w["q"][0, :] = torch.maximum(w["q"][0], w["p"][0])
    w["p"][4] = 0                                  # an empty row
    w["p"][5] = 0
    w["q"][5] = 1
    out = run(w, flags=ops.DEVERR_PROBS)
    assert out.tokens[0] >= 0 and out.tokens[4] == -1 and out.tokens[5] == -1


@pytest.mark.parametrize("given", [True, False])
def test_values_that_are_no_numbers(given):
    w = batch([1, 1, 0, 0, 1], 500, seed=8)
    w["p"][0, ::3] = float("nan")
    w["q"][2, ::5] = float("nan")
    w["p"][4, 17] = float("-inf")
    w["p"][5, 20] = float("inf")
    w["p"][6, w["tokens"][7]] = float("nan")
    out = run(w, given, flags=ops.DEVERR_PROBS)
    assert out.tokens[5] == -1 and out.accepted[4] == 0


@pytest.mark.parametrize("requests", [1, 40, 160])              # clusters of 8, 4 and 1 blocks
@pytest.mark.parametrize("dtype,V", [(torch.float32, 70001), (torch.bfloat16, 70001)])
def test_the_edges_in_long_rows(dtype, V, requests):
    """Rows too long for registers: borders between tokens, nothing left over, no weight, values that are no numbers."""
    n = max(requests, 12)
    w = batch([1] * 6 + [0] * (n - 6), 64, dtype, seed=n)
    p, q = torch.zeros(len(w["tokens"]), V, dtype=dtype), torch.zeros(len(w["tokens"]), V, dtype=dtype)
    w["p"], w["q"] = p, q
    p[:, [5, 35000, 70000]] = torch.tensor([0.25, 0.25, 0.5], dtype=dtype)
    w["au"][:] = 0.9999
    w["tokens"][1:12:2] = 7                        # the first six requests' draft: p 0 and q 1
    q[0:12:2, 7] = 1
    q[2] = p[2]                                    # p nowhere above q: the target's own row
    p[4, :], q[4, 5] = 0, 1                        # an empty row, left over or not
    p[6, 40000] = float("inf")
    p[8, 60000], q[8, 35000] = float("nan"), float("nan")
    q[10, [5, 70000]] = 1                          # one token left over
    w["su"][:12] = torch.tensor([0.0, 0.25, 0.9, 0.3, 0.1, 0.99, 0.0, 0.25, 0.4999999, 0.5, 1.0, float("nan")])
    out = run(w, flags=ops.DEVERR_PROBS)
    assert out.tokens[0:12:2].tolist() == [5, 35000, -1, -1, 5, 35000]
    assert out.tokens[12:18].tolist() == [5, 35000, 35000, 70000, 70000, 70000]


def test_bad_tokens():
    w = batch([3, 2], 400, seed=9, near=0.0)
    w["au"][:] = 0
    w["tokens"][2], w["tokens"][5] = 400, -1
    for given in (True, False):
        out = run(w, given, flags=ops.DEVERR_TOKEN)
        assert out.accepted.tolist() == [1, 0]


def test_rows_outside_the_requests_stay():
    w = batch([2, 1, 3], 100, seed=10)
    w["cu"] = i32([1, 3, 3, 7])                    # the second has no rows; rows 0 and 7.. belong to none
    w["su"], w["cached"] = w["su"][:3], w["cached"][:3]
    out = run(w)
    assert out.tokens[0] == -7 and out.tokens[7:].eq(-7).all() and out.accepted[1] == 0


def test_bad_row_offsets():
    w = batch([2, 1, 3, 1], 100, seed=11)
    T = len(w["tokens"])
    w["cu"] = i32([0, 3, 2, T + 1, T])             # backwards, past the end, backwards again
    run(w, flags=ops.DEVERR_LENGTH)
    w["cu"] = i32([-1, 3, 5, 9, 11])
    run(w, flags=ops.DEVERR_LENGTH)


def test_outputs_of_its_own_and_lengths_in_place():
    w = batch([2, 0, 4], 5000, seed=12)
    g = {k: v.cuda() for k, v in w.items()}
    got = ops.verify_drafts(g["p"], g["q"], g["tokens"], g["cu"], g["au"], g["su"])
    want = ref.verify(w["p"], w["q"], w["tokens"].tolist(), w["cu"].tolist(), w["au"].tolist(), w["su"].tolist(), None,
                      [-1] * len(w["tokens"]))
    for a, b in zip(got, want):
        assert a.tolist() == b.tolist()
    lens = g["cached"].clone()
    out = ops.verify_drafts(g["p"], g["q"], g["tokens"], g["cu"], g["au"], g["su"], cached_lens=lens,
                            out=ops.Verified(got.accepted, got.tokens, lens))
    assert lens.tolist() == (w["cached"] + out.accepted.cpu() + 1).tolist()


def test_empty_batches():
    z = torch.zeros(0, 10, device="cuda")
    f, n = torch.zeros(0, device="cuda"), i32([], "cuda")
    out = ops.verify_drafts(z, None, n, i32([0], "cuda"), f, f)
    assert out.accepted.numel() == 0
    out = ops.verify_drafts(z, None, n, i32([0, 0, 0], "cuda"), f, torch.zeros(2, device="cuda"), cached_lens=i32([3, 4], "cuda"))
    assert out.kv_lens.tolist() == [3, 4] and out.accepted.tolist() == [0, 0]


def test_rows_whose_offsets_pass_32_bits():
    V, T = 1 << 20, 2100
    p = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
    p[:, V - 5] = 1
    p[T - 1, 7] = 3
    cu = i32([0, 1, T - 1, T], "cuda")
    tok = torch.full((T,), V - 5, dtype=torch.int32, device="cuda")
    out = ops.verify_drafts(p, None, tok, cu, torch.full((T,), 0.5, device="cuda"), torch.tensor([0.5, 0.5, 0.7], device="cuda"))
    assert out.accepted.tolist() == [0, T - 3, 0]
    assert out.tokens[:T - 1].eq(V - 5).all() and out.tokens[T - 1] == 7


def test_graph_and_stream():
    w = batch([3, 1, 0, 2], 32000, seed=13)
    g = {k: v.cuda() for k, v in w.items()}
    T = len(w["tokens"])
    out = ops.Verified(*[torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, T, 4)])
    call = lambda **kw: ops.verify_drafts(g["p"], g["q"], g["tokens"], g["cu"], g["au"], g["su"], g["cached"], out, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call(stream=side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (14, 15):
        w = batch([3, 1, 0, 2], 32000, seed=seed)
        for k, v in w.items():
            g[k].copy_(v)
        graph.replay()
        want = ref.verify(w["p"], w["q"], w["tokens"].tolist(), w["cu"].tolist(), w["au"].tolist(), w["su"].tolist(),
                          w["cached"].tolist(), [0] * T)
        for a, b in zip(out, want):
            assert a.tolist() == b.tolist()


def test_distribution():
    """200000 draws with one draft each: accepted or replaced, tokens follow the target."""
    B, V = 200000, 5
    p = torch.tensor([0.4, 0.1, 0.25, 0.05, 0.2])
    q = torch.tensor([0.1, 0.3, 0.2, 0.2, 0.2])
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.multinomial(q.cuda().expand(1, V), B, replacement=True, generator=g)[0].int()
    tokens = torch.stack([torch.zeros_like(x), x], 1).flatten()
    out = ops.verify_drafts(p.cuda().expand(2 * B, V).contiguous(), q.cuda().expand(2 * B, V).contiguous(), tokens,
                            torch.arange(0, 2 * B + 1, 2, dtype=torch.int32, device="cuda"),
                            torch.rand(2 * B, device="cuda", generator=g), torch.rand(B, device="cuda", generator=g))
    share = torch.bincount(out.tokens[::2], minlength=V).double().cpu() / B
    # six standard deviations of a share
    assert ((share - p.double()).abs() < 6 * torch.sqrt(p.double() * (1 - p.double()) / B)).all(), share
    assert abs(out.accepted.double().mean().item() - torch.minimum(p, q).sum().item()) < 6 * 0.5 / B ** 0.5


def test_refusals():
    w = {k: v.cuda() for k, v in batch([2, 1], 40, seed=16).items()}
    call = lambda **kw: ops.verify_drafts(**{**dict(target_probs=w["p"], draft_probs=w["q"], tokens=w["tokens"],
                                                    cu_ext=w["cu"], accept_u=w["au"], sample_u=w["su"]), **kw})
    for kw in (dict(draft_probs=w["q"].bfloat16()), dict(draft_probs=w["q"][:, :39]), dict(target_probs=w["p"].double()),
               dict(target_probs=w["p"][:3]), dict(target_probs=w["p"].t().contiguous().t()), dict(cu_ext=w["cu"][:2]),
               dict(accept_u=w["au"][:3]), dict(sample_u=w["su"].double()), dict(tokens=w["tokens"].long()),
               dict(cached_lens=w["cached"][:1]), dict(target_probs=w["p"].cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    both = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    with pytest.raises(ops.MsglError, match="overlaps"):
        call(out=ops.Verified(both[0], w["tokens"], both[1]))
    with pytest.raises(ops.MsglError, match="overlaps"):
        call(out=ops.Verified(both[0], torch.zeros_like(w["tokens"]), both[0]))
    with pytest.raises(ops.MsglError):
        call(target_probs=torch.zeros(5, 0, device="cuda"), draft_probs=None)
