"""Host-side behaviour of the rotary store, the draft verification and the page calls (no GPU).

Every call below fails a host check, or is a size query or a metadata check on host copies,
before anything is launched.
"""
import ctypes
import os
import subprocess

import pytest
import torch

from paged_kv_attention_24_gb300 import ops

INVALID, UNSUPPORTED, OUT_OF_RANGE, WORKSPACE = 1, 2, 4, 6
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_24_gb300 import build
    build.build()
    return ops.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def at(k):
    """A device address that nothing else of a call overlaps."""
    return (k + 1) << 24


def test_struct_layouts_match_the_header(tmp_path):
    structs = {"msgl_rope": ops._Rope, "msgl_new_tokens": ops._NewTokens, "msgl_draft_batch": ops._DraftBatch,
               "msgl_fork_out": ops._ForkOut, "msgl_compact_out": ops._CompactOut}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "msgl_attn.h"', "int main(void) {"]
    want = []
    for name, cls in structs.items():
        lines.append(f'printf("%zu\\n", sizeof({name}));')
        want.append(ctypes.sizeof(cls))
        for f, _ in cls._fields_:
            lines.append(f'printf("%zu\\n", offsetof({name}, {f}));')
            want.append(getattr(cls, f).offset)
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["return 0;", "}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    assert [int(x) for x in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()] == want


def test_device_error_bits_match_the_header():
    text = open(os.path.join(ROOT, "include", "msgl_attn.h")).read()
    for name in ("ROW", "TOKEN", "PROBS"):
        assert f"#define MSGL_DEVERR_{name} {getattr(ops, 'DEVERR_' + name):#x}u" in text


def test_rope_store_refusals(lib):
    axes = (ctypes.c_uint8 * 64)(*[0] * 64)

    def call(pool=(at(0), at(1), 256, 16, 8, 128), hq=16, turns=at(2), ax=axes, pairs=64, num_axes=1, factor=1.0,
             q_norm=None, k_norm=None, eps=1e-6, tokens=True, rope=True, **over):
        p = ops._Pool(*pool)
        n = ops._NewTokens(at(3), at(4), at(5), at(6), 16 * 128, 8 * 128, 8 * 128, 16 * 128, at(7), 4, at(8), 4, hq)
        for k, v in over.items():
            setattr(n, k, v)
        r = ops._Rope(turns, None if ax is None else ctypes.cast(ax, ctypes.c_void_p), pairs, num_axes, 0, factor)
        return lib.msgl_rope_store_kv(ctypes.byref(p), ctypes.byref(n) if tokens else None, ctypes.byref(r) if rope else None,
                                      q_norm, k_norm, eps, None, None)

    second = (ctypes.c_uint8 * 64)(*[0] * 63, 1)
    for want, kw in [(INVALID, dict(tokens=False)), (INVALID, dict(rope=False)), (INVALID, dict(turns=None)),
                     (INVALID, dict(turns=at(2) + 4)), (INVALID, dict(pairs=0)), (INVALID, dict(pairs=72)),
                     (UNSUPPORTED, dict(pairs=12)), (INVALID, dict(num_axes=0)), (INVALID, dict(num_axes=5)),
                     (INVALID, dict(ax=second)), (INVALID, dict(factor=float("inf"))), (INVALID, dict(factor=float("nan"))),
                     (INVALID, dict(q_norm=at(9), eps=-1.0)), (INVALID, dict(k_norm=at(9), eps=float("nan"))),
                     (INVALID, dict(q_norm=at(9) + 8)), (INVALID, dict(n_tokens=-1)), (INVALID, dict(hq=12)),
                     (UNSUPPORTED, dict(hq=8 * 65)), (UNSUPPORTED, dict(pool=(at(0), at(1), 256, 16, 8, 64))),
                     (INVALID, dict(pool=(None, at(1), 256, 16, 8, 128))), (INVALID, dict(q=None)), (INVALID, dict(v=None)),
                     (INVALID, dict(q_out=None)), (INVALID, dict(positions=None)), (INVALID, dict(out_loc=None)),
                     (INVALID, dict(q=at(3) + 8)), (INVALID, dict(k=at(4) + 2)), (INVALID, dict(q_out=at(6) + 4)),
                     (INVALID, dict(q_stride=16 * 128 - 8)), (INVALID, dict(k_stride=8 * 128 + 4)), (INVALID, dict(v_stride=0)),
                     (INVALID, dict(out_stride=2 ** 62)), (INVALID, dict(q_stride=-8)),
                     (INVALID, dict(ax=second, num_axes=2, axis_stride=3)), (INVALID, dict(ax=second, num_axes=2, axis_stride=2 ** 60)),
                     (INVALID, dict(ax=second, num_axes=2, axis_stride=-4)),
                     # q_out over an input, and over part of q
                     (INVALID, dict(q_out=at(4))), (INVALID, dict(q_out=at(5) + 3 * 2048)), (INVALID, dict(q_out=at(3) + 16)),
                     (INVALID, dict(q_out=at(3), out_stride=16 * 128 + 8)), (INVALID, dict(q_out=at(0) + 2048)),
                     (INVALID, dict(q_out=at(7) - 4096)), (INVALID, dict(q_out=at(2)))]:
        assert call(**kw) == want, (kw, lib.msgl_last_error())
        assert lib.msgl_last_error(), kw
    assert call(n_tokens=0, q=None, k=None, v=None, q_out=None, positions=None, out_loc=None) == 0


@pytest.mark.parametrize("tokens", [1, 2, 500])
def test_rope_store_refuses_columns_that_meet(lib, tokens):
    """k and q_out columns of rows of 48 heads, a token's q_out sharing 16 bytes or more with the k of a token."""
    row, k = 48 * 256, at(3) + 17 * 256
    p, r = ops._Pool(at(0), at(1), 256, 16, 8, 128), ops._Rope(at(2), None, 64, 1, 0, 1.0)
    for apart in {0, 1 - tokens, tokens - 1, tokens // 2, -(tokens // 2)}:
        for shift in (16 - 16 * 256, -16, 0, 8 * 256 - 16):
            n = ops._NewTokens(at(6), k, at(5), k + apart * row + shift, 16 * 128, row // 2, 8 * 128, row // 2, at(7), tokens,
                               at(8), tokens, 16)
            assert lib.msgl_rope_store_kv(ctypes.byref(p), ctypes.byref(n), ctypes.byref(r), None, None, 0.0, None, None) == INVALID
            assert b"q_out overlaps k" in lib.msgl_last_error(), (apart, shift)


def test_verify_drafts_refusals(lib):
    def call(batch=True, **over):
        d = ops._DraftBatch(at(0), at(1), 1000, 1000, 1000, 0, at(2), at(3), at(4), at(5), at(6), 3, 9, at(7), at(8), at(9))
        for k, v in over.items():
            setattr(d, k, v)
        return lib.msgl_verify_drafts(ctypes.byref(d) if batch else None, None, None)

    for want, kw in [(INVALID, dict(batch=False)), (INVALID, dict(num_reqs=-1)), (INVALID, dict(total_tokens=-1)),
                     (INVALID, dict(vocab=0)), (UNSUPPORTED, dict(vocab=2 ** 30 + 1)), (UNSUPPORTED, dict(num_reqs=2 ** 25)),
                     (INVALID, dict(cu_ext=None)), (INVALID, dict(sample_u=None)), (INVALID, dict(accepted=None)),
                     (INVALID, dict(kv_lens=None)), (INVALID, dict(target=None)), (INVALID, dict(tokens=None)),
                     (INVALID, dict(accept_u=None)), (INVALID, dict(out_tokens=None)), (INVALID, dict(target_stride=999)),
                     (INVALID, dict(draft_stride=-1)), (INVALID, dict(target_stride=2 ** 60)), (INVALID, dict(target=at(0) + 2)),
                     (INVALID, dict(draft=at(1) + 1, is_bf16=1)),
                     (INVALID, dict(accepted=at(9))), (INVALID, dict(out_tokens=at(2) + 4)), (INVALID, dict(kv_lens=at(3) + 12)),
                     (INVALID, dict(out_tokens=at(0) + 8 * 4000)), (INVALID, dict(accepted=at(1) + 35996)),
                     (INVALID, dict(kv_lens=at(6) + 4)), (INVALID, dict(accepted=at(6)))]:
        assert call(**kw) == want, (kw, lib.msgl_last_error())
        assert lib.msgl_last_error(), kw
    assert call(num_reqs=0, cu_ext=None, sample_u=None, accepted=None, kv_lens=None) == 0


def test_fork_refusals(lib):
    def call(slots=256, ps=16, table=at(0), rows=4, stride=8, width=8, parents=at(1), children=at(2), lens=at(3), forks=2,
             free=at(4), num_free=3, out=True, **over):
        o = ops._ForkOut(at(5), at(6), at(7), at(8))
        for k, v in over.items():
            setattr(o, k, v)
        return lib.msgl_fork_requests(slots, ps, table, rows, stride, width, parents, children, lens, forks, free, num_free,
                                      ctypes.byref(o) if out else None, None, None)

    for want, kw in [(INVALID, dict(out=False)), (UNSUPPORTED, dict(ps=3)), (INVALID, dict(slots=250)), (INVALID, dict(slots=-16)),
                     (UNSUPPORTED, dict(slots=2 ** 31 * 16)), (INVALID, dict(rows=-1)), (INVALID, dict(forks=-1)),
                     (INVALID, dict(num_free=-1)), (INVALID, dict(stride=7)), (INVALID, dict(width=-1)), (INVALID, dict(table=None)),
                     (INVALID, dict(parents=None)), (INVALID, dict(children=None)), (INVALID, dict(lens=None)),
                     (INVALID, dict(free=None)), (INVALID, dict(copy_src=None)), (INVALID, dict(copy_dst=None)),
                     (INVALID, dict(copy_tokens=None)), (INVALID, dict(pages_taken=None)),
                     (UNSUPPORTED, dict(stride=2 ** 30, width=2 ** 30)), (UNSUPPORTED, dict(forks=2 ** 31 - 1)),
                     (INVALID, dict(copy_src=at(0) + 4)), (INVALID, dict(pages_taken=at(5) + 4)), (INVALID, dict(copy_dst=at(3))),
                     (INVALID, dict(table=at(4) - 4 * 31))]:
        assert call(**kw) == want, (kw, lib.msgl_last_error())
        assert lib.msgl_last_error(), kw


def test_copy_refusals(lib):
    def call(pools=((at(0), at(1), 256, 16, 8, 128), (at(2), at(3), 256, 16, 8, 128)), src=at(4), dst=at(5), pairs=2, n=None):
        c = (ops._Pool * max(1, len(pools)))(*[ops._Pool(*p) for p in pools])
        return lib.msgl_copy_pages(ctypes.cast(c, ctypes.POINTER(ops._Pool)), len(pools) if n is None else n, src, dst, None,
                                   pairs, None, None, None)

    one = (at(0), at(1), 256, 16, 8, 128)
    for want, kw in [(INVALID, dict(pairs=-1)), (INVALID, dict(n=-1)), (UNSUPPORTED, dict(n=2 ** 15 + 1)), (INVALID, dict(src=None)),
                     (INVALID, dict(dst=None)), (INVALID, dict(pools=(one, (at(2), at(3), 128, 16, 8, 128)))),
                     (INVALID, dict(pools=(one, (at(2), at(3), 256, 8, 8, 128)))),
                     (INVALID, dict(pools=(one, (at(2), at(3), 256, 16, 4, 128)))), (INVALID, dict(pools=(one, (at(2), None, 256, 16, 8, 128)))),
                     (UNSUPPORTED, dict(pools=((at(0), at(1), 256, 16, 8, 64),))), (UNSUPPORTED, dict(pools=((at(0), at(1), 252, 12, 8, 128),))),
                     (INVALID, dict(pools=((at(0) + 8, at(1), 256, 16, 8, 128),)))]:
        assert call(**kw) == want, (kw, lib.msgl_last_error())
        assert lib.msgl_last_error(), kw
    assert lib.msgl_copy_pages(None, 1, at(4), at(5), None, 2, None, None, None) == INVALID
    assert call(pools=()) == 0 and call(pairs=0, src=None, dst=None) == 0


def test_page_map_refusals(lib):
    size = lib.msgl_page_map_workspace_size(256, 16)
    assert size > 0 and size % 256 == 0
    assert lib.msgl_page_map_workspace_size(1 << 20, 1) >= 3 * (1 << 20) // 8
    assert lib.msgl_page_map_workspace_size(-1, 16) == 0 and lib.msgl_page_map_workspace_size(16, 0) == 0

    def args(slots=256, ps=16, table=at(0), rows=4, stride=8, width=8, req_rows=None, lens=at(1), reqs=2, held=None):
        return slots, ps, table, rows, stride, width, req_rows, lens, reqs, held

    def free(pages=at(2), count=at(3), ws=at(4), ws_bytes=size, **kw):
        return lib.msgl_free_pages(*args(**kw), pages, count, ws, ws_bytes, None, None)

    def compact(out=True, ws=at(4), ws_bytes=size, over={}, **kw):
        o = ops._CompactOut(at(5), 8, at(6), at(7), at(8), at(9), at(10))
        for k, v in over.items():
            setattr(o, k, v)
        return lib.msgl_compact_pages(*args(**kw), ctypes.byref(o) if out else None, ws, ws_bytes, None, None)

    shared = [(UNSUPPORTED, dict(ps=3)), (INVALID, dict(slots=250)), (UNSUPPORTED, dict(slots=2 ** 31 * 16)), (INVALID, dict(rows=-1)),
              (INVALID, dict(stride=7)), (INVALID, dict(width=-1)), (INVALID, dict(table=None)), (INVALID, dict(reqs=-1)),
              (INVALID, dict(lens=None)), (UNSUPPORTED, dict(reqs=2 ** 31 - 1)), (UNSUPPORTED, dict(width=2 ** 30, stride=2 ** 30)),
              (WORKSPACE, dict(ws=None)), (WORKSPACE, dict(ws_bytes=size - 1)), (INVALID, dict(ws=at(4) + 128))]
    for want, kw in shared:
        for f in (free, compact):
            assert f(**kw) == want, (f, kw, lib.msgl_last_error())
            assert lib.msgl_last_error(), kw
    for want, kw in [(INVALID, dict(pages=None)), (INVALID, dict(count=None)), (INVALID, dict(pages=at(0) + 16)),
                     (INVALID, dict(count=at(2) + 60)), (INVALID, dict(held=at(2) + 63)), (INVALID, dict(pages=at(1) + 4))]:
        assert free(**kw) == want, (kw, lib.msgl_last_error())
    for want, kw in [(INVALID, dict(out=False)), (INVALID, dict(over=dict(page_ids=None))), (INVALID, dict(over=dict(remap=None))),
                     (INVALID, dict(over=dict(src=None))), (INVALID, dict(over=dict(dst=None))), (INVALID, dict(over=dict(num_moves=None))),
                     (INVALID, dict(over=dict(num_used=None))), (INVALID, dict(over=dict(stride=7))),
                     (INVALID, dict(over=dict(page_ids=at(0), stride=9))), (INVALID, dict(over=dict(page_ids=at(0) + 4))),
                     (INVALID, dict(over=dict(remap=at(7)))), (INVALID, dict(over=dict(num_used=at(9)))), (INVALID, dict(held=at(8) + 3))]:
        assert compact(**kw) == want, (kw, lib.msgl_last_error())


def test_tensors_must_be_on_the_gpu():
    t, n = torch.zeros(2, 4, dtype=torch.int32), i32(1, 2)
    b = torch.zeros(2, 8, 128, dtype=torch.bfloat16)

    class Pool:
        k = v = torch.zeros(64, 8, 128, dtype=torch.bfloat16)
        page_size = 16

    class Rope:
        turns, axes, adjacent, factor = torch.zeros(64, dtype=torch.int64), bytes(64), False, 1.0
    for call in (lambda: ops.rope_store_kv(Pool, b, b, b, n, n, Rope), lambda: ops.fork_requests(t, n, n, n, n, 64, 16),
                 lambda: ops.copy_pages([Pool], n, n), lambda: ops.free_pages(t, n, 64, 16), lambda: ops.compact_pages(t, n, 64, 16),
                 lambda: ops.verify_drafts(torch.zeros(2, 9), None, n, i32(0, 2), torch.zeros(2), torch.zeros(1))):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_rope_arguments():
    for kw in (dict(inv_freq=[]), dict(inv_freq=[1.0] * 7), dict(inv_freq=[1.0] * 72), dict(inv_freq=[float("nan")] * 8),
               dict(inv_freq=[1.0] * 8, axes=[0] * 7), dict(inv_freq=[1.0] * 8, axes=[4] * 8), dict(inv_freq=[1.0] * 8, axes=[-1] * 8),
               dict(inv_freq=[1.0] * 8, factor=float("inf"))):
        with pytest.raises(ValueError):
            ops.Rope(**kw)
    import math
    r = ops.Rope(torch.tensor([1.0, 0.25, -0.25, 7.0, 0.0, 1e-9, 2 * math.pi, 1e6], dtype=torch.float64), [0, 1, 2, 3, 0, 1, 2, 3],
                 device="cpu")
    for t, f in zip(r.turns.tolist(), (1.0, 0.25, -0.25, 7.0, 0.0, 1e-9, 2 * math.pi, 1e6)):
        # the frequency as a part of a turn, to half a unit of its 53 bits (and whole turns dropped)
        off = (t % 2 ** 64) / 2 ** 64 - (f / (2 * math.pi)) % 1.0
        assert min(abs(off), 1 - abs(off)) <= abs(f) * 2 ** -52 / (2 * math.pi) + 2 ** -63
    assert r.axes == bytes([0, 1, 2, 3] * 2)


def expect(status, fragment, fn, *args, **kw):
    with pytest.raises(ops.MsglError) as e:
        fn(*args, **kw)
    assert e.value.status == status and fragment in str(e.value), str(e.value)


def test_check_fork_meta():
    table = torch.arange(24, dtype=torch.int32).reshape(6, 4)
    ok = dict(num_slots=100 * 16, page_size=16, req_table=table, parent_rows=i32(0, 0, -1, 1), child_rows=i32(2, 3, -1, 4),
              lens=i32(17, 32, 9, 64), free_pages=i32(50))
    ops.check_fork_meta(**ok)
    c = lambda status, fragment, **kw: expect(status, fragment, ops.check_fork_meta, **{**ok, **kw})
    c(OUT_OF_RANGE, "fork 3: row 6", child_rows=i32(2, 3, -1, 6))
    c(OUT_OF_RANGE, "fork 1: row -1", parent_rows=i32(0, -1, -1, 1))
    c(INVALID, "fork 3: row 0 is a parent", child_rows=i32(2, 3, -1, 0))
    c(INVALID, "fork 1: row 2 is an earlier", child_rows=i32(2, 2, -1, 4))
    c(INVALID, "fork 0: length -1", lens=i32(-1, 32, 9, 64))
    c(OUT_OF_RANGE, "fork 3: 65 keys", lens=i32(17, 32, 9, 65))
    c(OUT_OF_RANGE, "num_free = 0", free_pages=i32())
    c(OUT_OF_RANGE, "free_pages[0] = 100", free_pages=i32(100))
    c(INVALID, "free_pages[0] = 1 is in use", free_pages=i32(1))
    bad = table.clone()
    bad[1, 1] = 77
    c(OUT_OF_RANGE, "fork 3: page_ids[1] = 77", req_table=bad, num_slots=70 * 16)
    with pytest.raises(ValueError):
        ops.check_fork_meta(**{**ok, "lens": i32(1)})


def test_check_copy_meta():
    ops.check_copy_meta(160, 16, i32(0, 1, -1, 0), i32(5, 6, -1, 7), i32(0, 16, 99, 3))
    expect(OUT_OF_RANGE, "pair 1: page 10", ops.check_copy_meta, 160, 16, i32(0, 1), i32(5, 10))
    expect(OUT_OF_RANGE, "pair 0: page -1", ops.check_copy_meta, 160, 16, i32(-1, 1), i32(5, 6))
    expect(INVALID, "pair 1: 17 tokens", ops.check_copy_meta, 160, 16, i32(0, 1), i32(5, 6), i32(1, 17))
    expect(INVALID, "pair 1: page 5 is an earlier", ops.check_copy_meta, 160, 16, i32(0, 1), i32(5, 5))
    expect(INVALID, "pair 0: page 1 is written and read", ops.check_copy_meta, 160, 16, i32(0, 1), i32(1, 5))
    ops.check_copy_meta(160, 16, i32(5, 0), i32(5, 6))       # a page onto itself
    expect(INVALID, "pair 0: page 5 is written and read", ops.check_copy_meta, 160, 16, i32(5, 5), i32(5, 6))
    with pytest.raises(ValueError):
        ops.check_copy_meta(160, 16, i32(0, 1), i32(1))


def test_check_held_meta():
    table = torch.arange(12, dtype=torch.int32).reshape(3, 4)
    ops.check_held_meta(12 * 16, 16, table, i32(0, 64, 33))
    ops.check_held_meta(12 * 16, 16, table, i32(5, 64, 33), i32(-1, 0, 2))
    expect(OUT_OF_RANGE, "request 1: row 3", ops.check_held_meta, 192, 16, table, i32(0, 1), i32(0, 3))
    expect(INVALID, "request 0: length -1", ops.check_held_meta, 192, 16, table, i32(-1, 1))
    expect(OUT_OF_RANGE, "request 1: 65 keys", ops.check_held_meta, 192, 16, table, i32(1, 65))
    expect(OUT_OF_RANGE, "request 2: page_ids[2] = 10", ops.check_held_meta, 160, 16, table, i32(1, 1, 33))


def test_check_draft_meta():
    f = lambda *x: torch.tensor(x)
    ok = dict(vocab=10, tokens=i32(99, 3, 9, -5, 0), cu_ext=i32(0, 3, 3, 5), accept_u=f(0.0, 0.5, 7.0, 0.9, -1.0),
              sample_u=f(0.0, 9.0, 0.99))
    ops.check_draft_meta(**ok)
    c = lambda status, fragment, **kw: expect(status, fragment, ops.check_draft_meta, **{**ok, **kw})
    c(INVALID, "request 1: rows [3, 2)", cu_ext=i32(0, 3, 2, 5))
    c(INVALID, "request 2: rows [3, 6)", cu_ext=i32(0, 3, 3, 6))
    c(OUT_OF_RANGE, "tokens[2] = 10", tokens=i32(99, 3, 10, -5, 0))
    c(INVALID, "accept_u[1] = 1", accept_u=f(0.0, 1.0, 7.0, 0.9, -1.0))
    c(INVALID, "request 0: sample_u", sample_u=f(float("nan"), 9.0, 0.99))
    c(INVALID, "vocab", vocab=0)
    with pytest.raises(ValueError):
        ops.check_draft_meta(**{**ok, "accept_u": f(0.0)})
