"""Buffers that a call around the step may not be given twice (no GPU): every call below is refused by a host check before
anything is launched."""
import ctypes

import pytest

from paged_kv_attention_24_gb300 import ops

INVALID = 1


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_24_gb300 import build
    build.build()
    return ops.load()


def at(k):
    """A device address that nothing else of a call overlaps."""
    return (k + 1) << 24


def rope(lib, q_norm=None, k_norm=None, pool=(at(0), at(1)), hq=8, **over):
    """Four tokens of hq/8 heads, three axes; each buffer on its own but for what `over` says."""
    p = ops._Pool(*pool, 256, 16, 8, 128)
    n = ops._NewTokens(at(3), at(4), at(5), at(6), hq * 128, 8 * 128, 8 * 128, hq * 128, at(7), 4, at(8), 4, hq)
    turns = over.pop("turns", at(2))
    for k, v in over.items():
        assert hasattr(n, k)
        setattr(n, k, v)
    r = ops._Rope(turns, None, 64, 3, 0, 1.0)
    return lib.msgl_rope_store_kv(ctypes.byref(p), ctypes.byref(n), ctypes.byref(r), q_norm, k_norm, 1e-6, None, None)


@pytest.mark.parametrize("name,over", [
    ("k", dict(k=at(3))), ("v", dict(v=at(3))), ("positions", dict(positions=at(3))), ("out_loc", dict(out_loc=at(3))),
    ("rope->turns", dict(turns=at(3))), ("q_norm", dict(q_norm=at(3))), ("k_norm", dict(k_norm=at(3))),
    ("the K pool", dict(pool=(at(3), at(1)))), ("the V pool", dict(pool=(at(0), at(3))))])
def test_rotation_in_place_spares_q_alone(lib, name, over):
    assert rope(lib, q_out=at(3), **over) == INVALID
    assert lib.msgl_last_error() == f"q_out overlaps {name}".encode()


def verify(lib, **over):
    d = ops._DraftBatch(at(0), at(1), 1000, 1000, 1000, 0, at(2), at(3), at(4), at(5), at(6), 3, 9, at(7), at(8), at(9))
    for k, v in over.items():
        assert hasattr(d, k)
        setattr(d, k, v)
    return lib.msgl_verify_drafts(ctypes.byref(d), None, None)


@pytest.mark.parametrize("name", ["tokens", "cu_ext", "accept_u", "sample_u", "target", "draft"])
def test_lengths_in_place_spare_the_cached_lengths_alone(lib, name):
    assert verify(lib, kv_lens=at(6), **{name: at(6)}) == INVALID
    assert lib.msgl_last_error() == f"kv_lens overlaps {name}".encode()


@pytest.mark.parametrize("name", ["accepted", "out_tokens"])
def test_no_other_output_lies_over_the_cached_lengths(lib, name):
    assert verify(lib, kv_lens=at(6), **{name: at(6)}) == INVALID
    assert verify(lib, **{name: at(6)}) == INVALID


@pytest.mark.parametrize("pool", ["K", "V"])
@pytest.mark.parametrize("name", ["q", "k", "v", "positions", "out_loc", "rope->turns", "q_norm", "k_norm"])
def test_no_input_of_the_rotary_store_lies_in_the_pools(lib, name, pool):
    """(a token's rows are stored while another's are read)"""
    first = at(0 if pool == "K" else 1)
    for where in (first, first + 255 * 2048, first + 128 * 2048 - 2048):
        kw = {"turns" if name == "rope->turns" else name: where}
        assert rope(lib, **kw) == INVALID
        assert lib.msgl_last_error() == f"the {pool} pool overlaps {name}".encode()


def test_the_two_pools_of_the_rotary_store_are_two(lib):
    for v in (at(0), at(0) + 255 * 2048, at(0) - 255 * 2048):
        assert rope(lib, pool=(at(0), v)) == INVALID
        assert lib.msgl_last_error() == b"the K pool overlaps the V pool"


def page_map(lib, compact, ws=at(10), **over):
    """16 pages, 4 rows of 8 columns, 2 requests."""
    b = dict(req_table=at(0), req_rows=at(1), lens=at(2), held=at(3), pages=at(4), num_free=at(5), page_ids=at(4), remap=at(5),
             src=at(6), dst=at(7), num_moves=at(8), num_used=at(9))
    assert not set(over) - set(b)
    b.update(over)
    args = 256, 16, b["req_table"], 4, 8, 8, b["req_rows"], b["lens"], 2, b["held"]
    tail = ws, lib.msgl_page_map_workspace_size(256, 16), None, None
    if not compact:
        return lib.msgl_free_pages(*args, b["pages"], b["num_free"], *tail)
    out = ops._CompactOut(b["page_ids"], 8, b["remap"], b["src"], b["dst"], b["num_moves"], b["num_used"])
    return lib.msgl_compact_pages(*args, ctypes.byref(out), *tail)


IN = [("req_table", 128), ("req_rows", 8), ("lens", 8), ("held", 16)]
FREE = [("pages", 64), ("num_free", 4)]
COMPACT = [("page_ids", 128), ("remap", 64), ("src", 32), ("dst", 32), ("num_moves", 4), ("num_used", 4)]


@pytest.mark.parametrize("compact,name,size", [(False, *x) for x in IN + FREE] + [(True, *x) for x in IN + COMPACT])
def test_the_page_calls_workspace_is_scratch_of_its_own(lib, compact, name, size):
    need = lib.msgl_page_map_workspace_size(256, 16)
    for where in (at(10), at(10) + need - size, at(10) + 4 - size):
        assert page_map(lib, compact, **{name: where}) == INVALID, where - at(10)
        assert b"workspace" in lib.msgl_last_error() and name.encode() in lib.msgl_last_error()


def test_the_table_in_place_is_not_the_workspace_either(lib):
    assert page_map(lib, True, req_table=at(10), page_ids=at(10)) == INVALID
    assert b"workspace" in lib.msgl_last_error()
