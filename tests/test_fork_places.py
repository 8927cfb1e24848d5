"""Which place among the free pages a fork takes when forks in front of it are refused: the numbers written out."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import i32

pytestmark = pytest.mark.gpu

PS, PAGES = 16, 60
FREE = [50, 51, 52, 53]


@pytest.mark.parametrize("name,parent,child,length,flag,place", [
    # (the fork in the middle of three; the last one's place, -1: refused for want of pages)
    ("served", 0, 4, 17, 0, 2),
    ("served, no tail", 0, 4, 32, 0, 1),
    ("padding", -1, -1, 17, 0, 1),
    ("parent outside", 8, 4, 17, ops.DEVERR_ROW, 1),
    ("child outside", 0, -1, 17, ops.DEVERR_ROW, 1),
    ("negative length", 0, 4, -15, ops.DEVERR_LENGTH, 1),
    ("too long", 0, 4, 65, ops.DEVERR_LENGTH, 1),
    ("its own parent", 2, 2, 17, ops.DEVERR_ROW, 2),
    ("a child that is a parent", 0, 1, 17, ops.DEVERR_ROW, 2),
    ("a partly filled page outside", 7, 4, 17, ops.DEVERR_PAGE_RANGE, 2),
])
def test_places_behind_a_fork(name, parent, child, length, flag, place):
    table = torch.arange(32, dtype=torch.int32).reshape(8, 4)
    table[7, 1] = PAGES
    t, status = table.cuda(), ops.new_status()
    # the first and the last fork are in order; row 1 is the last one's parent
    f = ops.fork_requests(t, i32([0, parent, 1], "cuda"), i32([3, child, 5], "cuda"), i32([5, length, 18], "cuda"),
                          i32(FREE, "cuda"), PAGES * PS, PS, status=status)
    assert ops.read_status(status) == flag
    want = table.clone()
    want[3, 0] = FREE[0]
    want[5, :2] = torch.tensor([4, FREE[place]])
    served = name in ("served", "served, no tail")
    if served:
        want[4, :2] = torch.tensor([0, FREE[1] if length == 17 else 1])
    assert torch.equal(t.cpu(), want)
    middle = (1, FREE[1], 1) if name == "served" else (-1, -1, 0)
    assert list(zip(f.src.tolist(), f.dst.tolist(), f.tokens.tolist())) == [(0, FREE[0], 5), middle, (5, FREE[place], 2)]
    assert f.pages_taken.tolist() == [place + 1]


def test_both_of_one_child_keep_their_places():
    table = torch.arange(32, dtype=torch.int32).reshape(8, 4)
    t, status = table.cuda(), ops.new_status()
    f = ops.fork_requests(t, i32([0, 1, 0], "cuda"), i32([3, 3, 4], "cuda"), i32([5, 6, 7], "cuda"), i32(FREE, "cuda"), PAGES * PS,
                          PS, status=status)
    assert ops.read_status(status) == ops.DEVERR_ROW
    assert f.dst.tolist() == [-1, -1, FREE[2]] and f.pages_taken.tolist() == [3]
    want = table.clone()
    want[4, 0] = FREE[2]
    assert torch.equal(t.cpu(), want)


@pytest.mark.parametrize("free,taken", [([], 0), ([50], 1), ([50, 51], 2), ([50, 51, 52], 2)])
def test_no_more_places_than_free_pages(free, taken):
    t, status = torch.arange(32, dtype=torch.int32).reshape(8, 4).cuda(), ops.new_status()
    f = ops.fork_requests(t, i32([0, 1], "cuda"), i32([3, 4], "cuda"), i32([5, 6], "cuda"), i32(free, "cuda"), PAGES * PS, PS,
                          status=status)
    assert f.pages_taken.tolist() == [taken] and f.dst.tolist() == (free + [-1, -1])[:2]
    assert ops.read_status(status) == (0 if len(free) >= 2 else ops.DEVERR_NO_PAGES)
