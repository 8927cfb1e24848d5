"""The pools of a page copy as Python objects: sequences of any kind, and one that changes while it is looked through."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import i32

pytestmark = pytest.mark.gpu


def pool(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return ops.KVPool(*[torch.randn(4 * 16, 2, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)], 16)


def copied(p):
    return torch.equal(p.k[48:], p.k[16:32]) and torch.equal(p.v[48:], p.v[16:32])


@pytest.mark.parametrize("kind", [list, tuple, iter])
def test_sequences(kind):
    pools = [pool(i) for i in range(3)]
    ops.copy_pages(kind(pools), i32([1], "cuda"), i32([3], "cuda"))
    assert all(copied(p) for p in pools)


def test_a_list_that_shrinks_on_the_way():
    pools = [pool(i) for i in range(5)]
    given = list(pools)

    class Shrinks:
        v, page_size = pools[0].v, 16

        @property
        def k(self):
            given.clear()
            return pools[0].k
    given[0] = Shrinks()
    ops.copy_pages(given, i32([1], "cuda"), i32([3], "cuda"))
    assert given == [] and all(copied(p) for p in pools)


def test_no_sequence():
    with pytest.raises(TypeError, match="sequence of KVPool"):
        ops.copy_pages(7, i32([1], "cuda"), i32([3], "cuda"))
