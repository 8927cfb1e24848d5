"""msgl_check_step_meta names the request, not its row of the resident table, and refuses what the kernel refuses."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops

INVALID, OUT_OF_RANGE = 1, 4


@pytest.fixture(scope="module", autouse=True)
def lib():
    from paged_kv_attention_24_gb300 import build
    build.build()
    return ops.load()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def test_the_request_is_named():
    table = torch.tensor([[3, -1, -1], [0, 7, -1], [1, 2, 99]], dtype=torch.int32)
    good = dict(num_slots=160, page_size=16, req_table=table, req_rows=i32(2, 1, 0), cached_lens=i32(32, 20, 16),
                new_lens=i32(0, 1, 0), free_pages=i32(5), total_tokens=1)
    ops.check_step_meta(**good)
    for cached, fragment in ((i32(32, 20, 17), "request 2: page_ids[1] = -1"),
                             (i32(33, 20, 16), "request 0: page_ids[2] = 99")):
        with pytest.raises(ops.MsglError) as e:
            ops.check_step_meta(**dict(good, cached_lens=cached))
        assert e.value.status == OUT_OF_RANGE and fragment in str(e.value), str(e.value)


def test_a_length_past_int32():
    """The kernel refuses a request of more than 2^31 - 1 tokens however wide the table is."""
    pages = 2 ** 31 // 256
    table = torch.zeros(1, pages + 1, dtype=torch.int32)
    args = dict(num_slots=256 * (pages + 2), page_size=256, req_table=table, req_rows=None,
                cached_lens=i32(2 ** 31 - 1 - 200), free_pages=i32(1, 2), total_tokens=1000)
    ops.check_step_meta(**dict(args, new_lens=i32(200)))
    with pytest.raises(ops.MsglError) as e:
        ops.check_step_meta(**dict(args, new_lens=i32(201)))
    assert e.value.status == INVALID and "request 0" in str(e.value), str(e.value)
