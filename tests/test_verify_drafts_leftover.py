"""Draft verification where the leftover of p over q has no finite sum (a draft row that holds masked logits in place of
probabilities): the token comes from p, in rows that stay in registers and in longer ones."""
import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("requests", [1, 100])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 70001])
def test_a_leftover_without_a_finite_sum(V, dtype, requests):
    p, q = (torch.zeros(2 * requests, V, dtype=dtype, device="cuda") for _ in range(2))
    p[::2, [3, V - 2]] = torch.tensor([0.25, 0.75], dtype=dtype, device="cuda")
    q[::2, 7] = float("-inf")                      # p - q is infinite here, where p has no weight
    q[::2, 5] = 1                                  # the draft: p 0, so that it does not stand
    T = 2 * requests
    su = torch.tensor([(b % 4) / 4 for b in range(requests)], device="cuda")
    status = ops.new_status()
    got = ops.verify_drafts(p, q, torch.full((T,), 5, dtype=torch.int32, device="cuda"), i32(range(0, T + 1, 2), "cuda"),
                            torch.full((T,), 0.5, device="cuda"), su, status=status)
    assert got.accepted.tolist() == [0] * requests and ops.read_status(status) == 0
    # a border of the running sum (0.25) belongs to the token behind it
    assert got.tokens.tolist() == [x for b in range(requests) for x in (3 if b % 4 == 0 else V - 2, -1)]
