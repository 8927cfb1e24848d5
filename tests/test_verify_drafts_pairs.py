"""Draft verification by two blocks a request (a full decode batch) over rows too long for registers."""
import pytest
import torch

from tests.test_verify_drafts import batch, run, test_the_edges_in_long_rows as edges_in_long_rows

pytestmark = pytest.mark.gpu

# 73 to 152 requests get two blocks each (on 152 SMs); longer than 12288 tokens of fp32, or 16384 of bf16, is too long


@pytest.mark.parametrize("dtype,V", [(torch.float32, 12289), (torch.float32, 20011), (torch.bfloat16, 33333)])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("requests", [90, 128])
def test_rows_too_long_for_registers(requests, given, dtype, V):
    w = batch([i % 3 for i in range(requests)], V, dtype, seed=V + requests, near=0.3)
    w["su"][:3] = torch.tensor([0.0, 0.9999999, 1.0])
    run(w, given)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_their_edges(dtype):
    edges_in_long_rows(dtype, 70001, 100)
