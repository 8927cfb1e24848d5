"""Small angles of the rotary store: the slow pairs of long-context bases, near position 0, keep their digits."""
import math

import pytest
import torch

from paged_kv_attention_24_gb300 import ops
from tests.step_reference import i32

pytestmark = pytest.mark.gpu

# cos, sin of a small angle, at which the one cannot hide the other: with (x, y) = (1, 0) a pair becomes (cos, sin), so
# that y' is the sine alone.  Its error, relative to itself: the frequency as 64 bits of a turn (2^-64 over 2^-34 of a
# turn or more: 2^-30), its quotient (2^-53), the angle's rounding (2^-24), the sine (two units of 2^-23), one fused
# product (2^-24): below 2^-21; then half a step of bf16.
SLACK = 2.0 ** -21
HALF = torch.finfo(torch.bfloat16).eps / 2


@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("scale", [1.0, 1 / 32])
@pytest.mark.parametrize("base", [5e5, 1e7, 1e8])
def test_slow_pairs(base, scale, adjacent):
    f = [base ** (-j / 64) * scale for j in range(64)]
    at = [1, -1, 2, 3, 7, -100, 1000, 0]
    T, H = len(at), 4
    y_at = slice(1, None, 2) if adjacent else slice(64, None)
    x = torch.ones(T, H, 128, dtype=torch.bfloat16, device="cuda")
    x[..., y_at] = 0
    pool = ops.KVPool(*[torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)], 1)
    loc = torch.arange(T, dtype=torch.int32, device="cuda")
    out = ops.rope_store_kv(pool, x, x, x, i32(at, "cuda"), loc, ops.Rope(f, adjacent=adjacent))
    sines = torch.tensor([[math.sin(p * w) for w in f] for p in at], dtype=torch.float64)[:, None, :]
    small = torch.tensor([[abs(p * w) < 0.5 for w in f] for p in at])[:, None, :].expand(T, H, 64)
    for got in (out, pool.k):
        off = (got[..., y_at].double().cpu() - sines).abs()
        assert (off <= sines.abs() * (HALF * (1 + SLACK) + SLACK))[small].all(), (off / sines.abs())[small].nan_to_num().max()
