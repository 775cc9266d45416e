"""GPU tests of how mfd_tree_attention puts the parts of a cut item together:
parts of a row that have next to no weight."""
import math

import pytest
import torch

from test_gpu_attention import call, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,dtype,N", [(64, "bf16", 1), (128, "fp16", 1), (256, "bf16", 1), (128, "bf16", 40)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_value_that_is_not_finite_under_a_tiny_weight(bad, D, dtype, N):
    """A long item whose first keys score 300 powers of two below the others:
    their weights are nothing in 32 bits, but more than zero, so a NaN there
    is still the row's, and so is an infinity."""
    ctx = 20000
    s = make(1, N, 4, 2, D, 64, [ctx], [N], dtype=dtype, seed=61)
    c = s["cache"]
    s["q"] = torch.ones_like(s["q"])
    s["scale"] = 1.0
    for p in range(0, 512, 64):
        c.k[int(c.block_table[0, p // 64])] = -208.0 / D * (1 + 2 ** -5)
    rest = sorted({int(c.block_table[0, p // 64]) for p in range(512, ctx + N, 64)})
    c.k[rest] = 0.0
    page = int(c.block_table[0, 0])
    c.v[page, 1, 3, 5] = bad
    out, lse, st = call(s)
    assert st == 0
    want = torch.full_like(out[0, :, 2:, 5], bad)
    got = out[0, :, 2:, 5]
    assert bool((torch.isnan(got) if math.isnan(bad) else got == want).all()), got
    fine = torch.ones(D, dtype=torch.bool, device="cuda")
    fine[5] = False
    assert bool(torch.isfinite(out[0, :, 2:][..., fine].float()).all()) and bool(torch.isfinite(out[0, :, :2].float()).all())
    assert bool(torch.isfinite(lse).all())
