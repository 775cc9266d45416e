"""GPU tests of mfd_tree_attention where a row does not see an entry that is
not finite, in the corners: one row under a mask that hides its own entry."""
import math

import pytest
import torch

import attn_helpers as ah
from test_gpu_attention import call, check, make

pytestmark = pytest.mark.gpu


def _entry(c, r, p):
    return int(c.block_table[r, p // c.page_size]), p % c.page_size


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype,cache", [("bf16", "same"), ("fp16", "same"), ("bf16", "e4m3"), ("fp16", "e4m3")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_one_row_that_does_not_see_itself(bad, dtype, cache, D):
    """N = 1 with a mask: a clear bit hides the row's own entry, whatever it
    holds, with and without a context; a set bit shows it."""
    ctx = [0, 100, 128, 60, 0, 1000]
    sees = [False, False, False, True, True, False]
    R = len(ctx)
    s = make(R, 1, 8, 2, D, 16, ctx, [1] * R, dtype=dtype, cache=cache, seed=51)
    s["vis"][:, 0, 0] = torch.tensor(sees)
    s["words"] = ah.mask_words(s["vis"]).cuda()
    c = s["cache"]
    for r in range(R):
        page, slot = _entry(c, r, ctx[r])
        if cache == "e4m3":
            c.v_exp[page, 1, slot] = 255
        else:
            c.v[page, 1, slot, 3] = bad
    out, lse, st = call(s)
    assert st == 0
    for r in (0,):
        assert bool((out[r] == 0).all()) and bool((lse[r] == -math.inf).all())
    for r in (1, 2, 5):
        assert bool(torch.isfinite(out[r].float()).all()) and bool(torch.isfinite(lse[r]).all())
    check(s, out, lse)
