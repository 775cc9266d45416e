"""GPU tests of mfd_tree_attention where a row does not see an entry that is
not finite, in the corners: one row under a mask that hides its own entry, and
8-bit rows whose values leave the queries' type."""
import math

import pytest
import torch

import attn_helpers as ah
from test_gpu_attention import call, check, make
from tree_verified_speculative_gb300 import mfd

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


def _as_read(c, ty):
    """The cache with its rows as mfd_kv_read gives them in `ty`."""
    out = mfd.KVCache(c.n_pages, c.page_size, c.Hk, c.D, c.n_req, c.max_pages, ty)
    out.block_table.copy_(c.block_table)
    for x, e, y in ((c.k, c.k_exp, out.k), (c.v, c.v_exp, out.v)):
        held = x.view(torch.uint8).view(torch.float8_e4m3fn).float().double() * ah.two_to(e.long() - 127)[..., None]
        held = torch.where((e == 255)[..., None], torch.full_like(held, math.nan), held)
        y.copy_(held.float().to(ty))  # one rounding: a held value is exact in 32 bits (or past their range too)
    return out


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("dtype,low", [("fp16", 135), ("bf16", 247)])
@pytest.mark.parametrize("R", [1, 48])
def test_8bit_values_past_the_types_range(R, dtype, low, D):
    """Value rows of nodes whose power of two takes some of their elements past
    the type's largest number: those are the infinities that mfd_kv_read gives,
    and reach the rows that see the node alone.  Rows at the first such power
    whose elements stay inside are values like any other."""
    N, ctx = 70, 100
    s = make(R, N, 8, 2, D, 16, [ctx] * R, [N] * R, dtype=dtype, cache="e4m3", seed=52)
    c = s["cache"]
    g = torch.Generator("cuda").manual_seed(53)
    hit = {5: low + 1, 11: low + 2, 12: low + (15 if dtype == "fp16" else 3), 40: low + 3, 63: low + 1}
    inside = {7: low, 28: low}
    for r in range(R):
        for node, code in {**hit, **inside}.items():
            page, slot = _entry(c, r, ctx + node)
            # one sign per column: a row that sees several such nodes has one infinity there
            sign = 1.0 - 2.0 * (torch.arange(D, device="cuda") % 2)
            u = torch.rand(D, device="cuda", generator=g)
            if node in inside:
                x = 16.0 + 224.0 * u  # 240 times the power at most
            else:  # bf16: sums of what stays finite have to stay inside 32 bits
                x = 2.0 ** -9 + 2.0 ** -7 * u if dtype == "bf16" else 0.1 + 200.0 * u
                x[5::8] = 440.0
            c.v.view(torch.uint8)[page, 1, slot] = (x * sign).to(torch.float8_e4m3fn).view(torch.uint8)
            c.v_exp[page, 1, slot] = code if node in hit or dtype == "fp16" else 200
    ty = s["q"].dtype
    read = _as_read(c, ty)
    out, lse, st = call(s)
    assert st == 0
    vis = s["vis"].cuda()
    sees = vis[:, :, list(hit)].any(-1)
    assert int(sees.sum()) > 3 * R and int((~sees).sum()) > 3 * R
    assert bool(torch.isfinite(out[~sees].float()).all())
    assert bool(torch.isinf(out[sees].float()).any())
    assert bool(torch.isfinite(out[:, :, :4].float()).all())  # the other key head's rows
    check(dict(s, cache=read), out, lse)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_8bit_keys_past_the_types_range(D):
    """The same for a node's key: rows that do not see it do not change."""
    N, ctx = 70, 100
    s = make(1, N, 8, 2, D, 16, [ctx], [N], dtype="fp16", cache="e4m3", seed=54)
    c = s["cache"]
    want, wl, _ = call(s)
    page, slot = _entry(c, 0, ctx + 9)
    c.k_exp[page, 1, slot] = 150
    out, lse, st = call(s)
    assert st == 0
    hidden = ~s["vis"][0, :, 9].cuda()
    assert int(hidden.sum()) > 5
    assert torch.equal(out[0, hidden].view(torch.int16), want[0, hidden].view(torch.int16))
    assert torch.equal(lse[0, hidden], wl[0, hidden])
