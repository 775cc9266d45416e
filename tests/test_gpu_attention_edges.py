"""GPU tests of mfd_tree_attention where its own steps can go wrong: maxima
that keep growing, rows of the 8-bit cache at the ends of their range, NaN in
the context, many requests, items cut in many parts, odd head groupings."""
import math

import pytest
import torch

import attn_helpers as ah
from test_gpu_attention import call, check, make
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu


def _entry(c, r, p):
    return int(c.block_table[r, p // c.page_size]), p % c.page_size


@pytest.mark.parametrize("D,dtype,N,cache", [(128, "bf16", 1, "same"), (128, "fp16", 65, "same"), (256, "bf16", 70, "same"),
                                             (64, "fp16", 200, "same"), (128, "bf16", 33, "e4m3"), (256, "fp16", 3, "e4m3")])
def test_maxima_that_keep_growing(D, dtype, N, cache):
    """Keys along the queries' direction with a length that grows with the
    position: every tile's scores are far above the last one's, so the running
    maximum moves and what has been summed is scaled down again and again."""
    ctx = 1500
    s = make(1, N, 4, 2, D, 64, [ctx], [N], dtype=dtype, cache="same", seed=21)
    c = s["cache"]
    s["q"] = (s["q"] * 0.1 + 1.0).to(s["q"].dtype)
    for p in range(0, ctx + N):
        page, slot = _entry(c, 0, p)
        c.k[page, :, slot] = c.k[page, :, slot] * 0.05 + (p // 100) * 0.6
    if cache == "e4m3":
        q8 = mfd.KVCache(c.n_pages, 64, 2, D, 1, c.max_pages, torch.float8_e4m3fn)
        q8.block_table.copy_(c.block_table)
        for x, t, e in ((c.k, q8.k, q8.k_exp), (c.v, q8.v, q8.v_exp)):
            x = torch.nan_to_num(x.float(), nan=0.0)
            held, code = ah.quantise_rows(x, s["q"].dtype)
            t.view(torch.uint8).copy_((held * ah.two_to(127 - code.long())[..., None]).float().to(torch.float8_e4m3fn).view(torch.uint8))
            e.copy_(code)
        s["cache"] = q8
    s["scale"] = 1.0
    out, lse, st = call(s)
    assert st == 0
    assert lse.max().item() > 0.6 * 14 * D * 0.5
    check(s, out, lse)


@pytest.mark.parametrize("dtype,D,exps", [("bf16", 128, (135, 150, 240)), ("bf16", 64, (20, 134, 136)), ("fp16", 128, (1, 90, 96)),
                                          ("fp16", 256, (94, 100, 134)), ("bf16", 256, (1, 127, 139))])
def test_8bit_rows_at_the_ends_of_their_range(dtype, D, exps):
    """Rows whose power of two has no number of the operand type (or a
    subnormal one): values exactly as they read back.  Large value rows sit at
    places that get little weight in the sum of the others only if the kernel
    scales them right, so each is checked on its own: one visible position."""
    for e in exps:
        s = make(1, 1, 4, 2, D, 16, [0], [1], dtype=dtype, cache="e4m3", seed=22)
        c = s["cache"]
        page, slot = _entry(c, 0, 0)
        c.k_exp[page, :, slot] = 127
        c.v_exp[page, :, slot] = e
        out, lse, st = call(s)
        assert st == 0
        _, V = ah.entries(c, 0, 0, 1)
        want = V[0].repeat_interleave(2, 0).to(s["q"].dtype)
        assert torch.equal(out[0, 0], want), e
        # the same power on the keys: the score is the product, in fp32
        c.v_exp[page, :, slot] = 127
        c.k_exp[page, :, slot] = e
        s["q"] = torch.full_like(s["q"], 2.0 ** -6)
        out, lse, st = call(s)
        K, _ = ah.entries(c, 0, 0, 1)
        ty = s["q"].dtype
        z = (K.to(ty).double()[0].repeat_interleave(2, 0) * 2.0 ** -6).sum(-1) * s["scale"]
        lim = D * 2.0 ** -22 * K.abs().sum(-1).max().item() * 2.0 ** -6 * s["scale"] + 1e-5
        assert bool(((lse[0, 0].double() - z).abs() <= lim).all()), (e, lse, z)


@pytest.mark.parametrize("cache", ["same", "e4m3"])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_in_the_context_reaches_every_row(cache, where):
    s = make(2, 40, 8, 2, 128, 16, [300, 200], [40, 40], cache=cache, seed=23)
    c = s["cache"]
    page, slot = _entry(c, 0, 77)
    if cache == "e4m3":
        (c.k_exp if where == "k" else c.v_exp)[page, 1, slot] = 255
    else:
        (c.k if where == "k" else c.v)[page, 1, slot, 5] = math.nan
    out, lse, st = call(s)
    assert st == 0
    hit = out[0, :, 4:]  # key head 1
    assert bool(torch.isnan(hit[..., 5]).all())
    if where == "k" or cache == "e4m3":
        assert bool(torch.isnan(hit).all())
    assert bool(torch.isfinite(out[0, :, :4].float()).all()) and bool(torch.isfinite(out[1].float()).all())


@pytest.mark.parametrize("R,N,Hq,Hk,D,mask,cache", [(70, 9, 4, 2, 64, "tree", "same"), (45, 100, 4, 1, 64, "causal", "same"),
                                                     (300, 1, 4, 2, 64, "causal", "e4m3"), (33, 40, 8, 1, 128, "causal", "e4m3"),
                                                     (1, 1200, 8, 2, 64, "causal", "same"), (36, 70, 6, 2, 256, "causal", "same")])
def test_many_requests_and_items(R, N, Hq, Hk, D, mask, cache):
    gen = torch.Generator().manual_seed(5)
    ctx = torch.randint(0, 500, (R,), generator=gen).tolist()
    nodes = torch.randint(0, N + 1, (R,), generator=gen).tolist()
    nodes[0] = N
    s = make(R, N, Hq, Hk, D, 32, ctx, nodes, cache=cache, mask=mask, seed=24)
    out, lse, st = call(s)
    assert st == 0
    check(s, out, lse)


def test_all_requests_empty():
    s = make(3, 5, 4, 2, 64, 16, [0, 10, 0], [0, 0, 0], mask="causal", seed=25)
    out, lse, st = call(s)
    assert st == 0
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_back_to_back_calls_share_scratch():
    """Calls of different shapes on one scratch and one stream, queued without
    a wait between them, give what each gives alone."""
    a = make(1, 257, 16, 4, 256, 64, [900], [257], seed=26)
    b = make(4, 1, 32, 8, 128, 16, [3000, 10, 700, 1500], [1] * 4, mask="causal", cache="e4m3", seed=27)
    c = make(2, 65, 8, 2, 80, 16, [100, 400], [65, 30], dtype="fp16", seed=28)
    cases = [a, b, c]
    alone = [call(s) for s in cases]
    need = max(mfd.mfd_tree_attention_workspace_bytes(*s["q"].shape[:3], s["cache"].Hk, s["q"].shape[3]) for s in cases)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(s["q"]) for s in cases]
    for _ in range(20):
        for s, o in zip(cases, outs):
            mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["words"], s["scale"], o, None, st, ws)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for o, (w, _, _) in zip(outs, alone):
        assert torch.equal(o.view(torch.int16), w.view(torch.int16))
