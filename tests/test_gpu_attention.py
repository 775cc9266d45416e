"""GPU tests of mfd_tree_attention against the 64-bit plain form: types, head
layouts, page sizes, lengths from none to long, tree masks, rows that see
nothing, values that must not leak, streams, graphs."""
import math

import pytest
import torch

import attn_helpers as ah
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu


def make(R, N, Hq, Hk, D, ps, ctx, nodes, dtype="bf16", cache="same", layout="head", mask="tree", seed=0, stale=math.nan):
    """A case's tensors: cache with `stale` in every slot no position uses."""
    gen = torch.Generator().manual_seed(seed)
    cg = torch.Generator("cuda").manual_seed(seed)
    ty = ah.DT[dtype]
    lens = [c + n for c, n in zip(ctx, nodes)]
    max_pages = max(1, (max(c + N for c in ctx) + ps - 1) // ps)
    n_pages = sum((x + ps - 1) // ps for x in lens) + 3
    c = mfd.KVCache(n_pages, ps, Hk, D, R, max_pages, ah.DT["e4m3"] if cache == "e4m3" else ty, layout)
    ah.fill_table(c.block_table, lens, ps, n_pages, gen)
    for t, e in ((c.k, c.k_exp), (c.v, c.v_exp)):
        x = torch.randn(t.shape, generator=cg, device="cuda")
        if t is c.v:
            x = x + 0.5
        live = torch.zeros((n_pages, ps), dtype=torch.bool, device="cuda")
        for r in range(R):
            i = torch.arange(lens[r], device="cuda")
            live[c.block_table[r, i // ps].long(), i % ps] = True
        x = torch.where(live[:, None, :, None], x, torch.full_like(x, stale))
        if e is None:
            t.copy_(x.to(ty))
        else:
            held, code = ah.quantise_rows(x, ty)
            t.view(torch.uint8).copy_((torch.nan_to_num(held) * ah.two_to(127 - code.long().clamp(0, 247))[..., None])
                                      .float().to(torch.float8_e4m3fn).view(torch.uint8))
            e.copy_(code)
    q = torch.randn((R, N, Hq, D), generator=cg, device="cuda").to(ty)
    vis = None
    if mask == "tree":
        vis = torch.stack([ah.tree_visible(N, gen) for _ in range(R)])
        for r in range(R):
            vis[r, nodes[r]:] = False
    return dict(q=q, cache=c, ctx=torch.tensor(ctx, dtype=torch.int32, device="cuda"),
                nodes=torch.tensor(nodes, dtype=torch.int32, device="cuda"), vis=vis,
                words=None if vis is None else ah.mask_words(vis).cuda(), scale=1.0 / math.sqrt(D))


def call(s, stream=None, lse=True):
    R, N, Hq, D = s["q"].shape
    out = torch.full((R, N, Hq, D), 7.0, dtype=s["q"].dtype, device="cuda")
    lse = torch.full((R, N, Hq), 7.0, device="cuda") if lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(mfd.mfd_tree_attention_workspace_bytes(R, N, Hq, s["cache"].Hk, D), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)
    torch.cuda.synchronize()
    mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["words"], s["scale"], out, lse, status, ws, stream)
    torch.cuda.synchronize()
    return out, lse, int(status.item())


def check(s, out, lse):
    D, dtype = s["q"].shape[-1], s["q"].dtype
    want, wl, pv, sv, qk = ah.attention64(s["q"], s["cache"], s["ctx"].tolist(), s["nodes"].tolist(), s["vis"], s["scale"])
    got = out.double()
    fine = torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got[~fine & ~torch.isnan(want)], want[~fine & ~torch.isnan(want)])
    lim = ah.attention_bound(want, pv, sv, qk, dtype, D)
    err = (got - want).abs()
    assert bool((err <= lim)[fine].all()), (err / lim.clamp_min(1e-30))[fine].max().item()
    if lse is not None:
        lf = torch.isfinite(wl)
        assert torch.equal(lse[~lf & ~torch.isnan(wl)].double(), wl[~lf & ~torch.isnan(wl)])
        assert torch.equal(torch.isnan(lse), torch.isnan(wl))
        le = (lse.double() - wl).abs()
        assert bool((le <= ah.lse_bound(wl, qk, D))[lf].all()), le[lf].max().item()


CASES = [
    # R, N, Hq, Hk, D, ps, ctx, nodes, dtype, cache, layout, mask
    (1, 1, 8, 8, 64, 16, [0], [1], "bf16", "same", "head", "causal"),
    (1, 1, 8, 2, 128, 16, [1], [1], "bf16", "same", "head", "causal"),
    (3, 1, 32, 8, 128, 32, [127, 128, 700], [1, 1, 1], "bf16", "same", "head", "causal"),
    (2, 1, 7, 1, 80, 16, [63, 65], [1, 1], "fp16", "same", "token", "causal"),
    (2, 1, 16, 4, 256, 64, [255, 1000], [1, 1], "bf16", "same", "head", "causal"),
    (2, 1, 4, 4, 16, 256, [300, 3], [1, 1], "fp16", "same", "head", "causal"),
    (4, 1, 32, 8, 128, 32, [5, 1000, 0, 333], [1, 1, 1, 1], "bf16", "e4m3", "head", "causal"),
    (1, 9, 8, 8, 64, 16, [0], [9], "bf16", "same", "head", "tree"),
    (2, 33, 8, 2, 128, 64, [200, 0], [33, 20], "bf16", "same", "head", "tree"),
    (2, 65, 32, 8, 128, 16, [129, 1], [65, 64], "bf16", "same", "token", "tree"),
    (1, 257, 16, 4, 256, 64, [777], [257], "bf16", "same", "head", "tree"),
    (1, 257, 12, 4, 192, 128, [300], [250], "fp16", "same", "token", "tree"),
    (3, 129, 12, 2, 96, 128, [511, 37, 250], [129, 0, 77], "fp16", "same", "head", "tree"),
    (2, 129, 32, 8, 128, 64, [900, 64], [129, 100], "bf16", "e4m3", "head", "tree"),
    (2, 65, 16, 4, 256, 32, [300, 0], [65, 65], "bf16", "e4m3", "token", "tree"),
    (2, 50, 14, 2, 80, 16, [100, 200], [50, 49], "fp16", "e4m3", "head", "tree"),
    (1, 513, 4, 1, 64, 16, [65], [513], "bf16", "same", "head", "tree"),
    (2, 300, 8, 2, 128, 64, [0, 150], [300, 123], "bf16", "same", "head", "causal"),
    (1, 777, 7, 1, 80, 16, [33], [777], "fp16", "same", "head", "causal"),
    (1, 2, 128, 1, 128, 16, [40], [2], "bf16", "same", "head", "causal"),
    (5, 17, 3, 3, 48, 16, [0, 1, 2, 126, 400], [17, 16, 1, 0, 17], "bf16", "same", "head", "tree"),
    (40, 3, 8, 4, 64, 16, list(range(0, 400, 10)), [3] * 40, "bf16", "same", "head", "causal"),
    (1, 1, 8, 2, 128, 64, [20000], [1], "bf16", "same", "head", "causal"),
    (1, 1, 16, 4, 256, 64, [9001], [1], "fp16", "e4m3", "head", "causal"),
    (2, 20, 8, 2, 128, 128, [9000, 2500], [20, 20], "bf16", "e4m3", "head", "tree"),
    (1, 130, 8, 1, 64, 32, [5000], [130], "fp16", "same", "head", "tree"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_against_the_definition(i):
    s = make(*CASES[i], seed=i)
    out, lse, st = call(s)
    assert st == 0
    check(s, out, lse)
    again, lse2, _ = call(s)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16)) and torch.equal(lse, lse2)


def test_rows_that_see_nothing():
    """Mask rows of zeros with no context, rows past n_nodes, requests without
    nodes: zeros and -inf, whatever the cache holds."""
    s = make(2, 40, 8, 2, 64, 16, [0, 0], [40, 0], seed=3)
    s["vis"][0, 5:30] = False
    s["words"] = ah.mask_words(s["vis"]).cuda()
    out, lse, st = call(s)
    assert st == 0
    assert bool((out[0, 5:30] == 0).all()) and bool((out[1] == 0).all())
    assert bool((lse[0, 5:30] == -math.inf).all()) and bool((lse[1] == -math.inf).all())
    check(s, out, lse)


@pytest.mark.parametrize("D,cache", [(64, "same"), (128, "same"), (256, "same"), (128, "e4m3")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_a_row_does_not_see_does_not_reach_it(bad, D, cache):
    """A NaN or an infinity in one node's key and in another's value reaches
    the rows below those nodes alone."""
    N = 90
    s = make(1, N, 8, 2, D, 16, [100], [N], cache=cache, seed=4, stale=bad)
    c = s["cache"]
    for node, t, e in ((7, c.k, c.k_exp), (11, c.v, c.v_exp), (12, c.v, c.v_exp)):
        p = 100 + node
        page, slot = int(c.block_table[0, p // 16]), p % 16
        if e is None:
            t[page, 1, slot, 3] = bad
        else:
            e[page, 1, slot] = 255
    out, lse, st = call(s)
    assert st == 0
    vis = s["vis"][0].cuda()
    clean = ~(vis[:, 7] | vis[:, 11] | vis[:, 12])
    assert int(clean.sum()) > 5 and int((~clean).sum()) > 2
    assert bool(torch.isfinite(out[0, clean].float()).all())
    want, *_ = ah.attention64(s["q"], c, [100], [N], s["vis"], s["scale"])
    good = torch.isfinite(want)
    assert torch.equal(torch.isfinite(out.double()) & good, good)
    assert bool(torch.isfinite(out[0, :, :4].float()).all())  # the other key head's rows
    hit = vis[:, 11] & ~vis[:, 7]
    if cache == "same" and not math.isnan(bad):
        assert bool((out[0, hit, 4:, 3] == math.inf).all())


def test_masked_lowest_scores():
    """Scores at the edge of the range: large keys the row does not see."""
    s = make(1, 40, 4, 4, 64, 16, [33], [40], seed=5)
    c = s["cache"]
    for node in (3, 9):
        p = 33 + node
        c.k[int(c.block_table[0, p // 16]), :, p % 16] *= 1e4
    out, lse, st = call(s)
    assert st == 0
    check(s, out, lse)


def test_packed_queries_and_no_lse():
    """Queries cut from a packed projection (token stride above Hq * D)."""
    s = make(2, 33, 8, 2, 128, 16, [70, 10], [33, 33], seed=6)
    want, _, _ = call(s)
    packed = torch.randn((2, 33, 12, 128), device="cuda").to(torch.bfloat16)
    packed[:, :, :8] = s["q"]
    s["q"] = packed[:, :, :8]
    got, _, st = call(s, lse=False)
    assert st == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_layouts_give_the_same_bits():
    a = make(2, 65, 8, 2, 128, 32, [300, 90], [65, 50], layout="head", seed=7)
    c = a["cache"]
    k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.k, c.v))
    b = dict(a, cache=mfd.KVCache.from_tensors(k, v, c.block_table))
    x, y = call(a), call(b)
    assert torch.equal(x[0].view(torch.int16), y[0].view(torch.int16)) and torch.equal(x[1], y[1])


def test_another_stream():
    s = make(1, 65, 8, 2, 128, 16, [500], [65], seed=8)
    want, _, _ = call(s)
    side = torch.cuda.Stream()
    got, _, st = call(s, stream=side)
    assert st == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))


def test_offsets_past_32_bits():
    """Pages whose elements start past 2^32 in the cache's storage."""
    ps, Hk, D = 256, 8, 128
    n_pages = (1 << 32) // (ps * Hk * D) + 8
    s = make(1, 5, 16, Hk, D, ps, [700], [5], mask="causal", seed=9)
    small = s["cache"]
    big = mfd.KVCache(n_pages, ps, Hk, D, 1, small.max_pages)
    used = small.block_table[0, :3].long()
    far = torch.tensor([n_pages - 1, n_pages - 3, n_pages - 2], device="cuda")
    big.k[far], big.v[far] = small.k[used], small.v[used]
    big.block_table[0, :3] = far.int()
    want, _, _ = call(s)
    got, _, st = call(dict(s, cache=big))
    assert st == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))
    del big
    torch.cuda.empty_cache()


def test_graph_replays_with_other_lengths():
    """One captured call, replayed after the lengths on the device changed."""
    s = make(2, 33, 8, 2, 128, 16, [600, 350], [33, 30], seed=10)
    R, N, Hq, D = s["q"].shape
    out = torch.empty_like(s["q"])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(mfd.mfd_tree_attention_workspace_bytes(R, N, Hq, 2, D), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["words"], s["scale"], out, None, status, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["words"], s["scale"], out, None, status, ws)
    for ctx, nodes in (([600, 350], [33, 30]), ([100, 351], [20, 29]), ([0, 9], [33, 0])):
        s["ctx"].copy_(torch.tensor(ctx, dtype=torch.int32))
        s["nodes"].copy_(torch.tensor(nodes, dtype=torch.int32))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        want, _, _ = call(s)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_device_refusals():
    """Lengths and pages outside the cache set the status; the call returns
    and the next one is right."""
    s = make(2, 33, 8, 2, 128, 16, [100, 60], [33, 33], seed=11)
    want, _, _ = call(s)
    for key, val in (("ctx", [-1, 60]), ("nodes", [34, 33]), ("nodes", [-1, 33]), ("ctx", [100000, 60])):
        _, _, st = call(dict(s, **{key: torch.tensor(val, dtype=torch.int32, device="cuda")}))
        assert st == mfd.MFD_ERR_INPUT, (key, val)
    table = s["cache"].block_table.clone()
    for page in (-5, s["cache"].n_pages, 1 << 30):
        s["cache"].block_table[1, 2] = page
        _, _, st = call(s)
        assert st == mfd.MFD_ERR_INPUT, page
    s["cache"].block_table.copy_(table)
    got, _, st = call(s)
    assert st == 0 and torch.equal(got.view(torch.int16), want.view(torch.int16))
