"""GPU tests of the norm-and-rotation, the cache's append, read-back and
commit against the 64-bit plain form."""
import math

import pytest
import torch

import attn_helpers as ah
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu
THETA, EPS = 1.0e6, 1e-6


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def bound(want, x, w, dtype, D):
    """Half a step of the type at the result, plus fp32: the mean of D squares,
    the root and two products (D / 8 + 16 roundings), then the turn of a pair
    (cosine and sine good to 2^-23, three more roundings) on elements at most
    as large as the row's largest, and half the type's smallest step."""
    y = ah.norm64(x, w, EPS)
    fp32 = (D / 8 + 32) * 2.0 ** -24 * y.abs().amax(-1, keepdim=True)
    info = torch.finfo(dtype)
    return info.eps / 2 * (want.abs() + fp32) + fp32 + info.smallest_normal * info.eps / 2


def packed(R, N, Hq, Hk, D, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    qkv = torch.randn((R, N, Hq + 2 * Hk, D), device="cuda", generator=g).to(dtype)
    w = [(1 + 0.3 * torch.randn(D, device="cuda", generator=g)).to(dtype) for _ in range(2)]
    return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:], w[0], w[1]


NORM = [  # T, Hq, Hk, D, rot, interleaved, dtype, norms
    (1, 1, 1, 16, 16, False, "bf16", (1, 1)),
    (7, 8, 2, 64, 64, False, "bf16", (1, 1)),
    (33, 32, 8, 128, 128, False, "bf16", (1, 1)),
    (5, 16, 4, 256, 64, False, "fp16", (1, 0)),
    (5, 16, 4, 256, 256, True, "bf16", (0, 1)),
    (9, 28, 4, 80, 40, False, "fp16", (1, 1)),
    (9, 7, 7, 80, 80, False, "bf16", (0, 0)),
    (9, 3, 1, 48, 46, True, "fp16", (1, 1)),
    (4, 3, 1, 192, 2, False, "bf16", (1, 1)),
    (4, 3, 1, 96, 0, False, "bf16", (1, 1)),
    (300, 5, 3, 112, 56, False, "bf16", (1, 1)),
]


@pytest.mark.parametrize("i", range(len(NORM)))
@pytest.mark.parametrize("far", [0, 1 << 20, (1 << 31) - 400])
def test_norm_and_rotation(i, far):
    T, Hq, Hk, D, rot, inter, dt, (nq, nk) = NORM[i]
    dtype = ah.DT[dt]
    q, k, _, qw, kw = packed(1, T, Hq, Hk, D, dtype, i)
    qw, kw = qw if nq else None, kw if nk else None
    pos = (far + torch.arange(T, device="cuda")).to(torch.int32)
    qo, ko = (torch.empty(x.shape, dtype=dtype, device="cuda") for x in (q, k))
    st = status()
    phase = mfd.rope_phases(THETA, rot)
    mfd.mfd_qk_norm_rope(q, k, qw, kw, EPS, phase, rot, inter, pos, qo, ko, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for x, w, y in ((q, qw, qo), (k, kw, ko)):
        # the angle in 64 bits loses pos * 2^-53 turns of inv_freq's own rounding: below fp32 at these positions
        want = ah.rope64(ah.norm64(x, w, EPS), pos[None], rot, THETA, inter)
        err = (y.double() - want).abs()
        lim = bound(want, x, w, dtype, D) + 2.0 ** -50 * far * ah.norm64(x, w, EPS).abs().amax(-1, keepdim=True)
        assert bool((err <= lim).all()), (err / lim).max().item()


def test_norm_and_rotation_in_place():
    q, k, _, qw, kw = packed(1, 40, 8, 2, 128, torch.bfloat16, 3)
    q, k = q.contiguous(), k.contiguous()
    pos = torch.arange(40, device="cuda", dtype=torch.int32)
    qo, ko, st = torch.empty_like(q), torch.empty_like(k), status()
    phase = mfd.rope_phases(THETA, 128)
    mfd.mfd_qk_norm_rope(q, k, qw, kw, EPS, phase, 128, False, pos, qo, ko, st)
    mfd.mfd_qk_norm_rope(q, k, qw, kw, EPS, phase, 128, False, pos, q, k, st)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), qo.view(torch.int16)) and torch.equal(k.view(torch.int16), ko.view(torch.int16))


APPEND = [  # R, N, Hq, Hk, D, ps, ctx, nodes, rot, interleaved, dtype, cache, layout
    (1, 1, 8, 2, 128, 16, [0], [1], 128, False, "bf16", "same", "head"),
    (3, 1, 32, 8, 128, 16, [15, 16, 700], [1, 1, 0], 128, False, "bf16", "same", "token"),
    (2, 33, 16, 4, 256, 64, [63, 1], [33, 20], 64, True, "fp16", "same", "head"),
    (2, 40, 28, 4, 80, 32, [31, 200], [40, 39], 40, False, "bf16", "same", "head"),
    (2, 1, 8, 2, 64, 16, [5, 31], [1, 1], 64, False, "bf16", "e4m3", "head"),
    (2, 65, 32, 8, 128, 64, [100, 3], [65, 64], 128, False, "bf16", "e4m3", "token"),
    (1, 50, 16, 4, 256, 128, [99], [50], 64, False, "fp16", "e4m3", "head"),
    (2, 17, 7, 1, 48, 16, [0, 30], [17, 9], 24, False, "fp16", "e4m3", "head"),
]


@pytest.mark.parametrize("i", range(len(APPEND)))
def test_append_and_read(i):
    R, N, Hq, Hk, D, ps, ctx, nodes, rot, inter, dt, kind, layout = APPEND[i]
    dtype = ah.DT[dt]
    gen = torch.Generator().manual_seed(i)
    max_pages = (max(ctx) + N + ps - 1) // ps
    n_pages = R * max_pages + 2
    c = mfd.KVCache(n_pages, ps, Hk, D, R, max_pages, ah.DT["e4m3"] if kind == "e4m3" else dtype, layout)
    c.k.view(torch.uint8).fill_(0x33)
    c.v.view(torch.uint8).fill_(0x33)
    if kind == "e4m3":
        c.k_exp.fill_(120)
        c.v_exp.fill_(120)
    ah.fill_table(c.block_table, [x + n for x, n in zip(ctx, nodes)], ps, n_pages, gen)
    before = [x.clone() for x in (c.k, c.v)]
    q, k, v, qw, kw = packed(R, N, Hq, Hk, D, dtype, i)
    pos = torch.randint(0, 5000, (R, N), generator=gen, dtype=torch.int32).cuda()
    tc, tn = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ctx, nodes))
    qo, st = torch.full((R, N, Hq, D), 7.0, dtype=dtype, device="cuda"), status()
    mfd.mfd_kv_append(q, k, v, qw, kw, EPS, mfd.rope_phases(THETA, rot), rot, inter, pos, tc, tn, qo, c, st)
    L = max(x + n for x, n in zip(ctx, nodes)) + 3
    ko, vo = (torch.full((R, L, Hk, D), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    mfd.mfd_kv_read(c, torch.zeros_like(tc), tc + tn, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    want_q = ah.rope64(ah.norm64(q, qw, EPS), pos, rot, THETA, inter)
    want_k = ah.rope64(ah.norm64(k, kw, EPS), pos, rot, THETA, inter)
    touched = torch.zeros((n_pages, ps), dtype=torch.bool, device="cuda")
    for r in range(R):
        n = nodes[r]
        assert bool((qo[r, n:] == 0).all())
        assert bool((ko[r, ctx[r] + n:] == 0).all()) and bool((vo[r, ctx[r] + n:] == 0).all())
        assert bool(((qo[r, :n].double() - want_q[r, :n]).abs() <= bound(want_q[r, :n], q[r, :n], qw, dtype, D)).all())
        K, V = ah.entries(c, r, 0, ctx[r] + n)
        assert torch.equal(ko[r, :ctx[r] + n].double(), K) and torch.equal(vo[r, :ctx[r] + n].double(), V)
        t = torch.arange(ctx[r], ctx[r] + n, device="cuda")
        touched[c.block_table[r, t // ps].long(), t % ps] = True
        K, V = K[ctx[r]:], V[ctx[r]:]
        lim = bound(want_k[r, :n], k[r, :n], kw, dtype, D)
        if kind == "same":
            assert torch.equal(V, v[r, :n].double())
            assert bool(((K - want_k[r, :n]).abs() <= lim).all())
        else:
            held, code = ah.quantise_rows(v[r, :n], dtype)
            assert torch.equal(V, held)  # as it comes: one exact scaling, one rounding
            assert torch.equal(c.v_exp[c.block_table[r, t // ps].long(), :, t % ps], code)
            # half a step of the held grid (2^-4 of the value, 2^-10 of the row's power of two) around the fp32 key
            e = c.k_exp[c.block_table[r, t // ps].long(), :, t % ps]
            top = want_k[r, :n].abs().amax(-1)
            p = ah.two_to(e.long() - 127)
            assert bool((top * (1 - 2.0 ** -18) <= 448 * p).all()) and bool((top * (1 + 2.0 ** -18) > 224 * p).all())
            grid = torch.maximum(want_k[r, :n].abs() * 2.0 ** -4, p[..., None] * 2.0 ** -10)
            assert bool(((K - want_k[r, :n]).abs() <= grid * (1 + 2.0 ** -10) + lim).all())
    for x, y in zip((c.k, c.v), before):  # no other entry changed
        same = (x.view(torch.uint8).view(n_pages, Hk, ps, -1) if layout == "head" else x.view(torch.uint8)) == y.view(torch.uint8)
        assert bool(same.transpose(1, 2)[~touched].all())


def test_append_without_queries():
    q, k, v, _, kw = packed(1, 20, 4, 2, 64, torch.bfloat16, 1)
    ctx, pos = torch.tensor([10], dtype=torch.int32, device="cuda"), torch.arange(20, device="cuda", dtype=torch.int32)[None]
    caches = []
    for with_q in (True, False):
        c = mfd.KVCache(2, 16, 2, 64, 1, 2)
        c.k.zero_()
        c.v.zero_()
        c.block_table.copy_(torch.tensor([[1, 0]], dtype=torch.int32))
        st = status()
        mfd.mfd_kv_append(q if with_q else None, k, v, None, kw, EPS, mfd.rope_phases(THETA, 64), 64, False, pos, ctx, None,
                          torch.empty_like(q).contiguous() if with_q else None, c, st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        caches.append(c)
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_e4m3_rows_at_the_edges(dt):
    """Rows of zeros, of the largest and smallest numbers, on the grid's
    borders, with infinities and NaN."""
    dtype = ah.DT[dt]
    info = torch.finfo(dtype)
    D = 64
    rows = [torch.zeros(D), torch.full((D,), info.max), torch.full((D,), info.tiny), torch.full((D,), info.smallest_normal * info.eps),
            torch.linspace(-448, 448, D), torch.linspace(-449, 449, D), torch.linspace(-1.75, 1.75, D), torch.linspace(-2, 2, D),
            torch.full((D,), 248.0 / 256) * info.max, torch.tensor([math.inf] + [1.0] * (D - 1)),
            torch.tensor([1.0] * (D - 1) + [math.nan]), torch.tensor([-math.inf] * D), 2.0 ** -torch.arange(D).float(),
            17 * 2.0 ** -torch.arange(D).float().clamp(0, 20), torch.tensor([-0.0, 1e-3] * (D // 2)), torch.tensor([math.nan] * D)]
    x = torch.stack(rows).to(dtype).cuda()[None, :, None, :].contiguous()
    n = x.shape[1]
    c = mfd.KVCache(1, 16, 1, D, 1, 1, torch.float8_e4m3fn)
    st, zero = status(), torch.zeros(1, dtype=torch.int32, device="cuda")
    mfd.mfd_kv_append(None, x, x, None, None, 0.0, None, 0, False, torch.zeros((1, n), dtype=torch.int32, device="cuda"), zero, None,
                      None, c, st)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    mfd.mfd_kv_read(c, zero, zero + n, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    held, code = ah.quantise_rows(x, dtype)
    assert torch.equal(c.v_exp[0, 0], code[0, :, 0]) and torch.equal(c.k_exp[0, 0], code[0, :, 0])
    want = held.to(dtype)
    for got in (ko, vo):
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)])


@pytest.mark.parametrize("kind,layout,D", [("bf16", "head", 128), ("bf16", "token", 256), ("e4m3", "head", 80), ("e4m3", "token", 64)])
def test_commit(kind, layout, D):
    R, N, L, ps, Hk = 5, 40, 16, 16, 3
    ctx, nodes = [0, 15, 100, 31, 7], [40, 40, 33, 40, 1]
    paths = [[0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 39], [0], [0, 2, 3, 32], [0, 20, 21, 30, 39], [0]]
    gen = torch.Generator().manual_seed(1)
    c = mfd.KVCache(60, ps, Hk, D, R, 10, ah.DT[kind], layout)
    ah.fill_table(c.block_table, [x + N for x in ctx], ps, 60, gen)
    x = torch.randint(0, 120, c.k.shape, device="cuda", dtype=torch.uint8) if kind == "e4m3" else torch.randn(c.k.shape, device="cuda")
    for t in (c.k, c.v):
        (t.view(torch.uint8) if kind == "e4m3" else t).copy_(x)
        x = x.flip(0)
    if kind == "e4m3":
        c.k_exp.copy_(torch.randint(100, 140, c.k_exp.shape, device="cuda"))
        c.v_exp.copy_(torch.randint(100, 140, c.v_exp.shape, device="cuda"))
    want = [[y.clone() for y in ah.entries(c, r, 0, ctx[r] + N)] for r in range(R)]
    path = torch.full((R, L + 1), -1, dtype=torch.int32)
    for r in range(R):
        path[r, :len(paths[r])] = torch.tensor(paths[r], dtype=torch.int32)
        for y in want[r]:
            src = y[[ctx[r] + p for p in paths[r]]].clone()
            y[ctx[r]:ctx[r] + len(paths[r])] = src
    tc = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st = status()
    mfd.mfd_kv_commit(c, tc, torch.tensor([len(p) - 1 for p in paths], dtype=torch.int32, device="cuda"), path.cuda(),
                      torch.tensor(nodes, dtype=torch.int32, device="cuda"), tc, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert tc.tolist() == [x + len(p) for x, p in zip(ctx, paths)]
    for r in range(R):
        for got, y in zip(ah.entries(c, r, 0, ctx[r] + N), want[r]):
            assert torch.equal(got, y)


def test_device_refusals():
    """Bad lengths, paths and pages set the status and change nothing else."""
    R, N, Hk, D, ps = 2, 8, 2, 64, 16
    c = mfd.KVCache(6, ps, Hk, D, R, 3)
    c.block_table.copy_(torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32))
    c.k.zero_()
    c.v.zero_()
    q, k, v, _, _ = packed(R, N, 4, Hk, D, torch.bfloat16, 2)
    pos = torch.zeros((R, N), dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def append(ctx, nodes):
        st = status()
        mfd.mfd_kv_append(None, k, v, None, None, EPS, None, 0, False, pos, ctx, nodes, None, c, st)
        torch.cuda.synchronize()
        return int(st.item())

    for ctx, nodes in ((i32(-1, 50), i32(8, 0)), (i32(0, 0), i32(9, 0)), (i32(0, 0), i32(-1, 0)), (i32(48, 0), i32(1, 0))):
        assert append(ctx, nodes) == mfd.MFD_ERR_INPUT
    c.block_table[0, 0] = 6
    assert append(i32(0, 0), i32(8, 0)) == mfd.MFD_ERR_INPUT
    c.block_table[0, 0] = -1
    assert append(i32(0, 0), i32(8, 0)) == mfd.MFD_ERR_INPUT
    c.block_table[0, 0] = 0
    assert bool((c.k == 0).all()) and bool((c.v == 0).all())
    assert append(i32(0, 5), i32(8, 8)) == 0
    before = c.k.clone()

    def commit(ctx, acc, path, nodes):
        st, new = status(), i32(0, 0)
        mfd.mfd_kv_commit(c, ctx, acc, torch.tensor(path, dtype=torch.int32, device="cuda"), nodes, new, st)
        torch.cuda.synchronize()
        return int(st.item()), new.tolist()

    good = [0, 1, 2]
    for acc, bad in ((2, [1, 2, 3]), (2, [0, 2, 2]), (2, [0, 3, 8]), (3, good), (-1, good), (1, [0, -1, -1])):
        assert commit(i32(0, 5), i32(acc, 0), [bad, [0, -1, -1]], i32(8, 8)) == (mfd.MFD_ERR_INPUT, [0, 6])
    assert commit(i32(47, 5), i32(2, 0), [good, good], i32(8, 8)) == (mfd.MFD_ERR_INPUT, [47, 6])
    assert torch.equal(c.k, before)
    ko, vo, st = (torch.full((R, 9, Hk, D), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)), None, status()
    ko, vo = ko
    mfd.mfd_kv_read(c, i32(44, -1), i32(9, 3), ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == mfd.MFD_ERR_INPUT
    assert torch.equal(ko[0, :4], c.k[2, :, 12:16].transpose(0, 1)) and bool((ko[0, 4:] == 0).all()) and bool((vo[1] == 0).all())
