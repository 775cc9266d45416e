"""GPU tests of the norms with gates against their formulas in 64 bits."""
import math

import pytest
import torch

from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def normal(gen, *shape):
    return torch.randn(shape, device="cuda", generator=gen)


def norm64(x, w):
    x = x.double()
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w.double()


def act64(x, act):
    x = x.double()
    return x if act == "none" else torch.sigmoid(x) * (x if act == "silu" else 1)


def off(want, n, dtype):
    """Half a step of the type, its smallest one, and fp32: a mean of n squares
    (n / 8 + 16 roundings in the longest chain), the exponential's 2^-21 and its
    argument's rounding, and eight products."""
    info = torch.finfo(dtype)
    return want.abs() * (info.eps / 2 + 2.0 ** -20 + (n / 8 + 64) * 2.0 ** -24) + info.smallest_normal * info.eps / 2


@pytest.mark.parametrize("T,heads,D,dt,act", [(1, 1, 8, "bf16", "silu"), (1, 32, 128, "bf16", "silu"), (7, 3, 24, "fp16", "sigmoid"),
                                             (33, 5, 40, "bf16", "none"), (130, 12, 64, "fp16", "silu"), (9, 7, 136, "bf16", "silu"),
                                             (1000, 4, 256, "bf16", "sigmoid"), (3, 1024, 80, "fp16", "silu")])
@pytest.mark.parametrize("packed", [False, True])
def test_gated(T, heads, D, dt, act, packed):
    g = torch.Generator("cuda").manual_seed(T + D)
    dtype = DT[dt]
    both = (normal(g, T, 2 * heads * D + 16) * 2).to(dtype)
    x, z = (t.unflatten(1, (heads, D)) for t in (both[:, :heads * D], both[:, heads * D:2 * heads * D]))
    if not packed:
        x, z = x.contiguous(), z.contiguous()
    w = (1 + 0.3 * normal(g, D)).to(dtype)
    out = torch.empty((T, heads, D), dtype=dtype, device="cuda")
    mfd.mfd_gated_norm(x, z, w, EPS, act, out)
    torch.cuda.synchronize()
    want = norm64(x, w) * act64(z, act)
    err = (out.double() - want).abs()
    assert bool((err <= off(want, D, dtype)).all()), (err / off(want, D, dtype)).max().item()
    if not packed:  # in place, of either
        for to in (x, z):
            a, b = x.clone(), z.clone()
            mfd.mfd_gated_norm(a, b, w, EPS, act, a if to is x else b)
            assert torch.equal(a if to is x else b, out)


def test_gated_at_the_ends():
    """Rows of zeros, of the type's largest numbers (their squares pass fp32
    only in bf16: then the formula in fp32 gives 0), gates far out, NaN in one
    row only."""
    for dtype in DT.values():
        top = torch.finfo(dtype).max
        x = torch.ones((8, 2, 64), dtype=dtype, device="cuda")
        z = torch.ones_like(x)
        x[0] = 0
        z[1], z[2] = top, -top
        x[3, 0, 5] = math.nan
        z[4, 1, 7] = math.nan
        x[5] = 2.0 ** -14
        w, out = torch.ones(64, dtype=dtype, device="cuda"), torch.empty_like(x)
        mfd.mfd_gated_norm(x, z, w, EPS, "silu", out)
        torch.cuda.synchronize()
        want = norm64(x, w) * act64(z, "silu")
        assert bool((out[0] == 0).all()) and bool((out[2] == 0).all())
        assert bool(torch.isnan(out[3, 0]).all()) and bool(torch.isfinite(out[3, 1]).all())
        assert torch.equal(torch.isnan(out[4]), torch.isnan(want[4]))
        for i in (1, 5, 6):
            assert bool(((out[i].double() - want[i]).abs() <= off(want[i], 64, dtype)).all())


CASES = [(1, 8, "bf16", "none", None, True, True), (1, 2560, "bf16", "none", None, True, True), (5, 264, "fp16", "sigmoid", "rows", False, True),
         (3, 4096, "bf16", "silu", "one", True, False), (9, 4104, "bf16", "none", "rows", True, True), (2, 8200, "fp16", "sigmoid", "one", True, True),
         (4, 16384, "bf16", "silu", "rows", True, True), (300, 1024, "fp16", "none", None, False, False), (33, 256, "bf16", "sigmoid", "rows", True, True),
         # more rows than blocks are resident
         (700, 5600, "bf16", "silu", "rows", True, True), (701, 6400, "fp16", "sigmoid", "one", True, True),
         (403, 8320, "fp16", "none", "rows", True, True), (5000, 264, "bf16", "silu", None, True, True)]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_residual(i):
    T, H, dt, act, gate, post, pre = CASES[i]
    g = torch.Generator("cuda").manual_seed(i)
    dtype, scale = DT[dt], 0.6
    y, r = normal(g, T, H).to(dtype), (3 * normal(g, T, H)).to(dtype)
    wide = normal(g, T, H + 8).to(dtype)
    z = None if gate is None else wide[:, 8:] if gate == "rows" else wide[0, 8:].clone()
    wa, wb = ((1 + 0.3 * normal(g, H)).to(dtype) if f else None for f in (post, pre))
    ro, xo = torch.empty_like(y), torch.empty_like(y) if pre else None
    mfd.mfd_residual_norm(y, r, wa, z, act, scale, wb, EPS, ro, xo)
    torch.cuda.synchronize()
    t = (norm64(y, wa) if post else y.double()) * (act64(z, act) if gate else 1)
    want = r.double() + scale * t
    fp32 = off(scale * t.abs() + r.double().abs(), H, torch.float32)  # the sum's terms
    lim = fp32 + off(want, H, dtype)
    assert bool(((ro.double() - want).abs() <= lim).all())
    if pre:
        x = norm64(want, wb)
        grow = (x.abs().amax(-1, keepdim=True) / want.abs().amax(-1, keepdim=True).clamp_min(1e-30)) * 2
        assert bool(((xo.double() - x).abs() <= off(x, H, dtype) + fp32 * grow + 2.0 ** -20 * x.abs()).all())
    # in place: the residual over itself, the normed row over y
    a, b = y.clone(), r.clone()
    mfd.mfd_residual_norm(a, b, wa, z, act, scale, wb, EPS, b, a if pre else None)
    torch.cuda.synchronize()
    assert torch.equal(b, ro) and (not pre or torch.equal(a, xo))


def test_residual_keeps_rows_apart():
    T, H = 6, 512
    g = torch.Generator("cuda").manual_seed(1)
    y, r = (normal(g, T, H).to(torch.bfloat16) for _ in range(2))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    outs = []
    for bad in (False, True):
        if bad:
            y[2, 7], r[4, 9] = math.nan, math.inf
        ro, xo = torch.empty_like(y), torch.empty_like(y)
        mfd.mfd_residual_norm(y, r, w, None, "none", 1.0, w, EPS, ro, xo)
        torch.cuda.synchronize()
        outs.append((ro, xo))
    keep = torch.tensor([0, 1, 3, 5], device="cuda")
    for a, b in zip(*outs):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(outs[1][0][2]).all()) and bool(torch.isnan(outs[1][1][2]).all())


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("act", ["sigmoid", "silu"])
def test_gates_far_below_zero(dt, act):
    """Down to where the type's smallest number ends, and up to where a sigmoid is 1."""
    dtype = DT[dt]
    z = torch.cat([torch.arange(-110, -80, 0.125), torch.arange(-20, 100, 0.5)]).to(dtype).cuda()
    z = z[:z.numel() // 8 * 8].view(-1, 1, 8).contiguous()
    x, w, out = torch.ones_like(z), torch.ones(8, dtype=dtype, device="cuda"), torch.empty_like(z)
    mfd.mfd_gated_norm(x, z, w, 0.0, act, out)
    rows = z.flatten().expand(2, -1).contiguous()
    y, r = torch.ones_like(rows), torch.empty_like(rows)
    mfd.mfd_residual_norm(y, torch.zeros_like(y), None, rows, act, 1.0, None, EPS, r, None)
    torch.cuda.synchronize()
    want = act64(z, act)
    # the exponential's argument, 1.45 |z| + 32 at most, is rounded to 2^-24 of itself
    lim = off(want, 8, dtype) + (1.45 * z.double().abs() + 32) * 2.0 ** -24 * want.abs()
    assert bool(((out.double() - want).abs() <= lim).all())
    assert bool(((r.double() - want.flatten()).abs() <= lim.flatten()).all())
    assert dt == "fp16" or float(out[z == -88.5].double().abs().max()) > 0


@pytest.mark.parametrize("T,H,dt", [(1, 2560, "bf16"), (5, 264, "fp16"), (300, 1024, "fp16"), (5000, 264, "bf16"), (2500, 2560, "bf16"),
                                    (701, 6400, "bf16"), (403, 8320, "bf16"), (403, 16384, "fp16")])
def test_residual_and_the_next_norm(T, H, dt):
    """The plain end of a block, without a norm of its output and without a gate: one sum
    a row, for rows that all are resident and for more."""
    g = torch.Generator("cuda").manual_seed(T)
    dtype = DT[dt]
    y, r = normal(g, T, H).to(dtype), (3 * normal(g, T, H)).to(dtype)
    w = (1 + 0.3 * normal(g, H)).to(dtype)
    ro, xo = torch.empty_like(y), torch.empty_like(y)
    mfd.mfd_residual_norm(y, r, None, None, "none", 1.0, w, EPS, ro, xo)
    torch.cuda.synchronize()
    want = r.double() + y.double()
    fp32 = 2.0 ** -24 * want.abs()  # the sum, rounded once
    assert bool(((ro.double() - want).abs() <= fp32 + off(want, 0, dtype)).all())
    x = norm64(want, w)
    # a row's sum of squares carries twice the relative error of its terms, its root once
    assert bool(((xo.double() - x).abs() <= off(x, H, dtype) + 2.0 ** -22 * x.abs()).all())
    for over in ("residual", "y"):  # in place: the sum over one input, the normed row over the other
        a, b = y.clone(), r.clone()
        sum_to, x_to = (b, a) if over == "residual" else (a, b)
        mfd.mfd_residual_norm(a, b, None, None, "none", 1.0, w, EPS, sum_to, x_to)
        torch.cuda.synchronize()
        assert torch.equal(sum_to, ro) and torch.equal(x_to, xo)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_rows_of_the_largest_numbers(dt):
    """Their squares are summed in fp32: past its largest number (bf16 only) a row's norm
    is 0; rows beside it are as without it."""
    dtype = DT[dt]
    top = torch.finfo(dtype).max
    x = torch.ones((4, 2, 64), dtype=dtype, device="cuda")
    x[1] = top
    x[2, 0, ::2] = -top
    w, out = torch.ones(64, dtype=dtype, device="cuda"), torch.empty_like(x)
    mfd.mfd_gated_norm(x, torch.ones_like(x), w, EPS, "none", out)
    y, w2 = x.flatten(1), torch.ones(128, dtype=dtype, device="cuda")
    ro, xo = torch.empty_like(y), torch.empty_like(y)
    mfd.mfd_residual_norm(y, torch.ones_like(y), w2, None, "none", 1.0, w2, EPS, ro, xo)
    torch.cuda.synchronize()
    want = norm64(x, w)
    want_y = norm64(y, w2)
    if dt == "bf16":
        want[1] = want[2, 0] = want_y[1] = want_y[2] = 0
    assert bool(((out.double() - want).abs() <= off(want, 64, dtype)).all())
    want_r = 1 + want_y
    assert bool(((ro.double() - want_r).abs() <= off(want_r, 128, dtype) + off(want_y, 128, torch.float32)).all())
    want_x = norm64(want_r, w2)
    assert bool(((xo.double() - want_x).abs() <= off(want_x, 128, dtype) + off(want_y, 128, torch.float32).abs() * 4).all())


def test_more_elements_than_32_bits_count():
    """The last rows of 2^31 elements and more."""
    T, H = 135000, 16384
    g = torch.Generator("cuda").manual_seed(2)
    dtype = torch.bfloat16
    y, r = (torch.zeros((T, H), dtype=dtype, device="cuda") for _ in range(2))
    last = slice(T - 3, T)
    y[last], r[last] = normal(g, 3, H).to(dtype), normal(g, 3, H).to(dtype)
    w = (1 + 0.3 * normal(g, H)).to(dtype)
    small = [torch.empty((3, H), dtype=dtype, device="cuda") for _ in range(2)]
    mfd.mfd_residual_norm(y[last].clone(), r[last].clone(), w, y[last].clone(), "sigmoid", 1.0, w, EPS, *small)
    x = y.clone()
    mfd.mfd_residual_norm(y, r, w, x, "sigmoid", 1.0, w, EPS, r, y)
    torch.cuda.synchronize()
    assert torch.equal(r[last], small[0]) and torch.equal(y[last], small[1]) and not bool(r[:T - 3].any()) and not bool(y[:T - 3].any())
    heads = x.view(T, 64, 256)
    mfd.mfd_gated_norm(heads[last].clone(), heads[last].clone(), w[:256], EPS, "silu", small[0].view(3, 64, 256))
    mfd.mfd_gated_norm(heads, heads, w[:256], EPS, "silu", y.view(T, 64, 256))
    torch.cuda.synchronize()
    assert torch.equal(y[last], small[0]) and not bool(y[:T - 3].any())
