"""GPU tests of the gated delta rule over rows, trees and accepted paths
against the 64-bit plain form."""
import math

import pytest
import torch

from delta_helpers import Rows, i32, path_to, random_tree
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu

RULE = [  # R, N, Hk, Hv, Dk, Dv, dtype, normalize, live rows
    (1, 1, 1, 1, 16, 16, "bf16", True, None),
    (1, 1, 16, 32, 128, 128, "bf16", True, None),
    (5, 1, 2, 6, 64, 80, "fp16", True, [1, 0, 1, 1, 0]),
    (40, 1, 4, 8, 128, 128, "bf16", False, None),
    (2, 2, 2, 2, 128, 256, "bf16", True, [2, 1]),
    (3, 15, 1, 3, 48, 48, "fp16", False, [15, 0, 7]),
    (2, 17, 4, 4, 112, 144, "bf16", True, [17, 16]),
    (2, 63, 2, 4, 128, 128, "bf16", True, None),
    (2, 64, 2, 4, 128, 128, "fp16", True, None),
    (2, 65, 2, 4, 128, 128, "bf16", False, [65, 64]),
    (3, 128, 1, 2, 96, 192, "bf16", True, [128, 127, 1]),
    (4, 129, 2, 2, 64, 64, "fp16", True, [129, 128, 65, 0]),
    (1, 200, 1, 1, 16, 256, "bf16", True, None),
    (3, 333, 2, 6, 80, 112, "fp16", False, [333, 31, 257]),
    (1, 1000, 2, 4, 128, 128, "bf16", True, None),
    (2, 777, 1, 1, 128, 128, "fp16", True, [777, 640]),
]


@pytest.mark.parametrize("i", range(len(RULE)))
def test_rule(i):
    """From slots to others, one of the requests from the zero state."""
    R, N, Hk, Hv, Dk, Dv, dt, norm, live = RULE[i]
    x = Rows(R, N, Hk, Hv, Dk, Dv, dt, norm, seed=i)
    before = x.state.s.clone()
    src = [(r * 7 + 3) % R if R % 7 else r for r in range(R)]
    src[R // 2] = -1
    dst = [R + (r + 1) % R for r in range(R)]
    x.rule(None if live is None else i32(live), i32(src), i32(dst))
    torch.cuda.synchronize()
    assert int(x.st.item()) == 0
    for r in range(R):
        n = N if live is None else live[r]
        out, S, size = x.want(r, n, before[src[r]] if src[r] >= 0 else None)
        x.check_out(r, n, out, size)
        x.check_state(x.state.s[dst[r]], S, size, n)
    assert torch.equal(x.state.s[:R], before[:R])


@pytest.mark.parametrize("N", [1, 5, 100])
def test_rule_in_place_and_without_a_new_state(N):
    R = 3
    x, y, z = (Rows(R, N, 2, 4, 64, 64, seed=3, slots=R) for _ in range(3))
    before = x.state.s.clone()
    x.rule()
    y.rule(None, i32([0, 1, 2]), None)
    z.rule(None, None, i32([-1, -1, -1]))
    torch.cuda.synchronize()
    assert int(x.st.item()) == int(y.st.item()) == int(z.st.item()) == 0
    assert torch.equal(x.state.s, y.state.s) and torch.equal(z.state.s, before)
    assert torch.equal(x.out, y.out) and torch.equal(x.out, z.out)
    for r in range(R):
        _, S, size = x.want(r, N, before[r])
        x.check_state(x.state.s[r], S, size, N)


def test_rule_one_state_for_several_requests():
    """A prompt's state read by all requests of the call (and by a tree's)."""
    R, N = 4, 70
    x = Rows(R, N, 1, 2, 128, 128, seed=4, slots=R + 1)
    before = x.state.s.clone()
    x.rule(None, i32([0] * R), i32([1, 2, 3, 4]))
    torch.cuda.synchronize()
    for r in range(R):
        out, S, size = x.want(r, N, before[0])
        x.check_out(r, N, out, size)
        x.check_state(x.state.s[r + 1], S, size, N)


@pytest.mark.parametrize("N,cut", [(300, 123), (130, 1), (64, 63), (20, 9)])
def test_a_prompt_in_two_stretches(N, cut):
    """Rows 0 .. cut - 1 and the rest: the same within the bounds of each."""
    a, b = Rows(2, N, 2, 4, 128, 128, seed=5, slots=2), Rows(2, N, 2, 4, 128, 128, seed=5, slots=2)
    before = a.state.s.clone()
    a.rule()
    for lo, hi in ((0, cut), (cut, N)):
        parts = [t[:, lo:hi].contiguous() for t in (b.g, b.beta)]
        out = torch.empty((2, hi - lo, 4, 128), dtype=b.dtype, device="cuda")
        for r in range(2):  # a stretch of a longer buffer: one request a call
            mfd.mfd_delta_rule(b.q[r:r + 1, lo:hi], b.k[r:r + 1, lo:hi], b.v[r:r + 1, lo:hi], parts[0][r:r + 1], parts[1][r:r + 1],
                               b.eps, b.scale, None, out[r:r + 1], b.state, i32([r]), i32([r]), b.st)
        b.out[:, lo:hi] = out
    torch.cuda.synchronize()
    assert int(a.st.item()) == int(b.st.item()) == 0
    for r in range(2):
        out, S, size = a.want(r, N, before[r])
        for x in (a, b):
            x.check_out(r, N, out, size)
            x.check_state(x.state.s[r], S, size, N)


@pytest.mark.parametrize("N", [1, 20, 64, 150])
def test_decays_at_their_ends(N):
    """log decay 0 (all is kept), -inf (nothing is), and very negative ones."""
    x = Rows(1, N, 1, 4, 64, 64, seed=6)
    x.g[:, :, 0] = 0
    x.g[:, ::3, 1] = -math.inf
    x.g[:, :, 2] = -200.0
    x.g[:, :, 3] = -1e-7
    before = x.state.s.clone()
    x.rule(None, i32([0]), i32([1]))
    torch.cuda.synchronize()
    out, S, size = x.want(0, N, before[0])
    x.check_out(0, N, out, size)
    x.check_state(x.state.s[1], S, size, N)


@pytest.mark.parametrize("N", [3, 64, 100, 200])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_nothing_reaches_the_rows_before(N, what, bad):
    """A NaN or an infinity in row i: rows before it are as without it, bit for
    bit or within the bounds (another form of the same sums); from it on what
    the formula says is not a number is none, and other columns (for a value)
    and other heads are not touched."""
    i = N // 2
    x = Rows(1, N, 2, 2, 64, 64, seed=7)
    before = x.state.s.clone()
    out, S, size = x.want(0, N, before[0])
    t = getattr(x, what)
    if what in ("g", "beta"):
        t[0, i, 1] = bad
    else:
        t[0, i, 1, 5] = bad
    x.rule(None, i32([0]), i32([1]))
    torch.cuda.synchronize()
    got = x.out[0].double()
    lim = 2.0 ** -7 * (out.abs() + x.scale * size)  # the type's step at size, twice over
    assert bool(((got - out).abs() <= lim)[:, 0].all()), "the other head"
    assert bool(((got - out).abs() <= lim)[:i].all()), "rows before"
    x.check_state(x.state.s[1, :1], S[:1], size[:1], N)
    if what == "v":
        keep = torch.arange(64, device="cuda") != 5
        assert bool(((got - out).abs() <= lim)[:, 1, keep].all()), "other columns"
        assert not bool(torch.isfinite(got[i:, 1, 5]).any())
        x.check_state(x.state.s[1, 1:, :, keep], S[1:, :, keep], size[1:, keep], N)
    elif what == "q":
        assert not bool(torch.isfinite(got[i, 1]).any()) or bad == math.inf
        assert bool(((got - out).abs() <= lim)[i + 1:].all()), "rows after"
        x.check_state(x.state.s[1], S, size, N)
    elif math.isnan(bad):
        assert not bool(torch.isfinite(got[i:, 1]).any()) and not bool(torch.isfinite(x.state.s[1, 1]).any())


@pytest.mark.parametrize("N", [1, 30, 64, 130])
def test_rows_past_the_end_are_not_read(N):
    """NaN behind n_nodes, in every input and in the outputs' memory."""
    live = [N - 1, N // 2, N]
    x, y = Rows(3, N, 1, 2, 64, 64, seed=8), Rows(3, N, 1, 2, 64, 64, seed=8)
    for r, n in enumerate(live):
        for t in (y.q, y.k, y.v, y.g, y.beta, y.out):
            t[r, n:] = math.nan
    for t in (x, y):
        t.rule(i32(live), i32([0, 1, 2]), i32([3, 4, 5]))
    torch.cuda.synchronize()
    assert torch.equal(x.out, y.out) and torch.equal(x.state.s, y.state.s)


TREE = [  # R, N, Hk, Hv, Dk, Dv, dtype, normalize, live
    (1, 1, 1, 1, 16, 16, "bf16", True, None),
    (1, 2, 1, 2, 128, 128, "bf16", True, None),
    (2, 17, 2, 4, 64, 80, "fp16", True, [17, 5]),
    (1, 64, 2, 2, 128, 128, "bf16", True, None),
    (3, 65, 2, 4, 128, 128, "bf16", True, [65, 0, 64]),
    (2, 66, 1, 1, 128, 256, "fp16", False, [66, 65]),
    (2, 129, 2, 4, 128, 128, "bf16", True, [129, 100]),
    (1, 130, 1, 3, 96, 48, "bf16", False, None),
    (2, 257, 1, 2, 128, 128, "bf16", True, [257, 256]),
    (1, 300, 1, 1, 48, 112, "fp16", True, None),
    (1, 513, 1, 2, 128, 128, "bf16", True, None),
    (2, 450, 1, 1, 64, 144, "bf16", True, [450, 385]),
]


@pytest.mark.parametrize("i", range(len(TREE)))
@pytest.mark.parametrize("back", [1, 5, 40, 600])
def test_tree(i, back):
    """Trees from near chains (back 1) to near stars (back 600)."""
    R, N, Hk, Hv, Dk, Dv, dt, norm, live = TREE[i]
    gen = torch.Generator().manual_seed(i)
    x = Rows(R, N, Hk, Hv, Dk, Dv, dt, norm, seed=20 + i)
    before = x.state.s.clone()
    live = live or [N] * R
    par = [random_tree(N, gen, back=back) for _ in range(R)]
    src = list(range(R))[::-1]
    src[0] = -1 if R > 1 else src[0]
    parent = i32(par)
    for r in range(R):
        parent[r, live[r]:] = -7  # not read
    x.tree(parent, i32(live), i32(src))
    torch.cuda.synchronize()
    assert int(x.st.item()) == 0 and torch.equal(x.state.s, before)
    for r in range(R):
        out, _, size = x.want(r, live[r], before[src[r]] if src[r] >= 0 else None, par[r])
        x.check_out(r, live[r], out, size)


@pytest.mark.parametrize("N", [8, 64, 100, 300])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
def test_a_node_reaches_only_nodes_below_it(N, what):
    gen = torch.Generator().manual_seed(N)
    x, y = Rows(1, N, 2, 2, 64, 64, seed=9), Rows(1, N, 2, 2, 64, 64, seed=9)
    par = random_tree(N, gen, back=12)
    node = N // 3
    t = getattr(y, what)
    if what in ("g", "beta"):
        t[0, node, 1] = math.nan
    else:
        t[0, node, 1, 5] = math.nan
    for z in (x, y):
        z.tree(i32([par]), None, i32([0]))
    torch.cuda.synchronize()
    below = torch.tensor([node in path_to(par, j) for j in range(N)], device="cuda")
    if what == "q":
        below = torch.arange(N, device="cuda") == node
    assert torch.equal(x.out[0, ~below], y.out[0, ~below]) and torch.equal(x.out[0, :, 0], y.out[0, :, 0])
    if what == "v":
        keep = torch.arange(64, device="cuda") != 5
        assert torch.equal(x.out[..., keep], y.out[..., keep])
        assert bool(torch.isnan(y.out[0, below, 1, 5]).all())
    else:
        assert bool(torch.isnan(y.out[0, below, 1]).all())


def test_tree_decays_at_their_ends():
    N, gen = 90, torch.Generator().manual_seed(2)
    x = Rows(1, N, 1, 4, 64, 64, seed=10)
    x.g[:, :, 0] = 0
    x.g[:, ::3, 1] = -math.inf
    x.g[:, :, 2] = -200.0
    x.g[:, :, 3] = -1e-7
    par = random_tree(N, gen, back=9)
    x.tree(i32([par]), None, i32([1]))
    torch.cuda.synchronize()
    out, _, size = x.want(0, N, x.state.s[1], par)
    x.check_out(0, N, out, size)


def paths(par, live, L, gen):
    path, accept = torch.full((len(par), L + 1), -1, dtype=torch.int32), []
    for r, p in enumerate(par):
        chain = path_to(p, int(torch.randint(0, live[r], (1,), generator=gen)))[:L + 1]
        path[r, :len(chain)] = torch.tensor(chain, dtype=torch.int32)
        accept.append(len(chain) - 1)
    return path.cuda(), accept


@pytest.mark.parametrize("R,N,Hk,Hv,Dk,Dv,dt,norm,L", [(1, 1, 1, 1, 16, 16, "bf16", True, 1), (3, 40, 2, 4, 128, 128, "bf16", True, 16),
                                                    (40, 129, 1, 4, 128, 128, "fp16", True, 15), (5, 513, 1, 3, 80, 208, "bf16", False, 8)])
def test_commit(R, N, Hk, Hv, Dk, Dv, dt, norm, L):
    gen = torch.Generator().manual_seed(N)
    x = Rows(R, N, Hk, Hv, Dk, Dv, dt, norm, seed=30)
    before = x.state.s.clone()
    par = [random_tree(N, gen, back=3) for _ in range(R)]
    path, accept = paths(par, [N] * R, L, gen)
    src = list(range(R))
    src[-1] = -1 if R > 1 else 0
    x.commit(i32(accept), path, None if R == 1 else i32([N] * R), i32(src), i32([R + r for r in range(R)]))
    torch.cuda.synchronize()
    assert int(x.st.item()) == 0 and torch.equal(x.state.s[:R], before[:R])
    for r in range(R):
        rows = path[r, :accept[r] + 1].tolist()
        _, S, size = x.want(r, len(rows), before[src[r]] if src[r] >= 0 else None, rows=rows)
        x.check_state(x.state.s[R + r], S, size, len(rows))


@pytest.mark.parametrize("N", [5, 64, 200])
@pytest.mark.parametrize("what", ["alike", "in turn", "zero"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_keys_that_repeat(N, what, dt):
    """One key over and over, two in turn, none: what a row takes back is what the
    rows before it put there."""
    gen = torch.Generator().manual_seed(N)
    x = Rows(1, N, 1, 2, 128, 64, dt, True, seed=N, slots=2)
    if what == "zero":
        x.k.zero_()
    else:
        period = 1 if what == "alike" else 2
        x.k.copy_(x.k[:, torch.arange(N, device="cuda") % period].clone())
    x.g.mul_(0.01)
    x.beta.copy_(1 - x.beta * 0.01)
    before = x.state.s.clone()
    x.rule(None, i32([0]), i32([1]))
    torch.cuda.synchronize()
    out, S, size = x.want(0, N, before[0])
    x.check_out(0, N, out, size)
    x.check_state(x.state.s[1], S, size, N)
    par = random_tree(N, gen)
    x.tree(i32([par]), None, i32([0]))
    torch.cuda.synchronize()
    out, _, size = x.want(0, N, before[0], par)
    x.check_out(0, N, out, size)
    assert int(x.st.item()) == 0


@pytest.mark.parametrize("R,Hv", [(45, 16), (300, 4)])
@pytest.mark.parametrize("form", ["rule", "commit"])
def test_more_heads_than_blocks(form, R, Hv):
    """Blocks walk several heads, of requests of unlike lengths; a request that is
    refused in between leaves the others as they are."""
    gen = torch.Generator().manual_seed(R)
    N = 7
    x = Rows(R, N, 2, Hv, 32, 48, "bf16", True, seed=R)
    before = x.state.s.clone()
    rows = torch.randint(0 if form == "rule" else 1, N + 1, (R,), generator=gen).tolist()
    wrong = R // 3
    dst = i32([R + r for r in range(R)])
    if form == "rule":
        live = list(rows)
        live[wrong] = N + 1
        x.rule(i32(live), None, dst)
    else:
        accept = [n - 1 for n in rows]
        accept[wrong] = N
        x.commit(i32(accept), torch.arange(N, dtype=torch.int32).repeat(R, 1).cuda(), None, None, dst)
    torch.cuda.synchronize()
    assert int(x.st.item()) == mfd.MFD_ERR_INPUT and torch.equal(x.state.s[:R], before[:R])
    for r in range(R):
        if r == wrong:
            assert torch.equal(x.state.s[R + r], before[R + r]) and (form == "commit" or bool((x.out[r] == 0).all()))
            continue
        out, S, size = x.want(r, rows[r], before[r])
        if form == "rule":
            x.check_out(r, rows[r], out, size)
        x.check_state(x.state.s[R + r], S, size, rows[r])


def test_device_refusals():
    """Lengths, slots, parents and paths that are none: the status is set, the
    request's outputs are zero, its state stays, and the others' are right."""
    R, N = 2, 70

    def run(form, *a, **kw):
        x = Rows(R, N, 1, 2, 64, 64, seed=11, slots=4)
        before = x.state.s.clone()
        getattr(x, form)(*a, **kw)
        torch.cuda.synchronize()
        return int(x.st.item()), x, before

    good = i32([0, 1])
    for kw in (dict(nodes=i32([-1, N])), dict(nodes=i32([N + 1, N])), dict(src=i32([4, 1]), dst=good), dict(src=i32([-2, 1]), dst=good),
               dict(src=good, dst=i32([4, 1])), dict(src=good, dst=i32([-2, 1]))):
        code, x, before = run("rule", **kw)
        assert code == mfd.MFD_ERR_INPUT
        assert bool((x.out[0] == 0).all()) and torch.equal(x.state.s[0], before[0])
        out, S, size = x.want(1, N, before[1])
        x.check_out(1, N, out, size)
        x.check_state(x.state.s[1], S, size, N)
    gen = torch.Generator().manual_seed(1)
    par = random_tree(N, gen)
    bad = []
    for at, to in ((0, 0), (0, -2), (5, 5), (5, -1), (69, 69), (30, 1 << 30), (30, -(1 << 31))):
        p = list(par)
        p[at] = to
        bad.append(p)
    bad.append([i - 1 for i in range(N)])  # too deep
    for p in bad:
        code, x, before = run("tree", i32([p, par]))
        assert code == mfd.MFD_ERR_INPUT and torch.equal(x.state.s, before)
        assert bool((x.out[0] == 0).all())
        out, _, size = x.want(1, N, before[1], par)
        x.check_out(1, N, out, size)
    for kw in (dict(nodes=i32([-1, N])), dict(nodes=i32([N + 1, N])), dict(src=i32([4, 1])), dict(src=i32([-2, 1]))):
        code, x, before = run("tree", i32([par, par]), **kw)
        assert code == mfd.MFD_ERR_INPUT and bool((x.out[0] == 0).all())
    fine = [0, 1, 2, 3]
    for accept, path in ((-1, fine), (4, fine), (2, [1, 2, 3, 4]), (2, [0, 2, 2, 3]), (3, [0, 3, 2, 5]), (1, [0, N, 0, 0]), (1, [0, -1, 0, 0])):
        code, x, before = run("commit", i32([accept, 3]), i32([path, fine]))
        assert code == mfd.MFD_ERR_INPUT and torch.equal(x.state.s[0], before[0])
        _, S, size = x.want(1, 4, before[1], rows=fine)
        x.check_state(x.state.s[1], S, size, 4)
