"""GPU tests of the gated delta rule where rows differ in size by many orders:
each row is held to its own size, which no later row enters."""
import math

import pytest
import torch

from delta_helpers import Rows, i32, random_tree, unit

pytestmark = pytest.mark.gpu


def sized(x, r, n, S, parent=None, rows=None):
    """The 64-bit rule over rows of request r, and how far fp32 may be off.
    (out, its bound [n, Hv, Dv], S, its bound [Hv, Dv], for any element of the column.)

    With L = max(1, |1 - beta k^2|), which a row's map lengthens a column by at
    most, a state's column is no longer than N' = e^g N L + beta |k| |v|.  A row's
    sums take that much in, so its step is off by at most c N', and what was off
    before goes through the same map: E' = e^g E L + c N'.  c: sums of Dk and of
    64 products in fp32, which the tensor cores cut off instead of rounding (2^-23
    each), in every one of two such sums (S^T k; the updates), and eight factors
    of 22 bits.  The form for many rows sums over pairs of rows what the map does
    one by one: E' holds these pairs, as it adds N' at each row."""
    rows = list(range(n)) if rows is None else rows
    at = torch.tensor(rows, device="cuda")
    Hv, Dk, Dv = x.Hv, x.Dk, x.Dv
    head = torch.arange(Hv, device="cuda") * x.Hk // Hv
    q, k = unit(x.q[r, at], x.normalize)[:, head], unit(x.k[r, at], x.normalize)[:, head]
    v, a, beta = x.v[r, at].double(), torch.exp(x.g[r, at].double()), x.beta[r, at].double()
    S = torch.zeros((Hv, Dk, Dv), dtype=torch.float64, device="cuda") if S is None else S.double()
    c = (2 * (Dk + 64) + 8 * 4) * 2.0 ** -23 / 2
    info = torch.finfo(x.dtype)
    states, outs, lims = [(S, S.norm(dim=1), torch.zeros((Hv, Dv), dtype=torch.float64, device="cuda"))], [], []
    for i in range(n):
        S, N, E = states[0 if parent is not None and parent[i] < 0 else i if parent is None else parent[i] + 1]
        d, b = a[i][:, None], beta[i][:, None]
        L = (1 - b * (k[i] * k[i]).sum(-1, keepdim=True)).abs().clamp_min(1)
        S = d[..., None] * S
        u = b * (v[i] - torch.einsum("hkv,hk->hv", S, k[i]))
        S = S + k[i][:, :, None] * u[:, None, :]
        N = d * N * L + b * k[i].norm(dim=-1, keepdim=True) * v[i].abs()
        E = d * E * L + c * N
        states.append((S, N, E))
        want = x.scale * torch.einsum("hkv,hk->hv", S, q[i])
        fp32 = abs(x.scale) * q[i].norm(dim=-1, keepdim=True) * (E + c * N)
        outs.append(want)
        lims.append(fp32 + info.eps / 2 * (want.abs() + fp32) + info.smallest_normal * info.eps / 2)
    S, N, E = states[-1]
    return torch.stack(outs), torch.stack(lims), S, E + 2.0 ** -24 * N


def check(x, want, lim, S=None, lim_S=None, got=None, r=0):
    torch.cuda.synchronize()
    assert int(x.st.item()) == 0
    if want is not None:
        err = ((x.out[r, :len(want)].double() - want).abs() / lim).flatten(1).amax(1).tolist()
        assert all(e <= 1 for e in err), [f"{e:.3g}" for e in err]
    if S is not None:
        err = ((got.double() - S).abs() / lim_S[:, None]).amax().item()
        assert err <= 1, err


@pytest.mark.parametrize("N", [1, 4, 17, 18, 70])
@pytest.mark.parametrize("top", [1e30, 1e33])
@pytest.mark.parametrize("Dk", [16, 128])
def test_large_values_and_short_memories(N, top, Dk):
    """Values far up, and decays that leave next to nothing of the state: finite
    from the first row to the last, in each form."""
    x = Rows(2, N, 1, 2, Dk, 64, "bf16", True, seed=N)
    x.v.mul_(top)
    x.g.copy_(-5 - 22 * torch.rand(x.g.shape, device="cuda", generator=x.gen))
    x.g[:, 0] = -27.0
    x.rule(None, i32([-1, 0]), i32([2, 3]))
    before = x.state.s.clone()
    for r in range(2):
        out, lim, S, lim_S = sized(x, r, N, None if r == 0 else before[0])
        check(x, out, lim, S, lim_S, x.state.s[2 + r], r)
    path = list(range(min(N, 17)))
    x.commit(i32([len(path) - 1] * 2), i32([path + [-1] * (17 - len(path))] * 2), None, i32([-1, 0]), i32([2, 3]))
    for r in range(2):
        _, _, S, lim_S = sized(x, r, len(path), None if r == 0 else before[0])
        check(x, None, None, S, lim_S, x.state.s[2 + r])


def one_request(x, src=-1):
    """The rule from slot src to slot 1, checked."""
    before = None if src < 0 else x.state.s[src].clone()
    x.rule(None, i32([src]), i32([1]))
    out, lim, S, lim_S = sized(x, 0, x.N, before)
    check(x, out, lim, S, lim_S, x.state.s[1])


@pytest.mark.parametrize("N,at", [(16, 12), (64, 60), (64, 1), (200, 130)])
@pytest.mark.parametrize("dt,size,top", [("bf16", 1.0, 1e6), ("bf16", 1.0, 1e10), ("bf16", 1.0, 1e20), ("bf16", 1e-3, 1e30),
                                         ("fp16", 1e-3, 6e4)])
def test_a_large_row_takes_nothing_from_the_others(N, at, dt, size, top):
    """Rows before it keep what they have, rows behind it what its decay leaves them."""
    x = Rows(1, N, 1, 2, 64, 64, dt, True, seed=N)
    x.v.mul_(size / x.v.float().std().item())
    x.v[0, at] = (x.v[0, at].float().sign() * top).to(x.dtype)
    x.g.clamp_(max=-0.1)
    x.g[0, at + 1:at + 3] = -20.0
    one_request(x)
    x.state.s[0].mul_(size)
    one_request(x, 0)


@pytest.mark.parametrize("N", [20, 129, 300])
@pytest.mark.parametrize("dt,size,top", [("bf16", 1.0, 1e10), ("bf16", 1e-3, 1e30), ("fp16", 1e-3, 6e4)])
def test_a_large_node_takes_nothing_from_the_others(N, dt, size, top):
    """The same in a tree: large nodes among others, and below them, behind short memories."""
    x = Rows(1, N, 1, 2, 64, 64, dt, True, seed=N)
    x.v.mul_(size / x.v.float().std().item())
    x.v[0, 5::11] = (x.v[0, 5::11].float().sign() * top).to(x.dtype)
    x.g.clamp_(max=-0.1)
    x.g[0, 2::3] = -20.0
    x.state.s[0].mul_(size)
    par = random_tree(N, torch.Generator().manual_seed(N), back=9)
    x.tree(i32([par]), None, i32([0]))
    out, lim, _, _ = sized(x, 0, N, x.state.s[0], par)
    check(x, out, lim)


@pytest.mark.parametrize("N", [17, 64, 200])
@pytest.mark.parametrize("dt,size", [("bf16", 1.0), ("bf16", 1e-10), ("fp16", 1e-2)])
def test_a_large_row_that_is_forgotten(N, dt, size):
    """Nothing of it is left where the next row's decay is 0: not in the outputs, not in
    the state."""
    x = Rows(1, N, 1, 2, 64, 64, dt, True, seed=N + 1)
    x.v.mul_(size)
    x.v[0, N // 2] = 6e4
    x.g.clamp_(max=-0.1)
    x.g[0, N // 2 + 1] = -math.inf
    one_request(x)


@pytest.mark.parametrize("N", [17, 64])
@pytest.mark.parametrize("step", [1e3, 1e5, 1e7])
def test_a_large_step_takes_nothing_from_the_others(N, step):
    x = Rows(1, N, 1, 2, 64, 64, "bf16", True, seed=N + 2)
    x.g.clamp_(max=-0.1)
    x.beta[0, N // 2] = step
    x.g[0, N // 2 + 1] = -30.0
    one_request(x)


@pytest.mark.parametrize("N", [1, 17, 64, 130])
@pytest.mark.parametrize("size", [1e-12, 1e-24, 1e-30])
def test_small_values(N, size):
    """From the zero state, and from one of their size."""
    x = Rows(1, N, 1, 2, 64, 64, "bf16", True, seed=N + 3)
    x.v.mul_(size)
    one_request(x)
    x.state.s[0].mul_(size)
    one_request(x, 0)


@pytest.mark.parametrize("dt,length", [("fp16", 1e-4), ("fp16", 3e-3), ("fp16", 50.0), ("bf16", 1e-8), ("bf16", 1e-15), ("bf16", 1e-25), ("bf16", 1e8)])
def test_keys_and_queries_of_any_length(dt, length):
    """Some rows' keys and queries far shorter or longer than the others', brought to one."""
    N = 130
    x = Rows(1, N, 1, 2, 128, 64, dt, True, seed=7)
    x.k[0, 3::5].mul_(length)
    x.q[0, 4::7].mul_(length)
    x.g.clamp_(max=-0.1)
    one_request(x, 0)


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("N", [17, 64, 100])
def test_little_is_left_of_a_stretch(N, dt):
    """The last row's decay takes all rows' parts of the state down by 2^-20: what is left
    is as exact as before."""
    x = Rows(1, N, 1, 2, 128, 64, dt, True, seed=N + 4)
    x.g.clamp_(max=-0.1)
    x.g[0, -1] = -14.0
    x.beta[0, -1] = 0.0
    one_request(x, 0)


@pytest.mark.parametrize("N", [17, 64, 100])
@pytest.mark.parametrize("dt,size", [("bf16", 1e-6), ("fp16", 0.05), ("fp16", 1e-3)])
def test_a_state_of_unlike_rows(N, dt, size):
    """A row of the state that no key and no query meets, far larger than the rest: what
    meets it not is as it would be without it, but for 2^-39 of it with fp16."""
    x = Rows(1, N, 1, 2, 64, 64, dt, True, seed=N + 5)
    for t in (x.q, x.k):
        t[..., 0] = 0
    x.v.mul_(size)
    x.g.clamp_(max=-0.1)
    x.state.s.mul_(size)
    rest = x.state.s[0].clone()
    rest[:, 0] = 0
    x.state.s[0, :, 0] = 6e4
    par = random_tree(N, torch.Generator().manual_seed(N), back=9)
    # a row takes in Dk elements of the state that are off by that, and its keys and queries
    # are of length one; a step by each row before (17 nodes of a path) adds to what is off
    floor = 0 if dt == "bf16" else 2.0 ** -39 * 6e4 * 64 ** 0.5
    for form in ("rule", "tree"):
        if form == "rule":
            x.rule(None, i32([0]), i32([1]))
        else:
            x.tree(i32([par]), None, i32([0]))
        out, lim, S, lim_S = sized(x, 0, N, rest, par if form == "tree" else None)
        passed = torch.cumsum(torch.exp(torch.cumsum(x.g[0].double(), 0)), 0)[..., None] if form == "rule" else torch.full((1, 1, 1), 17.0, device="cuda")
        lim = lim + abs(x.scale) * floor * (1 + passed)
        check(x, out, lim)
        if form == "rule":
            check(x, None, None, S[:, 1:], lim_S + floor * (1 + passed[-1]), x.state.s[1, :, 1:])


@pytest.mark.parametrize("N", [1, 3, 17, 64, 100])
@pytest.mark.parametrize("what", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_no_number_in_the_formula_is_none(N, what, bad):
    """A NaN or an infinity in row i: outputs and state are finite where the 64-bit form's
    are, and nowhere else."""
    i = N // 2
    x = Rows(1, N, 2, 2, 64, 64, seed=N)
    t = getattr(x, what)
    if what in ("g", "beta"):
        t[0, i, 1] = bad
    else:
        t[0, i, 1, 5] = bad
    par = random_tree(N, torch.Generator().manual_seed(N), back=5)
    before = x.state.s[0].clone()
    x.rule(None, i32([0]), i32([1]))
    torch.cuda.synchronize()
    out, S, _ = x.want(0, N, before)
    assert torch.equal(torch.isfinite(x.out[0]), torch.isfinite(out))
    assert torch.equal(torch.isfinite(x.state.s[1]), torch.isfinite(S))
    x.tree(i32([par]), None, i32([0]))
    torch.cuda.synchronize()
    out, _, _ = x.want(0, N, before, par)
    assert torch.equal(torch.isfinite(x.out[0]), torch.isfinite(out))
    assert int(x.st.item()) == 0


@pytest.mark.parametrize("N", [1, 17, 64, 100])
@pytest.mark.parametrize("length", [1.0, 1e15])
def test_a_state_far_up(N, length):
    """A state of 1e25 and, of every fifth row, keys and queries so long that their products
    with it pass fp32 before they are divided by their length; in a column of it a NaN."""
    x = Rows(1, N, 1, 2, 64, 64, "bf16", True, seed=N + 6)
    x.k[0, ::5].mul_(length)
    x.q[0, ::5].mul_(length)
    x.g.clamp_(max=-0.1)
    x.state.s[0].mul_(1e25)
    x.state.s[0, 1, 3, 7] = math.nan
    x.rule(None, i32([0]), i32([1]))
    before = x.state.s[0].clone()
    torch.cuda.synchronize()
    assert bool(torch.isnan(x.out[0, :, 1, 7]).all()) and bool(torch.isnan(x.state.s[1, 1, :, 7]).all())
    before[1, :, 7] = 0
    x.out[0, :, 1, 7] = 0
    x.state.s[1, 1, :, 7] = 0
    out, lim, S, lim_S = sized(x, 0, N, before)
    out[:, 1, 7] = 0
    S[1, :, 7] = 0
    check(x, out, lim, S, lim_S, x.state.s[1])
