"""GPU tests of the gated delta rule where rows differ in size by many orders:
each row is held to its own size, which no later row enters."""
import pytest
import torch

from delta_helpers import Rows, i32, unit

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


@pytest.mark.parametrize("N", [1, 4, 17])
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
