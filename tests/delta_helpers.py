"""Inputs and the 64-bit plain form for the recurrent layers' tests: row by
row from the definitions in include/mfd.h, with torch only for storage and
products."""
import math

import torch

from tree_verified_speculative_gb300 import mfd

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def unit(x, normalize):
    x = x.double()
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS) if normalize else x


def rule64(q, k, v, g, beta, normalize, scale, S, parent=None):
    """One request: q, k [n, Hk, Dk], v [n, Hv, Dv], g, beta [n, Hv], S [Hv, Dk,
    Dv] (None: zero).  (out [n, Hv, Dv], S after the last row, size [Hv, Dv]:
    the largest column length of any state and value seen)."""
    n, Hv, Dv = v.shape
    Hk, Dk = k.shape[1:]
    S = torch.zeros((Hv, Dk, Dv), dtype=torch.float64, device=v.device) if S is None else S.double()
    head = torch.arange(Hv, device=v.device) * Hk // Hv
    q, k = unit(q, normalize)[:, head], unit(k, normalize)[:, head]
    out = torch.zeros((n, Hv, Dv), dtype=torch.float64, device=v.device)
    size = S.norm(dim=1)
    states = []
    for i in range(n):
        at = S if parent is None or parent[i] < 0 else states[parent[i]]
        a = torch.exp(g[i].double())[:, None, None]
        at = torch.where(a == 0, torch.zeros_like(at), at * a) if torch.isfinite(at).all() else at * a
        u = beta[i].double()[:, None] * (v[i].double() - torch.einsum("hkv,hk->hv", at, k[i]))
        at = at + k[i][:, :, None] * u[:, None, :]
        out[i] = scale * torch.einsum("hkv,hk->hv", at, q[i])
        size = torch.maximum(size, torch.maximum(at.norm(dim=1), v[i].double().abs()))
        if parent is None:
            S = at
        else:
            states.append(at)
    return out, S, size


def noise(Dk, rows):
    """How far fp32 may be off, relative to the largest column of a state or
    value (with keys of length one and beta in (0, 1) a row's map of the state
    lengthens no column, so what one step adds stays at most that): for a step
    the sums of Dk products and of 64 rows' (2^-24 each of their length, by
    Cauchy and Schwarz) and six operands of 22 bits; a step is 16 rows, or what
    is left of them."""
    return ((Dk + 64) * 2.0 ** -24 + 6 * 2.0 ** -22) * (2 + rows / 16)


def out_bound(want, size, q, normalize, scale, Dk, dtype):
    """For out [n, Hv, Dv] of one request: the above times the query's length,
    and half a step of the type at the result."""
    n, Hv, _ = want.shape
    length = unit(q, normalize).norm(dim=-1).repeat_interleave(Hv // q.shape[1], 1)[..., None]
    info = torch.finfo(dtype)
    fp32 = abs(scale) * length * size * noise(Dk, n)
    return fp32 + info.eps / 2 * (want.abs() + fp32) + info.smallest_normal * info.eps / 2


class Rows:
    """The rows of R requests, cut from one packed projection, and states."""

    def __init__(self, R, N, Hk, Hv, Dk, Dv, dtype="bf16", normalize=True, seed=0, slots=None):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.gen, self.R, self.N, self.Hk, self.Hv, self.Dk, self.Dv = gen, R, N, Hk, Hv, Dk, Dv
        self.dtype, self.normalize, self.eps = DT[dtype], normalize, EPS if normalize else None
        x = self.normal(R, N, 2 * Hk * Dk + Hv * Dv)
        if not normalize:
            x[..., :2 * Hk * Dk] *= 0.7 / math.sqrt(Dk)
        x = x.to(self.dtype)
        self.q, self.k = x[..., :Hk * Dk].unflatten(2, (Hk, Dk)), x[..., Hk * Dk:2 * Hk * Dk].unflatten(2, (Hk, Dk))
        self.v = x[..., 2 * Hk * Dk:].unflatten(2, (Hv, Dv))
        rate = torch.exp(torch.rand(Hv, device="cuda", generator=gen) * 7 - 6)
        self.g = -rate * torch.nn.functional.softplus(self.normal(R, N, Hv))
        self.beta = torch.sigmoid(self.normal(R, N, Hv))
        self.scale = Dk ** -0.5
        self.state = mfd.DeltaState(slots or 2 * R, Hv, Dk, Dv)
        self.state.s.copy_(0.5 * self.normal(*self.state.s.shape))
        self.out = torch.full((R, N, Hv, Dv), 7.0, dtype=self.dtype, device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def normal(self, *shape):
        return torch.randn(shape, device="cuda", generator=self.gen)

    def rule(self, nodes=None, src=None, dst=None):
        mfd.mfd_delta_rule(self.q, self.k, self.v, self.g, self.beta, self.eps, self.scale, nodes, self.out, self.state, src,
                           dst, self.st)

    def tree(self, parent, nodes=None, src=None):
        mfd.mfd_delta_tree(self.q, self.k, self.v, self.g, self.beta, self.eps, self.scale, parent, nodes, self.out, self.state,
                           src, self.st)

    def commit(self, accept, path, nodes=None, src=None, dst=None):
        mfd.mfd_delta_commit(self.k, self.v, self.g, self.beta, self.eps, accept, path, nodes, self.state, src, dst, self.st)

    def want(self, r, n, S, parent=None, rows=None):
        rows = torch.arange(n, device="cuda") if rows is None else torch.tensor(rows, device="cuda")
        return rule64(self.q[r, rows], self.k[r, rows], self.v[r, rows], self.g[r, rows], self.beta[r, rows], self.normalize,
                      self.scale, S, parent)

    def check_out(self, r, n, want, size):
        assert bool((self.out[r, n:] == 0).all())
        if n:
            lim = out_bound(want, size, self.q[r, :n], self.normalize, self.scale, self.Dk, self.dtype)
            err = (self.out[r, :n].double() - want).abs()
            assert bool((err <= lim).all()), (err / lim).max().item()
            # as a whole: half a step is 0.29 of a step on average, the fp32 part's roundings are as often up as down
            rel = ((self.out[r, :n].double() - want).norm() / want.norm()).item()
            assert rel <= torch.finfo(self.dtype).eps * 0.3 + 2.0 ** -19, rel

    def check_state(self, got, want, size, rows):
        err = (got.double() - want).abs()
        lim = size[:, None, :] * noise(self.Dk, rows)
        assert bool((err <= lim).all()), (err / lim).max().item()
        if rows:  # 22 bits of each operand and fp32 sums, as a whole: their roundings add up like a walk's steps
            rel = ((got.double() - want).norm() / want.norm()).item()
            assert rel <= 2.0 ** -21 * (2 + (rows / 64) ** 0.5), rel


def random_tree(N, gen, depth=16, back=40):
    """Parents of a random tree of N nodes, at most `depth` below the root."""
    par, dep = [-1] * N, [0] * N
    for i in range(1, N):
        p = max(0, i - 1 - int(torch.randint(0, back, (1,), generator=gen)))
        while dep[p] >= depth:
            p = par[p]
        par[i], dep[i] = p, dep[p] + 1
    return par


def path_to(par, node):
    chain = []
    while node >= 0:
        chain.append(node)
        node = par[node]
    return chain[::-1]
