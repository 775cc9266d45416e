"""What is measured of the target's recurrent layers: the gated delta rule, whose state takes the place of keys and
values in a cache, and the norms with gates around such a layer's output and around a block.

Five kinds of case, each one call:

  rule    mfd_delta_rule: rows one after the other (one new token, or a prompt), from a state to the next
  tree    mfd_delta_tree: a drafted tree's nodes, each behind its own path, over a state that stays
  commit  mfd_delta_commit: the state after the accepted path
  gated   mfd_gated_norm: norm of each head's output times its activated gate
  block   mfd_residual_norm: a block's output through its norm, gate and scale into the residual, and the next block's
          norm of it

`own` chooses between the library's calls and their plain form in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6
CHUNK = 64


def listed():
    heads = dict(Hk=16, Hv=32, Dk=128, Dv=128, normalize=True)
    return [
        # one user, one token at a time: the call's latency
        dict(name="rule_one_token", kind="rule", n_req=1, N=1, dtype="bf16", **heads),
        # a serving batch without drafts, one token each: the states' bytes
        dict(name="rule_batch_tokens", kind="rule", n_req=64, N=1, dtype="bf16", **heads),
        # one user's prompt: a chain, with one head's states for each SM at most
        dict(name="rule_prompt", kind="rule", n_req=1, N=4001, dtype="bf16", **heads),
        # prompts of a batch, ragged
        dict(name="rule_prompts", kind="rule", n_req=8, N=2000, dtype="bf16", **heads),
        # the default round: a 256-prefix tree for one request
        dict(name="tree_256", kind="tree", n_req=1, N=257, dtype="bf16", **heads),
        # 32 requests with 128-prefix trees
        dict(name="trees_batch", kind="tree", n_req=32, N=129, dtype="bf16", **heads),
        # one user's round: the accepted path kept
        dict(name="commit_one", kind="commit", n_req=1, N=65, dtype="bf16", **heads),
        # 32 users' rounds
        dict(name="commit_batch", kind="commit", n_req=32, N=257, dtype="bf16", **heads),
        # one token's heads
        dict(name="gated_one", kind="gated", T=1, heads=32, D=128, dtype="bf16", act="silu"),
        # prompts' heads, half precision
        dict(name="gated_prompts", kind="gated", T=16000, heads=32, D=128, dtype="fp16", act="silu"),
        # a tree's nodes through a block's end
        dict(name="block_tree", kind="block", T=257, H=2560, dtype="bf16", act="none", gate=None, post=True, pre=True),
        # prompts, a gate for each element
        dict(name="block_prompts", kind="block", T=15500, H=2560, dtype="bf16", act="sigmoid", gate="rows", post=True,
             pre=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["rule", "rule", "rule", "tree", "tree", "commit", "gated", "block"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    if kind == "gated":
        c = dict(kind=kind, heads=rng.choice([1, 4, 16, 24, 32, 48]), D=rng.choice([64, 80, 96, 128, 128, 192, 256]),
                 T=_log_int(rng, 1, 30000), dtype=dtype, act=rng.choice(["silu", "silu", "sigmoid"]))
        while c["T"] * c["heads"] * c["D"] > 16000 * 32 * 128:
            c["T"] //= 2
        return c
    if kind == "block":
        c = dict(kind=kind, H=8 * _log_int(rng, 32, 1024), T=_log_int(rng, 1, 30000), dtype=dtype,
                 act=rng.choice(["none", "sigmoid", "silu"]), gate=rng.choice([None, "rows", "one"]),
                 post=rng.random() < 0.6, pre=rng.random() < 0.8)
        while c["T"] * c["H"] > 15500 * 2560:
            c["T"] //= 2
        return c
    Hk = rng.choice([1, 2, 4, 8, 16])
    c = dict(kind=kind, Hk=Hk, Hv=Hk * rng.choice([1, 2, 2, 3]), Dk=rng.choice([64, 96, 128, 128, 128]),
             Dv=rng.choice([64, 80, 128, 128, 128, 192, 256]), normalize=rng.random() < 0.75, dtype=dtype)
    c["n_req"] = _log_int(rng, 1, 64)
    if kind == "rule":
        form = rng.choice(["one", "few", "prompt", "prompt"])
        c["N"] = {"one": 1, "few": _log_int(rng, 2, 60), "prompt": _log_int(rng, 61, 4000)}[form]
    else:
        c["N"] = _log_int(rng, 2, 513)
    # a drawn case costs no more than the largest listed ones
    most = {"rule": 8 * 2000, "tree": 32 * 129, "commit": 64 * 513}[kind] * 32
    while c["n_req"] > 1 and c["n_req"] * c["N"] * c["Hv"] > most:
        c["n_req"] //= 2
    return c


def lens(c):
    """Live rows of the case's requests: ragged, from the case alone."""
    q = np.arange(c["n_req"])
    part = 1.0 - 0.6 * np.mod(q * 0.6180339887, 1.0) if c["kind"] == "rule" else np.where(q % 3 == 2, 0.875, 1.0)
    return np.maximum(1, np.floor(c["N"] * part)).astype(np.int64)


# ------------------------------------------------------------------ inputs
def _tree(N, rng):
    """A random tree of N nodes, parents first, at most 15 deep: parents."""
    parent, depth = np.full(N, -1, np.int32), np.zeros(N, np.int32)
    back = rng.integers(1, 41, size=N)
    for i in range(1, N):
        p = max(0, i - int(back[i]))
        while depth[p] >= 15:
            p = parent[p]
        parent[i], depth[i] = p, depth[p] + 1
    return parent


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    ty = TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device=dev, generator=g)

    s = {"case": c}
    if c["kind"] == "gated":
        T, h, D = c["T"], c["heads"], c["D"]
        s["x"] = (normal(T, h, D) * torch.exp(normal(T, h, 1))).to(ty)
        # the gate is a stretch of a packed projection
        s["gate"] = normal(T, h * D + 64).to(ty)[:, 64:].unflatten(1, (h, D))
        s["w"] = (1.0 + 0.2 * normal(D)).to(ty)
        s["out"] = torch.empty((T, h, D), dtype=ty, device=dev)
        return s
    if c["kind"] == "block":
        T, H = c["T"], c["H"]
        s["y"] = (normal(T, H) * torch.exp(0.5 * normal(T, 1))).to(ty)
        s["residual"] = (normal(T, H) * 4.0 * torch.exp(0.7 * normal(H))).to(ty)
        s["w_post"] = (0.3 + 0.1 * normal(H)).to(ty) if c["post"] else None
        s["w_pre"] = (1.0 + 0.2 * normal(H)).to(ty) if c["pre"] else None
        s["gate"] = None if c["gate"] is None else normal(T if c["gate"] == "rows" else 1, H).to(ty)
        s["scale"] = 0.7
        s["residual_out"] = torch.empty((T, H), dtype=ty, device=dev)
        s["x_out"] = torch.empty((T, H), dtype=ty, device=dev) if c["pre"] else None
        return s
    rng = np.random.default_rng(seed)
    R, N, Hk, Hv, Dk, Dv = (c[n] for n in ("n_req", "N", "Hk", "Hv", "Dk", "Dv"))
    n = lens(c)
    # queries, keys and values: stretches of one projection, after its activation
    x = normal(R, N, 2 * Hk * Dk + Hv * Dv) * 1.2
    x = x * torch.sigmoid(x)
    if not c["normalize"]:
        x[..., :2 * Hk * Dk] *= 1.2 / math.sqrt(Dk)
    x = x.to(ty)
    s["q"], s["k"] = x[..., :Hk * Dk].unflatten(2, (Hk, Dk)), x[..., Hk * Dk:2 * Hk * Dk].unflatten(2, (Hk, Dk))
    s["v"] = x[..., 2 * Hk * Dk:].unflatten(2, (Hv, Dv))
    # log decays: heads that keep thousands of tokens and heads that keep a few
    rate = torch.exp(torch.rand(Hv, device=dev, generator=g) * 7.0 - 6.0)
    s["g"] = -rate * torch.nn.functional.softplus(normal(R, N, Hv))
    s["beta"] = torch.sigmoid(1.5 * normal(R, N, Hv))
    s["scale"] = 1.0 / math.sqrt(Dk)
    s["state"] = torch.zeros((2 * R, Hv, Dk, Dv), device=dev)
    s["state"][:R] = 0.3 * normal(R, Hv, Dk, Dv)
    src, dst = rng.permutation(R).astype(np.int32), R + rng.permutation(R).astype(np.int32)
    if N > 1:
        src[np.arange(R) % 4 == 3] = -1  # fresh requests
    s["src"], s["dst"] = torch.from_numpy(src).to(dev), torch.from_numpy(dst).to(dev)
    s["nodes"] = torch.from_numpy(n.astype(np.int32)).to(dev)
    s["out"] = torch.empty((R, N, Hv, Dv), dtype=ty, device=dev)
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=dev)
    if c["kind"] != "rule":
        parent = np.full((R, N), -1, np.int32)
        path = np.full((R, 16), -1, np.int32)
        accept = np.zeros(R, np.int32)
        for r in range(R):
            parent[r, :n[r]] = _tree(int(n[r]), rng)
            node, chain = int(rng.integers(0, n[r])), []
            while node >= 0:
                chain.append(node)
                node = int(parent[r, node])
            path[r, :len(chain)] = chain[::-1]
            accept[r] = len(chain) - 1
        s["parent"], s["path"] = torch.from_numpy(parent).to(dev), torch.from_numpy(path).to(dev)
        s["accept"] = torch.from_numpy(accept).to(dev)
    if own:  # the handle that a program makes once, over its states
        from tree_verified_speculative_gb300 import mfd
        s["handle"] = mfd.DeltaState.from_tensor(s["state"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from tree_verified_speculative_gb300 import mfd
    c = s["case"]
    if c["kind"] == "gated":
        mfd.mfd_gated_norm(s["x"], s["gate"], s["w"], EPS, c["act"], s["out"])
        return {"out": s["out"]}
    if c["kind"] == "block":
        mfd.mfd_residual_norm(s["y"], s["residual"], s["w_post"], s["gate"], c["act"], s["scale"], s["w_pre"], EPS,
                              s["residual_out"], s["x_out"])
        return {"residual": s["residual_out"]} | ({"x": s["x_out"]} if c["pre"] else {})
    eps = EPS if c["normalize"] else None
    kept = s["state"][c["n_req"]:]
    if c["kind"] == "rule":
        mfd.mfd_delta_rule(s["q"], s["k"], s["v"], s["g"], s["beta"], eps, s["scale"], s["nodes"], s["out"], s["handle"],
                           s["src"], s["dst"], s["status"])
        return {"out": s["out"], "state": kept}
    if c["kind"] == "tree":
        mfd.mfd_delta_tree(s["q"], s["k"], s["v"], s["g"], s["beta"], eps, s["scale"], s["parent"], s["nodes"], s["out"],
                           s["handle"], s["src"], s["status"])
        return {"out": s["out"]}
    mfd.mfd_delta_commit(s["k"], s["v"], s["g"], s["beta"], eps, s["accept"], s["path"], s["nodes"], s["handle"], s["src"],
                         s["dst"], s["status"])
    return {"state": kept}


def _run_plain(s):
    return {"gated": _plain_gated, "block": _plain_block, "rule": _plain_rule, "tree": _plain_tree,
            "commit": _plain_commit}[s["case"]["kind"]](s)


def _norm(x, w):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _act(x, act):
    return x if act == "none" else torch.sigmoid(x) if act == "sigmoid" else x * torch.sigmoid(x)


def _plain_gated(s):
    y = _norm(s["x"].float(), s["w"]) * _act(s["gate"].float(), s["case"]["act"])
    return {"out": y.to(s["x"].dtype)}


def _plain_block(s):
    ty = s["y"].dtype
    y = s["y"].float()
    if s["w_post"] is not None:
        y = _norm(y, s["w_post"])
    if s["gate"] is not None:
        y = y * _act(s["gate"].float(), s["case"]["act"])
    r = s["residual"].float() + s["scale"] * y
    out = {"residual": r.to(ty)}
    if s["w_pre"] is not None:
        out["x"] = _norm(r, s["w_pre"]).to(ty)
    return out


def _rows(s, x, heads):
    """[R, N, h, D] of the inputs in 32 bits as [R, heads, N, D], each head h repeated for the value heads that share it."""
    return x.float().transpose(1, 2).repeat_interleave(heads // x.shape[2], 1)


def _unit(x, c):
    return x * torch.rsqrt(x.square().sum(-1, keepdim=True) + EPS) if c["normalize"] else x


def _first(s):
    """The requests' states [R, Hv, Dk, Dv]; slot -1 is the zero state."""
    src = s["src"].long()
    return torch.where((src >= 0)[:, None, None, None], s["state"][src.clamp_min(0)], torch.zeros((), device=src.device))


def _inverse(A):
    """Inverse of I + A, A strictly lower triangular [.., n, n], n a power of two: of blocks twice as large, step by step."""
    n = A.shape[-1]
    T, size = torch.eye(n, device=A.device).expand(A.shape).clone(), 1
    block = torch.arange(n, device=A.device)
    while size < n:
        b = block // size
        below = (b[:, None] == b[None, :] + 1) & (b[:, None] % 2 == 1)  # the lower left block of each pair
        T = T - T @ torch.where(below, A, torch.zeros((), device=A.device)) @ T
        size *= 2
    return T


def _step(s, S, r, at):
    """States behind row at[r] of every request."""
    c = s["case"]
    k = _unit(s["k"][r, at].float(), c).repeat_interleave(c["Hv"] // c["Hk"], 1)[..., None]
    v, beta = s["v"][r, at].float()[:, :, None], s["beta"][r, at][..., None, None]
    kept = s["g"][r, at].exp()[..., None, None] * S
    return kept + k * (beta * (v - (k * kept).sum(2, keepdim=True)))


def _plain_rule(s):
    """One row as it is; more in chunks: within one, all rows' updates from a triangular system; from one to the next, the
    state."""
    c = s["case"]
    R, N, Hv, Dk, Dv = (c[n] for n in ("n_req", "N", "Hv", "Dk", "Dv"))
    dev = s["q"].device
    if N == 1:
        r, at = torch.arange(R, device=dev), torch.zeros(R, dtype=torch.int64, device=dev)
        S = _step(s, _first(s), r, at)
        s["state"][s["dst"].long()] = S
        q = s["scale"] * _unit(s["q"][:, 0].float(), c).repeat_interleave(Hv // c["Hk"], 1)
        return {"out": (q[..., None] * S).sum(2)[:, None].to(s["q"].dtype), "state": s["state"][R:]}
    n_chunk = (N + CHUNK - 1) // CHUNK
    live = (torch.arange(N, device=dev) < s["nodes"].long()[:, None])[:, None, :, None]

    def chunks(x):
        x = torch.where(live, x, torch.zeros((), device=dev, dtype=x.dtype))
        x = torch.nn.functional.pad(x, (0, 0, 0, n_chunk * CHUNK - N))
        return x.view(R, Hv, n_chunk, CHUNK, x.shape[-1])

    q, k = (chunks(_unit(_rows(s, s[n], Hv), c)) for n in ("q", "k"))
    v = chunks(_rows(s, s["v"], Hv))
    beta = chunks(s["beta"].transpose(1, 2)[..., None])
    total = chunks(s["g"].double().transpose(1, 2)[..., None]).cumsum(3)  # sums of log decays, in 64 bits
    i = torch.arange(CHUNK, device=dev)
    decay = torch.where(i[:, None] >= i, total - total.transpose(3, 4), -math.inf).float().exp()
    T = _inverse(torch.where(i[:, None] > i, beta * decay * (k @ k.transpose(3, 4)), torch.zeros((), device=dev)))
    P = s["scale"] * decay * (q @ k.transpose(3, 4))
    since = total.float().exp()
    until = (total[:, :, :, -1:] - total).float().exp()
    S, out = _first(s), []
    for j in range(n_chunk):
        u = T[:, :, j] @ (beta[:, :, j] * (v[:, :, j] - since[:, :, j] * (k[:, :, j] @ S)))
        out.append(s["scale"] * since[:, :, j] * (q[:, :, j] @ S) + P[:, :, j] @ u)
        S = since[:, :, j, -1:] * S + (k[:, :, j] * until[:, :, j]).transpose(2, 3) @ u
    s["state"][s["dst"].long()] = S
    out = torch.cat(out, 2)[:, :, :N]
    out = torch.where(live, out, torch.zeros((), device=dev)).transpose(1, 2)
    return {"out": out.to(s["q"].dtype).contiguous(), "state": s["state"][R:]}


def _above(parent):
    """bool [R, N, N]: [r, i, j] where j lies on the path from the root to i, i included."""
    R, N = parent.shape
    see = torch.eye(N, dtype=torch.bool, device=parent.device).repeat(R, 1, 1)
    p = parent.long()
    up = torch.arange(N, device=parent.device).expand(R, N)
    for _ in range(16):
        up = torch.where(up >= 0, torch.gather(p, 1, up.clamp_min(0)), up)
        see |= (torch.arange(N, device=parent.device) == up[..., None])
    return see


def _plain_tree(s):
    c = s["case"]
    N, Hv = c["N"], c["Hv"]
    dev = s["q"].device
    zero = torch.zeros((), device=dev)
    see = _above(s["parent"])[:, None]
    q, k = (_unit(_rows(s, s[n], Hv), c) for n in ("q", "k"))
    beta = s["beta"].transpose(1, 2)[..., None]
    g = s["g"].double().transpose(1, 2)
    total = see.double() @ g[..., None]  # along each node's path
    decay = torch.where(see, total - total.transpose(2, 3), -math.inf).float().exp()
    strict = see & ~torch.eye(N, dtype=torch.bool, device=dev)
    A = torch.where(strict, beta * decay * (k @ k.transpose(2, 3)), zero)
    S, since = _first(s), total.float().exp()
    first = beta * (_rows(s, s["v"], Hv) - since * (k @ S))
    u = first
    for _ in range(15):  # a node's update is right after as many steps as it has nodes above it
        u = first - A @ u
    out = s["scale"] * since * (q @ S) + (s["scale"] * decay * (q @ k.transpose(2, 3))) @ u
    live = (torch.arange(N, device=dev) < s["nodes"].long()[:, None])[:, None, :, None]
    out = torch.where(live, out, zero).transpose(1, 2)
    return {"out": out.to(s["q"].dtype).contiguous()}


def _plain_commit(s):
    R = s["case"]["n_req"]
    r = torch.arange(R, device=s["k"].device)
    S = _first(s)
    for j in range(s["path"].shape[1]):
        on = (j <= s["accept"].long())[:, None, None, None]
        S = torch.where(on, _step(s, S, r, s["path"][:, j].long().clamp_min(0)), S)
    s["state"][s["dst"].long()] = S
    return {"state": s["state"][R:]}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    if c["kind"] == "gated":
        n = c["T"] * c["heads"] * c["D"]
        return {"bytes": float(3 * 2 * n + 2 * c["D"]), "flops": 10.0 * n}
    if c["kind"] == "block":
        n = c["T"] * c["H"]
        tensors = 3 + (1 if c["pre"] else 0) + (1 if c["gate"] == "rows" else 0)
        return {"bytes": float(2 * n * tensors + 2 * c["H"] * (c["post"] + c["pre"] + (c["gate"] == "one"))), "flops": 12.0 * n}
    Hk, Hv, Dk, Dv = (c[n] for n in ("Hk", "Hv", "Dk", "Dv"))
    fresh = sum(1 for r in range(c["n_req"]) if r % 4 == 3) if c["N"] > 1 else 0
    state = Hv * Dk * Dv * 4
    rows = float(lens(c).sum())
    if c["kind"] == "commit":
        rows = min(rows, 6.0 * c["n_req"])  # about six accepted rows a request
        byts = rows * ((Hk * Dk + Hv * Dv) * 2 + 8 * Hv) + state * (2 * c["n_req"] - fresh)
        return {"bytes": byts, "flops": 4.0 * rows * Hv * Dk * Dv}
    byts = rows * ((2 * Hk * Dk + Hv * Dv) * 2 + 8 * Hv) + c["n_req"] * c["N"] * Hv * Dv * 2.0
    byts += state * (c["n_req"] * (2 if c["kind"] == "rule" else 1) - fresh)
    return {"bytes": float(byts), "flops": 6.0 * rows * Hv * Dk * Dv}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Row by row, node by node: S' = e^g S, u = beta (v - S'^T k), S = S' + k u^T, o = scale S^T q."""
    c = case
    s = prepare(c, seed)
    f64 = torch.float64

    def gate(x):
        sig = 1.0 / (1.0 + torch.exp(-x.to(f64)))
        return {"none": x.to(f64), "sigmoid": sig, "silu": x.to(f64) * sig}[c["act"]]

    def rms(x, w):
        return x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + EPS) * w.to(f64)

    if c["kind"] == "gated":
        return {"out": rms(s["x"].to(f64), s["w"]) * gate(s["gate"])}
    if c["kind"] == "block":
        y = s["y"].to(f64)
        y = rms(y, s["w_post"]) if c["post"] else y
        y = y * gate(s["gate"]) if c["gate"] else y
        r = s["residual"].to(f64) + s["scale"] * y
        return {"residual": r} | ({"x": rms(r, s["w_pre"])} if c["pre"] else {})

    R, N, Hk, Hv, Dk, Dv = (c[n] for n in ("n_req", "N", "Hk", "Hv", "Dk", "Dv"))
    n, src, dst = lens(c), s["src"].tolist(), s["dst"].tolist()

    def vectors(x, r):
        """Rows of request r for every value head, of length one where the case normalises."""
        x = x[r].to(f64)
        if c["normalize"]:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)
        return x[:, torch.arange(Hv, device=x.device) * Hk // Hv]

    def step(S, k, v, g, beta):
        S = S * torch.exp(g.to(f64))[:, None, None]
        u = beta.to(f64)[:, None] * (v.to(f64) - torch.einsum("hkv,hk->hv", S, k))
        return S + k[:, :, None] * u[:, None, :]

    out = torch.zeros((R, N, Hv, Dv), dtype=f64, device="cuda")
    state = torch.zeros((R, Hv, Dk, Dv), dtype=f64, device="cuda")
    if c["kind"] == "rule" and int(n.sum()) > 60000:
        return None
    for r in range(R):
        S = s["state"][src[r]].to(f64) if src[r] >= 0 else torch.zeros((Hv, Dk, Dv), dtype=f64, device="cuda")
        k, q = vectors(s["k"], r), vectors(s["q"], r)
        if c["kind"] == "commit":
            for i in s["path"][r, :int(s["accept"][r]) + 1].tolist():
                S = step(S, k[i], s["v"][r, i], s["g"][r, i], s["beta"][r, i])
            state[dst[r] - R] = S
            continue
        behind = [] if c["kind"] == "rule" else s["parent"][r].tolist()
        states = []
        for i in range(int(n[r])):
            at = S if not behind or behind[i] < 0 else states[behind[i]]
            at = step(at, k[i], s["v"][r, i], s["g"][r, i], s["beta"][r, i])
            out[r, i] = s["scale"] * torch.einsum("hkv,hk->hv", at, q[i])
            if behind:
                states.append(at)
            else:
                S = at
        state[dst[r] - R] = S
    if c["kind"] == "tree":
        return {"out": out}
    return {"state": state} if c["kind"] == "commit" else {"out": out, "state": state}
