"""What is measured of the target's attention over a paged key-value cache, the part of a decoding
round between the tree and its verification: the tree's nodes (or a prompt's tokens, or one new
token) get their query and key norms and position rotation, their keys and values are written into
the cache's pages, they attend to the cached context and to each other under the tree mask, and the
accepted path's entries are moved to where the next round expects them.

Four kinds of case, each one call (or the calls that only make sense together):

  attend  mfd_tree_attention
  append  mfd_kv_append into a cache of the values' own type
  store   mfd_kv_append into an E4M3 cache, then mfd_kv_read of context and new tokens
  accept  mfd_kv_append, then mfd_kv_commit of the accepted path

`own` chooses between the library's calls and their plain form in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}
EPS = 1e-6
THETA = 1.0e6


def listed():
    return [
        # one user, a short chat, one token at a time: the call's latency
        dict(name="attend_one_token", kind="attend", n_req=1, N=1, Hq=32, Hk=8, D=128, ctx=700, ps=16, dtype="bf16",
             cache="bf16", causal=True),
        # one user, one token over a long document: the cache's length is what there is to split
        dict(name="attend_one_long", kind="attend", n_req=1, N=1, Hq=32, Hk=8, D=128, ctx=200001, ps=64, dtype="bf16",
             cache="bf16", causal=True),
        # a serving batch without drafts, ragged contexts, the cache held in 8 bits
        dict(name="attend_batch_e4m3", kind="attend", n_req=32, N=1, Hq=32, Hk=8, D=128, ctx=16000, ps=32,
             dtype="bf16", cache="e4m3", causal=True),
        # the default round: a 256-prefix tree over one request's context, wide heads
        dict(name="attend_tree_256", kind="attend", n_req=1, N=257, Hq=16, Hk=4, D=256, ctx=8191, ps=64, dtype="bf16",
             cache="bf16", causal=False),
        # 32 requests with 128-prefix trees, the cache held in 8 bits
        dict(name="attend_trees_batch", kind="attend", n_req=32, N=129, Hq=32, Hk=8, D=128, ctx=6000, ps=64,
             dtype="bf16", cache="e4m3", causal=False),
        # prompts, before any tree: causal, odd head grouping and width, half precision
        dict(name="attend_prompts", kind="attend", n_req=3, N=1777, Hq=28, Hk=4, D=80, ctx=333, ps=16, dtype="fp16",
             cache="fp16", causal=True),
        # a serving batch without drafts: one token each
        dict(name="append_one_each", kind="append", n_req=32, N=1, Hq=32, Hk=8, D=128, ctx=5000, ps=16, dtype="bf16",
             cache="bf16", rot=128, inter=False, norm=True),
        # prompts of a model that rotates a part of each head, packed projections
        dict(name="append_prompts", kind="append", n_req=8, N=2000, Hq=16, Hk=4, D=256, ctx=100, ps=64, dtype="fp16",
             cache="fp16", rot=64, inter=True, norm=True),
        # trees into an 8-bit cache, and a stretch of the cache handed on in full width
        dict(name="store_trees", kind="store", n_req=4, N=257, Hq=32, Hk=8, D=128, ctx=900, ps=64, dtype="bf16",
             cache="e4m3", rot=128, inter=False, norm=True),
        # prompts behind a long context, handed on (a prefill machine to a decode machine)
        dict(name="store_long", kind="store", n_req=8, N=512, Hq=16, Hk=4, D=256, ctx=12000, ps=64, dtype="bf16",
             cache="e4m3", rot=64, inter=False, norm=True),
        # one user's round: 64 prefixes in, the accepted path kept
        dict(name="accept_one", kind="accept", n_req=1, N=65, Hq=32, Hk=8, D=128, ctx=2000, ps=16, dtype="bf16",
             cache="bf16", rot=128, inter=False, norm=True),
        # 32 users' rounds with 256-prefix trees
        dict(name="accept_batch", kind="accept", n_req=32, N=257, Hq=32, Hk=8, D=128, ctx=3000, ps=32, dtype="bf16",
             cache="bf16", rot=128, inter=False, norm=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "store", "accept"])
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    Hk = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 4, 6, 7, 8])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    ps = rng.choice([16, 32, 64, 128])
    c = dict(kind=kind, Hq=Hk * G, Hk=Hk, D=D, ps=ps, dtype=dtype)
    if kind == "attend":
        c["cache"] = rng.choice([dtype, "e4m3"])
        c["n_req"] = _log_int(rng, 1, 48)
        form = rng.choice(["one", "tree", "tree", "prompt"])
        c["N"] = {"one": 1, "tree": _log_int(rng, 9, 513), "prompt": _log_int(rng, 100, 2000)}[form]
        c["causal"] = form != "tree"
        c["ctx"] = _log_int(rng, 1, 150000) if form == "one" else _log_int(rng, 1, 12000)
        # a drawn case costs no more than the largest listed ones
        while c["n_req"] > 1 and (c["n_req"] * c["ctx"] * Hk * D > 32 * 16000 * 8 * 128 or
                                  c["n_req"] * (c["ctx"] + c["N"]) * c["N"] * Hk * G * D > 32 * 6000 * 129 * 32 * 128):
            c["n_req"] //= 2
        while (c["ctx"] + c["N"]) * c["N"] * Hk * G * D > 32 * 6000 * 129 * 32 * 128:
            c["ctx"] //= 2
            c["N"] = max(1, c["N"] * 3 // 4)
        return c
    c["cache"] = "e4m3" if kind == "store" else dtype
    c["rot"] = rng.choice([D, D, D // 2 // 8 * 8])
    c["inter"] = rng.random() < 0.3
    c["norm"] = rng.random() < 0.8
    c["n_req"] = _log_int(rng, 1, 32)
    c["N"] = _log_int(rng, 1, 513) if kind != "append" else _log_int(rng, 1, 2000)
    c["ctx"] = _log_int(rng, 1, 8000)
    while c["n_req"] > 1 and c["n_req"] * (c["N"] + c["ctx"]) * (c["Hq"] + 2 * Hk) * D > 8 * 12512 * 24 * 256:
        c["n_req"] //= 2
    return c


def lens(c):
    """(context lengths, node counts) of the case's requests: ragged, from the case alone."""
    q = np.arange(c["n_req"])
    part = 1.0 - 0.6 * np.mod(q * 0.6180339887, 1.0)
    ctx = np.maximum(0, np.floor(c["ctx"] * part)).astype(np.int64)
    nodes = np.where(q % 3 == 2, np.maximum(1, (c["N"] * 7) // 8), c["N"]).astype(np.int64)
    return ctx, nodes


# ------------------------------------------------------------------ inputs
def _tree(N, rng):
    """A random tree of N nodes, parents first, at most 15 deep: (parent, depth)."""
    parent, depth = np.full(N, -1, np.int32), np.zeros(N, np.int32)
    back = rng.integers(1, 41, size=N)
    for i in range(1, N):
        p = max(0, i - int(back[i]))
        while depth[p] >= 15:
            p = parent[p]
        parent[i], depth[i] = p, depth[p] + 1
    return parent, depth


def _bits(visible):
    """uint32 words (as int32) of boolean rows [.., N]."""
    N = visible.shape[-1]
    W = (N + 31) // 32
    v = np.zeros(visible.shape[:-1] + (W * 32,), np.uint64)
    v[..., :N] = visible
    words = (v.reshape(v.shape[:-1] + (W, 32)) << np.arange(32, dtype=np.uint64)).sum(-1)
    return words.astype(np.uint32).view(np.int32)


def prepare(case, seed):
    c = case
    dev = "cuda"
    g = torch.Generator(dev).manual_seed(seed)
    rng = np.random.default_rng(seed)
    R, N, Hq, Hk, D, ps = (c[k] for k in ("n_req", "N", "Hq", "Hk", "D", "ps"))
    ctx, nodes = lens(c)
    ty = TYPES[c["dtype"]]
    e4 = c["cache"] == "e4m3"
    max_pages = int((ctx + N).max() + ps - 1) // ps
    n_pages = int(((ctx + nodes + ps - 1) // ps).sum()) + 5
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.zeros((R, max_pages), np.int32)
    at = 0
    for r in range(R):
        n = int((ctx[r] + nodes[r] + ps - 1) // ps)
        table[r, :n] = perm[at:at + n]
        at += n
    # keys and values as a model leaves them: keys with a few strong channels, values with channel offsets
    shape = (n_pages, Hk, ps, D)
    gain = torch.exp(0.4 * torch.randn((Hk, 1, D), device=dev, generator=g))
    off = 0.5 * torch.randn((Hk, 1, D), device=dev, generator=g)
    s = {"case": c, "table": torch.from_numpy(table).to(dev),
         "ctx": torch.from_numpy(ctx.astype(np.int32)).to(dev), "nodes": torch.from_numpy(nodes.astype(np.int32)).to(dev)}
    for name in ("k", "v"):
        x = torch.randn(shape, device=dev, generator=g)
        x = x * gain if name == "k" else x + off
        if e4:
            s[name], s[name + "_exp"] = _quantise(x)
        else:
            s[name], s[name + "_exp"] = x.to(ty), None
        del x
    if c["kind"] == "attend":
        s["q"] = torch.randn((R, N, Hq, D), device=dev, generator=g).to(ty)
        s["scale"] = 1.0 / math.sqrt(D)
        s["mask"] = None
        if not c["causal"]:
            vis = np.zeros((R, N, N), bool)
            for r in range(R):
                parent, _ = _tree(N, rng)
                for i in range(int(nodes[r])):
                    if i:
                        vis[r, i] = vis[r, parent[i]]
                    vis[r, i, i] = True
            s["mask"] = torch.from_numpy(_bits(vis)).to(dev)
        s["out"] = torch.empty((R, N, Hq, D), dtype=ty, device=dev)
        s["lse"] = torch.empty((R, N, Hq), dtype=torch.float32, device=dev)
    else:
        # the packed projection that queries, keys and values are cut from
        qkv = torch.randn((R, N, Hq + 2 * Hk, D), device=dev, generator=g).to(ty)
        s["q"], s["kn"], s["vn"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk], qkv[:, :, Hq + Hk:]
        for w in ("q_w", "k_w"):
            s[w] = (1.0 + 0.2 * torch.randn((D,), device=dev, generator=g)).to(ty) if c["norm"] else None
        depth = np.zeros((R, N), np.int64)
        path = np.full((R, 16), -1, np.int32)
        accept = np.zeros(R, np.int32)
        for r in range(R):
            if c["kind"] == "append":
                depth[r] = np.arange(N)
                continue
            parent, depth[r] = _tree(N, rng)
            leaf, chain = int(rng.integers(0, nodes[r])), []
            while leaf >= 0:
                chain.append(leaf)
                leaf = int(parent[leaf])
            path[r, :len(chain)] = chain[::-1]
            accept[r] = len(chain) - 1
        s["pos"] = torch.from_numpy((ctx[:, None] + depth).astype(np.int32)).to(dev)
        s["path"], s["accept"] = torch.from_numpy(path).to(dev), torch.from_numpy(accept).to(dev)
        s["q_out"] = torch.empty((R, N, Hq, D), dtype=ty, device=dev)
        s["new_len"] = torch.empty((R,), dtype=torch.int32, device=dev)
        start, length = _stretch(c)
        s["start"], s["length"] = (torch.from_numpy(x.astype(np.int32)).to(dev) for x in (start, length))
        for name in ("k_out", "v_out"):
            s[name] = torch.empty((R, int(length.max()), Hk, D), dtype=ty, device=dev) if c["kind"] == "store" else None
    s["status"] = torch.zeros((1,), dtype=torch.int32, device=dev)
    if own:  # what a program makes once, when it loads its model: the cache's handle, phases, scratch
        from tree_verified_speculative_gb300 import mfd
        s["cache"] = mfd.KVCache.from_tensors(s["k"], s["v"], s["table"], s["k_exp"], s["v_exp"])
        if c["kind"] == "attend":
            s["ws"] = torch.empty((mfd.mfd_tree_attention_workspace_bytes(R, N, Hq, Hk, D),), dtype=torch.uint8,
                                  device=dev)
        else:
            s["phase"] = mfd.rope_phases(THETA, c["rot"], device=dev)
    return s


def _stretch(c):
    """(start, length) of the positions that a store case reads back: the last part of the context and the nodes."""
    ctx, nodes = lens(c)
    start = ctx // 3
    return start, ctx + nodes - start


def _power(e):
    """2^e in 32 bits, e from -126 to 127, built from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """E4M3 values and one power of two for each row of D: the smallest 2^e >= 2^-127 with max|x| <= 448 * 2^e, held as
    e + 127."""
    f, p = torch.frexp(x.abs().amax(-1))
    e = torch.where(f <= 0.875, p - 9, p - 8).clamp_min(-127)
    e = torch.where(f == 0, torch.full_like(e, -127), e)
    q = (x * _power(-e).unsqueeze(-1)).to(torch.float8_e4m3fn)
    return q, (e + 127).to(torch.uint8)


def _values(x, exp):
    x = x.float()
    return x if exp is None else x * 0.5 * _power(exp.to(torch.int32) - 126).unsqueeze(-1)


# ------------------------------------------------------------------ one pass
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from tree_verified_speculative_gb300 import mfd
    c = s["case"]
    if c["kind"] == "attend":
        mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["mask"], s["scale"], s["out"], s["lse"],
                               s["status"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    mfd.mfd_kv_append(s["q"], s["kn"], s["vn"], s["q_w"], s["k_w"], EPS, s["phase"], c["rot"], c["inter"], s["pos"],
                      s["ctx"], s["nodes"], s["q_out"], s["cache"], s["status"])
    if c["kind"] == "store":
        mfd.mfd_kv_read(s["cache"], s["start"], s["length"], s["k_out"], s["v_out"], s["status"])
        return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
    out = {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    if c["kind"] == "accept":
        mfd.mfd_kv_commit(s["cache"], s["ctx"], s["accept"], s["path"], s["nodes"], s["new_len"], s["status"])
        out["new_len"] = s["new_len"]
    return out


def _run_plain(s):
    c = s["case"]
    return _plain_attend(s) if c["kind"] == "attend" else _plain_append(s)


def _gather(s, t):
    """Keys and values [R, T, Hk, D] in 32 bits of positions t [R, T]."""
    ps = s["case"]["ps"]
    page = torch.gather(s["table"], 1, (t // ps).clamp(0, s["table"].shape[1] - 1)).long()
    slot = t % ps
    return [_values(s[n][page, :, slot], None if s[n + "_exp"] is None else s[n + "_exp"][page, :, slot])
            for n in ("k", "v")]


def _plain_attend(s):
    c = s["case"]
    R, N, Hq, Hk, D = (c[k] for k in ("n_req", "N", "Hq", "Hk", "D"))
    G = Hq // Hk
    dev = s["q"].device
    ctx, nodes = s["ctx"].long(), s["nodes"].long()
    T = s["table"].shape[1] * c["ps"]
    t = torch.arange(T, device=dev).expand(R, T)
    k, v = _gather(s, t)
    j = t - ctx[:, None]  # the node at position t, negative in the context
    n = torch.arange(N, device=dev)
    if s["mask"] is None:
        seen = j[:, None, :] <= n[None, :, None]
    else:
        word = torch.gather(s["mask"], 2, (j.clamp(0, N - 1) // 32)[:, None, :].expand(R, N, T))
        seen = ((word >> (j.clamp(0, N - 1) % 32)[:, None, :]) & 1).bool() | (j < 0)[:, None, :]
    seen = seen & (j < nodes[:, None])[:, None, :] & (n[None, :] < nodes[:, None])[:, :, None]
    q = s["q"].float().view(R, N, Hk, G, D).permute(0, 2, 1, 3, 4).reshape(R, Hk, N * G, D)
    z = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(s["scale"]).view(R, Hk, N, G, T)
    z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = z.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    v = torch.where((j < nodes[:, None])[:, :, None, None], v, torch.zeros((), device=dev))
    o = torch.matmul(p.view(R, Hk, N * G, T), v.permute(0, 2, 1, 3)).view(R, Hk, N, G, D)
    o = o / torch.where(l == 0, torch.ones_like(l), l)
    lse = (m + l.log()).squeeze(-1)
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(R, N, Hq, D).to(s["q"].dtype),
            "lse": lse.permute(0, 2, 1, 3).reshape(R, N, Hq)}


def _plain_norm_rope(x, w, s):
    """Root-mean-square norm over each head's D, times w, then the rotation of the first `rot` elements, in 32 bits."""
    c = s["case"]
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    h = c["rot"] // 2
    i = torch.arange(h, device=x.device, dtype=torch.float64)
    turn = s["pos"].double()[:, :, None] * torch.exp(-2.0 * i / c["rot"] * math.log(THETA))
    cos, sin = turn.cos().float()[:, :, None, :], turn.sin().float()[:, :, None, :]
    if c["inter"]:
        a, b = x[..., 0:2 * h:2], x[..., 1:2 * h:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :h], x[..., h:2 * h]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * h:]], -1)


def _plain_append(s):
    c = s["case"]
    R, N = c["n_req"], c["N"]
    ps, dev, ty = c["ps"], s["q"].device, s["q"].dtype
    ctx, nodes = s["ctx"].long(), s["nodes"].long()
    n = torch.arange(N, device=dev)
    live = n[None, :] < nodes[:, None]
    q = _plain_norm_rope(s["q"], s["q_w"], s)
    q = torch.where(live[:, :, None, None], q, torch.zeros((), device=dev)).to(ty)
    k, v = _plain_norm_rope(s["kn"], s["k_w"], s)[live], s["vn"][live].float()
    t = ctx[:, None] + n
    page = torch.gather(s["table"], 1, t // ps).long()[live]
    slot = (t % ps)[live]
    for name, x in (("k", k), ("v", v)):
        if s[name + "_exp"] is None:
            s[name][page, :, slot] = x.to(ty)
        else:
            e4, exp = _quantise(x)
            s[name].view(torch.uint8)[page, :, slot] = e4.view(torch.uint8)
            s[name + "_exp"][page, :, slot] = exp
    if c["kind"] == "store":
        i = torch.arange(s["k_out"].shape[1], device=dev)
        k, v = _gather(s, s["start"].long()[:, None] + i)
        there = (i[None, :] < s["length"].long()[:, None])[:, :, None, None]
        return {"q": q, "k": torch.where(there, k, torch.zeros((), device=dev)).to(ty),
                "v": torch.where(there, v, torch.zeros((), device=dev)).to(ty)}
    out = {"q": q, "k": s["k"], "v": s["v"]}
    if c["kind"] == "accept":
        i = torch.arange(s["path"].shape[1], device=dev)
        kept = i[None, :] <= s["accept"].long()[:, None]
        src, dst = ctx[:, None] + s["path"].long().clamp_min(0), ctx[:, None] + i
        at = [(torch.gather(s["table"], 1, (x // ps).clamp(0, s["table"].shape[1] - 1)).long()[kept], (x % ps)[kept])
              for x in (src, dst)]
        for name in ("k", "v"):
            s[name][at[1][0], :, at[1][1]] = s[name][at[0][0], :, at[0][1]]
        out["new_len"] = s["ctx"] + s["accept"] + 1
    return out


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    ctx, nodes = lens(c)
    Hq, Hk, D = c["Hq"], c["Hk"], c["D"]
    held = 1 if c["cache"] == "e4m3" else 2
    entry = 2 * Hk * (D * held + (1 if held == 1 else 0))  # one position's keys and values
    new = int(nodes.sum())
    if c["kind"] == "attend":
        among = nodes * (nodes + 1) / 2 if c["causal"] else nodes * np.minimum(nodes, 8)
        pairs = float((nodes * ctx + among).sum())
        masks = 0 if c["causal"] else c["n_req"] * c["N"] * ((c["N"] + 31) // 32) * 4
        rows = c["n_req"] * c["N"] * Hq
        return {"bytes": float((ctx + nodes).sum()) * entry + new * Hq * D * 2 + rows * (D * 2 + 4) + masks,
                "flops": 4.0 * pairs * Hq * D}
    byts = new * (Hq + 2 * Hk) * D * 2 + c["n_req"] * c["N"] * Hq * D * 2 + new * (entry + 4)
    if c["kind"] == "store":
        start, length = _stretch(c)
        byts += int(length.sum()) * entry + c["n_req"] * int(length.max()) * 2 * Hk * D * 2
    if c["kind"] == "accept":
        byts += c["n_req"] * 4 * 2 * entry  # about four accepted entries, read and written
    return {"bytes": float(byts), "flops": 10.0 * new * (Hq + Hk) * D}


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    ctx, nodes = lens(c)
    N, Hq, Hk, D, ps = (c[k] for k in ("N", "Hq", "Hk", "D", "ps"))
    dev = s["q"].device

    def two_to(e):
        return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)

    def entries(name, r, t):
        """Positions t of request r, [len(t), Hk, D]."""
        flat = s["table"][r, t // ps].long() * ps + t % ps
        x = s[name].to(torch.float64) if s[name].numel() < 1 << 26 else s[name]
        x = x.transpose(1, 2).reshape(-1, Hk, D)[flat].to(torch.float64)
        if s[name + "_exp"] is not None:
            x = x * two_to(s[name + "_exp"].transpose(1, 2).reshape(-1, Hk)[flat].long() - 127)[..., None]
        return x

    if c["kind"] == "attend":
        out = torch.zeros((c["n_req"], N, Hq, D), dtype=torch.float64, device=dev)
        lse = torch.full((c["n_req"], N, Hq), -math.inf, dtype=torch.float64, device=dev)
        for r in range(c["n_req"]):
            n, T = int(nodes[r]), int(ctx[r] + nodes[r])
            t = torch.arange(T, device=dev)
            K, V = entries("k", r, t), entries("v", r, t)
            hide = torch.zeros((n, T), dtype=torch.bool, device=dev)
            i = torch.arange(n, device=dev)
            if s["mask"] is None:
                hide[:, int(ctx[r]):] = i[None, :] > i[:, None]
            else:
                hide[:, int(ctx[r]):] = (s["mask"][r, :n][:, i // 32] >> (i % 32) & 1) == 0
            for h in range(Hq):
                z = (s["q"][r, :n, h].to(torch.float64) @ K[:, h * Hk // Hq].T) * s["scale"]
                z[hide] = -math.inf
                out[r, :n, h] = torch.softmax(z, -1) @ V[:, h * Hk // Hq]
                lse[r, :n, h] = torch.logsumexp(z, -1)
        return {"out": out, "lse": lse}

    def turned(x, w):
        x = x.to(torch.float64)
        if w is not None:
            x = x / torch.sqrt(torch.mean(x * x, -1, keepdim=True) + EPS) * w.to(torch.float64)
        rot = c["rot"]
        freq = THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
        e = torch.polar(torch.ones((), dtype=torch.float64, device=dev),
                        s["pos"].to(torch.float64)[..., None, None] * freq)
        y = x.clone()
        if c["inter"]:
            z = torch.complex(x[..., 0:rot:2].contiguous(), x[..., 1:rot:2].contiguous()) * e
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * e
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    q = turned(s["q"], s["q_w"])
    for r in range(c["n_req"]):
        q[r, int(nodes[r]):] = 0
    kn, vn = turned(s["kn"], s["k_w"]), s["vn"].to(torch.float64)
    if c["kind"] == "store":
        # A key next to a border of the 8-bit grid has no one value in 32 bits of norm and rotation: keys are left to the
        # comparison with the plain form.  Values are quantised as they come.
        start, length = _stretch(c)
        v = torch.zeros(s["v_out"].shape, dtype=torch.float64, device=dev)
        for r in range(c["n_req"]):
            t = torch.arange(int(start[r]), int(ctx[r]), device=dev)
            n = int(nodes[r])
            v[r, :len(t)] = entries("v", r, t)
            x = vn[r, :n]
            top = x.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(top / 448)).clamp_min(-127)
            e = torch.where(top > 448 * two_to(e), e + 1, torch.where(top <= 448 * two_to(e - 1), e - 1, e)).clamp_min(-127)
            y = x / two_to(e)
            step = two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
            v[r, len(t):len(t) + n] = torch.round(y / step) * step * two_to(e)
        return {"q": q, "k": None, "v": v}
    k, v = s["k"].to(torch.float64), s["v"].to(torch.float64)
    path, accept = s["path"].tolist(), s["accept"].tolist()
    for name, cache, x in (("k", k, kn), ("v", v, vn)):
        for r in range(c["n_req"]):
            i = torch.arange(int(nodes[r]), device=dev)
            t = int(ctx[r]) + i
            cache[s["table"][r, t // ps].long(), :, t % ps] = x[r, :len(i)]
            if c["kind"] == "accept":
                i = torch.arange(accept[r] + 1, device=dev)
                t = int(ctx[r]) + i
                cache[s["table"][r, t // ps].long(), :, t % ps] = x[r, path[r][:accept[r] + 1]]
    out = {"q": q, "k": k, "v": v}
    if c["kind"] == "accept":
        out["new_len"] = torch.tensor([int(a) + b + 1 for a, b in zip(ctx, accept)], dtype=torch.int32, device=dev)
    return out
