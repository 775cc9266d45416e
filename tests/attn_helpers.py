"""Inputs and the 64-bit plain form for the paged-cache tests: element by
element from the definitions in include/mfd.h, with torch only for storage
and products."""
import math

import torch

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def two_to(e):
    """2^e in 64 bits for integer e, exact."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def quantise_rows(x, dtype):
    """E4M3 rows of x [.., D] (any float type): (values held, in 64 bits;
    byte per row).  `dtype`: the type whose range the held values stay in."""
    x = x.double()
    top = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    m, p = torch.frexp(torch.where(bad, torch.ones_like(top), top))
    e = torch.where(m <= 0.875, p - 9, p - 8).clamp_min(-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.where(bad[..., None], torch.zeros_like(x), x) * two_to(-e)[..., None]
    step = two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
    held = torch.round(y / step) * step  # torch.round: to nearest even
    over = held.abs() * two_to(e)[..., None] > torch.finfo(dtype).max
    held = torch.where(over, torch.sign(held) * 240.0, held) * two_to(e)[..., None]
    held = torch.where(bad[..., None], torch.full_like(held, math.nan), held)
    return held, torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)


def rope64(x, pos, rot, theta, interleaved):
    """Rotation in 64 bits: x [.., H, D], pos [..]."""
    x = x.double().clone()
    h = rot // 2
    if h == 0:
        return x
    f = float(theta) ** (-2.0 * torch.arange(h, dtype=torch.float64, device=x.device) / rot)
    a = pos.double()[..., None, None] * f
    c, s = a.cos(), a.sin()
    u, v = (x[..., 0:rot:2].clone(), x[..., 1:rot:2].clone()) if interleaved else (x[..., :h].clone(), x[..., h:rot].clone())
    y, z = u * c - v * s, v * c + u * s
    if interleaved:
        x[..., 0:rot:2], x[..., 1:rot:2] = y, z
    else:
        x[..., :h], x[..., h:rot] = y, z
    return x


def norm64(x, w, eps):
    x = x.double()
    return x if w is None else x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()


def fill_table(table, lens, ps, n_pages, gen):
    """Distinct random pages for lens[q] positions of each request."""
    perm = torch.randperm(n_pages, generator=gen)
    at = 0
    table.fill_(-1)  # entries no position uses are never read
    for q, n in enumerate(lens):
        k = (int(n) + ps - 1) // ps
        table[q, :k] = perm[at:at + k].to(torch.int32).to(table.device)
        at += k


def entries(cache, q, lo, hi):
    """Positions lo..hi-1 of request q in 64 bits: k, v [n, Hk, D]."""
    t = torch.arange(lo, hi, device=cache.k.device)
    page, slot = cache.block_table[q, t // cache.page_size].long(), t % cache.page_size
    out = []
    for x, e in ((cache.k, cache.k_exp), (cache.v, cache.v_exp)):
        if e is None:
            y = x[page, :, slot].double()
        else:
            y = x.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float().double()
            code = e[page, :, slot]
            y = y * two_to(code.long() - 127)[..., None]
            y = torch.where((code == 255)[..., None], torch.full_like(y, math.nan), y)
        out.append(y)
    return out


def tree_visible(N, gen, depth=15):
    """A random tree of N nodes, parents first: bool [N, N], row i its path."""
    vis = torch.zeros((N, N), dtype=torch.bool)
    dep = [0] * N
    par = [-1] * N
    for i in range(N):
        if i:
            p = max(0, i - 1 - int(torch.randint(0, 40, (1,), generator=gen)))
            while dep[p] >= depth:
                p = par[p]
            par[i], dep[i] = p, dep[p] + 1
            vis[i] = vis[p]
        vis[i, i] = True
    return vis


def mask_words(vis):
    """bool [.., N] to int32 words [.., ceil(N / 32)]."""
    N = vis.shape[-1]
    W = (N + 31) // 32
    v = torch.zeros(vis.shape[:-1] + (W * 32,), dtype=torch.int64)
    v[..., :N] = vis.long()
    w = (v.view(vis.shape[:-1] + (W, 32)) << torch.arange(32)).sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def attention64(q, cache, ctx, nodes, visible, scale):
    """The definition, row by row of (request, head): out, lse and the error
    bound's ingredients: sum p |v| and the largest sum |q k| scale, each for
    every row.  visible: bool [n_req, N, N] or None (causal)."""
    R, N, Hq, D = q.shape
    G = Hq // cache.Hk
    dev = q.device
    out = torch.zeros((R, N, Hq, D), dtype=torch.float64, device=dev)
    lse = torch.full((R, N, Hq), -math.inf, dtype=torch.float64, device=dev)
    pv, sv = torch.zeros_like(out), torch.zeros_like(out)
    qk = torch.zeros_like(lse)
    for r in range(R):
        n, c = int(nodes[r]), int(ctx[r])
        if n == 0:
            continue
        K, V = entries(cache, r, 0, c + n)
        see = torch.ones((n, c + n), dtype=torch.bool, device=dev)
        see[:, c:] = torch.ones((n, n), dtype=torch.bool, device=dev).tril() if visible is None else visible[r, :n, :n].to(dev)
        some = see.any(-1)
        for h in range(Hq):
            k, v, x = K[:, h // G], V[:, h // G], q[r, :n, h].double()
            z = torch.where(see, (x @ torch.nan_to_num(k, 0, 0, 0).T) * scale, -math.inf)
            if not torch.isfinite(k).all():
                bad = ~torch.isfinite(k).all(-1)
                for t in bad.nonzero().flatten().tolist():
                    zt = (x * k[t]).sum(-1) * scale
                    z[:, t] = torch.where(see[:, t], zt, -math.inf)
            m = z.amax(-1, keepdim=True)
            p = torch.where(see, torch.exp(z - torch.where(some[:, None], m, 0.0)), 0.0)
            l = p.sum(-1, keepdim=True)
            w = p / torch.where(some[:, None], l, 1.0)
            vf = torch.nan_to_num(v, 0, 0, 0)
            o = w @ vf
            for t in (~torch.isfinite(v).all(-1)).nonzero().flatten().tolist():
                add = torch.where(torch.isfinite(v[t]), torch.zeros_like(v[t]), v[t])
                o = torch.where(see[:, t, None], o + add, o)
            out[r, :n, h] = torch.where(some[:, None], o, 0.0)
            lse[r, :n, h] = torch.where(some, (m + l.log()).squeeze(-1), -math.inf)
            pv[r, :n, h] = w @ vf.abs()
            sv[r, :n, h] = see.double() @ vf.abs() / torch.where(some[:, None], l, 1.0)
            qk[r, :n, h] = torch.where(see, (x.abs() @ torch.nan_to_num(k, 0, 0, 0).abs().T) * scale, 0.0).amax(-1)
    return out, lse, pv, sv, qk


def attention_bound(out, pv, sv, qk, dtype, D):
    """How far a correct kernel can be: scores are D fp32 products and sums
    (an absolute error d each, which changes a weight by a factor e^d, in the
    numerator and in the sum), exp2 and sums in fp32 (2^-18 together), each
    weight rounded to the type (half a step, and half of fp16's smallest step
    below its normal range), the result rounded to the type."""
    half = torch.finfo(dtype).eps / 2
    d = (D + 8) * 2.0 ** -23 * qk[..., None]
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return (half + 2 * d + 2.0 ** -18) * pv + tiny * (sv + 1) + half * out.abs() * (1 + 2.0 ** -6)


def lse_bound(lse, qk, D):
    return (D + 8) * 2.0 ** -23 * qk + 2.0 ** -20 * (1 + lse.abs())
