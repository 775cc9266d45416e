"""Greedy decoding of a small random target with drafted trees, on one GPU.

One round, as a serving loop runs it: the drafter's logits become a tree
(mfd_logits_topk, mfd_build_tree); the target scores every node in one pass, in
which each layer appends the nodes' keys and values to its paged cache
(mfd_kv_append) and attends under the tree mask (mfd_tree_attention); the walk
accepts a path (mfd_verify); each layer keeps that path's entries
(mfd_kv_commit).  The prompt goes through the same two calls, causally, and so
does the one-token decoding that the result is compared with.

The drafter is a stand-in: it knows the target's continuation and gets each
position of each mode wrong with some probability.

    python examples/tree_decode.py [--cache e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
from tree_verified_speculative_gb300 import mfd  # noqa: E402

EPS, THETA = 1e-6, 1.0e4


class Target:
    """A random decoder with grouped-query attention over paged caches."""

    def __init__(self, n_req, max_len, cache_dtype, layers=2, H=256, Hq=8, Hk=2, D=64, V=1000, page_size=16, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device="cuda") / shape[-1] ** 0.5).to(torch.bfloat16)

        self.H, self.Hq, self.Hk, self.D, self.V, self.n_req = H, Hq, Hk, D, V, n_req
        self.embed, self.head = 2.0 * weight(V, H), 4.0 * weight(V, H)
        self.layers = [dict(qkv=weight((Hq + 2 * Hk) * D, H), o=weight(H, Hq * D), up=weight(4 * H, H), down=weight(H, 4 * H),
                            q_w=1 + 0.1 * weight(D), k_w=1 + 0.1 * weight(D)) for _ in range(layers)]
        pages = (max_len + page_size - 1) // page_size
        self.caches = []
        for _ in range(layers):
            c = mfd.KVCache(n_req * pages, page_size, Hk, D, n_req, pages, cache_dtype)
            c.block_table.copy_(torch.randperm(n_req * pages, generator=torch.Generator().manual_seed(seed)).view(n_req, pages))
            self.caches.append(c)
        self.phase = mfd.rope_phases(THETA, D)
        self.ctx = torch.zeros(n_req, dtype=torch.int32, device="cuda")
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = {}

    def forward(self, tokens, pos, n_nodes=None, mask=None):
        """Logits [n_req, N, V] of N rows per request behind the context."""
        R, N = tokens.shape
        if N not in self.ws:
            n = mfd.mfd_tree_attention_workspace_bytes(R, N, self.Hq, self.Hk, self.D)
            self.ws[N] = torch.empty(n, dtype=torch.uint8, device="cuda")
        x = self.embed[tokens.clamp_min(0).long()]
        for w, cache in zip(self.layers, self.caches):
            qkv = (_norm(x) @ w["qkv"].T).view(R, N, self.Hq + 2 * self.Hk, self.D)
            q, k, v = qkv.split([self.Hq, self.Hk, self.Hk], dim=2)
            q_out = torch.empty((R, N, self.Hq, self.D), dtype=x.dtype, device="cuda")
            mfd.mfd_kv_append(q, k, v, w["q_w"], w["k_w"], EPS, self.phase, self.D, False, pos, self.ctx, n_nodes, q_out,
                              cache, self.status)
            o = torch.empty_like(q_out)
            mfd.mfd_tree_attention(q_out, cache, self.ctx, n_nodes, mask, self.D ** -0.5, o, None, self.status, self.ws[N])
            x = x + o.view(R, N, -1) @ w["o"].T
            x = x + torch.relu(_norm(x) @ w["up"].T) @ w["down"].T
        return _norm(x).float() @ self.head.float().T

    def keep(self, accept_len, path_nodes, n_nodes):
        """Keeps the accepted path in every layer and moves the context's end."""
        new = torch.empty_like(self.ctx)
        for cache in self.caches:
            mfd.mfd_kv_commit(cache, self.ctx, accept_len, path_nodes, n_nodes, new, self.status)
        self.ctx = new

    def prompt(self, tokens):
        """All but the last token into the cache; the last is the first anchor."""
        n = tokens.shape[1] - 1
        pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(self.n_req, n).contiguous()
        self.forward(tokens[:, :n], pos)
        self.ctx += n
        return tokens[:, n].to(torch.int32)


def _norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS)).to(x.dtype)


def decode_one_by_one(target, prompt, n):
    """Greedy tokens [n_req, n], one per pass."""
    token, out = target.prompt(prompt), []
    for _ in range(n):
        logits = target.forward(token[:, None], target.ctx[:, None].contiguous())
        target.ctx = target.ctx + 1
        token = logits[:, 0].argmax(-1).to(torch.int32)
        out.append(token)
    return torch.stack(out, 1)


def decode_trees(target, prompt, n, future, K=4, L=7, topk=8, B=31, wrong=0.25, seed=1):
    """Greedy tokens [n_req, n], a tree per pass, and the number of passes.
    future [n_req, >= n + L]: what the stand-in drafter draws on."""
    R, V = target.n_req, target.V
    g = torch.Generator("cuda").manual_seed(seed)
    rd = mfd.Round(R, K, L, topk, B, V)
    rd.anchor.copy_(target.prompt(prompt))
    temperature, seeds = torch.zeros(R, device="cuda"), torch.zeros(R, dtype=torch.int64, device="cuda")
    out, rounds = [[] for _ in range(R)], 0
    while min(len(o) for o in out) < n:
        draft = torch.randn((R, K, L, V), generator=g, device="cuda")
        at = torch.tensor([len(o) for o in out], device="cuda")[:, None] + torch.arange(L, device="cuda")
        want = torch.gather(future, 1, at.clamp_max(future.shape[1] - 1).long())[:, None, :].expand(R, K, L)
        miss = torch.rand((R, K, L), generator=g, device="cuda") < wrong
        want = torch.where(miss, torch.randint(0, V, (R, K, L), generator=g, device="cuda"), want.long())
        draft.scatter_add_(3, want[..., None], torch.full((R, K, L, 1), 9.0, device="cuda"))
        rd.base_pos.copy_(target.ctx)
        rd.logits_topk(draft.view(R * K * L, V))
        rd.build_tree()
        logits = target.forward(rd.token, rd.pos, rd.n_nodes, rd.mask)
        rd.verify(logits.contiguous(), temperature, seeds)
        target.keep(rd.accept_len, rd.path_nodes, rd.n_nodes)
        accept = rd.accept_len.tolist()
        tokens = rd.out_tokens.tolist()
        for r in range(R):
            out[r] += tokens[r][:accept[r] + 1]
        rd.anchor.copy_(torch.tensor([o[-1] for o in out], dtype=torch.int32))
        rounds += 1
    assert int(rd.status.item()) == 0 and int(target.status.item()) == 0
    return torch.tensor([o[:n] for o in out], device="cuda"), rounds


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--requests", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args(argv)
    dtype = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    prompt = torch.randint(0, 1000, (a.requests, 37), device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    size = prompt.shape[1] + a.tokens + 64
    one = decode_one_by_one(Target(a.requests, size, dtype), prompt, a.tokens + 8)
    tree, rounds = decode_trees(Target(a.requests, size, dtype), prompt, a.tokens, one)
    same = (tree == one[:, :a.tokens]).float().mean().item()
    print(f"{a.tokens} tokens for {a.requests} requests in {rounds} passes ({a.cache} cache); "
          f"{100 * same:.1f}% as decoded one by one")
    return tree, one, rounds, prompt


if __name__ == "__main__":
    main()
