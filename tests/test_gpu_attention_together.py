"""GPU tests of the paged-cache calls as a round makes them: append, attention
and commit captured as one graph, rounds on two streams at once, and caches
whose pages start past 2^32 elements."""
import math

import pytest
import torch

import attn_helpers as ah
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu
EPS, THETA = 1e-6, 1.0e4


class Layer:
    """One layer's round: the rows' projections, a cache, what the calls write."""

    def __init__(self, R, N, Hq, Hk, D, ps, ctx, kind="bf16", seed=0, pages=None):
        g = torch.Generator("cuda").manual_seed(seed)
        gen = torch.Generator().manual_seed(seed)
        self.R, self.N, self.Hq, self.D, self.L = R, N, Hq, D, 15
        max_pages = (max(ctx) + 3 * N + ps - 1) // ps
        n_pages = R * max_pages + 1 if pages is None else pages
        self.c = mfd.KVCache(n_pages, ps, Hk, D, R, max_pages, ah.DT[kind])
        table = torch.randperm(R * max_pages, generator=gen).to(torch.int32).view(R, max_pages)
        self.c.block_table.copy_(table + (n_pages - R * max_pages))  # the storage's last pages
        used = self.c.block_table.flatten().long()
        for t, e in ((self.c.k, self.c.k_exp), (self.c.v, self.c.v_exp)):
            for p in used.split(64):
                x = torch.randn((len(p),) + t.shape[1:], device="cuda", generator=g)
                t.view(torch.uint8)[p] = x.to(t.dtype).view(torch.uint8)
                if e is not None:
                    e[p] = 126
        self.qkv = torch.randn((R, N, Hq + 2 * Hk, D), device="cuda", generator=g).to(torch.bfloat16)
        self.w = [(1 + 0.1 * torch.randn(D, device="cuda", generator=g)).to(torch.bfloat16) for _ in range(2)]
        self.q, self.k, self.v = self.qkv.split([Hq, Hk, Hk], dim=2)
        vis = torch.stack([ah.tree_visible(N, gen) for _ in range(R)])
        self.mask = ah.mask_words(vis).cuda()
        path, acc = torch.full((R, 16), -1, dtype=torch.int32), torch.zeros(R, dtype=torch.int32)
        for r in range(R):
            chain = vis[r, N - 1].nonzero().flatten()
            path[r, :len(chain)], acc[r] = chain.to(torch.int32), len(chain) - 1
        self.path, self.acc = path.cuda(), acc.cuda()
        self.ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        self.pos = (self.ctx[:, None] + vis.sum(-1).cuda() - 1).to(torch.int32)
        self.nodes = torch.full((R,), N, dtype=torch.int32, device="cuda")
        self.phase = mfd.rope_phases(THETA, D)
        self.q_out, self.out = (torch.zeros((R, N, Hq, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.lse = torch.zeros((R, N, Hq), device="cuda")
        self.st = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((mfd.mfd_tree_attention_workspace_bytes(R, N, Hq, Hk, D),), 0xA5, dtype=torch.uint8, device="cuda")

    def round(self):
        mfd.mfd_kv_append(self.q, self.k, self.v, *self.w, EPS, self.phase, self.D, False, self.pos, self.ctx, self.nodes,
                          self.q_out, self.c, self.st)
        mfd.mfd_tree_attention(self.q_out, self.c, self.ctx, self.nodes, self.mask, self.D ** -0.5, self.out, self.lse,
                               self.st, self.ws)
        mfd.mfd_kv_commit(self.c, self.ctx, self.acc, self.path, self.nodes, self.ctx, self.st)

    def state(self):
        pages = self.c.block_table.flatten().long()
        out = [self.q_out, self.out, self.ctx] + [t.view(torch.uint8)[pages] for t in (self.c.k, self.c.v)]
        out += [e[pages] for e in (self.c.k_exp, self.c.v_exp) if e is not None]
        assert int(self.st.item()) == 0
        return [x.clone() for x in out] + [self.lse.view(torch.int32).clone()]


def same(a, b):
    return all(torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x,
                           y.view(torch.int16) if y.dtype == torch.bfloat16 else y) for x, y in zip(a, b))


SHAPES = [(1, 65, 8, 2, 128, 16, [700], "bf16"), (3, 33, 8, 2, 128, 64, [500, 0, 90], "e4m3"),
          (2, 129, 8, 2, 256, 32, [300, 1000], "bf16"), (8, 9, 4, 4, 64, 16, [40 * i for i in range(8)], "e4m3")]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_a_round_as_one_graph(i):
    """Append, attention and commit captured together and replayed three
    times (each replay's context is what the one before left), against the
    same calls with a wait after each."""
    *a, kind = SHAPES[i]
    plain, made = Layer(*a, kind, seed=i), Layer(*a, kind, seed=i)
    want = []
    for _ in range(3):
        for step in (0, 1, 2):
            if step == 0:
                mfd.mfd_kv_append(plain.q, plain.k, plain.v, *plain.w, EPS, plain.phase, plain.D, False, plain.pos, plain.ctx,
                                  plain.nodes, plain.q_out, plain.c, plain.st)
            elif step == 1:
                mfd.mfd_tree_attention(plain.q_out, plain.c, plain.ctx, plain.nodes, plain.mask, plain.D ** -0.5, plain.out,
                                       plain.lse, plain.st, plain.ws)
            else:
                mfd.mfd_kv_commit(plain.c, plain.ctx, plain.acc, plain.path, plain.nodes, plain.ctx, plain.st)
            torch.cuda.synchronize()
        want.append(plain.state())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        made.round()
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert same(made.state(), w)
    again = Layer(*a, kind, seed=i)  # and queued on a stream without a wait
    for _ in range(3):
        again.round()
    torch.cuda.synchronize()
    assert same(again.state(), want[-1])


def test_two_streams_with_a_workspace_each():
    """Rounds of two shapes on two streams at once give what each gives alone."""
    shapes = [SHAPES[0], SHAPES[1]]
    want = []
    for i, (*a, kind) in enumerate(shapes):
        x = Layer(*a, kind, seed=10 + i)
        x.round()
        torch.cuda.synchronize()
        want.append(x.state())
    for _ in range(10):
        both = [Layer(*a, kind, seed=10 + i) for i, (*a, kind) in enumerate(shapes)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for x, s in zip(both, streams):
            with torch.cuda.stream(s):
                x.round()
        torch.cuda.synchronize()
        assert all(same(x.state(), w) for x, w in zip(both, want))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_past_2_to_the_32(kind):
    """The same round over pages whose elements start past 2^32 in the cache's
    storage: append, attention, commit and read give the same bits."""
    a = (2, 20, 8, 8, 128, 256, [700, 100], kind)
    small = Layer(*a, seed=20)
    big = Layer(*a, seed=20, pages=(1 << 32) // (256 * 8 * 128) + 2 * small.c.max_pages + 2)
    first = int(big.c.block_table.min())
    assert first * 256 * 8 * 128 > 1 << 32
    out = []
    for x in (small, big):
        x.round()
        L = 800
        ko, vo = (torch.empty((2, L, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mfd.mfd_kv_read(x.c, torch.zeros_like(x.ctx), x.ctx, ko, vo, x.st)
        torch.cuda.synchronize()
        out.append(x.state() + [ko.clone(), vo.clone()])
    assert bool(torch.isfinite(out[0][1].float()).all()) and not math.isnan(out[0][-1].float().sum().item())
    assert same(*out)
    del big, small, x
    torch.cuda.empty_cache()
