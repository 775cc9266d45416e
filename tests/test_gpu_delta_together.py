"""GPU tests of the recurrent layers' calls as a serving loop makes them: with
the round's own trees and walks, as one graph, on two streams, over states far
into their storage, and in a decoding loop."""
import os
import sys

import numpy as np
import pytest
import torch

from delta_helpers import EPS, Rows, i32, random_tree
from tree_verified_speculative_gb300 import mfd

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu


def test_rounds_with_the_library_s_trees_and_walks():
    """A prompt, then three rounds: mfd_build_tree's tree through the layer,
    mfd_verify's path committed; each round against the 64-bit rule from the
    state that the last one should have left."""
    R, K, L, topk, B, V = 3, 4, 7, 8, 63, 512
    N = B + 1
    rng = np.random.default_rng(3)
    rd = mfd.Round(R, K, L, topk, B, V)
    prompt = Rows(R, 150, 2, 4, 128, 128, seed=40, slots=R)
    state = prompt.state
    state.s.zero_()
    lens = [150, 64, 97]
    prompt.rule(i32(lens), i32([-1] * R), i32([0, 1, 2]))
    want, rows = [], lens[:]
    for r in range(R):
        _, S, size = prompt.want(r, lens[r], None)
        prompt.check_state(state.s[r], S, size, lens[r])
        want.append(S)
    for step in range(3):
        x = Rows(R, N, 2, 4, 128, 128, seed=50 + step)
        x.state = state
        logits = torch.from_numpy((3 * rng.standard_normal((R * K * L, V))).astype(np.float32)).cuda()
        rd.status.zero_()
        rd.logits_topk(logits)
        rd.build_tree()
        x.tree(rd.parent, rd.n_nodes)
        target = torch.from_numpy(rng.standard_normal((R, N, V)).astype(np.float32))
        par, tok, n = rd.parent.tolist(), rd.token.cpu(), rd.n_nodes.tolist()
        for r in range(R):  # the walk follows a path some nodes deep
            node = n[r] - 1 - step
            while node > 0:
                target[r, par[r][node], tok[r, node]] += 20.0
                node = par[r][node]
        rd.verify(target.cuda(), torch.zeros(R, device="cuda"), torch.zeros(R, dtype=torch.int64, device="cuda"))
        before = state.s.clone()
        x.commit(rd.accept_len, rd.path_nodes, rd.n_nodes)
        torch.cuda.synchronize()
        assert int(rd.status.item()) == 0 and int(x.st.item()) == 0
        assert max(rd.accept_len.tolist()) >= 1
        for r in range(R):
            out, _, size = x.want(r, n[r], before[r], par[r][:n[r]])
            x.check_out(r, n[r], out, size)
            path = rd.path_nodes[r, :int(rd.accept_len[r]) + 1].tolist()
            _, S, size = x.want(r, len(path), want[r], rows=path)
            rows[r] += len(path)
            x.check_state(state.s[r], S, size, rows[r])
            want[r] = S


class Layer:
    """One recurrent layer's round: tree, gated norm, residual norm, commit."""

    def __init__(self, R, N, seed, dtype="bf16"):
        gen = torch.Generator().manual_seed(seed)
        self.x = Rows(R, N, 2, 4, 128, 128, dtype, seed=seed)
        par = [random_tree(N, gen, back=12) for _ in range(R)]
        path = torch.full((R, 17), -1, dtype=torch.int32)
        acc = []
        for r, p in enumerate(par):
            chain, j = [], N - 1
            while j >= 0:
                chain.append(j)
                j = p[j]
            path[r, :len(chain)], n = torch.tensor(chain[::-1], dtype=torch.int32), len(chain)
            acc.append(n - 1)
        self.parent, self.path, self.acc = i32(par), path.cuda(), i32(acc)
        dt = self.x.dtype
        self.z, self.w = self.x.normal(R, N, 4, 128).to(dt), (1 + 0.1 * self.x.normal(128)).to(dt)
        self.res, self.ones = self.x.normal(R, N, 512).to(dt), torch.ones(512, dtype=dt, device="cuda")
        self.normed, self.out = torch.zeros_like(self.z), torch.zeros_like(self.res)

    def round(self):
        x = self.x
        x.tree(self.parent)
        mfd.mfd_gated_norm(x.out, self.z, self.w, EPS, "silu", self.normed)
        mfd.mfd_residual_norm(self.normed.view(self.res.shape), self.res, self.ones, None, "none", 0.5, self.ones, EPS, self.res,
                              self.out)
        x.commit(self.acc, self.path)

    def prompt(self):
        self.x.rule()

    def all(self):
        assert int(self.x.st.item()) == 0
        bits = [t.view(torch.int16) for t in (self.x.out, self.normed, self.res, self.out)] + [self.x.state.s.view(torch.int32)]
        return [t.clone() for t in bits]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("R,N,dt", [(1, 65, "bf16"), (3, 129, "fp16"), (40, 20, "bf16")])
def test_a_round_as_one_graph(R, N, dt):
    """Captured once and replayed three times, each replay from the state and
    residual that the one before left: the bits of the calls made one by one,
    with a wait after each and without."""
    a, b, c = (Layer(R, N, 60, dt) for _ in range(3))
    want = []
    for _ in range(3):
        a.prompt()
        torch.cuda.synchronize()
        a.round()
        torch.cuda.synchronize()
        want.append(a.all())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b.prompt()
        b.round()
    for w in want:
        graph.replay()
        torch.cuda.synchronize()
        assert same(b.all(), w)
    for _ in range(3):
        c.prompt()
        c.round()
    torch.cuda.synchronize()
    assert same(c.all(), want[-1])


def test_two_streams_at_once():
    shapes = [(2, 129, 70), (5, 40, 71)]
    want = []
    for R, N, seed in shapes:
        x = Layer(R, N, seed)
        x.prompt()
        x.round()
        torch.cuda.synchronize()
        want.append(x.all())
    for _ in range(5):
        both, streams = [Layer(*s) for s in shapes], [torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for x, s in zip(both, streams):
            with torch.cuda.stream(s):
                x.prompt()
                x.round()
        torch.cuda.synchronize()
        assert all(same(x.all(), w) for x, w in zip(both, want))


def test_a_stream_given_by_hand():
    x, y = Rows(2, 70, 1, 2, 64, 64, seed=72), Rows(2, 70, 1, 2, 64, 64, seed=72)
    x.rule(None, i32([0, 1]), i32([2, 3]))
    s, src, dst = torch.cuda.Stream(), i32([0, 1]), i32([2, 3])
    torch.cuda.synchronize()
    mfd.mfd_delta_rule(y.q, y.k, y.v, y.g, y.beta, y.eps, y.scale, None, y.out, y.state, src, dst, y.st, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(x.out, y.out) and torch.equal(x.state.s, y.state.s)


@pytest.mark.parametrize("N", [1, 80])
def test_states_past_2_to_the_32_elements(N):
    """Slots whose elements start past 2^32: all three forms give the bits that
    they give near the start."""
    slots = (1 << 32) // (8 * 128 * 128) + 4
    gen = torch.Generator().manual_seed(1)
    outs = []
    par, path = [random_tree(N, gen)], torch.zeros((1, 17), dtype=torch.int32, device="cuda")
    big = torch.empty((slots, 8, 128, 128), dtype=torch.float32, device="cuda")
    for far in (False, True):
        x = Rows(1, N, 2, 8, 128, 128, seed=73, slots=3)
        first = slots - 3 if far else 0
        if far:
            big[first:] = x.state.s
            x.state = mfd.DeltaState.from_tensor(big)
        x.rule(None, i32([first]), i32([first + 1]))
        out = x.out.clone()
        x.tree(i32(par), None, i32([first + 1]))
        x.commit(i32([0]), path, None, i32([first + 1]), i32([first + 2]))
        torch.cuda.synchronize()
        assert int(x.st.item()) == 0
        outs.append([out, x.out.clone(), x.state.s[first:first + 3].clone()])
    assert same(*outs)
    del big, x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("R,N", [(700, 1), (700, 20), (600, 66)])
def test_many_requests(R, N):
    x = Rows(R, N, 1, 1, 64, 64, seed=74)
    before = x.state.s.clone()
    live = [1 + (r * 37) % N for r in range(R)]
    x.rule(i32(live), None, i32([R + r for r in range(R)]))
    torch.cuda.synchronize()
    assert int(x.st.item()) == 0
    for r in list(range(0, R, 61)) + [R - 1]:
        out, S, size = x.want(r, live[r], before[r])
        x.check_out(r, live[r], out, size)
        x.check_state(x.state.s[R + r], S, size, live[r])


def test_a_long_prompt():
    """5,000 rows, two of the heads without any decay."""
    x = Rows(1, 5000, 1, 3, 64, 128, seed=75)
    x.g[:, :, 1:] = 0
    before = x.state.s.clone()
    x.rule(None, i32([0]), i32([1]))
    torch.cuda.synchronize()
    out, S, size = x.want(0, 5000, before[0])
    x.check_out(0, 5000, out, size)
    x.check_state(x.state.s[1], S, size, 5000)


def test_results_do_not_change_from_run_to_run():
    gen = torch.Generator().manual_seed(4)
    par = [random_tree(129, gen, back=9) for _ in range(6)]
    outs = []
    for _ in range(4):
        x = Rows(6, 129, 2, 4, 128, 128, seed=76)
        x.rule(None, None, i32([6, 7, 8, 9, 10, 11]))
        a = x.out.clone()
        x.tree(i32(par), None, i32([6, 7, 8, 9, 10, 11]))
        torch.cuda.synchronize()
        outs.append([a, x.out.clone(), x.state.s.clone()])
    assert all(same(o, outs[0]) for o in outs[1:])


def test_trees_decode_a_hybrid_target_s_greedy_tokens():
    """Attention and recurrent layers in turn: the tokens are those of one token
    at a time but for near ties (a tree's sums are grouped otherwise, and each
    layer's activations are rounded to bf16)."""
    import tree_decode as td

    tree, one, rounds, _ = td.main(["--hybrid", "--tokens", "48"])
    assert rounds <= 30
    assert (tree == one[:, :48]).float().mean().item() > 0.9
