"""GPU test of a whole decoding loop over the paged cache: trees drafted,
scored in one pass, walked and committed give the target's own greedy tokens."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_trees_decode_the_targets_greedy_tokens(cache):
    """Every token is the target's argmax given the tokens before it, as one
    causal pass over the whole sequence scores them (a third grouping of the
    same sums, so a logit may differ by its bf16 activations' rounding: two
    layers of a few roundings of 2^-8 on logits of size 16 at most)."""
    import tree_decode as td

    tree, one, rounds, prompt = td.main(["--cache", cache, "--tokens", "48"])
    assert rounds <= 30  # most rounds accept several drafted tokens
    dtype = torch.bfloat16 if cache == "bf16" else torch.float8_e4m3fn
    t = td.Target(2, 256, dtype)
    seq = torch.cat([prompt, tree], 1)
    n = seq.shape[1] - 1
    pos = torch.arange(n, dtype=torch.int32, device="cuda").expand(2, n).contiguous()
    logits = t.forward(seq[:, :n], pos)[:, prompt.shape[1] - 1:]
    got = torch.gather(logits, 2, tree[..., None].long())[..., 0]
    top = logits.amax(-1)
    assert bool((got >= top - 16 * 2 ** -5).all()), (top - got).max().item()
    assert (tree == one[:, :48]).float().mean().item() > 0.9
