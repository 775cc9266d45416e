"""Attention while another stream keeps the GPU's memory busy: warps of a CTA are then held up against
one another.  No wait runs out and the bits do not change."""
import pytest
import torch

import test_gpu_attention as base
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu

CASES = [
    # R, N, Hq, Hk, D, ps, ctx, nodes, dtype, cache, layout, mask
    (22, 1, 28, 4, 64, 16, [7678 - 200 * i for i in range(22)], [1] * 22, "bf16", "e4m3", "head", "causal"),
    (16, 1, 32, 8, 128, 32, [5000 - 170 * i for i in range(16)], [1] * 16, "bf16", "e4m3", "head", "causal"),
    (3, 65, 16, 4, 256, 16, [900, 2500, 1700], [65, 65, 40], "fp16", "e4m3", "head", "tree"),
    (3, 129, 16, 4, 64, 16, [900, 2500, 1700], [129, 129, 77], "bf16", "e4m3", "head", "tree"),
    (3, 129, 16, 4, 128, 16, [900, 2500, 1700], [129, 129, 77], "bf16", "same", "head", "tree"),
    (2, 257, 16, 4, 256, 16, [900, 2500], [257, 200], "bf16", "same", "head", "tree"),
    (5, 1, 16, 4, 256, 16, [4000, 2500, 17, 3000, 900], [1] * 5, "bf16", "same", "head", "causal"),
    (8, 3, 12, 2, 64, 16, [4000, 2500, 17, 3000, 900, 5, 700, 1800], [3] * 8, "fp16", "same", "token", "tree"),
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_under_load(i):
    s = base.make(*CASES[i], seed=40 + i)
    R, N, Hq, D = s["q"].shape
    out, lse, st = base.call(s)
    assert st == 0
    base.check(s, out, lse)
    side = torch.cuda.Stream()
    x, y = torch.ones(1 << 26, device="cuda"), torch.empty(1 << 26, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(mfd.mfd_tree_attention_workspace_bytes(R, N, Hq, s["cache"].Hk, D), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(out) for _ in range(40)]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):
            y.copy_(x)
    for o in outs:
        mfd.mfd_tree_attention(s["q"], s["cache"], s["ctx"], s["nodes"], s["words"], s["scale"], o, None, status, ws)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for o in outs:
        assert torch.equal(o.view(torch.int16), out.view(torch.int16))
