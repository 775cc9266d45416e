"""GPU tests of the cache's handle: the addresses that calls get are those of
the tensors that the handle shows."""
import pytest
import torch

from test_gpu_attention import call, check, make
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["same", "e4m3"])
def test_an_assigned_block_table_is_the_one_that_is_read(cache):
    s = make(2, 17, 4, 2, 64, 16, [100, 40], [17, 17], cache=cache, seed=71)
    c = s["cache"]
    want, wl, _ = call(s)
    # the pages somewhere else, the old table left with what it must not be read for
    shift = torch.roll(torch.arange(c.n_pages, device="cuda"), 1)
    inverse = torch.argsort(shift)
    for t in (c.k, c.v, c.k_exp, c.v_exp):
        if t is not None:
            t.view(torch.uint8).copy_(t.view(torch.uint8)[shift].clone())
    old = c.block_table
    table = torch.where(old >= 0, inverse[old.clamp_min(0).long()].int(), old)
    wider = torch.full((2, c.max_pages + 3), -1, dtype=torch.int32, device="cuda")
    wider[:, :c.max_pages] = table
    old.fill_(0)
    c.block_table = wider
    assert c.block_table is wider and c.max_pages == wider.shape[1]
    got, lse, st = call(s)
    assert st == 0
    assert torch.equal(got.view(torch.int16), want.view(torch.int16)) and torch.equal(lse, wl)
    check(s, got, lse)


def test_the_other_tensors_and_sizes_stay():
    c = mfd.KVCache(4, 16, 2, 64, 1, 4)
    k, table = c.k, c.block_table
    for name in ("k", "v", "k_exp", "v_exp", "n_pages", "Hk", "page_size", "D", "n_req", "max_pages"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    for bad in (table.long(), table[0], torch.zeros((1, 8), dtype=torch.int32, device="cuda")[:, ::2], table.cpu()):
        with pytest.raises(AssertionError):
            c.block_table = bad
    assert c.k is k and c.block_table is table and c.max_pages == 4
    c.layer = 3  # a caller's own attribute
    assert c.layer == 3
