"""GPU tests of E4M3 rows whose keys leave fp16's range: the norm's weight and
the rotation are applied in fp32, and what is held stays inside."""
import math

import pytest
import torch

import attn_helpers as ah
from tree_verified_speculative_gb300 import mfd

pytestmark = pytest.mark.gpu


def held_rows(x, top):
    """E4M3 rows of x [.., D] in 64 bits, no held value past `top`: (values,
    bytes, how near an element comes to a border between two held values,
    relative to it)."""
    x = x.double()
    m, p = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, p - 9, p - 8)
    y = x * ah.two_to(-e)[..., None]
    step = ah.two_to(torch.frexp(y.abs().clamp_min(2.0 ** -6))[1] - 4)
    low = torch.floor(y.abs() / step)
    near = ((y.abs() / step - low - 0.5).abs() * step / y.abs().clamp_min(1e-30)).amin().item()
    held = torch.round(y / step) * step
    # every value of the grid (positive E4M3 numbers) that is inside, with the row's power
    grid = torch.arange(0, 127, device=x.device, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
    inside = grid * ah.two_to(e)[..., None] <= top
    most = torch.where(inside, grid, torch.zeros_like(grid)).amax(-1, keepdim=True)
    held = torch.sign(held) * torch.minimum(held.abs(), most)
    return held * ah.two_to(e)[..., None], (e + 127).to(torch.uint8), near


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("each", [1, 4, 16])
def test_keys_that_the_norms_weight_takes_past_fp16(each, D):
    """Rows with `each` elements of one size and zeros otherwise, their mean
    square one, times weights up to fp16's largest: the key is the weight times
    a power of two, up to 16 * 65504."""
    n = 32
    g = torch.Generator("cuda").manual_seed(D + each)
    k = torch.zeros((1, n, 1, D), device="cuda")
    for i in range(n):
        at = torch.randperm(D, device="cuda", generator=g)[:each]
        k[0, i, 0, at] = math.sqrt(D / each) * (1 - 2 * torch.randint(0, 2, (each,), device="cuda", generator=g).float())
    w = (65504 * (1 - 0.9 * torch.rand(D, device="cuda", generator=g) ** 3)).to(torch.float16)
    k = k.to(torch.float16)
    root = math.sqrt(D / each)
    exact = root == int(root)
    v = torch.randn((1, n, 1, D), device="cuda", generator=g).to(torch.float16)
    c = mfd.KVCache(2, 16, 1, D, 1, 2, torch.float8_e4m3fn)
    c.block_table.copy_(torch.tensor([[1, 0]], dtype=torch.int32))
    st, zero = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    mfd.mfd_kv_append(None, k, v, None, w, 0.0, None, 0, False, torch.zeros((1, n), dtype=torch.int32, device="cuda"), zero,
                      None, None, c, st)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    mfd.mfd_kv_read(c, zero, zero + n, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool(torch.isfinite(ko).all())
    want = ah.norm64(k, w, 0.0)
    assert want.abs().max().item() > 70000
    held, code, near = held_rows(want, 65504.0)
    if exact and near > 2.0 ** -20:  # else the fp32 key may round to the border's other side
        page, slot = c.block_table[0, torch.arange(n, device="cuda") // 16].long(), torch.arange(n, device="cuda") % 16
        assert torch.equal(c.k_exp[page, 0, slot], code[0, :, 0])
        assert torch.equal(ko.double(), held)
    # a half step of the grid, or past fp16 the largest number of the grid inside
    p = ah.two_to(code.long() - 127)[..., None]
    lim = torch.maximum(want.abs() * 2.0 ** -4, p * 2.0 ** -10) * (1 + 2.0 ** -10)
    over = want.abs() > 61440
    assert bool(((ko.double() - want).abs() <= lim)[~over].all())
    assert bool((ko.double()[over] == (torch.sign(want) * 61440)[over]).all())
    assert int(over.sum()) > 0


def test_values_keep_their_row_at_fp16s_largest():
    """Values are fp16 as they come: 65504 is held as 61440, as before."""
    D = 64
    x = torch.full((1, 1, 1, D), 65504.0, dtype=torch.float16, device="cuda")
    c = mfd.KVCache(1, 16, 1, D, 1, 1, torch.float8_e4m3fn)
    st, zero = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    mfd.mfd_kv_append(None, x, x, None, None, 0.0, None, 0, False, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), zero,
                      None, None, c, st)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    mfd.mfd_kv_read(c, zero, zero + 1, ko, vo, st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((ko == 61440).all()) and bool((vo == 61440).all())
    assert int(c.v_exp[0, 0, 0]) == 135
