"""CPU tests of what the paged-cache calls' binding refuses before any address
is taken: tensors of a type whose elements are smaller than the kernels read."""
from types import SimpleNamespace

import pytest
import torch

from tree_verified_speculative_gb300 import mfd

BF16, I32 = torch.bfloat16, torch.int32


def _call(name, phase=None, status=None):
    R, N, Hq, Hk, D = 2, 3, 4, 2, 64
    cache = SimpleNamespace(n_req=R, Hk=Hk, D=D, _c=None)
    q, k = torch.zeros((R, N, Hq, D), dtype=BF16), torch.zeros((R, N, Hk, D), dtype=BF16)
    pos, n = torch.zeros((R, N), dtype=I32), torch.zeros(R, dtype=I32)
    phase = torch.zeros(D // 2, dtype=torch.int64) if phase is None else phase
    status = torch.zeros(1, dtype=I32) if status is None else status
    if name == "norm":
        mfd.mfd_qk_norm_rope(q, k, None, None, 0.0, phase, D, False, pos, q.clone(), k.clone(), status)
    elif name == "append":
        mfd.mfd_kv_append(q, k, k, None, None, 0.0, phase, D, False, pos, n, None, q.clone(), cache, status)
    elif name == "read":
        mfd.mfd_kv_read(cache, n, n, k.clone(), k.clone(), status)
    elif name == "commit":
        mfd.mfd_kv_commit(cache, n, n, torch.zeros((R, 4), dtype=I32), n, n.clone(), status)
    else:
        mfd.mfd_tree_attention(q, cache, n, None, None, 0.1, q.clone(), None, status, torch.zeros(1))


@pytest.mark.parametrize("name", ["norm", "append"])
@pytest.mark.parametrize("phase", [torch.zeros(32, dtype=I32), torch.zeros(32), torch.zeros(64, dtype=torch.uint8),
                                   torch.zeros(31, dtype=torch.int64)])
def test_phases_of_another_type_are_refused(name, phase):
    with pytest.raises(AssertionError, match="phases"):
        _call(name, phase=phase)


@pytest.mark.parametrize("name", ["norm", "append", "read", "commit", "attend"])
@pytest.mark.parametrize("dtype", [torch.uint8, torch.int16, torch.int64, torch.float32])
def test_a_status_of_another_type_is_refused(name, dtype):
    with pytest.raises(AssertionError, match="status"):
        _call(name, status=torch.zeros(1, dtype=dtype))


@pytest.mark.parametrize("name", ["norm", "append", "read", "commit", "attend"])
def test_the_right_types_go_on_to_the_device_check(name):
    with pytest.raises(AssertionError, match="device"):
        _call(name)
