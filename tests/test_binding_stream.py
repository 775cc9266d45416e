"""The stream that a call without one gets: torch's current one, by whatever
way this torch has to ask for it."""
from types import SimpleNamespace

import pytest
import torch

from tree_verified_speculative_gb300 import mfd


@pytest.mark.parametrize("missing", ["_raw_stream", "_raw_device"])
def test_a_torch_without_the_short_way(monkeypatch, missing):
    monkeypatch.setattr(mfd, missing, None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: SimpleNamespace(cuda_stream=1234))
    assert mfd._s(None) == 1234 and mfd._s(7) == 7


@pytest.mark.gpu
def test_the_current_stream():
    side = torch.cuda.Stream()
    assert mfd._s(None) == torch.cuda.current_stream().cuda_stream
    with torch.cuda.stream(side):
        assert mfd._s(None) == side.cuda_stream == mfd._s(side)
    assert mfd._s(None) == torch.cuda.current_stream().cuda_stream
