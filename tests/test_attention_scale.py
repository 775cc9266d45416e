"""CPU check of mfd_tree_attention's scale: refused where scale * log2 e, which
the kernel works with, is no 32-bit number; taken up to there."""
import numpy as np
import pytest

import test_attention_args as args
from test_attention_args import lib  # noqa: F401
from tree_verified_speculative_gb300 import mfd

LOG2E = np.float32(1.4426950408889634)
TOP = np.finfo(np.float32).max


@pytest.mark.parametrize("scale", [float(TOP), 3.0e38, 2.4e38])
def test_scales_past_the_range_are_refused(lib, scale):  # noqa: F811
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(scale) * LOG2E)
    assert args.attend(lib, args.cache(), scale=scale) == mfd.MFD_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [2.3e38, 1.0, 1e-30, 1.5e-45])
def test_scales_inside_go_on(lib, scale):  # noqa: F811
    """The next check is the workspace's."""
    assert args.attend(lib, args.cache(), scale=scale, ws=None) == mfd.MFD_ERR_WORKSPACE
