"""The operators between blocks at the ends of their ranges: no points at all, deviations whose squares
pass float32's range, long sums of like terms, and more work items than a launch has work-groups.

References and bounds are those of test_gpu_between_ops: U = 2^-24 is float32's unit roundoff, and the
bounds count it.  A float32 chain of n like terms may be off by n / 3 U, so that sums within 128 U (weights'
gradients) and 32 U (means) of the magnitudes that they add are sums of short chains.
"""
import math

import pytest
import torch

from tests.gpu_helpers import announce
from tests.test_gpu_between_ops import (ACTS, EPS, TYPES, U, _act64, _both, _case, _close, _factor, _gen,
                                        _L, _randn, _Ref, _split)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("last", [False, True])
def test_statistics_without_points(last):
    """Entries without points: their statistics are written, as zeros."""
    L = _L()
    announce("group_norm without points", last)
    x = torch.empty((3, 0, 6) if last else (3, 6, 0), device="cuda")
    stats = torch.full((2, 3, 2), math.nan, device="cuda")
    y, got = L.group_norm_fwd(x, 2, channels_last=last, stats=stats)
    assert got is stats and y.shape == x.shape
    assert torch.equal(stats, torch.zeros_like(stats))
    many = torch.empty((70_001, 0, 12) if last else (70_001, 12, 0), device="cuda")
    out = torch.full((2 * 70_001 * 12 + 1,), 7.0, device="cuda")
    L.group_norm_fwd(many, 12, channels_last=last, stats=out[:-1].view(2, 70_001, 12))
    assert not out[:-1].any() and float(out[-1]) == 7.0
    L.group_norm_fwd(many[:0], 12, channels_last=last, stats=out[:0].view(2, 0, 12))
