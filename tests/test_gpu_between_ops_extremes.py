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
from tests.test_gpu_between_ops import (EPS, TYPES, U, _act64, _both, _case, _close, _factor, _gen,
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


# (last, channels, groups, grid, batch): rows, groups in 64, 256 and 1024 threads, two passes with several
# planes to a strip and several strips to a plane, channels last with and without whole vectors
FAR = [(False, 4096, 2, (), 5), (False, 8192, 1, (), 3), (False, 20_000, 1, (), 2), (False, 24, 1, (40,), 3),
       (False, 8, 2, (2048,), 3), (False, 8, 1, (4095,), 2), (False, 20, 1, (3000,), 2),
       (False, 2, 1, (70_001,), 2), (False, 300, 1, (3,), 2), (True, 64, 8, (777,), 2),
       (True, 45, 9, (1300,), 2), (True, 4, 4, (9001,), 1), (True, 1, 1, (5003,), 2),
       (True, 128, 1, (20_000,), 1)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("case", FAR, ids=str)
def test_deviations_whose_squares_pass_the_range(case, dtype):
    """A few elements 2.5e19 and more from the rest: their squares, 6e38 and more, are beyond float32, the
    variance, a share of 1 / m of their sum, is not."""
    L = _L()
    last, channels, groups, grid, batch = case
    announce("group_norm far elements", case, dtype)
    x, gamma, beta, gy = _case(FAR.index(case), channels, groups, grid, dtype, last, batch)
    flat = x.view(-1)
    m = math.prod(grid) * channels // groups
    for k, value in ((0, 2.5e19), (flat.numel() // 2, -3e19), (flat.numel() - 1, 2e19)):
        flat[k] = value
    ref = _Ref(x, groups, gamma, beta, None, last, None)
    assert m >= 300 and bool(torch.isfinite(ref.rstd.float()).all()) and float(ref.rstd.min()) > 1e-19
    _, stats, _ = _both(L, x, groups, gamma, beta, gy, None, last, None)
    assert float(stats[1].min()) > 1e-19
    # non-finite ones still are: the other groups keep their bits
    y0, s0 = L.group_norm_fwd(x, groups, gamma, beta, channels_last=last)
    for value in (math.inf, math.nan):
        bad = x.clone()
        bad.view(-1)[0] = value
        y, s = L.group_norm_fwd(bad, groups, gamma, beta, channels_last=last)
        own = torch.zeros_like(s0[0], dtype=torch.bool)
        own[0, 0] = True
        assert bool(s[1][own].isnan().all()) and torch.equal(s[:, ~own], s0[:, ~own])


# [batch, points, channels], groups, channels last: groups of one or few channels, whose statistics are
# joined from many parts
NARROW = [((1, 1 << 20, 1), 1), ((1, 1 << 18, 2), 2), ((2, 65_536, 4), 4), ((1, 65_536, 8), 8),
          ((2, 16_384, 16), 16), ((1, 300_001, 3), 3), ((1, 70_003, 6), 6), ((3, 30_011, 12), 6)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16], ids=str)
@pytest.mark.parametrize("shape,groups", NARROW, ids=str)
def test_narrow_groups_of_many_points(shape, groups, dtype):
    """Means far from zero and gradients of one sign, joined from hundreds of parts."""
    L = _L()
    announce("group_norm narrow", shape, groups, dtype)
    g = _gen(sum(shape))
    gamma, beta = 1 + 0.3 * _randn(g, shape[2]), 0.3 * _randn(g, shape[2])
    for mean, up in ((1700.7, 1.7), (901.3, 0.9), (1.1, 1.1)):
        x = (mean + _randn(g, *shape)).to(dtype)
        gy = torch.full(shape, up, device="cuda").to(dtype)
        _both(L, x, groups, gamma, beta, gy, None, True, None)
        y, stats, _ = _both(L, torch.full_like(x, mean), groups, gamma, beta, gy, None, True, None)


# (last, channels, groups, grid, batch, dtype): many entries, or long runs of points, to a channel
MANY = [(True, 64, 8, (4,), 65_536, 0), (True, 8, 2, (2,), 300_000, 0), (True, 6, 3, (3,), 40_000, 0),
        (True, 1, 1, (2,), 1 << 21, 0), (False, 8, 4, (2,), 300_000, 0), (False, 20, 5, (6,), 90_001, 0),
        (False, 2, 1, (12_000,), 3000, 0), (False, 4, 1, (), 1 << 25, 0), (False, 20, 4, (), 1 << 22, 0),
        (False, 1030, 1, (3,), 4100, 0), (True, 8, 2, (2,), 300_000, 1), (False, 8, 4, (2,), 300_000, 2),
        (False, 1, 1, (1 << 22,), 100, 0), (True, 4, 1, (1 << 18,), 800, 0)]


@pytest.mark.parametrize("up", [1.1, 0.9])
@pytest.mark.parametrize("case", MANY, ids=str)
def test_weight_gradients_of_many_rows(case, up):
    """Gradients of one sign and one size, over as many rows as a batch has: float32's rounding errors
    then add up in one direction."""
    L = _L()
    last, channels, groups, grid, batch, kind = case
    dtype = TYPES[kind]
    announce("group_norm many rows", case, up)
    g = _gen(batch + channels)
    shape = (batch,) + grid + (channels,) if last else (batch, channels) + grid
    x = torch.empty(shape, dtype=dtype, device="cuda")
    step = max(1, (1 << 24) // math.prod(shape[1:]))
    for at in range(0, batch, step):
        x[at:at + step] = _randn(g, *x[at:at + step].shape)
    gamma, beta = 1 + 0.3 * _randn(g, channels), 0.3 * _randn(g, channels)
    gy = torch.full(shape, up, device="cuda").to(dtype)
    _, stats = L.group_norm_fwd(x, groups, gamma, beta, None, EPS, last)
    got = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, None, last, want=("gamma", "beta"))
    both = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, None, last)
    assert torch.equal(both["gamma"], got["gamma"]) and torch.equal(both["beta"], got["beta"])
    sums = [0, 0, 0, 0]
    for at in range(0, batch, step):
        part = slice(at, at + step)
        ref = _Ref(x[part], groups, gamma, beta, None, last, None)
        if at == 0 or at + step >= batch:
            ref.check_bwd(gy[part], {"x": both["x"][part], "gamma": None, "beta": None})
        v = _split(gy[part], groups, last)
        for i, t in enumerate((v * ref.h, 128 * U * v * (ref.h.abs() + ref.kappa) + 2 * U * v * ref.h.abs(),
                               v, 130 * U * v)):
            sums[i] = sums[i] + t.sum((0, 3)).view(-1)
    _close("grad_gamma", got["gamma"], sums[0], sums[1])
    _close("grad_beta", got["beta"], sums[2], sums[3])


@pytest.mark.parametrize("case", [(False, 4, 1, (), 1 << 26, 1), (False, 4096, 32, (), 200_000, 1)], ids=str)
def test_weight_gradients_of_many_tokens(case):
    """More partial rows of tokens than are added up at a time."""
    test_weight_gradients_of_many_rows(case, 1.1)


# (last, channels, groups, grid, batch): more than 2^20 work items in one pass or both, of work-groups of
# 64, 256 and 1024 threads, of two passes with several planes to a strip, and channels last
LOOPS = [(False, 8, 4, (2,), 300_001), (False, 128, 1, (3,), (1 << 20) + 3), (False, 300, 1, (3,), (1 << 20) + 3),
         (False, 1030, 1, (3,), 215_000), (True, 4, 2, (2,), (1 << 20) + 5), (True, 6, 3, (3,), (1 << 20) + 5),
         (True, 8, 2, (2,), (1 << 20) + 5), (True, 3, 1, (2,), (1 << 20) + 5)]


@pytest.mark.parametrize("act,mask", [(None, None), ("silu", (0.3, 5, 1))], ids=["plain", "silu-dropout"])
@pytest.mark.parametrize("case", LOOPS, ids=str)
def test_more_work_items_than_work_groups(case, act, mask):
    """Work-groups that go on to a second item, with the shared memory of the first."""
    L = _L()
    last, channels, groups, grid, batch = case
    dtype = torch.float32 if channels < 100 else torch.bfloat16
    announce("group_norm loops", case, act, mask)
    g = _gen(batch + channels)
    shape = (batch,) + grid + (channels,) if last else (batch, channels) + grid
    n = math.prod(shape[1:])
    x, gy = (torch.empty(shape, dtype=dtype, device="cuda") for _ in range(2))
    step = max(1, (1 << 25) // n)
    for at in range(0, batch, step):
        x[at:at + step] = 0.7 + _randn(g, *x[at:at + step].shape)
        gy[at:at + step] = 0.5 + _randn(g, *x[at:at + step].shape)
    gamma, beta = 1 + 0.3 * _randn(g, channels), 0.3 * _randn(g, channels)
    drop = None if mask is None else L.Dropout(*mask)
    y, stats = L.group_norm_fwd(x, groups, gamma, beta, act, EPS, last, drop)
    got = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, act, last, drop)
    sums = {}
    for at in range(0, batch, step):
        part = slice(at, at + step)
        f = None if mask is None else _factor(x[part].shape, *mask, first=at * n)
        ref = _Ref(x[part], groups, gamma, beta, act, last, f)
        ref.check_fwd(y[part], stats[:, part])
        ref.check_bwd(gy[part], {"x": got["x"][part], "gamma": None, "beta": None})
        up = _split(gy[part], groups, last) * ref.f
        v = up * _act64(ref.u, act)[1]
        off = 2 * U * v.abs() if act is None else up.abs() * (16 * U + 1.2 * ref.off)
        for k, t, o in (("gamma", v * ref.h, 128 * U * v.abs() * (ref.h.abs() + ref.kappa)
                         + off * ref.h.abs()), ("beta", v, 128 * U * v.abs() + off)):
            s = sums.setdefault(k, [0, 0])
            s[0] = s[0] + t.sum((0, 3)).view(-1)
            s[1] = s[1] + o.sum((0, 3)).view(-1)
    for k, (t, o) in sums.items():
        _close("grad_" + k, got[k], t, o)


def test_more_strips_than_work_groups():
    """Planes of a strip and a little more, as many as make over 2^20 work items of each pass.  The entries
    are one entry in memory, so that all their outputs are the same bits."""
    L = _L()
    announce("group_norm loops of strips")
    g = _gen(77)
    for channels, batch in ((9, 116_600), (5, 104_900)):
        x = (_randn(g, 1, channels, 4100) + 0.7).expand(batch, -1, -1)
        gy = (_randn(g, 1, channels, 4100) + 0.5).expand(batch, -1, -1)
        gamma, beta = 1 + 0.3 * _randn(g, channels), 0.3 * _randn(g, channels)
        y, stats = L.group_norm_fwd(x, 1, gamma, beta, "gelu")
        ref = _Ref(x[:1], 1, gamma, beta, "gelu", False, None)
        ref.check_fwd(y[:1], stats[:, :1])
        assert bool((stats == stats[:, :1]).all())
        assert all(bool((y[at:at + 4096] == y[:1]).all()) for at in range(0, batch, 4096))
        got = L.group_norm_bwd(x, 1, gamma, beta, stats, gy, "gelu", out={"x": y})
        ref.check_bwd(gy[:1], {"x": got["x"][:1], "gamma": None, "beta": None})
        assert all(bool((y[at:at + 4096] == y[:1]).all()) for at in range(0, batch, 4096))
        del y, got
