"""The operators between blocks on the GPU: group norm with its activation and dropout, and dropout
by itself, forward and backward, against plain float64 formulas.

Tolerances are elementwise and follow from the arithmetic, as in test_gpu_train_ops: U = 2^-24 is
float32's unit roundoff and a half-format result adds its own, half a step.  The mask of a dropout is
compared exactly: what is dropped is 0, and nothing else is.
"""
import math

import pytest
import torch

from tests.gpu_helpers import announce

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}
TYPES = [torch.float32, torch.bfloat16, torch.float16]
ACTS = [None, "gelu", "silu"]
EPS = 1e-5
M32 = 0xffffffff


def _L():
    from fno_spectral_convolution_amd import binding
    return binding


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _close(name, got, want, bound):
    got = got.double()
    bad = (~((got - want).abs() <= bound)) & ~((got == want) | (got.isnan() & want.isnan()))
    n = int(bad.sum())
    worst = float(((got - want).abs() / bound.clamp_min(1e-300)).nan_to_num(0, 0, 0).max()) \
        if got.numel() else 0.0
    print(f"    {name}: worst error {worst:.3f} of its bound", flush=True)
    assert n == 0, f"{name}: {n} of {got.numel()} outside their bounds (worst {worst:.2f})"


def _in_range(v, dtype):
    """v with infinity where it rounds to that in half: from 65520 on, half way between the largest
    number, 65504, and 2^16."""
    return torch.where(v.abs() >= 65520, v * math.inf, v) if dtype == torch.float16 else v


# ---- the mask ----------------------------------------------------------------------------------
def _philox(block, draw, seed):
    """Words of Philox4x32-10 of the counters (block, draw): int64 tensors, values below 2^32."""
    a, b = block & M32, block >> 32
    c, d = (torch.full_like(block, v) for v in (draw & M32, draw >> 32))
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = ((q >> 32) & M32) ^ b ^ k0, q & M32, ((p >> 32) & M32) ^ d ^ k1, p & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return torch.stack([a, b, c, d], -1)


def _factor(shape, p, seed, draw, first=0, device="cuda"):
    """What dropout multiplies each element by: 0, or 65536 / (65536 - T)."""
    n, t = math.prod(shape), round(p * 65536)
    blocks = torch.arange(first // 8, (first + n + 7) // 8 + 1, dtype=torch.int64, device=device)
    w = _philox(blocks, draw, seed)
    bits = torch.stack([w & 0xffff, w >> 16], -1).reshape(-1)[first % 8:first % 8 + n]
    return torch.where(bits >= t, 65536 / (65536 - t), 0.0).double().view(shape)


MASKS = [(0.1, 7, 0), (0.5, 0x9E3779B97F4A7C15, (1 << 40) + 3), (0.25, (1 << 63) + 5, (1 << 64) - 1),
         (1 / 65536, 1, 1), (65535 / 65536, 2, 9)]


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (1, 4096), (3, 5), (1003, 37), (5, 8, 9),
                                   (2, 20, 63, 65), (70_001,), (4, 262_147)], ids=str)
@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_dropout(shape, dtype):
    L = _L()
    announce("dropout", shape, dtype)
    g = _gen(sum(shape))
    x, r = (_randn(g, *shape) + 3.0).to(dtype), _randn(g, *shape).to(dtype)
    for p, seed, draw in MASKS:
        f = _factor(shape, p, seed, draw)
        drop = L.Dropout(p, seed, draw)
        # one product with a factor that is rounded itself; with a residual one more sum
        want = x.double() * f
        y = L.dropout_fwd(x, drop)
        assert torch.equal(y == 0, f == 0)
        _close("y", y, _in_range(want, dtype),
               (2 * U + ROUND[dtype] * (1 + 4 * U)) * want.abs() + TINY[dtype])
        both = want + r.double()
        off = 2 * U * want.abs() + U * both.abs()
        _close("y + residual", L.dropout_fwd(x, drop, r), _in_range(both, dtype),
               off + ROUND[dtype] * (both.abs() + off) + TINY[dtype])
        assert torch.equal(L.dropout_bwd(x, drop), y)
    assert torch.equal(L.dropout_fwd(x, L.Dropout(0.0, 1)), x)
    assert torch.equal(L.dropout_bwd(x, L.Dropout(0.0, 1)), x)
    assert not torch.equal(L.dropout_fwd(x, L.Dropout(0.5, 1, 2)), L.dropout_fwd(x, L.Dropout(0.5, 1, 3))) \
        or x.numel() < 64


def test_dropout_share_and_independence():
    """The share that is dropped, and its correlation between neighbours, draws and seeds: sums of n
    independent bits, within six of their deviations."""
    L = _L()
    announce("dropout share")
    n = 1 << 22
    one = torch.ones(n, device="cuda")
    for p in (0.1, 0.5, 0.37):
        masks = [L.dropout_fwd(one, L.Dropout(p, s, d)) != 0
                 for s, d in ((1, 0), (1, 1), (2, 0), (1 << 32, 0), (1, 1 << 32))]
        q = round(p * 65536) / 65536
        for m in masks:
            assert abs(float((~m).double().mean()) - q) <= 6 * math.sqrt(q * (1 - q) / n)
        pairs = [(masks[0][k:], masks[0][:-k]) for k in (1, 2, 7, 8, 64)] + \
            [(masks[i], masks[j]) for i in range(5) for j in range(i)]
        for u, v in pairs:
            cov = float(((u.double() - (1 - q)) * (v.double() - (1 - q))).mean())
            assert abs(cov) <= 6 * q * (1 - q) / math.sqrt(n - 64)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
def test_dropout_strides_alignment_in_place(dtype):
    L = _L()
    announce("dropout strides", dtype)
    g = _gen(4)
    for shape in ((29, 65), (5, 7), (300, 3), (3, 4, 1031)):
        n = math.prod(shape[1:])

        def cut(off, gap, fill=77.0):
            buf = torch.full((off + shape[0] * (n + gap),), fill, dtype=dtype, device="cuda")
            return buf, buf[off:].view(shape[0], n + gap)[:, :n].unflatten(1, shape[1:])

        x0, r0 = (_randn(g, *shape) + 2).to(dtype), _randn(g, *shape).to(dtype)
        drop = L.Dropout(0.3, 99, 4)
        want, plain = L.dropout_fwd(x0, drop, r0), L.dropout_fwd(x0, drop)
        for off, gap in ((0, 0), (1, 0), (3, 5), (0, 8), (8, 1)):
            _, x = cut(off, gap)
            _, r = cut(off + 1, gap + 2)
            x.copy_(x0)
            r.copy_(r0)
            ybuf, y = cut(off + 2, gap + 3)
            L.dropout_fwd(x, drop, r, out=y)
            assert torch.equal(y, want)
            y.fill_(77.0)
            assert bool((ybuf == 77.0).all()), "written outside its entries"
            assert torch.equal(L.dropout_fwd(x, drop, r, out=r), want)
            L.dropout_bwd(x, drop, out=x)
            assert torch.equal(x, plain)
        one = x0[:1].expand(shape)  # one entry for all
        assert torch.equal(L.dropout_fwd(one, drop, one), L.dropout_fwd(one.contiguous(), drop, one.contiguous()))


def test_dropout_drops_what_is_not_finite():
    L = _L()
    announce("dropout non-finite")
    for v in (math.inf, -math.inf, math.nan):
        x = torch.full((1000,), v, device="cuda")
        f = _factor((1000,), 0.5, 3, 0)
        y = L.dropout_fwd(x, L.Dropout(0.5, 3))
        assert not y[f == 0].any() and not torch.isfinite(y[f != 0]).any()


def test_dropout_no_elements():
    L = _L()
    announce("dropout no elements")
    for shape in ((0,), (0, 5), (5, 0, 3)):
        x = torch.empty(shape, device="cuda")
        assert L.dropout_fwd(x, L.Dropout(0.5, 3), x).shape == x.shape
        assert L.dropout_bwd(x, L.Dropout(0.5, 3)).shape == x.shape


def test_dropout_offsets_past_32_bits():
    """Elements beyond 2^32, packed and in entries 2^31 elements apart."""
    L = _L()
    announce("dropout long offsets")
    n = (1 << 32) + 4101
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    y = L.dropout_fwd(x, L.Dropout(0.5, 11, 2), out=x)
    for first in (0, (1 << 31) - 2048, (1 << 32) - 2048, n - 4097):
        assert torch.equal(y[first:first + 4097].double(), _factor((4097,), 0.5, 11, 2, first))
    del x, y
    stride = (1 << 31) + 9
    buf = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    v = buf.as_strided((3, 1001), (stride, 1))
    v.fill_(1.0)
    L.dropout_fwd(v, L.Dropout(0.5, 11, 2), out=v)
    assert torch.equal(v.double(), _factor((3, 1001), 0.5, 11, 2))


# ---- group norm --------------------------------------------------------------------------------
def _split(t, groups, last):
    """[batch, groups, channels of a group, points]"""
    t = t.double()
    if last:
        t = t.movedim(-1, 1)
    return t.reshape(t.shape[0], groups, t.shape[1] // groups, -1)


def _join(t, like, last):
    shape = (like.shape[0], like.shape[-1]) + like.shape[1:-1] if last else like.shape
    t = t.reshape(shape)
    return t.movedim(1, -1) if last else t


def _act64(u, act):
    """act(u), act'(u)"""
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(u / math.sqrt(2)))
        return u * cdf, cdf + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return u * s, s * (1 + u * (1 - s))
    return u, torch.ones_like(u)


class _Ref:
    """The operator in float64, with the magnitudes that its bounds are made of."""

    def __init__(self, x, groups, gamma, beta, act, last, factor, eps=EPS):
        self.x, self.groups, self.last, self.act = x, groups, last, act
        v = _split(x, groups, last)
        side = (1, groups, v.shape[2], 1)
        one = torch.ones(side, dtype=torch.float64, device=x.device)
        self.ga = one if gamma is None else gamma.double().view(side)
        self.be = 0 * one if beta is None else beta.double().view(side)
        over = (2, 3)
        self.mean = v.mean(over, keepdim=True)
        self.rstd = 1 / torch.sqrt(((v - self.mean) ** 2).mean(over, keepdim=True) + eps)
        self.h = (v - self.mean) * self.rstd
        self.kappa = v.abs().amax(over, keepdim=True) * self.rstd
        self.u = self.ga * self.h + self.be
        self.off = 32 * U * ((self.h.abs() + self.kappa) * (1 + self.h.abs()) * self.ga.abs()
                             + self.be.abs())
        self.f = torch.ones((), dtype=torch.float64, device=x.device) if factor is None \
            else _split(factor, groups, last)

    def check_fwd(self, y, stats):
        v, _ = _act64(self.u, self.act)
        # |act'| < 1.13; GELU's erf is off by 1.5e-7 = 2.5 U, SiLU's exponential by |u| U and less
        off = self.off if self.act is None else 1.13 * self.off + 8 * U * self.u.abs()
        want = v * self.f
        off = (off + 2 * U * v.abs()) * self.f
        d = self.x.dtype
        bound = off + ROUND[d] * (want.abs() + off) + torch.where(self.f == 0, 0.0, TINY[d])
        _close("y", y, _join(want, y, self.last), _join(bound, y, self.last))
        if stats is not None:
            flat = self.mean.shape[:2]
            top = _split(self.x, self.groups, self.last).abs().amax((2, 3))
            _close("mean", stats[0], self.mean.view(flat), 32 * U * top)
            _close("rstd", stats[1], self.rstd.view(flat),
                   (32 * U * (1 + self.kappa) * self.rstd).view(flat))

    def check_bwd(self, gy, got):
        up = _split(gy, self.groups, self.last) * self.f
        g = up * _act64(self.u, self.act)[1]
        # |act''| < 1.2; the slope itself is off by a few U
        og = 2 * U * g.abs() if self.act is None else up.abs() * (16 * U + 1.2 * self.off)
        if got["x"] is not None:
            v, ov, h, r, k = g * self.ga, og * self.ga.abs(), self.h, self.rstd, self.kappa

            def mean(t):
                return t.mean((2, 3), keepdim=True)

            want = r * (v - mean(v) - h * mean(v * h))
            a1, a2 = mean(v.abs()), mean((v * h).abs())
            mag = (v.abs() + a1 + h.abs() * a2) * (1 + k) + k * a2 + h.abs() * k * a1
            off = r * (32 * U * mag + ov + mean(ov) + h.abs() * mean(ov * h.abs()))
            d = self.x.dtype
            _close("grad_x", got["x"], _join(want, gy, self.last),
                   _join(off + ROUND[d] * (want.abs() + off) + TINY[d], gy, self.last))
        sums = (0, 3)
        if got["gamma"] is not None:
            _close("grad_gamma", got["gamma"], (g * self.h).sum(sums).view(-1),
                   (128 * U * g.abs() * (self.h.abs() + self.kappa) + og * self.h.abs())
                   .sum(sums).view(-1))
        if got["beta"] is not None:
            _close("grad_beta", got["beta"], g.sum(sums).view(-1),
                   (128 * U * g.abs() + og).sum(sums).view(-1))


# (channels, groups, grid), for a few entries each: groups of one channel and of all, odd widths and
# grids, groups around a wave, a work-group and its registers, planes within and beyond them
FIELDS = [
    (1, 1, (1,)), (1, 1, (2,)), (6, 3, (1,)), (4, 2, (3,)), (4, 4, (7,)), (20, 4, (64, 64)),
    (20, 5, (63, 65)), (20, 1, (24, 10, 6)), (64, 8, (33, 31)), (45, 9, (17, 15)), (3, 3, (8195,)),
    (8, 2, (2048,)), (7, 7, (16384,)), (2, 1, (70_001,)), (6, 2, (32_771,)), (640, 32, (5, 6)),
    (130, 2, (9, 7)), (256, 16, (16, 16)), (33, 11, (255,)), (12, 3, (1024,)), (96, 1, (31, 3)),
    (513, 3, (11,)), (40, 8, (129,)), (24, 6, (513,)), (1030, 5, (4,)), (2000, 1, (3,)),
]


def _case(i, channels, groups, grid, dtype, last, batch=3):
    g = _gen(channels * 31 + sum(grid) + i)
    shape = (batch,) + grid + (channels,) if last else (batch, channels) + grid
    x = (_randn(g, *shape) * 2 + 0.7).to(dtype)
    gamma, beta = 1 + 0.3 * _randn(g, channels), 0.3 * _randn(g, channels)
    return x, gamma, beta, _randn(g, *shape).to(dtype)


def _both(L, x, groups, gamma, beta, gy, act, last, mask, check=True):
    drop = None if mask is None else L.Dropout(*mask)
    y, stats = L.group_norm_fwd(x, groups, gamma, beta, act, EPS, last, drop)
    got = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, act, last, drop)
    if check:
        ref = _Ref(x, groups, gamma, beta, act, last,
                   None if mask is None else _factor(x.shape, *mask))
        ref.check_fwd(y, stats)
        ref.check_bwd(gy, got)
    return y, stats, got


@pytest.mark.parametrize("last", [False, True], ids=["first", "last"])
@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("i", range(len(FIELDS)), ids=[str(f) for f in FIELDS])
def test_group_norm(i, dtype, last):
    L = _L()
    channels, groups, grid = FIELDS[i]
    k = i + TYPES.index(dtype) + (1 if last else 0)
    act, mask = ACTS[k % 3], (None, (0.2, 5, 1), None, (0.4, 1 << 50, 77))[k % 4]
    announce("group_norm", channels, groups, grid, dtype, last, act, mask)
    x, gamma, beta, gy = _case(i, channels, groups, grid, dtype, last)
    _, stats, got = _both(L, x, groups, gamma, beta, gy, act, last, mask)
    drop = None if mask is None else L.Dropout(*mask)
    again = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, act, last, drop)
    assert all(torch.equal(got[k], again[k]) for k in got)


# rows of tokens, a norm for each head: (batch, channels, groups)
TOKENS = [(1, 1, 1), (3, 7, 1), (5, 12, 12), (8, 1024, 16), (130, 96, 3), (33, 511, 7), (2, 4096, 32),
          (9, 2050, 2), (3, 16384, 1), (2, 33000, 3), (1, 70_001, 1), (2000, 20, 4), (10_000, 6, 2),
          (513, 768, 12), (7, 5120, 40), (4, 45, 9), (300, 8, 1), (5, 8191, 1), (2, 40_000, 2)]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", TOKENS, ids=str)
def test_group_norm_tokens(shape, dtype):
    L = _L()
    batch, channels, groups = shape
    k = sum(shape) + TYPES.index(dtype)
    act, mask = ACTS[k % 3], (None, (0.1, 6, 2))[k % 2]
    announce("group_norm tokens", shape, dtype, act, mask)
    x, gamma, beta, gy = _case(k, channels, groups, (), dtype, False, batch)
    a = _both(L, x, groups, gamma, beta, gy, act, False, mask)
    b = _both(L, x, groups, gamma, beta, gy, act, True, mask, check=False)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert all(torch.equal(a[2][n], b[2][n]) for n in a[2])


# (last, channels, groups, grid, batch): work-groups of 64, 256 and 1024 threads and beyond, whole
# vectors and ragged ones, pairs of lanes, one entry and one row, rows around the work-groups' rounds,
# partial sums joined by the second pass and before it
EDGES = [(True, c, g, (p,), b) for c, g, p, b in (
    (8, 2, 70, 3), (16, 4, 300, 2), (24, 1, 33, 1), (40, 10, 129, 3), (64, 8, 4000, 1), (136, 17, 65, 2),
    (320, 32, 100, 2), (328, 41, 9, 5), (4, 4, 1000, 2), (12, 1, 5000, 1), (132, 3, 77, 1),
    (1048, 8, 17, 2), (64, 64, 777, 2), (128, 1, 20_000, 2), (264, 2, 16_384, 1))] + \
    [(False, c, g, (p,), b) for c, g, p, b in (
        (2, 1, 1024, 1), (2, 1, 1026, 2), (8, 1, 1023, 1), (8, 2, 2048, 3), (8, 2, 2050, 1),
        (4, 1, 4096, 2), (4, 1, 4098, 1), (8, 1, 4095, 2), (1, 1, 16_384, 1), (1, 1, 16_392, 3),
        (2, 1, 16_385, 1), (1, 1, 32_768, 2), (1, 1, 32_776, 1), (5, 1, 4100, 2), (300, 2, 8, 2),
        (40, 1, 520, 1), (9, 3, 20_480, 1), (3, 1, 66_000, 2), (2048, 1, 6, 1), (700, 7, 17, 3))] + \
    [(False, c, g, (), b) for c, g, b in (
        (64, 1, 4), (64, 1, 513), (256, 32, 31), (256, 32, 32), (256, 32, 129), (1024, 4, 64),
        (4096, 2, 5), (8192, 1, 3), (8200, 1, 3), (72, 9, 1000), (17 * 24, 17, 300), (2056, 8, 260))]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("case", EDGES, ids=str)
def test_group_norm_edges(case, dtype):
    L = _L()
    last, channels, groups, grid, batch = case
    k = EDGES.index(case)
    act, mask = ACTS[k % 3], ((0.3, 5, 1) if k % 3 != 2 or last else None)
    announce("group_norm edges", case, dtype, act, mask)
    x, gamma, beta, gy = _case(k, channels, groups, grid, dtype, last, batch)
    _, stats, want = _both(L, x, groups, gamma, beta, gy, act, last, mask)
    drop = None if mask is None else L.Dropout(*mask)
    args = (x, groups, gamma, beta, stats)
    for keys in (("x",), ("gamma",), ("beta",)):
        got = L.group_norm_bwd(*args, gy, act, last, drop, want=keys)
        assert torch.equal(got[keys[0]], want[keys[0]])
    over = gy.clone()
    got = L.group_norm_bwd(*args, over, act, last, drop, out={"x": over})
    assert all(torch.equal(got[n], want[n]) for n in want)


@pytest.mark.parametrize("dtype,last,field", [
    (torch.float32, False, (8, 2, (3_000_001,))), (torch.bfloat16, False, (5, 1, (9_000_000,))),
    (torch.float32, True, (20, 4, (1_200_003,))), (torch.float16, True, (45, 9, (1_100_001,))),
    (torch.float32, False, (4096, 32, ())), (torch.bfloat16, False, (6150, 6, ()))], ids=str)
def test_group_norm_outputs_past_the_cache(dtype, last, field):
    """Outputs over 128 MB, which go past the caches, at odd places too."""
    L = _L()
    channels, groups, grid = field
    batch = 2 if grid else 12_000
    announce("group_norm large", dtype, last, field)
    x, gamma, beta, gy = _case(9, channels, groups, grid, dtype, last, batch)
    assert x.numel() * x.element_size() > 128 << 20
    n = math.prod(x.shape[1:])
    mask = (0.2, 9, 3)
    buf = torch.empty(x.numel() + 64, dtype=dtype, device="cuda")
    y = buf[1:1 + x.numel()].view(x.shape)
    _, stats = L.group_norm_fwd(x, groups, gamma, beta, "silu", EPS, last, L.Dropout(*mask), out=y)
    got = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, "silu", last, L.Dropout(*mask))
    sums = {}
    step = 1 if grid else 3000
    for at in range(0, batch, step):
        part = slice(at, at + step)
        f = _factor(x[part].shape, *mask, first=at * n)
        ref = _Ref(x[part], groups, gamma, beta, "silu", last, f)
        ref.check_fwd(y[part], stats[:, part])
        ref.check_bwd(gy[part], {"x": got["x"][part], "gamma": None, "beta": None})
        up = _split(gy[part], groups, last) * ref.f
        g = up * _act64(ref.u, "silu")[1]
        og = up.abs() * (16 * U + 1.2 * ref.off)
        for k, v, o in (("gamma", g * ref.h, 128 * U * g.abs() * (ref.h.abs() + ref.kappa) + og * ref.h.abs()),
                        ("beta", g, 128 * U * g.abs() + og)):
            s = sums.setdefault(k, [0, 0])
            s[0] = s[0] + v.sum((0, 3)).view(-1)
            s[1] = s[1] + o.sum((0, 3)).view(-1)
        del ref, f, up, g, og
    for k, (v, o) in sums.items():
        _close("grad_" + k, got[k], v, o)


SOME = [(False, (20, 4, (9, 7))), (True, (20, 4, (9, 7))), (False, (6, 2, (12_000,))),
        (True, (45, 9, (300,))), (False, (24, 1, (3,))), (True, (300, 4, (65,))), (False, (96, 4, ())),
        (False, (5000, 2, ())), (False, (33, 3, (40_001,)))]


@pytest.mark.parametrize("last,field", SOME, ids=str)
def test_group_norm_optional_arguments(last, field):
    L = _L()
    announce("group_norm optional", last, field)
    channels, groups, grid = field
    x, gamma, beta, gy = _case(2, channels, groups, grid, torch.float32, last, 4)
    drop = L.Dropout(0.2, 8, 1)
    for ga, be in ((None, None), (gamma, None), (None, beta)):
        y, none = L.group_norm_fwd(x, groups, ga, be, "gelu", EPS, last, want_stats=False)
        assert none is None
        _Ref(x, groups, ga, be, "gelu", last, None).check_fwd(y, None)
        _both(L, x, groups, ga, be, gy, "silu", last, None)
    y, stats = L.group_norm_fwd(x, groups, gamma, beta, "gelu", EPS, last, drop)
    want = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, "gelu", last, drop)
    for keys in (("x",), ("gamma",), ("beta",), ("gamma", "beta"), ("x", "beta"), ()):
        got = L.group_norm_bwd(x, groups, gamma, beta, stats, gy, "gelu", last, drop, want=keys)
        for k in want:
            assert (got[k] is None) == (k not in keys)
            if k in keys:
                assert torch.equal(got[k], want[k]), (keys, k)
    # a large mean: the deviations come from the data itself, not from E[x^2] - E[x]^2
    _both(L, x + 3000.0, groups, gamma, beta, gy, "silu", last, None)
    # constant data: no deviation at all
    _both(L, torch.full_like(x, 2.5), groups, gamma, beta, gy, "gelu", last, None)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("last,field", SOME, ids=str)
def test_group_norm_strides_alignment_in_place(last, field, dtype):
    L = _L()
    announce("group_norm strides", last, field, dtype)
    channels, groups, grid = field
    x0, gamma, beta, gy0 = _case(3, channels, groups, grid, dtype, last)
    shape, n = x0.shape, math.prod(x0.shape[1:])

    def cut(off, gap):
        buf = torch.full((off + shape[0] * (n + gap),), 77.0, dtype=dtype, device="cuda")
        return buf, buf[off:].view(shape[0], n + gap)[:, :n].unflatten(1, shape[1:])

    drop = L.Dropout(0.3, 5, 6)
    y0, stats0 = L.group_norm_fwd(x0, groups, gamma, beta, "silu", EPS, last, drop)

    def bwd(x, gy, out):
        return L.group_norm_bwd(x, groups, gamma, beta, stats0, gy, "silu", last, drop, out={"x": out})

    want = bwd(x0, gy0, torch.empty_like(x0))
    for off, gap in ((1, 0), (3, 5), (0, 8), (8, 1)):
        _, x = cut(off, gap)
        _, gy = cut(off + 2, gap + 3)
        x.copy_(x0)
        gy.copy_(gy0)
        ybuf, y = cut(off + 1, gap + 2)
        _, stats = L.group_norm_fwd(x, groups, gamma, beta, "silu", EPS, last, drop, out=y)
        assert torch.equal(y, y0) and torch.equal(stats, stats0)
        y.fill_(77.0)
        assert bool((ybuf == 77.0).all()), "the forward wrote outside its entries"
        gbuf, gx = cut(off + 5, gap + 4)
        got = bwd(x, gy, gx)
        assert all(torch.equal(got[k], want[k]) for k in want)
        gx.fill_(77.0)
        assert bool((gbuf == 77.0).all()), "the backward wrote outside its entries"
        # in place: grad_x over grad_y, then over x; y over x
        got = bwd(x, gy, gy)
        assert all(torch.equal(got[k], want[k]) for k in want)
        gy.copy_(gy0)
        got = bwd(x, gy, x)
        assert all(torch.equal(got[k], want[k]) for k in want)
        x.copy_(x0)
        L.group_norm_fwd(x, groups, gamma, beta, "silu", EPS, last, drop, out=x)
        assert torch.equal(x, y0)
    # one entry for all (stride 0)
    xs, gs = x0[:1].expand(shape), gy0[:1].expand(shape)
    _both(L, xs, groups, gamma, beta, gs, "gelu", last, (0.3, 5, 6))


@pytest.mark.parametrize("last,field", SOME, ids=str)
def test_group_norm_non_finite_groups_stay_apart(last, field):
    L = _L()
    announce("group_norm non-finite", last, field)
    channels, groups, grid = field
    x, gamma, beta, gy = _case(4, channels, groups, grid, torch.float32, last)
    y0, s0, g0 = _both(L, x, groups, gamma, beta, gy, None, last, None, check=False)
    for value in (math.inf, -math.inf, math.nan):
        bad = x.clone()
        own = torch.zeros_like(_split(x, groups, last), dtype=torch.bool)
        own[1, groups // 2] = True
        own = _join(own, x, last)
        _split_at = own.nonzero()[int(own.sum()) // 2]
        bad[tuple(_split_at)] = value
        y, s, g = _both(L, bad, groups, gamma, beta, gy, None, last, None, check=False)
        assert bool(y[own].isnan().all()) and bool(g["x"][own].isnan().all())
        y[own], g["x"][own] = y0[own], g0["x"][own]
        assert torch.equal(y, y0) and torch.equal(g["x"], g0["x"])


@pytest.mark.parametrize("last", [False, True])
def test_group_norm_no_rows(last):
    L = _L()
    announce("group_norm no rows", last)
    for shape in ((0, 6), (0, 6, 6), (3, 6, 0), (3, 0, 6)):
        channels = shape[-1] if last else shape[1]
        if channels != 6:
            continue
        x = torch.empty(shape, device="cuda")
        y, stats = L.group_norm_fwd(x, 3, channels_last=last)
        assert y.shape == x.shape and stats.shape == (2, shape[0], 3)
        out = {k: torch.full((6,), 9.0, device="cuda") for k in ("gamma", "beta")}
        L.group_norm_bwd(x, 3, None, None, stats, x, channels_last=last, out=out)
        assert not out["gamma"].any() and not out["beta"].any()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("last,field", SOME[:7], ids=str)
def test_group_norm_against_differences(last, field, act):
    """Directional differences of L = sum w * y, mask included: a four-point rule of the float32
    forward.  Its error is O(e^4) = 1e-6 relative from the rule and U |y| sqrt(n) / e ~ 1e-5 from
    rounding, on derivatives of size sqrt(n)."""
    L = _L()
    announce("group_norm differences", last, field, act)
    channels, groups, grid = field
    x, gamma, beta, w = _case(5, channels, groups, grid, torch.float32, last, 2)
    g = _gen(6)
    drop = L.Dropout(0.25, 3, 3)
    _, stats = L.group_norm_fwd(x, groups, gamma, beta, act, EPS, last, drop)
    got = L.group_norm_bwd(x, groups, gamma, beta, stats, w, act, last, drop)

    def loss(x, gamma, beta):
        y = L.group_norm_fwd(x, groups, gamma, beta, act, EPS, last, drop)[0]
        return float((y.double() * w.double()).sum())

    e = 1.0 / 64  # exact steps in float32
    for k, base in (("x", x), ("gamma", gamma), ("beta", beta)):
        d = _randn(g, *base.shape)
        args = {"x": x, "gamma": gamma, "beta": beta}

        def at(t):
            args[k] = base + t * d
            return loss(**args)

        diff = (8 * (at(e) - at(-e)) - (at(2 * e) - at(-2 * e))) / (12 * e)
        want = float((got[k].double() * d.double()).sum())
        size = float(got[k].double().norm())
        print(f"    {k}: difference {diff:.6f}, gradient {want:.6f}", flush=True)
        assert abs(diff - want) <= 1e-3 * size + 1e-3 * abs(want)


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("last,field", [(False, (4, 2, (300,))), (True, (12, 3, (500,))),
                                        (False, (3, 1, (30_000,))), (False, (2050, 1, ())),
                                        (True, (130, 2, (999,)))], ids=str)
def test_group_norm_of_large_means(last, field, dtype):
    """Data whose mean's square passes float32's range, and the sum of its squared deviations too
    where a group is large, while its variance does not."""
    L = _L()
    announce("group_norm large means", last, field, dtype)
    channels, groups, grid = field
    x, gamma, beta, gy = _case(7, channels, groups, grid, torch.float32, last)
    big = 30000.0 if dtype == torch.float16 else 2.5e19
    x = (big * (1 + 0.01 * x)).to(dtype)
    y, stats, got = _both(L, x, groups, gamma, beta, gy.to(dtype), None, last, None)
    assert bool(torch.isfinite(y).all())


def test_group_norm_offsets_past_32_bits():
    """Entries 2^31 elements apart, planes of 2^30 points, and channels-last rows beyond 2^31."""
    L = _L()
    announce("group_norm long offsets")
    stride = (1 << 31) + 24
    buf = torch.empty(2 * stride + (1 << 21), dtype=torch.bfloat16, device="cuda")
    for last, field in SOME:
        channels, groups, grid = field
        x0, gamma, beta, _ = _case(8, channels, groups, grid, torch.bfloat16, last)
        x = buf.as_strided(x0.shape, (stride,) + x0.stride()[1:])
        x.copy_(x0)
        y0, s0 = L.group_norm_fwd(x0, groups, gamma, beta, "gelu", EPS, last)
        y, s = L.group_norm_fwd(x, groups, gamma, beta, "gelu", EPS, last, out=x)
        assert torch.equal(y, y0) and torch.equal(s, s0)
    del buf, x, y
    n = (1 << 30) + 5
    for last in (False, True):
        shape = (1, n, 3) if last else (1, 3, n)
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        x.fill_(-1.0)
        at = (slice(None), slice(0, 1 << 29)) if last else (slice(None), slice(None), slice(0, 1 << 29))
        x[at] = 1.0
        share = (1 << 29) / n  # of ones: the mean and variance follow
        mean, var = 2 * share - 1, 1 - (2 * share - 1) ** 2
        y, stats = L.group_norm_fwd(x, 1, eps=0.0, channels_last=last, out=x,
                                    drop=L.Dropout(0.5, 3, 1))
        r = 1 / math.sqrt(var)
        # a thread's moments join a few hundred times, the parts after them ten times more
        assert abs(float(stats[0]) - mean) <= 512 * U and abs(float(stats[1]) - r) <= 512 * U
        flat = y.view(-1)
        for first in (0, flat.numel() - 4099):
            f = _factor((4099,), 0.5, 3, 1, first)
            ones = flat[first:first + 4099]
            want = f * ((1 if first == 0 else -1) - mean) * r
            _close("y", ones, want, (2.0 ** -8 + 1024 * U) * want.abs())
        del x, y, flat, ones


def _all(L, s):
    y, _ = L.group_norm_fwd(s["x"], 4, s["gamma"], s["beta"], "gelu", EPS, False, s["drop"],
                            out=s["y"], stats=s["stats"], ws=s["ws"])
    L.group_norm_bwd(s["x"], 4, s["gamma"], s["beta"], s["stats"], s["gy"], "gelu", False, s["drop"],
                     out=s["grads"], ws=s["ws"])
    t, _ = L.group_norm_fwd(s["xl"], 4, s["gamma"], s["beta"], "silu", EPS, True, s["drop"],
                            out=s["yl"], stats=s["stats2"], ws=s["ws"])
    L.group_norm_bwd(s["xl"], 4, s["gamma"], s["beta"], s["stats2"], s["gyl"], "silu", True, s["drop"],
                     out=s["grads2"], ws=s["ws"])
    L.dropout_fwd(y, s["drop"], s["x"], out=s["sum"])
    L.dropout_bwd(s["sum"], s["drop"], out=s["back"])


def _state(L, seed, points=333):
    g = _gen(seed)
    x, xl = _randn(g, 2, 20, points), _randn(g, 2, points, 20)
    s = {"x": x, "gy": _randn(g, *x.shape), "xl": xl, "gyl": _randn(g, *xl.shape),
         "gamma": 1 + 0.1 * _randn(g, 20), "beta": 0.1 * _randn(g, 20),
         "ws": torch.empty(1 << 22, dtype=torch.uint8, device="cuda"),
         "counter": torch.zeros(1, dtype=torch.int64, device="cuda")}
    s["drop"] = L.Dropout(0.3, 21, 1, s["counter"])
    for k in ("y", "sum", "back"):
        s[k] = torch.empty_like(x)
    s["yl"] = torch.empty_like(xl)
    s["stats"], s["stats2"] = (torch.empty(2, 2, 4, device="cuda") for _ in range(2))
    for k, like in (("grads", x), ("grads2", xl)):
        s[k] = {"x": torch.empty_like(like), "gamma": torch.empty(20, device="cuda"),
                "beta": torch.empty(20, device="cuda")}
    return s


def _outputs(s):
    return [s[k] for k in ("y", "sum", "back", "yl", "stats", "stats2")] + \
        [t for k in ("grads", "grads2") for t in s[k].values()]


@pytest.mark.parametrize("points", [333, 40_000])
def test_graph_replays_match_eager(points):
    """Every replay takes the counter as it is then: other masks, and the eager call's."""
    L = _L()
    announce("between ops in a graph", points)
    eager, cap = _state(L, 7, points), _state(L, 7, points)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _all(L, _state(L, 8, points))
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _all(L, cap)
        cap["counter"] += 3
    seen = []
    for k in range(4):
        x = _randn(_gen(40 + k), *eager["x"].shape)
        for s in (eager, cap):
            s["x"].copy_(x)
        _all(L, eager)
        eager["counter"] += 3
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(_outputs(eager), _outputs(cap))), k
        f = _factor(x.shape, 0.3, 21, 1 + 3 * k)
        assert torch.equal(cap["y"] == 0, f == 0)
        seen.append(cap["y"] == 0)
    assert not any(torch.equal(seen[i], seen[j]) for i in range(4) for j in range(i))


def test_calls_run_on_the_current_stream():
    """Inputs written on a stream behind other work, with no synchronisation, and two streams at once,
    each with its own workspace."""
    L = _L()
    announce("between ops behind a stream's own work")
    new, s = _state(L, 9, 4001), _state(L, 10, 4001)
    _all(L, _state(L, 8, 4001))
    busy = torch.ones(1 << 28, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    other = _state(L, 9, 4001)
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        for _ in range(60):
            busy.mul_(1.0)  # 2 GB each
        for k in ("x", "gy", "xl", "gyl", "gamma", "beta"):
            s[k].copy_(new[k])
        ready = torch.cuda.Event()
        ready.record()
        _all(L, s)
    still_busy = not ready.query()
    with torch.cuda.stream(b):
        b.wait_event(ready)
        _all(L, other)
    torch.cuda.synchronize()
    assert still_busy, "the other work was too short to tell streams apart"
    _all(L, new)
    torch.cuda.synchronize()
    for got in (s, other):
        assert all(torch.equal(p, q) for p, q in zip(_outputs(got), _outputs(new)))


def test_refusals():
    L = _L()
    announce("between ops refusals")
    x = torch.zeros(4, 8, 6, device="cuda")
    st = torch.zeros(2, 4, 2, device="cuda")
    drop = L.Dropout(0.5, 1)
    with pytest.raises(L.FnoError, match="groups"):
        L.group_norm_fwd(x, 3)
    with pytest.raises(ValueError, match="act"):
        L.group_norm_fwd(x, 2, act="relu")
    with pytest.raises(ValueError, match="gamma"):
        L.group_norm_fwd(x, 2, torch.ones(6, device="cuda"))
    with pytest.raises(ValueError, match="gamma"):
        L.group_norm_fwd(x, 2, torch.ones(8, device="cuda"), channels_last=True)
    with pytest.raises(ValueError, match="out"):
        L.group_norm_fwd(x, 2, out=x[:2])
    with pytest.raises(ValueError, match="stats"):
        L.group_norm_bwd(x, 2, None, None, st[:1], x)
    with pytest.raises(ValueError, match="stats"):
        L.group_norm_bwd(x, 4, None, None, st, x)
    with pytest.raises(ValueError, match="grad_y"):
        L.group_norm_bwd(x, 2, None, None, st, x.bfloat16())
    with pytest.raises(ValueError, match="packed"):
        L.group_norm_fwd(x.transpose(1, 2), 2)
    with pytest.raises(ValueError, match="residual"):
        L.dropout_fwd(x, drop, x[:2])
    with pytest.raises(ValueError, match="out"):
        L.dropout_bwd(x, drop, out=x.bfloat16())
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8),
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20)):
        with pytest.raises(ValueError, match="ws"):
            L.group_norm_fwd(x, 2, ws=ws)
    big = torch.zeros(1, 8, 1 << 20, device="cuda")
    with pytest.raises(L.FnoError, match="workspace"):
        L.group_norm_fwd(big, 2, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(L.FnoError, match="workspace"):
        L.group_norm_bwd(big, 2, None, None, torch.zeros(2, 1, 2, device="cuda"), big,
                         ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert not x.any()
