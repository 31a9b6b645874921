"""The training operators on the GPU: layer norm forward and backward, the gradient norm with
clipping, and AdamW, against plain float64 formulas.

Tolerances are elementwise and follow from the arithmetic: U = 2^-24 is float32's unit roundoff,
a half-format result adds its own (2^-8 bfloat16, 2^-11 half).  Every quantity is a short chain of
float32 operations on sums of at most a few hundred roundings' depth on one path, so each bound is
a constant times U times the sum of the magnitudes that enter the result.
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
EPS = 1e-5


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


def _sides(x, v, one):
    if v is None:
        return torch.full((), one, dtype=torch.float64, device=x.device)
    return v.double().view((1, -1) + (1,) * (x.dim() - 2))


def _norm64(x, gamma, beta, eps):
    """y, mean, rstd, h, kappa (the row's condition: its largest magnitude over its deviation)."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = 1.0 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    h = (x - mean) * rstd
    kappa = x.abs().amax(1, keepdim=True) * rstd
    return _sides(x, gamma, 1.0) * h + _sides(x, beta, 0.0), mean, rstd, h, kappa


def _check_fwd(x, gamma, beta, y, stats, eps=EPS):
    want, mean, rstd, h, kappa = _norm64(x, gamma, beta, eps)
    ga, be = _sides(x, gamma, 1.0).abs(), _sides(x, beta, 0.0).abs()
    # the mean is off by a few U of the row's magnitude, the deviation's square by as much
    off = 32 * U * ((h.abs() + kappa) * (1 + h.abs()) * ga + be)
    _close("y", y, want, off + ROUND[x.dtype] * (want.abs() + off) + TINY[x.dtype])
    if stats is not None:
        _close("mean", stats[0], mean.squeeze(1), 32 * U * x.double().abs().amax(1))
        _close("rstd", stats[1], rstd.squeeze(1), 32 * U * ((1 + kappa) * rstd).squeeze(1))


def _check_bwd(x, gamma, gy, got, eps=EPS):
    _, mean, rstd, h, kappa = _norm64(x, gamma, None, eps)
    up = gy.double()
    g = up * _sides(x, gamma, 1.0)
    m1, m2 = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    a1, a2 = g.abs().mean(1, keepdim=True), (g * h).abs().mean(1, keepdim=True)
    if got["x"] is not None:
        want = rstd * (g - m1 - h * m2)
        mag = (g.abs() + a1 + h.abs() * a2) * (1 + kappa) + kappa * a2 + h.abs() * kappa * a1
        off = 32 * U * rstd * mag
        _close("grad_x", got["x"], want, off + ROUND[x.dtype] * (want.abs() + off) + TINY[x.dtype])
    rows = [0] + list(range(2, x.dim()))
    if got["gamma"] is not None:
        _close("grad_gamma", got["gamma"], (up * h).sum(rows),
               128 * U * (up.abs() * (h.abs() + kappa)).sum(rows))
    if got["beta"] is not None:
        _close("grad_beta", got["beta"], up.sum(rows), 128 * U * up.abs().sum(rows))


# [batch, channels] rows and [batch, channels, *grid] fields: one entry, one row, widths around
# every power of two and around the lanes' vectors, long rows, odd grids, few and many points
SHAPES = [
    (1, 1), (3, 1), (1, 2), (5, 3), (7, 8), (130, 31), (65, 33), (9, 64), (300, 65), (4, 127),
    (2, 256), (17, 257), (33, 511), (6, 1000), (5, 1024), (3, 1025), (3, 2047), (2, 2049),
    (7, 4096), (2, 4103), (1, 8192), (2, 8200), (3, 16384), (2, 16391), (2, 33000), (1, 70001),
    (2000, 20), (10000, 7), (513, 768),
    (1, 1, 1, 1), (2, 1, 5), (1, 20, 1, 1), (3, 20, 7), (2, 20, 63, 65), (1, 32, 256), (2, 32, 257),
    (3, 64, 64, 64), (2, 64, 1001), (1, 65, 300), (2, 100, 333), (1, 128, 512), (2, 129, 260),
    (1, 200, 1030), (2, 256, 100), (1, 257, 515), (2, 513, 9), (700, 5, 2), (40, 33, 3),
    (5, 20, 24, 10, 6), (1, 7, 4099),
]


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_norm(shape, dtype):
    L = _L()
    announce("layer_norm", shape, dtype)
    g = _gen(sum(shape) * 7 + TYPES.index(dtype))
    x = (_randn(g, *shape) * 2 + 0.7).to(dtype)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    gy = _randn(g, *shape).to(dtype)
    y, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    _check_fwd(x, gamma, beta, y, stats)
    got = L.layer_norm_bwd(x, gamma, stats, gy)
    _check_bwd(x, gamma, gy, got)
    again = L.layer_norm_bwd(x, gamma, stats, gy)
    assert all(torch.equal(got[k], again[k]) for k in got)


# widths and extents at which another kernel, vector width or number of waves takes over
EDGES = [(3, d) for d in (7, 8, 9, 15, 16, 63, 128, 129, 512, 513, 2048, 4097, 8191, 8193, 12288,
                          16383, 16385)] + \
    [(n, 96) for n in (511, 512, 513)] + \
    [(2, c, p) for c in (8, 9, 48, 49, 72, 73, 101, 120, 121, 255) for p in (255, 256, 261)] + \
    [(1, 20, 21503), (1, 20, 21505), (3, 24, 255), (13, 24, 255), (1, 3, 1), (6, 257, 2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=str)
@pytest.mark.parametrize("shape", EDGES, ids=str)
def test_layer_norm_edges(shape, dtype):
    L = _L()
    announce("layer_norm edges", shape, dtype)
    g = _gen(sum(shape))
    x, gy = (_randn(g, *shape) - 0.4).to(dtype), _randn(g, *shape).to(dtype)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    y, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    _check_fwd(x, gamma, beta, y, stats)
    _check_bwd(x, gamma, gy, L.layer_norm_bwd(x, gamma, stats, gy))
    # in place, and the weight gradients alone: the same bits
    want = L.layer_norm_bwd(x, gamma, stats, gy)
    alone = L.layer_norm_bwd(x, gamma, stats, gy, want=("gamma", "beta"))
    over = gy.clone()
    got = L.layer_norm_bwd(x, gamma, stats, over, out={"x": over})
    assert torch.equal(over, want["x"])
    for k in ("gamma", "beta"):
        assert torch.equal(got[k], want[k]) and torch.equal(alone[k], want[k])


@pytest.mark.parametrize("shape", [(37, 257), (5, 4100), (3, 20, 130), (2, 300, 70)], ids=str)
def test_layer_norm_optional_arguments(shape):
    L = _L()
    announce("layer_norm optional", shape)
    g = _gen(5)
    x, gy = _randn(g, *shape), _randn(g, *shape)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    for ga, be in ((None, None), (gamma, None), (None, beta)):
        y, none = L.layer_norm_fwd(x, ga, be, EPS, want_stats=False)
        assert none is None
        _check_fwd(x, ga, be, y, None)
    full, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    want = L.layer_norm_bwd(x, gamma, stats, gy)
    for keys in (("x",), ("gamma",), ("beta",), ("gamma", "beta"), ("x", "beta"), ()):
        got = L.layer_norm_bwd(x, gamma, stats, gy, want=keys)
        for k in want:
            assert (got[k] is None) == (k not in keys)
            if k in keys:
                assert torch.equal(got[k], want[k]), (keys, k)
    got = L.layer_norm_bwd(x, None, stats, gy)
    _check_bwd(x, None, gy, got)
    # a large mean: the deviations come from the rows themselves, not from E[x^2] - E[x]^2
    far = x + 3000.0
    y, stats = L.layer_norm_fwd(far, gamma, beta, EPS)
    _check_fwd(far, gamma, beta, y, stats)
    # constant rows: no deviation at all
    flat = torch.full_like(x, 2.5)
    y, stats = L.layer_norm_fwd(flat, gamma, beta, EPS)
    _check_fwd(flat, gamma, beta, y, stats)
    _check_bwd(flat, gamma, gy, L.layer_norm_bwd(flat, gamma, stats, gy))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(29, 65), (11, 1031), (4, 5000), (3, 17000), (2, 20, 67),
                                   (3, 64, 515), (2, 140, 33), (2, 300, 21)], ids=str)
def test_layer_norm_strides_alignment_in_place(shape, dtype):
    L = _L()
    announce("layer_norm strides", shape, dtype)
    g = _gen(9)
    n = math.prod(shape[1:])

    def cut(off, gap):  # a field whose entries lie `gap` apart, `off` elements into a buffer
        buf = torch.full((off + shape[0] * (n + gap),), 77.0, dtype=dtype, device="cuda")
        return buf, buf[off:].view(shape[0], n + gap)[:, :n].unflatten(1, shape[1:])

    x0, gy0 = (_randn(g, *shape) + 0.3).to(dtype), _randn(g, *shape).to(dtype)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    y0, stats0 = L.layer_norm_fwd(x0, gamma, beta, EPS)
    want = L.layer_norm_bwd(x0, gamma, stats0, gy0)
    for off, gap in ((1, 0), (3, 5), (0, 8), (8, 1)):
        _, x = cut(off, gap)
        _, gy = cut(off + 2, gap + 3)
        x.copy_(x0)
        gy.copy_(gy0)
        ybuf, y = cut(off + 1, gap + 2)
        L.layer_norm_fwd(x, gamma, beta, EPS, out=y)
        assert torch.equal(y, y0)
        y.fill_(77.0)
        assert bool((ybuf == 77.0).all()), "the forward wrote outside its rows"
        gbuf, gx = cut(off + 5, gap + 4)
        got = L.layer_norm_bwd(x, gamma, stats0, gy, out={"x": gx})
        assert torch.equal(gx, want["x"])
        assert torch.equal(got["gamma"], want["gamma"]) and torch.equal(got["beta"], want["beta"])
        gx.fill_(77.0)
        assert bool((gbuf == 77.0).all()), "the backward wrote outside its rows"
        # in place: grad_x over grad_y, then over x; y over x
        got = L.layer_norm_bwd(x, gamma, stats0, gy, out={"x": gy})
        assert torch.equal(gy, want["x"]) and torch.equal(got["gamma"], want["gamma"])
        gy.copy_(gy0)
        got = L.layer_norm_bwd(x, gamma, stats0, gy, out={"x": x})
        assert torch.equal(x, want["x"]) and torch.equal(got["beta"], want["beta"])
        x.copy_(x0)
        L.layer_norm_fwd(x, gamma, beta, EPS, out=x)
        assert torch.equal(x, y0)
    # one entry for all (stride 0), as the gradient of a sum comes
    xs, gs = x0[:1].expand(shape), gy0[:1].expand(shape)
    y, stats = L.layer_norm_fwd(xs, gamma, beta, EPS)
    _check_fwd(xs, gamma, beta, y, stats)
    _check_bwd(xs, gamma, gs, L.layer_norm_bwd(xs, gamma, stats, gs))


@pytest.mark.parametrize("shape", [(7, 100), (5, 3000), (3, 9001), (2, 20, 300), (2, 70, 90),
                                   (2, 400, 12)], ids=str)
def test_layer_norm_non_finite_rows_stay_apart(shape):
    L = _L()
    announce("layer_norm non-finite", shape)
    g = _gen(3)
    x, gy = _randn(g, *shape), _randn(g, *shape)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    y0, s0 = L.layer_norm_fwd(x, gamma, beta, EPS)
    g0 = L.layer_norm_bwd(x, gamma, s0, gy)["x"]
    for value in (math.inf, -math.inf, math.nan):
        bad = x.clone()
        at = (1, shape[1] // 2) + tuple(n // 2 for n in shape[2:])
        bad[at] = value
        row = (1, slice(None)) + at[2:]
        y, s = L.layer_norm_fwd(bad, gamma, beta, EPS)
        gx = L.layer_norm_bwd(bad, gamma, s, gy)["x"]
        assert bool(y[row].isnan().all()) and bool(gx[row].isnan().all())
        y[row], gx[row] = y0[row], g0[row]
        assert torch.equal(y, y0) and torch.equal(gx, g0)


def test_layer_norm_no_rows():
    L = _L()
    announce("layer_norm no rows")
    for shape in ((0, 5), (0, 5, 4), (3, 5, 0)):
        x = torch.empty(shape, device="cuda")
        y, stats = L.layer_norm_fwd(x)
        assert y.shape == x.shape and stats.numel() == 0
        out = {"gamma": torch.full((5,), 9.0, device="cuda"),
               "beta": torch.full((5,), 9.0, device="cuda")}
        L.layer_norm_bwd(x, None, stats, x, out=out)
        assert not out["gamma"].any() and not out["beta"].any()


@pytest.mark.parametrize("shape", [(12, 130), (3, 5000), (2, 20, 66), (2, 300, 9)], ids=str)
def test_layer_norm_against_differences(shape):
    """Directional differences of L = sum w * norm(x): a four-point rule of the float32 forward.
    Its error is O(e^4) = 1e-6 relative from the rule and U |y| sqrt(n) / e ~ 1e-5 from rounding,
    on derivatives of size sqrt(n)."""
    L = _L()
    announce("layer_norm differences", shape)
    g = _gen(21)
    x, w = _randn(g, *shape), _randn(g, *shape)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    _, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    got = L.layer_norm_bwd(x, gamma, stats, w)

    def loss(x, gamma, beta):
        return float((L.layer_norm_fwd(x, gamma, beta, EPS)[0].double() * w.double()).sum())

    e = 1.0 / 64  # exact steps in float32
    for k, base in (("x", x), ("gamma", gamma), ("beta", beta)):
        d = _randn(g, *base.shape)
        args = {"x": x, "gamma": gamma, "beta": beta}

        def at(t):
            args[k] = base + t * d
            return loss(**args)

        diff = (8 * (at(e) - at(-e)) - (at(2 * e) - at(-2 * e))) / (12 * e)
        want = float((got[k].double() * d.double()).sum())
        size = float(got[k].double().norm() * 1.0)
        print(f"    {k}: difference {diff:.6f}, gradient {want:.6f}", flush=True)
        assert abs(diff - want) <= 1e-3 * size + 1e-3 * abs(want)


def test_layer_norm_offsets_past_32_bits():
    """Rows 2^31 elements apart, and a field whose channels are: every offset is 64 bits wide."""
    L = _L()
    announce("layer_norm long offsets")
    g = _gen(2)
    stride = (1 << 31) + 24
    buf = torch.empty(2 * stride + 4096, dtype=torch.bfloat16, device="cuda")
    for d in (100, 2056):
        x0 = _randn(g, 3, d).bfloat16()
        x = buf.as_strided((3, d), (stride, 1))
        x.copy_(x0)
        y0, s0 = L.layer_norm_fwd(x0)
        y, s = L.layer_norm_fwd(x, out=x)
        assert torch.equal(x, y0) and torch.equal(s, s0)
    del buf, x, y
    npts = (1 << 30) + 5
    x = torch.empty((1, 3, npts), dtype=torch.bfloat16, device="cuda")
    tail = _randn(g, 1, 3, 4096).bfloat16()
    x[:, :, :4096] = tail
    x[:, :, -4096:] = tail
    y0, _ = L.layer_norm_fwd(tail)
    y, _ = L.layer_norm_fwd(x, want_stats=False)
    assert torch.equal(y[:, :, :4096], y0) and torch.equal(y[:, :, -4096:], y0)


@pytest.mark.parametrize("shape,dtype", [
    ((70_001, 2048), torch.bfloat16), ((17_001, 4096), torch.float32), ((140_003, 512), torch.float32),
    ((5, 64, 262_144), torch.float32), ((3, 20, 1_200_032), torch.float32), ((9, 17, 500_000), torch.float32),
    ((3, 40, 1_200_064), torch.bfloat16)], ids=str)
def test_layer_norm_outputs_past_the_cache(shape, dtype):
    """Outputs over 256 MB, which go past the caches: the bits of calls on parts of the batch."""
    L = _L()
    announce("layer_norm large", shape, dtype)
    g = _gen(sum(shape))
    x, gy = (_randn(g, *shape) - 0.4).to(dtype), _randn(g, *shape).to(dtype)
    assert x.numel() * x.element_size() > 256 << 20
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    y, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    got = L.layer_norm_bwd(x, gamma, stats, gy)
    sums = {k: torch.zeros(shape[1], dtype=torch.float64, device="cuda") for k in ("gamma", "beta")}
    mags = {k: torch.zeros_like(v) for k, v in sums.items()}
    step = max(1, shape[0] // 3)
    for at in range(0, shape[0], step):
        part = slice(at, min(at + step, shape[0]))
        yp, sp = L.layer_norm_fwd(x[part], gamma, beta, EPS)
        assert torch.equal(y[part], yp)
        assert all(torch.equal(a[part], b) for a, b in zip(stats, sp))
        assert torch.equal(got["x"][part], L.layer_norm_bwd(x[part], gamma, sp, gy[part], want=("x",))["x"])
        few = slice(at, min(at + 1, shape[0])) if x.dim() > 2 else slice(at, at + 100)
        _check_fwd(x[few], gamma, beta, y[few], [v[few] for v in stats])
        for b in range(part.start, part.stop, 1 if x.dim() > 2 else 10_000):
            c = slice(b, min(b + (1 if x.dim() > 2 else 10_000), part.stop))
            _, _, _, h, kappa = _norm64(x[c], gamma, beta, EPS)
            up = gy[c].double()
            rows = [0] + list(range(2, x.dim()))
            sums["gamma"] += (up * h).sum(rows)
            mags["gamma"] += (up.abs() * (h.abs() + kappa)).sum(rows)
            sums["beta"] += up.sum(rows)
            mags["beta"] += up.abs().sum(rows)
    for k in ("gamma", "beta"):
        _close("grad_" + k, got[k], sums[k], 128 * U * mags[k])


# ---- tensor lists ------------------------------------------------------------------------------
def _norm_of(ts):
    return math.sqrt(sum(float((t.abs() if t.is_complex() else t).double().square().sum())
                         for t in ts))


def _lists(g, sizes, dtypes, packed):
    """Tensors of the sizes, their dtypes in turn; packed: cut one after another from one byte
    buffer per dtype, at element-size alignment."""
    out = []
    for i, n in enumerate(sizes):
        dt = dtypes[i % len(dtypes)]
        v = (_randn(g, n) * 0.1).to(dt)
        if packed:
            buf = torch.zeros(n + 3, dtype=dt, device="cuda")
            buf[i % 3:i % 3 + n] = v
            v = buf[i % 3:i % 3 + n]
        out.append(v)
    return out


SIZES = [
    [1], [0], [], [8192], [8191, 8193, 1, 0, 7], [100_003], [3, 0, 0, 70_000, 0],
    [1 + (i * 37) % 900 for i in range(250)], [2_000_003, 17, 65_536], [5, 0] * 51,
]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], [torch.float16], TYPES],
                         ids=["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_grad_norm_and_clip(sizes, dtypes, packed):
    L = _L()
    announce("grad_norm", len(sizes), sum(sizes), dtypes, packed)
    g = _gen(len(sizes) + sum(sizes))
    ts = _lists(g, sizes, dtypes, packed)
    norm = _norm_of(ts)
    for max_norm, scale in ((math.inf, 1.0), (max(norm * 0.5, 1e-3), 1.0), (norm * 2 + 1, 8.0),
                            (max(norm / 64, 1e-3), 8.0)):
        rec = L.grad_norm(ts, max_norm, scale).double().tolist()
        want = norm / scale
        factor = (1.0 if want <= max_norm else max_norm / want) / scale
        assert abs(rec[0] - want) <= 4 * U * want
        assert abs(rec[1] - factor) <= 4 * U * factor
        assert L.grad_norm(ts, max_norm, scale).double().tolist() == rec
        outs = [torch.full_like(t, 5.0) for t in ts]
        wide = [torch.full(t.shape, 5.0, device="cuda") for t in ts]
        assert L.clip_grad_norm(ts, max_norm, scale, out=outs).double().tolist() == rec
        assert L.clip_grad_norm(ts, max_norm, scale, out=wide).double().tolist() == rec
        for t, o, f in zip(ts, outs, wide):
            exact = t.double() * factor
            _close("clipped f32", f, exact, 4 * U * exact.abs() + TINY[torch.float32])
            _close("clipped", o, exact, (4 * U + ROUND[t.dtype]) * exact.abs() + TINY[t.dtype])
        copies = [t.clone() for t in ts]
        L.clip_grad_norm(copies, max_norm, scale)
        assert all(torch.equal(a, b) for a, b in zip(copies, outs))


def test_clip_leaves_neighbours_alone():
    L = _L()
    announce("clip neighbours")
    for dt in TYPES:
        buf = torch.ones(40_000, dtype=dt, device="cuda")
        cuts = [buf[1:2], buf[5:5 + 8191], buf[9001:9001 + 17_003], buf[30_000:30_007]]
        keep = torch.ones_like(buf, dtype=torch.bool)
        for c in cuts:
            at = c.storage_offset()
            keep[at:at + c.numel()] = False
        L.clip_grad_norm(cuts, 1.0)
        assert bool((buf[keep] == 1).all()) and bool((buf[~keep] < 1).all())


def test_grad_norm_range_and_non_finite():
    L = _L()
    announce("grad_norm range")
    for size in (1e30, 1e-30, 3e38, 1e-42):
        t = torch.full((5000,), size, device="cuda")
        n = float(t[0].double()) * math.sqrt(5000)
        rec = L.grad_norm([t], 1.0).double().tolist()
        if n < 3.4e38:
            assert abs(rec[0] - n) <= 4 * U * n + 2.0 ** -149
        else:
            assert rec[0] == math.inf
        assert abs(rec[1] - min(1.0, 1.0 / n)) <= 4 * U * min(1.0, 1.0 / n) + 2.0 ** -149
    for value in (math.inf, -math.inf, math.nan):
        for dt in TYPES:
            ts = [torch.ones(300, dtype=dt, device="cuda"), torch.ones(9001, dtype=dt,
                                                                      device="cuda")]
            ts[1][9000] = value
            rec = L.clip_grad_norm(ts, 1.0).tolist()
            assert not math.isfinite(rec[0]) and math.isnan(rec[1])
            assert all(bool(t.isnan().all()) for t in ts)
    z = [torch.zeros(100, device="cuda")]
    assert L.clip_grad_norm(z, 1.0, 4.0).tolist() == [0.0, 0.25] and not z[0].any()


def test_grad_norm_complex_and_repeated():
    L = _L()
    announce("grad_norm complex")
    g = _gen(8)
    w = torch.complex(_randn(g, 3, 5, 7), _randn(g, 3, 5, 7))
    norm = _norm_of([w, w])
    rec = L.grad_norm([w, w]).tolist()  # listed twice, counted twice
    assert abs(rec[0] - norm) <= 4 * U * norm and rec[1] == 1.0
    want = w * (0.5 / _norm_of([w]))
    L.clip_grad_norm([w], 0.5)
    assert float((w - want).abs().max()) <= 8 * U * float(want.abs().max())


@pytest.mark.parametrize("dtype,wide", [(torch.float32, False), (torch.bfloat16, False),
                                        (torch.float16, True)], ids=str)
def test_clip_past_the_cache(dtype, wide):
    """Outputs over 256 MB, which go past the caches."""
    L = _L()
    announce("clip large", dtype, wide)
    g = _gen(9)
    ts = [(_randn(g, n) * 0.1).to(dtype) for n in (50_000_003, 1, 90_000_001, 4097)]
    outs = [torch.empty(t.shape, dtype=torch.float32 if wide else dtype, device="cuda") for t in ts]
    assert sum(o.numel() * o.element_size() for o in outs) > 256 << 20
    norm = _norm_of(ts)
    rec = L.clip_grad_norm(ts, norm / 2, 8.0, out=outs).double().tolist()
    # norm / 8 stays below norm / 2: the factor is the scale's, exact
    assert abs(rec[0] - norm / 8) <= 4 * U * norm / 8 and rec[1] == 0.125
    for t, o in zip(ts, outs):
        assert torch.equal(o, (t.float() * 0.125).to(o.dtype))
    L.clip_grad_norm(ts, norm / 2, 8.0)
    for t, o in zip(ts, outs):
        assert torch.equal(t, o.to(dtype))


def test_grad_norm_past_32_bits():
    L = _L()
    announce("grad_norm long")
    n = (1 << 32) + 70_001
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[0], t[n - 1], t[1 << 32] = 3.0, 4.0, 12.0
    rec = L.clip_grad_norm([t], 6.5).tolist()
    assert rec == [13.0, 0.5]
    assert (float(t[0]), float(t[n - 1]), float(t[1 << 32])) == (1.5, 2.0, 6.0)


def _adamw64(p, g, m, v, t, lr, b1, b2, eps, wd, f):
    g = g.double() * f
    m1 = b1 * m.double() + (1 - b1) * g
    v1 = b2 * v.double() + (1 - b2) * g * g
    up = (m1 / (1 - b1 ** t)) / (torch.sqrt(v1 / (1 - b2 ** t)) + eps)
    return p.double() * (1 - lr * wd) - lr * up, m1, v1, up


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtypes", [[torch.float32], [torch.bfloat16], TYPES],
                         ids=["f32", "bf16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{sum(s)}")
def test_adamw(sizes, dtypes, packed):
    L = _L()
    announce("adamw", len(sizes), sum(sizes), dtypes, packed)
    g = _gen(sum(sizes))
    for step, lr, (b1, b2), eps, wd, rec in (
            (1, 1e-2, (0.9, 0.999), 1e-8, 0.0, None), (7, 1e-3, (0.9, 0.95), 1e-6, 0.1, 0.25),
            (1_000_000, 3e-4, (0.0, 0.5), 0.0, 0.01, 1.0)):
        ps, ms = (_lists(g, sizes, [torch.float32], packed) for _ in range(2))
        vs = [v.square_() + 1e-4 for v in _lists(g, sizes, [torch.float32], packed)]
        gs = _lists(g, sizes, dtypes, packed)
        record = None if rec is None else torch.tensor([9.0, rec], device="cuda")
        want = [_adamw64(*q, step, lr, b1, b2, eps, wd, 1.0 if rec is None else rec)
                for q in zip(ps, gs, ms, vs)]
        old = [[t.clone().double() for t in ts] for ts in (ps, gs, ms)]
        L.adamw(ps, gs, ms, vs, step, lr, (b1, b2), eps, wd, record=record)
        for i, (p1, m1, v1, up) in enumerate(want):
            f = 1.0 if rec is None else rec
            # the first moment may cancel: its magnitude is that of its two terms
            mag = b1 * old[2][i].abs() + (1 - b1) * old[1][i].abs() * f
            _close("exp_avg", ms[i], m1, 4 * U * mag)
            _close("exp_avg_sq", vs[i], v1, 6 * U * v1)
            den = torch.sqrt(v1 / (1 - b2 ** step)) + eps
            _close("param", ps[i], p1, 4 * U * old[0][i].abs()
                   + lr * 24 * U * (mag / (1 - b1 ** step)) / den)


def test_adamw_skips_after_non_finite_gradients():
    L = _L()
    announce("adamw skip")
    g = _gen(1)
    p, m, v = (_randn(g, 20_000) for _ in range(3))
    keep = [t.clone() for t in (p, m, v)]
    grad = torch.ones(20_000, device="cuda")
    grad[77] = math.inf
    rec = L.grad_norm([grad], 1.0)
    L.adamw([p], [grad], [m], [v], 3, 1e-2, record=rec)
    assert all(torch.equal(a, b) for a, b in zip((p, m, v), keep))


def test_adamw_complex_parameters():
    L = _L()
    announce("adamw complex")
    g = _gen(4)
    w, gw = (torch.complex(_randn(g, 4, 9), _randn(g, 4, 9)) for _ in range(2))
    p = torch.view_as_real(w).clone()
    m, v = torch.zeros_like(p), torch.zeros_like(p)
    mw, vw = torch.zeros_like(w), torch.zeros_like(w)
    L.adamw([p], [torch.view_as_real(gw).contiguous()], [m], [v], 1, 1e-2)
    L.adamw([w], [gw], [mw], [vw], 1, 1e-2)
    assert torch.equal(torch.view_as_real(w), p) and torch.equal(torch.view_as_real(mw), m)


def test_refusals():
    """What needs a GPU to be asked: wrong shapes, lists that do not match."""
    L = _L()
    announce("train ops refusals")
    x = torch.zeros(4, 8, 6, device="cuda")
    st = torch.zeros(2, 4, 6, device="cuda")
    with pytest.raises(ValueError, match="gamma"):
        L.layer_norm_fwd(x, torch.ones(7, device="cuda"))
    with pytest.raises(ValueError, match="gamma"):
        L.layer_norm_fwd(x, torch.ones(8))
    with pytest.raises(ValueError, match="out"):
        L.layer_norm_fwd(x, out=x[:2])
    with pytest.raises(ValueError, match="stats"):
        L.layer_norm_bwd(x, None, st[:1], x)
    with pytest.raises(ValueError, match="grad_y"):
        L.layer_norm_bwd(x, None, st, x.bfloat16())
    with pytest.raises(ValueError, match="one GPU"):
        L.TensorList([x, x.cpu()])
    with pytest.raises(ValueError, match="float32"):
        L.TensorList([x.double()])
    a, b, h = L.TensorList([x]), L.TensorList([x, x]), L.TensorList([x.half()])
    short, other = L.TensorList([x[:2]]), L.TensorList([x.bfloat16()])
    rec = torch.zeros(2, device="cuda")
    for grads, out in ((a, b), (a, short), (a, h), (h, other)):
        with pytest.raises(L.FnoError):
            L.clip_grad_norm(grads, 1.0, out=out)
    same = L.fno_tensor(x.data_ptr(), 4, 1, 0), L.fno_tensor(x.data_ptr(), 4, 0, 0)
    for bad in (0.0, -1.0, math.nan):
        with pytest.raises(L.FnoError):
            L.grad_norm(a, bad)
        if bad != 1.0:
            with pytest.raises(L.FnoError):
                L.grad_norm(a, 1.0, bad)
    with pytest.raises(L.FnoError):
        L.grad_norm(a, 1.0, math.inf)
    with pytest.raises(L.FnoError, match="workspace"):
        L.grad_norm(a, 1.0, ws=torch.empty(0, dtype=torch.uint8, device="cuda"))
    with pytest.raises(L.FnoError, match="workspace"):
        L.grad_norm(a, 1.0, ws=torch.empty(4, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="record"):
        L.grad_norm(a, record=rec[:1])
    with pytest.raises(ValueError, match="record"):
        L.adamw(a, a, a, a, 1, 1e-3, record=rec.half())
    for lists in ((a, b, a, a), (a, a, b, a), (a, a, a, b), (a, short, a, a), (a, a, short, a)):
        with pytest.raises(L.FnoError, match="another number"):
            L.adamw(*lists, 1, 1e-3)
    for lists in ((h, h, a, a), (a, a, h, a), (a, a, a, h)):
        with pytest.raises(L.FnoError, match="float32"):
            L.adamw(*lists, 1, 1e-3)
    # a half gradient cannot widen over itself
    tables = [torch.empty(4096, dtype=torch.uint8, device="cuda") for _ in same]
    import ctypes
    handles = []
    for t, e in zip(tables, same):
        handles.append(L.fno_tensor_list_create(1, ctypes.addressof(e), t.data_ptr(), 4096,
                                                torch.cuda.current_stream().cuda_stream))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    assert L._lib.fno_clip_grad_norm(handles[0], handles[1], 1.0, 1.0, rec.data_ptr(),
                                     ws.data_ptr(), ws.numel(), None) == L.FNO_ERR_INVALID_ARGUMENT
    for hd in handles:
        L.fno_tensor_list_destroy(hd)
    torch.cuda.synchronize()
    assert not x.any() and not rec.any()


# ---- streams and graphs ------------------------------------------------------------------------
def _everything(L, s):
    y, stats = L.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS, out=s["y"], stats=s["stats"])
    gr = L.layer_norm_bwd(s["x"], s["gamma"], s["stats"], s["gy"], out=s["grads"], ws=s["ws"])
    assert gr["gamma"] is s["grads"]["gamma"]
    rec = L.clip_grad_norm(s["lists"][0], 0.5, out=s["lists"][1], record=s["record"],
                           ws=s["ws2"])
    L.adamw(*s["lists"][2:], 1, 1e-2, record=rec)


def _state(L, seed):
    g = _gen(seed)
    x = _randn(g, 2, 20, 333)
    s = {"x": x, "gy": _randn(g, *x.shape), "gamma": 1 + 0.1 * _randn(g, 20),
         "beta": 0.1 * _randn(g, 20), "y": torch.empty_like(x),
         "stats": torch.empty(2, 2, 333, device="cuda"),
         "grads": {"x": torch.empty_like(x), "gamma": torch.empty(20, device="cuda"),
                   "beta": torch.empty(20, device="cuda")},
         "half": _randn(g, 30_001).half(), "record": torch.empty(2, device="cuda"),
         "ws": torch.empty(1 << 20, dtype=torch.uint8, device="cuda"),
         "ws2": torch.empty(1 << 20, dtype=torch.uint8, device="cuda")}
    s["clipped"] = [torch.empty(20, device="cuda"), torch.empty(20, device="cuda"),
                    torch.empty(30_001, device="cuda")]
    s["m"], s["v"] = ([torch.zeros(20, device="cuda") for _ in range(2)] for _ in range(2))
    s["lists"] = [L.TensorList(t) for t in (
        [s["grads"]["gamma"], s["grads"]["beta"], s["half"]], s["clipped"],
        [s["gamma"], s["beta"]], s["clipped"][:2], s["m"], s["v"])]
    return s


def _outputs(s):
    return [s["y"], s["stats"], s["record"], s["gamma"], s["beta"]] + list(s["grads"].values()) \
        + s["clipped"] + s["m"] + s["v"]


def test_side_stream():
    L = _L()
    announce("train ops on a side stream")
    a, b = _state(L, 6), _state(L, 6)
    _everything(L, a)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(L, b)
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(_outputs(a), _outputs(b)))


def test_graph_replays_match_eager():
    L = _L()
    announce("train ops in a graph")
    eager, cap = _state(L, 7), _state(L, 7)
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _everything(L, _state(L, 8))
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(L, cap)
        with pytest.raises(L.FnoError, match="capture"):
            L.TensorList([cap["x"]])
    for k in range(4):
        x = _randn(_gen(40 + k), 2, 20, 333)
        eager["x"].copy_(x)
        cap["x"].copy_(x)
        _everything(L, eager)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(_outputs(eager), _outputs(cap))), k


def test_norm_workspace_refused():
    """A workspace that is not packed memory of the fields' device; no call goes out."""
    L = _L()
    announce("layer_norm workspace refusals")
    x, st = torch.zeros(2, 8, 1 << 16, device="cuda"), torch.zeros(2, 2, 1 << 16, device="cuda")
    for ws in (torch.zeros(1 << 20, dtype=torch.uint8),
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 20),
               torch.zeros(2 << 20, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError, match="ws"):
            L.layer_norm_bwd(x, None, st, x, ws=ws)


def test_layer_norm_more_channels_than_a_launch_has_threads():
    """From 2^29 channels on the weight gradients have more columns than a launch of 64 to a work-group
    has threads for (2^32); the header allows up to 2^31."""
    L = _L()
    announce("layer_norm very long rows")
    c = (1 << 29) + 67
    out = {"gamma": torch.full((c,), 9.0, device="cuda")}
    none = torch.empty((0, c), dtype=torch.bfloat16, device="cuda")
    L.layer_norm_bwd(none, None, none.new_empty((2, 0), dtype=torch.float32), none, want=(), out=out)
    assert not out["gamma"].any()
    part = torch.randn(1 << 20, generator=_gen(3), device="cuda").bfloat16()
    x = torch.empty((1, c), dtype=torch.bfloat16, device="cuda")
    gy = torch.empty_like(x)
    ends = (slice(0, 1 << 20), slice(c - (1 << 20), c))
    x.zero_(), gy.zero_()
    for s in ends:
        x[0, s], gy[0, s] = part, part.flip(0)
    stats = torch.tensor([[0.25], [2.0]], device="cuda")
    got = L.layer_norm_bwd(x, None, stats, gy, want=("beta",), out=out)
    for s in ends:
        # one row: each sum is one product, of exact factors but for the rounding of x - mean
        want = part.flip(0).double() * (part.double() - 0.25) * 2.0
        _close("grad_gamma", got["gamma"][s], want, 4 * U * want.abs())
        assert torch.equal(got["beta"][s], part.flip(0).float())
    assert not got["beta"][1 << 20:c - (1 << 20)].any()


def test_layer_norm_most_channels():
    """One row of 2^31 - 1 entries, the most there may be: an index of its last vector's bias sums
    passes 31 bits."""
    L = _L()
    announce("layer_norm longest row")
    c = (1 << 31) - 1
    part = torch.randn(1 << 20, generator=_gen(5), device="cuda").bfloat16()
    x = torch.zeros((1, c), dtype=torch.bfloat16, device="cuda")
    gy = torch.zeros_like(x)
    ends = (slice(0, 1 << 20), slice(c - (1 << 20), c))
    for s in ends:
        gy[0, s] = part
    stats = torch.tensor([[0.25], [2.0]], device="cuda")
    got = L.layer_norm_bwd(x, None, stats, gy, want=("beta",))["beta"]
    for s in ends:
        assert torch.equal(got[s], part.float())
    assert int(got.count_nonzero()) == 2 * int(part.count_nonzero())


@pytest.mark.parametrize("lr,wd", [(2e-6, 0.01), (1e-5, 0.01), (3e-5, 0.02)])
def test_adamw_small_decay_counts(lr, wd):
    """A decay below a parameter's rounding still counts on average: rounding p - lr wd p - step once
    is as often up as down, where a factor 1 - lr wd, rounded to float32 by itself, is off by up to
    2^-25 for every parameter alike (at lr wd = 2e-8 by all of it).  Each result is off by its own
    rounding, at most 2^-24 (parameters in [1, 2)) and independent between parameters, since the
    steps spread over many roundings: the mean of n errors stays within six times
    2^-24 / sqrt(3 n), plus the steps' own float32 roundings, which are relative to them."""
    L = _L()
    announce("adamw decay", lr, wd)
    g = _gen(31)
    n = 1 << 20
    p = 1 + torch.rand(n, generator=g, device="cuda")
    gr, m = _randn(g, n), _randn(g, n)
    v = _randn(g, n).square() + 0.5
    b1, b2, eps = 0.9, 0.99, 1e-8
    want, _, _, up = _adamw64(p, gr, m, v, 5, lr, b1, b2, eps, wd, 1.0)
    L.adamw([p], [gr], [m], [v], 5, lr, (b1, b2), eps, wd)
    mean = float((p.double() - want).mean())
    bound = 6 * 2.0 ** -24 / math.sqrt(3 * n) + 24 * U * (lr * float(up.abs().mean()) + 2 * lr * wd)
    print(f"    mean error {mean:.3e}, bound {bound:.3e}, decay {lr * wd * 1.5:.3e}", flush=True)
    assert abs(mean) <= bound


@pytest.mark.parametrize("shape", [(3, 64, 1 << 19), (5, 32, 1 << 19), (2, 100, 1 << 19)], ids=str)
def test_layer_norm_outputs_past_the_cache_planes_2mb_apart(shape):
    """As above, where the forward keeps all its waves."""
    test_layer_norm_outputs_past_the_cache(shape, torch.float32)


def test_adamw_takes_finite_gradients_of_a_norm_above_float32():
    """The recorded norm is infinity, the factor 5e-41 (subnormal: to 2^-149 / 5e-41 = 3e-5 of
    itself), and the update is made."""
    L = _L()
    announce("adamw, norm above float32")
    grad = torch.full((5000,), 3e38, device="cuda")
    p, m, v = torch.ones(5000, device="cuda"), torch.zeros(5000, device="cuda"), \
        torch.zeros(5000, device="cuda")
    rec = L.grad_norm([grad], 1.0)
    assert rec[0] == math.inf and bool(rec[1].isfinite())
    L.adamw([p], [grad], [m], [v], 1, 1e-2, (0.9, 0.99), 1e-8, 0.0, record=rec)
    want = 0.1 / math.sqrt(5000)
    _close("exp_avg", m, torch.full_like(m, want, dtype=torch.float64),
           torch.full_like(m, 4e-5 * want, dtype=torch.float64))
    _close("param", p, torch.full_like(p, 0.99, dtype=torch.float64),
           torch.full_like(p, 4 * U, dtype=torch.float64))


def _call_each(L, s, rec, ws):
    """Every operator once, outputs of its own but for the gradient list, which is s's."""
    y, stats = L.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
    gr = L.layer_norm_bwd(s["x"], s["gamma"], stats, s["x"])
    L.grad_norm(s["list"], 0.5, record=rec[0], ws=ws[0])
    clipped = [torch.empty_like(t) for t in s["grads"]]
    L.clip_grad_norm(s["list"], 0.5, out=clipped, record=rec[1], ws=ws[1])
    p, m, v = ([torch.full_like(t, one) for t in s["grads"]] for one in (1.0, 0.0, 0.0))
    L.adamw(p, s["list"], m, v, 1, 1e-2, record=rec[0])
    return [y, stats, *gr.values(), *rec, *clipped, *p, *m, *v]


def test_calls_run_on_the_current_stream():
    """Each stream's inputs are written on it behind some milliseconds of other work, with no
    synchronisation: a call that went out on another stream would read what was there before.  Both
    streams use one tensor list, each with its own workspace and record."""
    L = _L()
    announce("train ops behind a stream's own work")
    g = _gen(12)
    new = {"x": _randn(g, 3, 20, 4001), "gamma": 1 + 0.1 * _randn(g, 20), "beta": _randn(g, 20),
           "grads": [_randn(g, n) for n in (20_011, 5, 70_003)]}
    s = {k: [torch.ones_like(t) for t in v] if isinstance(v, list) else torch.ones_like(v)
         for k, v in new.items()}
    s["list"] = L.TensorList(s["grads"])
    recs = [[torch.zeros(2, device="cuda") for _ in range(2)] for _ in range(3)]
    wss = [[torch.empty(1 << 16, dtype=torch.uint8, device="cuda") for _ in range(2)]
           for _ in range(3)]
    busy = torch.ones(1 << 28, device="cuda")
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    _call_each(L, s, recs[2], wss[2])  # what a process's first calls take is done
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        for _ in range(60):
            busy.mul_(1.0)  # 2 GB each
        for k, v in new.items():
            for d, src in zip(s[k], v) if isinstance(v, list) else [(s[k], v)]:
                d.copy_(src)
        ready = torch.cuda.Event()
        ready.record()
        got_a = _call_each(L, s, recs[0], wss[0])
    still_busy = not ready.query()
    with torch.cuda.stream(b):
        b.wait_event(ready)
        got_b = _call_each(L, s, recs[1], wss[1])
    torch.cuda.synchronize()
    assert still_busy, "the other work was too short to tell streams apart"
    want_new = _call_each(L, s, recs[2], wss[2])
    torch.cuda.synchronize()
    assert all(torch.equal(s[k], new[k]) for k in ("x", "gamma", "beta"))
    for got in (got_a, got_b):
        assert len(got) == len(want_new) and all(torch.equal(p, q) for p, q in zip(got, want_new))


@pytest.mark.parametrize("dtype", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(3, w) for w in (1025, 1032, 1536, 2049, 5000, 9000, 20000)]
                         + [(2, 20, 300), (1, 256, 300), (1, 9000, 5)], ids=str)
def test_layer_norm_of_large_means(shape, dtype):
    """Rows whose mean's square passes float32's range, and from 9000 entries on the sum of their
    squared deviations too, while their variance does not.  Waves that hold none of a row's entries
    (the last one at 1025 to 1536, the half types) add nothing to the joined deviations."""
    L = _L()
    announce("layer_norm large means", shape, dtype)
    g = _gen(shape[1])
    big = 30000.0 if dtype == torch.float16 else 2.5e19
    x = (big * (1 + 0.01 * _randn(g, *shape))).to(dtype)
    gamma, beta = 1 + 0.3 * _randn(g, shape[1]), 0.3 * _randn(g, shape[1])
    gy = _randn(g, *shape).to(dtype)
    y, stats = L.layer_norm_fwd(x, gamma, beta, EPS)
    assert bool(torch.isfinite(y).all())
    _check_fwd(x, gamma, beta, y, stats)
    _check_bwd(x, gamma, gy, L.layer_norm_bwd(x, gamma, stats, gy))
