"""What stands between two blocks of a training stack, as it is measured: the group norm with its
activation and dropout in one pass, over fields [batch, channels, *grid] and channels-last data,
and the dropout by itself with a residual; each forward and backward.

A case is a dict of plain values, `prepare` makes its inputs on the GPU from a seed, and `run` is
one pass.  With `own` false `run` computes in elementary torch operations in float32 and rounds
once at the end; with `own` true it calls the library.  `exact` is the definition in float64.

Dropout takes its mask from a counter: element i of a tensor (in the row-major order of its shape)
is dropped where its 16 bits are below T = round(65536 p), and the rest is multiplied by
65536 / (65536 - T).  The bits are half (i even: the lower) of word (i % 8) / 2 of Philox4x32-10
(Salmon et al., SC 2011) of the counter (i / 8, draw), 64 bits each, under the 64-bit key seed.
"""
import math

import torch

own = False  # set from outside: whether run() calls the library

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}
LOW = 0xffffffff
ACTS = {"none": None, "gelu": "gelu", "silu": "silu"}


def listed():
    def group(name, op, type, batch, channels, groups, points, last, act, p):
        return dict(name=name, op=op, type=type, batch=batch, channels=channels, groups=groups,
                    points=points, last=last, act=act, p=p, gap=0, residual=False)

    def drop(name, op, type, batch, channels, points, gap, residual, p):
        return dict(name=name, op=op, type=type, batch=batch, channels=channels, groups=1,
                    points=points, last=False, act="none", p=p, gap=gap, residual=residual)

    return [
        # ---- group norm, forward
        # one decode step of a small batch, a norm for each head of 64: nothing but latency
        group("group_fwd_heads8", "group_fwd", "bf16", 8, 1024, 16, 1, True, "none", 0.0),
        # one 2D layer of width 20 on 64^2, batch 4
        group("group_fwd_layer2d", "group_fwd", "f32", 4, 20, 4, 64 * 64, False, "gelu", 0.0),
        # channels last on an odd grid, five channels to a group
        group("group_fwd_last_odd", "group_fwd", "f16", 3, 45, 9, 63 * 65, True, "silu", 0.0),
        # channels last of an image-like feature map in half precision
        group("group_fwd_last_map", "group_fwd", "bf16", 8, 128, 32, 256 * 256, True, "silu", 0.0),
        # between two blocks of the 2D training step: 8 x 64 channels x 512^2, with its dropout
        group("group_fwd_train2d", "group_fwd", "f32", 8, 64, 8, 512 * 512, False, "gelu", 0.1),
        # ---- group norm, backward
        # one 2D layer: latency, and the sums for the weights' gradients
        group("group_bwd_layer2d", "group_bwd", "f32", 4, 20, 4, 64 * 64, False, "gelu", 0.1),
        # a training batch of tokens, a norm for each of 32 heads
        group("group_bwd_rows", "group_bwd", "bf16", 8192, 4096, 32, 1, True, "none", 0.0),
        # a channels-last feature map of few entries and many channels
        group("group_bwd_last_map", "group_bwd", "f16", 4, 320, 32, 96 * 96, True, "silu", 0.1),
        # between two blocks of the 3D training step: 2 x 20 channels x 128^3
        group("group_bwd_train3d", "group_bwd", "f32", 2, 20, 5, 128 ** 3, False, "gelu", 0.0),
        # ---- dropout
        # a few tokens onto their residual: latency
        drop("drop_fwd_tokens8", "drop_fwd", "bf16", 8, 1024, 1, 0, True, 0.1),
        # rows cut out of wider ones, an odd width
        drop("drop_bwd_rows_odd", "drop_bwd", "f16", 1003, 1537, 1, 7, False, 0.25),
        # a block's output in the 2D training step, onto the residual
        drop("drop_fwd_train2d", "drop_fwd", "bf16", 8, 64, 512 * 512, 0, True, 0.1),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["group_fwd", "group_bwd", "group_fwd", "group_bwd", "drop_fwd", "drop_bwd"])
    c = dict(op=op, type=rng.choice(["f32", "bf16", "f16"]), groups=1, last=False, act="none",
             gap=0, residual=False)
    if op.startswith("drop"):
        c["channels"] = _log(rng, 3, 8192)
        c["batch"] = _log(rng, 1, 16)
        c["points"] = _log(rng, 1, max(2, 100_000_000 // (c["channels"] * c["batch"])))
        c["gap"] = rng.choice([0, 0, rng.randrange(1, 70)])
        c["residual"] = op == "drop_fwd" and rng.random() < 0.5
        c["p"] = round(rng.uniform(0.02, 0.6), 3)
        return c
    c["act"] = rng.choice(["none", "gelu", "silu"])
    c["p"] = rng.choice([0.0, round(rng.uniform(0.02, 0.5), 3)])
    c["groups"] = rng.choice([1, 2, 4, 5, 8, 16, 32, rng.randrange(1, 33)])
    form = rng.choice(["field", "last", "tokens", "field", "last"])
    if form == "tokens":  # rows of heads
        c["channels"] = c["groups"] * _log(rng, 16, 512)
        c["points"], c["last"] = 1, True
        c["batch"] = _log(rng, 1, max(2, min(32768, 40_000_000 // c["channels"])))
        c["gap"] = rng.choice([0, 0, rng.randrange(1, 70)])
        return c
    c["channels"] = c["groups"] * _log(rng, 1, max(2, 640 // c["groups"]))
    c["batch"] = _log(rng, 1, 32)
    c["points"] = _log(rng, 30, max(31, 60_000_000 // (c["channels"] * c["batch"])))
    c["last"] = form == "last"
    return c


def _shape(case):
    b, c, p = case["batch"], case["channels"], case["points"]
    if p == 1:
        return (b, c)
    return (b, p, c) if case["last"] else (b, c, p)


def _per_channel(case, v):
    """A vector [channels] as it broadcasts over the case's data."""
    return v if case["last"] or case["points"] == 1 else v.unsqueeze(1)


def _grouped(case, x):
    """Data as [batch, groups, rest] or [batch, points, groups, rest], and the axes of a norm."""
    g = case["groups"]
    if case["last"] and case["points"] > 1:
        return x.unflatten(2, (g, -1)), (1, 3)
    return x.reshape(x.shape[0], g, -1), (2,)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    kind, shape, c = TYPES[case["type"]], _shape(case), case["channels"]

    def data(at, by):
        """Activations with a mean and a scale of their own per channel, entries `gap` apart."""
        n = math.prod(shape[1:])
        wide = torch.empty((shape[0], n + case["gap"]), dtype=kind, device="cuda")
        step = max(1, (1 << 28) // n)
        for i in range(0, shape[0], step):
            part = (min(step, shape[0] - i),) + shape[1:]
            wide[i:i + step, :n] = (normal(*part) * by + at).reshape(part[0], n).to(kind)
        return wide[:, :n].unflatten(1, shape[1:])

    s = {"case": case, "seed": (0x5eed0000 + seed * 0x100000001) % 2 ** 63, "draw": 3,
         # the draws that the training run has taken so far: a count that lives on the device
         "counter": torch.full((1,), 8 * seed, dtype=torch.int64, device="cuda"),
         "x": data(_per_channel(case, normal(c)), _per_channel(case, torch.exp(0.5 * normal(c))))}
    if case["residual"]:
        s["residual"] = data(0.0, 1.0)
    if case["op"].startswith("group"):
        s["gamma"], s["beta"] = 1.0 + 0.2 * normal(c), 0.2 * normal(c)
    if case["op"] == "group_bwd":
        x, over = _grouped(case, s["x"].float())
        mean = x.mean(over, keepdim=True)
        rstd = ((x - mean).square().mean(over) + EPS).rsqrt()
        s["stats"] = torch.stack([mean.reshape(rstd.shape), rstd])
        s["grad_y"] = data(0.0, 1.0)
    if own:
        from fno_spectral_convolution_amd import binding
        s["drop"] = binding.Dropout(case["p"], s["seed"], s["draw"], s["counter"]) \
            if case["p"] else None
    return s


def _threshold(case):
    return round(case["p"] * 65536)


def _plain_keep(s, shape):
    """The mask: True where an element is kept."""
    n = math.prod(shape)
    at = torch.arange((n + 7) // 8, device="cuda")
    count = s["counter"][0] + s["draw"]
    a, b, c, d = at & LOW, at >> 32, count & LOW, count >> 32
    k0, k1 = s["seed"] & LOW, s["seed"] >> 32
    for _ in range(10):
        p, q = a * 0xD2511F53, c * 0xCD9E8D57  # 64-bit products, their top bit the sign
        a, b, c, d = (q >> 32 & LOW) ^ b ^ k0, q & LOW, (p >> 32 & LOW) ^ d ^ k1, p & LOW
        k0, k1 = (k0 + 0x9E3779B9) & LOW, (k1 + 0xBB67AE85) & LOW
    words = torch.stack([a, b, c, d], 1)
    bits = torch.stack([words & 0xffff, words >> 16], 2).reshape(-1)[:n]
    return (bits >= _threshold(s["case"])).view(shape)


def _plain_drop(s, v):
    if not s["case"]["p"]:
        return v
    return torch.where(_plain_keep(s, v.shape), v * (65536 / (65536 - _threshold(s["case"]))), 0.0)


def _plain_norm(s, x, mean, rstd):
    """(x - mean) rstd, and that times gamma plus beta."""
    case = s["case"]
    parts, over = _grouped(case, x)
    h = ((parts - mean) * rstd).reshape(x.shape)
    return h, h * _per_channel(case, s["gamma"]) + _per_channel(case, s["beta"])


def _plain_group_fwd(s):
    case = s["case"]
    x = s["x"].float()
    parts, over = _grouped(case, x)
    mean = parts.mean(over, keepdim=True)
    rstd = ((parts - mean).square().mean(over, keepdim=True) + EPS).rsqrt()
    u = _plain_norm(s, x, mean, rstd)[1]
    if case["act"] == "gelu":
        u = 0.5 * u * (1.0 + torch.erf(u * math.sqrt(0.5)))
    elif case["act"] == "silu":
        u = u / (1.0 + torch.exp(-u))
    flat = (case["batch"], case["groups"])
    return {"y": _plain_drop(s, u).to(s["x"].dtype),
            "stats": torch.stack([mean.reshape(flat), rstd.reshape(flat)])}


def _plain_group_bwd(s):
    case = s["case"]
    x, g = s["x"].float(), _plain_drop(s, s["grad_y"].float())
    parts, over = _grouped(case, x)
    side = [n if i not in over else 1 for i, n in enumerate(parts.shape)]
    mean, rstd = s["stats"][0].view(side), s["stats"][1].view(side)
    h, u = _plain_norm(s, x, mean, rstd)
    if case["act"] == "gelu":
        g = g * (0.5 * (1.0 + torch.erf(u * math.sqrt(0.5))) +
                 u * torch.exp(-0.5 * u * u) * math.sqrt(0.5 / math.pi))
    elif case["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-u))
        g = g * sig * (1.0 + u * (1.0 - sig))
    axis = -1 if case["last"] or case["points"] == 1 else 1
    rows = [i for i in range(x.dim()) if i != axis % x.dim()]
    grads = {"gamma": (g * h).sum(rows), "beta": g.sum(rows)}
    g = _grouped(case, g * _per_channel(case, s["gamma"]))[0]
    h = _grouped(case, h)[0]
    gx = (g - g.mean(over, keepdim=True) - h * (g * h).mean(over, keepdim=True)) * rstd
    return {"x": gx.reshape(x.shape).to(s["x"].dtype), **grads}


def _plain_drop_pass(s):
    y = _plain_drop(s, s["x"].float())
    if s["case"]["residual"]:
        y = y + s["residual"].float()
    return y.to(s["x"].dtype)


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"group_fwd": _plain_group_fwd, "group_bwd": _plain_group_bwd,
                "drop_fwd": _plain_drop_pass, "drop_bwd": _plain_drop_pass}[op](s)
    from fno_spectral_convolution_amd import binding
    if op == "drop_fwd":
        return binding.dropout_fwd(s["x"], s["drop"], s.get("residual"))
    if op == "drop_bwd":  # x: the gradient at the output
        return binding.dropout_bwd(s["x"], s["drop"])
    if op == "group_fwd":
        y, stats = binding.group_norm_fwd(s["x"], case["groups"], s["gamma"], s["beta"],
                                          ACTS[case["act"]], EPS, case["last"], s["drop"])
        return {"y": y, "stats": stats}
    return binding.group_norm_bwd(s["x"], case["groups"], s["gamma"], s["beta"], s["stats"],
                                  s["grad_y"], ACTS[case["act"]], case["last"], s["drop"])


def work(case):
    w, c = WIDTH[case["type"]], case["channels"]
    n, sides = case["batch"] * c * case["points"], case["batch"] * case["groups"]
    if case["op"].startswith("drop"):  # x, the residual; y
        return {"bytes": (3 if case["residual"] else 2) * n * w, "flops": 2 * n}
    if case["op"] == "group_fwd":  # x; gamma, beta; y; the statistics
        return {"bytes": 2 * n * w + 8 * c + 8 * sides, "flops": 12 * n}
    # x, grad_y; gamma, beta, the statistics; grad_x; grad_gamma, grad_beta
    return {"bytes": 3 * n * w + 16 * c + 8 * sides, "flops": 20 * n}


def _exact_multiplier(s, n):
    """What dropout multiplies n elements by, 0 or the scale, from products of 16-bit halves."""
    t, seed = _threshold(s["case"]), s["seed"]
    if t == 0:
        return torch.ones(n, dtype=torch.float64, device="cuda")
    blocks = torch.arange(-(-n // 8), dtype=torch.int64, device="cuda")
    number = int(s["counter"]) + s["draw"]
    x = [blocks % 2 ** 32, blocks // 2 ** 32, torch.full_like(blocks, number % 2 ** 32),
         torch.full_like(blocks, number // 2 ** 32)]

    def times(v, m):
        """High and low word of a product of two 32-bit numbers."""
        low, high = v * (m % 65536), v * (m // 65536)
        mid = low // 65536 + high
        return mid // 65536, mid % 65536 * 65536 + low % 65536

    for r in range(10):
        key = ((seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32)
        h0, l0 = times(x[0], 0xD2511F53)
        h1, l1 = times(x[2], 0xCD9E8D57)
        x = [torch.bitwise_xor(torch.bitwise_xor(h1, x[1]), key[0]), l1,
             torch.bitwise_xor(torch.bitwise_xor(h0, x[3]), key[1]), l0]
    out = torch.empty((blocks.numel(), 8), dtype=torch.float64, device="cuda")
    for e in range(8):
        half = x[e // 2] % 65536 if e % 2 == 0 else x[e // 2] // 65536
        out[:, e] = (half >= t) * (65536 / (65536 - t))
    return out.view(-1)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    shape = s["x"].shape
    keep = _exact_multiplier(s, s["x"].numel()).view(shape)
    if case["op"].startswith("drop"):
        y = s["x"].double() * keep
        return y + s["residual"].double() if case["residual"] else y
    # everything as [batch, groups, channels of a group, points]
    b, c, k, p = case["batch"], case["channels"], case["groups"], case["points"]

    def split(t):
        t = t.double()
        if case["last"] and p > 1:
            t = t.transpose(1, 2)
        return t.reshape(b, k, c // k, p)

    def join(t):
        t = t.reshape(b, c, p)
        return (t.transpose(1, 2) if case["last"] and p > 1 else t).reshape(shape)

    x, m = split(s["x"]), c // k * p
    mu = x.sum((2, 3), keepdim=True) / m
    sigma = torch.sqrt(((x - mu) ** 2).sum((2, 3), keepdim=True) / m + EPS)
    z = (x - mu) / sigma
    del x
    gamma, beta = (s[n].double().view(1, k, c // k, 1) for n in ("gamma", "beta"))
    u = gamma * z + beta
    if case["act"] == "gelu":  # u times the normal distribution function, and its density
        cdf = torch.special.ndtr(u)
        slope = cdf + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
        u = u * cdf
    elif case["act"] == "silu":
        sig = torch.sigmoid(u)
        slope = sig + u * sig * (1 - sig)
        u = u * sig
    else:
        slope = 1.0
    if case["op"] == "group_fwd":
        return {"y": join(u) * keep, "stats": torch.stack([mu.view(b, k), 1 / sigma.view(b, k)])}
    up = split(s["grad_y"].double() * keep) * slope
    grads = {"gamma": (up * z).sum((0, 3)).view(c), "beta": up.sum((0, 3)).view(c)}
    up = up * gamma
    # the Jacobian of z = (x - mu) / sigma, group by group: (1 - 1/m - z z^T / m) / sigma
    along = (up * z).sum((2, 3), keepdim=True) / m
    grads["x"] = join((up - up.sum((2, 3), keepdim=True) / m - z * along) / sigma)
    return grads
