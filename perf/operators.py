"""The training operators of a stack, as they are measured: the layer norm's forward and backward
pass, the global gradient norm with clipping, and the AdamW update that takes its clipping.

A case is a dict of plain values, `prepare` makes its inputs on the GPU from a seed, and `run` is
one pass.  With `own` false `run` computes in elementary torch operations in float32 and rounds
once at the end; with `own` true it calls the library.  `exact` is the definition in float64.
"""
import math
import random

import torch

own = False  # set from outside: whether run() calls the library

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
WIDTH = {"f32": 4, "bf16": 2, "f16": 2}

# Real tensor lists: the element counts (complex weights as two numbers an entry) of one block of
# the workloads of that name, and the number of blocks.  Norm weights and biases come after the
# bypass and its bias.
MODELS = {
    # one 2D layer of width 20 with 12 x 12 modes
    "layer2d_64": ((2 * 20 * 20 * 12 * 12 * 2, 400, 20, 20, 20), 1),
    # the 2D training step's factorised weights: core 32 x 32 x 32 x 16 and its four factors
    "train2d_512_tfno": ((32 * 32 * 32 * 16 * 2, 64 * 32 * 2, 64 * 32 * 2, 64 * 32 * 2,
                          32 * 16 * 2, 64 * 64, 64, 64, 64), 4),
    # the 3D training step: four corners of 20 x 20 channels and 16^3 modes
    "train3d_128": ((4 * 20 * 20 * 16 ** 3 * 2, 400, 20, 20, 20), 4),
}

LR, BETAS, ADAM_EPS, DECAY = 1e-3, (0.9, 0.95), 1e-8, 0.01


def listed():
    return [
        # ---- layer norm, forward: rows of tokens (points = 1) and fields [batch, channels, points]
        # one decode step of a small batch: nothing but latency
        dict(name="norm_fwd_tokens8", op="norm_fwd", type="bf16", batch=8, channels=1024, points=1,
             gap=0),
        # a ragged prompt with an odd width, rows cut out of wider ones
        dict(name="norm_fwd_rows_odd", op="norm_fwd", type="f16", batch=1003, channels=1537,
             points=1, gap=7),
        # between two blocks of the 2D training step: 8 x 64 channels x 512^2
        dict(name="norm_fwd_train2d", op="norm_fwd", type="f32", batch=8, channels=64,
             points=512 * 512, gap=0),
        # ---- layer norm, backward
        # a few tokens: latency of the row pass and of the weight gradient's reduction
        dict(name="norm_bwd_tokens", op="norm_bwd", type="f32", batch=48, channels=640, points=1,
             gap=0),
        # a training batch of tokens
        dict(name="norm_bwd_rows", op="norm_bwd", type="bf16", batch=8192, channels=4096, points=1,
             gap=0),
        # a 2D field of an odd grid (63 x 65)
        dict(name="norm_bwd_field_odd", op="norm_bwd", type="f32", batch=5, channels=20,
             points=63 * 65, gap=0),
        # between two blocks of the 3D training step: 2 x 20 channels x 128^3
        dict(name="norm_bwd_train3d", op="norm_bwd", type="f32", batch=2, channels=20,
             points=128 ** 3, gap=0),
        # ---- gradient norm and clipping, into a second set of buffers (in place the second pass
        # would find nothing left to clip)
        # the factorised 2D training step's 36 gradients
        dict(name="clip_tfno2d", op="clip", type="f32", model="train2d_512_tfno", tensors=0,
             total=0, layout=0, align=1, scale=1.0),
        # many half-precision gradients of odd sizes, packed into one flat buffer; the loss scale is
        # taken out on the way to float32, where they do not underflow
        dict(name="clip_many_f16", op="clip", type="f16", model="", tensors=301, total=150_000_001,
             layout=11, align=1, scale=65536.0),
        # ---- one optimiser step: the gradients' norm, and AdamW on the clipped gradients
        # one 2D layer: latency
        dict(name="adamw_layer2d", op="adamw", type="f32", model="layer2d_64", tensors=0, total=0,
             layout=0, align=1, scale=1.0),
        # many bfloat16 gradients of float32 parameters, each tensor on its own 64-entry boundary
        dict(name="adamw_many_bf16", op="adamw", type="bf16", model="", tensors=147,
             total=30_000_000, layout=12, align=64, scale=1.0),
        # the 3D training step's 20 parameters (52 million numbers)
        dict(name="adamw_train3d", op="adamw", type="f32", model="train3d_128", tensors=0, total=0,
             layout=0, align=1, scale=1.0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "norm_fwd", "norm_bwd", "clip", "adamw"])
    kind = rng.choice(["f32", "bf16", "f16"])
    if op in ("norm_fwd", "norm_bwd"):
        if rng.random() < 0.5:  # tokens
            width = _log(rng, 64, 16384)
            rows = _log(rng, 1, max(2, 40_000_000 // width))
            return dict(op=op, type=kind, batch=rows, channels=width, points=1,
                        gap=rng.choice([0, 0, rng.randrange(1, 70)]))
        channels = rng.choice([rng.randrange(1, 129), 20, 32, 64])
        batch = rng.randrange(1, 17)
        points = _log(rng, 30, max(31, 60_000_000 // (channels * batch)))
        return dict(op=op, type=kind, batch=batch, channels=channels, points=points, gap=0)
    tensors = _log(rng, 1, 500)
    most = 100_000_000 if op == "clip" else 30_000_000
    total = max(4 * tensors, _log(rng, 1000, most))
    return dict(op=op, type=kind, model="", tensors=tensors, total=total,
                layout=rng.randrange(1 << 30), align=rng.choice([1, 1, 64]),
                scale=65536.0 if kind == "f16" else 1.0)


def _sizes(case):
    """Element counts of a case's tensors: a model's own, or `tensors` of them that add up to
    `total`, spread over two to three powers of ten (a model's matrices and its vectors)."""
    if case["model"]:
        block, blocks = MODELS[case["model"]]
        return list(block) * blocks
    r = random.Random(case["layout"])
    share = [math.exp(r.uniform(0.0, 6.0)) for _ in range(case["tensors"])]
    unit = case["total"] / sum(share)
    sizes = [max(1, int(s * unit)) for s in share]
    sizes[0] += max(0, case["total"] - sum(sizes))
    return sizes


def _spans(case):
    """(start, elements) of each tensor in the flat buffer, and the buffer's length."""
    at, spans = 0, []
    for n in _sizes(case):
        spans.append((at, n))
        at = -(-(at + n) // case["align"]) * case["align"]
    return spans, at


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    kind = TYPES[case["type"]]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        b, c, p = case["batch"], case["channels"], case["points"]
        shape = (b, c) if p == 1 else (b, c, p)
        # activations with a mean and a scale of their own per channel
        at, by = normal(1, c, 1), torch.exp(0.5 * normal(1, c, 1))
        wide = torch.empty((b, c * p + case["gap"]), dtype=kind, device="cuda")
        for i in range(0, b, 4096):
            n = min(4096, b - i)
            wide[i:i + n, :c * p] = (normal(n, c, p) * by + at).reshape(n, c * p).to(kind)
        x = wide[:, :c * p].unflatten(1, shape[1:])
        s = {"case": case, "x": x, "gamma": 1.0 + 0.2 * normal(c), "beta": 0.2 * normal(c)}
        if case["op"] == "norm_bwd":
            f = x.float()
            mean = f.mean(1)
            var = (f - mean.unsqueeze(1)).square().mean(1)
            s["stats"] = torch.stack([mean, (var + EPS).rsqrt()])
            s["grad_y"] = normal(*shape).to(kind)
        return s
    spans, length = _spans(case)
    names = ["grad", "out"] if case["op"] == "clip" else ["grad", "param", "exp_avg", "exp_avg_sq"]
    to = kind if case["op"] == "clip" and case["type"] != "f16" else torch.float32
    flat = {"grad": torch.zeros(length, dtype=kind, device="cuda")}
    for start, n in spans:  # a scale of its own for each tensor's gradient
        size = 1e-3 * math.exp(2.0 * random.Random(start + seed).uniform(-1, 1)) / 4
        if case["scale"] != 1.0:
            size *= 1.0 / 64  # far below what half holds without the loss scale
        flat["grad"][start:start + n] = normal(n) * (size * case["scale"])
    for name in names[1:]:
        flat[name] = torch.zeros(length, dtype=to, device="cuda")
    if case["op"] == "adamw":
        for start, n in spans:
            flat["param"][start:start + n] = 0.02 * normal(n)
            flat["exp_avg"][start:start + n] = 3e-4 * normal(n)
            flat["exp_avg_sq"][start:start + n] = (3e-4 * normal(n)).square() + 1e-9
    lists = {k: [v[a:a + n] for a, n in spans] for k, v in flat.items()}
    norm = float(flat["grad"].double().norm()) / case["scale"]
    if own:  # the lists that a training program makes once for its buffers, and keeps
        from fno_spectral_convolution_amd import binding
        lists = {k: binding.TensorList(v) for k, v in lists.items()}
    # some steps are clipped, and some are not
    return {"case": case, "flat": flat, "lists": lists, "step": 100,
            "max_norm": norm * (0.5 if seed % 4 else 2.0)}


def _plain_norm_fwd(s):
    x = s["x"].float()
    side = (1, -1) + (1,) * (x.dim() - 2)
    mean = x.mean(1, keepdim=True)
    off = x - mean
    rstd = (off.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = off * rstd * s["gamma"].view(side) + s["beta"].view(side)
    return {"y": y.to(s["x"].dtype), "stats": torch.stack([mean.squeeze(1), rstd.squeeze(1)])}


def _plain_norm_bwd(s):
    x, gy = s["x"].float(), s["grad_y"].float()
    mean, rstd = s["stats"][0].unsqueeze(1), s["stats"][1].unsqueeze(1)
    xhat = (x - mean) * rstd
    g = gy * s["gamma"].view((1, -1) + (1,) * (x.dim() - 2))
    gx = (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True)) * rstd
    rows = [0] + list(range(2, x.dim()))
    return {"x": gx.to(s["x"].dtype), "gamma": (gy * xhat).sum(rows), "beta": gy.sum(rows)}


def _plain_clip_factor(s):
    """The norm of the gradients without their loss scale, and what clipping multiplies them by."""
    grad, scale = s["flat"]["grad"].float(), s["case"]["scale"]
    norm = grad.square().sum().sqrt() / scale
    return grad, norm, torch.clamp(s["max_norm"] / norm, max=1.0) / scale


def _plain_clip(s):
    grad, norm, factor = _plain_clip_factor(s)
    s["flat"]["out"].copy_(grad * factor)
    return {"out": s["flat"]["out"], "norm": norm}


def _plain_adamw(s):
    grad, norm, factor = _plain_clip_factor(s)
    p, m, v = (s["flat"][k] for k in ("param", "exp_avg", "exp_avg_sq"))
    g = grad * factor
    m.mul_(BETAS[0]).add_(g, alpha=1 - BETAS[0])
    v.mul_(BETAS[1]).add_(g.square(), alpha=1 - BETAS[1])
    by = v.sqrt().div_(math.sqrt(1 - BETAS[1] ** s["step"])).add_(ADAM_EPS)
    p.mul_(1 - LR * DECAY).sub_(m / by, alpha=LR / (1 - BETAS[0] ** s["step"]))
    return {"param": p, "exp_avg": m, "exp_avg_sq": v, "norm": norm}


def run(s):
    op = s["case"]["op"]
    if op == "adamw":
        s["step"] += 1
    if not own:
        return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "clip": _plain_clip,
                "adamw": _plain_adamw}[op](s)
    from fno_spectral_convolution_amd import binding
    if op == "norm_fwd":
        y, stats = binding.layer_norm_fwd(s["x"], s["gamma"], s["beta"], EPS)
        return {"y": y, "stats": stats}
    if op == "norm_bwd":
        return binding.layer_norm_bwd(s["x"], s["gamma"], s["stats"], s["grad_y"])
    at, scale = s["lists"], s["case"]["scale"]
    if op == "clip":
        record = binding.clip_grad_norm(at["grad"], s["max_norm"], scale, out=at["out"])
        return {"out": s["flat"]["out"], "norm": record[0]}
    record = binding.grad_norm(at["grad"], s["max_norm"], scale)
    binding.adamw(at["param"], at["grad"], at["exp_avg"], at["exp_avg_sq"], s["step"], LR, BETAS,
                  ADAM_EPS, DECAY, record=record)
    return {"param": s["flat"]["param"], "exp_avg": s["flat"]["exp_avg"],
            "exp_avg_sq": s["flat"]["exp_avg_sq"], "norm": record[0]}


def work(case):
    w = WIDTH[case["type"]]
    if case["op"] in ("norm_fwd", "norm_bwd"):
        rows = case["batch"] * case["points"]
        n = rows * case["channels"]
        if case["op"] == "norm_fwd":  # x; gamma, beta; y; the statistics
            return {"bytes": 2 * n * w + 8 * case["channels"] + 8 * rows, "flops": 8 * n}
        # x, grad_y; gamma, the statistics; grad_x; grad_gamma, grad_beta
        return {"bytes": 3 * n * w + 12 * case["channels"] + 8 * rows, "flops": 14 * n}
    n = sum(_sizes(case))
    if case["op"] == "clip":  # the gradients, their clipped form
        return {"bytes": n * (w + (2 if case["type"] == "bf16" else 4)) + 4, "flops": 3 * n}
    # the gradients; parameters and both moments read and written
    return {"bytes": n * (w + 24) + 4, "flops": 16 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        d = case["channels"]
        x = s["x"].double().reshape(case["batch"], d, -1)
        gamma, beta = (s[k].double()[None, :, None] for k in ("gamma", "beta"))
        mu = x.sum(1) / d
        sigma = torch.sqrt(((x - mu[:, None]) ** 2).sum(1) / d + EPS)
        z = (x - mu[:, None]) / sigma[:, None]
        if case["op"] == "norm_fwd":
            del x
            return {"y": (gamma * z + beta).reshape(s["x"].shape),
                    "stats": torch.stack([mu, 1 / sigma]).reshape((2,) + s["x"][:, 0].shape)}
        up = s["grad_y"].double().reshape(case["batch"], d, -1)
        grads = {"gamma": (up * z).sum((0, 2)), "beta": up.sum((0, 2))}
        up = up * gamma
        # the Jacobian of z = (x - mu) / sigma, row by row: (1 - 1/d - z z^T / d) / sigma
        along = (up * z).sum(1, keepdim=True) / d
        grads["x"] = ((up - up.sum(1, keepdim=True) / d - z * along) / sigma[:, None]) \
            .reshape(s["x"].shape)
        return grads
    raw = s["flat"]["grad"].double() / case["scale"]
    norm = torch.linalg.vector_norm(raw)
    clipped = raw * min(1.0, s["max_norm"] / float(norm))
    if case["op"] == "clip":
        return {"out": clipped, "norm": norm}
    t = s["step"] + 1
    m = BETAS[0] * s["flat"]["exp_avg"].double() + (1 - BETAS[0]) * clipped
    v = BETAS[1] * s["flat"]["exp_avg_sq"].double() + (1 - BETAS[1]) * clipped ** 2
    unbiased = (m / (1 - BETAS[0] ** t)) / (torch.sqrt(v / (1 - BETAS[1] ** t)) + ADAM_EPS)
    p = s["flat"]["param"].double()
    return {"param": p - LR * DECAY * p - LR * unbiased, "exp_avg": m, "exp_avg_sq": v,
            "norm": norm}
