"""The training operators as a stack uses them: a stack with layer norms against the oracle's
blocks and plain norms in float64, AdamW over its parameters against the formula, and the example
run, whose loss falls."""
import math

import numpy as np
import pytest

import oracle.fno_oracle as O
from fno_spectral_convolution_amd import inputs
from fno_spectral_convolution_amd.configs import F16_LOSS_SCALE, Workload
from tests.gpu_helpers import TOL_F32, announce, check, tol_for

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _norm(z, gamma, beta):
    s = (1, -1) + (1,) * (z.ndim - 2)
    mean = z.mean(1, keepdims=True)
    r = 1.0 / np.sqrt(((z - mean) ** 2).mean(1, keepdims=True) + EPS)
    h = (z - mean) * r
    return gamma.reshape(s) * h + beta.reshape(s), h, r


def _norm_bwd(h, r, gamma, gy):
    s = (1, -1) + (1,) * (h.ndim - 2)
    rows = (0,) + tuple(range(2, h.ndim))
    g = gy * gamma.reshape(s)
    gx = r * (g - g.mean(1, keepdims=True) - h * (g * h).mean(1, keepdims=True))
    return gx, (gy * h).sum(rows), gy.sum(rows)



def _reference(wl, hi):
    """Output, loss and gradients of the normed stack (GELU between norm and block, and last)."""
    tanh, nb = bool(wl.mixed), len(hi["blocks"])
    h, xs, saved = np.asarray(hi["x"], np.float64), [], []
    for i, b in enumerate(hi["blocks"]):
        if i:
            h, hn, r = _norm(h, b["gamma"].astype(np.float64), b["beta"].astype(np.float64))
            saved.append((hn, r))
        xs.append(h)
        f = O.block_fwd(h, b["w"], b["wb"], b["bias"], wl.modes, tanh=tanh, act=i == nb - 1,
                        input_gelu=i > 0)
        h = f["y"]
    out = {"y": h}
    if not wl.train:
        return out
    out["loss"], g = O.mse_loss_grad(h, hi["target"])
    out["grads"] = [None] * nb
    for i in reversed(range(nb)):
        b = hi["blocks"][i]
        k = O.block_bwd(xs[i], b["w"], b["wb"], b["bias"], wl.modes, g, tanh=tanh,
                        act=i == nb - 1, input_gelu=i > 0)
        out["grads"][i] = {"w": k["grad_w"], "wb": k["grad_wb"], "bias": k["grad_bias"]}
        g = k["grad_x"]
        if i:
            hn, r = saved[i - 1]
            g, gg, gb = _norm_bwd(hn, r, b["gamma"].astype(np.float64), g)
            out["grads"][i].update(gamma=gg, beta=gb)
    out["grad_x"] = g
    return out


# a stack's error is a block's, once for each block it went through and came back by
def _tol(wl):
    return 2 * wl.blocks * tol_for(wl.mixed)


@pytest.mark.parametrize("mixed", [False, True, "f16"])
@pytest.mark.parametrize("shape", [(3, 16, (32, 64), (6, 10)), (2, 20, (17, 30), (5, 7)),
                                   (2, 6, (8, 10, 12), (3, 3, 4))], ids=str)
def test_normed_training_stack(shape, mixed):
    from fno_spectral_convolution_amd.stack import StackRunner
    batch, c, grid, modes = shape
    announce("normed stack", shape, mixed)
    wl = Workload("t", 41, batch, c, grid, modes, 3, mixed, True, norm=True)
    for fuse in (True, False):
        r = StackRunner(wl, fuse_loss=fuse)
        r.step()
        ref = _reference(wl, r.host)
        scale = r.grad_scale
        assert scale == (F16_LOSS_SCALE if mixed == "f16" else 1.0)
        assert abs(float(r.loss) - ref["loss"]) <= _tol(wl) * ref["loss"]
        check("grad_x", r.grad_x.cpu().numpy() / scale, ref["grad_x"], _tol(wl))
        for i, g in enumerate(r.grads):
            assert set(g) == set(ref["grads"][i])
            for k in g:
                check(f"block {i} {k}", g[k].cpu().numpy() / scale, ref["grads"][i][k], _tol(wl))


@pytest.mark.parametrize("blocks", [1, 3])
def test_normed_forward_stack(blocks):
    from fno_spectral_convolution_amd.stack import StackRunner
    announce("normed forward stack", blocks)
    wl = Workload("t", 42, 2, 20, (30, 40), (6, 8), blocks, False, False, norm=True)
    r = StackRunner(wl)
    y = r.step().cpu().numpy()
    check("y", y, _reference(wl, r.host)["y"], _tol(wl))


def test_normed_tucker_stack_matches_its_lists():
    """A factorised stack trains its core and factors: lists, buffers and update go together."""
    import torch

    from fno_spectral_convolution_amd.optim import AdamW
    from fno_spectral_convolution_amd.stack import StackRunner
    announce("normed tucker stack")
    wl = Workload("t", 43, 2, 16, (16, 32), (4, 6), 2, False, True, norm=True,
                  tucker_ranks=(8, 8, 6, 4))
    r = StackRunner(wl)
    ps, gs = r.parameters(), r.gradients()
    assert len(ps) == len(gs) == 2 * (1 + 4 + 2) + 2
    assert all(p.shape == g.shape and p.dtype == g.dtype for p, g in zip(ps, gs))
    opt = AdamW(ps, gs, 1e-3)
    first = None
    for _ in range(30):
        r.step()
        opt.step()
        first = float(r.loss) if first is None else first
    torch.cuda.synchronize()
    assert float(r.loss) < first
    assert all(bool(torch.isfinite(torch.view_as_real(p) if p.is_complex() else p).all())
               for p in ps)


@pytest.mark.parametrize("mixed", [False, "f16"])
def test_optimiser_steps(mixed):
    """Three clipped steps of AdamW on the stack's own gradients, against float64."""
    from fno_spectral_convolution_amd.optim import AdamW
    from fno_spectral_convolution_amd.stack import StackRunner
    announce("optimiser steps", mixed)
    wl = Workload("t", 44, 2, 16, (16, 32), (4, 6), 2, mixed, True, norm=True)
    r = StackRunner(wl)
    lr, betas, eps, wd, top = 1e-2, (0.9, 0.99), 1e-8, 0.02, 1e-3
    opt = AdamW(r.parameters(), r.gradients(), lr, betas, eps, wd, max_norm=top)

    def flat(ts):
        return np.concatenate([t.cpu().numpy().ravel().view(np.float32).astype(np.float64)
                               for t in ts])

    p = flat(r.parameters())
    m, v = np.zeros_like(p), np.zeros_like(p)
    for t in range(1, 4):
        r.step()
        g = flat(r.gradients()) / r.grad_scale
        opt.step(r.grad_scale)
        norm = np.linalg.norm(g)
        assert abs(float(opt.grad_norm) - norm) <= 2e-6 * norm
        g *= min(1.0, top / norm)
        m = betas[0] * m + (1 - betas[0]) * g
        v = betas[1] * v + (1 - betas[1]) * g * g
        p -= lr * wd * p + lr * (m / (1 - betas[0] ** t)) / (np.sqrt(v / (1 - betas[1] ** t)) + eps)
        check(f"step {t} parameters", flat(r.parameters()), p, TOL_F32)
        check(f"step {t} exp_avg", flat(opt.exp_avg), m, TOL_F32)
        check(f"step {t} exp_avg_sq", flat(opt.exp_avg_sq), v, TOL_F32)
        p, m, v = flat(r.parameters()), flat(opt.exp_avg), flat(opt.exp_avg_sq)
    assert opt.steps == 3


@pytest.mark.parametrize("precision", ["f32", "bf16", "f16"])
def test_example_learns(precision):
    import examples.train_stack as ex
    announce("example", precision)
    losses, norms = ex.train(steps=40, precision=precision, verbose=False)
    assert all(math.isfinite(x) for x in losses + norms)
    assert losses[-1] < 0.5 * losses[0]


def test_norm_parameters_are_seeded():
    wl = Workload("t", 45, 1, 8, (8, 8), (2, 2), 3, False, False, norm=True)
    a, b = inputs.block_params(wl), inputs.block_params(wl)
    assert "gamma" not in a[0] and a[1]["gamma"].dtype == np.float32
    assert np.array_equal(a[2]["gamma"], b[2]["gamma"])
    assert not np.array_equal(a[1]["gamma"], a[2]["gamma"])


def test_optimiser_step_refused_during_capture():
    """A captured step would replay one update's number and learning rate: it is refused, and the
    optimiser goes on as if it had not been asked."""
    import torch

    from fno_spectral_convolution_amd.optim import AdamW
    announce("optimiser step during capture")
    p, g = torch.ones(3000, device="cuda"), torch.ones(3000, device="cuda")
    opt = AdamW([p], [g], 1e-2)
    opt.step()
    torch.cuda.synchronize()
    before, graph, x = p.clone(), torch.cuda.CUDAGraph(), torch.zeros(64, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        x += 1
        with pytest.raises(RuntimeError, match="captur"):
            opt.step()
    graph.replay()
    torch.cuda.synchronize()
    assert opt.steps == 1 and torch.equal(p, before) and float(x[0]) == 1.0
    opt.step()
    assert opt.steps == 2 and bool((p < before).all())
