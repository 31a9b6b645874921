"""Group norm and dropout as a stack uses them: training stacks against the oracle's blocks and plain
norms and masks in float64, a captured step whose replays take new masks, and the example run."""
import math

import numpy as np
import pytest

import oracle.fno_oracle as O
from fno_spectral_convolution_amd.configs import F16_LOSS_SCALE, Workload
from tests.gpu_helpers import announce, check, tol_for

pytestmark = pytest.mark.gpu

EPS = 1e-5


def _gelu(u):
    """GELU and its slope"""
    erf = np.vectorize(math.erf, otypes=[np.float64])
    cdf = 0.5 * (1 + erf(u / math.sqrt(2)))
    return u * cdf, cdf + u * np.exp(-u * u / 2) / math.sqrt(2 * math.pi)


def _split(t, groups):
    return t.reshape(t.shape[0], groups, -1)


def _factor(shape, p, seed, draw):
    from tests.test_gpu_between_ops import _factor as f
    return f(shape, p, seed, draw, device="cpu").numpy() if p else 1.0


def _reference(wl, hi, seed, draws):
    """Output, loss and gradients of the stack at a step that begins with `draws`."""
    tanh, nb = bool(wl.mixed), len(hi["blocks"])
    h, xs, saved = np.asarray(hi["x"], np.float64), [], [None]
    side = (1, -1) + (1,) * len(wl.grid)
    inner = wl.norm == "group"  # GELU in the norm, not in the block
    for i, b in enumerate(hi["blocks"]):
        if i:
            f = _factor(h.shape, wl.dropout if wl.train else 0.0, seed, i + draws)
            keep = {"f": f}
            if wl.norm == "group":
                s = _split(h, wl.groups)
                mean = s.mean(2, keepdims=True)
                r = 1 / np.sqrt(((s - mean) ** 2).mean(2, keepdims=True) + EPS)
                hn = ((s - mean) * r).reshape(h.shape)
                ga, be = (b[k].astype(np.float64).reshape(side) for k in ("gamma", "beta"))
                h, slope = _gelu(ga * hn + be)
                keep.update(hn=hn, r=r, ga=ga, slope=slope)
            h = h * f
            saved.append(keep)
        xs.append(h)
        fw = O.block_fwd(h, b["w"], b["wb"], b["bias"], wl.modes, tanh=tanh,
                         act=i == nb - 1 or not inner)
        h = fw["y"]
    out = {"y": h}
    if not wl.train:
        return out
    out["loss"], g = O.mse_loss_grad(h, hi["target"])
    out["grads"] = [None] * nb
    for i in reversed(range(nb)):
        b = hi["blocks"][i]
        k = O.block_bwd(xs[i], b["w"], b["wb"], b["bias"], wl.modes, g, tanh=tanh,
                        act=i == nb - 1 or not inner)
        out["grads"][i] = {"w": k["grad_w"], "wb": k["grad_wb"], "bias": k["grad_bias"]}
        g = k["grad_x"]
        if i:
            c = saved[i]
            g = g * c["f"]
            if inner:
                g = g * c["slope"]
                rows = (0,) + tuple(range(2, g.ndim))
                out["grads"][i].update(gamma=(g * c["hn"]).sum(rows), beta=g.sum(rows))
                v, hs = _split(g * c["ga"], wl.groups), _split(c["hn"], wl.groups)
                g = (c["r"] * (v - v.mean(2, keepdims=True)
                               - hs * (v * hs).mean(2, keepdims=True))).reshape(g.shape)
    out["grad_x"] = g
    return out


def _tol(wl):  # a block's, once for each block that the step goes through and comes back by
    return 2 * wl.blocks * tol_for(wl.mixed)


@pytest.mark.parametrize("mixed", [False, True, "f16"])
@pytest.mark.parametrize("norm,dropout", [("group", 0.0), ("group", 0.2), (False, 0.2)])
@pytest.mark.parametrize("shape", [(3, 16, 4, (32, 64), (6, 10)), (2, 20, 5, (17, 30), (5, 7)),
                                   (2, 6, 2, (8, 10, 12), (3, 3, 4))], ids=str)
def test_training_stack(shape, norm, dropout, mixed):
    from fno_spectral_convolution_amd.stack import StackRunner
    batch, c, groups, grid, modes = shape
    announce("stack", shape, norm, dropout, mixed)
    wl = Workload("t", 51, batch, c, grid, modes, 3, mixed, True, norm=norm, groups=groups,
                  dropout=dropout)
    for fuse in (True, False):
        r = StackRunner(wl, fuse_loss=fuse, dropout_seed=77)
        for step in range(2):  # the second step draws other masks
            r.step()
            ref = _reference(wl, r.host, 77, 3 * step)
            scale = r.grad_scale
            assert scale == (F16_LOSS_SCALE if mixed == "f16" else 1.0)
            assert abs(float(r.loss) - ref["loss"]) <= _tol(wl) * ref["loss"]
            check("grad_x", r.grad_x.cpu().numpy() / scale, ref["grad_x"], _tol(wl))
            for i, g in enumerate(r.grads):
                assert set(g) == set(ref["grads"][i])
                for k in g:
                    check(f"block {i} {k}", g[k].cpu().numpy() / scale, ref["grads"][i][k], _tol(wl))


@pytest.mark.parametrize("blocks", [1, 3])
def test_forward_stack_drops_nothing(blocks):
    from fno_spectral_convolution_amd.stack import StackRunner
    announce("group normed forward stack", blocks)
    wl = Workload("t", 52, 2, 20, (30, 40), (6, 8), blocks, False, False, norm="group", groups=4,
                  dropout=0.3)
    r = StackRunner(wl)
    y = r.step().cpu().numpy()
    check("y", y, _reference(wl, r.host, 0, 0)["y"], _tol(wl))


def test_captured_step_takes_new_masks():
    """A captured step and the optimiser-free rest of it: each replay moves the draws on, and gives the
    bits of an eager run's same step."""
    import torch

    from fno_spectral_convolution_amd.stack import StackRunner
    announce("captured stack step")
    wl = Workload("t", 53, 2, 16, (16, 32), (4, 6), 3, False, True, norm="group", groups=4,
                  dropout=0.25)
    eager, cap = StackRunner(wl, dropout_seed=5), StackRunner(wl, dropout_seed=5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        cap.step()  # what a process's first calls take is done
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    cap.draws.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cap.step()
    losses = []
    for k in range(4):
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert int(cap.draws) == int(eager.draws) == 3 * (k + 1)
        assert torch.equal(cap.loss, eager.loss) and torch.equal(cap.grad_x, eager.grad_x)
        assert all(torch.equal(a, b) for a, b in zip(cap.gradients(), eager.gradients()))
        losses.append(float(cap.loss))
    assert len(set(losses)) == 4


def test_tucker_stack_with_dropout_steps():
    import torch

    from fno_spectral_convolution_amd.optim import AdamW
    from fno_spectral_convolution_amd.stack import StackRunner
    announce("tucker stack with group norm and dropout")
    wl = Workload("t", 54, 2, 16, (16, 32), (4, 6), 2, False, True, norm="group", groups=2,
                  dropout=0.1, tucker_ranks=(8, 8, 6, 4))
    r = StackRunner(wl)
    ps, gs = r.parameters(), r.gradients()
    assert len(ps) == len(gs) == 2 * (1 + 4 + 2) + 2
    opt = AdamW(ps, gs, 1e-3)
    for _ in range(3):
        r.step()
        opt.step()
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(torch.view_as_real(p) if p.is_complex() else p).all())
               for p in ps + gs)


@pytest.mark.parametrize("precision", ["f32", "bf16", "f16"])
def test_example_runs(precision):
    import examples.train_stack as ex
    announce("example with group norm and dropout", precision)
    losses, norms = ex.train(steps=4, precision=precision, verbose=False, norm="group", dropout=0.1)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses + norms)
    assert all(n > 0 for n in norms)


def test_refusals():
    from fno_spectral_convolution_amd.stack import StackRunner
    base = ("t", 55, 1, 8, (8, 8), (2, 2), 2, False, True)
    with pytest.raises(ValueError, match="groups"):
        StackRunner(Workload(*base, norm="group", groups=3))
    with pytest.raises(ValueError, match="norm must be"):
        StackRunner(Workload(*base, norm="batch"))
    with pytest.raises(ValueError, match="dropout goes with"):
        StackRunner(Workload(*base, norm="layer", dropout=0.1))
    with pytest.raises(ValueError, match="p must"):
        StackRunner(Workload(*base, dropout=1.0))
