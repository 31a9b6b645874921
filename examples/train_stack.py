"""Trains a small 2D FNO stack with layer norms on a made-up operator, on one MI355X.

    python examples/train_stack.py [--steps N] [--precision f32|bf16|f16]

The data stands for a PDE's solution operator: inputs are Gaussian random fields a, targets GELU(u)
(what a stack that ends in a GELU can give) of their screened-Poisson solutions
u = (1 - 0.01 Laplace)^-1 a, a new batch each step.  Each step is the stack's forward, loss and
backward, then AdamW with the gradients clipped to a global norm.
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from fno_spectral_convolution_amd import inputs  # noqa: E402
from fno_spectral_convolution_amd.configs import Workload  # noqa: E402
from fno_spectral_convolution_amd.optim import AdamW  # noqa: E402
from fno_spectral_convolution_amd.stack import StackRunner  # noqa: E402

PRECISIONS = {"f32": False, "bf16": "bf16", "f16": "f16"}


def batch(wl, step):
    """Inputs and targets [B, C, N, N]: every channel a field of its own."""
    n = wl.grid[0]
    a = inputs.grf(inputs.rng(wl.cfg_id, inputs.STREAM_INPUT, step), wl.batch * wl.width, wl.grid)
    k = np.fft.fftfreq(n, 1.0 / n)
    k2 = k[:, None] ** 2 + np.fft.rfftfreq(n, 1.0 / n)[None, :] ** 2
    u = np.fft.irfft2(np.fft.rfft2(a) / (1.0 + 0.01 * k2), s=wl.grid)
    a, u = (torch.from_numpy(v.astype(np.float32).reshape((wl.batch, wl.width) + wl.grid))
            for v in (a, u))
    return a, torch.nn.functional.gelu(u)


def train(steps=60, precision="f32", lr=1e-2, max_norm=0.1, verbose=True):
    """Losses and gradient norms of the run."""
    wl = Workload("example", 90, 4, 20, (64, 64), (12, 12), 3, PRECISIONS[precision], True,
                  norm=True)
    runner = StackRunner(wl)
    opt = AdamW(runner.parameters(), runner.gradients(), lr, max_norm=max_norm)
    losses, norms = [], []
    for i in range(steps):
        a, u = batch(wl, i)
        runner.x_in.copy_(a)
        runner.target.copy_(u)
        runner.step()
        opt.step(runner.grad_scale)
        losses.append(float(runner.loss))
        norms.append(float(opt.grad_norm))
        if verbose and (i % 10 == 0 or i == steps - 1):
            print(f"step {i:4d}  loss {losses[-1]:.5f}  gradient norm {norms[-1]:.4f}", flush=True)
    return losses, norms


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--precision", choices=sorted(PRECISIONS), default="f32")
    args = ap.parse_args()
    train(args.steps, args.precision)
