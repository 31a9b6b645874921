"""AdamW with clipping by the global gradient norm, over lists of tensors, through libfno.

``AdamW(runner.parameters(), runner.gradients(), lr)`` keeps the two moments of every parameter
and the tensor lists of its calls; ``step(grad_scale)`` takes one update from the gradients that
are in their buffers: the norm in one pass over them, then the update in one pass over everything,
which takes the clipping and the loss scale out of the gradients as it reads them.
"""
from __future__ import annotations

from . import binding as L


class AdamW:
    """params: float32 or complex64 (as pairs) tensors, updated in place.  grads: as many tensors
    of the same sizes, in the buffers that every step's gradients come in; float32, bfloat16,
    float16 or complex64.  max_norm: the global norm that gradients are clipped to (inf: none)."""

    def __init__(self, params, grads, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 max_norm=float("inf")):
        import torch
        self.lr, self.betas, self.eps = lr, betas, eps
        self.weight_decay, self.max_norm = weight_decay, max_norm
        params = list(params)
        self.exp_avg, self.exp_avg_sq = ([torch.zeros_like(p) for p in params] for _ in range(2))
        self._params, self._grads = L.TensorList(params), L.TensorList(grads)
        self._m, self._v = L.TensorList(self.exp_avg), L.TensorList(self.exp_avg_sq)
        self.record = torch.zeros(2, dtype=torch.float32, device=self._params.device)
        self.steps = 0

    @staticmethod
    def _capturing(stream):
        import torch
        return torch.cuda.is_current_stream_capturing()

    @property
    def grad_norm(self):
        """The gradients' global norm at the last step, without the loss scale (a device tensor)."""
        return self.record[0]

    def step(self, grad_scale=1.0):
        """One update from the gradients in their buffers, which carry the loss scale grad_scale.
        Where one of them is infinite or NaN, parameters and moments stay as they are (and the step
        still counts in the bias corrections).  Not during a stream capture: the update's number and
        the learning rate are values of the launch, and a replay would repeat them."""
        if L._on_stream(self._params.index, self._capturing):
            raise RuntimeError("AdamW.step cannot be captured: a replay would repeat this step's "
                               "number and learning rate")
        self.steps += 1
        L.grad_norm(self._grads, self.max_norm, grad_scale, record=self.record)
        L.adamw(self._params, self._grads, self._m, self._v, self.steps, self.lr, self.betas,
                self.eps, self.weight_decay, record=self.record)
