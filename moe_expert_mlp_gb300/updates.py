"""Orthogonalised updates of a list of weight gradients on one GPU.

Like the layer, the object allocates its buffers once (momenta, results, one
workspace that its calls use in turn) and issues a fixed sequence of C-ABI calls
on one stream, so a step can be captured in a CUDA graph.
"""
from __future__ import annotations

import math

import torch

from . import _lib as L


class OrthogonalUpdates:
    """grads: bf16 or fp32 tensors [E, rows, cols] (a matrix an expert) or [rows,
    cols], with unit stride along a row; they are read at each step, where they
    are.  momentum 0 keeps none.  scale: a number, or a function of (rows, cols);
    by default 0.2 sqrt(max(rows, cols)), with which an update's elements have the
    same size whatever the matrix's.  sizes: those (rows, cols) for each gradient
    that holds more than its weight has, such as rows of padding, which the default
    would count; None: the gradients' own.  Results: outs (bf16), to be subtracted
    from the weights times the learning rate; momenta (fp32)."""

    def __init__(self, grads, momentum=0.95, dampening=0.0, nesterov=True, steps=5,
                 coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=None, sizes=None):
        self.grads = list(grads)
        if sizes is not None and len(sizes) != len(self.grads):
            raise ValueError(f"{len(sizes)} sizes for {len(self.grads)} gradients")
        names = {torch.bfloat16: "bf16", torch.float32: "fp32"}
        self.descs, self.outs, self.momenta = [], [], []
        size = 256
        for i, g in enumerate(self.grads):
            if g.dtype not in names or g.dim() not in (2, 3) or not g.is_cuda:
                raise ValueError(f"gradient {i}: expected a bf16 or fp32 CUDA tensor of two or three "
                                 f"dimensions, got {g.dtype} of shape {tuple(g.shape)} on {g.device}")
            rows, cols = g.shape[-2:]
            of = (rows, cols) if sizes is None else tuple(sizes[i])
            if sizes is not None and not (0 < of[0] <= rows and 0 < of[1] <= cols):
                raise ValueError(f"gradient {i}: a size of {of} in matrices of {(rows, cols)}")
            if scale is None:
                by = 0.2 * math.sqrt(max(of))
            else:
                by = scale(*of) if callable(scale) else scale
            self.descs.append(L.make_orthogonalize_desc(
                g.shape[0] if g.dim() == 3 else 1, rows, cols, grad_dtype=names[g.dtype],
                steps=steps, coefficients=coefficients, eps=eps, momentum=momentum,
                dampening=dampening, nesterov=nesterov, scale=by))
            size = max(size, L.moe_orthogonalize_workspace_size(self.descs[-1]))
            self.outs.append(torch.zeros(g.shape, dtype=torch.bfloat16, device=g.device))
            self.momenta.append(torch.zeros(g.shape, dtype=torch.float32, device=g.device)
                                if momentum else None)
        self.ws = torch.empty(size, dtype=torch.uint8,
                              device=self.grads[0].device if self.grads else "cpu")

    def step(self, stream=None):
        """The momenta's next values and the updates they give."""
        for desc, g, out, m in zip(self.descs, self.grads, self.outs, self.momenta):
            L.moe_orthogonalize(desc, g, out, self.ws, m, stream=stream)
        return self.outs
