"""Layer norm's device buffers around the C entry points of
include/mamba_norm.h.

``LayerNorm`` owns the output, the row statistics, the gradients and the
workspace, allocated once, so that ``forward`` and ``backward`` issue only
kernel launches.  Rows are [rows, dim] views of whatever is normed.
"""
from __future__ import annotations

import torch

from . import _lib


class LayerNorm:
    def __init__(self, dims: _lib.NormDims, device="cuda"):
        self.dims = d = dims
        f, kw = torch.float32, dict(device=device)
        self.y = torch.empty((d.rows, d.dim), dtype=d.y_dtype, **kw)
        self.dx = torch.empty((d.rows, d.dim), dtype=d.x_dtype, **kw)
        self.mean, self.rstd = torch.empty(d.rows, dtype=f, **kw), torch.empty(d.rows, dtype=f, **kw)
        pad = -(-d.dim // 64) * 64
        self._param_grads = torch.zeros(2 * pad, dtype=f, **kw)   # one fill clears both
        self.dw, self.db = self._param_grads[:d.dim], self._param_grads[pad:pad + d.dim]
        self.workspace = torch.empty(_lib.layernorm_workspace_bytes(d), dtype=torch.uint8, **kw)

    def zero_grads(self):
        """The weight's and bias's gradients accumulate; clear them once per step."""
        self._param_grads.zero_()

    def forward(self, x, w=None, b=None, stream=None):
        _lib.layernorm_fwd(self.dims, x, w, b, y=self.y, mean=self.mean, rstd=self.rstd, stream=stream)
        return self.y

    def backward(self, x, w, dy, d_add=None, mean=None, rstd=None, stream=None):
        """dx (+ d_add); d_w and d_b are added to ``dw`` and ``db``.  mean and rstd: the forward's, by default the
        latest ``forward`` of this object's."""
        _lib.layernorm_bwd(self.dims, x, w, self.mean if mean is None else mean, self.rstd if rstd is None else rstd,
                           dy, d_add, dx=self.dx, d_w=self.dw, d_b=self.db, workspace=self.workspace, stream=stream)
        return self.dx
