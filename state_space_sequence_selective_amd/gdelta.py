"""One gated delta rule core's device buffers around the C entry points of
include/mamba_gdelta.h.

``GatedDeltaCore`` owns the output, the last state and, for training, what the
backward reads, every gradient and the workspace, allocated once, so that
``forward``, ``backward`` and ``step`` issue only kernel launches.
"""
from __future__ import annotations

import torch

from . import _lib

INPUTS = ("q", "k", "v", "a_raw", "b_raw", "a_log", "dt_bias")
PARAMS = ("a_log", "dt_bias")   # their gradients accumulate


class GatedDeltaCore:
    def __init__(self, dims: _lib.GDeltaDims, device="cuda", train=True):
        self.dims = d = dims
        self.train = train
        s, at, f = d.shapes(), d.act_dtype, torch.float32
        kw = dict(device=device)
        self.y = torch.empty(s["v"], dtype=at, **kw)
        self.h_last = torch.empty(s["state"], dtype=f, **kw)
        self.workspace = torch.empty(_lib.gdelta_workspace_bytes(d) if train or d.seqlen > _lib.GDELTA_STEP_TOKENS else 0,
                                     dtype=torch.uint8, **kw)
        self.saved, self.grads, self._had_h0 = None, {}, False
        if train:
            self.saved = torch.empty(_lib.gdelta_saved_bytes(d), dtype=torch.uint8, **kw)
            shp = dict(q=(s["qk"], at), k=(s["qk"], at), v=(s["v"], at), a_raw=(s["gate"], f), b_raw=(s["gate"], f))
            self.grads = {n: torch.empty(sh, dtype=dt, **kw) for n, (sh, dt) in shp.items()}
            # the accumulating parameter gradients share one block, so clearing them is one fill
            pad = -(-d.heads // 64) * 64
            self._param_grads = torch.zeros(2 * pad, dtype=f, **kw)
            for i, n in enumerate(PARAMS):
                self.grads[n] = self._param_grads[i * pad:i * pad + d.heads]

    def zero_grads(self):
        """The parameter gradients accumulate; clear them once per step."""
        self._param_grads.zero_()

    def forward(self, inp: dict, h0=None, stream=None):
        """y; the state behind the last token is in ``h_last`` (h0 may be ``h_last`` itself)."""
        _lib.gdelta_fwd(self.dims, *(inp[n] for n in INPUTS), h0, y=self.y, h_last=self.h_last, saved=self.saved,
                        workspace=self.workspace if self.workspace.numel() else None, stream=stream)
        self._had_h0 = h0 is not None
        return self.y

    def backward(self, inp: dict, dy, stream=None):
        """Every input's gradient, for the latest ``forward`` of the same inputs."""
        if not self.train:
            raise ValueError("backward needs a core made with train=True")
        g = self.grads
        _lib.gdelta_bwd(self.dims, *(inp[n] for n in INPUTS), self.saved, dy, d_q=g["q"], d_k=g["k"], d_v=g["v"],
                        d_a_raw=g["a_raw"], d_b_raw=g["b_raw"], d_a_log=g["a_log"], d_dt_bias=g["dt_bias"],
                        workspace=self.workspace, has_h0=self._had_h0, stream=stream)
        return g

    def step(self, inp: dict, state, stream=None):
        """y of a decoding step's tokens; ``state`` is updated in place."""
        _lib.gdelta_step(self.dims, *(inp[n] for n in INPUTS), state, y=self.y, stream=stream)
        return self.y
