"""The vocabulary's loss on the GPU: softmax cross entropy of the logits x W^T
with its gradient, the logits never stored.

Every step runs in the CUDA library (mom_linear_ce_fwd, mom_linear_ce_bwd); this
module holds the weight, the outputs and the workspaces and passes pointers.
"""
from __future__ import annotations

from typing import Dict, Optional

import torch

from . import binding as B


class LMHead:
    """weight [vocab, d_model], bf16 or float32.  Outputs and workspaces are
    made once per shape and written again by the next call of that shape;
    calls of one head must not overlap on the GPU."""

    def __init__(self, weight: torch.Tensor):
        if weight.dim() != 2:
            raise ValueError("the head's weight is [vocab, d_model]")
        B.dtype_code(weight.dtype)
        self.w = weight
        self.vocab, self.d_model = weight.shape
        self.dtype, self.device = weight.dtype, weight.device
        self._bufs = {}
        self._held = []

    def _buf(self, name, shape, dtype):
        key = (name, tuple(shape), dtype)
        t = self._bufs.get(key)
        if t is None:
            t = self._bufs[key] = torch.empty(shape, dtype=dtype, device=self.device)
        return t

    def _ws(self, name, nbytes, stream):
        key = ("ws", name)
        t = self._bufs.get(key)
        with torch.cuda.stream(stream):            # None: the current stream
            if t is None or t.numel() < nbytes:
                t = self._bufs[key] = B.new_workspace(nbytes, self.device)
            if torch.cuda.is_current_stream_capturing() and not any(t is h for h in self._held):
                self._held.append(t)    # a graph keeps its workspace when a larger one takes its place
        return t

    def loss(self, x: torch.Tensor, targets: torch.Tensor, stream=None) -> Dict[str, torch.Tensor]:
        """x [N, d_model], targets [N] int32 (negative: padding).  Returns
        ``loss`` [N] (0 for padding), ``lse`` [N], the ``mean`` loss over the
        rows with a target and ``inv_count`` = 1 / their number (0-d)."""
        n = x.shape[0]
        loss, lse = self._buf("loss", (n,), torch.float32), self._buf("lse", (n,), torch.float32)
        mean = self._buf(("mean", n), (2,), torch.float32)
        ws = self._ws("fwd", B.mom_linear_ce_workspace_size(n, self.d_model, self.vocab, self.dtype, False), stream)
        B.mom_linear_ce_fwd(x, self.w, targets, loss, lse, mean, ws, stream=stream)
        return dict(loss=loss, lse=lse, mean=mean[0], inv_count=mean[1])

    def backward(self, x: torch.Tensor, targets: torch.Tensor, dloss: Optional[torch.Tensor] = None,
                 stream=None) -> Dict[str, torch.Tensor]:
        """Gradients for the loss just run on the same x and targets (its lse
        is read): ``dx`` [N, d_model] and ``dw`` [vocab, d_model] in the
        weight's type, of the mean loss, or with dloss [N] float32 of
        sum(dloss * loss)."""
        n = x.shape[0]
        lse = self._bufs.get(("lse", (n,), torch.float32))
        if lse is None:
            raise ValueError("backward follows a loss call of the same shape")
        scale = None if dloss is not None else self._buf(("mean", n), (2,), torch.float32)[1:2]
        dx = self._buf("dx", (n, self.d_model), self.dtype)
        dw = self._buf("dw", (self.vocab, self.d_model), self.dtype)
        ws = self._ws("bwd", B.mom_linear_ce_workspace_size(n, self.d_model, self.vocab, self.dtype, True), stream)
        B.mom_linear_ce_bwd(x, self.w, targets, lse, dloss, scale, dx, dw, ws, stream=stream)
        return dict(dx=dx, dw=dw)

    def device_errors(self):
        """(code, info) of every workspace with a recorded violation."""
        errs = {}
        for key, t in self._bufs.items():
            if key[0] == "ws":
                code, info = B.mom_get_error(t)
                if code:
                    errs[key[1]] = (code, info)
        return errs
