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
    made once and written again: loss, lse, mean, inv_count and dx by the next
    call with the same number of rows, dw by the next backward of any number.
    A caller who needs them longer gives tensors of its own (out, saved, dw
    below).  Every number of rows keeps its outputs as long as the head lives.
    Calls of one head must not overlap on the GPU."""

    def __init__(self, weight: torch.Tensor):
        if weight.dim() != 2:
            raise ValueError("the head's weight is [vocab, d_model]")
        B.dtype_code(weight.dtype)
        self.w = weight
        self.vocab, self.d_model = weight.shape
        self.dtype, self.device = weight.dtype, weight.device
        self._bufs, self._ws, self._made_on, self._held = {}, {}, {}, []

    def _fwd_bufs(self, n):
        b = self._bufs.get(("fwd", n))
        if b is None:
            new = lambda k: torch.empty(k, dtype=torch.float32, device=self.device)
            loss, lse, mean = new(n), new(n), new(2)
            size = B.mom_linear_ce_workspace_size(n, self.d_model, self.vocab, self.dtype, False)
            b = self._bufs["fwd", n] = (loss, lse, mean, mean[0], mean[1], mean[1:2], size)
        return b

    def _bwd_bufs(self, n):
        b = self._bufs.get(("bwd", n))
        if b is None:
            size = B.mom_linear_ce_workspace_size(n, self.d_model, self.vocab, self.dtype, True)
            b = self._bufs["bwd", n] = (torch.empty((n, self.d_model), dtype=self.dtype, device=self.device), size)
        return b

    def _dw(self):
        dw = self._bufs.get("dw")
        if dw is None:
            dw = self._bufs["dw"] = torch.empty((self.vocab, self.d_model), dtype=self.dtype, device=self.device)
        return dw

    def new_loss(self, n) -> Dict[str, torch.Tensor]:
        """Outputs of a loss call of n rows for the caller to keep (loss's
        ``out``, backward's ``saved``)."""
        new = lambda k: torch.empty(k, dtype=torch.float32, device=self.device)
        both = new(2)
        return dict(loss=new(n), lse=new(n), mean=both[0], inv_count=both[1], mean_inv=both)

    def _workspace(self, name, nbytes):
        t = self._ws.get(name)
        if t is None or t.numel() < nbytes:
            t = self._ws[name] = B.new_workspace(nbytes, self.device)
            self._made_on[name] = B.current_stream_id(self.device)
        elif B.current_stream_id(self.device) != self._made_on[name]:
            # freed when a larger one takes its place, but not before this stream is done with it
            t.record_stream(torch.cuda.current_stream(self.device))
        if torch.cuda.is_current_stream_capturing() and not any(t is h for h in self._held):
            self._held.append(t)    # a graph keeps its workspace when a larger one takes its place
        return t

    def loss(self, x: torch.Tensor, targets: torch.Tensor, stream=None,
             out: Optional[Dict[str, torch.Tensor]] = None) -> Dict[str, torch.Tensor]:
        """x [N, d_model], targets [N] int32 (negative: padding).  Returns
        ``loss`` [N] (0 for padding), ``lse`` [N], the ``mean`` loss over the
        rows with a target and ``inv_count`` = 1 / their number (0-d); with
        ``out`` (new_loss(N)) in the tensors given there."""
        if stream is not None:      # buffers that a first call makes belong to its stream
            with torch.cuda.stream(stream):
                return self.loss(x, targets, out=out)
        loss, lse, both, mean, inv_count, _, size = self._fwd_bufs(x.shape[0])
        if out is not None:
            if "mean_inv" not in out:
                raise ValueError("out is a dict that new_loss made")
            loss, lse, both = out["loss"], out["lse"], out["mean_inv"]
        B.mom_linear_ce_fwd(x, self.w, targets, loss, lse, both, self._workspace("fwd", size))
        return out if out is not None else dict(loss=loss, lse=lse, mean=mean, inv_count=inv_count)

    def backward(self, x: torch.Tensor, targets: torch.Tensor, dloss: Optional[torch.Tensor] = None, stream=None,
                 saved: Optional[Dict[str, torch.Tensor]] = None,
                 dw: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
        """Gradients for a loss on the same x and targets, whose lse and
        inv_count are read: from ``saved``, what loss(.., out=) wrote, or else
        from this head's last loss call with N rows -- which must have been that
        one: where another loss of N rows, an evaluation say, comes between the
        two, give ``saved``.  ``dx`` [N, d_model] and ``dw`` [vocab, d_model]
        in the weight's type, of the mean loss, or with dloss [N] float32 of
        sum(dloss * loss); dw into the tensor given, or else into the head's one
        (overwritten by every backward)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(x, targets, dloss, saved=saved, dw=dw)
        n = x.shape[0]
        if saved is not None:
            lse, inv_count = saved["lse"], saved["inv_count"].view(1)
        else:
            fwd = self._bufs.get(("fwd", n))
            if fwd is None:
                raise ValueError("backward follows a loss call of the same shape")
            lse, inv_count = fwd[1], fwd[5]
        dx, size = self._bwd_bufs(n)
        if dw is None:
            dw = self._dw()
        B.mom_linear_ce_bwd(x, self.w, targets, lse, dloss, None if dloss is not None else inv_count, dx, dw,
                            self._workspace("bwd", size))
        return dict(dx=dx, dw=dw)

    def device_errors(self):
        """(code, info) of every workspace with a recorded violation."""
        errs = {}
        for name, t in self._ws.items():
            code, info = B.mom_get_error(t)
            if code:
                errs[name] = (code, info)
        return errs
