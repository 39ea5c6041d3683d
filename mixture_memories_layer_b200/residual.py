"""A stack of Mixture-of-Memories blocks in a residual stream, on the GPU.

    h_0     = norm(x_0) w_pre[0]
    y_i     = block_i(h_i)
    x_{i+1} = x_i + res_scale[i] sigmoid(gate_i) norm(y_i) w_post[i]
    h_{i+1} = norm(x_{i+1}) w_pre[i+1]          (the last one: w_final)

The norms, gates and additions between two blocks are one call
(mom_residual_norm), which also keeps the block's input stream as an 8-bit
checkpoint: the backward pass restores the blocks' inputs and the stream from
it (mom_residual_norm, mom_residual_norm_bwd) instead of from x_i and h_i.  A
caller to whom 8 bits are too few keeps x_i in its own type (act8=False).
Everything runs in the CUDA library; this module holds buffers and passes
pointers.
"""
from __future__ import annotations

from typing import Dict, List, Optional, Sequence

import torch

from . import binding as B
from .block import MoMBlock, RMS_EPS


class MoMStack:
    """blocks: MoMBlock, one a level; norms: for each level a dict of w_pre,
    w_post [d_model] and optionally res_scale [d_model], float32; w_final
    [d_model]: the norm after the last block.  ``stream_dtype``: the residual
    stream's type (bf16 or float32).  ``act8``: each block's input stream is
    kept for the backward pass in 8 bits; False: in stream_dtype, 2 or 4 bytes
    an element, and the gradients carry no other rounding of it."""

    def __init__(self, blocks: Sequence[MoMBlock], norms: Sequence[Dict[str, torch.Tensor]], w_final: torch.Tensor,
                 eps: float = RMS_EPS, stream_dtype: torch.dtype = torch.bfloat16, act8: bool = True):
        if len(blocks) != len(norms) or not blocks:
            raise ValueError("one norms entry a block")
        if len(set(id(b) for b in blocks)) != len(blocks):
            raise ValueError("every level has a block of its own (it keeps its forward's activations)")
        B.dtype_code(stream_dtype)
        self.blocks, self.norms, self.w_final, self.eps = list(blocks), list(norms), w_final, eps
        self.dtype, self.stream_dtype, self.act8 = blocks[0].dtype, stream_dtype, act8
        self.d_model, self.device = blocks[0].d_model, blocks[0].device
        if any(b.d_model != self.d_model for b in blocks):
            raise ValueError("the blocks' d_model differ")
        if any(b.dtype != self.dtype for b in blocks):
            raise ValueError("the blocks are of different types")
        self._bufs = {}
        self._ran = None            # what the last forward was given (None: none, or not to its end)

    def _buf(self, name, shape, dtype):
        key = (name, tuple(shape), dtype)
        t = self._bufs.get(key)
        if t is None:
            t = self._bufs[key] = torch.empty(shape, dtype=dtype, device=self.device)
        return t

    def _k8(self, i, n):
        groups = -(-self.d_model // B.MOM_ACT8_GROUP)
        return (self._buf("codes%d" % i, (n, self.d_model), torch.int8),
                self._buf("scales%d" % i, (n, groups), torch.float32))

    def _stream(self, i, n):
        """Block i's input stream (without 8-bit checkpoints; the last one: the output)."""
        return self._buf("x%d" % i, (n, self.d_model), self.stream_dtype)

    def _kept(self, i, n):
        """What the backward pass reads for it."""
        return self._k8(i, n) if self.act8 else self._stream(i, n)

    def _check_gates(self, gates):
        if gates is not None and len(gates) != len(self.blocks):
            raise ValueError("gates has %d entries for %d blocks" % (len(gates), len(self.blocks)))

    def _given(self, n, cu_seqlens, gates):
        """What a backward has to share with the forward just run: the numbers
        of rows and sequences, and each level's kind of gate."""
        kinds = [g if g is None else "token" if g.numel() == n else "element" for g in gates or [None] * len(self.blocks)]
        return n, cu_seqlens.numel() - 1, kinds

    def _w_next(self, i):
        return self.norms[i + 1]["w_pre"] if i + 1 < len(self.blocks) else self.w_final

    # -------------------------------------------------------------- forward
    def forward(self, x: torch.Tensor, cu_seqlens: torch.Tensor, gates: Optional[List] = None,
                stream=None) -> Dict[str, torch.Tensor]:
        """x [N, d_model] (stream_dtype), cu_seqlens [S+1] int32 (device);
        gates: None, or one entry a block (None, or logits [N], [N, 1] or
        [N, d_model] in the blocks' type).  Returns ``h`` [N, d_model], the
        normed output, and ``x``, the stream after the last block (both
        written again by the next call); x itself is left as it is."""
        if stream is not None:      # buffers that a first call makes, the blocks' too, belong to its stream
            with torch.cuda.stream(stream):
                return self.forward(x, cu_seqlens, gates)
        self._check_gates(gates)
        n = x.shape[0]
        st = torch.cuda.current_stream(self.device)
        self._ran = None
        h = self._buf("h", (n, self.d_model), self.dtype)
        first = None if self.act8 else self._stream(0, n)
        out = self._buf("x", (n, self.d_model), self.stream_dtype) if self.act8 else None
        B.mom_residual_norm(x, None, None, None, None, self.norms[0]["w_pre"], self.eps, first, h, stream=st)
        if first is not None:
            x = first
        for i, blk in enumerate(self.blocks):
            y = blk.forward(h, cu_seqlens, stream=st)["y"]
            w = self.norms[i]
            if not self.act8:
                out = self._stream(i + 1, n)
            B.mom_residual_norm(x, y, gates[i] if gates else None, w["w_post"], w.get("res_scale"), self._w_next(i),
                                self.eps, out, h, pack=self._k8(i, n) if self.act8 else None, stream=st)
            x = out
        self._ran = self._given(n, cu_seqlens, gates)
        return dict(h=h, x=out)

    # ------------------------------------------------------------- backward
    def backward(self, cu_seqlens: torch.Tensor, dh: torch.Tensor, dx: Optional[torch.Tensor] = None,
                 gates: Optional[List] = None, stream=None) -> Dict:
        """Gradients of <dh, h> + <dx, x> for the forward just run with the
        same cu_seqlens and gates (what it kept and the blocks' buffers are
        read, which the next forward of any size overwrites; dh, dx [N,
        d_model] float32).  Returns ``dx`` [N, d_model]
        float32, the gradient of the input stream, ``dw_final`` and ``levels``:
        for each block dw_pre, dw_post, dres_scale, dgate (where it has them)
        and ``block``, the block's own gradients (MoMBlock.backward)."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.backward(cu_seqlens, dh, dx, gates)
        self._check_gates(gates)
        n = dh.shape[0]
        if self._ran != self._given(n, cu_seqlens, gates):
            raise ValueError("backward of %d rows in %d sequences: the forward just run must have had the same, and the "
                             "same kinds of gates" % (n, cu_seqlens.numel() - 1))
        st = torch.cuda.current_stream(self.device)
        f32 = torch.float32
        g = self._buf("dx", (n, self.d_model), f32)
        ws = self._bufs.get(("ws", n))
        if ws is None:
            ws = self._bufs[("ws", n)] = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, self.d_model),
                                                         self.device)
        levels: List[Dict] = [None] * len(self.blocks)
        vec = lambda name, i: self._buf("%s%d" % (name, i), (self.d_model,), f32)
        dw_next = vec("dw_final", 0)
        dw_final = dw_next
        h = self._buf("h_restored", (n, self.d_model), self.dtype)      # (the forward's h stays the caller's)
        dy = self._buf("dy", (n, self.d_model), self.dtype)
        for i in reversed(range(len(self.blocks))):
            blk, w, kept = self.blocks[i], self.norms[i], self._kept(i, n)
            gate = gates[i] if gates else None
            lev = dict(dw_post=vec("dw_post", i))
            if w.get("res_scale") is not None:
                lev["dres_scale"] = vec("dres_scale", i)
            if gate is not None:
                lev["dgate"] = self._buf("dgate%d" % i, gate.shape, gate.dtype)
            y = blk.block_buffers(n, cu_seqlens.numel() - 1)["y"]
            B.mom_residual_norm_bwd(kept, y, gate, w["w_post"], w.get("res_scale"), self._w_next(i), self.eps, dx, dh, g,
                                    dy, lev.get("dgate"), lev["dw_post"], lev.get("dres_scale"), dw_next, ws, stream=st)
            B.mom_residual_norm(kept, None, None, None, None, w["w_pre"], self.eps, None, h, stream=st)
            lev["block"] = blk.backward(h, cu_seqlens, dy, stream=st)
            levels[i] = lev
            dx, dh, dw_next = g, lev["block"]["dx"], vec("dw_pre", i)
            lev["dw_pre"] = dw_next
        # the norm before the first block
        B.mom_residual_norm_bwd(self._kept(0, n), None, None, None, None, self.norms[0]["w_pre"], self.eps, dx, dh, g, None,
                                None, None, None, dw_next, ws, stream=st)
        return dict(dx=g, dw_final=dw_final, levels=levels)

    # --------------------------------------------------------------- decode
    def decode_step(self, x: torch.Tensor, states: Sequence, gates: Optional[List] = None,
                    stream=None) -> Dict[str, torch.Tensor]:
        """One token a sequence: x [B, d_model] (stream_dtype); states: for
        each block (state, conv_sh, conv_mem) of MoMBlock.decode_step, updated
        in place.  Returns ``h`` and ``x`` as forward."""
        if stream is not None:
            with torch.cuda.stream(stream):
                return self.decode_step(x, states, gates)
        self._check_gates(gates)
        n = x.shape[0]
        st = torch.cuda.current_stream(self.device)
        h = self._buf("dec_h", (n, self.d_model), self.dtype)
        out = self._buf("dec_x", (n, self.d_model), self.stream_dtype)
        B.mom_residual_norm(x, None, None, None, None, self.norms[0]["w_pre"], self.eps, None, h, stream=st)
        for i, blk in enumerate(self.blocks):
            y, _ = blk.decode_step(h, *states[i], stream=st)
            w = self.norms[i]
            B.mom_residual_norm(x, y, gates[i] if gates else None, w["w_post"], w.get("res_scale"), self._w_next(i),
                                self.eps, out, h, stream=st)
            x = out
        return dict(h=h, x=out)
