"""Plain fp64 numpy forms of the operators around the blocks in a training
step: the residual stream's norms, the 8-bit activation checkpoints and the
vocabulary's cross entropy, with their gradients.  Test infrastructure only;
shares no code with the CUDA path.

The functions named *_size give, element by element, the sum of the magnitudes
that meet in an output: rounding errors are bounded relative to it.
"""
from __future__ import annotations

import numpy as np

GROUP = 128


def _rms(a, eps):
    return np.sqrt(np.mean(a * a, axis=1, keepdims=True) + eps)


def sigmoid(z):
    return 1.0 / (1.0 + np.exp(-z))


def _gate(gate, n):
    return 1.0 if gate is None else sigmoid(gate.reshape(n, -1))


def residual_norm(x, y, gate, w_post, res_scale, w_pre, eps):
    """(x_out, h); y, gate, res_scale, w_pre may be None."""
    n = x.shape[0]
    if y is not None:
        u = y / _rms(y, eps) * w_post * _gate(gate, n)
        x = x + (u if res_scale is None else u * res_scale)
    return x, None if w_pre is None else x / _rms(x, eps) * w_pre


def residual_norm_bwd(x, y, gate, w_post, res_scale, w_pre, eps, dx_out, dh):
    """Gradients of <dx_out, x_out> + <dh, h>: a dict of dx, dy, dgate,
    dw_post, dres_scale, dw_pre and, under "size", the same of magnitudes."""
    n, d = x.shape
    x_out, _ = residual_norm(x, y, gate, w_post, res_scale, None, eps)
    out, size = {}, {}
    D = np.zeros_like(x) if dx_out is None else dx_out.copy()
    S = np.abs(D)
    if dh is not None:
        r = 1.0 / _rms(x_out, eps)
        nx = x_out * r
        dn = dh * w_pre
        D = D + r * (dn - nx * np.mean(dn * nx, axis=1, keepdims=True))
        # x_out = x + u may cancel: one rounding of it is half an ulp of x_out,
        # but u's own error (a chain of products) stays in |u|, so what n_x
        # carries is relative to (|x| + |u|) / rms, not to |n_x|
        an = (np.abs(x) + np.abs(x_out - x)) * r
        S = S + r * (np.abs(dn) + an * np.mean(np.abs(dn) * an, axis=1, keepdims=True))
        out["dw_pre"], size["dw_pre"] = np.sum(dh * nx, axis=0), np.sum(np.abs(dh) * an, axis=0)
    out["dx"], size["dx"] = D, S
    if y is not None:
        ry = 1.0 / _rms(y, eps)
        ny = y * ry
        sg = _gate(gate, n)
        s = np.ones(d) if res_scale is None else res_scale
        coef = s * w_post
        A, sA = np.sum(D * sg * ny, axis=0), np.sum(S * sg * np.abs(ny), axis=0)
        out["dw_post"], size["dw_post"] = s * A, np.abs(s) * sA
        if res_scale is not None:
            out["dres_scale"], size["dres_scale"] = w_post * A, np.abs(w_post) * sA
        if gate is not None:
            dg, sdg = D * coef * ny * sg * (1 - sg), S * np.abs(coef * ny) * sg
            if gate.size == n and not (gate.ndim == 2 and gate.shape[1] == d and d > 1):
                dg, sdg = dg.sum(axis=1).reshape(gate.shape), sdg.sum(axis=1).reshape(gate.shape)
            out["dgate"], size["dgate"] = dg, sdg
        u, su = D * sg * coef, S * sg * np.abs(coef)
        out["dy"] = ry * (u - ny * np.mean(u * ny, axis=1, keepdims=True))
        size["dy"] = ry * (su + np.abs(ny) * np.mean(su * np.abs(ny), axis=1, keepdims=True))
    out["size"] = size
    return out


def act8_pack(x):
    """(codes int8, scales float32): groups of 128 channels of a row."""
    n, d = x.shape
    x = np.asarray(x, np.float64)
    codes = np.zeros((n, d), np.int8)
    scales = np.zeros((n, -(-d // GROUP)), np.float32)
    for g in range(scales.shape[1]):
        blk = x[:, g * GROUP:(g + 1) * GROUP]
        m = np.max(np.abs(blk), axis=1)                 # NaN if any is
        bad = ~np.isfinite(m)
        s = np.where(bad, np.nan, np.where(m < 2.0 ** -100, 0.0, np.where(bad, 0.0, m) / 127.0)).astype(np.float32)
        scales[:, g] = s
        s64 = s.astype(np.float64)[:, None]
        ok = s64[:, 0] > 0
        q = np.zeros_like(blk)
        q[ok] = np.rint(blk[ok] / s64[ok])              # numpy's rint rounds ties to even
        codes[:, g * GROUP:(g + 1) * GROUP] = q.astype(np.int8)
    return codes, scales


def act8_unpack(codes, scales):
    """The restored values: code * scale, rounded once to float32."""
    d = codes.shape[1]
    s = np.repeat(scales.astype(np.float64), GROUP, axis=1)[:, :d]
    return (codes.astype(np.float64) * s).astype(np.float32)


def linear_ce(x, w, targets):
    """(loss, lse, z) of the logits z = x w^T; targets < 0 or >= vocab: loss 0."""
    z = x @ w.T
    m = z.max(axis=1, keepdims=True)
    lse = (m + np.log(np.sum(np.exp(z - m), axis=1, keepdims=True)))[:, 0]
    live = (targets >= 0) & (targets < w.shape[0])
    loss = np.where(live, lse - z[np.arange(len(targets)), np.where(live, targets, 0)], 0.0)
    return loss, lse, z


def linear_ce_grad(x, w, targets, weights):
    """(dx, dw, g) of sum_t weights[t] loss[t]."""
    _, lse, z = linear_ce(x, w, targets)
    live = np.nonzero((targets >= 0) & (targets < w.shape[0]))[0]
    g = np.zeros_like(z)
    g[live] = np.exp(z[live] - lse[live, None])
    g[live, targets[live]] -= 1.0
    g[live] *= weights[live, None]
    return g @ w, g.T @ x, g
