"""The measured cases of the training-step operators around a Mixture-of-Memories
block: the residual stream's norms (before and after the block, with the gate and
the residual scale), the 8-bit activation checkpoints that its backward reads, and
the vocabulary's softmax cross entropy with its gradient.

With ``own`` false ``run`` computes each operator in elementary torch operations
in 32 bits; with ``own`` true it makes the calls of mixture_memories_layer_b200.

Formulas (row t, channel c, d channels, RMS norms with eps):

  x'    = x + res_scale * sigmoid(gate) * (y / rms(y)) * w_post      rms(a) = sqrt(mean(a^2) + eps)
  h     = (x' / rms(x')) * w_pre
  8-bit checkpoint: groups of 128 channels of a row, scale = float32(max|x| / 127),
          code = round_half_even(x / scale), restored x = code * scale
  loss_t = log(sum_v exp(z_tv)) - z_t,target,   z = x W^T;  targets < 0 are padding (loss 0)
"""
import math

import torch

own = False

EPS = 1e-5
GROUP = 128
PAD = -100

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one token of each of 256 sequences between two blocks (serving): latency
        dict(name="norm_decode", op="norm", n=256, d=1024, x="bf16", t="bf16", y=True, gate="token", scale=True, pre=True),
        # a batch of 8 x 2048 tokens of the 380M shape between two blocks
        dict(name="norm_train", op="norm", n=16384, d=1024, x="bf16", t="bf16", y=True, gate="elem", scale=True,
             pre=True),
        # float32 everywhere, a width that no vector load divides
        dict(name="norm_f32_odd", op="norm", n=6001, d=1537, x="f32", t="f32", y=True, gate="token", scale=False,
             pre=True),
        # the gradients of norm_train's call, its stream read from the 8-bit checkpoint
        dict(name="norm_bwd_train", op="norm_bwd", n=16384, d=1024, x="q8", t="bf16", g="f32", y=True, gate="elem",
             scale=True, pre=True),
        # float32, odd sizes, one gate a token: its gradient is a sum over the row
        dict(name="norm_bwd_f32_odd", op="norm_bwd", n=3001, d=1021, x="f32", t="f32", g="f32", y=True, gate="token",
             scale=True, pre=True),
        # a block's input stream kept in 8 bits in the forward pass and restored with
        # its pre-norm in the backward pass, at the wider model's size
        dict(name="ckpt_cycle", op="ckpt_norm", n=16384, d=2048, x="bf16", t="bf16"),
        # packing and restoring alone, float32, a ragged last group
        dict(name="ckpt_f32_odd", op="ckpt", n=4999, d=1000, x="f32"),
        # log-likelihoods of a few tokens (scoring): the vocabulary's matrix is read once
        dict(name="ce_score", op="ce", n=64, d=1024, v=32000, t="bf16", grad=False),
        # a training step's loss and gradients on 8 x 2048 tokens
        dict(name="ce_train", op="ce", n=16384, d=1024, v=32000, t="bf16", grad=True),
        # a short batch against a large vocabulary whose size nothing divides
        dict(name="ce_vocab_odd", op="ce", n=2047, d=1024, v=65003, t="bf16", grad=True),
        # float32 throughout, every size odd
        dict(name="ce_f32_odd", op="ce", n=1001, d=515, v=8009, t="f32", grad=True),
    ]


def _spread(rng, lo, hi):
    """A size spread over its logarithm; half of the draws are left ragged."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and n >= 16:
        n = n // 8 * 8
    return max(lo, min(hi, n))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "ckpt_norm", "ckpt", "ce", "ce"])
    if op == "ce":
        t = rng.choice(["bf16", "bf16", "f32"])
        # float32 costs six times the products of bf16: its sizes stay smaller
        d = _spread(rng, 64, 2048 if t == "bf16" else 1024)
        v = _spread(rng, 1000, 65003 if t == "bf16" else 16000)
        most = 16384 * 1024 * 32000 if t == "bf16" else 4096 * 1024 * 8192
        n = _spread(rng, 1, max(1, min(16384, most // (d * v))))
        return dict(op=op, n=n, d=d, v=v, t=t, grad=rng.random() < 0.7)
    d = _spread(rng, 64, 8192)
    n = _spread(rng, 1, max(1, min(32768, 16384 * 1024 // d)))
    if op == "ckpt":
        return dict(op=op, n=n, d=d, x=rng.choice(["bf16", "f32"]))
    x, t = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f32", "f32")])
    if op == "ckpt_norm":
        return dict(op=op, n=n, d=d, x=x, t=t)
    case = dict(op=op, n=n, d=d, x=x, t=t, y=True, gate=rng.choice(["none", "token", "elem"]),
                scale=rng.random() < 0.5, pre=rng.random() < 0.8)
    if case["pre"] and rng.random() < 0.2:
        case.update(y=False, gate="none", scale=False)      # the norm before the first block
    if op == "norm_bwd":
        case["g"] = rng.choice(["f32", "bf16"])
        if rng.random() < 0.4:
            case["x"] = "q8"
    return case


# -------------------------------------------------------------------- inputs

def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(dtype)


def _stream(gen, n, d, dtype):
    """A residual stream: channels of unequal size, tokens of unequal size."""
    x = torch.randn((n, d), generator=gen, device="cuda")
    x *= torch.exp(0.5 * torch.randn((1, d), generator=gen, device="cuda"))
    x *= torch.exp(0.3 * torch.randn((n, 1), generator=gen, device="cuda"))
    return x.to(dtype)


def _quantise(x):
    """(codes int8, scales float32 [n, groups], restored float32) of a checkpoint."""
    n, d = x.shape
    g = -(-d // GROUP)
    xp = torch.zeros((n, g * GROUP), device=x.device, dtype=torch.float32)
    xp[:, :d] = x.float()
    xp = xp.view(n, g, GROUP)
    s = (xp.abs().amax(dim=2).double() / 127.0).float()
    # values next to a border between two codes: the quotient in 64 bits
    q = torch.round(xp.double() / torch.where(s > 0, s, torch.ones_like(s)).double()[:, :, None]).float()
    r = (q * s[:, :, None]).view(n, g * GROUP)[:, :d].contiguous()
    return q.view(n, g * GROUP)[:, :d].to(torch.int8).contiguous(), s.contiguous(), r


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 1000003 + 17)
    op, n, d = case["op"], case["n"], case["d"]
    s = dict(case=case)
    if op == "ce":
        dt = DT[case["t"]]
        s["x"] = _normal(gen, (n, d), dt)
        s["w"] = _normal(gen, (case["v"], d), dt, 2.5 / math.sqrt(d))
        tg = torch.randint(0, case["v"], (n,), generator=gen, device="cuda", dtype=torch.int32)
        if n >= 4:                                           # some padding, as a packed batch has
            pad = torch.rand((n,), generator=gen, device="cuda") < 0.1
            pad[0] = False
            tg = torch.where(pad, torch.full_like(tg, PAD), tg)
        s["targets"] = tg
        if own:
            from mixture_memories_layer_b200.lm_head import LMHead
            s["head"] = LMHead(s["w"])
        return s
    xdt = torch.float32 if case["x"] in ("f32", "q8") else torch.bfloat16
    s["x"] = _stream(gen, n, d, xdt)
    if op in ("norm", "norm_bwd"):
        t = DT[case["t"]]
        if case["x"] == "q8":
            s["codes"], s["scales"], _ = _quantise(s["x"].to(torch.bfloat16))
        s["y"] = _normal(gen, (n, d), t, 0.7) if case["y"] else None
        s["gate"] = (None if case["gate"] == "none" else
                     _normal(gen, (n, 1) if case["gate"] == "token" else (n, d), t, 1.0))
        s["w_post"] = 1.0 + 0.2 * _normal(gen, (d,), torch.float32) if case["y"] else None
        s["res_scale"] = 0.5 + 0.1 * _normal(gen, (d,), torch.float32) if case["scale"] else None
        s["w_pre"] = 1.0 + 0.2 * _normal(gen, (d,), torch.float32) if case["pre"] else None
        if op == "norm_bwd":
            g = DT[case["g"]]
            s["dx_out"] = _normal(gen, (n, d), g, 1e-2)
            s["dh"] = _normal(gen, (n, d), g, 1e-2) if case["pre"] else None
    elif op == "ckpt_norm":
        s["w_pre"] = 1.0 + 0.2 * _normal(gen, (d,), torch.float32)
    if own:
        _buffers(s)
    return s


def _buffers(s):
    """What a program that calls the library keeps: outputs and workspaces."""
    from mixture_memories_layer_b200 import binding as B
    case = s["case"]
    op, n, d = case["op"], case["n"], case["d"]
    new = lambda shape, dt: torch.empty(shape, dtype=dt, device="cuda")
    f32 = torch.float32
    if op == "norm":
        s["x_out"] = new((n, d), s["x"].dtype) if case["y"] else None
        s["h"] = new((n, d), DT[case["t"]]) if case["pre"] else None
    elif op == "norm_bwd":
        g, t = DT[case["g"]], DT[case["t"]]
        s["dx"] = new((n, d), g)
        s["dy"] = new((n, d), t) if case["y"] else None
        s["dgate"] = new(tuple(s["gate"].shape), t) if s["gate"] is not None else None
        s["dw_post"] = new((d,), f32) if case["y"] else None
        s["dres_scale"] = new((d,), f32) if case["scale"] else None
        s["dw_pre"] = new((d,), f32) if case["pre"] else None
        s["ws"] = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, d))
    else:
        s["k8"] = B.new_act8(n, d)
        s["x_hat"] = new((n, d), s["x"].dtype)
        if op == "ckpt_norm":
            s["h"] = new((n, d), DT[case["t"]])


# --------------------------------------------------------------------- a pass

def run(state):
    return _own(state) if own else _plain(state)


def _own(s):
    from mixture_memories_layer_b200 import binding as B
    case = s["case"]
    op = case["op"]
    if op == "ce":
        r = s["head"].loss(s["x"], s["targets"])
        out = dict(loss=r["loss"], lse=r["lse"], mean=r["mean"])
        if case["grad"]:
            g = s["head"].backward(s["x"], s["targets"])
            out.update(dx=g["dx"], dw=g["dw"])
        return out
    if op == "norm":
        B.mom_residual_norm(s["x"], s["y"], s["gate"], s["w_post"], s["res_scale"], s["w_pre"], EPS, s["x_out"],
                            s["h"])
        return {k: s[k] for k in ("x_out", "h") if s[k] is not None}
    if op == "norm_bwd":
        x = (s["codes"], s["scales"]) if case["x"] == "q8" else s["x"]
        B.mom_residual_norm_bwd(x, s["y"], s["gate"], s["w_post"], s["res_scale"], s["w_pre"], EPS, s["dx_out"],
                                s["dh"], s["dx"], s["dy"], s["dgate"], s["dw_post"], s["dres_scale"], s["dw_pre"],
                                s["ws"])
        return {k: s[k] for k in ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre") if s[k] is not None}
    B.mom_act_pack8(s["x"], s["k8"])
    if op == "ckpt":
        B.mom_act_unpack8(s["k8"], s["x_hat"])
        return dict(x_hat=s["x_hat"], scales=s["k8"][1])
    B.mom_residual_norm(s["k8"], None, None, None, None, s["w_pre"], EPS, s["x_hat"], s["h"])
    return dict(x_hat=s["x_hat"], scales=s["k8"][1], h=s["h"])


def _rms(a):
    return torch.rsqrt((a * a).mean(dim=1, keepdim=True) + EPS)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "ce":
        return _plain_ce(s)
    if op == "norm":
        x = s["x"].float()
        out = {}
        if case["y"]:
            y = s["y"].float()
            u = y * _rms(y) * s["w_post"]
            if s["gate"] is not None:
                u = u * (1.0 / (1.0 + torch.exp(-s["gate"].float())))
            if s["res_scale"] is not None:
                u = u * s["res_scale"]
            x = x + u
            out["x_out"] = x.to(s["x"].dtype)
        if case["pre"]:
            out["h"] = (x * _rms(x) * s["w_pre"]).to(DT[case["t"]])
        return out
    if op == "norm_bwd":
        return _plain_bwd(s)
    _, scales, r = _quantise(s["x"])
    out = dict(x_hat=r.to(s["x"].dtype), scales=scales)
    if op == "ckpt_norm":
        out["h"] = (r * _rms(r) * s["w_pre"]).to(DT[case["t"]])
    return out


def _plain_bwd(s):
    case = s["case"]
    t, gt = DT[case["t"]], DT[case["g"]]
    if case["x"] == "q8":
        x = s["codes"].float() * s["scales"].repeat_interleave(GROUP, dim=1)[:, :case["d"]]
    else:
        x = s["x"].float()
    out = {}
    if case["y"]:
        y = s["y"].float()
        ry = _rms(y)
        yn = y * ry
        sg = 1.0 / (1.0 + torch.exp(-s["gate"].float())) if s["gate"] is not None else None
        coef = s["w_post"] if s["res_scale"] is None else s["w_post"] * s["res_scale"]
        gc = coef if sg is None else sg * coef
        x = x + yn * gc
    dx = s["dx_out"].float()
    if case["pre"]:
        dh = s["dh"].float()
        r = _rms(x)
        xn = x * r
        out["dw_pre"] = (dh * xn).sum(dim=0)
        dn = dh * s["w_pre"]
        dx = dx + r * (dn - xn * (dn * xn).mean(dim=1, keepdim=True))
    out["dx"] = dx.to(gt)
    if case["y"]:
        a = dx * yn if sg is None else dx * yn * sg
        col = a.sum(dim=0)
        out["dw_post"] = col if s["res_scale"] is None else col * s["res_scale"]
        if s["res_scale"] is not None:
            out["dres_scale"] = col * s["w_post"]
        if sg is not None:
            dg = a * coef * (1.0 - sg)
            out["dgate"] = (dg.sum(dim=1, keepdim=True) if case["gate"] == "token" else dg).to(t)
        du = dx * gc
        out["dy"] = (ry * (du - yn * (du * yn).mean(dim=1, keepdim=True))).to(t)
    return {k: out[k] for k in ("dx", "dy", "dgate", "dw_post", "dres_scale", "dw_pre") if k in out}


def _plain_ce(s):
    case = s["case"]
    x, w, tg = s["x"].float(), s["w"].float(), s["targets"].long()
    z = x @ w.t()
    m = z.amax(dim=1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(dim=1, keepdim=True)
    lse = (m + torch.log(total))[:, 0]
    live = tg >= 0
    at = tg.clamp(min=0)[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    count = live.sum().clamp(min=1).float()
    out = dict(loss=loss, lse=lse, mean=loss.sum() / count)
    if case["grad"]:
        wt = torch.where(live, 1.0 / count, torch.zeros_like(lse))[:, None]
        p *= wt / total
        p.scatter_add_(1, at, -wt)
        out["dx"] = (p @ w).to(s["x"].dtype)
        out["dw"] = (p.t() @ x).to(s["w"].dtype)
    return out


# ------------------------------------------------------------ the definition

def exact(case, seed):
    """The outputs from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, d = case["op"], case["d"]
    f = lambda a: None if a is None else a.to(torch.float64)
    if op == "ce":
        return _exact_ce(s)
    if op in ("ckpt", "ckpt_norm"):
        x = f(s["x"])
        hat, scales = torch.empty_like(x), torch.empty((case["n"], -(-d // GROUP)), device="cuda")
        for j in range(scales.shape[1]):
            blk = x[:, j * GROUP:(j + 1) * GROUP]
            sc = (blk.abs().max(dim=1).values / 127.0).float()
            scales[:, j] = sc
            sc = sc.double()[:, None]
            hat[:, j * GROUP:(j + 1) * GROUP] = torch.where(sc > 0, torch.round(blk / sc) * sc, torch.zeros_like(blk))
        out = dict(x_hat=hat, scales=scales.double())
        if op == "ckpt_norm":
            out["h"] = hat / torch.sqrt((hat ** 2).sum(1, keepdim=True) / d + EPS) * f(s["w_pre"])
        return out
    if case["x"] == "q8":
        x = torch.stack([s["codes"][:, c].double() * s["scales"][:, c // GROUP].double() for c in range(d)], dim=1)
    else:
        x = f(s["x"])
    # the forward pass, as one differentiable function of its inputs
    leaves = {"x": x, "y": f(s["y"]), "gate": f(s["gate"]), "w_post": f(s["w_post"]),
              "res_scale": f(s["res_scale"]), "w_pre": f(s["w_pre"])}
    leaves = {k: a.requires_grad_(op == "norm_bwd") for k, a in leaves.items() if a is not None}
    stream = leaves["x"]
    if case["y"]:
        y = leaves["y"]
        add = y / torch.sqrt((y ** 2).sum(1, keepdim=True) / d + EPS) * leaves["w_post"]
        if "gate" in leaves:
            add = add / (1.0 + torch.exp(-leaves["gate"]))
        if "res_scale" in leaves:
            add = add * leaves["res_scale"]
        stream = stream + add
    h = None
    if case["pre"]:
        h = stream / torch.sqrt((stream ** 2).sum(1, keepdim=True) / d + EPS) * leaves["w_pre"]
    if op == "norm":
        out = {}
        if case["y"]:
            out["x_out"] = stream
        if h is not None:
            out["h"] = h
        return out
    total = (stream * f(s["dx_out"])).sum()
    if h is not None:
        total = total + (h * f(s["dh"])).sum()
    names = list(leaves)
    grads = dict(zip(names, torch.autograd.grad(total, [leaves[k] for k in names])))
    at = dict(dx="x", dy="y", dgate="gate", dw_post="w_post", dres_scale="res_scale", dw_pre="w_pre")
    return {k: grads[v] for k, v in at.items() if v in grads}


def _exact_ce(s):
    case = s["case"]
    n, d, v = case["n"], case["d"], case["v"]
    w = s["w"].double()
    tg = s["targets"].long()
    count = max(1, int((tg >= 0).sum()))
    loss, lse = torch.zeros(n, device="cuda").double(), torch.zeros(n, device="cuda").double()
    dx = torch.zeros((n, d), device="cuda").double() if case["grad"] else None
    dw = torch.zeros((v, d), device="cuda").double() if case["grad"] else None
    for r in range(0, n, 1024):
        x = s["x"][r:r + 1024].double()
        z = torch.mm(x, w.T)
        lse[r:r + 1024] = torch.logsumexp(z, dim=1)
        rows = torch.nonzero(tg[r:r + 1024] >= 0)[:, 0]
        cols = tg[r:r + 1024][rows]
        loss[r + rows] = lse[r + rows] - z[rows, cols]
        if case["grad"]:
            g = torch.zeros_like(z)
            g[rows] = torch.softmax(z[rows], dim=1) / count
            g[rows, cols] -= 1.0 / count
            dx[r:r + 1024] = torch.mm(g, w)
            dw += torch.mm(g.T, x)
    out = dict(loss=loss, lse=lse, mean=loss.sum() / count)
    if case["grad"]:
        out.update(dx=dx, dw=dw)
    return out


# ------------------------------------------------------------------ the floor

def work(case):
    op, n, d = case["op"], case["n"], case["d"]
    size = {"bf16": 2, "f32": 4, "q8": 1}
    if op == "ce":
        e, v = size[case["t"]], case["v"]
        b = n * d * e + v * d * e + n * 12
        fl = 2 * n * d * v
        if case["grad"]:
            # the logits once, the two products of the gradient
            b += n * d * e + v * d * e
            fl *= 3
        return dict(bytes=b, flops=fl)
    el = n * d
    groups = n * (-(-d // GROUP)) * 4
    if op in ("ckpt", "ckpt_norm"):
        # the stream in, codes and scales out and in again, the restored stream (and h) out
        b = el * (2 * size[case["x"]] + 2) + 2 * groups
        if op == "ckpt_norm":
            b += el * size[case["t"]] + 4 * d
        return dict(bytes=b, flops=8 * el)
    e = size[case["t"]]
    gate = 0 if case["gate"] == "none" else n * e if case["gate"] == "token" else el * e
    b = el * size[case["x"]] + (groups if case["x"] == "q8" else 0) + gate + 12 * d
    if case["y"]:
        b += el * e
    if op == "norm":
        b += (el * size[case["x"]] if case["y"] else 0) + (el * e if case["pre"] else 0)
        return dict(bytes=b, flops=12 * el)
    g = size[case["g"]]
    b += el * g * (3 if case["pre"] else 2) + (el * e if case["y"] else 0) + gate + 12 * d
    return dict(bytes=b, flops=30 * el)
