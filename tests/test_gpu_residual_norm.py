"""The residual stream's norms, their adjoint and the 8-bit activation
checkpoints on the GPU against fp64 (oracle/train_ops.py).

Tolerances.  Outputs: half a step of the output's type relative to the value
(torch.finfo(t).eps / 2) plus float32 arithmetic.  Each element passes through
at most ~40 float32 roundings (two row sums of at most 32 serial terms a lane,
5 shuffles and 16 warps each enter with half their weight through the square
root; the sigmoid, the products): 128 roundings of 2^-24 = 2^-17 of the
magnitudes that meet in it bound them.  A column sum adds one rounding a row.
Checkpoints are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T

pytestmark = pytest.mark.gpu

EPS = 1e-5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F32 = 2.0 ** -17


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _close(got, ref, size, extra=F32):
    half = torch.finfo(got.dtype).eps / 2
    g = _np(got)
    assert g.shape == ref.shape
    lim = half * np.abs(ref) + extra * size + 1e-30
    bad = ~(np.abs(g - ref) <= lim)
    assert not bad.any(), (int(bad.sum()), float(np.nanmax(np.abs(g - ref) / lim)))


def _inputs(n, d, x, t, gate, scale=True, pre=True, y=True, seed=0):
    from mixture_memories_layer_b200 import binding as B
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + n * 31 + d)
    r = lambda shape, dt, std=1.0: (torch.randn(shape, generator=g, device="cuda") * std).to(dt)
    p = dict(x=r((n, d), torch.bfloat16 if x == "bf16" else torch.float32, 1.5), y=r((n, d), DT[t]) if y else None,
             gate={"none": None, "token": r((n, 1), DT[t]), "elem": r((n, d), DT[t])}[gate],
             w_post=1 + r((d,), torch.float32, 0.3) if y else None,
             res_scale=0.5 + r((d,), torch.float32, 0.2) if scale else None,
             w_pre=1 + r((d,), torch.float32, 0.3) if pre else None)
    x64 = p["x"]
    if x == "q8":
        k8 = B.new_act8(n, d)
        B.mom_act_pack8(p["x"], k8)
        x64 = torch.empty_like(p["x"])
        B.mom_act_unpack8(k8, x64)
        p["x"] = k8
    return p, x64


def _ref(p, x64):
    q = {k: _np(v) for k, v in p.items() if k != "x"}
    return dict(q, x=_np(x64))


SIZES = [(1, 1024), (1, 1), (3, 7), (5, 8), (33, 64), (9, 127), (17, 128), (4, 256), (6, 257), (130, 1000),
         (64, 1024), (11, 1537), (5, 2048), (7, 5000), (3, 8192), (2, 12288), (3, 16384), (3, 16383)]


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("x,t,gate", [("bf16", "bf16", "elem"), ("f32", "bf16", "token"), ("f32", "f32", "elem"),
                                      ("q8", "bf16", "none"), ("q8", "f32", "token")])
def test_forward_against_fp64(n, d, x, t, gate):
    from mixture_memories_layer_b200 import binding as B
    p, x64 = _inputs(n, d, x, t, gate)
    x_out = torch.empty((n, d), dtype=x64.dtype, device="cuda")
    h = torch.empty((n, d), dtype=DT[t], device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=x_out, h=h)
    q = _ref(p, x64)
    xo, hh = T.residual_norm(**q, eps=EPS)
    size = np.abs(q["x"]) + np.abs(xo - q["x"])
    _close(x_out, xo, size)
    r = 1 / np.sqrt(np.mean(xo * xo, axis=1, keepdims=True) + EPS)
    _close(h, hh, size * r * np.abs(q["w_pre"]) + np.abs(hh))


@pytest.mark.parametrize("n,d", SIZES)
@pytest.mark.parametrize("x,t,g,gate,scale", [("bf16", "bf16", "bf16", "elem", True), ("f32", "bf16", "f32", "token", False),
                                              ("f32", "f32", "f32", "elem", True), ("q8", "bf16", "f32", "none", True),
                                              ("q8", "f32", "f32", "token", True), ("bf16", "bf16", "f32", "none", False)])
def test_backward_against_fp64(n, d, x, t, g, gate, scale):
    from mixture_memories_layer_b200 import binding as B
    p, x64 = _inputs(n, d, x, t, gate, scale=scale, seed=1)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    dx_out = torch.randn((n, d), generator=gen, device="cuda").to(DT[g])
    dh = torch.randn((n, d), generator=gen, device="cuda").to(DT[g])
    got = _backward(p, dx_out, dh, DT[t])
    ref = T.residual_norm_bwd(**_ref(p, x64), eps=EPS, dx_out=_np(dx_out), dh=_np(dh))
    for k, v in got.items():
        if v is None:
            continue
        cols = k.startswith("dw") or k == "dres_scale"
        tok = k == "dgate" and gate == "token"
        _close(v, ref[k], ref["size"][k], F32 + (n * 2.0 ** -24 if cols else d * 2.0 ** -24 / 32 if tok else 0))


def _backward(p, dx_out, dh, t, want=None):
    from mixture_memories_layer_b200 import binding as B
    like = dx_out if dx_out is not None else dh
    n, d = like.shape
    e = lambda shape, dt: torch.full(shape, float("nan"), dtype=dt, device="cuda")
    y = p["y"] is not None
    o = dict(dx=e((n, d), like.dtype), dy=e((n, d), t) if y else None,
             dgate=e(tuple(p["gate"].shape), t) if p["gate"] is not None else None,
             dw_post=e((d,), torch.float32) if y else None,
             dres_scale=e((d,), torch.float32) if p["res_scale"] is not None else None,
             dw_pre=e((d,), torch.float32) if dh is not None else None)
    ws = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, d))
    B.mom_residual_norm_bwd(**p, eps=EPS, dx_out=dx_out, dh=dh, **o, ws=ws)
    return o


@pytest.mark.parametrize("d", [1024, 515])
def test_the_norm_before_the_first_block_and_the_stream_after_the_last(d):
    from mixture_memories_layer_b200 import binding as B
    n = 37
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    a, b = (torch.randn((n, d), generator=gen, device="cuda") for _ in range(2))
    # no block: h = norm(x) alone, dx = dx_out + its adjoint
    p, x64 = _inputs(n, d, "bf16", "bf16", "none", scale=False, y=False)
    h = torch.empty((n, d), dtype=torch.bfloat16, device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=None, h=h)
    q = _ref(p, x64)
    _, hh = T.residual_norm(**q, eps=EPS)
    _close(h, hh, 2 * np.abs(hh))
    for dx_out in (a, None):
        ref = T.residual_norm_bwd(**q, eps=EPS, dx_out=_np(dx_out), dh=_np(b))
        got = _backward(p, dx_out, b, torch.bfloat16)
        for k in ("dx", "dw_pre"):
            _close(got[k], ref[k], ref["size"][k], F32 + n * 2.0 ** -24)
    # no norm after it: x_out alone, the gradient from dx_out alone
    p, x64 = _inputs(n, d, "f32", "bf16", "elem", pre=False)
    x_out = torch.empty((n, d), device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=x_out, h=None)
    q = _ref(p, x64)
    xo, _ = T.residual_norm(**q, eps=EPS)
    _close(x_out, xo, np.abs(q["x"]) + np.abs(xo - q["x"]))
    ref = T.residual_norm_bwd(**q, eps=EPS, dx_out=_np(a), dh=None)
    got = _backward(p, a, None, torch.bfloat16)
    assert torch.equal(got["dx"], a)
    for k in ("dy", "dgate", "dw_post", "dres_scale"):
        _close(got[k], ref[k], ref["size"][k], F32 + n * 2.0 ** -24)


def test_gradients_are_differences_of_the_forward():
    """Along random directions, float32, steps of 2^-7: the difference quotient
    of a sum over the outputs against the adjoint.  The quotient's error is the
    second derivative's (step^2, below 2^-14 x ~8 of the directional size) and
    the outputs' rounding over the step (2^-24 x 2^7 x sqrt of the terms)."""
    from mixture_memories_layer_b200 import binding as B
    n, d = 24, 96
    p, _ = _inputs(n, d, "f32", "f32", "elem", seed=5)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(9)
    r = lambda t: torch.randn(t.shape, generator=gen, device="cuda")
    dx_out, dh = r(p["x"]), r(p["x"])
    got = _backward(p, dx_out, dh, torch.float32)

    def f(q):
        x_out, h = torch.empty_like(q["x"]), torch.empty_like(q["x"])
        B.mom_residual_norm(**q, eps=EPS, x_out=x_out, h=h)
        return float((dx_out.double() * x_out.double()).sum() + (dh.double() * h.double()).sum())
    step = 2.0 ** -7
    for name, out in dict(x="dx", y="dy", gate="dgate", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre").items():
        v = r(p[name])
        v /= v.norm()
        num = (f({**p, name: p[name] + step * v}) - f({**p, name: p[name] - step * v})) / (2 * step)
        want = float((got[out].double() * v.double()).sum())
        assert abs(num - want) < 2e-3 * float(got[out].double().norm()), name


def test_outputs_may_take_their_inputs_place():
    from mixture_memories_layer_b200 import binding as B
    n, d = 65, 768
    p, _ = _inputs(n, d, "bf16", "bf16", "elem", seed=2)
    x_out, h = torch.empty_like(p["x"]), torch.empty_like(p["y"])
    B.mom_residual_norm(**p, eps=EPS, x_out=x_out, h=h)
    q = {k: v.clone() for k, v in p.items()}
    B.mom_residual_norm(**q, eps=EPS, x_out=q["x"], h=q["y"])
    assert torch.equal(q["x"], x_out) and torch.equal(q["y"], h)
    dx_out, dh = torch.randn((n, d), device="cuda"), torch.randn((n, d), device="cuda")
    got = _backward(p, dx_out, dh, torch.bfloat16)
    q = {k: v.clone() for k, v in p.items()}
    ws = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, d))
    dgate = torch.empty_like(p["gate"])
    g = dx_out.clone()
    B.mom_residual_norm_bwd(**q, eps=EPS, dx_out=g, dh=dh, dx=g, dy=q["y"], dgate=dgate, dw_post=None, dres_scale=None,
                            dw_pre=None, ws=ws)
    assert torch.equal(g, got["dx"]) and torch.equal(q["y"], got["dy"]) and torch.equal(dgate, got["dgate"])


def test_rows_of_other_alignments_and_rows_beyond_are_left():
    """Rows that start at odd element addresses, and a call over the first rows
    of larger arrays."""
    from mixture_memories_layer_b200 import binding as B
    n, d = 9, 1024
    for off in (1, 4):
        flat = torch.randn(n * d + off, device="cuda").bfloat16()
        x = flat[off:].view(n, d)
        p, _ = _inputs(n, d, "bf16", "bf16", "token", seed=4)
        p["x"] = x
        big = torch.full((n + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
        h = torch.full((n + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
        B.mom_residual_norm(**p, eps=EPS, x_out=big[:n], h=h[:n])
        q = _ref(p, x)
        xo, hh = T.residual_norm(**q, eps=EPS)
        size = np.abs(q["x"]) + np.abs(xo - q["x"])
        _close(big[:n], xo, size)
        assert torch.all(big[n:] == 7) and torch.all(h[n:] == 7)
        k8 = B.new_act8(n, d)
        B.mom_act_pack8(x, k8)
        c, s = T.act8_pack(_np(x))
        assert np.array_equal(k8[0].cpu().numpy(), c) and np.array_equal(k8[1].cpu().numpy(), s)


def test_no_rows():
    from mixture_memories_layer_b200 import binding as B
    d = 64
    p, _ = _inputs(0, d, "bf16", "bf16", "elem")
    z = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=z, h=z)
    got = _backward(p, z, z, torch.bfloat16)
    for k in ("dw_post", "dres_scale", "dw_pre"):
        assert torch.all(got[k] == 0)
    k8 = B.new_act8(0, d)
    B.mom_act_pack8(z, k8)
    B.mom_act_unpack8(k8, z)


def test_a_row_of_zeros_and_a_row_of_nan_keep_to_themselves():
    from mixture_memories_layer_b200 import binding as B
    n, d = 6, 300
    p, _ = _inputs(n, d, "f32", "f32", "token", seed=8)
    clean_x, clean_h = torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=clean_x, h=clean_h)
    p["y"][2] = 0
    p["x"][2] = 0
    p["y"][4, 7] = float("nan")
    x_out, h = torch.empty((n, d), device="cuda"), torch.empty((n, d), device="cuda")
    B.mom_residual_norm(**p, eps=EPS, x_out=x_out, h=h)
    rows = [0, 1, 3, 5]
    assert torch.equal(x_out[rows], clean_x[rows]) and torch.equal(h[rows], clean_h[rows])
    assert torch.all(h[2] == 0) and torch.all(torch.isnan(h[4]))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 127), (5, 128), (7, 129), (4, 256), (33, 1000), (300, 1024), (3, 16390),
                                 (2, 70001)])
def test_checkpoints_bit_for_bit(dt, n, d):
    from mixture_memories_layer_b200 import binding as B
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n * d)
    x = (torch.randn((n, d), generator=gen, device="cuda") *
         torch.exp(4 * torch.randn((n, 1), generator=gen, device="cuda"))).to(DT[dt])
    k8 = B.new_act8(n, d)
    B.mom_act_pack8(x, k8)
    c, s = T.act8_pack(_np(x))
    assert np.array_equal(k8[1].cpu().numpy(), s)
    assert np.array_equal(k8[0].cpu().numpy(), c)
    back = torch.empty_like(x)
    B.mom_act_unpack8(k8, back)
    want = torch.as_tensor(T.act8_unpack(c, s)).to(DT[dt])
    assert torch.equal(back.cpu(), want)


def test_checkpoint_ties_extremes_and_non_finite_groups():
    from mixture_memories_layer_b200 import binding as B
    d = 1024
    x = torch.zeros((6, d), device="cuda")
    # all halves of a scale of 2, then of a scale that is not a power of two
    x[0, :512] = torch.arange(-256, 256, device="cuda").float() * 0.99
    x[1] = (torch.arange(d, device="cuda").float() % 255 - 127) * 0.5 * 3
    x[2, ::128] = 254.0
    x[2, 1::128] = torch.tensor([1., 3., 5., 7., -1., -3., -5., 253.], device="cuda")
    x[3] = 3e38
    x[3, 1] = -1e-45
    x[4, 3], x[4, 300], x[4, 600] = float("inf"), float("nan"), float("-inf")
    x[5, :128] = 2.0 ** -101
    x[5, 128:256] = 2.0 ** -100
    for dt in (torch.float32, torch.bfloat16):
        y = x.to(dt)
        for width in (d, 1023):                    # 16-byte rows and single elements
            z = y[:, :width].contiguous()
            k8 = B.new_act8(6, width)
            B.mom_act_pack8(z, k8)
            c, s = T.act8_pack(_np(z))
            assert np.array_equal(k8[1].cpu().numpy(), s, equal_nan=True)
            assert np.array_equal(k8[0].cpu().numpy(), c)
            back = torch.empty((6, width), device="cuda")
            B.mom_act_unpack8(k8, back)
            assert np.array_equal(back.cpu().numpy(), T.act8_unpack(c, s), equal_nan=True)


@pytest.mark.parametrize("n,d", [(70, 1024), (13, 777)])
def test_the_stream_is_packed_while_it_is_read(n, d):
    from mixture_memories_layer_b200 import binding as B
    for y in (True, False):
        p, _ = _inputs(n, d, "bf16", "bf16", "elem" if y else "none", scale=y, y=y, seed=6)
        x = p["x"].clone()
        plain, packed = torch.empty_like(x), torch.empty_like(x)
        h0, h1 = torch.empty_like(x), torch.empty_like(x)
        B.mom_residual_norm(**p, eps=EPS, x_out=plain, h=h0)
        k8, alone = B.new_act8(n, d), B.new_act8(n, d)
        p["x"] = packed.copy_(x)
        B.mom_residual_norm(**p, eps=EPS, x_out=packed, h=h1, pack=k8)       # x_out in x's place
        B.mom_act_pack8(x, alone)
        assert torch.equal(k8[0], alone[0]) and torch.equal(k8[1], alone[1])
        assert torch.equal(plain, packed) and torch.equal(h0, h1)


def test_another_stream_and_a_captured_graph():
    from mixture_memories_layer_b200 import binding as B
    n, d = 200, 1024
    p, _ = _inputs(n, d, "bf16", "bf16", "elem", seed=11)
    a, b = torch.randn((n, d), device="cuda"), torch.randn((n, d), device="cuda")
    want = _backward(p, a, b, torch.bfloat16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    e = lambda t: torch.zeros_like(t)
    o = {k: e(v) for k, v in want.items()}
    ws = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, d))
    torch.cuda.synchronize()
    B.mom_residual_norm_bwd(**p, eps=EPS, dx_out=a, dh=b, **o, ws=ws, stream=s)
    s.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.mom_residual_norm_bwd(**p, eps=EPS, dx_out=a, dh=b, **o, ws=ws)
    for k in o:
        o[k].zero_()
    p["y"].mul_(0.5)
    want = _backward(p, a, b, torch.bfloat16)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o[k], want[k]) for k in want)


# more rows than the GPU holds at once: every CTA walks several, the copies
# ahead of it wrap around their slots
MANY = [(20000, 200, "bf16", "bf16"), (12001, 256, "q8", "f32"), (4003, 1024, "f32", "f32"), (1701, 2048, "q8", "bf16"),
        (901, 4000, "bf16", "bf16"), (401, 8192, "f32", "bf16"), (310, 9000, "q8", "bf16"), (3001, 1021, "f32", "bf16"),
        (905, 3001, "bf16", "bf16"), (403, 7777, "f32", "f32")]


@pytest.mark.parametrize("n,d,x,t", MANY)
def test_many_rows_forward(n, d, x, t):
    test_forward_against_fp64(n, d, x, t, "token" if n % 2 else "elem")


@pytest.mark.parametrize("n,d,x,t", MANY)
def test_many_rows_backward(n, d, x, t):
    test_backward_against_fp64(n, d, x, t, "f32", "token" if n % 2 else "elem", n % 4 != 1)


@pytest.mark.parametrize("n,d,dt", [(9001, 1024, "bf16"), (40001, 256, "f32"), (2003, 8200, "bf16"), (3001, 1001, "f32")])
def test_many_rows_restore_and_norm(n, d, dt):
    """The checkpoint of many rows, restored with its norm: the stream bit for
    bit as mom_act_unpack8 restores it."""
    from mixture_memories_layer_b200 import binding as B
    p, _ = _inputs(n, d, dt, dt, "none", scale=False, y=False, seed=21)
    k8 = B.new_act8(n, d)
    B.mom_act_pack8(p["x"], k8)
    codes, scales = T.act8_pack(_np(p["x"]).astype(np.float32))
    assert np.array_equal(k8[0].cpu().numpy(), codes) and np.array_equal(k8[1].cpu().numpy(), scales)
    x_hat, x_out, h = torch.empty_like(p["x"]), torch.empty_like(p["x"]), torch.empty_like(p["x"])
    B.mom_act_unpack8(k8, x_hat)
    B.mom_residual_norm(k8, None, None, None, None, p["w_pre"], EPS, x_out, h)
    assert torch.equal(x_hat, x_out)
    x32 = torch.empty((n, d), device="cuda")
    B.mom_act_unpack8(k8, x32)
    _, hh = T.residual_norm(x=_np(x32), y=None, gate=None, w_post=None, res_scale=None, w_pre=_np(p["w_pre"]), eps=EPS)
    r = np.abs(hh)
    _close(h, hh, r)


def test_gates_at_their_ends():
    """Gates of +-infinity, large and small logits: exactly 0 or the whole
    block, and a gradient that does not cancel (1 - sigma = e^-z / (1 + e^-z)
    for z > 0)."""
    from mixture_memories_layer_b200 import binding as B
    n, d = 12, 512
    p, x64 = _inputs(n, d, "f32", "f32", "token", seed=31)
    z = torch.tensor([float("inf"), float("-inf"), 200.0, -200.0, 80.0, -80.0, 30.0, -30.0, 15.0, -15.0, 8.0, 0.0],
                     device="cuda").view(n, 1)
    for gate in (z, z.expand(n, d).contiguous()):
        q = dict(p, gate=gate)
        x_out, h = torch.empty_like(p["x"]), torch.empty_like(p["x"])
        B.mom_residual_norm(**q, eps=EPS, x_out=x_out, h=h)
        whole, none = torch.empty_like(x_out), torch.empty_like(h)
        B.mom_residual_norm(**dict(q, gate=None), eps=EPS, x_out=whole, h=none)
        assert torch.equal(x_out[0], whole[0]) and torch.equal(x_out[1], p["x"][1])
        gen = torch.Generator(device="cuda")
        gen.manual_seed(5)
        dx_out = torch.randn((n, d), generator=gen, device="cuda")
        dh = torch.randn((n, d), generator=gen, device="cuda")
        got = _backward(q, dx_out, dh, torch.float32)
        assert torch.all(got["dgate"][:2] == 0)
        # |z| <= 15, where float64 forms 1 - sigma to 2^-30: the error stays
        # relative to sigma (1 - sigma).  The exponential adds two ulps and its
        # argument's rounding, |z| 2^-24 relative, to the 2^-17 above; a token's
        # gate is a sum over the row.
        mid = slice(8, 12)
        ref = T.residual_norm_bwd(**dict(_ref(q, x64), gate=_np(gate.clamp(-300, 300))), eps=EPS, dx_out=_np(dx_out),
                                  dh=_np(dh))
        zz = _np(z)[mid]
        size = ref["size"]["dgate"][mid] / (1 + np.exp(zz))
        lim = (F32 + 2.0 ** -22 + np.abs(zz) * 2.0 ** -23 + d * 2.0 ** -24 / 32) * size
        assert np.all(np.abs(_np(got["dgate"])[mid] - ref["dgate"][mid]) <= lim)
