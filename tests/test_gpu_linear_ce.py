"""The vocabulary's cross entropy on the GPU against fp64 (oracle/train_ops.py).

Tolerances, per element and from the magnitudes that meet in it.  With u =
2^-24 and P = |x| |w|^T: a logit is a chain of ceil(d / 16) tensor-core
additions (each may truncate: 2u of the running magnitude) of exact products,
so |dz| <= 2u (ceil(d / 16) + 16) P; float32 operands run six such chains and
drop parts below 2^-22 of a product.  lse follows max |dz| with the
exponentials' and the sum's error (2^-21) and its own rounding; loss adds z's.
A gradient's entry g = r (p - [target]) carries |dz| + |dlse| + 2^-20 of r p
(or r) and half a step of bf16, 2^-8 (float32: its parts' 2^-22); dx and dw
add one product's chain and half a step of their own type."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
U = 2.0 ** -24


def _np(t):
    return t.detach().double().cpu().numpy()


def _problem(n, d, v, t, seed=0, pad=0.2, std=2.5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 104729 + n + 3 * d + 7 * v)
    x = torch.randn((n, d), generator=g, device="cuda").to(DT[t])
    w = (torch.randn((v, d), generator=g, device="cuda") * (std / d ** 0.5)).to(DT[t])
    tg = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    if n > 1:
        tg[torch.rand(n, generator=g, device="cuda") < pad] = -100
    return x, w, tg


def _chain(k, t):
    steps = -(-k // 16) * (6 if t == "f32" else 1) + 16
    return 2 * U * steps + (2.0 ** -22 if t == "f32" else 0)


def _limits(x, w, tg, r, t):
    """(dz, dlse, dloss, ddx, ddw) error bounds, without the outputs' own rounding."""
    n, d = x.shape
    v = w.shape[0]
    loss, lse, z = T.linear_ce(x, w, tg)
    dz = _chain(d, t) * (np.abs(x) @ np.abs(w).T)
    dlse = dz.max(axis=1) + 2.0 ** -21 + 4 * U * np.abs(lse)
    at = np.where((tg >= 0) & (tg < v), tg, 0)
    dloss = dlse + dz[np.arange(n), at] + 2 * U * np.abs(lse)
    _, _, g = T.linear_ce_grad(x, w, tg, r)
    live = ((tg >= 0) & (tg < v))[:, None]
    p = np.exp(z - lse[:, None]) * live
    hot = (np.arange(v)[None, :] == tg[:, None]) * live
    half = 2.0 ** -8 if t == "bf16" else 2.0 ** -22
    dg = np.abs(r)[:, None] * (p * (dz + dlse[:, None] + 2.0 ** -20) + 4 * U * (p + hot)) + half * np.abs(g)
    ag = np.abs(g) + dg
    ddx = dg @ np.abs(w) + _chain(v, t) * (ag @ np.abs(w))
    ddw = dg.T @ np.abs(x) + _chain(n, t) * (ag.T @ np.abs(x))
    return dlse, dloss, ddx, ddw


def _check(x, w, tg, t, dloss=None):
    from mixture_memories_layer_b200.lm_head import LMHead
    n, d = x.shape
    head = LMHead(w)
    f = head.loss(x, tg)
    g = head.backward(x, tg, dloss)
    assert head.device_errors() == {}
    X, W, G = _np(x), _np(w), tg.cpu().numpy()
    count = max(1, int((G >= 0).sum()))
    r = _np(dloss) if dloss is not None else np.full(n, 1.0 / count)
    loss, lse, _ = T.linear_ce(X, W, G)
    dx, dw, _ = T.linear_ce_grad(X, W, G, r)
    e_lse, e_loss, e_dx, e_dw = _limits(X, W, G, r, t)
    half = torch.finfo(DT[t]).eps / 2

    def close(got, ref, lim, name):
        bad = ~(np.abs(_np(got) - ref) <= lim)
        assert not bad.any(), (name, int(bad.sum()), float(np.nanmax(np.abs(_np(got) - ref) / (lim + 1e-300))))
    close(f["lse"], lse, e_lse, "lse")
    close(f["loss"], loss, np.where(G >= 0, e_loss, 0.0), "loss")
    close(f["mean"], loss.sum() / count, e_loss.max() + U * np.abs(loss).sum() / count, "mean")
    close(g["dx"], dx, e_dx + half * np.abs(dx) + 1e-38, "dx")
    close(g["dw"], dw, e_dw + half * np.abs(dw) + 1e-38, "dw")
    return head, f, g


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("n,d,v", [(1, 1, 1), (1, 64, 2), (2, 7, 5), (3, 64, 256), (17, 100, 257), (64, 128, 1000),
                                   (128, 64, 512), (129, 65, 300), (300, 256, 2100), (257, 72, 511), (5, 1024, 4001),
                                   (40, 2056, 130), (700, 24, 33)])
def test_loss_and_gradients_against_fp64(n, d, v, t):
    _check(*_problem(n, d, v, t), t)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_weights_of_the_rows(t):
    x, w, tg = _problem(90, 96, 700, t, seed=3)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    r = torch.randn(90, generator=gen, device="cuda")
    r[5] = 0
    _check(x, w, tg, t, r)


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_only_padding_and_one_class(t):
    x, w, tg = _problem(33, 64, 300, t, seed=4)
    tg.fill_(-1)
    head, f, g = _check(x, w, tg, t)
    assert float(f["mean"]) == 0 and float(f["inv_count"]) == 0
    assert torch.all(g["dx"] == 0) and torch.all(g["dw"] == 0) and torch.all(f["loss"] == 0)
    x, w, tg = _problem(33, 64, 1, t, seed=5)
    head, f, g = _check(x, w, tg, t)          # the softmax of one class is 1
    assert torch.all(f["loss"].abs() < 1e-5)


def test_large_logits_and_a_sure_prediction():
    """Logits of several hundred: the exponentials must not overflow, and the
    target of the winning class has loss 0."""
    x, w, tg = _problem(64, 64, 600, "bf16", seed=6, std=60.0)
    _check(x, w, tg, "bf16")
    z = _np(x) @ _np(w).T
    tg = torch.as_tensor(z.argmax(axis=1).astype(np.int32)).cuda()
    _check(x, w, tg, "bf16")


def test_infinite_and_nan_logits_stay_in_their_rows():
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(40, 64, 700, "bf16", seed=7, pad=0.0)
    tg[9] = -100
    clean = {k: v.clone() for k, v in LMHead(w).loss(x, tg).items()}
    x2 = x.clone()
    x2[3, 5] = float("nan")
    x2[9, 1] = float("inf")
    head = LMHead(w)
    f = head.loss(x2, tg)
    g = head.backward(x2, tg, torch.ones(40, device="cuda"))
    rows = [i for i in range(40) if i not in (3, 9)]
    assert torch.equal(f["loss"][rows], clean["loss"][rows])
    assert torch.isnan(f["loss"][3]) and f["loss"][9] == 0
    assert torch.all(torch.isfinite(g["dx"][rows].float())) and torch.all(g["dx"][9] == 0)
    assert torch.all(torch.isnan(g["dx"][3]))
    # a class whose logits are -inf for every token takes no part
    w3 = w.clone()
    x3 = x.abs()
    w3[100] = float("-inf")
    keep = torch.arange(700, device="cuda") != 100
    tg3 = torch.where(tg == 100, torch.full_like(tg, 101), tg)
    f3 = LMHead(w3).loss(x3, tg3)
    t4 = torch.where(tg3 > 100, tg3 - 1, tg3)
    f4 = LMHead(w3[keep].contiguous()).loss(x3, t4)
    assert torch.allclose(f3["lse"], f4["lse"], rtol=1e-6, atol=1e-6)


def test_a_target_beyond_the_vocabulary_is_recorded_and_counts_as_padding():
    from mixture_memories_layer_b200 import binding as B
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(50, 64, 300, "bf16", seed=8)
    tg[7] = 300
    ok = tg.clone()
    ok[7] = -100
    head, ref = LMHead(w), LMHead(w)
    f, r = head.loss(x, tg), ref.loss(x, ok)
    assert head.device_errors() == {"fwd": (B.MOM_DEVERR_TARGET, 7)}
    g, h = head.backward(x, tg), ref.backward(x, ok)
    assert all(torch.equal(f[k], r[k]) for k in f) and all(torch.equal(g[k], h[k]) for k in g)


def test_no_tokens():
    from mixture_memories_layer_b200.lm_head import LMHead
    w = torch.randn((300, 64), device="cuda").bfloat16()
    head = LMHead(w)
    x, tg = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    f = head.loss(x, tg)
    g = head.backward(x, tg)
    assert float(f["mean"]) == 0 and f["loss"].numel() == 0 and torch.all(g["dw"] == 0) and g["dx"].shape == (0, 64)


def test_repeats_bit_for_bit_and_leaves_the_neighbours():
    """Two calls give the same bits, and writes stop at the arrays' ends."""
    from mixture_memories_layer_b200 import binding as B
    for t, (n, d, v) in (("bf16", (77, 200, 901)), ("bf16", (77, 203, 901)), ("f32", (50, 61, 333)), ("f32", (50, 64, 333))):
        x, w, tg = _problem(n, d, v, t, seed=9)
        outs = []
        for _ in range(2):
            e = lambda k, dt: torch.full((k + 64,), 3.0, dtype=dt, device="cuda")
            loss, lse, dx, dw = e(n, torch.float32), e(n, torch.float32), e(n * d, DT[t]), e(v * d, DT[t])
            mean = torch.empty(2, device="cuda")
            ws = B.new_workspace(B.mom_linear_ce_workspace_size(n, d, v, DT[t], False))
            B.mom_linear_ce_fwd(x, w, tg, loss[:n], lse[:n], mean, ws)
            ws = B.new_workspace(B.mom_linear_ce_workspace_size(n, d, v, DT[t], True))
            B.mom_linear_ce_bwd(x, w, tg, lse[:n], None, mean[1:2], dx[:n * d].view(n, d), dw[:v * d].view(v, d), ws)
            for a, k in ((loss, n), (lse, n), (dx, n * d), (dw, v * d)):
                assert torch.all(a[k:] == 3)
            outs.append((loss, lse, mean, dx, dw))
        assert all(torch.equal(a, b) for a, b in zip(*outs))


def _torch64(x, w, tg):
    """Sampled rows and classes of a large problem in float64 on the GPU."""
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, dim=1)
    live = tg >= 0
    loss = torch.where(live, lse - z.gather(1, tg.long().clamp(min=0)[:, None])[:, 0], torch.zeros_like(lse))
    g = torch.exp(z - lse[:, None])
    g.scatter_add_(1, tg.long().clamp(min=0)[:, None], -torch.ones_like(lse)[:, None])
    g *= (live / live.sum().clamp(min=1))[:, None]
    return loss, lse, g @ w.double(), g.t() @ x.double()


@pytest.mark.parametrize("n,d,v,t", [(4096, 512, 9001, "bf16"), (33000, 64, 3001, "bf16"), (200, 1024, 40000, "bf16"),
                                     (9000, 264, 2050, "f32"), (64, 520, 20011, "f32")])
def test_several_tiles_pieces_and_slots(n, d, v, t):
    """Sizes with several tiles a CTA, more than one row sweep (n > 32768) and
    split K axes, by 2-norm: bf16 two roundings of at most 2^-8 each in the
    gradient's chain (g and the output), float32 1e-5."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(n, d, v, t, seed=10)
    head = LMHead(w)
    f, g = head.loss(x, tg), head.backward(x, tg)
    ref = _torch64(x, w, tg)
    lim = 2.0 ** -7 if t == "bf16" else 1e-5
    for name, got, want, m in (("loss", f["loss"], ref[0], 1e-5), ("lse", f["lse"], ref[1], 1e-5),
                               ("dx", g["dx"], ref[2], lim), ("dw", g["dw"], ref[3], lim)):
        err = float((got.double() - want).norm() / want.norm())
        assert err < m, (name, err)


def test_pieces_of_the_vocabulary():
    """Several pieces (n large enough that a piece is a part of the
    vocabulary): the same against float64, by 2-norm as above."""
    from mixture_memories_layer_b200 import binding as B
    from mixture_memories_layer_b200.lm_head import LMHead
    n, d, v = 131072, 64, 4500             # 512 MB / (2 n) = 2048 classes a piece
    x, w, tg = _problem(n, d, v, "bf16", seed=11)
    head = LMHead(w)
    f, g = head.loss(x, tg), head.backward(x, tg)
    assert B.mom_linear_ce_workspace_size(n, d, v, torch.bfloat16, True) < 2 * n * v * 2 // 3
    ref = _torch64(x, w, tg)
    for got, want, lim in ((f["loss"], ref[0], 1e-5), (g["dx"], ref[2], 2.0 ** -7), (g["dw"], ref[3], 2.0 ** -7)):
        assert float((got.double() - want).norm() / want.norm()) < lim


def test_another_stream_and_captured_graphs():
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(150, 128, 900, "bf16", seed=12)
    head = LMHead(w)
    want = {**{k: v.clone() for k, v in head.loss(x, tg).items()}, **{k: v.clone() for k, v in head.backward(x, tg).items()}}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other = LMHead(w)
    got = {**other.loss(x, tg, stream=s), **other.backward(x, tg, stream=s)}
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    head.loss(x, tg), head.backward(x, tg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = {**head.loss(x, tg), **head.backward(x, tg)}
    # a larger call replaces the workspaces; the graph keeps its own
    x2, _, tg2 = _problem(600, 128, 900, "bf16", seed=13)
    head.loss(x2, tg2), head.backward(x2, tg2)
    x.mul_(0.5)
    ref = LMHead(w)
    want = {**ref.loss(x, tg), **ref.backward(x, tg)}
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)


@pytest.mark.parametrize("t", ["bf16", "f32"])
@pytest.mark.parametrize("live", [1, 63, 64, 65, 127, 128, 129, 256, 257, 300])
def test_rows_with_a_target_at_the_tiles_edges(t, live):
    """Only rows that have a target take part in the gradient; their number
    falls on and beside the edges of 64 (K of dw) and 256 (rows of a tile)."""
    x, w, tg = _problem(300, 72, 333, t, seed=20, pad=0.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(live)
    tg[torch.randperm(300, generator=g, device="cuda")[live:]] = -100
    _, f, b = _check(x, w, tg, t)
    assert torch.all(b["dx"][tg < 0] == 0)
    r = torch.randn(300, generator=g, device="cuda")
    _check(x, w, tg, t, r)


@pytest.mark.parametrize("t,d", [("bf16", 64), ("bf16", 65), ("f32", 64)])
def test_padding_rows_may_hold_anything(t, d):
    """NaN and infinities in x and dloss of rows without a target: loss, dx and
    dw bit for bit as with zeros there."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(200, d, 500, t, seed=22, pad=0.5)
    pad = (tg < 0).nonzero()[:, 0]
    r = torch.rand(200, device="cuda")
    x0, x1, r0, r1 = x.clone(), x.clone(), r.clone(), r.clone()
    x0[pad], r0[pad] = 0, 0
    x1[pad[::2]], x1[pad[1::2]], r1[pad] = float("nan"), float("inf"), float("nan")
    outs = []
    for xx, rr in ((x0, r0), (x1, r1)):
        head = LMHead(w)
        f = head.loss(xx, tg)
        outs.append((f["loss"].clone(), f["mean"].clone(), *[v.clone() for v in head.backward(xx, tg).values()],
                     *[v.clone() for v in head.backward(xx, tg, rr).values()]))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    assert torch.all(outs[0][2][pad] == 0)


@pytest.mark.parametrize("n,d,v,t,pad", [(20000, 64, 700, "bf16", 0.8), (40000, 40, 300, "f32", 0.5), (16385, 72, 257, "bf16", 0.1),
                                         (12000, 512, 1000, "bf16", 0.0), (4096, 64, 132000, "bf16", 0.3),
                                         (200, 360, 8000, "f32", 0.1), (3000, 300, 6000, "f32", 0.1),
                                         (70000, 33, 9000, "bf16", 0.3), (40000, 41, 5000, "f32", 0.3)])
def test_long_batches_and_slots(n, d, v, t, pad):
    """Rows counted in chunks (n > 16384), token and vocabulary axes split into
    slots, several pieces with slots, several pieces of ragged rows, tiles of
    128 and 256 columns; by 2-norm,
    bf16 two roundings of at most 2^-8 each, float32 1e-5 (a logit's float32
    error in its exponential is the largest)."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(n, d, v, t, seed=23, pad=pad)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2)
    r = torch.rand(n, generator=gen, device="cuda") + 0.5
    head = LMHead(w)
    f, g = head.loss(x, tg), {k: a.clone() for k, a in head.backward(x, tg).items()}
    h = head.backward(x, tg, r)
    loss, lse, dx, dw = _torch64(x, w, tg)
    lim = 2.0 ** -7 if t == "bf16" else 1e-5
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())
    assert rel(f["loss"], loss) < 1e-5 and rel(f["lse"], lse) < 1e-5
    assert rel(g["dx"], dx) < lim and rel(g["dw"], dw) < lim
    assert torch.all(g["dx"][tg < 0] == 0) and torch.all(h["dx"][tg < 0] == 0)
    # rows' weights: dx scales by them; dw from the rows' scaled x
    count = (tg >= 0).sum()
    assert rel(h["dx"], dx * (r * count).double()[:, None]) < lim
    z = torch.exp(x.double() @ w.double().t() - lse[:, None])
    z.scatter_add_(1, tg.long().clamp(min=0)[:, None], -torch.ones_like(lse)[:, None])
    assert rel(h["dw"], z.t() @ (x.double() * (r * (tg >= 0)).double()[:, None])) < lim


def test_gradients_are_differences_of_the_loss():
    """float32, along random directions: (L(x + e a) - L(x - e a)) / 2e of the
    mean loss against <dx, a>, the same for w.  Error: the third derivative
    (e^2 times a constant of the order of the direction's logits cubed, e =
    2^-8 and logits of about 1: 2^-16 x 8) and the loss's own float32 error,
    2^-21 x 8 / 2e = 2^-11."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(60, 48, 200, "f32", seed=24, std=1.0)
    head = LMHead(w)
    head.loss(x, tg)
    grads = {k: v.double().clone() for k, v in head.backward(x, tg).items()}
    gen = torch.Generator(device="cuda")
    gen.manual_seed(4)
    e = 2.0 ** -8
    for name, t in (("dx", x), ("dw", w)):
        for _ in range(4):
            a = torch.randn(t.shape, generator=gen, device="cuda") / 48 ** 0.5
            out = []
            for s in (e, -e):
                xx, ww = (x + s * a, w) if name == "dx" else (x, w + s * a)
                loss = LMHead(ww.contiguous()).loss(xx.contiguous(), tg)["loss"].double()
                out.append(loss.sum() / (tg >= 0).sum())
            got, want = float((out[0] - out[1]) / (2 * e)), float((grads[name] * a).sum())
            assert abs(got - want) < 2.0 ** -11 + 2.0 ** -13, (name, got, want)


@pytest.mark.parametrize("t,d", [("bf16", 72), ("f32", 65)])
def test_a_workspace_at_any_16_bytes(t, d):
    from mixture_memories_layer_b200 import binding as B
    n, v = 130, 700
    x, w, tg = _problem(n, d, v, t, seed=25)
    outs = []
    for off in (0, 16, 48, 240):
        loss, lse, mean = (torch.empty(k, device="cuda") for k in (n, n, 2))
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = [B.new_workspace(B.mom_linear_ce_workspace_size(n, d, v, DT[t], b) + off)[off:] for b in (0, 1)]
        B.mom_linear_ce_fwd(x, w, tg, loss, lse, mean, ws[0])
        B.mom_linear_ce_bwd(x, w, tg, lse, None, mean[1:2], dx, dw, ws[1])
        assert all(B.mom_get_error(a) == (0, 0) for a in ws)
        outs.append((loss, lse, mean, dx, dw))
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o, outs[0]))
