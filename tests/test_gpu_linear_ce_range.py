"""The vocabulary's cross entropy at the ends of the number range: classes masked
by finite values, logits far from 0, the largest float32 values and infinities,
and the parts of a float32 operand.  Against fp64 (oracle/train_ops.py);
tolerances as in test_gpu_linear_ce.py unless a test derives its own."""
import numpy as np
import pytest
import torch

from oracle import train_ops as T
from tests.test_gpu_linear_ce import DT, U, _chain, _limits, _np, _problem

pytestmark = pytest.mark.gpu

LOWEST = {"bf16": torch.finfo(torch.bfloat16).min, "f32": torch.finfo(torch.float32).min}


def _masked(t, value, at, count, n=70, v=700):
    """A problem whose classes at .. at + count - 1 have a logit of about
    `value` for every token: x's first channel is 1 and carries a bias.  Also
    the kept classes' indices."""
    d = 72 if t == "bf16" else 65
    x, w, tg = _problem(n, d, v, t, seed=30)
    x[:, 0] = 1
    w[at:at + count, 0] = value
    keep = torch.ones(v, dtype=torch.bool, device="cuda")
    keep[at:at + count] = False
    first = int(keep.nonzero()[0, 0])
    tg = torch.where((tg >= at) & (tg < at + count), torch.full_like(tg, first), tg)
    return x, w, tg, keep


def _check_masked(x, w, tg, keep, t, gradient=True):
    """Loss and gradients are those of the kept classes alone; a masked class'
    probability is 0, so its row of dw is 0 and it adds nothing to dx."""
    from mixture_memories_layer_b200.lm_head import LMHead
    n = x.shape[0]
    X, G = _np(x), tg.cpu().numpy()
    Wk = _np(w[keep])
    index = (torch.cumsum(keep.int(), 0) - 1).cpu().numpy()
    Gk = np.where(G >= 0, index[np.where(G >= 0, G, 0)], G)
    r = np.full(n, 1.0 / (G >= 0).sum())
    head = LMHead(w)
    f = head.loss(x, tg)
    loss, lse, _ = T.linear_ce(X, Wk, Gk)
    e_lse, e_loss, e_dx, e_dw = _limits(X, Wk, Gk, r, t)
    assert np.all(np.abs(_np(f["lse"]) - lse) <= e_lse), np.abs(_np(f["lse"]) - lse).max()
    assert np.all(np.abs(_np(f["loss"]) - loss) <= np.where(G >= 0, e_loss, 0.0))
    assert np.isfinite(float(f["mean"])) and abs(float(f["mean"]) - loss.sum() * r[0]) <= e_loss.max() + 8 * U
    if not gradient:
        return
    g = head.backward(x, tg)
    dx, dw, _ = T.linear_ce_grad(X, Wk, Gk, r)
    half = torch.finfo(DT[t]).eps / 2
    assert np.all(np.abs(_np(g["dx"]) - dx) <= e_dx + half * np.abs(dx))
    assert np.all(np.abs(_np(g["dw"][keep]) - dw) <= e_dw + half * np.abs(dw))
    assert torch.all(g["dw"][~keep] == 0)
    assert head.device_errors() == {}


@pytest.mark.parametrize("at,count", [(0, 40), (128, 128), (300, 32), (320, 64), (660, 40), (0, 650), (50, 650)])
@pytest.mark.parametrize("t,value", [("bf16", v) for v in (-1e9, -1e10, -1e30, LOWEST["bf16"])] +
                         [("f32", v) for v in (-1e9, -1e10, -1e30, LOWEST["f32"] / 2)])
def test_classes_masked_by_finite_values(t, value, at, count):
    """32 and more neighbouring masked classes: whole chunks, half tiles and
    tiles that hold nothing else, at the vocabulary's start, inside and end."""
    _check_masked(*_masked(t, value, at, count), t)


@pytest.mark.parametrize("t,value", [(t, v) for t in ("bf16", "f32") for v in (1.0, 2.0 ** 24, 1e10, 1e30, -1e10, -1e30)] +
                         [("bf16", LOWEST["bf16"]), ("bf16", -LOWEST["bf16"])])
def test_equal_logits_of_any_size(t, value):
    _check_equal(t, value)


def _check_equal(t, value):
    """All classes share one logit, whatever its size: lse is that logit plus
    log v, rounded (twice, and log v's own 2^-21)."""
    from mixture_memories_layer_b200.lm_head import LMHead
    n, d, v = 40, 64, 700
    x, w, tg = _problem(n, d, v, t, seed=31)
    x[:, 0] = 1
    w.zero_()
    w[:, 0] = value
    value = float(w[0, 0])
    f = LMHead(w).loss(x, tg)
    want = value + np.log(float(v))
    assert np.all(np.abs(_np(f["lse"]) - want) <= 2 * U * abs(want) + 2.0 ** -21 * np.log(v))


def _integers(t, n=60, d=64, v=700, offset=2 ** 20, seed=32):
    """x and w of -1, 0 and 1 with a bias of `offset` through x's first channel:
    every logit and every partial sum of one is an integer below 2^21, exact in
    float32 under any rounding."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randint(-1, 2, (n, d), generator=g, device="cuda").to(DT[t])
    w = torch.randint(-1, 2, (v, d), generator=g, device="cuda").to(DT[t])
    x[:, 0] = 1
    w[:, 0] = offset
    tg = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
    tg[::7] = -1
    return x, w, tg


@pytest.mark.parametrize("value", [0.0, 2.0 ** 20, -2.0 ** 20])
@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_the_loss_keeps_its_digits_far_from_zero(t, value):
    """loss = (max - z_target) + log(sum): the first term is exact for integer
    logits, so what is left is the exponentials' and the sum's error, 2^-19,
    and the rounding of the terms -- not 2^-24 of the logits, 2^-4 here."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _integers(t, offset=value)
    f = LMHead(w).loss(x, tg)
    G = tg.cpu().numpy()
    loss, lse, _ = T.linear_ce(_np(x), _np(w), G)
    lim = 2.0 ** -19 + 8 * U * (np.abs(loss) + np.log(w.shape[0]))
    assert np.all(np.abs(_np(f["loss"]) - loss) <= lim), np.abs(_np(f["loss"]) - loss).max()
    assert abs(float(f["mean"]) - loss.sum() / (G >= 0).sum()) <= lim.max()


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_a_sure_prediction_of_a_large_logit(t):
    """The winning class leads by 8 at a logit of 2^20: the loss is log(1 + ..
    exp(-8) ..), of the order of 0.2, and the equal logits' loss log v."""
    from mixture_memories_layer_b200.lm_head import LMHead
    n, d, v = 33, 64, 700
    x = torch.zeros((n, d), device="cuda").to(DT[t])
    w = torch.zeros((v, d), device="cuda").to(DT[t])
    x[:, 0], x[:, 1] = 1, 1
    w[:, 0] = 2.0 ** 20
    w[333, 1] = 8
    tg = torch.full((n,), 333, dtype=torch.int32, device="cuda")
    f = LMHead(w).loss(x, tg)
    want = np.log1p((v - 1) * np.exp(-8.0))
    assert np.all(np.abs(_np(f["loss"]) - want) <= 2.0 ** -19 + 8 * U * np.log(v))
    w[333, 1] = 0
    f = LMHead(w).loss(x, tg)
    assert np.all(np.abs(_np(f["loss"]) - np.log(v)) <= 2.0 ** -19 + 8 * U * np.log(v))


@pytest.mark.parametrize("t", ["bf16", "f32"])
def test_the_gradients_exponent_is_a_difference(t):
    """g = exp(z - lse) - [target] of the lse that is given: with integer logits
    and an integer lse of 2^20 the exponent is exact, so p has only its own
    error, 2^-22 of the exponential and 2^-24 of the exponent's |z - lse| log2 e,
    and g its rounding (bf16, or three parts)."""
    from mixture_memories_layer_b200 import binding as B
    x, w, tg = _integers(t, seed=33)
    n, d = x.shape
    v = w.shape[0]
    X, W, G = _np(x), _np(w), tg.cpu().numpy()
    z = X @ W.T
    lse = z.max(axis=1) + 3
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = B.new_workspace(B.mom_linear_ce_workspace_size(n, d, v, DT[t], True))
    r = torch.rand(n, device="cuda") + 0.5
    B.mom_linear_ce_bwd(x, w, tg, torch.as_tensor(lse, dtype=torch.float32, device="cuda"), r, None, dx, dw, ws)
    live = G >= 0
    e = z - lse[:, None]
    p = np.exp(e) * live[:, None]
    hot = (np.arange(v)[None, :] == G[:, None]) * live[:, None]
    R = _np(r)[:, None]
    g = R * (p - hot)
    half = torch.finfo(DT[t]).eps / 2
    dg = np.abs(R) * (p * (2.0 ** -21 + 3 * U * np.abs(e)) + 4 * U * (p + hot)) + (half if t == "bf16" else 2.0 ** -22) * np.abs(g)
    for got, want, lim in ((dx, g @ W, dg @ np.abs(W) + _chain(v, t) * (np.abs(g) @ np.abs(W))),
                           (dw, g.T @ X, dg.T @ np.abs(X) + _chain(n, t) * (np.abs(g).T @ np.abs(X)))):
        assert np.all(np.abs(_np(got) - want) <= lim + half * np.abs(want)), np.abs(_np(got) - want).max()


@pytest.mark.parametrize("n,d,v,t", [(70, 72, 700, "bf16"), (300, 65, 9001, "f32"), (2000, 64, 9000, "bf16"), (20, 130, 40001, "bf16")])
def test_the_gradient_forms_the_losss_logits_again(n, d, v, t):
    """Logits of 1e10: a class' exponent is 0 (the largest) or below -1000, if the
    gradient's logit is the one that the loss saw, bit for bit, whatever tiles
    the two took.  Then g = [largest] - [target], and dx, dw are exact sums of
    rows (rounded; bf16 weights are 1)."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(n, d, v, t, seed=34)
    w = (w.float() * 1e10).to(DT[t])
    head = LMHead(w)
    f = head.loss(x, tg)
    g = head.backward(x, tg, torch.ones(n, device="cuda"))
    X, W, G = _np(x), _np(w), tg.cpu().numpy()
    z = X @ W.T
    order = np.sort(z, axis=1)
    sure = order[:, -1] - order[:, -2] > 2e6          # rows whose largest logit leads by many ulps (2^10)
    assert sure.mean() > 0.9
    top = z.argmax(axis=1)
    want = np.where((G >= 0)[:, None], W[top] - W[np.where(G >= 0, G, 0)], 0.0)
    mag = np.abs(W[top]) + np.abs(W[np.where(G >= 0, G, 0)])
    lim = torch.finfo(DT[t]).eps / 2 * np.abs(want) + 2.0 ** -21 * mag
    ok = np.abs(_np(g["dx"]) - want) <= lim
    assert np.all(ok[sure]) and torch.all(torch.isfinite(g["dx"].float())) and torch.all(torch.isfinite(g["dw"].float()))
    assert torch.all(torch.isfinite(f["loss"]))


@pytest.mark.parametrize("at,count", [(0, 40), (128, 128), (300, 32), (320, 64), (660, 40), (0, 650), (50, 650)])
def test_float32_classes_masked_by_the_lowest_value(at, count):
    _check_masked(*_masked("f32", LOWEST["f32"], at, count), "f32")


@pytest.mark.parametrize("value", [LOWEST["f32"], -LOWEST["f32"], 3.391e38])
def test_float32_logits_of_the_largest_size(value):
    _check_equal("f32", value)


@pytest.mark.parametrize("at,count", [(0, 40), (128, 128), (660, 40), (0, 699), (333, 1)])
def test_float32_classes_masked_by_minus_infinity(at, count):
    """A -inf in w counts as the lowest float32 value: in the loss a masked
    class as in bf16, and in the gradient 0 times a finite number."""
    x, w, tg, keep = _masked("f32", float("-inf"), at, count)
    _check_masked(x, w, tg, keep, "f32")
    # whole rows of -inf, against tokens without a negative channel
    x = x.abs()
    w[at:at + count] = float("-inf")
    _check_masked(x, w, tg, keep, "f32")


def test_float32_values_up_to_the_largest():
    """Values that round to infinity in bf16 are split like any other: in a
    channel of x that no class uses and in one of w that no token uses they
    leave logits and the other channels' gradients bit for bit, and their own
    gradients are 2^100 times those of values 2^100 times smaller (both within
    a chain of the magnitudes; weights of 1/4 and a class for each token keep
    the sums finite)."""
    from mixture_memories_layer_b200.lm_head import LMHead
    n, d, v = 50, 65, 300
    x, w, tg = _problem(n, d, v, "f32", seed=35, pad=0.0)
    tg = torch.arange(n, dtype=torch.int32, device="cuda") * 5
    big = torch.tensor([3.4028234663852886e38, 3.3961775292304957e38, 3.3895313892515355e38, 3.391e38], device="cuda")
    x[:, 3], w[:, 3], x[:, 7], w[:, 7] = 0, 0, 0, 0
    x3 = big.repeat(13)[:n] * torch.where(torch.arange(n, device="cuda") % 3 == 0, -1.0, 1.0)
    w7 = -big.repeat(75)[:v]
    r = torch.full((n,), 0.25, device="cuda")
    outs = []
    for scale in (1.0, 2.0 ** -100):
        x[:, 3], w[:, 7] = x3 * scale, w7 * scale
        head = LMHead(w)
        f = head.loss(x, tg)
        outs.append({**{k: a.clone() for k, a in f.items()}, **{k: _np(a) for k, a in head.backward(x, tg, r).items()}})
    a, b = outs
    assert all(torch.equal(a[k], b[k]) for k in ("loss", "lse", "mean"))
    other = [c for c in range(d) if c not in (3, 7)]
    assert np.array_equal(a["dx"][:, other], b["dx"][:, other]) and np.array_equal(a["dw"][:, other], b["dw"][:, other])
    X, W = _np(x), _np(w)
    X[:, 3], W[:, 7] = 0, 0
    g = np.abs(T.linear_ce_grad(X, W, tg.cpu().numpy(), np.full(n, 0.25))[2])
    for got, want, k, mag in ((a["dw"][:, 3], b["dw"][:, 3], n, g.T @ np.abs(_np(x3))),
                              (a["dx"][:, 7], b["dx"][:, 7], v, g @ np.abs(_np(w7)))):
        assert np.all(np.abs(got - want * 2.0 ** 100) <= 2 * _chain(k, "f32") * 1.01 * mag)


def test_float32_infinities_and_nan_stay_in_their_rows():
    """An infinity or a NaN in x makes its row NaN and no other; a +inf in w, or
    a NaN, every row."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(40, 65, 700, "f32", seed=36, pad=0.0)
    tg[9] = -100
    clean = LMHead(w).loss(x, tg)["loss"].clone()
    x2 = x.clone()
    x2[3, 5], x2[4, 6], x2[5, 7], x2[9, 1] = float("nan"), float("inf"), float("-inf"), float("inf")
    head = LMHead(w)
    f = head.loss(x2, tg)
    rows = [i for i in range(40) if i not in (3, 4, 5, 9)]
    assert torch.equal(f["loss"][rows], clean[rows]) and f["loss"][9] == 0
    assert torch.all(torch.isnan(f["loss"][3:6])) and torch.all(torch.isnan(f["lse"][3:6]))
    g = head.backward(x2, tg, torch.ones(40, device="cuda"))
    assert torch.all(torch.isfinite(g["dx"][rows])) and torch.all(torch.isnan(g["dx"][3:6])) and torch.all(g["dx"][9] == 0)
    for bad in (float("inf"), float("nan")):
        w2 = w.clone()
        w2[17, 3] = bad
        assert torch.all(torch.isnan(LMHead(w2).loss(x, tg)["lse"]))


def test_float32_parts_hold_every_bit():
    """One channel and one class: lse is the product x w, of a full mantissa
    and a power of two, bit for bit.  Two classes with logits of 0: g = -+1/2,
    and dw and dx repeat all 24 bits of x and w within 1.5 x 2^-20 (p: 2^-22 of
    the exponential and 2 x 2^-24 of its exponent; six truncated products, 2 x
    2^-24 each).  Without the third part they would be off by up to 2^-17."""
    from mixture_memories_layer_b200.lm_head import LMHead
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    bits = torch.randint(1 << 23, 1 << 24, (64,), generator=g, device="cuda", dtype=torch.int32) | 1
    full = bits.float() * 2.0 ** -23 * torch.where(torch.arange(64, device="cuda") % 2 == 0, 1.0, -1.0)
    zero = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    for k in (0, 5, -30):
        x, w = torch.zeros((64, 65), device="cuda"), torch.zeros((1, 65), device="cuda")
        x[:, 40], w[0, 40] = full, 2.0 ** k
        assert torch.equal(LMHead(w).loss(x, zero(64))["lse"], full * 2.0 ** k)
        x = torch.zeros((1, 65), device="cuda")
        for j in range(0, 64, 9):
            x[0, 40], w[0, 40] = 2.0 ** k, full[j]
            assert torch.equal(LMHead(w).loss(x, zero(1))["lse"], (full * 2.0 ** k)[j:j + 1])
    lim = 1.5 * 2.0 ** -20 * full.abs()
    head = LMHead(torch.zeros((2, 64), device="cuda"))
    x = full[None].clone()
    head.loss(x, zero(1))
    dw = head.backward(x, zero(1))["dw"]
    assert torch.all((dw[0] + full / 2).abs() <= lim) and torch.all((dw[1] - full / 2).abs() <= lim)
    head = LMHead(torch.stack([full, torch.zeros_like(full)]))
    x = torch.zeros((1, 64), device="cuda")
    head.loss(x, zero(1))
    dx = head.backward(x, zero(1))["dx"]
    assert torch.all((dx[0] + full / 2).abs() <= lim)


def test_a_target_beyond_the_vocabulary_is_recorded_in_the_gradient():
    """The gradient's own workspace keeps the violation too, and the row counts
    as padding."""
    from mixture_memories_layer_b200 import binding as B
    for t, n, row in (("bf16", 50, 7), ("f32", 20, 19), ("bf16", 20000, 17001)):
        x, w, tg = _problem(n, 64, 300, t, seed=37)
        tg[row] = 300 + row
        lse = torch.full((n,), 5.0, device="cuda")
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws = B.new_workspace(B.mom_linear_ce_workspace_size(n, 64, 300, DT[t], True))
        B.mom_linear_ce_bwd(x, w, tg, lse, None, None, dx, dw, ws)
        assert B.mom_get_error(ws) == (B.MOM_DEVERR_TARGET, row)
        assert torch.all(dx[row] == 0)
        tg[row] = -100
        dx2, dw2 = torch.empty_like(x), torch.empty_like(w)
        ws = B.new_workspace(B.mom_linear_ce_workspace_size(n, 64, 300, DT[t], True))
        B.mom_linear_ce_bwd(x, w, tg, lse, None, None, dx2, dw2, ws)
        assert B.mom_get_error(ws) == (0, 0) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
