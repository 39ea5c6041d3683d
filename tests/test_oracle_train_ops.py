"""The fp64 forms of the training-step operators, pinned by finite differences,
pure-Python sums and closed forms (CPU)."""
import math

import numpy as np
import pytest

from oracle import train_ops as T

EPS = 1e-5


def _problem(rng, n, d, gate):
    g = {"none": None, "token": rng.standard_normal((n, 1)), "elem": rng.standard_normal((n, d))}[gate]
    return dict(x=rng.standard_normal((n, d)), y=rng.standard_normal((n, d)), gate=g,
                w_post=1 + 0.3 * rng.standard_normal(d), res_scale=0.5 + 0.2 * rng.standard_normal(d),
                w_pre=1 + 0.3 * rng.standard_normal(d))


def test_residual_norm_is_the_formula_element_by_element():
    rng = np.random.default_rng(0)
    p = _problem(rng, 3, 5, "elem")
    x_out, h = T.residual_norm(**p, eps=EPS)
    for t in range(3):
        ry = math.sqrt(sum(v * v for v in p["y"][t]) / 5 + EPS)
        want = [p["x"][t, c] + p["res_scale"][c] / (1 + math.exp(-p["gate"][t, c])) * p["y"][t, c] / ry * p["w_post"][c]
                for c in range(5)]
        rx = math.sqrt(sum(v * v for v in want) / 5 + EPS)
        assert np.allclose(x_out[t], want, rtol=1e-13)
        assert np.allclose(h[t], [want[c] / rx * p["w_pre"][c] for c in range(5)], rtol=1e-13)


@pytest.mark.parametrize("gate", ["none", "token", "elem"])
def test_residual_norm_gradients_are_central_differences(gate):
    rng = np.random.default_rng(1)
    p = _problem(rng, 4, 6, gate)
    dx_out, dh = rng.standard_normal((4, 6)), rng.standard_normal((4, 6))
    got = T.residual_norm_bwd(**p, eps=EPS, dx_out=dx_out, dh=dh)

    def f(q):
        x_out, h = T.residual_norm(**q, eps=EPS)
        return np.sum(dx_out * x_out) + np.sum(dh * h)
    names = dict(x="dx", y="dy", gate="dgate", w_post="dw_post", res_scale="dres_scale", w_pre="dw_pre")
    for name, out in names.items():
        if p[name] is None:
            continue
        num = np.zeros_like(p[name])
        for i in np.ndindex(num.shape):
            hi, lo = ({**p, name: p[name].copy()} for _ in range(2))
            hi[name][i] += 1e-5
            lo[name][i] -= 1e-5
            num[i] = (f(hi) - f(lo)) / 2e-5
        assert np.max(np.abs(got[out] - num)) < 1e-7 * max(1.0, np.max(np.abs(num))), name


def test_act8_restores_within_half_a_step_and_ties_go_to_even():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 300)).astype(np.float32)
    codes, scales = T.act8_pack(x)
    assert scales.shape == (5, 3) and np.max(np.abs(codes.astype(int))) == 127
    step = np.repeat(scales, 128, axis=1)[:, :300]
    assert np.all(np.abs(T.act8_unpack(codes, scales) - x) <= step * (0.5 + 1e-6))
    # scale 2: 1, 3, 5 lie half way between codes
    codes, scales = T.act8_pack(np.array([[254.0, 1.0, 3.0, 5.0, -1.0, -3.0]]))
    assert scales[0, 0] == 2.0 and codes[0].tolist() == [127, 0, 2, 2, 0, -2]


def test_act8_zeros_and_non_finite_groups():
    x = np.zeros((3, 256))
    x[1, 5] = np.inf
    x[2, 200] = np.nan
    codes, scales = T.act8_pack(x)
    r = T.act8_unpack(codes, scales)
    assert np.all(r[0] == 0) and np.all(np.isnan(r[1, :128])) and np.all(r[1, 128:] == 0)
    assert np.all(r[2, :128] == 0) and np.all(np.isnan(r[2, 128:]))


def test_linear_ce_is_the_sum_and_its_gradient_central_differences():
    rng = np.random.default_rng(3)
    x, w = rng.standard_normal((4, 3)), rng.standard_normal((5, 3))
    tg = np.array([2, -100, 4, 0])
    wt = np.array([0.5, 7.0, -1.0, 2.0])
    loss, lse, z = T.linear_ce(x, w, tg)
    for t in range(4):
        zs = [sum(x[t, c] * w[v, c] for c in range(3)) for v in range(5)]
        want = math.log(sum(math.exp(a) for a in zs))
        assert abs(lse[t] - want) < 1e-13
        assert abs(loss[t] - (0.0 if tg[t] < 0 else want - zs[tg[t]])) < 1e-13
    dx, dw, _ = T.linear_ce_grad(x, w, tg, wt)
    f = lambda a, b: np.sum(wt * T.linear_ce(a, b, tg)[0])
    for arr, got, which in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(arr.shape):
            hi, lo = arr.copy(), arr.copy()
            hi[i] += 1e-5
            lo[i] -= 1e-5
            num = (f(hi, w) - f(lo, w) if which == 0 else f(x, hi) - f(x, lo)) / 2e-5
            assert abs(got[i] - num) < 1e-8
    assert np.all(dx[1] == 0)


def test_linear_ce_a_gradient_without_the_target_term_fails_the_differences():
    rng = np.random.default_rng(4)
    x, w, tg = rng.standard_normal((3, 4)), rng.standard_normal((6, 4)), np.array([1, 5, 2])
    dx, _, g = T.linear_ce_grad(x, w, tg, np.ones(3))
    planted = (g + (np.arange(6)[None, :] == tg[:, None])) @ w
    hi, lo = x.copy(), x.copy()
    hi[0, 0] += 1e-5
    lo[0, 0] -= 1e-5
    num = (T.linear_ce(hi, w, tg)[0].sum() - T.linear_ce(lo, w, tg)[0].sum()) / 2e-5
    assert abs(dx[0, 0] - num) < 1e-8 < abs(planted[0, 0] - num)
