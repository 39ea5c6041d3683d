"""The vocabulary's cross entropy on long batches and in pieces of the vocabulary,
row by row against float64: a lost, doubled or misplaced row of dx or dw is an
error of its own size, which a norm over all rows would not show.

Per row, in 2-norms.  A bf16 g is off by half a step, 2^-8 of its magnitude, a
float32 one by 2^-22; its probability by dz + dlse, twice a logit's error; the
products' sum by its chain (float32: of 128 of K, 48 truncated additions of
2^-23, continued in registers by one rounding each): all relative to the row of
|g| |w| or |g|^T |x|.  The output adds half a step of its own type."""
import pytest
import torch

from tests.test_gpu_linear_ce import DT, U, _chain, _problem

pytestmark = pytest.mark.gpu


def _grad64(x, w, tg, r):
    """(loss, lse, g) in float64 on the GPU, g = r (p - [target])."""
    z = x.double() @ w.double().t()
    lse = torch.logsumexp(z, dim=1)
    live = tg >= 0
    at = tg.long().clamp(min=0)[:, None]
    loss = torch.where(live, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
    z.sub_(lse[:, None]).exp_()
    z.scatter_add_(1, at, -torch.ones_like(lse)[:, None])
    z.mul_((r * live)[:, None])
    return loss, lse, z


def _check_rows(name, got, want, mag, rel, half):
    err, size = (got.double() - want).norm(dim=1), want.norm(dim=1)
    lim = half * size + rel * mag.norm(dim=1)
    bad = ~(err <= lim)
    assert not bad.any(), (name, int(bad.sum()), int(bad.nonzero()[0]), float((err / lim).nan_to_num().max()))
    live = size > 0
    shown = (size > 2 * lim)[live].float().mean()      # rows whose loss would show
    assert shown > 0.99, (name, float(shown))


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("n,d,v,t,pad", [(131072, 64, 4500, "bf16", 0.2), (70000, 33, 9000, "bf16", 0.3),
                                         (33000, 64, 3001, "bf16", 0.2), (16385, 72, 257, "bf16", 0.1),
                                         (40000, 41, 5000, "f32", 0.3), (9000, 264, 2050, "f32", 0.2),
                                         (300, 256, 70001, "bf16", 0.1), (64, 520, 20011, "f32", 0.2)])
def test_every_row_of_the_gradients(n, d, v, t, pad, weighted):
    """Several pieces, row sweeps (32768), counted chunks (16384), slots, ragged
    rows: each row of dx and dw, of the mean loss and of weighted rows."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, w, tg = _problem(n, d, v, t, seed=40, pad=pad)
    tg[torch.arange(0, n, 16384, device="cuda")] = 1          # the chunks' first rows have targets
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)
    dloss = torch.rand(n, generator=gen, device="cuda") + 0.5 if weighted else None
    head = LMHead(w)
    f = head.loss(x, tg)
    b = head.backward(x, tg, dloss)
    r = dloss.double() if weighted else (1.0 / (tg >= 0).sum()).double().expand(n)
    loss, lse, g = _grad64(x, w, tg, r)
    X, W = x.double(), w.double()
    dz = _chain(d, t) * float((X.abs() @ W.abs().t()).max())
    assert float((f["lse"].double() - lse).abs().max()) <= dz + 2.0 ** -20 + 4 * U * float(lse.abs().max())
    assert float((f["loss"].double() - loss).abs().max()) <= 2 * dz + 2.0 ** -20 + 4 * U * float(loss.max())
    half = torch.finfo(DT[t]).eps / 2
    seg = lambda k: _chain(k, t) if t == "bf16" else 2 * U * 64 + U * (k // 128 + 1) + 2.0 ** -22
    dg = (half if t == "bf16" else 2.0 ** -22) + 2 * dz + 2.0 ** -20
    dx, dw = g @ W, g.t() @ X
    g.abs_()
    _check_rows("dx", b["dx"], dx, g @ W.abs(), dg + seg(v), half)
    _check_rows("dw", b["dw"], dw, g.t() @ X.abs(), dg + seg(n), half)
    assert torch.all(b["dx"][tg < 0] == 0) and head.device_errors() == {}
