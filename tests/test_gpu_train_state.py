"""What MoMStack and LMHead keep between their calls, on the GPU: side streams,
results that another call must not change, and refusals."""
import pytest
import torch

from tests.test_gpu_stack import BF, _build

pytestmark = pytest.mark.gpu


def _flat(r, prefix=""):
    """Every tensor of a nested result, copied."""
    if torch.is_tensor(r):
        return {prefix: r.clone()}
    items = r.items() if isinstance(r, dict) else enumerate(r)
    return {k: v for i, a in items for k, v in _flat(a, "%s.%s" % (prefix, i)).items()}


def _same(got, want):
    """Bit for bit, but for the blocks' own weight gradients, whose partial sums
    meet in any order: a sum of n terms differs by at most n 2^-24 of their
    magnitudes, and 2^-14 of the largest entry covers the 100 rows here."""
    assert got.keys() == want.keys()
    for k in want:
        if ".block.d" in k and not k.endswith(".dx"):
            lim = 2.0 ** -14 * float(want[k].abs().max())
            assert float((got[k] - want[k]).abs().max()) <= lim, k
        else:
            assert torch.equal(got[k], want[k]), k


def _batch(w, lens, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n = sum(lens)
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device="cuda")
    x = torch.randn((n, w.d_model), generator=g, device="cuda").to(BF)
    return x, cu, torch.randn((n, w.d_model), generator=g, device="cuda"), torch.randn((n, 1), generator=g, device="cuda").to(BF)


def test_a_stack_on_a_side_stream():
    """The same as on the current stream, for the first call and again."""
    w, _, _, _, _, stack, _ = _build(2, 71)
    _, _, _, _, _, other, _ = _build(2, 71)
    x, cu, dh, gate = _batch(w, (40, 1, 24), 3)
    gates = [gate, None]
    want = {**_flat(stack.forward(x, cu, gates)), **_flat(stack.backward(cu, dh, gates=gates), "g")}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):
        out = other.forward(x, cu, gates, stream=s)
        grads = other.backward(cu, dh, gates=gates, stream=s)
        s.synchronize()
        _same({**_flat(out), **_flat(grads, "g")}, want)
        torch.cuda.synchronize()
