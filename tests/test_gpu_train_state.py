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


def _tokens(n, d, v, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((n, d), generator=g, device="cuda").to(BF)
    return x, torch.randint(-20, v, (n,), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("capture", [False, True])
def test_a_gradient_after_an_evaluation_of_the_same_size(capture):
    """A loss kept by the caller gives the same gradients when other losses of
    the same number of rows came between; without it they are the last one's."""
    from mixture_memories_layer_b200.lm_head import LMHead
    x, tg = _tokens(130, 64, 500, 1)
    x2, tg2 = _tokens(130, 64, 500, 2)
    w = _tokens(500, 64, 1, 3)[0]
    ref = LMHead(w)
    want_loss = _flat(ref.loss(x, tg))
    want = _flat(ref.backward(x, tg))
    head = LMHead(w)
    keep = head.new_loss(130)
    torch.cuda.synchronize()

    def step():
        head.loss(x, tg, out=keep)
        head.loss(x2, tg2)
        return head.backward(x, tg, saved=keep)
    got = step()
    if capture:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        for t in (*keep.values(), *got.values()):
            t.zero_()
        graph.replay()
    assert all(torch.equal(want_loss["." + k], keep[k]) for k in ("loss", "lse", "mean", "inv_count"))
    assert all(torch.equal(want["." + k], got[k]) for k in got)
    assert not torch.equal(head.backward(x, tg)["dx"], want[".dx"])
    head.loss(x, tg)
    assert torch.equal(head.backward(x, tg)["dx"], want[".dx"])


def test_weight_gradients_of_two_micro_batches():
    """dw is the head's one buffer, whatever the number of rows; a tensor of the
    caller's is left alone by the next call."""
    from mixture_memories_layer_b200.lm_head import LMHead
    w = _tokens(500, 64, 1, 3)[0]
    a, b = _tokens(100, 64, 500, 4), _tokens(200, 64, 500, 5)
    alone = []
    for x, tg in (a, b):
        h = LMHead(w)
        h.loss(x, tg)
        alone.append(h.backward(x, tg)["dw"].clone())
    head = LMHead(w)
    mine = [torch.full_like(w, 7.0) for _ in range(2)]
    for (x, tg), dw in zip((a, b), mine):
        head.loss(x, tg)
        assert head.backward(x, tg, dw=dw)["dw"] is dw
    assert all(torch.equal(x, y) for x, y in zip(mine, alone))
    g = []
    for x, tg in (a, b):
        head.loss(x, tg)
        g.append(head.backward(x, tg))
    assert g[0]["dw"] is g[1]["dw"] and torch.equal(g[1]["dw"], alone[1])
    assert torch.equal(mine[0], alone[0])
    for bad in (w[:-1], w.float(), torch.empty((64, 500), dtype=BF, device="cuda").t()):
        with pytest.raises(ValueError, match="dw"):
            head.backward(*a, dw=bad)


def test_a_stack_refuses_another_batchs_backward():
    """A forward of another size in between (the blocks' routing tables are its
    own now); the right order gives what the sizes give alone."""
    w, _, _, _, _, stack, _ = _build(2, 81)
    x, cu, dh, gate = _batch(w, (40, 25), 7)
    x2, cu2, dh2, gate2 = _batch(w, (30, 9), 8)
    alone = []
    for a in ((x, cu, dh, gate), (x2, cu2, dh2, gate2)):
        fresh = _build(2, 81)[5]
        fresh.forward(a[0], a[1], [a[3], None])
        alone.append(_flat(fresh.backward(a[1], a[2], gates=[a[3], None])))
    with pytest.raises(ValueError, match="forward"):
        stack.backward(cu, dh, gates=[gate, None])
    stack.forward(x, cu, [gate, None])
    stack.forward(x2, cu2, [gate2, None])
    with pytest.raises(ValueError, match="forward"):
        stack.backward(cu, dh, gates=[gate, None])
    _same(_flat(stack.backward(cu2, dh2, gates=[gate2, None])), alone[1])
    stack.forward(x, cu, [gate, None])
    _same(_flat(stack.backward(cu, dh, gates=[gate, None])), alone[0])


@pytest.mark.parametrize("stream_dtype", [BF, torch.float32])
def test_a_stack_that_keeps_its_stream_in_its_own_type(stream_dtype):
    """The forward's bits are those with 8-bit checkpoints; the gradients at the
    first block are those of the norm's adjoint on the input itself, bit for
    bit, and no longer those on a restored one."""
    from mixture_memories_layer_b200 import binding as B
    from mixture_memories_layer_b200.residual import MoMStack
    w, _, _, _, _, stack, _ = _build(2, 91, stream_dtype)
    plain = MoMStack(_build(2, 91)[5].blocks, stack.norms, stack.w_final, stack.eps, stream_dtype, act8=False)
    x, cu, dh, gate = _batch(w, (50, 3, 33), 9)
    x = x.to(stream_dtype) + (0.001 if stream_dtype == torch.float32 else 0)
    keep = x.clone()
    gates = [gate, None]
    want = _flat(stack.forward(x, cu, gates))
    quant = _flat(stack.backward(cu, dh, gates=gates))
    n, d = x.shape
    one = MoMStack(plain.blocks[:1], plain.norms[:1], plain.w_final, plain.eps, stream_dtype, act8=False)
    one.forward(x, cu, [gate])
    y = one.blocks[0].block_buffers(n, 3)["y"]
    vec = lambda: torch.empty(d, device="cuda")
    dx, dy, dgate, dwp, dsc, dwf = torch.empty_like(dh), torch.empty_like(y), torch.empty_like(gate), vec(), vec(), vec()
    ws = B.new_workspace(B.mom_residual_norm_bwd_workspace_size(n, d))
    nm = one.norms[0]
    B.mom_residual_norm_bwd(keep, y, gate, nm["w_post"], nm["res_scale"], one.w_final, one.eps, None, dh, dx, dy, dgate,
                            dwp, dsc, dwf, ws)
    x.zero_()                                  # the stack has its own copy
    g = one.backward(cu, dh, gates=[gate])
    lev = g["levels"][0]
    assert torch.equal(g["dw_final"], dwf) and torch.equal(lev["dw_post"], dwp)
    assert torch.equal(lev["dres_scale"], dsc) and torch.equal(lev["dgate"], dgate)
    x.copy_(keep)
    got = _flat(plain.forward(x, cu, gates))
    assert all(torch.equal(got[k], want[k]) for k in want) and torch.equal(x, keep)
    x.zero_()
    exact = _flat(plain.backward(cu, dh, gates=gates))
    assert exact.keys() == quant.keys()
    # 8 bits: half a code is 1/254 of a group's largest; the gradients differ, by less than a tenth
    for k in (".dx", ".dw_final", ".levels.0.dw_pre", ".levels.1.dw_post"):
        r = float((exact[k] - quant[k]).norm() / exact[k].norm())
        assert 0 < r < 0.1, (k, r)
    x.copy_(keep)
    _same(_flat(plain.forward(x, cu, gates)), want)
    _same(_flat(plain.backward(cu, dh, gates=gates)), exact)
