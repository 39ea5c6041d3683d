"""The training-step operators together, as a program uses them: a stack of
Mixture-of-Memories blocks in a residual stream (norms before and after each
block, gates, residual scales, the stream kept as 8-bit checkpoints) under the
vocabulary's cross entropy, forward and backward against the fp64 forms
(oracle/train_ops.py, oracle/mom_block.py, oracle/mom_block_bwd.py, under the
GPU's routing), and decode continuing a prefill.

Error measure: 2-norm of the difference over the 2-norm.  A block is held to
2e-2 in each direction (its own tests); two blocks forward 4e-2, and their
gradients, which carry both passes, 8e-2.  A wrong index, sign, gate or dropped
term shows as an O(1) error."""
import numpy as np
import pytest
import torch

from mixture_memories_layer_b200 import synth
from oracle import mom_block as blk
from oracle import mom_block_bwd as bbwd
from oracle import train_ops as T
from tests.gpu_helpers import to_np

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-5
V = 700


def _rel(got, ref):
    ref = np.asarray(ref, np.float64)
    return float(np.linalg.norm(np.asarray(got, np.float64) - ref) / np.linalg.norm(ref))


def _build(n_blocks, seed, stream_dtype=BF):
    from mixture_memories_layer_b200 import block as BL
    from mixture_memories_layer_b200.lm_head import LMHead
    from mixture_memories_layer_b200.residual import MoMStack
    w = synth.Workload("small_block", 0, 0, 256, 2, 128, 4, 2, "bf16", seed=seed, block=True)
    rng = np.random.default_rng(seed)
    D = w.d_model
    ps = [synth.make_weights(w, np.random.default_rng(seed + 1 + i)) for i in range(n_blocks)]
    f = lambda a: np.asarray(a, np.float32)
    norms = [dict(w_pre=f(1 + 0.2 * rng.standard_normal(D)), w_post=f(1 + 0.2 * rng.standard_normal(D)))
             for _ in range(n_blocks)]
    norms[0]["res_scale"] = f(0.7 + 0.1 * rng.standard_normal(D))
    w_final = f(1 + 0.2 * rng.standard_normal(D))
    w_head = torch.as_tensor(f(rng.standard_normal((V, D)) * 2 / D ** 0.5)).to(BF)
    cuda = lambda a: torch.as_tensor(a).cuda()
    blocks = [BL.MoMBlock(BL.pack_block_weights(p, BF), w.heads, w.d_head, w.top_k) for p in ps]
    stack = MoMStack(blocks, [{k: cuda(v) for k, v in n.items()} for n in norms], cuda(w_final), EPS, stream_dtype)
    return w, ps, norms, w_final, w_head, stack, LMHead(w_head.cuda())


@pytest.mark.parametrize("stream_dtype", [BF, torch.float32])
def test_a_training_step_of_two_blocks_and_the_head(stream_dtype):
    w, ps, norms, w_final, w_head, stack, head = _build(2, 31, stream_dtype)
    H, d, K, D = w.heads, w.d_head, w.top_k, w.d_model
    lens = (70, 1, 29, 12)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    n = int(cu[-1])
    rng = np.random.default_rng(5)
    x = torch.as_tensor(rng.standard_normal((n, D)).astype(np.float32)).to(stream_dtype)
    gates = [torch.as_tensor(rng.standard_normal((n, 1)).astype(np.float32)).to(BF),
             torch.as_tensor(rng.standard_normal((n, D)).astype(np.float32)).to(BF)]
    tg = rng.integers(0, V, n).astype(np.int32)
    tg[cu[1:] - 1] = -100                                  # no next token at a sequence's end
    cu_d, tg_d, gates_d = torch.as_tensor(cu).cuda(), torch.as_tensor(tg).cuda(), [g.cuda() for g in gates]
    xd = x.cuda()
    for _ in range(2):                                     # the second step over the first one's buffers
        out = stack.forward(xd, cu_d, gates_d)
        loss = head.loss(out["h"], tg_d)
        g = head.backward(out["h"], tg_d)
        grads = stack.backward(cu_d, g["dx"].float(), gates=gates_d)
    torch.cuda.synchronize()
    assert torch.equal(xd.cpu(), x) and head.device_errors() == {}
    assert all(b.device_errors() == {} for b in stack.blocks)

    # fp64, forward
    f64 = lambda t: t.double().cpu().numpy()
    xs, hs, ys, fwds = [f64(x)], [], [], []
    hs.append(T.residual_norm(xs[0], None, None, None, None, norms[0]["w_pre"].astype(np.float64), EPS)[1])
    pre = [n_["w_pre"].astype(np.float64) for n_ in norms] + [w_final.astype(np.float64)]
    post = [n_["w_post"].astype(np.float64) for n_ in norms]
    scl = [n_["res_scale"].astype(np.float64) if "res_scale" in n_ else None for n_ in norms]
    idxs = [b.buffers(n, len(lens))["idx"].cpu().numpy() for b in stack.blocks]
    for i in range(2):
        r = blk.block_forward(hs[i], ps[i], cu, K, H, d, forced_idx=idxs[i])
        ys.append(r["y"])
        xo, h = T.residual_norm(xs[i], r["y"], f64(gates[i]), post[i], scl[i], pre[i + 1], EPS)
        xs.append(xo)
        hs.append(h)
    assert _rel(to_np(out["x"]), xs[2]) < 4e-2 and _rel(to_np(out["h"]), hs[2]) < 4e-2
    l64, _, _ = T.linear_ce(hs[2], f64(w_head), tg)
    count = int((tg >= 0).sum())
    assert abs(float(loss["mean"]) - l64.sum() / count) < 4e-2 * l64.sum() / count
    # fp64, backward
    dh, dw_head, _ = T.linear_ce_grad(hs[2], f64(w_head), tg, np.full(n, 1.0 / count))
    assert _rel(to_np(g["dw"]), dw_head) < 8e-2
    dx = None
    for i in (1, 0):
        r = T.residual_norm_bwd(xs[i], ys[i], f64(gates[i]), post[i], scl[i], pre[i + 1], EPS, dx, dh)
        lev = grads["levels"][i]
        assert _rel(to_np(lev["dgate"]), r["dgate"]) < 8e-2 and _rel(to_np(lev["dw_post"]), r["dw_post"]) < 8e-2
        if scl[i] is not None:
            assert _rel(to_np(lev["dres_scale"]), r["dres_scale"]) < 8e-2
        nxt = grads["dw_final"] if i == 1 else grads["levels"][1]["dw_pre"]
        assert _rel(to_np(nxt), r["dw_pre"]) < 8e-2
        b = bbwd.block_backward(hs[i], ps[i], cu, K, H, d, r["dy"], forced_idx=idxs[i])
        for name, ref in (("dw_o", b["dw_o"]), ("dw_norm", b["dw_norm"]), ("dx", b["dx"])):
            assert _rel(to_np(lev["block"][name]), ref) < 8e-2, (i, name)
        dx, dh = r["dx"], b["dx"]
    r = T.residual_norm_bwd(xs[0], None, None, None, None, pre[0], EPS, dx, dh)
    assert _rel(to_np(grads["levels"][0]["dw_pre"]), r["dw_pre"]) < 8e-2
    assert _rel(to_np(grads["dx"]), r["dx"]) < 8e-2


def test_the_backward_reads_the_checkpoints():
    """The stream that the backward sees is the restored one: the checkpoints
    are those of each block's input, and the input may be overwritten after
    the forward."""
    from mixture_memories_layer_b200 import binding as B
    w, ps, norms, w_final, w_head, stack, head = _build(2, 41)
    cu = torch.tensor([0, 40, 90], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x = torch.randn((90, w.d_model), generator=g, device="cuda").to(BF)
    dh = torch.randn((90, w.d_model), generator=g, device="cuda")
    keep = x.clone()
    stack.forward(x, cu)
    first = {k: v.clone() for k, v in stack.backward(cu, dh).items() if torch.is_tensor(v)}
    k8 = B.new_act8(90, w.d_model)
    B.mom_act_pack8(keep, k8)
    assert torch.equal(stack._k8(0, 90)[0], k8[0]) and torch.equal(stack._k8(0, 90)[1], k8[1])
    stack.forward(x, cu)
    x.zero_()
    again = stack.backward(cu, dh)
    assert all(torch.equal(first[k], again[k]) for k in first)


def test_decode_continues_a_prefill():
    w, ps, norms, w_final, w_head, stack, head = _build(2, 51)
    lens = (20, 7, 33)
    rng = np.random.default_rng(6)
    seqs = [torch.as_tensor(rng.standard_normal((l + 1, w.d_model)).astype(np.float32)).to(BF).cuda() for l in lens]
    cum = lambda ls: torch.tensor(np.concatenate([[0], np.cumsum(ls)]), dtype=torch.int32, device="cuda")
    full = stack.forward(torch.cat(seqs), cum([l + 1 for l in lens]))
    ends = np.cumsum([l + 1 for l in lens]) - 1
    want_h, want_x = to_np(full["h"])[ends], to_np(full["x"])[ends]
    cu = cum(lens)
    stack.forward(torch.cat([s[:-1] for s in seqs]), cu)
    states = []
    for b in stack.blocks:
        f = b.block_buffers(sum(lens), len(lens))
        st = torch.empty((len(lens), w.n_mem + 1, w.heads, w.d_head, w.d_head), device="cuda")
        st[:, :w.n_mem] = f["h_mem"].permute(1, 0, 2, 3, 4)
        st[:, w.n_mem] = f["h_shared"]
        states.append((st,) + b.conv_state(f, cu))
    out = stack.decode_step(torch.stack([s[-1] for s in seqs]), states)
    assert _rel(to_np(out["x"]), want_x) < 4e-2 and _rel(to_np(out["h"]), want_h) < 4e-2


def test_a_stack_refuses_what_it_cannot_hold():
    from mixture_memories_layer_b200.residual import MoMStack
    w, ps, norms, w_final, w_head, stack, head = _build(1, 61)
    b, n = stack.blocks[0], stack.norms[0]
    with pytest.raises(ValueError):
        MoMStack([b, b], [n, n], stack.w_final)
    with pytest.raises(ValueError):
        MoMStack([b], [n, n], stack.w_final)
    with pytest.raises(ValueError):
        MoMStack([], [], stack.w_final)
    with pytest.raises(ValueError, match="gates"):
        stack.forward(torch.zeros((4, w.d_model), dtype=BF, device="cuda"),
                      torch.tensor([0, 4], dtype=torch.int32, device="cuda"), gates=[None, None])
