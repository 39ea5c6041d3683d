"""What MoMStack and LMHead do on the host, without a GPU: the library's calls
are replaced by records of their arguments (CPU)."""
import contextlib

import pytest
import torch

N, D, V = 6, 8, 10


class Stream:
    cuda_stream = 77

    def __init__(self, name):
        self.name = name


class Recorder:
    """Which stream was current as each buffer was made and each call launched."""

    def __init__(self, monkeypatch):
        from mixture_memories_layer_b200 import binding as B
        self.default, self.calls, self.made = Stream("default"), [], []
        self.current = self.default

        @contextlib.contextmanager
        def stream(s):
            before, self.current = self.current, s
            yield
            self.current = before
        monkeypatch.setattr(torch.cuda, "stream", stream)
        monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: self.current)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
        monkeypatch.setattr(B, "current_stream_id", lambda device: self.current.name)
        for name in ("empty", "zeros"):
            make = getattr(torch, name)
            monkeypatch.setattr(torch, name, lambda *a, make=make, **k: (self.made.append(self.current), make(*a, **k))[1])
        for name in ("mom_linear_ce_fwd", "mom_linear_ce_bwd", "mom_residual_norm", "mom_residual_norm_bwd"):
            monkeypatch.setattr(B, name, lambda *a, name=name, stream=None, **k:
                                self.calls.append((name, stream or self.current, a, k)))


class Block:
    """A block that keeps its buffers as MoMBlock does."""

    def __init__(self, rec, d_model=D, dtype=torch.bfloat16):
        self.rec, self.d_model, self.dtype, self.device, self.made = rec, d_model, dtype, torch.device("cpu"), {}

    def block_buffers(self, n, n_seq):
        if n not in self.made:
            self.made[n] = torch.empty((n, self.d_model), dtype=self.dtype)
        return dict(y=self.made[n])

    def forward(self, x, cu, stream=None):
        self.rec.calls.append(("block", stream, (x,), {}))
        return self.block_buffers(x.shape[0], cu.numel() - 1)

    def backward(self, x, cu, dy, stream=None):
        self.rec.calls.append(("block_bwd", stream, (x,), {}))
        return dict(dx=torch.empty(x.shape, dtype=torch.float32))

    def decode_step(self, x, stream=None):
        self.rec.calls.append(("block_dec", stream, (x,), {}))
        return self.block_buffers(x.shape[0], 1)["y"], None


@pytest.fixture
def rec(monkeypatch):
    from mixture_memories_layer_b200 import build
    build.build(verbose=False)
    return Recorder(monkeypatch)


def _stack(rec, levels=2, **kw):
    from mixture_memories_layer_b200.residual import MoMStack
    w = torch.ones(D)
    return MoMStack([Block(rec) for _ in range(levels)], [dict(w_pre=w, w_post=w) for _ in range(levels)], w, **kw)


def _cu(*ends):
    return torch.tensor((0,) + ends, dtype=torch.int32)


@pytest.mark.parametrize("side", [False, True])
def test_buffers_are_made_on_the_stream_that_uses_them(rec, side):
    """The caching allocator hands memory out in the order of the stream that it
    is made on: a buffer made on the current stream and written on another one
    could still be in use by a kernel queued on the first."""
    from mixture_memories_layer_b200.lm_head import LMHead
    head, stack = LMHead(torch.zeros((V, D))), _stack(rec)
    x, tg = torch.zeros((N, D)), torch.zeros(N, dtype=torch.int32)
    xs, dh = torch.zeros((N, D), dtype=torch.bfloat16), torch.zeros((N, D))
    rec.made.clear()
    s = Stream("side") if side else None
    head.loss(x, tg, stream=s)
    head.backward(x, tg, stream=s)
    head.backward(x, tg, torch.ones(N), stream=s)
    stack.forward(xs, _cu(2, N), stream=s)
    stack.backward(_cu(2, N), dh, stream=s)
    stack.decode_step(xs, [(), ()], stream=s)
    want = s or rec.default
    assert len(rec.made) > 20 and all(m is want for m in rec.made)
    assert len(rec.calls) > 15 and all(c[1] is want for c in rec.calls)
    assert rec.current is rec.default


def test_a_workspace_outlives_the_streams_that_use_it(rec, monkeypatch):
    """A workspace that a larger one replaces goes back to the allocator, which
    must know every stream that used it besides the one that it was made on."""
    from mixture_memories_layer_b200 import binding as B
    from mixture_memories_layer_b200.lm_head import LMHead

    class Workspace:
        def __init__(self, nbytes):
            self.nbytes, self.used_on = nbytes, []

        def numel(self):
            return self.nbytes

        def record_stream(self, stream):
            self.used_on.append(stream.name)
    made = []
    monkeypatch.setattr(B, "new_workspace", lambda nbytes, device=None: (made.append(Workspace(nbytes)), made[-1])[1])
    head = LMHead(torch.zeros((V, D)))
    x, tg = torch.zeros((N, D)), torch.zeros(N, dtype=torch.int32)
    a, b = Stream("a"), Stream("b")
    head.loss(x, tg, stream=a)
    head.loss(x, tg, stream=a)
    assert len(made) == 1 and made[0].used_on == []
    head.loss(x, tg, stream=b)
    head.loss(x, tg)
    assert len(made) == 1 and set(made[0].used_on) == {"b", "default"}
    n = 100000
    head.loss(torch.zeros((n, D)), torch.zeros(n, dtype=torch.int32), stream=b)
    head.loss(x, tg, stream=b)
    assert len(made) == 2 and made[1].used_on == []
    head.loss(x, tg, stream=a)
    assert made[1].used_on == ["a"]


def test_the_heads_own_and_the_callers_outputs(rec):
    """What a call reads and writes: the head's own tensors, one set a number of
    rows and one dw, or the caller's."""
    from mixture_memories_layer_b200.lm_head import LMHead
    head = LMHead(torch.zeros((V, D)))
    x, tg = torch.zeros((N, D)), torch.zeros(N, dtype=torch.int32)
    with pytest.raises(ValueError, match="loss"):
        head.backward(x, tg)
    own = head.loss(x, tg)
    assert head.loss(x, tg)["lse"] is own["lse"] and head.loss(x[:2], tg[:2])["lse"] is not own["lse"]
    with pytest.raises(ValueError, match="new_loss"):
        head.loss(x, tg, out=own)
    keep = head.new_loss(N)
    assert head.loss(x, tg, out=keep) is keep
    _, _, a, _ = rec.calls[-1]
    assert a[3] is keep["loss"] and a[4] is keep["lse"] and a[5] is keep["mean_inv"]
    assert keep["mean"].data_ptr() == a[5].data_ptr() and keep["inv_count"].data_ptr() == a[5].data_ptr() + 4
    g = head.backward(x, tg)
    _, _, a, _ = rec.calls[-1]
    assert a[3] is own["lse"] and a[5].data_ptr() == own["inv_count"].data_ptr() and a[7] is g["dw"]
    mine = torch.zeros((V, D))
    g2 = head.backward(x, tg, saved=keep, dw=mine)
    _, _, a, _ = rec.calls[-1]
    assert a[3] is keep["lse"] and a[5].data_ptr() == keep["inv_count"].data_ptr() and tuple(a[5].shape) == (1,)
    assert a[7] is mine and g2["dw"] is mine and g2["dx"] is g["dx"]
    assert head.backward(x[:2], tg[:2])["dw"] is g["dw"]      # one dw, whatever the number of rows
    other = LMHead(torch.zeros((V, D)))
    assert other.backward(x, tg, saved=keep, dw=mine)["dw"] is mine      # no loss call of its own is needed


def test_a_stack_refuses_a_backward_without_its_forward(rec):
    """Its checkpoints and the blocks' buffers would be uninitialised, or those
    of another batch."""
    stack = _stack(rec)
    xs, dh = torch.zeros((N, D), dtype=torch.bfloat16), torch.zeros((N, D))
    tok, el = torch.zeros((N, 1), dtype=torch.bfloat16), torch.zeros((N, D), dtype=torch.bfloat16)

    def refused(*a, **k):
        before = len(rec.calls)
        with pytest.raises(ValueError, match="forward"):
            stack.backward(*a, **k)
        assert len(rec.calls) == before
    refused(_cu(2, N), dh)                                        # none yet
    stack.forward(xs, _cu(2, N), [tok, None])
    refused(_cu(2, 4), dh[:4], gates=[tok[:4], None])             # other rows
    refused(_cu(2, 3, N), dh, gates=[tok, None])                  # other sequences
    for gates in (None, [None, None], [None, tok], [el, None], [tok, tok]):
        refused(_cu(2, N), dh, gates=gates)
    stack.backward(_cu(2, N), dh, gates=[tok[:, 0], None])        # a token's gate may be [N] or [N, 1]
    stack.backward(_cu(2, N), dh, gates=[tok, None])              # again, from the same forward
    stack.decode_step(xs[:3], [(), ()])
    stack.backward(_cu(2, N), dh, gates=[tok, None])              # decoding leaves what it reads
    stack.forward(xs[:4], _cu(1, 4))
    refused(_cu(2, N), dh, gates=[tok, None])                     # the blocks' routing tables are the last forward's
    stack.backward(_cu(1, 4), dh[:4])
    stack.forward(xs, _cu(3, 4, N), [tok, None])
    refused(_cu(2, N), dh, gates=[tok, None])                     # overwritten since
    stack.blocks[1].forward = lambda *a, **k: 1 / 0
    with pytest.raises(ZeroDivisionError):
        stack.forward(xs, _cu(3, 4, N), [tok, None])
    refused(_cu(3, 4, N), dh, gates=[tok, None])                  # not to its end


def test_a_stack_refuses_blocks_of_two_types(rec):
    from mixture_memories_layer_b200.residual import MoMStack
    w = dict(w_pre=torch.ones(D), w_post=torch.ones(D))
    with pytest.raises(ValueError, match="type"):
        MoMStack([Block(rec), Block(rec, dtype=torch.float32)], [w, w], torch.ones(D))
    with pytest.raises(ValueError, match="d_model"):
        MoMStack([Block(rec), Block(rec, d_model=2 * D)], [w, w], torch.ones(D))


@pytest.mark.parametrize("act8", [True, False])
def test_what_a_stack_keeps_for_its_backward(rec, act8):
    """8-bit checkpoints, or the stream itself in buffers of each level's own
    (the caller's input is copied: it may be overwritten after the forward)."""
    stack = _stack(rec, 3, act8=act8)
    x = torch.zeros((N, D), dtype=torch.bfloat16)
    out = stack.forward(x, _cu(N))
    fwd = [c[2:] for c in rec.calls if c[0] == "mom_residual_norm"]
    rec.calls.clear()
    stack.backward(_cu(N), torch.zeros((N, D)))
    bwd = [c[2][0] for c in rec.calls if c[0] == "mom_residual_norm_bwd"]
    restored = [c[2][0] for c in rec.calls if c[0] == "mom_residual_norm"]
    assert fwd[0][0][0] is x and len(fwd) == 4 and len(bwd) == 4 and len(restored) == 3
    if act8:
        codes = [k["pack"][0] for _, k in fwd[1:]]
        assert all(c is b[0] for c, b in zip(codes, reversed(bwd[:3]))) and all(c is r[0] for c, r in zip(codes, reversed(restored)))
        assert bwd[3][0] is bwd[2][0] and len({id(b[0]) for b in bwd}) == 3
        assert all(b[0].dtype == torch.int8 for b in bwd)
    else:
        ins, outs = [a[0] for a, _ in fwd], [a[7] for a, _ in fwd]
        assert all(k.get("pack") is None for _, k in fwd)
        assert all(i is o for i, o in zip(ins[1:], outs)) and len({id(o) for o in outs}) == 4
        assert all(b is o for b, o in zip(reversed(bwd[:3]), outs)) and bwd[3] is outs[0]
        assert all(r is o for r, o in zip(reversed(restored), outs))
        assert out["x"] is outs[3]
