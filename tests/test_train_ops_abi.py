"""The training-step operators refuse bad arguments on the host, before any
launch (CPU)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from mixture_memories_layer_b200 import build
    build.build(verbose=False)
    from mixture_memories_layer_b200 import binding
    return binding


fake, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)


def test_residual_norm_validates(lib):
    B, L = lib, lib.lib

    def call(x=fake, codes=None, scales=None, y=fake, gate=fake, mode=1, w_post=fake, s=fake, w_pre=fake, eps=1e-5, n=4,
             d=64, x_dt=B.MOM_BF16, dt=B.MOM_BF16, x_out=fake, h=fake, oc=None, os=None):
        return L.mom_residual_norm(x, codes, scales, y, gate, mode, w_post, s, w_pre, eps, n, d, x_dt, dt, x_out, h, oc,
                                   os, None)
    A, U = B.MOM_ERR_ARG, B.MOM_ERR_UNSUPPORTED
    assert call(d=0) == A and call(n=-1) == A and call(eps=-1.0) == A and call(eps=float("nan")) == A
    assert call(d=B.MOM_NORM_MAX_D + 1) == U and call(n=1 << 31) == U
    assert call(dt=5) == A and call(x_dt=-1) == A and call(mode=3) == A
    assert call(x_dt=B.MOM_BF16, dt=B.MOM_F32) == U
    assert call(x=None) == A                                     # neither a stream nor a checkpoint
    assert call(codes=fake, scales=fake) == A                    # both
    assert call(x=None, codes=fake) == A
    assert call(gate=None) == A and call(mode=0) == A            # gate and mode disagree
    assert call(y=None, gate=None, mode=0, w_post=None) == A     # a residual scale without a block
    assert call(y=None, gate=None, mode=0, s=None) == A
    assert call(w_post=None) == A and call(w_pre=None) == A
    assert call(x_out=None, h=None) == A
    assert call(oc=fake) == A                                    # codes without scales
    assert call(x=None, codes=fake, scales=fake, oc=fake, os=fake) == A
    for k in ("x", "y", "gate", "w_post", "s", "w_pre", "x_out", "h"):
        assert call(**{k: odd}) == A, k
    assert call(n=0, x=None, y=None, gate=None, mode=0, w_post=None, s=None, w_pre=None, x_out=None, h=None) == B.MOM_OK


def test_residual_norm_bwd_validates(lib):
    B, L = lib, lib.lib
    size = L.mom_residual_norm_bwd_workspace_size(4, 64)
    assert size > B.MOM_WS_HEADER_BYTES

    def call(x=fake, y=fake, gate=fake, mode=2, w_post=fake, s=fake, w_pre=fake, n=4, d=64, dxo=fake, dh=fake,
             g_dt=B.MOM_F32, dx=fake, dy=fake, dgate=fake, dwp=fake, dsc=fake, dwq=fake, ws=fake, nb=size):
        return L.mom_residual_norm_bwd(x, None, None, y, gate, mode, w_post, s, w_pre, 1e-5, n, d, B.MOM_BF16,
                                       B.MOM_BF16, dxo, dh, g_dt, dx, dy, dgate, dwp, dsc, dwq, ws, nb, None)
    A = B.MOM_ERR_ARG
    assert call(nb=size - 1) == A and call(ws=None) == A and call(g_dt=7) == A
    assert call(dx=None) == A and call(dy=None) == A and call(dxo=None, dh=None) == A
    assert call(dh=None) == A                                    # dw_pre wanted without a pre-norm
    assert call(w_pre=None) == A
    assert call(s=None) == A                                     # dres_scale without a scale
    assert call(gate=None, mode=0) == A                          # dgate without a gate
    assert call(y=None, gate=None, mode=0, w_post=None, s=None) == A          # dy without a block
    for k in ("dxo", "dh", "dx", "dy", "dgate", "dwp", "dsc", "dwq"):
        assert call(**{k: odd}) == A, k


def test_act8_validates(lib):
    B, L = lib, lib.lib
    A = B.MOM_ERR_ARG
    for f in (lambda x=fake, dt=B.MOM_F32, n=2, d=8, c=fake, s=fake: L.mom_act_pack8(x, dt, n, d, c, s, None),
              lambda x=fake, dt=B.MOM_F32, n=2, d=8, c=fake, s=fake: L.mom_act_unpack8(c, s, n, d, x, dt, None)):
        assert f(x=None) == A and f(c=None) == A and f(s=None) == A and f(dt=9) == A and f(n=-1) == A and f(d=0) == A
        assert f(x=odd) == A and f(s=odd) == A
        assert f(n=0, x=None, c=None, s=None) == B.MOM_OK


def test_linear_ce_validates(lib):
    B, L = lib, lib.lib
    A, U = B.MOM_ERR_ARG, B.MOM_ERR_UNSUPPORTED
    fsize = L.mom_linear_ce_workspace_size(4, 64, 100, B.MOM_BF16, 0)
    bsize = L.mom_linear_ce_workspace_size(4, 64, 100, B.MOM_BF16, 1)

    def fwd(x=fake, w=fake, t=fake, dt=B.MOM_BF16, n=4, d=64, v=100, loss=fake, lse=fake, mean=None, ws=fake, nb=fsize):
        return L.mom_linear_ce_fwd(x, w, t, dt, n, d, v, loss, lse, mean, ws, nb, None)

    def bwd(x=fake, w=fake, t=fake, lse=fake, dl=None, ds=None, dt=B.MOM_BF16, n=4, d=64, v=100, dx=fake, dw=fake,
            ws=fake, nb=bsize):
        return L.mom_linear_ce_bwd(x, w, t, lse, dl, ds, dt, n, d, v, dx, dw, ws, nb, None)
    for f, nb in ((fwd, fsize), (bwd, bsize)):
        assert f(n=-1) == A and f(d=0) == A and f(v=0) == A and f(dt=4) == A
        assert f(ws=None) == A and f(nb=nb - 1) == A
        assert f(x=None) == A and f(w=None) == A and f(t=None) == A
        assert f(x=odd) == A and f(w=odd) == A and f(t=odd) == A
        big = 1 << 62
        assert f(n=(1 << 30) + 1, nb=big) == U and f(v=(1 << 30) + 1, nb=big) == U and f(d=(1 << 20) + 1, nb=big) == U
    assert fwd(loss=None) == A and fwd(lse=odd) == A and fwd(mean=odd) == A
    assert fwd(n=0, x=None, w=None, t=None, loss=None, lse=None) == B.MOM_OK
    assert bwd(lse=None) == A and bwd(dx=None) == A and bwd(dw=None) == A and bwd(dx=odd) == A and bwd(dw=odd) == A
    assert bwd(dl=odd) == A and bwd(ds=odd) == A


def test_workspaces_hold_the_piece_and_not_the_logits(lib):
    L, B = lib.lib, lib
    n, d, v = 16384, 1024, 262144
    f = L.mom_linear_ce_workspace_size(n, d, v, B.MOM_BF16, 0)
    b = L.mom_linear_ce_workspace_size(n, d, v, B.MOM_BF16, 1)
    assert f < n * v * 2 / 16 and b < n * v * 2 / 8
    assert L.mom_linear_ce_workspace_size(n, d, 2 * v, B.MOM_BF16, 1) <= b + (1 << 20)


def test_the_binding_refuses_other_shapes_types_and_host_tensors(lib):
    B = lib
    x = torch.zeros((4, 64))
    w = torch.ones(64)
    with pytest.raises(ValueError, match="shape"):
        B.mom_residual_norm(x, torch.zeros((4, 32)), None, w, None, w, 1e-5, x, x)
    with pytest.raises(ValueError, match="gate"):
        B.mom_residual_norm(x, x, torch.zeros((4, 2)), w, None, w, 1e-5, x, x)
    with pytest.raises(ValueError, match="float32"):
        B.mom_residual_norm(x, x, None, w.double(), None, w, 1e-5, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.mom_residual_norm(x, x, None, w, None, w, 1e-5, x, x)
    with pytest.raises(ValueError, match="scales"):
        B.mom_act_pack8(x, (torch.zeros((4, 64), dtype=torch.int8), torch.zeros((4, 2))))
    with pytest.raises(ValueError, match="targets"):
        B.mom_linear_ce_fwd(x, torch.zeros((10, 64)), torch.zeros(4, dtype=torch.int64), w[:4], w[:4], None, x)
    with pytest.raises(ValueError, match="w has shape|w is"):
        B.mom_linear_ce_fwd(x, torch.zeros((10, 64)).bfloat16(), torch.zeros(4, dtype=torch.int32), w[:4], w[:4], None, x)
