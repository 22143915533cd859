"""Host-side argument checks of the operators around the MLP: each refusal has
its documented status code and comes before any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    import block_scaled_mlp_gb300 as mx
    return mx.lib()


P = ctypes.c_void_p(0x10000)
ODD = ctypes.c_void_p(0x10008)


def _fwd(L, x=P, res=P, w=P, M=64, d=96, eps=1e-5, r=P, rstd=P, y=P, axis=3, layout=1, mode=0, q=(P, P, P, P), ck=(P, P)):
    return L.mx_add_rmsnorm_fwd(x, res, w, M, d, eps, r, rstd, y, axis, layout, mode, *q, *ck, None)


def test_norm_forward_refusals(L):
    assert _fwd(L, x=None) == 1 and _fwd(L, w=None) == 1 and _fwd(L, rstd=None) == 1
    assert _fwd(L, r=None) == 1                                    # a residual needs r
    assert _fwd(L, M=-1) == 1 and _fwd(L, d=0) == 1
    assert _fwd(L, axis=4) == 1 and _fwd(L, layout=2) == 1 and _fwd(L, mode=2) == 1
    assert _fwd(L, eps=-1e-5) == 1 and _fwd(L, eps=float("nan")) == 1 and _fwd(L, eps=float("inf")) == 1
    assert _fwd(L, q=(None, P, P, P)) == 1 and _fwd(L, q=(P, P, P, None)) == 1
    assert _fwd(L, ck=(P, None)) == 1
    assert _fwd(L, d=104) == 4 and _fwd(L, d=100, axis=0, ck=(None, None)) == 4
    assert _fwd(L, M=33) == 4                                      # columnwise rows
    assert _fwd(L, d=16416) == 4
    assert _fwd(L, x=ODD) == 2 and _fwd(L, ck=(ODD, P)) == 2 and _fwd(L, y=ODD) == 2
    assert b"aligned" in L.mx_last_error()
    assert _fwd(L, M=0, x=None, r=None, rstd=None) == 0            # no rows: nothing to do


def test_norm_backward_refusals(L):
    def bwd(dy=P, r=P, ck=(None, None), rstd=P, w=P, dres=P, M=64, d=96, dx=P, dw=P, ws=P):
        return L.mx_add_rmsnorm_bwd(dy, r, *ck, rstd, w, dres, M, d, dx, dw, ws, None)

    assert bwd(dy=None) == 1 and bwd(dw=None) == 1 and bwd(ws=None) == 1 and bwd(dx=None) == 1
    assert bwd(r=None) == 1 and bwd(ck=(P, P)) == 1 and bwd(r=None, ck=(P, None)) == 1   # exactly one saved form
    assert bwd(M=-1) == 1 and bwd(d=100) == 4 and bwd(r=None, ck=(P, P), d=104) == 4 and bwd(d=16416) == 4
    assert bwd(dy=ODD) == 2 and bwd(dres=ODD) == 2
    assert L.mx_add_rmsnorm_bwd_workspace(0, 96) == 0 and L.mx_add_rmsnorm_bwd_workspace(1, 96) == 96 * 4


def test_checkpoint_refusals(L):
    for call in (L.mx_ckpt8_save, L.mx_ckpt8_load):
        rest = (P, P) if call is L.mx_ckpt8_save else (P,)
        head = (P,) if call is L.mx_ckpt8_save else (P, P)
        assert call(None, *head[1:], 4, 64, *rest, None) == 1
        assert call(*head, -1, 64, *rest, None) == 1 and call(*head, 4, 0, *rest, None) == 1
        assert call(*head, 4, 48, *rest, None) == 4 and call(*head, 1 << 40, 1 << 30, *rest, None) == 4
        assert call(ODD, *head[1:], 4, 64, *rest, None) == 2
        assert call(*head, 0, 64, *rest, None) == 0
    assert L.mx_swiglu_ckpt8_fwd(None, 4, 64, P, P, P, None) == 1 and L.mx_swiglu_ckpt8_fwd(P, 4, 48, P, P, P, None) == 4
    assert L.mx_swiglu_ckpt8_fwd(P, 4, 64, ODD, P, P, None) == 2
    assert L.mx_swiglu_ckpt8_bwd(P, P, P, 4, 64, None, P, None) == 1 and L.mx_swiglu_ckpt8_bwd(P, P, P, 4, 64, P, ODD, None) == 2
    assert L.mx_swiglu_ckpt8_bwd(P, P, P, -4, 64, P, P, None) == 1


def test_ragged_refusals(L):
    def mm(mode=0, a=P, b=P, M=100, N=64, K=72, offs=P, E=4, c=P):
        return L.mx_ragged_mm(mode, a, b, M, N, K, offs, E, c, None, None)

    for mode in (0, 1, 2):
        assert mm(mode, a=None) == 1 and mm(mode, b=None) == 1 and mm(mode, offs=None) == 1 and mm(mode, c=None) == 1
        assert mm(mode, N=60) == 4 and mm(mode, K=60) == 4 and mm(mode, M=-1) == 1 and mm(mode, N=0) == 1
        assert mm(mode, E=0) == 1 and mm(mode, E=1025) == 1 and mm(mode, M=1 << 31) == 4
        assert mm(mode, a=ODD) == 2 and mm(mode, b=ODD) == 2 and mm(mode, c=ODD) == 2
    assert mm(3) == 1 and mm(-1) == 1
    assert mm(0, M=0, a=None, b=None) == 0
