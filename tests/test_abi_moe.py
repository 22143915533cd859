"""Host-side argument checks of routing, grouping, combining and FP8 with 128-blocks: each refusal has its documented
status code and comes before any CUDA call."""
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
BYTE = ctypes.c_void_p(0x10001)


def test_route_refusals(L):
    def route(l=P, kind=0, T=5, E=64, k=8, score=0, bias=P, groups=8, top=4, renorm=1, scale=1.0, ids=P, w=P):
        return L.mx_moe_route(l, kind, T, E, k, score, bias, groups, top, renorm, scale, ids, w, None)

    assert route(l=None) == 1 and route(ids=None) == 1 and route(w=None) == 1
    assert route(kind=2) == 1 and route(score=2) == 1 and route(score=-1) == 1 and route(T=-1) == 1
    assert route(E=0) == 1 and route(E=1025) == 1 and route(k=0) == 1 and route(k=33) == 1 and route(E=4, k=5, groups=1, top=1) == 1
    assert route(groups=0) == 1 and route(groups=5) == 1 and route(E=330, groups=33) == 1
    assert route(top=0) == 1 and route(top=9) == 1 and route(k=9, top=1) == 1
    assert route(scale=float("nan")) == 1 and route(scale=float("inf")) == 1
    assert route(T=1 << 31) == 4
    assert route(l=BYTE) == 2 and route(l=ctypes.c_void_p(0x10002), kind=1) == 2 and route(ids=BYTE) == 2 and route(bias=BYTE) == 2
    assert route(T=0, l=None, ids=None, w=None) == 0


def test_route_backward_refusals(L):
    def bwd(dw=P, l=P, kind=0, ids=P, T=5, E=64, k=8, score=1, renorm=1, scale=1.0, dl=P):
        return L.mx_moe_route_bwd(dw, l, kind, ids, T, E, k, score, renorm, scale, dl, None, None)

    assert bwd(dw=None) == 1 and bwd(l=None) == 1 and bwd(ids=None) == 1 and bwd(dl=None) == 1
    assert bwd(kind=3) == 1 and bwd(score=7) == 1 and bwd(E=1025) == 1 and bwd(k=65) == 1 and bwd(scale=float("inf")) == 1
    assert bwd(dl=BYTE) == 2 and bwd(dw=BYTE) == 2 and bwd(T=-1) == 1 and bwd(T=1 << 31) == 4
    assert bwd(T=0, dw=None, l=None) == 0


def test_token_group_refusals(L):
    def group(ids=P, R=9000, E=4, offs=P, dst=P, src=P, ws=P):
        return L.mx_token_group(ids, R, E, offs, dst, src, ws, None, None)

    assert group(ids=None) == 1 and group(offs=None) == 1 and group(dst=None) == 1 and group(src=None) == 1 and group(ws=None) == 1
    assert group(R=-1) == 1 and group(E=0) == 1 and group(E=1025) == 1 and group(R=1 << 31) == 4 and group(dst=BYTE) == 2 and group(ws=ODD) == 2
    assert L.mx_token_group_workspace(0, 4) == 0 and L.mx_token_group_workspace(8192, 352) == 0      # one CTA
    assert L.mx_token_group_workspace(8193, 4) == 9 * 4 * 4 and L.mx_token_group_workspace(1025, 353) == 2 * 353 * 4
    assert L.mx_token_group_workspace(10, 0) == 0 and L.mx_token_group_workspace(1 << 32, 4) == 0


def test_combine_refusals(L):
    def fwd(rows=P, n=40, d=64, dst=P, T=10, k=4, w=P, add=P, out=P):
        return L.mx_moe_combine(rows, n, d, dst, T, k, w, add, out, None, None)

    def bwd(dout=P, rows=P, n=40, d=64, dst=P, src=P, T=10, k=4, w=P, drows=P, dw=P):
        return L.mx_moe_combine_bwd(dout, rows, n, d, dst, src, T, k, w, drows, dw, None, None)

    for call in (fwd, bwd):
        assert call(rows=None) == 1 and call(dst=None) == 1 and call(n=-1) == 1 and call(T=-1) == 1 and call(d=0) == 1
        assert call(k=0) == 1 and call(k=33) == 1 and call(d=60) == 4 and call(T=1 << 31) == 4 and call(n=1 << 31) == 4
        assert call(rows=ODD) == 2 and call(dst=BYTE) == 2 and call(w=BYTE) == 2
    assert fwd(out=None) == 1 and fwd(out=ODD) == 2 and fwd(add=ODD) == 2 and fwd(T=0, rows=None, out=None) == 0
    assert bwd(dout=None) == 1 and bwd(src=None) == 1 and bwd(w=None) == 1 and bwd(drows=None) == 1 and bwd(dw=None) == 1
    assert bwd(dout=ODD) == 2 and bwd(drows=ODD) == 2 and bwd(T=0, n=0) == 0


def test_fp8_block_cast_refusals(L):
    def rows(x=P, n_in=40, cols=64, src=None, n=40, div=1, q=P, s=P):
        return L.mx_fp8_block_quantize(x, n_in, cols, src, n, div, q, s, None, None)

    assert rows(x=None) == 1 and rows(q=None) == 1 and rows(s=None) == 1 and rows(n_in=-1, n=-1) == 1 and rows(cols=0) == 1
    assert rows(n=41) == 1 and rows(div=2) == 1 and rows(src=P, div=0) == 1
    assert rows(cols=72) == 4 and rows(n_in=1 << 31, n=1 << 31) == 4
    assert rows(x=ODD) == 2 and rows(q=ODD) == 2 and rows(src=BYTE) == 2
    assert rows(n_in=0, n=0, x=None, q=None) == 0

    def weight(w=P, E=3, N=64, K=48, q=P, qt=P, s=P):
        return L.mx_fp8_block_quantize_weight(w, E, N, K, q, qt, s, None)

    assert weight(w=None) == 1 and weight(q=None) == 1 and weight(s=None) == 1 and weight(N=0) == 1 and weight(E=-1) == 1
    assert weight(N=72) == 4 and weight(K=72) == 4 and weight(E=65536) == 4
    assert weight(w=ODD) == 2 and weight(qt=ODD) == 2 and weight(E=0, w=None) == 0


def test_fp8_block_mm_refusals(L):
    def mm(mode=0, a=P, sa=P, w=P, sw=P, M=100, N=64, K=48, offs=P, E=4, c=P):
        return L.mx_fp8_block_mm(mode, a, sa, w, sw, M, N, K, offs, E, c, None, None)

    for mode in (0, 1):
        assert mm(mode, a=None) == 1 and mm(mode, sa=None) == 1 and mm(mode, w=None) == 1 and mm(mode, sw=None) == 1
        assert mm(mode, c=None) == 1 and mm(mode, M=-1) == 1 and mm(mode, N=0) == 1 and mm(mode, K=0) == 1
        assert mm(mode, E=0) == 1 and mm(mode, E=1025) == 1 and mm(mode, offs=None) == 1          # dense: one expert
        assert mm(mode, N=72) == 4 and mm(mode, K=40) == 4 and mm(mode, M=1 << 31) == 4
        assert mm(mode, a=ODD) == 2 and mm(mode, w=ODD) == 2 and mm(mode, c=ODD) == 2 and mm(mode, sa=BYTE) == 2
        assert mm(mode, M=0, a=None, c=None) == 0
    assert mm(2) == 1 and mm(-1) == 1


def test_binding_refuses_what_is_not_there():
    import torch
    import block_scaled_mlp_gb300 as mx
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: mx.moe_route(x, 2), lambda: mx.token_group(ids, 4), lambda: mx.moe_combine(x, ids, k=1),
                 lambda: mx.fp8_block_quantize(x), lambda: mx.fp8_block_quantize_weight(x), lambda: mx.fp8_block_mm(x, x),
                 lambda: mx.fp8_block_mm_dgrad(mx.Fp8Block(x, x), mx.Fp8BlockWeight(x, None, x))):
        with pytest.raises(mx.MxError):
            call()
