"""Rows back to tokens and the gradients, against 64-bit references.

out: k products and an addend added in fp32, each step off by 2^-24 of the sum of magnitudes, one rounding to bf16
(2^-8).  drows: a product, 2^-24, rounded to bf16.  dweights: d products added in fp32 in any order."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _case(T, k, d, seed, E=9, padded=False):
    g = torch.Generator().manual_seed(seed)
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    offs, dst, src = mx.token_group_pad(ids.view(-1), max(E, k)) if padded else mx.token_group(ids, max(E, k))
    rows = _bf16((src.numel(), d), seed + 1).cuda()
    return rows, dst, src, torch.rand((T, k), generator=g).cuda(), _bf16((T, d), seed + 2).cuda(), _bf16((T, d), seed + 3).cuda()


def _close(got, ref, tol):
    got = got.cpu().double()
    assert got.shape == ref.shape and torch.isfinite(got).all() and ((got - ref).abs() <= tol).all(), ((got - ref).abs() - tol).max()


@pytest.mark.parametrize("T,k,d", [(1, 1, 8), (1, 8, 7168), (3, 2, 16), (17, 4, 1000), (130, 8, 264), (64, 32, 72), (257, 3, 2056),
                                   (5, 6, 20000), (1021, 2, 512)])
@pytest.mark.parametrize("padded", [False, True])
def test_forward_and_backward(T, k, d, padded):
    rows, dst, src, w, add, dout = _case(T, k, d, T + d, padded=padded)
    R = rows.cpu().double()[dst.cpu().long()].view(T, k, d)
    W, A, D = w.cpu().double()[..., None], add.cpu().double(), dout.cpu().double()
    for weights, addend in ((w, add), (w, None), (None, add), (None, None)):
        out = mx.moe_combine(rows, dst, weights=weights, k=k, add=addend)
        f = W if weights is not None else 1.0
        ref, mag = (R * f).sum(1), (R.abs() * f).sum(1)
        if addend is not None:
            ref, mag = ref + A, mag + A.abs()
        _close(out, ref, ref.abs() * 2.0 ** -8 + mag * ((k + 1) * 2.0 ** -24))
    drows, dw = mx.moe_combine_bwd(dout, rows, dst, src, w)
    ref = torch.zeros_like(rows.cpu().double())
    ref[dst.cpu().long()] = (W * D[:, None]).reshape(T * k, d)
    _close(drows, ref, ref.abs() * (2.0 ** -8 + 2.0 ** -23))
    _close(dw, (R * D[:, None]).sum(2), (R * D[:, None]).abs().sum(2) * (d * 2.0 ** -24))
    assert not drows[src < 0].any()


def test_rows_that_were_not_placed():
    """Negative places add nothing and get no gradient; places past the end are reported too."""
    rows, dst, src, w, add, dout = _case(40, 4, 136, 3)
    clean = mx.moe_combine(rows, dst, w), *mx.moe_combine_bwd(dout, rows, dst, src, w)
    bad = dst.clone().view(40, 4)
    gone = bad[7].clone().long()
    bad[7] = -1
    rows[gone] = float("nan")
    src = src.clone()
    src[gone] = -1
    out = mx.moe_combine(rows, bad, w)
    drows, dw = mx.moe_combine_bwd(dout, rows, bad, src, w)
    keep = [t for t in range(40) if t != 7]
    assert torch.equal(out[keep], clean[0][keep]) and not out[7].any()
    assert torch.equal(dw[keep], clean[2][keep]) and not dw[7].any()
    live = torch.ones(160, dtype=torch.bool, device="cuda")
    live[gone] = False
    assert torch.equal(drows[live], clean[1][live]) and not drows[gone].any()
    bad[7] = 160
    for call in (lambda e: mx.moe_combine(rows, bad, w, err=e), lambda e: mx.moe_combine_bwd(dout, rows, bad, src, w, err=e)[0]):
        err = mx.ErrorWord()
        again = call(err)
        assert err.value() == 8 and torch.isfinite(again).all()


@pytest.mark.parametrize("T", [40, 700])
def test_maps_that_are_not_inverse(T):
    """A row that two routed rows name gets the gradient of the one that it holds, one that none names gets zeros; both are
    reported, and each row is written once."""
    k, d = 4, 136
    rows, dst, src, w, _, dout = _case(T, k, d, 7)
    clean, dw0 = mx.moe_combine_bwd(dout, rows, dst, src, w)
    two = dst.clone()
    lost = int(two[5])
    two[5] = two[9]  # routed rows 5 and 9 name one row; the row that held 5 is named by none
    err = mx.ErrorWord()
    drows, dw = mx.moe_combine_bwd(dout, rows, two, src, w, err=err)
    assert err.value() == 8
    want = clean.clone()
    want[lost] = 0
    assert torch.equal(drows, want)
    assert torch.equal(dw.view(-1)[6:], dw0.view(-1)[6:])
    far = src.clone()
    far[lost] = T * k  # a routed row that there is not
    err = mx.ErrorWord()
    drows, _ = mx.moe_combine_bwd(dout, rows, dst, far, w, err=err)
    assert err.value() == 8 and torch.equal(drows, want)


def test_sum_is_the_gradient_of_the_gather():
    """<gather(x), r> = <x, combine(r)> with weights of one, to the outputs' bf16 rounding."""
    T, k, d = 50, 3, 256
    rows, dst, src, _, _, x = _case(T, k, d, 11)
    r = mx.moe_combine(rows, dst, k=k).double()
    a, b = (mx.gather_rows(x, src, div=k).double() * rows.double()).sum(), (x.double() * r).sum()
    assert abs(a - b) <= 2.0 ** -8 * (x.double() * r).abs().sum()


def test_gradients_against_differences():
    T, k, d = 12, 3, 64
    rows, dst, src, w, _, dout = _case(T, k, d, 5)
    drows, dw = mx.moe_combine_bwd(dout, rows, dst, src, w)
    at = dst.cpu().long()
    loss = lambda r, v: ((r[at].view(T, k, d) * v[..., None]).sum(1) * dout.cpu().double()).sum()  # noqa: E731
    r, v = rows.cpu().double(), w.cpu().double()
    g = torch.Generator().manual_seed(2)
    u, q = torch.randn(r.shape, generator=g, dtype=torch.float64), torch.randn(v.shape, generator=g, dtype=torch.float64)
    h = 1e-3  # bilinear: differences are exact but for rounding
    for grad, num, t in ((drows, loss(r + h * u, v) - loss(r - h * u, v), u), (dw, loss(r, v + h * q) - loss(r, v - h * q), q)):
        grad = grad.cpu().double()
        assert abs(num / (2 * h) - (grad * t).sum()) <= (grad * t).abs().sum() * 2.0 ** -8 + 1e-6


def test_no_tokens():
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    none = z(0, t=torch.int32)
    assert mx.moe_combine(z(0, 64), none, k=2).shape == (0, 64)
    src = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    drows, dw = mx.moe_combine_bwd(z(0, 64), torch.ones((3, 64), dtype=torch.bfloat16, device="cuda"), none, src, z(0, 2, t=torch.float32))
    assert drows.shape == (3, 64) and not drows.any() and dw.shape == (0, 2)
    out = mx.moe_combine(z(0, 64), torch.full((4,), -1, dtype=torch.int32, device="cuda"), k=2)
    assert out.shape == (2, 64) and not out.any()


def test_refuses_tensors_it_cannot_take():
    rows, dst, src, w, add, dout = _case(6, 2, 64, 1)
    bad = [lambda: mx.moe_combine(rows.float(), dst, w), lambda: mx.moe_combine(rows, dst), lambda: mx.moe_combine(rows, dst[:11], w),
           lambda: mx.moe_combine(rows, dst, w, k=3), lambda: mx.moe_combine(rows, dst, w.bfloat16()),
           lambda: mx.moe_combine(rows, dst.long(), w), lambda: mx.moe_combine(rows, dst, w, add=add[:5]),
           lambda: mx.moe_combine(rows, dst, w, add=add.float()), lambda: mx.moe_combine(rows[:, :60].contiguous(), dst, w),
           lambda: mx.moe_combine(rows[:, ::2], dst, w), lambda: mx.moe_combine(rows, dst, k=0), lambda: mx.moe_combine(rows, dst, k=33),
           lambda: mx.moe_combine_bwd(dout[:, :32].contiguous(), rows, dst, src, w), lambda: mx.moe_combine_bwd(dout, rows, dst, src[:4], w),
           lambda: mx.moe_combine_bwd(dout, rows, dst[:4], src, w), lambda: mx.moe_combine_bwd(dout, rows, dst, src, w[:5])]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()
