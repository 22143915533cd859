"""Ragged expert products against 64-bit references.

Products of bf16 values are exact in fp32; a sum of C of them in fp32 is off
by at most C * 2^-24 of the sum of magnitudes in any order (the tensor core
may truncate instead of rounding: 2^-23), and the result is rounded once to
bf16 (2^-8 of the value at most).
"""
import numpy as np
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _close(got, ref, mag, C):
    got = got.cpu().double()
    assert got.shape == ref.shape
    tol = ref.abs() * 2.0 ** -8 + mag * (C * 2.0 ** -23)
    worst = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
    assert torch.isfinite(got).all() and worst <= 0, worst


def _case(counts, spare, N, K, seed):
    M = sum(counts) + spare
    x, dout, w = _bf16((M, K), seed), _bf16((M, N), seed + 1, 0.1), _bf16((len(counts), N, K), seed + 2, 0.05)
    return x, dout, w, torch.tensor(np.cumsum(counts), dtype=torch.int32)


def _check(counts, spare, N, K, seed=0):
    x, dout, w, offs = _case(counts, spare, N, K, seed)
    err = mx.ErrorWord()
    X, D, W, O = x.cuda(), dout.cuda(), w.cuda(), offs.cuda()
    out = mx.ragged_mm(X, W, O, err=err)
    dx = mx.ragged_mm_dgrad(D, W, O, err=err)
    dw = mx.ragged_mm_wgrad(D, X, O, err=err)
    torch.cuda.synchronize()
    err.check()
    M, ends = x.shape[0], [0] + offs.tolist()
    ref = dict(out=torch.zeros(M, N).double(), dx=torch.zeros(M, K).double(), dw=torch.zeros(w.shape).double())
    mag = {k: v.clone() for k, v in ref.items()}
    x, dout, w = x.double(), dout.double(), w.double()
    for e in range(len(counts)):
        r = slice(ends[e], ends[e + 1])
        for dst, f in ((ref, lambda t: t), (mag, torch.abs)):
            dst["out"][r] = f(x[r]) @ f(w[e]).t()
            dst["dx"][r] = f(dout[r]) @ f(w[e])
            dst["dw"][e] = f(dout[r]).t() @ f(x[r])
    _close(out, ref["out"], mag["out"], K)
    _close(dx, ref["dx"], mag["dx"], N)
    _close(dw, ref["dw"], mag["dw"], max(counts + [1]))
    return out, dx, dw


@pytest.mark.parametrize("counts", [[64], [1], [16], [17], [63], [65], [128], [1, 2, 3], [0, 0, 5, 0], [100, 0, 33, 64, 1],
                                    [256], [257, 255], [300, 1, 0, 700, 31]])
@pytest.mark.parametrize("N,K", [(256, 128), (264, 72), (8, 8), (520, 1000)])
def test_products(counts, N, K):
    _check(counts, 0, N, K, sum(counts) + N)


@pytest.mark.parametrize("counts", [[1], [8, 0, 3], [33, 1], [64, 64, 64], [300, 17], [257, 0, 600, 31]])
@pytest.mark.parametrize("N,K", [(1032, 2056), (4096, 512), (264, 4096)])
def test_few_tiles_and_long_contractions(counts, N, K):
    _check(counts, 3, N, K, sum(counts) + K)


@pytest.mark.parametrize("counts", [[128], [129, 31], [40, 64, 0, 90], [127, 1, 128, 0, 7], [600, 3], [1000]])
@pytest.mark.parametrize("N,K", [(1032, 264), (200, 2056), (4104, 512)])
def test_tiles_of_128_rows(counts, N, K):
    out, dx, _ = _check(counts, 5, N, K, sum(counts) + N)
    assert not out[-5:].any() and not dx[-5:].any()


@pytest.mark.parametrize("counts,N,K", [([8], 512, 7168), ([8], 7168, 512), ([31, 2], 1000, 1032), ([100], 1024, 4096),
                                        ([60, 3], 2048, 1600), ([64], 2304, 1544), ([65, 64, 1], 1800, 2048),
                                        ([0, 3, 0, 1, 0], 1288, 3000), ([33, 31], 264, 1024)])
@pytest.mark.parametrize("spare", [0, 40])
def test_contractions_shared_by_pairs(counts, N, K, spare):
    """Few tiles: two and four pairs a tile, tiles of 32 and of 64 rows; other groups' and spare rows hold NaN."""
    out, dx, _ = _check(counts, spare, N, K, sum(counts) + N)
    n = sum(counts)
    assert not out[n:].any() and not dx[n:].any()
    x, dout, w, offs = (t.cuda() for t in _case(counts, spare, N, K, sum(counts) + N))
    last = max(e for e, c in enumerate(counts) if c)
    start = sum(counts[:last])
    x[:start], dout[:start], x[n:], dout[n:] = (float("nan"),) * 4
    out2, dx2 = mx.ragged_mm(x, w, offs), mx.ragged_mm_dgrad(dout, w, offs)
    assert torch.equal(out2[start:n].cpu(), out[start:n].cpu()) and torch.equal(dx2[start:n].cpu(), dx[start:n].cpu())
    assert not out2[n:].any() and not dx2[n:].any()
    err = mx.ErrorWord()
    bad = offs.clone()
    bad[-1] = -1
    assert not mx.ragged_mm(x, w, bad, err).any() and not mx.ragged_mm_dgrad(dout, w, bad, err).any()
    with pytest.raises(mx.MxError):
        err.check()


@pytest.mark.parametrize("counts,spare,N,K", [([5, 9, 0, 2], 77, 128, 256), ([0, 0], 40, 64, 64), ([700, 20], 1, 512, 320),
                                              ([3] * 40, 5, 136, 200), ([0] * 7, 9, 40, 24)])
def test_spare_rows_are_zero(counts, spare, N, K):
    out, dx, _ = _check(counts, spare, N, K, 3)
    n = sum(counts)
    assert not out[n:].any() and not dx[n:].any()


def test_many_experts():
    r = np.random.default_rng(1)
    _check([int(c) for c in r.integers(0, 5, 1024)], 3, 32, 40)
    _check([int(c) for c in r.multinomial(3000, r.dirichlet([0.3] * 64))], 0, 384, 256)


def test_no_rows():
    w = _bf16((3, 64, 128), 1).cuda()
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, d = w.new_empty((0, 128)), w.new_empty((0, 64))
    assert mx.ragged_mm(x, w, offs).shape == (0, 64) and mx.ragged_mm_dgrad(d, w, offs).shape == (0, 128)
    dw = mx.ragged_mm_wgrad(d, x, offs)
    assert dw.shape == (3, 64, 128) and not dw.any()


@pytest.mark.parametrize("counts", [[40, 23, 50], [200, 300, 90]])
def test_other_groups_and_spare_rows_do_not_leak(counts):
    """NaN and infinity in one group's rows (and behind the last) stay out of every other group's results."""
    N, K = 264, 328
    x, dout, w, offs = _case(counts, 30, N, K, 5)
    clean = [f(*a) for f, a in ((mx.ragged_mm, (x.cuda(), w.cuda(), offs.cuda())),
                                (mx.ragged_mm_dgrad, (dout.cuda(), w.cuda(), offs.cuda())),
                                (mx.ragged_mm_wgrad, (dout.cuda(), x.cuda(), offs.cuda())))]
    a, b = offs[0].item(), offs[1].item()
    x[a:b], dout[a:b] = float("nan"), float("inf")
    x[offs[2].item():], dout[offs[2].item():] = float("nan"), float("nan")
    out = mx.ragged_mm(x.cuda(), w.cuda(), offs.cuda())
    dx = mx.ragged_mm_dgrad(dout.cuda(), w.cuda(), offs.cuda())
    dw = mx.ragged_mm_wgrad(dout.cuda(), x.cuda(), offs.cuda())
    keep = [i for i in range(x.shape[0]) if not a <= i < b]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert torch.equal(dw[[0, 2]], clean[2][[0, 2]])
    assert torch.isnan(out[a:b]).all() and torch.isnan(dw[1]).all()


@pytest.mark.parametrize("ends", [[10, 5, 60], [-1, 5, 60], [10, 20, 65], [70, 70, 70]])
def test_bad_offsets_are_reported_and_give_zeros(ends):
    x, dout, w, _ = _case([20, 20, 24], 0, 64, 128, 1)
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for call in (lambda e: mx.ragged_mm(x.cuda(), w.cuda(), offs, err=e), lambda e: mx.ragged_mm_dgrad(dout.cuda(), w.cuda(), offs, err=e),
                 lambda e: mx.ragged_mm_wgrad(dout.cuda(), x.cuda(), offs, err=e)):
        err = mx.ErrorWord()
        c = call(err)
        torch.cuda.synchronize()
        assert err.value() == 8 and not c.any()


def test_gradients_against_differences():
    """The product is bilinear: central differences are exact up to rounding, the gradients are off by their bf16
    rounding, 2^-8 of each term."""
    x, dout, w, offs = _case([5, 0, 40, 19], 0, 72, 56, 9)
    dx = mx.ragged_mm_dgrad(dout.cuda(), w.cuda(), offs.cuda()).cpu().double()
    dw = mx.ragged_mm_wgrad(dout.cuda(), x.cuda(), offs.cuda()).cpu().double()
    e = torch.repeat_interleave(torch.arange(4), torch.tensor([5, 0, 40, 19]))
    loss = lambda a, b: (dout.double() * torch.einsum("tk,tnk->tn", a, b[e])).sum()  # noqa: E731
    x, w = x.double(), w.double()
    for seed in range(4):
        g = torch.Generator().manual_seed(seed)
        v, u = torch.randn(x.shape, generator=g, dtype=torch.float64), torch.randn(w.shape, generator=g, dtype=torch.float64)
        h = 1e-3
        for grad, num, t in ((dx, loss(x + h * v, w) - loss(x - h * v, w), v), (dw, loss(x, w + h * u) - loss(x, w - h * u), u)):
            assert abs(num / (2 * h) - (grad * t).sum()) <= (grad * t).abs().sum() * 2.0 ** -8 + 1e-5


def test_repeatable_and_on_another_stream():
    x, dout, w, offs = (t.cuda() for t in _case([100, 0, 33, 420, 1], 11, 520, 392, 2))

    def once():
        return mx.ragged_mm(x, w, offs), mx.ragged_mm_dgrad(dout, w, offs), mx.ragged_mm_wgrad(dout, x, offs)

    a = once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = once()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_refuses_tensors_it_cannot_take():
    x, dout, w, offs = (t.cuda() for t in _case([5, 9], 0, 64, 128, 1))
    bad = [lambda: mx.ragged_mm(x.float(), w, offs), lambda: mx.ragged_mm(x, w[:1].contiguous(), offs),
           lambda: mx.ragged_mm(x[:, :64].contiguous(), w, offs), lambda: mx.ragged_mm(x, w, offs.long()),
           lambda: mx.ragged_mm(x, w.transpose(1, 2), offs), lambda: mx.ragged_mm(x, w, offs.cpu()),
           lambda: mx.ragged_mm_dgrad(x, w, offs), lambda: mx.ragged_mm_wgrad(dout[:10].contiguous(), x, offs),
           lambda: mx.ragged_mm(x[:, :124].contiguous(), w[:, :, :124].contiguous(), offs),
           lambda: mx.ragged_mm_wgrad(dout, x[:, 0], offs), lambda: mx.ragged_mm(x, w, offs[:0])]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()
