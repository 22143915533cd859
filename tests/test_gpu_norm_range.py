"""Where the norm's fp32 range ends, and that it does not end earlier."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64

pytestmark = pytest.mark.gpu


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64) * std).to(torch.bfloat16)


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("e", [-66, -40, 40, 56])
@pytest.mark.parametrize("M,d", [(3, 256), (5, 544), (400, 2080)])
def test_backward_of_small_and_large_rows(M, d, e, ckpt):
    """rstd's square may pass fp32, dx does not.  Tolerances as in test_gpu_norm: 2^-8 of a result (its bf16 rounding),
    2^-18 of the magnitudes in a sum, and rstd's own rounding."""
    r, w, dy = _bf16((M, d), M + d, 2.0 ** e), _bf16(d, 3), _bf16((M, d), 5)
    n = 1 / torch.sqrt((r.double() ** 2).mean(1))
    kept = mx.ckpt8_save(r.cuda()) if ckpt else r.cuda()
    dx, dw = mx.add_rmsnorm_bwd(dy.cuda(), kept, n.float().cuda(), w.cuda())
    at = ref64.int8_values(r.double()) if ckpt else r.double()
    gx, gw, mag, mw = ref64.rmsnorm_bwd(dy.double(), at, n, w.double())
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    assert torch.all((ref64.f64(dx) - gx).abs() <= gx.abs() * 2.0 ** -8 + mag * 2.0 ** -18)
    assert torch.all((ref64.f64(dw) - gw).abs() <= gw.abs() * 2.0 ** -8 + mw * 2.0 ** -18)


@pytest.mark.parametrize("axis", [0, 3])
@pytest.mark.parametrize("d", [256, 2080, 8192, 16384])
def test_statistic_of_a_row_with_one_large_value(d, axis):
    """One square of 2^24 beside ones: an fp32 sum drops each one that it adds to it.  The kernel adds at most eight
    squares in fp32 (four roundings of 2^-24 of the sum, halved by the root), the rest with its errors carried; rstd is
    rounded once (2^-24)."""
    M = 64
    x = torch.ones((M, d), dtype=torch.bfloat16)
    at = torch.randint(0, d, (M,), generator=torch.Generator().manual_seed(d))
    x[torch.arange(M), at] = 4096.0
    f = mx.add_rmsnorm_fwd(x.cuda(), torch.ones(d, dtype=torch.bfloat16).cuda(), eps=1e-5, axis=axis)
    n = ref64.rmsnorm(x.double(), torch.ones(d).double(), float(torch.tensor(1e-5)))[1]
    assert torch.all((ref64.f64(f["rstd"]) - n).abs() <= n * (2 + 1 + 0.1) * 2.0 ** -24)


@pytest.mark.parametrize("axis", [1, 3])
@pytest.mark.parametrize("d", [64, 1024, 16384])
def test_sum_of_squares_past_fp32(d, axis):
    """sum r^2 = 2^128: rstd and every result are zero; half of it: the norm."""
    M = 32
    over = torch.full((M, d), 2.0 ** 60, dtype=torch.bfloat16)
    over[:, 0] = 2.0 ** 64
    w = torch.ones(d, dtype=torch.bfloat16)
    f = mx.add_rmsnorm_fwd(over.cuda(), w.cuda(), axis=axis, layout=mx.SCALE_LINEAR)
    assert not f["rstd"].any() and not f["y"].any() and not f["q_row"].any() and not f["s_row"].any()
    under = torch.full((M, d), 2.0 ** 56, dtype=torch.bfloat16)
    f = mx.add_rmsnorm_fwd(under.cuda(), w.cuda(), axis=axis, layout=mx.SCALE_LINEAR)
    assert torch.all(f["rstd"] == 2.0 ** -56) and torch.all(f["y"] == 1)
    if d == 16384:                                            # sum r^2 = 2^128 with every |r| = 2^57
        f = mx.add_rmsnorm_fwd((under * 2).cuda(), w.cuda(), axis=axis, layout=mx.SCALE_LINEAR)
        assert not f["rstd"].any() and not f["y"].any()


@pytest.mark.parametrize("axis", [0, 1, 3])
def test_weights_past_the_product(axis):
    """|r w| < 2^128 is in range, whatever w is; from there on y is NaN, in that element alone."""
    M, d = 32, 256
    x = torch.ones((M, d), dtype=torch.bfloat16)
    x[:, 7] = 2.0
    w = torch.full((d,), 2.0 ** 100, dtype=torch.bfloat16)
    w[7] = 2.0 ** 127
    w[9] = 2.0 ** 127
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), axis=axis, layout=mx.SCALE_LINEAR)
    y = (x.double() * w.double()) / torch.sqrt((x.double() ** 2).mean(1, keepdim=True) + 1e-5)
    got = ref64.f64(f["y"])
    assert torch.isnan(got[:, 7]).all()
    keep = torch.arange(d) != 7
    assert torch.all((got - y).abs()[:, keep] <= y[:, keep] * (2.0 ** -8 + 2.5e-6))
    if axis:
        s = f["s_row"].view(M, d // 32)
        assert torch.all(s[:, 0] == 255) and not (s[:, 1:] == 255).any()
