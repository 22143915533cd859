"""The norm over clusters of CTAs: uneven slices, whose CTAs reach the exchange of the rows' sums at different times,
and a sum that replaces an input."""
import ctypes

import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64
from tests.test_gpu_norm import EPS, EY, _check_codes, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,d", [(32, 288), (64, 4128), (32, 8224), (96, 8480), (4096, 2080), (32, 16160)])
def test_uneven_slices(M, d):
    """The last CTA of a cluster has a few columns only.  Against 64 bits, and again and again bit for bit the same."""
    x, res, w = _inputs(M, d, True, M + d)
    X, R, W = x.cuda(), res.cuda(), w.cuda()
    want = mx.add_rmsnorm_fwd(X, W, R, eps=EPS, axis=mx.BOTH, layout=mx.SCALE_LINEAR, ckpt=True)
    r = (x.float() + res.float()).to(torch.bfloat16)
    y, n = ref64.rmsnorm(r.double(), w.double(), EPS)
    assert torch.equal(want["r"].cpu(), r)
    assert torch.all((ref64.f64(want["rstd"]) - n).abs() <= n * EY)
    _check_codes(want["q_row"], want["s_row"].view(M, d // 32), y)
    _check_codes(want["q_col"], want["s_col"].view(d, M // 32), y.t().contiguous())
    for _ in range(20):
        f = mx.add_rmsnorm_fwd(X, W, R, eps=EPS, axis=mx.BOTH, layout=mx.SCALE_LINEAR, ckpt=True)
        for k in ("rstd", "y", "q_row", "s_row", "q_col", "s_col"):
            assert torch.equal(f[k], want[k]), k
        assert torch.equal(f["ckpt"].codes, want["ckpt"].codes)


@pytest.mark.parametrize("axis", [1, 2, 3])
@pytest.mark.parametrize("M,d", [(64, 544), (32, 8192), (320, 2080)])
def test_sum_may_replace_an_input_with_codes(M, d, axis):
    x, res, w = (t.cuda() for t in _inputs(M, d, True, 8))
    want = mx.add_rmsnorm_fwd(x, w, res, eps=EPS, axis=axis, layout=mx.SCALE_LINEAR, ckpt=True)
    P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for into in ("x", "res"):
        a, b = x.clone(), res.clone()
        r = a if into == "x" else b
        new = {k: None if want[k] is None else torch.empty_like(want[k]) for k in ("rstd", "y", "q_row", "s_row", "q_col", "s_col")}
        ck = mx.Ckpt8(torch.empty_like(want["ckpt"].codes), torch.empty_like(want["ckpt"].scales))
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert mx.lib().mx_add_rmsnorm_fwd(P(a), P(b), P(w), M, d, EPS, P(r), P(new["rstd"]), P(new["y"]), axis, 0, 0,
                                           P(new["q_row"]), P(new["s_row"]), P(new["q_col"]), P(new["s_col"]), P(ck.codes),
                                           P(ck.scales), st) == 0
        assert torch.equal(r, want["r"])
        assert all(torch.equal(new[k], want[k]) for k in new if new[k] is not None)
        assert torch.equal(ck.codes, want["ckpt"].codes) and torch.equal(ck.scales, want["ckpt"].scales)


@pytest.fixture
def small_clusters():
    """As on a device that holds no cluster of more than eight CTAs."""
    assert mx.lib().mx_selftest_norm_clusters(8) == 0
    yield
    assert mx.lib().mx_selftest_norm_clusters(0) == 0


@pytest.mark.parametrize("M,d", [(32, 32), (32, 2304), (64, 7168), (32, 8224), (32, 16384), (4096, 8192), (2048, 12320)])
def test_clusters_of_eight(M, d, small_clusters):
    x, res, w = _inputs(M, d, True, M + d)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS, axis=mx.BOTH, layout=mx.SCALE_LINEAR, ckpt=True)
    r = (x.float() + res.float()).to(torch.bfloat16)
    y, n = ref64.rmsnorm(r.double(), w.double(), EPS)
    assert torch.equal(f["r"].cpu(), r)
    assert torch.all((ref64.f64(f["rstd"]) - n).abs() <= n * EY)
    _check_codes(f["q_row"], f["s_row"].view(M, d // 32), y)
    _check_codes(f["q_col"], f["s_col"].view(d, M // 32), y.t().contiguous())
    assert torch.equal(ref64.f64(mx.ckpt8_load(f["ckpt"])), ref64.int8_values(r.double()))


def test_refuses_other_cluster_limits():
    assert mx.lib().mx_selftest_norm_clusters(3) == 1 and mx.lib().mx_selftest_norm_clusters(-1) == 1
