"""Weights of small scores.  A score is exact to 2^-18 of itself, and below 2^-126, where fp32 has steps of 2^-149, to four of
those (two of the exponential's, a half for each of the roundings after it)."""
import numpy as np
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from test_gpu_route import SCORES, _scores

pytestmark = pytest.mark.gpu


def _check_weights(l, k, score, renorm, scale=1.0):
    ids, w = mx.moe_route(l, k, score=SCORES[score], renorm=renorm, scale=scale)
    s = np.take_along_axis(_scores(l.cpu().double().numpy(), score), ids.cpu().numpy().astype(np.int64), 1)
    t = s.sum(1, keepdims=True) + 1e-20 if renorm else 1.0
    want = scale * s / t
    # four steps of each of the k scores, and of the weight itself where that is so small
    tol = 2.0 ** -18 * np.abs(want) + scale * 4 * 2.0 ** -149 * (1 + k * s / t) / t + 2.0 ** -149
    off = np.abs(w.cpu().double().numpy() - want) - tol
    assert (off <= 0).all(), (off.max(), np.unravel_index(off.argmax(), off.shape))
    return w


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("k", [1, 3])
def test_sigmoid_of_very_negative_logits(dtype, renorm, k):
    l = torch.linspace(-104, -80, 600, dtype=torch.float64).repeat_interleave(8).view(600, 8)
    l = (l + torch.rand((600, 8), generator=torch.Generator().manual_seed(k), dtype=torch.float64) * 0.5).to(dtype).cuda()
    w = _check_weights(l, k, "sigmoid", renorm)
    if renorm:
        assert (w[l.max(1).values > -100] > 0).all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [4, 64, 1000])
def test_softmax_far_below_the_largest(renorm, E):
    """Differences that fp32 rounds by up to 2^-18: as much as a score may be off altogether."""
    g = torch.Generator().manual_seed(E)
    l = -torch.rand((800, E), generator=g) * 30 - 60
    l[:, 1] = torch.rand(800, generator=g) * 40
    _check_weights(l.cuda(), 4, "softmax", renorm, 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ordinary_logits(score):
    l = (torch.randn((500, 64), generator=torch.Generator().manual_seed(1)) * 8).cuda()
    for renorm in (True, False):
        _check_weights(l, 8, score, renorm)


@pytest.mark.parametrize("renorm", [True, False])
def test_logits_a_whole_range_apart(renorm):
    """Differences past fp32's largest number, and logits that are -inf among them."""
    g = torch.Generator().manual_seed(3)
    l = (torch.rand((40, 12), generator=g) * 2 - 1) * 3.4e38
    l[::2, 3] = -float("inf")
    l[::3, 7:] = torch.finfo(torch.float32).min
    l[::5, 0] = torch.finfo(torch.float32).max
    w = _check_weights(l.cuda(), 9, "softmax", renorm)
    assert torch.isfinite(w).all()
