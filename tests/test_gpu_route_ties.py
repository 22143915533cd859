"""Routing where ties and near-ties meet: experts that are equal by their inputs at the border of the k, with others before
them that fp32 cannot tell from them.  The numbers are those of c in double precision, equal ones by number."""
import numpy as np
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from test_gpu_route import _check, _logits, _scores

pytestmark = pytest.mark.gpu

SCORES = ["softmax", "sigmoid"]


def _next(x, n=1):
    """The fp32 value n steps above x."""
    x = np.float32(x)
    for _ in range(n):
        x = np.nextafter(x, np.float32(np.inf))
    return x


def _on_gpu(bias):
    return torch.from_numpy(np.asarray(bias, np.float32)).cuda()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("low,high", [(0.0, 2.0 ** -30), (0.003, _next(0.003)), (0.003, _next(0.003, 3)), (-0.25, _next(-0.25))])
@pytest.mark.parametrize("E,others", [(3, 0), (3, 5), (5, 0), (8, 56), (33, 200), (40, 0)])
def test_twins_behind_a_nearly_equal_one(score, low, high, E, others):
    """Expert 0 is worth a little less than all others of the first E, which are twins: the first k of those are chosen."""
    bias = _on_gpu([low] + [high] * (E - 1) + [-10.0] * others)
    l = torch.zeros((3, E + others), device="cuda")
    l[1] = 1.5
    for k in {1, 2, E // 2, min(E - 1, 32)}:
        ids, _ = _check(l, k, score=score, bias=bias)
        assert ids[0].tolist() == list(range(1, k + 1))
    ids, _ = _check(l, 2, score=score, bias=bias.flip(0).contiguous())      # the lesser one has the highest number
    assert ids[0].tolist() == [others, others + 1]


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("k", [2, 5, 8])
def test_several_levels_of_twins(score, k):
    """Levels one step apart, which fp32 sums cannot tell from one another, each with several experts."""
    for seed in range(60):
        g = np.random.default_rng(seed)
        E = int(g.integers(k + 1, 70))
        steps = g.integers(0, 4, E)
        bias = _on_gpu([_next(2e-3, int(n)) for n in steps])
        _check(torch.zeros((2, E), device="cuda"), k, score=score, bias=bias)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("groups,top", [(1, 1), (8, 4)])
def test_biases_that_have_walked(score, groups, top):
    """Balance biases after many steps of +-1e-3 in fp32: sums of one value that went other ways differ in their last bits.  A
    padding token has equal logits."""
    for seed in range(300):
        g = np.random.default_rng(seed)
        bias = np.zeros(64, np.float32)
        for _ in range(int(g.integers(20, 400))):
            bias += np.float32(1e-3) * np.sign(g.normal(size=64)).astype(np.float32)
        _check(torch.zeros((1, 64), device="cuda"), 8, score=score, bias=_on_gpu(bias), groups=groups, top_groups=top)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("groups,top", [(1, 1), (6, 3)])
def test_twins_of_several_logits(score, dtype, groups, top):
    """A few logits, each with the bias that brings its score to 0.7 to within some of the bias's steps: nearly all experts
    are as near as fp32 can tell, and many are twins."""
    for seed in range(80):
        g = np.random.default_rng(seed)
        l = torch.from_numpy(g.integers(-2, 3, (1, 48)).astype(np.float32) / 2).to(dtype)
        s = _scores(l.double().numpy(), score)[0]
        bias = [_next(0.7 - v, int(n)) for v, n in zip(s, g.integers(0, 3, 48))]
        _check(l.cuda(), int(g.integers(1, 13)), score=score, bias=_on_gpu(bias), groups=groups, top_groups=top)


@pytest.mark.parametrize("score", SCORES)
def test_one_large_score_among_small_ones(score):
    """Scores near one with biases near minus one beside scores near nothing: the one's fp32 value is off by far more than the
    others' are."""
    for seed in range(40):
        g = np.random.default_rng(seed)
        l = torch.from_numpy(np.r_[g.normal() + 9, g.normal(size=15) * 3 - 30].astype(np.float32))[None]
        s = _scores(l.double().numpy(), score)[0]
        bias = np.zeros(16, np.float32)
        bias[0] = -s[0]
        bias[1:] = s[0] + np.float64(bias[0]) + g.integers(-3, 4, 15) * 2.0 ** -26
        _check(l.cuda(), 4, score=score, bias=_on_gpu(bias))


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("groups,top", [(1, 1), (6, 3)])
def test_a_bias_of_a_masked_expert_does_not_matter(score, groups, top):
    """c of a logit of -inf is -inf, whatever the bias: a NaN there spoils the tokens that may choose the expert alone."""
    E = 48
    l = _logits(20, E, 3)
    bias = torch.from_numpy(np.random.default_rng(1).normal(size=E).astype(np.float32)).cuda() * 0.1
    bias[5] = bias[30] = float("nan")
    l[:12, 5] = -float("inf")
    l[:12, 30] = -float("inf")
    ids, w = _check(l[:12].contiguous(), 6, score=score, bias=bias, groups=groups, top_groups=top)
    got = mx.moe_route(l, 6, score=SCORES.index(score), bias=bias, groups=groups, top_groups=top)
    assert torch.equal(got[0][:12], ids) and torch.equal(got[1][:12], w)
    assert torch.isnan(got[1][12:]).all() and (got[0][12:] == torch.arange(6, device="cuda")).all()


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("k", [1, 4, 8])
def test_infinite_sums_at_the_border(score, k):
    """Masked experts right behind the k-th, fewer than k left, and biases of plus and minus infinity."""
    E, inf = 40, float("inf")
    for left in (k - 1, k, k + 1):
        l = torch.full((30, E), -inf)
        v = _logits(30, E, left).cpu()
        for t in range(30):
            at = torch.randperm(E, generator=torch.Generator().manual_seed(t))[:left]
            l[t, at] = v[t, at]
        bias = torch.from_numpy(np.random.default_rng(k).integers(-2, 3, E).astype(np.float32)).cuda() * 0.125
        _check(l.cuda(), k, score=score, bias=bias)
        _check(l.cuda(), k, score=score, bias=bias, groups=8, top_groups=4)
    l = _logits(30, E, 77)
    for seed in range(12):
        g = np.random.default_rng(seed)
        bias = g.choice([0.0, 0.25, inf, -inf], E, p=[0.4, 0.4, 0.1, 0.1] if seed % 2 else [0.05, 0.05, 0.1, 0.8])
        _check(l, k, score=score, bias=_on_gpu(bias))


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("far", [88.4, 88.7, 89.0, 95.0, 140.0, 1e4])
def test_doubts_with_logits_beyond_the_range_of_44_bits(score, far):
    """All experts of the groups that are taken are chosen, two of them are closer than fp32 can tell, and one has a logit
    that scores of 44 bits are not made for."""
    for groups, top, size in ((8, 3, 2), (31, 2, 3), (1, 1, 5), (4, 1, 9)):
        E = groups * size
        l = torch.full((4, E), -30.0)
        l[:, :size * top] = 2.0 if score == "softmax" else 1.0
        for t in range(4):
            l[t, t % size] = 2.0 - far if score == "softmax" else -far
        s = _scores(l.double().numpy(), score)[0]
        bias = np.zeros(E, np.float32)
        bias[:size * top] = np.float32(0.5) - s[:size * top].astype(np.float32)
        bias[1:size * top:2] = np.nextafter(bias[1:size * top:2], np.float32(1))
        _check(l.cuda(), size * top, score=score, bias=_on_gpu(bias), groups=groups, top_groups=top)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups", [(8, 4), (12, 4), (32, 4), (64, 8), (30, 5)])
def test_group_values_past_the_largest_number(score, dtype, E, groups):
    """Experts put out of reach by the lowest finite bias, or ahead by the largest: a sum of two is none of fp32's numbers, and
    still ahead of minus infinity or behind plus infinity."""
    big = float(np.finfo(np.float32).max)
    for seed in range(20):
        g = np.random.default_rng(seed)
        bias = g.choice([-big, -big, -3e38, 0.0, -np.inf] if seed % 2 else [big, 3e38, 0.0, float("inf"), 0.25], E)
        l = torch.from_numpy(g.normal(size=(6, E)).astype(np.float32))
        l[1] = 0.5
        l[2, torch.from_numpy(g.random(E) < 0.3)] = -float("inf")
        k, top, b = int(g.integers(1, E // groups + 1)), int(g.integers(1, groups)), _on_gpu(bias)
        # a group of plus and minus infinity is worth a NaN, which spoils its token
        two = np.sort(np.where(np.isneginf(l.numpy()), -np.inf, bias).reshape(6, groups, -1), 2)[:, :, -2:]
        spoilt = (np.isposinf(two[:, :, 1]) & np.isneginf(two[:, :, 0])).any(1)
        l = l.to(dtype).cuda()
        _check(l[torch.from_numpy(~spoilt).cuda()].contiguous(), k, score=score, bias=b, groups=groups, top_groups=top)
        w = mx.moe_route(l, k, score=SCORES.index(score), bias=b, groups=groups, top_groups=top)[1]
        assert torch.equal(torch.isnan(w).all(1).cpu(), torch.from_numpy(spoilt))


@pytest.mark.parametrize("binade", [3, 6, 10])
def test_scores_as_far_off_as_they_are(binade):
    """Of two experts, one whose fp32 score is too large by as much as there is among four million logits and one whose score
    is as much too small, with biases that leave the second a little more: fp32 puts the first ahead."""
    g = torch.Generator().manual_seed(binade)
    x = (-np.log(2) * binade - torch.rand(1 << 22, generator=g) * 0.3).cuda()
    got = mx.moe_route(x[:, None].contiguous(), 1, score=SCORES.index("sigmoid"), renorm=False)[1][:, 0].double()
    exact = 1 / (1 + torch.exp(-x.double()))
    off = (got - exact) / exact
    low, high = torch.topk(-off, 100).indices, torch.topk(off, 100).indices
    xl, el = x[low].cpu().numpy(), exact[low].cpu().numpy()
    xh, eh = x[high].cpu().numpy(), exact[high].cpu().numpy()
    bl, bh = (-el).astype(np.float32), (-eh).astype(np.float32)
    step = np.abs(np.spacing(bl)).max().astype(np.float64)
    for i in range(100):
        to_go = eh[i] + bh[i].astype(np.float64) - (el + bl.astype(np.float64))
        j = np.argmax(to_go % step)
        b = np.float32(bl[j].astype(np.float64) + np.ceil(to_go[j] / step) * step)
        for flip in (False, True):
            l, bias = [xh[i], xl[j]], [bh[i], b]
            if flip:
                l.reverse(), bias.reverse()
            for k in (1, 2):
                _check(torch.tensor([l + [-50.0]]).cuda(), k, score="sigmoid", bias=_on_gpu(bias + [-9.0]))
