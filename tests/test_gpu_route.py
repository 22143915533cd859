"""Routing and grouping against 64-bit references: expert numbers and row maps equal, weights within the stated 2^-18,
gradients within bounds that are derived where they stand."""
import numpy as np
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu

SCORES = {"softmax": mx.SCORE_SOFTMAX, "sigmoid": mx.SCORE_SIGMOID}


def _scores(l, score):
    if score == "sigmoid":
        return 1 / (1 + np.exp(-l))
    m = l.max(1, keepdims=True)
    e = np.exp(l - np.where(np.isneginf(m), 0, m))
    z = e.sum(1, keepdims=True)
    return e / np.where(z == 0, 1, z)


def _ref(logits, k, score="softmax", bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    """ids and weights, token by token, in 64 bits (logits without NaN)."""
    l = logits.detach().cpu().double().numpy()
    T, E = l.shape
    s = _scores(l, score)
    c = s if bias is None else s + bias.cpu().double().numpy()
    c = np.where(np.isneginf(l), -np.inf, c)
    ids = np.zeros((T, k), np.int32)
    for t in range(T):
        allowed = np.arange(E)
        if groups > 1:
            worth = np.sort(c[t].reshape(groups, -1), 1)[:, ::-1][:, :2].sum(1)
            best = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            allowed = [e for e in range(E) if e // (E // groups) in best]
        order = l[t] if bias is None else c[t]
        ids[t] = sorted(allowed, key=lambda e: (-order[e], e))[:k]
    sel = np.take_along_axis(s, ids, 1)
    return ids, scale * sel / (sel.sum(1, keepdims=True) + 1e-20 if renorm else 1)


def _check(logits, k, **kw):
    kw_dev = {n: SCORES[v] if n == "score" else v for n, v in kw.items()}
    ids, w = mx.moe_route(logits, k, **kw_dev)
    rid, rw = _ref(logits, k, **kw)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == rid.shape
    bad = np.nonzero((ids.cpu().numpy() != rid).any(1))[0]
    assert bad.size == 0, (bad[:5], ids[bad[:2]], rid[bad[:2]])
    assert np.all(np.abs(w.cpu().double().numpy() - rw) <= 2.0 ** -18 * np.abs(rw) + 1e-37)
    return ids, w


def _logits(T, E, seed, dtype=torch.float32, std=1.5):
    return (torch.randn((T, E), generator=torch.Generator().manual_seed(seed)) * std).to(dtype).cuda()


def _bias(E, seed):
    return (torch.round(torch.randn(E, generator=torch.Generator().manual_seed(seed)) * 20) * 1e-3).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (7, 5, 5), (33, 16, 1), (257, 43, 8), (100, 64, 8), (65, 100, 6),
                                   (40, 256, 8), (9, 300, 10), (5, 1000, 32), (3, 1024, 32), (4, 33, 32)])
def test_without_groups(dtype, score, T, E, k):
    l = _logits(T, E, T + E, dtype)
    _check(l, k, score=score)
    _check(l, k, score=score, bias=_bias(E, E), renorm=False, scale=2.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(64, 8, 4, 8), (256, 8, 4, 8), (24, 4, 2, 6), (30, 3, 1, 10), (30, 3, 3, 4), (8, 8, 3, 3),
                                            (96, 32, 5, 8), (640, 5, 2, 32), (1024, 32, 1, 32), (40, 2, 1, 20), (62, 31, 30, 7),
                                            (416, 13, 4, 6), (64, 1, 1, 8)])
def test_with_groups(dtype, score, E, groups, top, k):
    l = _logits(50, E, E + groups, dtype)
    for bias in (None, _bias(E, 3)):
        _check(l, k, score=score, bias=bias, groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(64, 1, 1), (64, 8, 3), (30, 3, 2)])
def test_equal_scores_go_by_number(score, E, groups, top):
    l = torch.zeros((40, E), device="cuda")
    l[1] = -0.0
    l[2, ::2] = -0.0                                                      # -0 is 0
    l[3:] = torch.randint(-2, 3, (37, E), generator=torch.Generator().manual_seed(1)).float()
    for bias in (None, torch.zeros(E, device="cuda"), torch.full((E,), 0.125, device="cuda"),
                 torch.randint(0, 2, (E,), generator=torch.Generator().manual_seed(2)).float().cuda()):
        _check(l, 6, score=score, bias=bias, groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,groups,top", [(64, 8, 4), (256, 8, 4), (96, 12, 3), (30, 5, 2), (1024, 32, 7), (16, 16, 5)])
def test_equal_logits_with_biases_of_few_steps(score, dtype, E, groups, top):
    """Padding tokens: their groups' values are sums of biases, which are alike often, exactly or to within a rounding."""
    l = torch.zeros((6, E), dtype=dtype, device="cuda")
    l[4:] = _logits(2, E, 3, dtype)
    for seed in range(12):
        g = torch.Generator().manual_seed(seed)
        steps = torch.randint(-3, 4, (E,), generator=g) if seed % 2 else torch.round(torch.randn(E, generator=g) * 20)
        _check(l, min(5, E // groups * top), score=score, bias=(steps.float() * 1e-3).cuda(), groups=groups, top_groups=top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_close_scores_are_ordered_in_double_precision(score, dtype):
    """A bias that undoes the scores to within fp32's rounding: c differs by less than fp32 scores are exact to."""
    E = 96
    l = _logits(300, E, 5, dtype, 0.5)
    s = _scores(l.cpu().double().numpy(), score)
    for t in range(0, 300, 20):
        bias = torch.from_numpy((0.7 - s[t]).astype(np.float32)).cuda()
        _check(l, 8, score=score, bias=bias)
        _check(l, 8, score=score, bias=bias, groups=12, top_groups=5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_empty_rows(score):
    E, inf = 48, float("inf")
    l = _logits(60, E, 9)
    keep = torch.randint(0, 2, (60, E), generator=torch.Generator().manual_seed(4)).bool().cuda()
    l[~keep] = -inf
    l[0] = -inf                                            # nothing left
    l[1] = -inf
    l[1, 17] = 0.5                                         # one expert
    l[2] = torch.finfo(torch.float32).min                  # a mask of the type's lowest value
    l[3, :40] = torch.finfo(torch.float32).min
    for bias in (None, _bias(E, 1)):
        for renorm in (True, False):
            ids, w = _check(l, 5, score=score, bias=bias, renorm=renorm)
            assert not w[0].any() and ids[0].tolist() == [0, 1, 2, 3, 4] and ids[1, 0] == 17
        _check(l, 5, score=score, bias=bias, groups=6, top_groups=3)


def test_extreme_logits():
    l = _logits(64, 32, 2)
    l[:16] *= 30
    l[16:32] *= 1e4
    l[32:48] *= 1e-20
    _check(l, 4, score="softmax")
    _check(l[32:].contiguous(), 4, score="sigmoid")
    _check(l, 4, score="softmax", renorm=False)
    b = torch.tensor([0.0, -float("inf"), 1e30, float("inf")] * 8, device="cuda")
    _check(l[48:].contiguous(), 4, score="softmax", bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_nan_spoils_its_token_only(score, dtype):
    l = _logits(20, 50, 7, dtype)
    clean = mx.moe_route(l, 4, score=SCORES[score])
    l[3, 49] = float("nan")
    l[8] = float("nan")
    hit = [3, 8]
    if score == "softmax":
        l[11, 2] = float("inf")
        hit.append(11)
    ids, w = mx.moe_route(l, 4, score=SCORES[score])
    rest = [t for t in range(20) if t not in hit]
    assert torch.equal(ids[rest], clean[0][rest]) and torch.equal(w[rest], clean[1][rest])
    assert torch.isnan(w[hit]).all() and ids[hit].tolist() == [[0, 1, 2, 3]] * len(hit)
    ids, w = mx.moe_route(l[12:].contiguous(), 4, score=SCORES[score], bias=torch.full((50,), float("nan"), device="cuda"))
    assert torch.isnan(w).all() and (ids == torch.arange(4, device="cuda")).all()


def _ref_bwd(dw, l, ids, score, renorm, scale):
    """dlogits in 64 bits, and the sum of the magnitudes that go into each."""
    l, dw, ids = l.detach().cpu().double().numpy(), dw.cpu().double().numpy(), ids.cpu().numpy().astype(np.int64)
    s = _scores(l, score)
    sel = np.take_along_axis(s, ids, 1)
    t = sel.sum(1, keepdims=True) + 1e-20 if renorm else np.ones((l.shape[0], 1))
    ds = scale * (dw - ((dw * sel).sum(1, keepdims=True) / t if renorm else 0)) / t
    mag = abs(scale) * (abs(dw) + ((abs(dw) * sel).sum(1, keepdims=True) / t if renorm else 0)) / t
    full, full_mag = np.zeros_like(s), np.zeros_like(s)
    for j in range(ids.shape[1]):
        np.add.at(full, (np.arange(len(l)), ids[:, j]), ds[:, j])
        np.add.at(full_mag, (np.arange(len(l)), ids[:, j]), mag[:, j])
    if score == "sigmoid":
        d = s / (1 + np.exp(l))
        return full * d, full_mag * d
    back, back_mag = (ds * sel).sum(1, keepdims=True), (mag * sel).sum(1, keepdims=True)
    return s * (full - back), s * (full_mag + back_mag)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (33, 43, 8), (100, 64, 8), (20, 256, 8), (5, 1024, 32), (7, 500, 31)])
def test_gradient(dtype, score, renorm, T, E, k):
    """fp32: a score is exact to 2^-18, the quotients and products after it add a few 2^-24, all relative to the
    magnitudes that are added; one rounding to the logits' type (fp32's is in the 2^-17)."""
    l = _logits(T, E, T + k, dtype)
    if T > 2:
        l[1, : E // 2] = -float("inf")
        l[2] = -float("inf")
    ids, _ = mx.moe_route(l, k, score=SCORES[score], bias=_bias(E, 2))
    dw = torch.randn((T, k), generator=torch.Generator().manual_seed(E)).cuda()
    if T > 4:
        ids[3, 1] = ids[3, 0]                              # an expert named twice
    dl = mx.moe_route_bwd(dw, l, ids, score=SCORES[score], renorm=renorm, scale=2.5)
    ref, mag = _ref_bwd(dw, l, ids, score, renorm, 2.5)
    tol = mag * 2.0 ** -17 + (np.abs(ref) * 2.0 ** -8 if dtype == torch.bfloat16 else 0) + 1e-37
    assert dl.dtype == dtype and dl.shape == l.shape
    got = dl.cpu().double().numpy()
    assert np.isfinite(got).all() and (np.abs(got - ref) <= tol).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_against_differences(score, renorm):
    """Central differences of the 64-bit weights with the ids held: their own error is third order in 1e-4."""
    l = _logits(12, 24, 3)
    ids, _ = mx.moe_route(l, 5, score=SCORES[score])
    dw = torch.randn((12, 5), generator=torch.Generator().manual_seed(1)).cuda()
    dl = mx.moe_route_bwd(dw, l, ids, score=SCORES[score], renorm=renorm).cpu().double().numpy()
    x, i = l.cpu().double().numpy(), ids.cpu().numpy().astype(np.int64)

    def loss(x):
        sel = np.take_along_axis(_scores(x, score), i, 1)
        return (dw.cpu().double().numpy() * (sel / sel.sum(1, keepdims=True) if renorm else sel)).sum()

    for seed in range(4):
        v = np.random.default_rng(seed).normal(size=x.shape)
        num = (loss(x + 1e-4 * v) - loss(x - 1e-4 * v)) / 2e-4
        assert abs(num - (dl * v).sum()) <= 1e-5 * (np.abs(dl * v).sum() + 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k", [(1, 24, 1), (300, 24, 1), (65, 256, 8), (9, 7, 3)])
def test_weights_that_cannot_change_have_no_gradient(dtype, score, T, E, k):
    """Renormalised weights of one expert are constant, and alike gradients of several add up to that of a constant: 0, and
    no rounding's rest (the 1e-20 in the sum is below fp32's rounding of it)."""
    l = _logits(T, E, T, dtype)
    ids, _ = mx.moe_route(l, k, score=SCORES[score])
    dw = torch.randn((T, 1), generator=torch.Generator().manual_seed(5)).expand(T, k).contiguous().cuda()
    assert not mx.moe_route_bwd(dw, l, ids, score=SCORES[score], scale=2.5).any()


def test_gradient_reports_bad_ids():
    l = _logits(6, 10, 1)
    ids = torch.tensor([[0, 1]] * 6, dtype=torch.int32, device="cuda")
    dw = torch.ones((6, 2), device="cuda")
    want = mx.moe_route_bwd(dw, l, ids, score=mx.SCORE_SIGMOID, renorm=False)
    ids[2, 1], ids[4, 0] = 10, -1
    err = mx.ErrorWord()
    got = mx.moe_route_bwd(dw, l, ids, score=mx.SCORE_SIGMOID, renorm=False, err=err)
    assert err.value() == 8
    want[2, 1] = 0
    want[4, 0] = 0
    assert torch.equal(got, want)


# ---------------------------------------------------------------- grouping


def _ref_group(ids, E):
    ids = np.asarray(ids).reshape(-1)
    ok = (ids >= 0) & (ids < E)
    order = [r for r in np.argsort(ids, kind="stable") if ok[r]]
    dst, src = np.full(ids.size, -1, np.int32), np.full(ids.size, -1, np.int32)
    for i, r in enumerate(order):
        dst[r], src[i] = i, r
    return np.cumsum(np.bincount(ids[ok], minlength=E)).astype(np.int32), dst, src


def _group(ids, E):
    err = mx.ErrorWord()
    out = mx.token_group(torch.as_tensor(ids, dtype=torch.int32, device="cuda"), E, err=err)
    return [t.cpu().numpy() for t in out], err.value()


@pytest.mark.parametrize("R,E,seed", [(1, 1, 0), (31, 3, 1), (64, 64, 2), (1000, 16, 2), (1024, 64, 8), (1025, 7, 3), (5000, 64, 4),
                                      (20000, 1000, 5), (4096, 1, 6), (40961, 1024, 7), (700000, 256, 9)])
def test_groups(R, E, seed):
    ids = np.random.default_rng(seed).integers(0, E, R).astype(np.int32)
    got, err = _group(ids, E)
    assert err == 0 and all(np.array_equal(a, b) for a, b in zip(got, _ref_group(ids, E)))


def test_groups_of_all_in_one_and_of_a_matrix():
    ids = np.full((777, 3), 3, np.int32)
    got, err = _group(ids, 5)
    assert err == 0 and got[0].tolist() == [0, 0, 0, 2331, 2331] and got[1].tolist() == list(range(2331))
    got, err = _group(np.zeros(0, np.int32), 4)
    assert err == 0 and got[0].tolist() == [0] * 4 and got[1].size == 0


@pytest.mark.parametrize("R", [6, 3000])
def test_bad_expert_ids_are_reported_and_not_placed(R):
    ids = np.random.default_rng(R).integers(0, 3, R).astype(np.int32)
    ids[[1, R - 1, R // 2]] = [5, -2, 3]
    got, err = _group(ids, 3)
    assert err == 8 and all(np.array_equal(a, b) for a, b in zip(got, _ref_group(ids, 3)))
    assert (got[2][-3:] == -1).all()


def test_refuses_tensors_it_cannot_take():
    l = _logits(4, 16, 1)
    ids, w = mx.moe_route(l, 2)
    bad = [lambda: mx.moe_route(l.double(), 2), lambda: mx.moe_route(l[0], 2), lambda: mx.moe_route(l.t(), 2),
           lambda: mx.moe_route(l.cpu(), 2), lambda: mx.moe_route(l, 0), lambda: mx.moe_route(l, 17), lambda: mx.moe_route(l, 2.0),
           lambda: mx.moe_route(l, 2, bias=torch.zeros(15, device="cuda")), lambda: mx.moe_route(l, 2, bias=l[0].bfloat16()),
           lambda: mx.moe_route(l, 2, groups=3), lambda: mx.moe_route(l, 9, groups=2), lambda: mx.moe_route(l, 2, score=2),
           lambda: mx.moe_route(l, 2, scale=float("nan")), lambda: mx.moe_route(l, 2, scale="a"),
           lambda: mx.moe_route(torch.zeros((4, 1025), device="cuda"), 2),
           lambda: mx.moe_route_bwd(w, l, ids.long()), lambda: mx.moe_route_bwd(w[:3], l, ids),
           lambda: mx.moe_route_bwd(w.bfloat16(), l, ids), lambda: mx.moe_route_bwd(w, l.half(), ids),
           lambda: mx.token_group(ids.long(), 16), lambda: mx.token_group(ids, 0), lambda: mx.token_group(ids, 1025),
           lambda: mx.token_group(ids.t(), 16)]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()


def test_no_tokens():
    l = torch.zeros((0, 8), device="cuda")
    ids, w = mx.moe_route(l, 2)
    assert ids.shape == w.shape == (0, 2) and mx.moe_route_bwd(w, l, ids).shape == (0, 8)
