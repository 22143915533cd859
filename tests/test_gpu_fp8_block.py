"""FP8 with 128-blocks against 64-bit references: codes and scales bit for bit, products within derived bounds.

A product of two E4M3 values is exact; a sum of C of them in fp32 is off by at most C * 2^-23 of the sum of magnitudes
(the tensor core may truncate), the product of the scales and the sums over the blocks by 2^-24 each more; one rounding
to bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu

LEAST = 2.0 ** -100


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _ref_rows(x):
    """(codes, scales [blocks, rows]) of a bf16 matrix on the host."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 128)).view(rows, -1, 128)
    m = v.abs().amax(2).clamp_min(LEAST)
    q = (v * 448 / m[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).view(rows, -1)[:, :cols]
    return q, (m.float() / 448).t()


def _ref_weight(w):
    E, N, K = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -K % 128, 0, -N % 128))
    v = v.view(E, v.shape[1] // 128, 128, v.shape[2] // 128, 128)
    m = v.abs().amax((2, 4)).clamp_min(LEAST)
    q = (v * 448 / m[:, :, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.reshape(E, v.shape[1] * 128, -1)[:, :N, :K], m.float() / 448


def _decode(codes):
    return codes.cpu().view(torch.float8_e4m3fn).double()


def _row_values(q):
    return _decode(q.codes) * q.scales.cpu().double().t().repeat_interleave(128, 1)[:, :q.codes.shape[1]]


def _weight_values(w):
    N, K = w.codes.shape[-2:]
    s = w.scales.cpu().double().view(-1, *w.scales.shape[-2:])
    return _decode(w.codes).view(-1, N, K) * s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


# ---------------------------------------------------------------- casts


def _rows_equal(x):
    q = mx.fp8_block_quantize(x.cuda())
    codes, scales = _ref_rows(x)
    assert torch.equal(q.codes.cpu(), codes) and torch.equal(q.scales.cpu(), scales)


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (7, 112), (33, 256), (100, 1000 // 16 * 16), (130, 2064), (2, 7168),
                                       (17, 32768)])
def test_rows(rows, cols):
    _rows_equal(_bf16((rows, cols), rows + cols))
    x = _bf16((rows, cols), rows, 1e-3)
    x[:, ::7] *= 300
    x[rows // 2] = 0
    _rows_equal(x)


def test_every_fraction_against_every_largest():
    """All 128 fractions of a block's largest with all 128 fractions of its values over six binades: every tie that two
    bf16 values can make."""
    m = (1 + torch.arange(128) / 128).bfloat16()
    rows = []
    for e in range(6):
        v = ((1 + torch.arange(128) / 128) * 2.0 ** -(e + 1)).bfloat16()
        rows.append(torch.cat([v.repeat(128, 1)[:, :127], m[:, None]], 1))
        rows.append(torch.cat([-v.repeat(128, 1)[:, 1:], m[:, None]], 1))
    x = torch.cat(rows)
    _rows_equal(x)
    _rows_equal(x * 2.0 ** 100)
    _rows_equal((x.double() * 2.0 ** -95).bfloat16())


@pytest.mark.parametrize("e", [-133, -126, -120, -101, -100, -99, -10, 0, 60, 119, 126])
def test_ends_of_the_range(e):
    x = (_bf16((4, 256), 3).clamp(-3.9, 3.9).double() * 2.0 ** (e - 1)).bfloat16()
    _rows_equal(x)
    w = x[:, :128].reshape(1, 4 * 8, 16)
    q = mx.fp8_block_quantize_weight(w.cuda())
    codes, scales = _ref_weight(w)
    assert torch.equal(q.codes.cpu(), codes) and torch.equal(q.scales.cpu(), scales)


def test_a_block_without_finite_values_spoils_itself_only():
    x = _bf16((6, 400), 1)
    clean = mx.fp8_block_quantize(x.cuda())
    x[1, 5], x[2, 399], x[4, 130] = float("nan"), float("inf"), -float("inf")
    q = mx.fp8_block_quantize(x.cuda())
    hit = torch.zeros((4, 6), dtype=torch.bool)
    hit[0, 1] = hit[3, 2] = hit[1, 4] = True
    at = hit.t().repeat_interleave(128, 1)[:, :400]
    assert torch.isnan(q.scales.cpu()[hit]).all() and torch.equal(q.scales.cpu()[~hit], clean.scales.cpu()[~hit])
    assert (q.codes.cpu()[at] == 0x7F).all() and torch.equal(q.codes.cpu()[~at], clean.codes.cpu()[~at])
    w = _bf16((2, 144, 272), 1)
    clean = mx.fp8_block_quantize_weight(w.cuda())
    w[1, 143, 271] = float("nan")
    q = mx.fp8_block_quantize_weight(w.cuda())
    assert torch.isnan(q.scales[1, 1, 2]) and (q.codes[1, 128:, 256:] == 0x7F).all() and (q.codes_t[1, 256:, 128:] == 0x7F).all()
    assert torch.equal(q.codes[0], clean.codes[0]) and torch.equal(q.codes[1, :128], clean.codes[1, :128])
    assert torch.equal(q.scales[1, 0], clean.scales[1, 0])


@pytest.mark.parametrize("T,cols,k", [(1, 128, 1), (5, 272, 3), (64, 1024, 8), (40, 48, 2)])
def test_rows_gathered(T, cols, k):
    x = _bf16((T, cols), T)
    src = torch.randperm(T * k, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    src[::5] = -1
    q = mx.fp8_block_quantize(x.cuda(), src=src.cuda(), div=k)
    want = mx.fp8_block_quantize(mx.gather_rows(x.cuda(), src.cuda(), div=k))
    assert torch.equal(q.codes, want.codes) and torch.equal(q.scales, want.scales)
    err = mx.ErrorWord()
    last = T * k - 1
    src[last] = T * k
    q = mx.fp8_block_quantize(x.cuda(), src=src.cuda(), div=k, err=err)
    assert err.value() == 8 and not q.codes[last].any()
    keep = list(range(last))
    assert torch.equal(q.codes[keep], want.codes[keep]) and torch.equal(q.scales[:, keep], want.scales[:, keep])


@pytest.mark.parametrize("E,N,K", [(1, 16, 16), (2, 128, 128), (3, 144, 272), (1, 1024, 512), (5, 48, 400), (2, 400, 48)])
def test_weights(E, N, K):
    w = _bf16((E, N, K), N + K, 0.02)
    codes, scales = _ref_weight(w)
    q = mx.fp8_block_quantize_weight(w.cuda())
    assert torch.equal(q.codes.cpu(), codes) and torch.equal(q.scales.cpu(), scales)
    assert torch.equal(q.codes_t.cpu(), codes.transpose(1, 2))
    alone = mx.fp8_block_quantize_weight(w.cuda(), transposed=False)
    assert alone.codes_t is None and torch.equal(alone.codes, q.codes) and torch.equal(alone.scales, q.scales)
    flat = mx.fp8_block_quantize_weight(w[0].cuda().contiguous())
    assert torch.equal(flat.codes, q.codes[0]) and torch.equal(flat.codes_t, q.codes_t[0]) and torch.equal(flat.scales, q.scales[0])


# ---------------------------------------------------------------- products


def _case(counts, spare, N, K, seed):
    M = sum(counts) + spare
    x, dout = mx.fp8_block_quantize(_bf16((M, K), seed).cuda()), mx.fp8_block_quantize(_bf16((M, N), seed + 1, 0.1).cuda())
    w = mx.fp8_block_quantize_weight(_bf16((len(counts), N, K), seed + 2, 0.05).cuda())
    return x, dout, w, torch.tensor(np.cumsum(counts), dtype=torch.int32).cuda()


def _close(got, ref, mag, C):
    got = got.cpu().double()
    assert got.shape == ref.shape
    tol = ref.abs() * 2.0 ** -8 + mag * (C * 2.0 ** -23 + (C // 128 + 3) * 2.0 ** -24)
    worst = ((got - ref).abs() - tol).max() if got.numel() else torch.tensor(-1.0)
    assert torch.isfinite(got).all() and worst <= 0, worst


def _check(counts, spare, N, K, seed=0):
    x, dout, w, offs = _case(counts, spare, N, K, seed)
    err = mx.ErrorWord()
    out, dx = mx.fp8_block_mm(x, w, offs, err=err), mx.fp8_block_mm_dgrad(dout, w, offs, err=err)
    torch.cuda.synchronize()
    err.check()
    X, D, W = _row_values(x), _row_values(dout), _weight_values(w)
    M, ends = X.shape[0], [0] + offs.tolist()
    ref = dict(out=torch.zeros(M, N).double(), dx=torch.zeros(M, K).double())
    mag = {k: v.clone() for k, v in ref.items()}
    for e in range(len(counts)):
        r = slice(ends[e], ends[e + 1])
        for dst, f in ((ref, lambda t: t), (mag, torch.abs)):
            dst["out"][r] = f(X[r]) @ f(W[e]).t()
            dst["dx"][r] = f(D[r]) @ f(W[e])
    _close(out, ref["out"], mag["out"], K)
    _close(dx, ref["dx"], mag["dx"], N)
    n = sum(counts)
    assert not out[n:].any() and not dx[n:].any()
    return out, dx


@pytest.mark.parametrize("counts", [[64], [1], [16], [33], [128], [1, 2, 3], [0, 0, 5, 0], [100, 0, 33, 64, 1], [256], [257, 255],
                                    [300, 1, 0, 700, 31]])
@pytest.mark.parametrize("N,K", [(256, 128), (272, 80), (16, 16), (528, 1008), (144, 400)])
def test_grouped_products(counts, N, K):
    _check(counts, 0, N, K, sum(counts) + N)


@pytest.mark.parametrize("counts", [[1], [8, 0, 3], [33, 1], [64, 64, 64], [300, 17]])
@pytest.mark.parametrize("N,K", [(1040, 2064), (4096, 512), (272, 7168)])
def test_long_contractions(counts, N, K):
    _check(counts, 3, N, K, sum(counts) + K)


# More than 64 rows a group and more small tiles than SMs: tiles of 256 x 256, in one or several waves, of an even and odd
# number of K blocks, the last features and rows of each in all places.
@pytest.mark.parametrize("counts,spare", [([300, 1, 0, 700, 31], 7), ([129, 0, 255, 256, 257, 640, 33, 31], 0), ([1000, 1500, 500], 45),
                                          ([2000], 0)])
@pytest.mark.parametrize("N,K", [(1424, 48), (1424, 272), (2064, 400), (2304, 640), (272, 1424), (1552, 16), (400, 2064)])
def test_large_tiles(counts, spare, N, K):
    out, dx = _check(counts, spare, N, K, sum(counts) + N + K)
    again = _check(counts, spare, N, K, sum(counts) + N + K)
    assert torch.equal(out, again[0]) and torch.equal(dx, again[1])


@pytest.mark.parametrize("counts,spare", [([5, 9, 0, 2], 77), ([0, 0], 40), ([700, 20], 1), ([3] * 40, 5), ([0] * 7, 9)])
def test_spare_rows_are_zero(counts, spare):
    _check(counts, spare, 144, 208, 3)


def test_many_experts():
    r = np.random.default_rng(1)
    _check([int(c) for c in r.integers(0, 5, 1024)], 3, 32, 48)
    _check([int(c) for c in r.multinomial(3000, r.dirichlet([0.3] * 64))], 0, 384, 256)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (1, 512, 1024), (31, 272, 144), (64, 1024, 2048), (200, 128, 128), (513, 384, 656),
                                   (2048, 1024, 512), (12001, 16, 144), (144, 12016, 48), (10000, 48, 272)])
def test_dense_products(M, N, K):
    x, dout, w, offs = _case([M], 0, N, K, M + N)
    out, dx = mx.fp8_block_mm(x, w, offs), mx.fp8_block_mm_dgrad(dout, w, offs)
    flat = mx.Fp8BlockWeight(w.codes[0], w.codes_t[0], w.scales[0])
    for ww in (w, flat):
        assert torch.equal(mx.fp8_block_mm(x, ww), out) and torch.equal(mx.fp8_block_mm_dgrad(dout, ww), dx)
    _check([M], 0, N, K, M + N)


def test_scales_of_very_different_size():
    """Neighbouring blocks 2^40 apart: the sums are of the largest block's size, the rest is kept as fp32 keeps it."""
    M, N, K = 40, 160, 640
    x = _bf16((M, K), 1)
    for b in range(5):
        x[:, b * 128:b * 128 + 128] *= 2.0 ** (20 * (b % 3) - 20)
    x[3:9] = 0
    q, w = mx.fp8_block_quantize(x.cuda()), mx.fp8_block_quantize_weight(_bf16((N, K), 2).cuda())
    X, W = _row_values(q), _weight_values(w)[0]
    _close(mx.fp8_block_mm(q, w), X @ W.t(), X.abs() @ W.abs().t(), K)


@pytest.mark.parametrize("counts,N,K", [([40, 23, 50], 272, 336), ([200, 300, 90], 272, 336), ([3, 5, 2], 272, 336),
                                        ([700, 500, 290], 1424, 336), ([700, 500, 290], 336, 1424)])
def test_other_groups_and_spare_rows_do_not_leak(counts, N, K):
    x, dout, w, offs = _case(counts, 30, N, K, 5)
    clean = mx.fp8_block_mm(x, w, offs), mx.fp8_block_mm_dgrad(dout, w, offs)
    a, b = offs[0].item(), offs[1].item()
    for t in (x, dout):
        for rows in (slice(a, b), slice(offs[2].item(), None)):
            t.codes[rows], t.scales[:, rows] = 0x7F, float("nan")
    out, dx = mx.fp8_block_mm(x, w, offs), mx.fp8_block_mm_dgrad(dout, w, offs)
    keep = [i for i in range(out.shape[0]) if not a <= i < b]
    assert torch.equal(out[keep], clean[0][keep]) and torch.equal(dx[keep], clean[1][keep])
    assert torch.isnan(out[a:b]).all() and torch.isnan(dx[a:b]).all()


@pytest.mark.parametrize("ends", [[10, 5, 60], [-1, 5, 60], [10, 20, 65], [70, 70, 70]])
def test_bad_offsets_are_reported_and_give_zeros(ends):
    x, dout, w, _ = _case([20, 20, 24], 0, 64, 128, 1)
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    for call in (lambda e: mx.fp8_block_mm(x, w, offs, err=e), lambda e: mx.fp8_block_mm_dgrad(dout, w, offs, err=e)):
        err = mx.ErrorWord()
        c = call(err)
        torch.cuda.synchronize()
        assert err.value() == 8 and not c.any()


def test_repeatable_and_on_another_stream():
    x, dout, w, offs = _case([100, 0, 33, 420, 1], 11, 528, 400, 2)
    once = lambda: (mx.fp8_block_mm(x, w, offs), mx.fp8_block_mm_dgrad(dout, w, offs))  # noqa: E731
    a = once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = once()
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_no_rows():
    w = mx.fp8_block_quantize_weight(_bf16((3, 64, 128), 1).cuda())
    offs = torch.zeros(3, dtype=torch.int32, device="cuda")
    x, d = (mx.fp8_block_quantize(torch.empty((0, n), dtype=torch.bfloat16, device="cuda")) for n in (128, 64))
    assert mx.fp8_block_mm(x, w, offs).shape == (0, 64) and mx.fp8_block_mm_dgrad(d, w, offs).shape == (0, 128)


def test_refuses_tensors_it_cannot_take():
    x, dout, w, offs = _case([5, 9], 0, 64, 128, 1)
    t = _bf16((4, 64), 1).cuda()
    src = torch.zeros(4, dtype=torch.int32, device="cuda")
    bad = [lambda: mx.fp8_block_quantize(t.float()), lambda: mx.fp8_block_quantize(t[:, :56].contiguous()),
           lambda: mx.fp8_block_quantize(t.t()), lambda: mx.fp8_block_quantize(t, div=2), lambda: mx.fp8_block_quantize(t, src.long()),
           lambda: mx.fp8_block_quantize(t, src, div=0), lambda: mx.fp8_block_quantize_weight(t[:, :24].contiguous()),
           lambda: mx.fp8_block_quantize_weight(t[0]), lambda: mx.fp8_block_mm(x, w), lambda: mx.fp8_block_mm(x.codes, w, offs),
           lambda: mx.fp8_block_mm(x, w.codes, offs), lambda: mx.fp8_block_mm(dout, w, offs), lambda: mx.fp8_block_mm_dgrad(x, w, offs),
           lambda: mx.fp8_block_mm(x, w, offs[:1]), lambda: mx.fp8_block_mm(x, w, offs.long()), lambda: mx.fp8_block_mm(x, w, offs.cpu()),
           lambda: mx.fp8_block_mm(mx.Fp8Block(x.codes, x.scales.t().contiguous()), w, offs),
           lambda: mx.fp8_block_mm(mx.Fp8Block(x.codes, x.scales.bfloat16()), w, offs),
           lambda: mx.fp8_block_mm(x, mx.Fp8BlockWeight(w.codes, None, w.scales[:1]), offs),
           lambda: mx.fp8_block_mm_dgrad(dout, mx.Fp8BlockWeight(w.codes, None, w.scales), offs)]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()
