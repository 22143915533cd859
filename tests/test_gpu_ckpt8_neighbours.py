"""A block that holds a NaN or an infinity spoils only itself: every other block's checkpoint codes and scales are bit
for bit those of the clean input, whichever block the kernels work on together with the spoilt one."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu
BAD = [float("nan"), float("inf"), float("-inf")]


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16)


def _same_elsewhere(got, want, bad):
    """bad [rows, cols / 32]: the spoilt blocks."""
    rows, cols = want.codes.shape
    assert torch.equal(got.scales.cpu() == 255, bad)
    assert torch.equal(got.scales.cpu()[~bad], want.scales.cpu()[~bad])
    a, b = (t.codes.cpu().view(rows, cols // 32, 32)[~bad] for t in (got, want))
    assert torch.equal(a, b), f"{int((a != b).sum())} of {a.numel()} codes"
    assert torch.isnan(mx.ckpt8_load(got).cpu().view(rows, cols // 32, 32)[bad]).all()


def _spoil(x, every, first, seed):
    """Blocks first, first + every, ... of x each get one bad value."""
    b = x.view(-1, 32)
    bad = torch.zeros(b.shape[0], dtype=torch.bool)
    bad[first::every] = True
    at = torch.nonzero(bad).flatten()
    col = torch.randint(0, 32, at.shape, generator=torch.Generator().manual_seed(seed))
    for i, v in enumerate(BAD):
        b[at[i::3], col[i::3]] = v
    return bad.view(x.shape[0], -1)


@pytest.mark.parametrize("every,first", [(2, 0), (2, 1), (7, 3), (1000, 0), (1000, 64), (128, 5)])
@pytest.mark.parametrize("rows,cols", [(257, 544), (8, 4096), (70, 64)])
def test_save(rows, cols, every, first):
    x = _bf16((rows, cols), rows + cols)
    want = mx.ckpt8_save(x.cuda())
    bad = _spoil(x, every, first, 1)
    _same_elsewhere(mx.ckpt8_save(x.cuda()), want, bad)


@pytest.mark.parametrize("half", ["g", "u"])
@pytest.mark.parametrize("M,h", [(3, 64), (65, 544), (9, 4096)])
def test_swiglu(M, h, half):
    """g and u of the same columns are one pair."""
    h13 = _bf16((M, 2 * h), M + h, 1.5)
    y0, want = mx.swiglu_ckpt8_fwd(h13.cuda())
    part = (h13[:, :h] if half == "g" else h13[:, h:]).contiguous()
    bad = torch.zeros((M, 2 * h // 32), dtype=torch.bool)
    blocks = _spoil(part, 3, 1, 2)
    if half == "g":
        h13[:, :h], bad[:, :h // 32] = part, blocks
    else:
        h13[:, h:], bad[:, h // 32:] = part, blocks
    y, got = mx.swiglu_ckpt8_fwd(h13.cuda())
    _same_elsewhere(got, want, bad)
    fine = torch.isfinite(h13[:, :h]) & torch.isfinite(h13[:, h:])
    assert torch.equal(y.cpu()[fine], y0.cpu()[fine])


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,d", [(2, 544), (3, 4096), (2, 16384), (400, 256), (400, 1024), (400, 2048), (400, 9216)])
def test_norm_rows(M, d, residual):
    """Every form that holds a row: the pairs are vectors of one row."""
    x, res, w = _bf16((M, d), d), _bf16((M, d), d + 1) if residual else None, torch.ones(d, dtype=torch.bfloat16)
    call = lambda: mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda() if residual else None, ckpt=True)["ckpt"]  # noqa: E731
    want = call()
    bad = _spoil(x, 5, 2, 3)
    _same_elsewhere(call(), want, bad)


@pytest.mark.parametrize("d", [64, 544, 8192])
@pytest.mark.parametrize("row", [0, 1, 2, 3, 13, 30])
def test_norm_rows_and_columns(row, d):
    """One bad row of a row block; its pair is the row beside it."""
    M = 64
    x, w = _bf16((M, d), d), torch.ones(d, dtype=torch.bfloat16)
    call = lambda: mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), axis=mx.BOTH, ckpt=True)["ckpt"]  # noqa: E731
    want = call()
    bad = torch.zeros((M, d // 32), dtype=torch.bool)
    for b, v in zip(range(0, d // 32, 2), BAD * 100):
        x[row, b * 32 + b % 32] = v
        bad[row, b] = True
    _same_elsewhere(call(), want, bad)
