"""8-bit activation checkpoints, and SwiGLU with one, against 64-bit references.

Saving is exact arithmetic: codes and scales have to be the definition's, bit
for bit, and a loaded value is the code times a power of two.  SwiGLU results
are fp32 with an approximate exponential and reciprocal (relative error of
the sigmoid below 8 * 2^-24 for |g| <= 88 and of the whole chain below 32 *
2^-24 of the magnitudes involved), then rounded to bf16 (2^-8 of the value).
Below g = -88 the exponential overflows and the sigmoid is zero, an absolute
error of e^-88 of the factors.
"""
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64

pytestmark = pytest.mark.gpu
EF = 32 * 2.0 ** -24
TINY = 1e-36


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * std).to(torch.bfloat16)


def _spread(rows, cols, seed):
    """Blocks over the whole exponent range, zero blocks, subnormals, ties and block maxima at the scale rule's step."""
    x = torch.randn((rows, cols), generator=_gen(seed), dtype=torch.float64)
    x = x.view(rows, cols // 32, 32) * torch.exp2(torch.randint(-135, 125, (rows, cols // 32, 1), generator=_gen(seed + 1)).double())
    x = x.float().to(torch.bfloat16)
    n = rows * (cols // 32)
    b = x.view(n, 32)
    b[0::7] = 0
    k = torch.arange(n)[1::7]
    b[k] = (torch.arange(32).float() - 15.5).to(torch.bfloat16)      # ties: halves at scale 1 below
    b[k, 0] = 127.0
    k = torch.arange(n)[2::7]
    b[k, 3] = torch.tensor(1.984375 * 2.0 ** 20).to(torch.bfloat16)  # 127 * 2^14: no larger scale
    k = torch.arange(n)[3::7]
    b[k, 3] = torch.tensor(1.9921875 * 2.0 ** 20).to(torch.bfloat16)  # the next bf16 needs one
    return x.view(rows, cols)


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (257, 544), (64, 7168), (1000, 64)])
def test_save_and_load_are_the_definition(rows, cols):
    x = _spread(rows, cols, rows + cols)
    ck = mx.ckpt8_save(x.cuda())
    e = ref64.blocks_exp2(x.double(), 127.0)
    assert torch.equal(ck.scales.cpu().long(), (e + 127).long())
    code = torch.round(x.double() / torch.exp2(e.double()).repeat_interleave(32, 1))
    assert code.abs().max() <= 127
    assert torch.equal(ck.codes.cpu().double(), code)
    back = mx.ckpt8_load(ck)
    assert torch.equal(ref64.f64(back), ref64.int8_values(x.double()))
    assert ck.nbytes() == rows * cols + rows * cols // 32
    again = mx.ckpt8_save(back)                      # what a checkpoint holds it keeps
    assert torch.equal(mx.ckpt8_load(again), back)


def test_non_finite_blocks_load_as_nan():
    x = _bf16((4, 128), 3)
    x[0, 40], x[1, 3], x[2, 127] = float("nan"), float("inf"), float("-inf")
    ck = mx.ckpt8_save(x.cuda())
    bad = torch.zeros((4, 4), dtype=torch.bool)
    bad[0, 1] = bad[1, 0] = bad[2, 3] = True
    assert torch.equal(ck.scales.cpu() == 255, bad)
    back = mx.ckpt8_load(ck).cpu().view(4, 4, 32)
    assert torch.isnan(back[bad]).all() and torch.isfinite(back[~bad]).all()


def _h13(M, h, seed):
    h13 = _bf16((M, 2 * h), seed, 1.5)
    h13[:, 3::37] *= 40                              # gates far out on both sides
    if M > 2:
        h13[M // 2] = 0
    return h13


@pytest.mark.parametrize("M,h", [(1, 32), (1, 2048), (3, 96), (333, 544), (65, 7168)])
def test_swiglu(M, h):
    h13, dy = _h13(M, h, M + h), _bf16((M, h), 7, 0.01)
    y, ck = mx.swiglu_ckpt8_fwd(h13.cuda())
    g, u = h13[:, :h].double(), h13[:, h:].double()
    ref = ref64.silu(g) * u
    assert torch.all((ref64.f64(y) - ref).abs() <= ref.abs() * (2.0 ** -8 + EF) + (g * u).abs() * TINY + 1e-40)
    alone = mx.ckpt8_save(h13.cuda())
    assert torch.equal(ck.codes, alone.codes) and torch.equal(ck.scales, alone.scales)

    dh13, again = mx.swiglu_ckpt8_bwd(dy.cuda(), ck)
    kept = ref64.int8_values(h13.double())
    g, u, d = kept[:, :h], kept[:, h:], dy.double()
    s = torch.sigmoid(g)
    ref = g * s * u
    assert torch.all((ref64.f64(again) - ref).abs() <= ref.abs() * (2.0 ** -8 + EF) + (g * u).abs() * TINY + 1e-40)
    dg, du = d * u * s * (1 + g * (1 - s)), d * g * s
    mag = (d * u).abs() * s * (1 + g.abs() * (1 - s))
    tiny = (d * u).abs() * (1 + g.abs()) * TINY + 1e-40
    assert torch.all((ref64.f64(dh13)[:, :h] - dg).abs() <= dg.abs() * 2.0 ** -8 + mag * EF * 2 + tiny)
    assert torch.all((ref64.f64(dh13)[:, h:] - du).abs() <= du.abs() * (2.0 ** -8 + EF) + (d * g).abs() * TINY + 1e-40)
    only, none = mx.swiglu_ckpt8_bwd(dy.cuda(), ck, y=False)
    assert none is None and torch.equal(only, dh13)


def test_swiglu_backward_against_differences():
    M, h = 4, 64
    h13, dy = _bf16((M, 2 * h), 31, 1.5), _bf16((M, h), 32)
    _, ck = mx.swiglu_ckpt8_fwd(h13.cuda())
    dh13 = ref64.f64(mx.swiglu_ckpt8_bwd(dy.cuda(), ck)[0])
    at = ref64.f64(mx.ckpt8_load(ck))
    loss = lambda a: (dy.double() * ref64.silu(a[:, :h]) * a[:, h:]).sum()  # noqa: E731
    e = 1e-5
    for seed in range(5):
        v = torch.randn(at.shape, generator=_gen(seed), dtype=torch.float64)
        num = (loss(at + e * v) - loss(at - e * v)) / (2 * e)
        assert abs(num - (dh13 * v).sum()) <= (dh13 * v).abs().sum() * 2.0 ** -8 + 1e-6


def test_swiglu_non_finite_gradients_stay_in_their_block():
    h13, dy = _bf16((2, 128), 1), _bf16((2, 64), 2)
    h13[0, 5] = float("inf")
    _, ck = mx.swiglu_ckpt8_fwd(h13.cuda())
    dh13, y = mx.swiglu_ckpt8_bwd(dy.cuda(), ck)
    assert torch.isnan(y[0, :32]).all() and torch.isfinite(y[0, 32:]).all() and torch.isfinite(y[1]).all()
    assert torch.isfinite(dh13[1]).all()


def test_no_rows_and_another_stream():
    y, ck = mx.swiglu_ckpt8_fwd(torch.empty((0, 128), dtype=torch.bfloat16, device="cuda"))
    assert y.shape == (0, 64) and ck.codes.shape == (0, 128)
    dh13, y = mx.swiglu_ckpt8_bwd(y, ck)
    assert dh13.shape == (0, 128) and mx.ckpt8_load(ck).shape == (0, 128)
    h13, dy = _h13(65, 544, 3).cuda(), _bf16((65, 544), 4).cuda()
    want = mx.swiglu_ckpt8_bwd(dy, mx.swiglu_ckpt8_fwd(h13)[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mx.swiglu_ckpt8_bwd(dy, mx.swiglu_ckpt8_fwd(h13)[1])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_refuses_tensors_it_cannot_take():
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    ck = mx.ckpt8_save(x)
    bad = [lambda: mx.ckpt8_save(x.float()), lambda: mx.ckpt8_save(x.view(-1)), lambda: mx.ckpt8_save(x[:, :64]),
           lambda: mx.ckpt8_save(x.view(8, 64)[:, :48].contiguous()), lambda: mx.ckpt8_save(x.cpu()),
           lambda: mx.ckpt8_load(x), lambda: mx.swiglu_ckpt8_fwd(x.view(16, 32)),
           lambda: mx.swiglu_ckpt8_bwd(x, ck), lambda: mx.swiglu_ckpt8_bwd(x[:2, :64].contiguous(), ck),
           lambda: mx.ckpt8_load(mx.Ckpt8(ck.codes, ck.scales[:, :2].contiguous()))]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()
