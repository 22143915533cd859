"""Norms whose result is an exact number: in rows of one magnitude a (or with zeros besides) y = r w n is w or 2 w up to
its sign, whatever a is, and codes, scales and bf16 values have to be that number's own, rounded once: a tie goes to
even, a maximum of 1.75 * 2^k keeps the smaller scale.  The reference's y is exact in 64 bits."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64

pytestmark = pytest.mark.gpu
MAGNITUDES = [1.0, 3.0, 0.5, 96.5, 2.0 ** -20, 7 * 2.0 ** 10, 1.9921875, 125.5 * 2.0 ** -30]


def _rows(M, d):
    """Rows of one magnitude and random signs; every second one with three zeros between its values."""
    g = torch.Generator().manual_seed(M + d)
    a = torch.tensor(MAGNITUDES, dtype=torch.float64)[torch.arange(M) % len(MAGNITUDES)]
    r = a[:, None] * (torch.randint(0, 2, (M, d), generator=g) * 2 - 1)
    sparse = torch.arange(M) // len(MAGNITUDES) % 2 == 1
    keep = torch.arange(d) % 4 == 1
    r[sparse] *= keep
    a = torch.where(sparse, a / 2, a)
    return r, a


def _weights(d):
    """Every significand of a bf16 number, over some powers of two; blocks whose largest is 1.75 and one step above."""
    j = torch.arange(d)
    w = (1 + (j * 37 % 128).double() / 128) * torch.exp2(-((j // 3) % 9).double())
    b = w.view(-1, 32)
    b[0::4] = b[0::4].clamp(max=1.75)
    b[0::4, 5] = 1.75
    b[1::4] = b[1::4].clamp(max=1.75)
    b[1::4, 9] = 1.7578125
    b[2::4] = 1.0625
    return w


def _bf16_of(y):
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -120))) - 7)
    return torch.round(y / step) * step


def _codes_of(y, floor):
    m = y.reshape(y.shape[0], -1, 32).abs().amax(-1)
    e = ref64.blocks_exp2(y, 448.0).double()
    if floor:
        e = torch.where(m == 0, -127.0, torch.floor(torch.log2(m.clamp_min(1e-300))) - 8)
    v = y / torch.exp2(e).repeat_interleave(32, 1)
    step = ref64.e4m3_step(v)
    return (torch.round(v / step) * step).clamp(-448, 448), (e + 127).to(torch.uint8)


@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("M,d,axis", [(1, 64, 1), (16, 544, 1), (16, 4096, 1), (16, 7168, 1), (2, 16384, 1), (400, 256, 1),
                                      (400, 1024, 1), (400, 4096, 1), (320, 12288, 1), (32, 64, 3), (64, 544, 3), (64, 7168, 3),
                                      (32, 16384, 3), (4096, 1024, 3)])
def test_exact_results(M, d, axis, floor):
    r, a = _rows(M, d)
    w = _weights(d)
    y = r * w / a[:, None]
    assert torch.equal((r * r).mean(1), a * a)
    x = r.to(torch.bfloat16)
    assert torch.equal(x.double(), r) and torch.equal(w.to(torch.bfloat16).double(), w)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.to(torch.bfloat16).cuda(), eps=0.0, axis=axis, layout=mx.SCALE_LINEAR,
                           scale_mode=mx.SCALE_FLOOR if floor else mx.SCALE_RCEIL)
    assert torch.equal(f["rstd"].cpu(), (1 / a).float())
    assert torch.equal(ref64.f64(f["y"]), _bf16_of(y))
    for bit, q, s, yy in ((1, "q_row", "s_row", y), (2, "q_col", "s_col", y.t().contiguous())):
        if axis & bit:
            code, byte = _codes_of(yy, floor)
            assert torch.equal(f[s].cpu().view(byte.shape), byte)
            assert torch.equal(f[q].cpu().view(torch.float8_e4m3fn).double(), code)


def test_residual_and_eps_that_complete_a_square():
    """mean r^2 = 3.5 and eps = 0.5: n is 1/2."""
    d, eps = 512, 0.5
    r = torch.tensor([0.0, 3.0, 2.0, 1.0], dtype=torch.float64).repeat(5, d // 4)
    assert torch.all((r * r).mean(1) + eps == 4.0)
    w = _weights(d)
    x = (r / 2).to(torch.bfloat16)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.to(torch.bfloat16).cuda(), x.cuda(), eps=eps, axis=mx.ROW, layout=mx.SCALE_LINEAR)
    y = r * w / 2
    code, byte = _codes_of(y, False)
    assert torch.equal(ref64.f64(f["y"]), _bf16_of(y))
    assert torch.equal(f["s_row"].cpu().view(byte.shape), byte)
    assert torch.equal(f["q_row"].cpu().view(torch.float8_e4m3fn).double(), code)
