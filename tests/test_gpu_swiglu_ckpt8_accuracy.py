"""The sigmoid of SwiGLU with a checkpoint within CUDA's documented bounds, for gates far out.

In units of 2^-24 of the value: e^-g by __expf 2 (2 + 1.173 |g|) (its bound is in units of the last place, 2^-23 at
most), the sum with 1 one, __fdividef four, and one for each of the two products that follow: 11 + 2.35 |g|.  The bf16
result adds half its step."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64

pytestmark = pytest.mark.gpu


def _within(got, ref, g):
    step = torch.exp2(torch.floor(torch.log2(ref.abs().clamp_min(2.0 ** -126))) - 7)
    off = (ref64.f64(got) - ref).abs() - step / 2
    assert torch.all(off <= ref.abs() * (11 + 2.35 * g.abs()) * 2.0 ** -24)


@pytest.mark.parametrize("lo,hi", [(-80, -40), (-40, -10), (-10, 0), (0, 10), (10, 80)])
def test_forward(lo, hi):
    M, h = 512, 2048
    gen = torch.Generator().manual_seed(hi)
    g = (torch.rand((M, h), generator=gen) * (hi - lo) + lo).to(torch.bfloat16)
    u = torch.randn((M, h), generator=gen).to(torch.bfloat16)
    y, _ = mx.swiglu_ckpt8_fwd(torch.cat([g, u], 1).cuda())
    _within(y, ref64.silu(g.double()) * u.double(), g.double())


@pytest.mark.parametrize("lo,hi", [(-80, -40), (-40, -10), (-10, 0), (0, 10), (10, 80)])
def test_backward(lo, hi):
    M, h = 512, 2048
    gen = torch.Generator().manual_seed(hi + 1)
    h13 = torch.cat([torch.rand((M, h), generator=gen) * (hi - lo) + lo, torch.randn((M, h), generator=gen)], 1)
    dy = torch.randn((M, h), generator=gen).to(torch.bfloat16)
    ck = mx.ckpt8_save(h13.to(torch.bfloat16).cuda())
    dh13, y = mx.swiglu_ckpt8_bwd(dy.cuda(), ck)
    at, d = ref64.f64(mx.ckpt8_load(ck)), dy.double()
    g, u = at[:, :h], at[:, h:]
    s = torch.sigmoid(g)
    _within(y, g * s * u, g)
    _within(dh13[:, h:], d * g * s, g)
