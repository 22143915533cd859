"""Dense FP8 products of few rows whose contraction is one K block and whose tiles are more than the SMs: a CTA takes several
tiles, and its second scale warp none of the first.  Right behind the cast that writes the scales, their results are those
of the same calls with a wait for the GPU between them, bit for bit."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu
F = 32768


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=torch.Generator().manual_seed(seed)) * std).to(torch.bfloat16).cuda()


def _case(direction, M, C):
    """The rows' shape, and the product of a cast of them."""
    if direction == "forward":
        w = mx.fp8_block_quantize_weight(_bf16((F, C), 1, 0.05), transposed=False)
        return w, lambda x: mx.fp8_block_mm(mx.fp8_block_quantize(x), w)
    w = mx.fp8_block_quantize_weight(_bf16((C, F), 1, 0.05))
    return w, lambda x: mx.fp8_block_mm_dgrad(mx.fp8_block_quantize(x), w)


def _apart(direction, w, x):
    """The same with the GPU waited for between the cast and the product."""
    q = mx.fp8_block_quantize(x)
    torch.cuda.synchronize()
    out = (mx.fp8_block_mm if direction == "forward" else mx.fp8_block_mm_dgrad)(q, w)
    torch.cuda.synchronize()
    return out


# Scales a factor of 2^30 apart from one call to the next: one of the call before shows.
INPUTS = [2.0 ** 15, 2.0 ** -15, 1.0, 2.0 ** -30, 2.0 ** 30]


@pytest.mark.parametrize("direction", ["forward", "gradient"])
@pytest.mark.parametrize("M,C", [(3, 128), (64, 128), (64, 16), (33, 112)])
def test_captured_behind_the_cast(direction, M, C):
    w, product = _case(direction, M, C)
    x = _bf16((M, C), 2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        product(x)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = [product(x) for _ in range(4)]
    torch.cuda.current_stream().wait_stream(s)
    for i, size in enumerate(INPUTS):
        x.copy_(_bf16((M, C), 3 + i) * size)
        want = _apart(direction, w, x)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for out in captured)


@pytest.mark.parametrize("direction", ["forward", "gradient"])
def test_back_to_back(direction):
    w, product = _case(direction, 48, 128)
    x = [_bf16((48, 128), i) * INPUTS[i % len(INPUTS)] for i in range(20)]
    torch.cuda.synchronize()
    got = [product(t) for t in x]
    torch.cuda.synchronize()
    assert all(torch.equal(a, _apart(direction, w, t)) for a, t in zip(got, x))
