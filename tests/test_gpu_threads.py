"""Calls of different sizes from several threads at once: none fails, and each result is that of the call alone."""
import sys
import threading

import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


def _flat(v):
    if isinstance(v, dict):
        return [t for x in v.values() for t in _flat(x)]
    if isinstance(v, mx.Ckpt8):
        return [v.codes, v.scales]
    if isinstance(v, (tuple, list)):
        return [t for x in v for t in _flat(x)]
    return [] if v is None else [v]


def _together(calls, rounds):
    """The calls at once, before any of them ran alone."""
    torch.cuda.synchronize()
    failed, got, old = [], [None] * len(calls), sys.getswitchinterval()
    sys.setswitchinterval(1e-5)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(rounds):
                try:
                    got[i] = _flat(calls[i]())
                except Exception as e:  # noqa: BLE001
                    failed.append((i, str(e)))
                    return
            s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    assert not failed, failed
    for call, mine in zip(calls, got):
        assert all(torch.equal(a, b) for a, b in zip(mine, _flat(call())))


def _bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_norm_into_columns_of_two_widths():
    calls = []
    for i, d in enumerate([64, 16384, 64, 16384]):
        x, w = _bf16((32, d), i), torch.ones(d, dtype=torch.bfloat16, device="cuda")
        calls.append(lambda x=x, w=w: mx.add_rmsnorm_fwd(x, w, axis=mx.BOTH))
    _together(calls, 2000)


@pytest.mark.parametrize("ckpt", [False, True])
def test_norm_backward_of_two_widths(ckpt):
    calls = []
    for i, d in enumerate([544, 16384, 544, 16384]):
        x, w, dy = _bf16((32, d), i), torch.ones(d, dtype=torch.bfloat16, device="cuda"), _bf16((32, d), 9 + i)
        f = mx.add_rmsnorm_fwd(x, w, ckpt=ckpt)
        kept = f["ckpt"] if ckpt else x
        calls.append(lambda w=w, dy=dy, kept=kept, n=f["rstd"]: mx.add_rmsnorm_bwd(dy, kept, n, w))
    _together(calls, 2000)


def test_ragged_products_of_several_shapes():
    """Several tile shapes, each of which asks the device once how many of its clusters it holds."""
    calls = []
    for i, (counts, N, K) in enumerate([([8], 512, 7168), ([100], 1024, 4096), ([300, 17], 264, 328), ([40] * 30, 1032, 264)]):
        offs = torch.tensor(counts, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        x, w = _bf16((sum(counts), K), i), _bf16((len(counts), N, K), i + 5)
        calls.append(lambda x=x, w=w, offs=offs: mx.ragged_mm(x, w, offs))
    _together(calls, 300)
