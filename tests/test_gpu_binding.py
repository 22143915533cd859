"""The compiled binding: what it refuses besides wrong tensors, and that other
threads run while a call waits."""
import sys
import threading

import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


def _x():
    return torch.zeros((32, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("name", ["axis", "layout", "scale_mode"])
@pytest.mark.parametrize("value", [1 << 32, (1 << 32) + 1, -(1 << 40), 1 << 80, 1.0, None, "1"])
def test_refuses_whole_numbers_out_of_range(name, value):
    x, w = _x()
    with pytest.raises(mx.MxError):
        mx.add_rmsnorm_fwd(x, w, **{"axis": mx.BOTH, name: value})


def test_refuses_flags_without_a_truth_value():
    x, w = _x()
    two = torch.ones(2)
    dy = torch.zeros((32, 32), dtype=torch.bfloat16, device="cuda")
    ck = mx.ckpt8_save(x)
    for call in (lambda: mx.add_rmsnorm_fwd(x, w, y=two), lambda: mx.add_rmsnorm_fwd(x, w, ckpt=two),
                 lambda: mx.swiglu_ckpt8_bwd(dy, ck, y=two)):
        with pytest.raises(mx.MxError):
            call()


def test_refuses_an_error_word_elsewhere():
    x, w = _x()
    offs = torch.tensor([32], dtype=torch.int32, device="cuda")
    w3 = torch.zeros((1, 64, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mx.MxError):
        mx.ragged_mm(x, w3, offs, mx.ErrorWord("cpu"))
    mx.ragged_mm(x, w3, offs, mx.ErrorWord()).sum().item()


def test_calls_from_several_threads():
    """Each thread on its own stream: the results are those of one thread."""
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [torch.randn((257, 512), generator=g, device="cuda").bfloat16() for _ in range(4)]
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    want = [(mx.ckpt8_load(mx.ckpt8_save(x)), mx.add_rmsnorm_fwd(x, w)["y"]) for x in xs]
    torch.cuda.synchronize()
    bad, old = [], sys.getswitchinterval()
    sys.setswitchinterval(1e-5)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                got = (mx.ckpt8_load(mx.ckpt8_save(xs[i])), mx.add_rmsnorm_fwd(xs[i], w)["y"])
                s.synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(old)
    assert not bad
