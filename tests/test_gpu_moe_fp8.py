"""Routing, grouping, combining and FP8 products together, as a layer uses them: against 64-bit autograd of the layer
without any rounding, in a CUDA graph, and from several threads.

What the roundings come to, normwise: E4M3 codes with a scale for 128 elements 2.6% of an operand, 3.7% of a product of two
of them, up to three such products behind one another on a gradient: 8%.  bf16 values 0.2% and an 8-bit checkpoint 0.75%
beside them."""
import importlib.util
import os
import sys
import threading

import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("moe_fp8_layer", os.path.join(ROOT, "examples", "moe_fp8_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _bf16(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


@pytest.mark.parametrize("T,d,h,E,k", [(1, 64, 32, 4, 2), (77, 160, 96, 5, 3), (300, 384, 256, 9, 4), (64, 256, 128, 1, 1)])
def test_layer_against_autograd(T, d, h, E, k):
    ex = _example()
    p = ex.init_params(d, h, E, seed=3)
    p["bias"] += 0.05 * torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda()
    if E > 4:
        p["bias"][E - 1] = -float("inf")                    # an expert without tokens
    x, residual, dout = _bf16((T, d), 1), _bf16((T, d), 2), _bf16((T, d), 4)
    q = ex.quantise_params(p)
    out, s = ex.forward(p, q, x, residual, k)
    dx, grads = ex.backward(p, q, s, dout)

    r = {n: t.double().requires_grad_() for n, t in p.items()}
    xx = x.double().requires_grad_()
    score = torch.sigmoid(xx @ r["router"].t()).gather(1, s["ids"].long())
    weights = ex.SCALE * score / score.sum(1, keepdim=True)
    ref, rows = residual.double(), []
    for j in range(k):
        e = s["ids"][:, j].long()
        g, u = torch.einsum("td,thd->th", xx, r["w13"][e]).chunk(2, 1)
        rows.append(torch.einsum("th,tdh->td", g * torch.sigmoid(g) * u, r["w2"][e]))
        ref = ref + weights[:, j, None] * rows[j]
    (ref * dout.double()).sum().backward()
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert rel(out, ref.detach()) < 0.08 and rel(s["weights"], weights.detach()) < 1e-5
    assert rel(dx, xx.grad) < 0.08 and rel(grads["w13"], r["w13"].grad) < 0.08 and rel(grads["w2"], r["w2"].grad) < 0.08
    # A weight's gradient dout . row is off by |dout| times a row's error, 8% of |row|; the logits' gradients are differences of
    # them: dl = scale (dw - sum dw s / t) / t s (1 - s), off by no more than the same with errors added up.
    with torch.no_grad():
        off = 0.08 * dout.double().norm(dim=1, keepdim=True) * torch.stack([row.norm(dim=1) for row in rows], 1)
        t = score.sum(1, keepdim=True)
        dl = ex.SCALE * (off + (off * score).sum(1, keepdim=True) / t) / t * score * (1 - score)
        dl = torch.zeros((T, E), dtype=torch.float64, device="cuda").scatter_(1, s["ids"].long(), dl)
        assert ((grads["router"].double() - r["router"].grad).abs() <= dl.t() @ x.double().abs() + 1e-6).all()
    if E > 4:
        assert not grads["w13"][E - 1].any() and not grads["w2"][E - 1].any()


def test_example_runs(capsys, monkeypatch):
    ex = _example()
    monkeypatch.setattr("sys.argv", ["moe_fp8_layer.py", "--tokens", "200", "--d", "256", "--h", "128", "--experts", "6", "--topk",
                                     "2", "--steps", "2"])
    ex.main()
    assert "ms a step" in capsys.readouterr().out


def _step(ex, p, x, residual, dout, k):
    q = ex.quantise_params(p)
    out, s = ex.forward(p, q, x, residual, k)
    dx, grads = ex.backward(p, q, s, dout)
    return [out, s["ids"], s["weights"], s["offs"], s["dst"], s["src"], s["rows"], dx, *grads.values()]


@pytest.mark.parametrize("T", [3, 200])
def test_capture_and_replay(T):
    ex = _example()
    d, h, E, k = 192, 96, 5, 2
    p = ex.init_params(d, h, E, seed=0)
    x, residual, dout = (torch.empty((T, d), dtype=torch.bfloat16, device="cuda") for _ in range(3))

    def fill(seed):
        for i, t in enumerate((x, residual, dout, p["w13"], p["w2"], p["bias"])):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(10 * seed + i)) * 0.3)

    fill(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(ex, p, x, residual, dout, k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = _step(ex, p, x, residual, dout, k)
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2):
        fill(seed)
        graph.replay()
        torch.cuda.synchronize()
        want = _step(ex, p, x, residual, dout, k)
        assert all(torch.equal(a, b) for a, b in zip(captured, want))


def test_two_graphs_at_once():
    """Two captured steps replayed on two streams at the same time: each has its own workspaces."""
    ex = _example()
    d, h, E, k = 256, 128, 16, 8
    graphs = []
    for i in range(2):
        p = ex.init_params(d, h, E, seed=i)
        a = [_bf16((1500, d), 3 * i + j) for j in range(3)]
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            want = _step(ex, p, *a, k)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                got = _step(ex, p, *a, k)
        graphs.append((g, s, got, want, (p, a)))
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s, *_ in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_calls_from_several_threads():
    """Several tile shapes and layouts at once, each of which asks the device once what it holds."""
    calls = []
    for i, (T, E, k, d, n) in enumerate([(5, 8, 2, 256, 7168), (2000, 300, 6, 528, 64), (700, 3, 1, 144, 2048), (9000, 64, 4, 128, 256)]):
        l, x = torch.randn((T, E), generator=torch.Generator().manual_seed(i)).cuda(), _bf16((T, d), i)
        w = mx.fp8_block_quantize_weight(_bf16((E, n, d), 9 + i))

        def call(l=l, x=x, w=w, E=E, k=k):
            ids, weights = mx.moe_route(l, k, score=mx.SCORE_SIGMOID, bias=l[0])
            offs, dst, src = mx.token_group(ids, E)
            rows = mx.fp8_block_mm(mx.fp8_block_quantize(x, src, k), w, offs)
            out = mx.moe_combine(rows, dst, weights)
            return [ids, weights, offs, dst, src, rows, out, *mx.moe_combine_bwd(out, rows, dst, src, weights)]

        calls.append(call)
    torch.cuda.synchronize()
    failed, got, old = [], [None] * len(calls), sys.getswitchinterval()
    sys.setswitchinterval(1e-5)

    def work(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(50):
                try:
                    got[i] = calls[i]()
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
        assert all(torch.equal(a, b) for a, b in zip(mine, call()))


def test_padded_layout():
    """The rows and gradients of the padded layout are those of the other, and its padding rows are zero."""
    T, k, d, E = 130, 3, 264, 7
    ids = mx.moe_route(torch.randn((T, E), generator=torch.Generator().manual_seed(2)).cuda(), k)[0]
    weights, y, dout = torch.rand((T, k), generator=torch.Generator().manual_seed(3)).cuda(), _bf16((T * k, d), 1), _bf16((T, d), 2)
    offs, dst, src = mx.token_group(ids, E)
    p_offs, p_dst, p_src = mx.token_group_pad(ids.view(-1), E)
    rows, p_rows = mx.gather_rows(y, src), mx.gather_rows(y, p_src)
    assert torch.equal(mx.moe_combine(rows, dst, weights), mx.moe_combine(p_rows, p_dst, weights))
    a, da = mx.moe_combine_bwd(dout, rows, dst, src, weights)
    b, db = mx.moe_combine_bwd(dout, p_rows, p_dst, p_src, weights)
    assert torch.equal(da, db) and torch.equal(a[dst.long()], b[p_dst.long()]) and not b[p_src < 0].any()


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 bytes and 2^31 elements: their last rows are those of the rows alone."""
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    R, cols = 70001, 32768
    tail = _bf16((3, cols), 1)
    x = torch.zeros((R, cols), dtype=torch.bfloat16, device="cuda")
    x[-3:] = tail
    q, want = mx.fp8_block_quantize(x), mx.fp8_block_quantize(tail)
    assert torch.equal(q.codes[-3:], want.codes) and torch.equal(q.scales[:, -3:], want.scales) and not q.codes[:-3].any()
    src = torch.tensor([R - 1, 0, R - 3], dtype=torch.int32, device="cuda")
    q2 = mx.fp8_block_quantize(x, src)
    assert torch.equal(q2.codes[0], want.codes[2]) and torch.equal(q2.codes[2], want.codes[0]) and not q2.codes[1].any()
    w = mx.fp8_block_quantize_weight(_bf16((128, cols), 2))
    out = mx.fp8_block_mm(q, w)
    # the products of few rows add in another order: two roundings to bf16 apart, 2^-8 each
    small = mx.fp8_block_mm(want, w)
    assert (out[-3:].double() - small.double()).norm() <= 2.0 ** -7 * small.double().norm() and not out[:-3].any()
    del q, q2, out
    dst = torch.arange(R, dtype=torch.int32, device="cuda").flip(0).contiguous()
    ones = torch.ones((R, 1), device="cuda")
    out = mx.moe_combine(x, dst, ones)
    assert torch.equal(out[:3], tail.flip(0)) and not out[3:].any()
    drows, dw = mx.moe_combine_bwd(out, x, dst, dst, ones)
    assert torch.equal(drows[-3:], tail) and not dw[3:].any() and (dw[:3] > 0).all()
    del x, out, drows
    wide = mx.fp8_block_quantize_weight(_bf16((32768, 128), 3))
    rows = torch.zeros((70001, 128), dtype=torch.bfloat16, device="cuda")
    rows[-3:] = tail[:, :128]
    out = mx.fp8_block_mm(mx.fp8_block_quantize(rows), wide)
    small = mx.fp8_block_mm(mx.fp8_block_quantize(tail[:, :128].contiguous()), wide)
    assert (out[-3:].double() - small.double()).norm() <= 2.0 ** -7 * small.double().norm() and not out[:-3].any()
