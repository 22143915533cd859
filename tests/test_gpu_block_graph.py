"""The operators around the MLP in a CUDA graph: captured on one stream, replayed with new inputs in the same buffers,
bit for bit what the calls give outside."""
import pytest
import torch

import block_scaled_mlp_gb300 as mx

pytestmark = pytest.mark.gpu


def _step(t):
    f = mx.add_rmsnorm_fwd(t["x"], t["w"], t["res"], axis=mx.BOTH, ckpt=True)
    h13 = mx.ragged_mm(f["y"], t["w13"], t["offs"])
    y, ck = mx.swiglu_ckpt8_fwd(h13)
    out = mx.ragged_mm(y, t["w2"], t["offs"])
    dy = mx.ragged_mm_dgrad(t["dout"], t["w2"], t["offs"])
    dh13, y2 = mx.swiglu_ckpt8_bwd(dy, ck)
    dw2, dw13 = mx.ragged_mm_wgrad(t["dout"], y2, t["offs"]), mx.ragged_mm_wgrad(dh13, f["y"], t["offs"])
    dn = mx.ragged_mm_dgrad(dh13, t["w13"], t["offs"])
    dx, dw = mx.add_rmsnorm_bwd(dn, f["ckpt"], f["rstd"], t["w"], dres=t["dout"])
    return [f["q_row"], f["s_row"], f["q_col"], f["s_col"], out, dw2, dw13, dx, dw, mx.ckpt8_load(f["ckpt"])]


def _fill(t, seed):
    g = torch.Generator().manual_seed(seed)
    for k, v in t.items():
        if k == "offs":
            cuts = torch.sort(torch.randint(0, 193, (v.numel(),), generator=g)).values
            v.copy_(cuts.to(torch.int32))
        else:
            v.copy_((torch.randn(v.shape, generator=g) * 0.3).to(torch.bfloat16))


def test_capture_and_replay():
    M, d, h, E = 192, 256, 160, 5
    new = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    t = dict(x=new(M, d), res=new(M, d), dout=new(M, d), w=new(d), w13=new(E, 2 * h, d), w2=new(E, d, h),
             offs=torch.empty(E, dtype=torch.int32, device="cuda"))
    _fill(t, 0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _step(t)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            captured = _step(t)
    torch.cuda.current_stream().wait_stream(s)
    for seed in (1, 2):
        _fill(t, seed)
        graph.replay()
        torch.cuda.synchronize()
        want = _step(t)
        assert all(torch.equal(a, b) for a, b in zip(captured, want))
