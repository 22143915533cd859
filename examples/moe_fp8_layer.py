"""A routed mixture-of-experts layer with FP8 products, forward and backward, from the library's operators.

    logits = x . router^T;  ids, weights = the k experts of each token (sigmoid scores, a bias for balance, renormalised)
    out    = residual + sum over the token's k experts of weight * w2[e] . swiglu(w13[e] . x)

The experts' products run in FP8 with a scale for 128 elements, on the groups as the router left them: tokens are quantised
on their way to their groups.  Weight gradients run in bf16, [g | u] is kept in 8 bits for the backward pass, and the
balance bias moves by a fixed step against the experts' loads, outside of the gradients.

    python examples/moe_fp8_layer.py [--tokens 8192 --d 2048 --h 1024 --experts 32 --topk 4 --steps 20]

d and h are multiples of 32; tokens, experts and groups have any sizes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mlp_gb300 as mx  # noqa: E402

SCALE = 2.5


def init_params(d, h, E, device="cuda", seed=0):
    """router [E, d] fp32, bias [E] fp32; w13 [E, 2h, d], w2 [E, d, h] bf16."""
    g = torch.Generator(device=device).manual_seed(seed)
    draw = lambda *s: torch.randn(s, generator=g, device=device) * s[-1] ** -0.5  # noqa: E731
    return dict(router=draw(E, d), bias=torch.zeros(E, device=device), w13=draw(E, 2 * h, d).to(torch.bfloat16),
                w2=draw(E, d, h).to(torch.bfloat16))


def quantise_params(p):
    """The experts' weights in FP8, once for every optimizer step."""
    return dict(w13=mx.fp8_block_quantize_weight(p["w13"]), w2=mx.fp8_block_quantize_weight(p["w2"]))


def forward(p, q, x, residual, k):
    """(out [T, d], saved) from x, residual [T, d] bf16."""
    E = p["router"].shape[0]
    logits = x.float() @ p["router"].t()
    ids, weights = mx.moe_route(logits, k, score=mx.SCORE_SIGMOID, bias=p["bias"], scale=SCALE)
    offs, dst, src = mx.token_group(ids, E)
    h13 = mx.fp8_block_mm(mx.fp8_block_quantize(x, src, k), q["w13"], offs)
    y, ck = mx.swiglu_ckpt8_fwd(h13)
    rows = mx.fp8_block_mm(mx.fp8_block_quantize(y), q["w2"], offs)
    out = mx.moe_combine(rows, dst, weights, add=residual)
    return out, dict(x=x, logits=logits, ids=ids, weights=weights, offs=offs, dst=dst, src=src, ck=ck, rows=rows)


def backward(p, q, s, dout):
    """(dx, gradients): of x without the residual path, whose gradient is dout itself, and of the parameters."""
    k = s["weights"].shape[1]
    drows, dweights = mx.moe_combine_bwd(dout, s["rows"], s["dst"], s["src"], s["weights"])
    dy = mx.fp8_block_mm_dgrad(mx.fp8_block_quantize(drows), q["w2"], s["offs"])
    dh13, y = mx.swiglu_ckpt8_bwd(dy, s["ck"])
    dw2 = mx.ragged_mm_wgrad(drows, y, s["offs"])
    dw13 = mx.ragged_mm_wgrad(dh13, mx.gather_rows(s["x"], s["src"], div=k), s["offs"])
    dx = mx.moe_combine(mx.fp8_block_mm_dgrad(mx.fp8_block_quantize(dh13), q["w13"], s["offs"]), s["dst"], k=k)
    dlogits = mx.moe_route_bwd(dweights, s["logits"], s["ids"], score=mx.SCORE_SIGMOID, scale=SCALE)
    dx = (dx.float() + dlogits @ p["router"]).to(torch.bfloat16)
    return dx, dict(router=dlogits.t() @ s["x"].float(), w13=dw13, w2=dw2)


def balance(p, offs, step=1e-3):
    """The bias against the loads: down for experts with more rows than the mean, up for the others."""
    load = torch.diff(offs, prepend=offs.new_zeros(1)).float()
    p["bias"] += step * torch.sign(load.mean() - load)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, v in (("tokens", 8192), ("d", 2048), ("h", 1024), ("experts", 32), ("topk", 4), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=v)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    p = init_params(a.d, a.h, a.experts)
    x, residual, dout = (torch.randn((a.tokens, a.d), generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))

    def step():
        q = quantise_params(p)
        _, saved = forward(p, q, x, residual, a.topk)
        backward(p, q, saved, dout)
        balance(p, saved["offs"])
        return saved

    for _ in range(3):
        saved = step()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(a.steps):
        saved = step()
    t1.record()
    torch.cuda.synchronize()
    load = torch.diff(saved["offs"], prepend=saved["offs"].new_zeros(1)).float()
    print(f"forward + backward: {t0.elapsed_time(t1) / a.steps:.3f} ms a step; fullest expert {float(load.max() / load.mean()):.2f} "
          f"times the mean")


if __name__ == "__main__":
    main()
