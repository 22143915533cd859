"""A pre-norm mixture-of-experts block, forward and backward, from the library's operators.

    r   = x + residual;  n = RMSNorm(r)
    out = shared_expert(n) + sum over the token's k experts of gate * expert(n)

The shared expert runs in MXFP8 on the codes that the norm writes (rows for its forward product, columns
for its weight gradient).  The routed experts run in bf16 on the groups as the router left them, with no padding rows.
For the backward pass r and both experts' [g | u] are kept in 8 bits; n and the activations are computed again from them.

    python examples/moe_block.py [--tokens 8192 --d 2048 --h 1024 --experts 32 --topk 4 --steps 20]

tokens, d and h are multiples of 128 (the MXFP8 products); the routed groups have any sizes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_mlp_gb300 as mx  # noqa: E402


def init_params(d, h, E, device="cuda", seed=0):
    """norm [d]; shared w13 [2h, d], w2 [d, h]; routed w13 [E, 2h, d], w2 [E, d, h]."""
    g = torch.Generator(device=device).manual_seed(seed)
    draw = lambda *s: (torch.randn(s, generator=g, device=device) * s[-1] ** -0.5).to(torch.bfloat16)  # noqa: E731
    return dict(norm=torch.ones(d, dtype=torch.bfloat16, device=device), w13s=draw(2 * h, d), w2s=draw(d, h),
                w13=draw(E, 2 * h, d), w2=draw(E, d, h))


def route(ids, E):
    """Expert-major order of the T*k routed rows: (offs [E], order, place), all int32 on the device; row i of the
    ordered list is routed row order[i], and routed row j is at place[j]."""
    flat = ids.reshape(-1)
    order = torch.argsort(flat, stable=True)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=order.device)
    counts = torch.zeros(E, dtype=torch.int64, device=ids.device).scatter_add_(0, flat, torch.ones_like(flat))
    return counts.cumsum(0).to(torch.int32), order.to(torch.int32), place.to(torch.int32)


def forward(p, x, residual, ids, gates, eps=1e-5):
    """(out [T, d], r [T, d], saved).  ids [T, k] int64 expert numbers, gates [T, k] bf16; T a multiple of 128."""
    T, d = x.shape
    E, k = p["w13"].shape[0], ids.shape[1]
    n = mx.add_rmsnorm_fwd(x, p["norm"], residual, eps=eps, axis=mx.BOTH, ckpt=True)
    # shared expert
    w13q, w2q = mx.quantize(p["w13s"]), mx.quantize(p["w2s"])
    h13 = mx.scaled_mm(n["q_row"], n["s_row"], w13q["q_row"], w13q["s_row"])
    y, shared_ck = mx.swiglu_ckpt8_fwd(h13)
    yq = mx.quantize(y, mx.ROW)
    shared = mx.scaled_mm(yq["q_row"], yq["s_row"], w2q["q_row"], w2q["s_row"])
    # routed experts
    offs, order, place = route(ids, E)
    rows = mx.gather_rows(n["y"], order, div=k)
    y, ck = mx.swiglu_ckpt8_fwd(mx.ragged_mm(rows, p["w13"], offs))
    routed = mx.gather_rows(mx.ragged_mm(y, p["w2"], offs), place).view(T, k, d)
    out = (shared.float() + (routed.float() * gates.float()[..., None]).sum(1)).to(torch.bfloat16)
    saved = dict(r=n["ckpt"], rstd=n["rstd"], n_col=(n["q_col"], n["s_col"]), w13q=w13q, w2q=w2q, shared=shared_ck, ck=ck,
                 offs=offs, order=order, place=place, gates=gates, eps=eps)
    return out, n["r"], saved


def backward(p, s, dout, dr):
    """Gradients of x (the residual's are the same) and of the parameters; dr is the gradient that reaches r later on."""
    T, d = dout.shape
    k = s["gates"].shape[1]
    # shared expert
    dq = mx.quantize(dout)
    dy = mx.scaled_mm(dq["q_row"], dq["s_row"], s["w2q"]["q_col"], s["w2q"]["s_col"])
    dh13, y = mx.swiglu_ckpt8_bwd(dy, s["shared"])
    yq, hq = mx.quantize(y, mx.COL), mx.quantize(dh13)
    dw2s = mx.scaled_mm(dq["q_col"], dq["s_col"], yq["q_col"], yq["s_col"])
    dw13s = mx.scaled_mm(hq["q_col"], hq["s_col"], *s["n_col"])
    dn = mx.scaled_mm(hq["q_row"], hq["s_row"], s["w13q"]["q_col"], s["w13q"]["s_col"]).float()
    # routed experts
    do = mx.gather_rows(dout, s["order"], div=k) * s["gates"].reshape(-1)[s["order"].long(), None]
    dh13, y = mx.swiglu_ckpt8_bwd(mx.ragged_mm_dgrad(do, p["w2"], s["offs"]), s["ck"])
    dw2 = mx.ragged_mm_wgrad(do, y, s["offs"])
    n = mx.add_rmsnorm_fwd(mx.ckpt8_load(s["r"]), p["norm"], eps=s["eps"])["y"]
    dw13 = mx.ragged_mm_wgrad(dh13, mx.gather_rows(n, s["order"], div=k), s["offs"])
    drows = mx.gather_rows(mx.ragged_mm_dgrad(dh13, p["w13"], s["offs"]), s["place"])
    dn += drows.view(T, k, d).float().sum(1)
    dx, dnorm = mx.add_rmsnorm_bwd(dn.to(torch.bfloat16), s["r"], s["rstd"], p["norm"], dres=dr)
    return dx, dict(norm=dnorm, w13s=dw13s, w2s=dw2s, w13=dw13, w2=dw2)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, v in (("tokens", 8192), ("d", 2048), ("h", 1024), ("experts", 32), ("topk", 4), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=v)
    a = ap.parse_args()
    g = torch.Generator(device="cuda").manual_seed(1)
    bf = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    p = init_params(a.d, a.h, a.experts)
    x, residual, dout, dr = (bf(a.tokens, a.d) for _ in range(4))
    scores = torch.randn((a.tokens, a.experts), generator=g, device="cuda")
    gates, ids = torch.softmax(scores, 1).topk(a.topk)
    gates = gates.to(torch.bfloat16)

    def step():
        out, r, saved = forward(p, x, residual, ids, gates)
        return saved, backward(p, saved, dout, dr)

    for _ in range(3):
        saved, _ = step()
    t0, t1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    t0.record()
    for _ in range(a.steps):
        step()
    t1.record()
    torch.cuda.synchronize()
    kept = sum(saved[k].nbytes() for k in ("r", "shared", "ck"))
    rows = a.tokens * (1 + a.topk)
    print(f"forward + backward: {t0.elapsed_time(t1) / a.steps:.3f} ms a step; checkpoints {kept / 2**20:.1f} MiB "
          f"({(a.tokens * a.d + rows * 3 * a.h) * 2 / 2**20:.1f} MiB for r, [g | u] and the activations in bf16)")


if __name__ == "__main__":
    main()
