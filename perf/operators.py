"""Measured cases of the operators around the MXFP8 MLP:

norm    residual addition + root-mean-square norm with the result in MXFP8 (and/or bf16), its
        backward pass, from the bf16 sum or from its 8-bit checkpoint
swiglu  SwiGLU that keeps [g | u] as an 8-bit checkpoint, and the backward pass from it
ckpt    the 8-bit checkpoint of a tensor by itself: saved and loaded
ragged  matrix products grouped by expert, group sizes not padded: forward, input gradient,
        weight gradient

``run`` computes a case with elementary torch operations in 32 bits, or, with ``own`` set, through
block_scaled_mlp_gb300.  E4M3 codes and E8M0 scales are returned as torch's 8-bit floating types
(the values that they stand for); an 8-bit checkpoint as the bf16 values that it loads as.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
EPS = 1e-5


def listed():
    return [
        # one decoded token of a d = 7168 MoE model: the norm before its MXFP8 projections
        dict(name="norm_token", op="norm", rows=1, d=7168, residual=True, y=False, axis="row", layout="mma", train=False,
             ckpt=False),
        # a ragged prefill: bf16 for the router and row codes for the projections
        dict(name="norm_prefill", op="norm", rows=1999, d=4096, residual=True, y=True, axis="row", layout="linear",
             train=False, ckpt=False),
        # the norm of a dense FFN block in training, first layer (no residual yet), bf16 result
        dict(name="norm_train_dense", op="norm", rows=8192, d=4096, residual=False, y=True, axis="none", layout="mma",
             train=True, ckpt=False),
        # the norm of a MoE block in training: row and column codes, the sum kept in 8 bits for the backward pass
        dict(name="norm_train_moe", op="norm", rows=16384, d=7168, residual=True, y=False, axis="both", layout="mma",
             train=True, ckpt=True),
        # a small odd microbatch through the experts' activation, forward and backward
        dict(name="swiglu_small", op="swiglu", rows=333, h=2048),
        # the activation of the Llama-3-8B FFN at 8192 tokens, forward and backward
        dict(name="swiglu_ffn", op="swiglu", rows=8192, h=14336),
        # a block's input kept in 8 bits and brought back
        dict(name="ckpt_small", op="ckpt", rows=257, d=5120),
        dict(name="ckpt_block", op="ckpt", rows=16384, d=7168),
        # 8 decoded tokens, top-8 of 64 experts: each hit expert's weights are read for one or two rows
        dict(name="ragged_decode", op="ragged", rows=64, spare=0, experts=64, n=4096, k=7168, alpha=0.3, part="fwd"),
        # a small odd training step with spare rows behind the last group
        dict(name="ragged_odd_step", op="ragged", rows=2041, spare=39, experts=16, n=1416, k=1000, alpha=1.0, part="step"),
        # a microbatch of the 16-expert layer, w2's products
        dict(name="ragged_moe16_step", op="ragged", rows=4096, spare=0, experts=16, n=5120, k=8192, alpha=3.0, part="step"),
        # the 64-expert layer's w13 products at full size (16384 tokens, top-8)
        dict(name="ragged_moe64_step", op="ragged", rows=131072, spare=0, experts=64, n=4096, k=7168, alpha=0.3,
             part="step"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    v = max(lo, min(hi, int(v / step + (0.5 if step > 1 else 0)) * step))
    return v if v != 3072 else v + step  # a width that no configuration here has


def draw(rng):
    op = rng.choice(["norm", "norm", "swiglu", "ckpt", "ragged", "ragged"])
    if op == "norm":
        axis = rng.choice(["none", "row", "both"])
        train = rng.random() < 0.5
        return dict(op=op, rows=_log(rng, 32, 16384, 32) if axis == "both" else _log(rng, 1, 16384), d=_log(rng, 512, 8192, 32),
                    residual=rng.random() < 0.7, y=axis == "none" or rng.random() < 0.3, axis=axis,
                    layout=rng.choice(["mma", "linear"]), train=train, ckpt=train and rng.random() < 0.5)
    if op == "swiglu":
        return dict(op=op, rows=_log(rng, 1, 8192), h=_log(rng, 512, 14336, 32))
    if op == "ckpt":
        return dict(op=op, rows=_log(rng, 1, 16384), d=_log(rng, 512, 7168, 32))
    return dict(op=op, rows=_log(rng, 1, 32768), spare=rng.choice([0, 0, 5, 100]), experts=_log(rng, 1, 64),
                n=_log(rng, 512, 7168, 8), k=_log(rng, 512, 7168, 8), alpha=rng.choice([0.3, 1.0, 10.0]),
                part=rng.choice(["fwd", "dgrad", "wgrad", "step"]))


# ---------------------------------------------------------------- inputs


def _counts(case):
    """Rows of each expert, from the case alone (a routing's skew by `alpha`)."""
    r = np.random.default_rng([case["rows"], case["experts"], case["n"], case["k"]])
    return r.multinomial(case["rows"], r.dirichlet([case["alpha"]] * case["experts"]))


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, std=1.0):
    """N(0, std^2) in bf16, drawn in slices so that a large tensor needs no second copy in 32 bits."""
    out = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    for part in out.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.numel(), generator=g, device=DEV).mul_(std))
    return out


def _activations(g, rows, d, std=1.0):
    """Activations of a transformer: normal, one channel in 256 twenty times larger, one row in 64 a zero padding row."""
    x = _normal(g, (rows, d), std)
    x[:, torch.randint(0, d, (max(1, d // 256),), generator=g, device=DEV)] *= 20
    if rows >= 64:
        x[torch.randint(0, rows, (rows // 64,), generator=g, device=DEV)] = 0
    return x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "norm":
        M, d = case["rows"], case["d"]
        s["x"] = _activations(g, M, d)
        s["res"] = _normal(g, (M, d), 2.0) if case["residual"] else None
        s["w"] = (torch.randn(d, generator=g, device=DEV) * 0.1 + 1).to(torch.bfloat16)
        if case["train"]:
            s["dy"] = _normal(g, (M, d), 1e-2)
            s["dres"] = _normal(g, (M, d), 1e-2) if case["residual"] else None
    elif op == "swiglu":
        s["h13"] = _activations(g, case["rows"], 2 * case["h"], 1.5)
        s["dy"] = _normal(g, (case["rows"], case["h"]), 1e-2)
    elif op == "ckpt":
        s["x"] = _activations(g, case["rows"], case["d"])
    else:
        E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
        counts = np.random.default_rng(seed).permutation(_counts(case))
        s["counts"] = [int(c) for c in counts]  # the router's numbers, on the host as well
        s["offs"] = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=DEV)
        if case["part"] != "dgrad":
            s["x"] = _normal(g, (M, k))
        if case["part"] != "fwd":
            s["dout"] = _normal(g, (M, n), 1e-2)
        if case["part"] != "wgrad":
            s["w"] = _normal(g, (E, n, k), 0.02)
    return s


def work(case):
    op = case["op"]
    if op == "norm":
        M, d = case["rows"], case["d"]
        a = M * d
        b = 2 * a + 2 * d + 4 * M + (4 * a if case["residual"] else 0)  # x, w, rstd; residual in, sum out
        b += (2 * a if case["y"] else 0) + {"none": 0, "row": 1, "both": 2}[case["axis"]] * (a + a // 32)
        if case["train"]:  # the kept sum written where it is one in 8 bits, and read again; dy, residual gradient, dx, dw
            b += (2 * (a + a // 32) if case["ckpt"] else 2 * a) + 4 * a + 4 * M + 4 * d + (2 * a if case["residual"] else 0)
        return {"bytes": b, "flops": a * (8 + (12 if case["train"] else 0))}
    if op == "swiglu":  # h13 in, y out, 8-bit h13 out and in again, dy in, dh13 and the recomputed y out
        a = case["rows"] * case["h"]
        return {"bytes": 4 * a + 2 * a + 2 * (2 * a + a // 16) + 2 * a + 4 * a + 2 * a, "flops": 30 * a}
    if op == "ckpt":
        a = case["rows"] * case["d"]
        return {"bytes": 2 * a + 2 * (a + a // 32) + 2 * a, "flops": 6 * a}
    E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
    hit = int((_counts(case) > 0).sum())
    m = case["rows"]
    fwd = 2 * (m * k + hit * n * k + M * n)
    dgrad = 2 * (m * n + hit * n * k + M * k)
    wgrad = 2 * (m * n + m * k + E * n * k)
    b = {"fwd": fwd, "dgrad": dgrad, "wgrad": wgrad, "step": fwd + dgrad + wgrad}[case["part"]]
    return {"bytes": b, "flops": 2 * m * n * k * (3 if case["part"] == "step" else 1)}


# ---------------------------------------------------------------- plain form


def _rceil(amax, bits, most):
    """Biased exponent byte of the smallest power of two 2^e with amax <= most * 2^bits * 2^e (most in [1, 2))."""
    man, e = torch.frexp(amax)
    e = e - 1 - bits + (man * 2 > most).to(torch.int32)
    e = torch.where(amax == 0, -127, e.clamp(-127, 127))
    return torch.where(torch.isfinite(amax), e + 127, 255)


def _tiled(scales):
    """[R, S] scale bytes in the block-scaled tensor core layout: 128 x 4 tiles of 512 bytes."""
    R, S = scales.shape
    rb, cb = -(-R // 128), -(-S // 4)
    full = torch.zeros((rb * 128, cb * 4), dtype=torch.uint8, device=scales.device)
    full[:R, :S] = scales
    return full.view(rb, 4, 32, cb, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _mx(y, layout):
    """E4M3 codes and E8M0 scales (RCEIL) of 32-element blocks along the rows of y (32 bits)."""
    rows, cols = y.shape
    blocks = y.reshape(rows, cols // 32, 32)
    e = _rceil(blocks.abs().amax(-1), 8, 1.75)
    q = torch.ldexp(blocks, (127 - e).unsqueeze(-1)).to(torch.float8_e4m3fn).reshape(rows, cols)
    s = e.to(torch.uint8)
    s = _tiled(s) if layout == "mma" else s.reshape(-1)
    return q, s.view(torch.float8_e8m0fnu)


def _int8(x):
    """The values that the 8-bit checkpoint of x (32 bits) holds: 32-element blocks, 8-bit whole numbers times 2^e."""
    rows, cols = x.shape
    blocks = x.reshape(rows, cols // 32, 32)
    e = _rceil(blocks.abs().amax(-1), 6, 127 / 64).unsqueeze(-1) - 127
    return torch.ldexp(torch.round(torch.ldexp(blocks, -e)), e).reshape(rows, cols)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        out = {}
        r = s["x"].float()
        if case["residual"]:
            out["r"] = (r + s["res"].float()).to(torch.bfloat16)
            r = out["r"].float()
        w = s["w"].float()
        out["rstd"] = rstd = torch.rsqrt((r * r).mean(-1) + EPS)
        y = r * rstd[:, None] * w
        if case["y"]:
            out["y"] = y.to(torch.bfloat16)
        if case["axis"] != "none":
            out["q_row"], out["s_row"] = _mx(y, case["layout"])
        if case["axis"] == "both":
            out["q_col"], out["s_col"] = _mx(y.t().contiguous(), case["layout"])
        if case["train"]:
            xhat = (_int8(r) if case["ckpt"] else r) * rstd[:, None]
            dy = s["dy"].float()
            gw = dy * w
            dx = rstd[:, None] * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
            if case["residual"]:
                dx = dx + s["dres"].float()
            out["dx"] = dx.to(torch.bfloat16)
            out["dw"] = (dy * xhat).sum(0).to(torch.bfloat16)
        return out
    if op == "swiglu":
        h = case["h"]
        h13 = s["h13"].float()
        g, u = h13[:, :h], h13[:, h:]
        y = g * u / (1 + torch.exp(-g))
        kept = _int8(h13)
        g, u, dy = kept[:, :h], kept[:, h:], s["dy"].float()
        sig = 1 / (1 + torch.exp(-g))
        dg = dy * u * sig * (1 + g * (1 - sig))
        du = dy * g * sig
        return dict(y=y.to(torch.bfloat16), dh13=torch.cat([dg, du], 1).to(torch.bfloat16),
                    y_again=(g * sig * u).to(torch.bfloat16))
    if op == "ckpt":
        return _int8(s["x"].float()).to(torch.bfloat16)
    out, part, a = {}, case["part"], 0
    E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
    if part in ("fwd", "step"):
        out["out"] = torch.zeros((M, n), dtype=torch.bfloat16, device=DEV)
    if part in ("dgrad", "step"):
        out["dx"] = torch.zeros((M, k), dtype=torch.bfloat16, device=DEV)
    if part in ("wgrad", "step"):
        out["dw"] = torch.zeros((E, n, k), dtype=torch.bfloat16, device=DEV)
    for e, c in enumerate(s["counts"]):  # groups of different sizes: one product each
        if c:
            w = s["w"][e].float() if "w" in s else None
            if "out" in out:
                out["out"][a:a + c] = s["x"][a:a + c].float() @ w.t()
            if "dx" in out:
                out["dx"][a:a + c] = s["dout"][a:a + c].float() @ w
            if "dw" in out:
                out["dw"][e] = s["dout"][a:a + c].float().t() @ s["x"][a:a + c].float()
        a += c
    return out


# ---------------------------------------------------------------- through the framework


def _own(s):
    import block_scaled_mlp_gb300 as mx
    case = s["case"]
    op = case["op"]
    if op == "norm":
        axis = {"none": 0, "row": mx.ROW, "both": mx.BOTH}[case["axis"]]
        layout = mx.SCALE_MMA if case["layout"] == "mma" else mx.SCALE_LINEAR
        f = mx.add_rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, y=case["y"], axis=axis, layout=layout,
                               ckpt=case["ckpt"])
        out = dict(rstd=f["rstd"])
        if case["residual"]:
            out["r"] = f["r"]
        if case["y"]:
            out["y"] = f["y"]
        if axis:
            out["q_row"], out["s_row"] = f["q_row"].view(torch.float8_e4m3fn), f["s_row"].view(torch.float8_e8m0fnu)
        if axis == mx.BOTH:
            out["q_col"], out["s_col"] = f["q_col"].view(torch.float8_e4m3fn), f["s_col"].view(torch.float8_e8m0fnu)
        if case["train"]:
            out["dx"], out["dw"] = mx.add_rmsnorm_bwd(s["dy"], f["ckpt"] if case["ckpt"] else f["r"], f["rstd"], s["w"],
                                                      dres=s["dres"])
        return out
    if op == "swiglu":
        y, kept = mx.swiglu_ckpt8_fwd(s["h13"])
        dh13, again = mx.swiglu_ckpt8_bwd(s["dy"], kept)
        return dict(y=y, dh13=dh13, y_again=again)
    if op == "ckpt":
        return mx.ckpt8_load(mx.ckpt8_save(s["x"]))
    out, part = {}, case["part"]
    if part in ("fwd", "step"):
        out["out"] = mx.ragged_mm(s["x"], s["w"], s["offs"])
    if part in ("dgrad", "step"):
        out["dx"] = mx.ragged_mm_dgrad(s["dout"], s["w"], s["offs"])
    if part in ("wgrad", "step"):
        out["dw"] = mx.ragged_mm_wgrad(s["dout"], s["x"], s["offs"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- in 64 bits, from the definitions


def _exp2_blocks(x, limit):
    """2^e of each 32-block of x, e the smallest (of -127 and up) with max|x| <= limit * 2^e; zero blocks: e = -127."""
    m = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(m, -127.0)
    nz = m > 0
    e[nz] = torch.ceil(torch.log2(m[nz] / limit)).clamp(-127, 127)
    e = torch.where(nz & (m > limit * torch.exp2(e)), e + 1, e)  # the logarithm may be a rounding off
    e = torch.where(nz & (e > -127) & (m <= limit * torch.exp2(e - 1)), e - 1, e)
    return torch.exp2(e)


def _exact_mx(y, layout):
    rows, cols = y.shape
    v = y.reshape(rows, cols // 32, 32)
    s = _exp2_blocks(v, 448.0)
    v = v / s
    ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)  # E4M3: 3 fraction bits, least exponent -6
    q = (torch.round(v / ulp) * ulp).clamp(-448, 448).reshape(rows, cols)
    s = s.reshape(rows, cols // 32)
    if layout == "mma":
        R, S = s.shape
        i = torch.arange(-(-R // 128) * 128, device=s.device)[:, None]
        j = torch.arange(-(-S // 4) * 4, device=s.device)[None, :]
        at = (i // 128 * -(-S // 4) + j // 4) * 512 + i % 32 * 16 + i % 128 // 32 * 4 + j % 4
        flat = torch.full((at.numel(),), 2.0 ** -127, dtype=torch.float64, device=s.device)
        flat[at[:R, :S].reshape(-1)] = s.reshape(-1)
        return q, flat
    return q, s.reshape(-1)


def _exact_int8(x):
    rows, cols = x.shape
    v = x.reshape(rows, cols // 32, 32)
    s = _exp2_blocks(v, 127.0)
    return (torch.round(v / s) * s).reshape(rows, cols)


def exact(case, seed):
    if case["op"] == "ragged" and work(case)["flops"] > 8e12:
        return None  # too many products for the card's 64-bit rate
    s = prepare(case, seed)
    wide = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() and v.numel() < 1 << 28 else v for k, v in s.items()}
    if case["op"] == "norm":
        out = {}
        r = wide["x"]
        if case["residual"]:
            r = (wide["x"] + wide["res"]).float().to(torch.bfloat16).double()  # the sum that the model carries on is bf16
            out["r"] = r
        inv = 1 / torch.sqrt(torch.sum(r ** 2, 1, keepdim=True) / case["d"] + EPS)
        out["rstd"] = inv[:, 0]
        y = wide["w"] * (r * inv)
        if case["y"]:
            out["y"] = y
        if case["axis"] in ("row", "both"):
            out["q_row"], out["s_row"] = _exact_mx(y, case["layout"])
        if case["axis"] == "both":
            out["q_col"], out["s_col"] = _exact_mx(y.t(), case["layout"])
        del y
        if case["train"]:
            kept = _exact_int8(r) if case["ckpt"] else r
            # y_j = w_j r_j n, n = (sum r^2 / d + eps)^-1/2: dr_i = w_i n dy_i - r_i n^3 / d sum_j dy_j w_j r_j
            dot = torch.sum(wide["dy"] * wide["w"] * kept, 1, keepdim=True)
            dx = wide["w"] * inv * wide["dy"] - kept * inv ** 3 * dot / case["d"]
            out["dx"] = dx + wide["dres"] if case["residual"] else dx
            out["dw"] = torch.sum(wide["dy"] * kept * inv, 0)
        return out
    if case["op"] == "swiglu":
        h = case["h"]
        h13 = wide["h13"]
        y = h13[:, :h] * torch.sigmoid(h13[:, :h]) * h13[:, h:]
        kept = _exact_int8(h13)
        g, u, dy = kept[:, :h], kept[:, h:], wide["dy"]
        p = torch.sigmoid(g)
        return dict(y=y, dh13=torch.cat([dy * u * (p + g * p * torch.sigmoid(-g)), dy * (g * p)], 1), y_again=g * p * u)
    if case["op"] == "ckpt":
        return _exact_int8(wide["x"])
    part, ends = case["part"], [0] + s["offs"].tolist()
    E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
    new = lambda *shape: torch.zeros(shape, dtype=torch.float64, device=DEV)  # noqa: E731
    out = {}
    if part != "dgrad" and part != "wgrad":
        out["out"] = new(M, n)
    if part in ("dgrad", "step"):
        out["dx"] = new(M, k)
    if part in ("wgrad", "step"):
        out["dw"] = new(E, n, k)
    for e in range(E):
        rows = slice(ends[e], ends[e + 1])
        if "out" in out:
            out["out"][rows] = torch.mm(s["x"][rows].double(), s["w"][e].double().t())
        if "dx" in out:
            out["dx"][rows] = torch.mm(s["dout"][rows].double(), s["w"][e].double())
        if "dw" in out:
            out["dw"][e] = torch.mm(s["dout"][rows].double().t(), s["x"][rows].double())
    return out
