"""Measured cases of the operators of a mixture-of-experts layer around its products, and of products in block-scaled FP8:

route    a router's scores to expert numbers and weights (softmax or sigmoid, a bias for balance, groups of experts,
         renormalised), the routed rows grouped by expert without padding, and the gradient of the router's logits
combine  the experts' rows weighted and summed back to tokens, and the gradient of rows and weights
quant    E4M3 codes with one fp32 scale for 128 elements of a row (rows gathered by routing or not), and weights with one
         for each 128 x 128 block, as they lie and transposed
mm       matrix products of such operands, dense or grouped by expert: forward and input gradient

``run`` computes a case with elementary torch operations in 32 bits (in 64 which experts are the largest and which code
is next to a value), or, with ``own`` set, through block_scaled_mlp_gb300.  E4M3 codes are returned as torch's 8-bit floating type.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LEAST = 2.0 ** -100  # the smallest largest-of-a-block that a scale is made for


def listed():
    return [
        # 8 decoded tokens of a 64-expert layer: top-8, softmax, renormalised
        dict(name="route_token", op="route", tokens=8, experts=64, k=8, score="softmax", bias=False, groups=1, top_groups=1,
             renorm=True, scale=1.0, wide=False, train=False),
        # a ragged prefill through a 16-expert top-1 layer with sigmoid gates, router in fp32
        dict(name="route_prefill", op="route", tokens=1999, experts=16, k=1, score="sigmoid", bias=False, groups=1,
             top_groups=1, renorm=False, scale=1.0, wide=True, train=False),
        # a training step of a 64-expert layer: balance bias, 8 groups of which 4 are taken, forward and backward
        dict(name="route_train", op="route", tokens=16384, experts=64, k=8, score="sigmoid", bias=True, groups=8,
             top_groups=4, renorm=True, scale=2.5, wide=True, train=True),
        # the same 8 decoded tokens' rows back to tokens, on top of a shared expert's output
        dict(name="combine_token", op="combine", tokens=8, k=8, d=7168, weighted=True, add=True, train=False),
        # a small odd microbatch, forward and backward
        dict(name="combine_odd", op="combine", tokens=1021, k=2, d=1000, weighted=True, add=False, train=True),
        # the 64-expert layer at full size, forward and backward
        dict(name="combine_train", op="combine", tokens=16384, k=8, d=7168, weighted=True, add=True, train=True),
        # the tokens of a prefill, each to its 8 experts, quantised on the way
        dict(name="quant_gather", op="quant", tokens=4096, k=8, d=7168, weight=False),
        # w2 of a 16-expert layer after an optimizer step: codes for the forward pass and transposed ones for the backward
        dict(name="quant_weights", op="quant", experts=16, n=5120, d=8192, transposed=True, weight=True),
        # 8 decoded tokens, top-8 of 64 experts: each hit expert's weights are read for one or two rows
        dict(name="mm_decode", op="mm", rows=64, spare=0, experts=64, n=4096, k=7168, alpha=0.3, part="fwd"),
        # a small odd training step with spare rows behind the last group
        dict(name="mm_odd_step", op="mm", rows=2041, spare=39, experts=16, n=1424, k=1008, alpha=1.0, part="step"),
        # w2 of a dense FFN at 8192 tokens
        dict(name="mm_dense", op="mm", rows=8192, spare=0, experts=0, n=4096, k=14336, alpha=1.0, part="fwd"),
        # the 64-expert layer's w13 products at full size (16384 tokens, top-8)
        dict(name="mm_moe64_step", op="mm", rows=131072, spare=0, experts=64, n=4096, k=7168, alpha=0.3, part="step"),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))
    return max(lo, min(hi, int(v / step + (0.5 if step > 1 else 0)) * step))


def draw(rng):
    op = rng.choice(["route", "route", "combine", "quant", "mm", "mm"])
    if op == "route":
        size, groups = rng.choice([(8, 8), (32, 8), (6, 4), (10, 3), (0, 1), (0, 1)])
        experts = size * groups or _log(rng, 4, 256)
        top = rng.randint(1, groups)
        return dict(op=op, tokens=_log(rng, 1, 16384), experts=experts, k=rng.randint(1, min(8, top * (experts // groups))),
                    score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, top_groups=top,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), wide=rng.random() < 0.5, train=rng.random() < 0.5)
    if op == "combine":
        weighted = rng.random() < 0.8
        return dict(op=op, tokens=_log(rng, 1, 8192), k=rng.randint(1, 8), d=_log(rng, 512, 7168, 8), weighted=weighted,
                    add=rng.random() < 0.5, train=weighted and rng.random() < 0.6)
    if op == "quant":
        if rng.random() < 0.5:
            return dict(op=op, tokens=_log(rng, 1, 4096), k=rng.choice([0, 1, 2, 8]), d=_log(rng, 512, 8192, 16), weight=False)
        return dict(op=op, experts=rng.randint(1, 16), n=_log(rng, 512, 7168, 16), d=_log(rng, 512, 7168, 16),
                    transposed=rng.random() < 0.6, weight=True)
    return dict(op=op, rows=_log(rng, 1, 32768), spare=rng.choice([0, 0, 5, 100]), experts=rng.choice([0, 1, 8, 16, 43, 64]),
                n=_log(rng, 512, 7168, 16), k=_log(rng, 512, 7168, 16), alpha=rng.choice([0.3, 1.0, 10.0]),
                part=rng.choice(["fwd", "dgrad", "step"]))


# ---------------------------------------------------------------- inputs


def _counts(case):
    """Rows of each expert, from the case alone (a routing's skew by `alpha`); a dense product is one group of all rows."""
    if not case["experts"]:
        return np.array([case["rows"] + case["spare"]])
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


def _experts(g, tokens, experts, k):
    """k different experts a token [tokens, k], some experts far more popular than others."""
    taste = torch.randn(experts, generator=g, device=DEV)
    return (torch.randn((tokens, experts), generator=g, device=DEV) + taste).topk(k, 1).indices


def _order(ids):
    """Rows grouped by expert: (row of each routed row, routed row of each row), whole numbers in 32 bits."""
    src = torch.argsort(ids.reshape(-1), stable=True)
    dst = torch.empty_like(src)
    dst[src] = torch.arange(src.numel(), device=DEV)
    return dst.to(torch.int32), src.to(torch.int32)


def _codes(g, rows, cols, std=1.0):
    """E4M3 codes and scales [cols / 128, rows] of normal rows, made in slices."""
    codes = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    scales = torch.empty((-(-cols // 128), rows), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 27) // cols)
    for a in range(0, rows, step):
        q, s = _quantise(_normal(g, (min(step, rows - a), cols), std))
        codes[a:a + step], scales[:, a:a + step] = q.view(torch.uint8), s
    return codes, scales


def _weight_codes(g, experts, n, k):
    codes = torch.empty((experts, n, k), dtype=torch.uint8, device=DEV)
    scales = torch.empty((experts, -(-n // 128), -(-k // 128)), dtype=torch.float32, device=DEV)
    for e in range(experts):
        q, s = _quantise_weight(_normal(g, (1, n, k), 0.02))
        codes[e], scales[e] = q[0].view(torch.uint8), s[0]
    return codes, scales


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "route":
        T, E = case["tokens"], case["experts"]
        taste = torch.randn(E, generator=g, device=DEV) * 0.5
        logits = torch.randn((T, E), generator=g, device=DEV) * 1.5 + taste
        if T >= 64:  # zero padding rows: all scores alike
            logits[torch.randint(0, T, (T // 64,), generator=g, device=DEV)] = 0
        s["logits"] = logits if case["wide"] else logits.to(torch.bfloat16)
        # as an update by a fixed step leaves it, against the popular ones
        s["bias"] = torch.round(-taste * 20 + torch.randn(E, generator=g, device=DEV) * 3) * 1e-3 if case["bias"] else None
        if case["train"]:
            s["dweights"] = torch.randn((T, case["k"]), generator=g, device=DEV) * 1e-2
    elif op == "combine":
        T, k, d = case["tokens"], case["k"], case["d"]
        s["rows"] = _normal(g, (T * k, d))
        s["dst"], s["src"] = _order(_experts(g, T, 64, k))
        s["weights"] = torch.softmax(torch.randn((T, k), generator=g, device=DEV), 1) if case["weighted"] else None
        s["add"] = _normal(g, (T, d)) if case["add"] else None
        if case["train"]:
            s["dout"] = _normal(g, (T, d), 1e-2)
    elif op == "quant":
        if case["weight"]:
            s["w"] = _normal(g, (case["experts"], case["n"], case["d"]), 0.02)
        else:
            s["x"] = _activations(g, case["tokens"], case["d"])
            s["src"] = _order(_experts(g, case["tokens"], 64, case["k"]))[1] if case["k"] else None
    else:
        E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
        counts = np.random.default_rng(seed).permutation(_counts(case))
        s["counts"] = [int(c) for c in counts]  # the router's numbers, on the host as well
        s["offs"] = torch.tensor(np.cumsum(counts), dtype=torch.int32, device=DEV) if E else None
        if case["part"] != "dgrad":
            s["x"] = _codes(g, M, k)
        if case["part"] != "fwd":
            s["dout"] = _codes(g, M, n, 1e-2)
        s["w"] = _weight_codes(g, E or 1, n, k)
        if case["part"] != "fwd":
            s["w_t"] = s["w"][0].transpose(1, 2).contiguous()
    return s


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        size = 4 if case["wide"] else 2
        b = T * E * size + 4 * E * (1 + case["bias"]) + 8 * T * k + 8 * T * k  # logits, bias, ends; ids and weights; both maps
        if case["train"]:
            b += 2 * T * E * size + 8 * T * k
        return {"bytes": b, "flops": T * E * (10 + (10 if case["train"] else 0)) + T * k * E}
    if op == "combine":
        T, k, d = case["tokens"], case["k"], case["d"]
        b = 2 * T * k * d + 4 * T * k * (1 + case["weighted"]) + 2 * T * d * (1 + case["add"])
        if case["train"]:
            b += 4 * T * k * d + 2 * T * d + 16 * T * k
        return {"bytes": b, "flops": T * k * d * (2 + (3 if case["train"] else 0))}
    if op == "quant":
        if case["weight"]:
            a = case["experts"] * case["n"] * case["d"]
            blocks = case["experts"] * -(-case["n"] // 128) * -(-case["d"] // 128)
            return {"bytes": a * (4 if case["transposed"] else 3) + 4 * blocks, "flops": 3 * a}
        T, d, R = case["tokens"], case["d"], case["tokens"] * (case["k"] or 1)
        return {"bytes": 2 * T * d + R * d + 4 * R * -(-d // 128) + (4 * R if case["k"] else 0), "flops": 3 * R * d}
    E, n, k, M = case["experts"], case["n"], case["k"], case["rows"] + case["spare"]
    counts = _counts(case)
    hit, m = int((counts > 0).sum()), int(counts.sum())
    kb, nb = -(-k // 128), -(-n // 128)
    weights = hit * (n * k + 4 * nb * kb)
    fwd = m * (k + 4 * kb) + weights + 2 * M * n
    dgrad = m * (n + 4 * nb) + weights + 2 * M * k
    return {"bytes": {"fwd": fwd, "dgrad": dgrad, "step": fwd + dgrad}[case["part"]],
            "flops": 2 * m * n * k * (2 if case["part"] == "step" else 1)}


# ---------------------------------------------------------------- plain form


def _scores(case, l):
    """Scores of logits in 64 bits; an expert with a logit of -inf has none."""
    if case["score"] == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(1, keepdim=True).clamp_min(-1e300))
    z = e.sum(1, keepdim=True)
    return e / torch.where(z == 0, 1, z)


def _select(case, l, s, bias):
    """The k largest experts of each token, larger ones first, ties by number: scores with the bias, of the top groups."""
    T, E, G = l.shape[0], case["experts"], case["groups"]
    c = s if bias is None else s + bias.double()
    c = torch.where(l == -math.inf, -math.inf, c)
    order = torch.sort(l if bias is None else c, dim=1, descending=True, stable=True).indices
    if G > 1:
        group = c.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(group, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]
        taken = torch.zeros((T, G), dtype=torch.int8, device=DEV).scatter_(1, best, 1).repeat_interleave(E // G, 1)
        order = order.gather(1, torch.sort(taken.gather(1, order), dim=1, descending=True, stable=True).indices)
    return order[:, :case["k"]]


def _quantise(x):
    """E4M3 codes of the rows of x and fp32 scales [cols / 128, rows]: a block's largest is 448 scales.  In 64 bits: values
    half way between two codes are common (7 divides the largest's fraction)."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 128)).view(rows, -1, 128)
    amax = v.abs().amax(2).clamp_min(LEAST)
    q = (v * 448 / amax.unsqueeze(2)).to(torch.float8_e4m3fn).view(rows, -1)[:, :cols]
    return q.contiguous(), (amax / 448).float().t().contiguous()


def _quantise_weight(w):
    """E4M3 codes of w [E, n, k] and fp32 scales [E, n / 128, k / 128], one for each 128 x 128 block."""
    E, n, k = w.shape
    v = torch.nn.functional.pad(w.double(), (0, -k % 128, 0, -n % 128))
    v = v.view(E, v.shape[1] // 128, 128, v.shape[2] // 128, 128)
    amax = v.abs().amax((2, 4)).clamp_min(LEAST)
    q = (v * 448 / amax[:, :, None, :, None]).to(torch.float8_e4m3fn)
    return q.view(E, v.shape[1] * 128, -1)[:, :n, :k].contiguous(), (amax / 448).float()


def _values(codes, scales):
    """What codes [rows, cols] with scales [cols / 128, rows] stand for, in 32 bits."""
    return codes.view(torch.float8_e4m3fn).float() * scales.t().repeat_interleave(128, 1)[:, :codes.shape[1]]


def _weight_values(codes, scales):
    """What the codes [n, k] with scales [n / 128, k / 128] stand for, in 32 bits."""
    n, k = codes.shape
    s = scales.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return codes.view(torch.float8_e4m3fn).float() * s


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["k"]
        l = s["logits"].double()
        score = _scores(case, l)
        ids = _select(case, l, score, s["bias"])
        sel = score.gather(1, ids)
        total = sel.sum(1, keepdim=True) + 1e-20 if case["renorm"] else 1.0
        out = dict(ids=ids.to(torch.int32), weights=(case["scale"] * sel / total).float())
        flat = ids.reshape(-1)
        counts = torch.zeros(E, dtype=torch.int64, device=DEV).scatter_add_(0, flat, torch.ones_like(flat))
        out["offs"] = counts.cumsum(0).to(torch.int32)
        out["dst"], out["src"] = _order(flat)
        if case["train"]:
            score, sel = score.float(), sel.float()
            ds = case["scale"] * s["dweights"]
            if case["renorm"]:
                total = total.float()
                ds = (ds - (ds * sel).sum(1, keepdim=True) / total) / total
            ds = torch.zeros_like(score).scatter_(1, ids, ds)
            if case["score"] == "sigmoid":
                dl = ds * score * (1 - score)
            else:
                dl = score * (ds - (ds * score).sum(1, keepdim=True))
            out["dlogits"] = dl.to(s["logits"].dtype)
        return out
    if op == "combine":
        T, k, d = case["tokens"], case["k"], case["d"]
        rows = s["rows"][s["dst"].long()].view(T, k, d).float()
        w = s["weights"][..., None] if case["weighted"] else 1.0
        total = (rows * w).sum(1)
        if case["add"]:
            total = total + s["add"].float()
        out = dict(out=total.to(torch.bfloat16))
        if case["train"]:
            dout = s["dout"].float()[:, None]
            out["drows"] = (dout * w).view(T * k, d)[s["src"].long()].to(torch.bfloat16)
            out["dweights"] = (rows * dout).sum(2)
        return out
    if op == "quant":
        if case["weight"]:
            q, scales = _quantise_weight(s["w"])
            out = dict(q=q, s=scales)
            if case["transposed"]:
                out["q_t"] = q.view(torch.uint8).transpose(1, 2).contiguous().view(torch.float8_e4m3fn)
            return out
        x = s["x"] if s["src"] is None else s["x"][s["src"].long() // case["k"]]
        q, scales = _quantise(x)
        return dict(q=q, s=scales)
    out, a = {}, 0
    M, n, k, part = case["rows"] + case["spare"], case["n"], case["k"], case["part"]
    if part != "dgrad":
        out["out"] = torch.zeros((M, n), dtype=torch.bfloat16, device=DEV)
        x = _values(*s["x"])
    if part != "fwd":
        out["dx"] = torch.zeros((M, k), dtype=torch.bfloat16, device=DEV)
        dout = _values(*s["dout"])
    for e, c in enumerate(s["counts"]):  # groups of different sizes: one product each
        if c:
            w = _weight_values(s["w"][0][e], s["w"][1][e])
            if "out" in out:
                out["out"][a:a + c] = x[a:a + c] @ w.t()
            if "dx" in out:
                out["dx"][a:a + c] = dout[a:a + c] @ w
        a += c
    return out


# ---------------------------------------------------------------- through the framework


def _own(s):
    import block_scaled_mlp_gb300 as mx
    case = s["case"]
    op = case["op"]
    if op == "route":
        score = mx.SCORE_SOFTMAX if case["score"] == "softmax" else mx.SCORE_SIGMOID
        ids, weights = mx.moe_route(s["logits"], case["k"], score=score, bias=s["bias"], groups=case["groups"],
                                    top_groups=case["top_groups"], renorm=case["renorm"], scale=case["scale"])
        out = dict(ids=ids, weights=weights)
        out["offs"], out["dst"], out["src"] = mx.token_group(ids, case["experts"])
        if case["train"]:
            out["dlogits"] = mx.moe_route_bwd(s["dweights"], s["logits"], ids, score=score, renorm=case["renorm"],
                                              scale=case["scale"])
        return out
    if op == "combine":
        out = dict(out=mx.moe_combine(s["rows"], s["dst"], weights=s["weights"], k=case["k"], add=s["add"]))
        if case["train"]:
            out["drows"], out["dweights"] = mx.moe_combine_bwd(s["dout"], s["rows"], s["dst"], s["src"], s["weights"])
        return out
    if op == "quant":
        if case["weight"]:
            w = mx.fp8_block_quantize_weight(s["w"], transposed=case["transposed"])
            out = dict(q=w.codes.view(torch.float8_e4m3fn), s=w.scales)
            if case["transposed"]:
                out["q_t"] = w.codes_t.view(torch.float8_e4m3fn)
            return out
        x = mx.fp8_block_quantize(s["x"], src=s["src"], div=case["k"] or 1)
        return dict(q=x.codes.view(torch.float8_e4m3fn), s=x.scales)
    out, part = {}, case["part"]
    w = mx.Fp8BlockWeight(s["w"][0], s.get("w_t"), s["w"][1])
    if part != "dgrad":
        out["out"] = mx.fp8_block_mm(mx.Fp8Block(*s["x"]), w, s["offs"])
    if part != "fwd":
        out["dx"] = mx.fp8_block_mm_dgrad(mx.Fp8Block(*s["dout"]), w, s["offs"])
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- in 64 bits, from the definitions


def _e4m3(v):
    """The E4M3 value next to v (3 fraction bits, least exponent -6, largest 448), ties to even."""
    _, e = torch.frexp(v)
    ulp = torch.exp2((e - 1).clamp_min(-6).double() - 3)
    return (torch.round(v / ulp) * ulp).clamp(-448, 448)


def _exact_route(case, s):
    l = s["logits"].double()
    T, E, k = case["tokens"], case["experts"], case["k"]
    p = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, 1)
    key = l if s["bias"] is None else p + s["bias"].double()
    taken = torch.ones((T, E), dtype=torch.bool, device=DEV)
    if case["groups"] > 1:  # a group's value: its two largest added
        c = (p if s["bias"] is None else key).view(T, case["groups"], -1)
        first = c.amax(2)
        at = (c == first[..., None]).to(torch.int8).argmax(2, keepdim=True)
        value = first + (c.scatter(2, at, -math.inf).amax(2) if c.shape[2] > 1 else 0)
        i = torch.arange(case["groups"], device=DEV)
        ahead = (value[:, None, :] > value[:, :, None]) | ((value[:, None, :] == value[:, :, None]) & (i[None, :] < i[:, None]))
        taken = (ahead.sum(2) < case["top_groups"]).repeat_interleave(E // case["groups"], 1)
    ids, left = [], torch.where(taken, key, -math.inf)
    for _ in range(k):
        top = (left == left.amax(1, keepdim=True)).to(torch.int8).argmax(1)  # the first of the largest
        ids.append(top)
        left = left.scatter(1, top[:, None], -math.inf)
    ids = torch.stack(ids, 1)
    chosen = torch.gather(p, 1, ids)
    denominator = chosen.sum(1, keepdim=True) + 1e-20
    out = dict(ids=ids.to(torch.int32), weights=chosen * case["scale"] / (denominator if case["renorm"] else 1))
    onehot = torch.zeros(E, dtype=torch.int64, device=DEV)
    onehot.index_add_(0, ids.flatten(), torch.ones(T * k, dtype=torch.int64, device=DEV))
    out["offs"] = torch.cumsum(onehot, 0).to(torch.int32)
    order = torch.argsort(ids.flatten().long() * (T * k) + torch.arange(T * k, device=DEV))  # by expert, then by number
    out["src"] = order.to(torch.int32)
    out["dst"] = torch.argsort(order).to(torch.int32)
    if case["train"]:
        dw = s["dweights"].double() * case["scale"]
        if case["renorm"]:  # w = p / t: dp = dw / t - (sum dw p) / t^2
            dw = dw / denominator - (dw * chosen).sum(1, keepdim=True) / denominator ** 2
        dp = torch.zeros_like(p)
        dp.scatter_(1, ids, dw)
        if case["score"] == "sigmoid":
            out["dlogits"] = dp * torch.sigmoid(l) * torch.sigmoid(-l)
        else:
            out["dlogits"] = p * dp - p * torch.einsum("te,te->t", dp, p)[:, None]
    return out


def exact(case, seed):
    if case["op"] == "mm" and work(case)["flops"] > 8e12:
        return None  # too many products for the card's 64-bit rate
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "combine":
        T, k, d = case["tokens"], case["k"], case["d"]
        w = s["weights"].double() if case["weighted"] else torch.ones((T, k), dtype=torch.float64, device=DEV)
        dst = s["dst"].long().view(T, k)
        total = s["add"].double() if case["add"] else torch.zeros((T, d), dtype=torch.float64, device=DEV)
        out = dict(out=total)
        if case["train"]:
            out["drows"] = torch.empty((T * k, d), dtype=torch.float64, device=DEV)
            out["dweights"] = torch.empty((T, k), dtype=torch.float64, device=DEV)
        for j in range(k):
            r = s["rows"][dst[:, j]].double()
            total += r * w[:, j:j + 1]
            if case["train"]:
                out["drows"][dst[:, j]] = s["dout"].double() * w[:, j:j + 1]
                out["dweights"][:, j] = torch.linalg.vecdot(r, s["dout"].double())
        return out
    if case["op"] == "quant":
        if case["weight"]:
            E, n, d = s["w"].shape
            q = torch.empty((E, n, d), dtype=torch.float64, device=DEV)
            scales = torch.empty((E, -(-n // 128), -(-d // 128)), dtype=torch.float64, device=DEV)
            for i in range(scales.shape[1]):
                for j in range(scales.shape[2]):
                    at = (slice(None), slice(i * 128, i * 128 + 128), slice(j * 128, j * 128 + 128))
                    v = s["w"][at].double()
                    m = v.abs().flatten(1).amax(1).clamp_min(LEAST)
                    scales[:, i, j] = m / 448
                    q[at] = _e4m3(v * 448 / m[:, None, None])
            return dict(q=q, s=scales, q_t=q.transpose(1, 2)) if case["transposed"] else dict(q=q, s=scales)
        x = s["x"] if s["src"] is None else s["x"][torch.div(s["src"].long(), case["k"], rounding_mode="floor")]
        q = torch.empty(x.shape, dtype=torch.float64, device=DEV)
        scales = torch.empty((-(-x.shape[1] // 128), x.shape[0]), dtype=torch.float64, device=DEV)
        for b in range(scales.shape[0]):
            v = x[:, b * 128:b * 128 + 128].double()
            m = v.abs().amax(1).clamp_min(LEAST)
            scales[b] = m / 448
            q[:, b * 128:b * 128 + 128] = _e4m3(v * 448 / m[:, None])
        return dict(q=q, s=scales)
    ends = [0] + (s["offs"].tolist() if s["offs"] is not None else [case["rows"] + case["spare"]])
    n, k, M = case["n"], case["k"], ends[-1] if s["offs"] is None else case["rows"] + case["spare"]
    new = lambda cols: torch.zeros((M, cols), dtype=torch.float64, device=DEV)  # noqa: E731
    out = {}
    if case["part"] in ("fwd", "step"):
        out["out"] = new(n)
    if case["part"] in ("dgrad", "step"):
        out["dx"] = new(k)
    at_n, at_k = torch.arange(n, device=DEV) // 128, torch.arange(k, device=DEV) // 128
    for e in range(len(ends) - 1):
        rows = slice(ends[e], ends[e + 1])
        w = s["w"][0][e].view(torch.float8_e4m3fn).double() * s["w"][1][e].double()[at_n[:, None], at_k]
        if "out" in out:
            x = s["x"][0][rows].view(torch.float8_e4m3fn).double() * s["x"][1][:, rows].double().t()[:, at_k]
            out["out"][rows] = torch.mm(x, w.t())
        if "dx" in out:
            dout = s["dout"][0][rows].view(torch.float8_e4m3fn).double() * s["dout"][1][:, rows].double().t()[:, at_n]
            out["dx"][rows] = torch.mm(dout, w)
    return out
