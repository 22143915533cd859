"""64-bit references of the operators around the MLP, for the tests: plain
torch in float64 on the host, from the definitions, one function per formula."""
import torch


def f64(t):
    return t.detach().cpu().double()


def blocks_exp2(x, limit):
    """2^e per 32-block of the rows of x: e the smallest, -127 and up, with max|x| <= limit * 2^e."""
    m = x.reshape(x.shape[0], -1, 32).abs().amax(-1)
    man, e = torch.frexp(m / limit)          # m / limit = man * 2^e, man in [0.5, 1)
    e = torch.where(man == 0.5, e - 1, e)    # exact powers of two need no larger scale
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(min=-127))
    return e


def int8_values(x):
    """What the 8-bit checkpoint of x holds."""
    s = torch.exp2(blocks_exp2(x, 127.0).double()).repeat_interleave(32, 1)
    return torch.round(x / s) * s


def e4m3_step(v):
    """Distance of neighbouring E4M3 values at |v| (v in units of the block's scale)."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)


def untile(scales, R, S):
    """MMA-layout scale bytes -> ([R, S], the padding bytes)."""
    rb, cb = -(-R // 128), -(-S // 4)
    full = scales.cpu().view(rb, cb, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rb * 128, cb * 4)
    live = torch.zeros_like(full, dtype=torch.bool)
    live[:R, :S] = True
    return full[:R, :S], full[~live]


def silu(g):
    return g * torch.sigmoid(g)


def rmsnorm(r, w, eps):
    n = 1 / torch.sqrt((r * r).mean(1) + eps)
    return r * n[:, None] * w, n


def rmsnorm_bwd(dy, r, n, w):
    """(dr, dw) and the sums of the magnitudes that went into each element."""
    n = n[:, None]
    g = dy * w
    c = (g * r).mean(1, keepdim=True) * n * n
    mag = n * (g.abs() + r.abs() * (g * r).abs().mean(1, keepdim=True) * n * n)
    t = dy * r * n
    return n * (g - r * c), t.sum(0), mag, t.abs().sum(0)
