"""add_rmsnorm_fwd / add_rmsnorm_bwd against 64-bit references.

Tolerances, from the arithmetic.  y is fp32: a sum of d squares added in a
tree at most 64 deep (relative error 64 * 2^-24, halved by the root), one
rounding each for n, r n and r n w: 40 * 2^-24 < EY = 2.5e-6 relative.  A code
is then within half an E4M3 step of y / scale, give or take EY; a scale byte
is exact unless the block's maximum is within EY of the step of the rule.
bf16 results add half a unit: 2^-8 of the value at most.  In the backward
pass the sums add up to 64 * 2^-24 = 2^-18 of the magnitudes involved, for dw
(rows per CTA + CTAs) * 2^-24 of them.
"""
import ctypes

import pytest
import torch

import block_scaled_mlp_gb300 as mx
from tests import ref64

pytestmark = pytest.mark.gpu
EY = 2.5e-6
EPS = 1e-5


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _bf16(shape, seed, std=1.0):
    return (torch.randn(shape, generator=_gen(seed)) * std).to(torch.bfloat16)


def _inputs(M, d, residual, seed):
    x = _bf16((M, d), seed)
    if d >= 64:
        x[:, 5::61] *= 30                       # outlier channels
    if M >= 3:
        x[M // 2] = 0
    res = _bf16((M, d), seed + 1, 2.0) if residual else None
    if residual and M >= 3:
        res[M // 2] = 0                         # a row of zeros: n = eps^-1/2
    w = (torch.randn(d, generator=_gen(seed + 2)) * 0.1 + 1).to(torch.bfloat16)
    return x, res, w


def _check_codes(q, s, y, floor=False, pad=None):
    """codes q [R, C] u8 and scale bytes s [R, C/32] against exact y [R, C]."""
    m = y.reshape(y.shape[0], -1, 32).abs().amax(-1)
    lo, hi = (ref64.blocks_exp2(y * f, 448.0) + 127 for f in (1 - EY, 1 + EY))
    if floor:
        lo, hi = (torch.where(m == 0, 0, (torch.floor(torch.log2(m.clamp_min(1e-300) * f)) - 8 + 127).clamp(min=0))
                  for f in (1 - EY, 1 + EY))
    s = s.cpu().double()
    assert torch.all((s >= lo) & (s <= hi))
    v = q.cpu().view(torch.float8_e4m3fn).double()
    t = y / torch.exp2(s - 127).repeat_interleave(32, 1)
    tol = ref64.e4m3_step(t) / 2 + t.abs() * EY + 1e-12
    tol = torch.where(t.abs() > 448, t.abs() - 448 + t.abs() * EY, tol)      # FLOOR saturates
    assert torch.all((v - t).abs() <= tol)


@pytest.mark.parametrize("floor", [False, True])
@pytest.mark.parametrize("layout", ["mma", "linear"])
@pytest.mark.parametrize("M,d,residual,axis", [(1, 32, True, 1), (1, 7168, True, 1), (5, 96, False, 1), (129, 544, True, 1),
                                               (33, 2080, True, 1), (2, 16384, True, 1), (3, 4096, False, 1),
                                               (32, 32, True, 3), (96, 544, True, 3), (160, 1056, False, 3),
                                               (32, 16384, True, 3), (64, 8192, True, 3), (64, 288, True, 2)])
def test_forward(M, d, residual, axis, layout, floor):
    x, res, w = _inputs(M, d, residual, M + d)
    lay = mx.SCALE_MMA if layout == "mma" else mx.SCALE_LINEAR
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), None if res is None else res.cuda(), eps=EPS, axis=axis, layout=lay,
                           scale_mode=mx.SCALE_FLOOR if floor else mx.SCALE_RCEIL, ckpt=True)
    r = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    assert torch.equal(f["r"].cpu(), r)
    y, n = ref64.rmsnorm(r.double(), w.double(), EPS)
    assert torch.all((ref64.f64(f["rstd"]) - n).abs() <= n * EY)
    assert torch.all((ref64.f64(f["y"]) - y).abs() <= y.abs() * (2.0 ** -8 + EY))
    for bit, q, s, yy in ((1, "q_row", "s_row", y), (2, "q_col", "s_col", y.t().contiguous())):
        if not axis & bit:
            assert f[q] is None and f[s] is None
            continue
        R, S = yy.shape[0], yy.shape[1] // 32
        if layout == "mma":
            s2, pad = ref64.untile(f[s], R, S)
            assert not pad.any()
        else:
            s2 = f[s].view(R, S)
        _check_codes(f[q], s2, yy, floor)
    assert torch.equal(ref64.f64(mx.ckpt8_load(f["ckpt"])), ref64.int8_values(r.double()))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("d,axis", [(8, 0), (32, 1), (200, 0), (256, 1), (512, 1), (520, 0), (544, 1), (1024, 1), (1032, 0),
                                    (1056, 1), (2080, 1), (4096, 1), (8192, 1), (8200, 0), (8224, 1), (16384, 1)])
def test_forward_of_many_rows(d, axis, residual):
    """More rows than two an SM: the forms that hold a row in a warp and in a CTA.  Padding reads zero in buffers
    that held something else."""
    M = 2 * 160 + 11
    x, res, w = _inputs(M, d, residual, 5 + d)
    P = lambda t: None if t is None else ctypes.c_void_p(t.data_ptr())  # noqa: E731
    r = x if res is None else (x.float() + res.float()).to(torch.bfloat16)
    xc, wc, rc = x.cuda(), w.cuda(), None if res is None else res.cuda()
    out_r, out_y, rstd = torch.empty_like(xc), torch.empty_like(xc), torch.empty(M, device="cuda")
    q = torch.full((M, d), 0xAB, dtype=torch.uint8, device="cuda")
    s = torch.full((mx.mma_scale_bytes(M, d) if axis else 1,), 0xAB, dtype=torch.uint8, device="cuda")
    ck, cs = torch.empty((M, d), dtype=torch.int8, device="cuda"), torch.empty((M, d // 32), dtype=torch.uint8, device="cuda")
    st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    assert mx.lib().mx_add_rmsnorm_fwd(P(xc), P(rc), P(wc), M, d, EPS, P(out_r) if residual else None, P(rstd), P(out_y), axis,
                                       1, 0, P(q) if axis else None, P(s) if axis else None, None, None,
                                       P(ck) if axis else None, P(cs) if axis else None, st) == 0
    y, n = ref64.rmsnorm(r.double(), w.double(), EPS)
    if residual:
        assert torch.equal(out_r.cpu(), r)
    assert torch.all((ref64.f64(rstd) - n).abs() <= n * EY)
    assert torch.all((ref64.f64(out_y) - y).abs() <= y.abs() * (2.0 ** -8 + EY))
    if axis:
        s2, pad = ref64.untile(s, M, d // 32)
        assert not pad.any()
        _check_codes(q, s2, y)
        assert torch.equal(ref64.f64(mx.ckpt8_load(mx.Ckpt8(ck, cs))), ref64.int8_values(r.double()))


@pytest.mark.parametrize("M,d", [(1, 8), (7, 40), (3, 1000), (2, 16376)])
def test_forward_widths_without_codes(M, d):
    x, res, w = _inputs(M, d, True, d)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    r = (x.float() + res.float()).to(torch.bfloat16)
    y, _ = ref64.rmsnorm(r.double(), w.double(), EPS)
    assert torch.equal(f["r"].cpu(), r)
    assert torch.all((ref64.f64(f["y"]) - y).abs() <= y.abs() * (2.0 ** -8 + EY))
    dy = _bf16((M, d), 3)
    dx, dw = mx.add_rmsnorm_bwd(dy.cuda(), f["r"], f["rstd"], w.cuda())
    _check_bwd(dx, dw, dy, r.double(), w, None)


def test_every_padding_byte_is_written():
    """Scale buffers that held something else before: the layout's padding reads zero afterwards."""
    M, d = 160, 544                                         # 2 x 128 rows, 17 scale columns of 20
    x, res, w = (t.cuda() for t in _inputs(M, d, True, 4))
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for axis in (1, 3):
        r, rstd = torch.empty_like(x), torch.empty(M, device="cuda")
        q = [torch.full((M * d,), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(2)]
        s = [torch.full((mx.mma_scale_bytes(*rc),), 0xAB, dtype=torch.uint8, device="cuda") for rc in ((M, d), (d, M))]
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert mx.lib().mx_add_rmsnorm_fwd(P(x), P(res), P(w), M, d, EPS, P(r), P(rstd), None, axis, 1, 0, P(q[0]), P(s[0]),
                                           P(q[1]), P(s[1]), None, None, st) == 0
        assert not ref64.untile(s[0], M, d // 32)[1].any()
        if axis == 3:
            assert not ref64.untile(s[1], d, M // 32)[1].any()
        else:
            assert torch.all(s[1] == 0xAB) and torch.all(q[1] == 0xAB)   # not asked for: not touched


def test_non_finite_rows_stay_in_their_row():
    M, d = 64, 256
    x, _, w = _inputs(M, d, False, 9)
    clean = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), axis=mx.BOTH, layout=mx.SCALE_LINEAR, ckpt=True)
    x[40, 7] = float("nan")
    x[41, 9] = float("inf")
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), axis=mx.BOTH, layout=mx.SCALE_LINEAR, ckpt=True)
    keep = [i for i in range(M) if i not in (40, 41)]
    for k in ("y", "q_row", "rstd"):
        assert torch.equal(f[k][keep], clean[k][keep])
    assert torch.isnan(f["y"][40]).all() and torch.isnan(f["y"][41, 9]) and not f["y"][41, :9].any()
    s = f["s_row"].view(M, d // 32)
    assert torch.all(s[40] == 255) and s[41, 0] == 255 and torch.all(s[41, 1:] == 0)
    assert torch.all(f["q_row"][40] == 0x7F)
    sc = f["s_col"].view(d, 2)
    assert torch.all(sc[:, 1] == 255) and torch.equal(sc[:, 0], clean["s_col"].view(d, 2)[:, 0])
    back = mx.ckpt8_load(f["ckpt"])
    assert torch.isnan(back[40, :32]).all() and torch.isnan(back[41, :32]).all()
    assert torch.equal(back[40, 32:], mx.ckpt8_load(clean["ckpt"])[40, 32:])


def _check_bwd(dx, dw, dy, r, w, dres):
    _, n = ref64.rmsnorm(r, w.double(), EPS)
    M = r.shape[0]
    gx, gw, mx_, mw = ref64.rmsnorm_bwd(dy.double(), r, n, w.double())
    if dres is not None:
        gx, mx_ = gx + dres.double(), mx_ + dres.double().abs()
    assert torch.all((ref64.f64(dx) - gx).abs() <= gx.abs() * 2.0 ** -8 + mx_ * 2.0 ** -18)
    depth = (M // 256 + 64) * 2.0 ** -24
    assert torch.all((ref64.f64(dw) - gw).abs() <= gw.abs() * 2.0 ** -8 + mw * (depth + EY))


@pytest.mark.parametrize("ckpt", [False, True])
@pytest.mark.parametrize("M,d,residual", [(1, 32, True), (1, 4096, False), (3, 544, True), (130, 1056, True),
                                          (1025, 2080, False), (700, 7168, True), (5, 16384, True), (40, 8224, True)])
def test_backward(M, d, residual, ckpt):
    x, res, w = _inputs(M, d, residual, M * 3 + d)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), None if res is None else res.cuda(), eps=EPS, y=False, ckpt=ckpt)
    dy = _bf16((M, d), 11, 0.01)
    dres = _bf16((M, d), 12, 0.01) if residual else None
    dx, dw = mx.add_rmsnorm_bwd(dy.cuda(), f["ckpt"] if ckpt else f["r"], f["rstd"], w.cuda(),
                                dres=None if dres is None else dres.cuda())
    r = f["r"].cpu().double()
    n = ref64.rmsnorm(r, w.double(), EPS)[1]
    if ckpt:                       # the statistics are the forward pass's, the values the checkpoint's
        r = ref64.int8_values(r)
    gx, gw, mag, mw = ref64.rmsnorm_bwd(dy.double(), r, n, w.double())
    if dres is not None:
        gx, mag = gx + dres.double(), mag + dres.double().abs()
    assert torch.all((ref64.f64(dx) - gx).abs() <= gx.abs() * 2.0 ** -8 + mag * 2.0 ** -18)
    assert torch.all((ref64.f64(dw) - gw).abs() <= gw.abs() * 2.0 ** -8 + mw * ((M // 256 + 64) * 2.0 ** -24 + EY))


def test_backward_against_differences():
    """<dx, v> and <dw, u> against central differences of the 64-bit forward pass; the gradients' bf16
    rounding contributes 2^-8 of each term, the differences h^2 and 1e-16 / h."""
    M, d = 6, 96
    x, res, w = _inputs(M, d, True, 21)
    x, res = x + 0, res + 0
    dy = _bf16((M, d), 22)
    f = mx.add_rmsnorm_fwd(x.cuda(), w.cuda(), res.cuda(), eps=EPS)
    dx, dw = mx.add_rmsnorm_bwd(dy.cuda(), f["r"], f["rstd"], w.cuda())
    r, w64, dy = f["r"].cpu().double(), w.double(), dy.double()
    live = r.abs().sum(1) > 0                    # the zero row bends within h: left to the formula's test
    r, dy, dx = r[live], dy[live], ref64.f64(dx)[live]
    loss = lambda a, b: (dy * ref64.rmsnorm(a, b, EPS)[0]).sum()  # noqa: E731
    h = 1e-5
    for seed in range(5):
        v = torch.randn(r.shape, generator=_gen(seed), dtype=torch.float64)
        num = (loss(r + h * v, w64) - loss(r - h * v, w64)) / (2 * h)
        assert abs(num - (dx * v).sum()) <= (dx * v).abs().sum() * 2.0 ** -8 + 1e-6
        u = torch.randn(w64.shape, generator=_gen(seed + 50), dtype=torch.float64)
        num = (loss(r, w64 + h * u) - loss(r, w64 - h * u)) / (2 * h)
        got = ref64.f64(dw)
        assert abs(num - (got * u).sum()) <= (got * u).abs().sum() * 2.0 ** -8 + 1e-6


def test_no_rows():
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    f = mx.add_rmsnorm_fwd(x, w, x.clone(), axis=mx.BOTH, ckpt=True)
    assert f["y"].shape == (0, 64) and f["q_col"].shape == (64, 0)
    dx, dw = mx.add_rmsnorm_bwd(x, f["r"], f["rstd"], w)
    assert dx.shape == (0, 64) and dw.shape == (64,) and not dw.any()


def test_repeatable_and_on_another_stream():
    x, res, w = (t.cuda() for t in _inputs(700, 1056, True, 5))
    dy = _bf16((700, 1056), 6).cuda()

    def once():
        f = mx.add_rmsnorm_fwd(x, w, res, axis=mx.ROW, ckpt=True)
        return [f["r"], f["y"], f["q_row"], f["s_row"], f["rstd"], *mx.add_rmsnorm_bwd(dy, f["ckpt"], f["rstd"], w, dres=res)]

    a = once()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = once()
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_sum_may_replace_an_input():
    M, d = 64, 544
    x, res, w = (t.cuda() for t in _inputs(M, d, True, 8))
    want = mx.add_rmsnorm_fwd(x, w, res, axis=mx.BOTH)
    P = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    for into in ("x", "res"):
        a, b = x.clone(), res.clone()
        r = a if into == "x" else b
        rstd, y = torch.empty(M, device="cuda"), torch.empty_like(x)
        st = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        assert mx.lib().mx_add_rmsnorm_fwd(P(a), P(b), P(w), M, d, EPS, P(r), P(rstd), P(y), 0, 0, 0, None, None, None, None,
                                           None, None, st) == 0
        assert torch.equal(r, want["r"]) and torch.equal(y, want["y"])


def test_refuses_tensors_it_cannot_take():
    x = torch.zeros((64, 96), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(96, dtype=torch.bfloat16, device="cuda")
    f = mx.add_rmsnorm_fwd(x, w)
    bad = [lambda: mx.add_rmsnorm_fwd(x.float(), w), lambda: mx.add_rmsnorm_fwd(x[:, ::2], w[::2].contiguous()),
           lambda: mx.add_rmsnorm_fwd(x, w[:64].contiguous()), lambda: mx.add_rmsnorm_fwd(x, w, x[:32].contiguous()),
           lambda: mx.add_rmsnorm_fwd(x.cpu(), w), lambda: mx.add_rmsnorm_fwd(x, w, eps=-1.0),
           lambda: mx.add_rmsnorm_fwd(x, w, eps=float("nan")), lambda: mx.add_rmsnorm_fwd(x[:33], w, axis=mx.COL),
           lambda: mx.add_rmsnorm_fwd(x.view(-1)[4:4 + 32 * 96].view(32, 96), w),
           lambda: mx.add_rmsnorm_fwd(x.view(128, 48), w[:48].contiguous(), axis=mx.ROW),
           lambda: mx.add_rmsnorm_bwd(x, f["r"][:32], f["rstd"], w), lambda: mx.add_rmsnorm_bwd(x, f["r"], f["rstd"][:32], w),
           lambda: mx.add_rmsnorm_bwd(x, mx.ckpt8_save(x[:32]), f["rstd"], w),
           lambda: mx.add_rmsnorm_bwd(x, None, f["rstd"], w)]
    for call in bad:
        with pytest.raises(mx.MxError):
            call()
