"""rms_norm_rows, rms_norm_rows_e4m3 and rms_norm_rows_backward against float64.

Tolerances: a thread adds up at most max(64, N / 256) squares and ten partial sums follow, each addition off by 2^-24 of
the sum: ADDS 2^-24 of the sum, half of that of rstd, with 6 more roundings for the quotient, eps, root, weight and products.
Then half a step of the element type; of e4m3, 2^-4 of the value, or 2^-10 of the scale below 2^-6 of it.
Backward: c = mean(g xhat) is off by (ADDS + 4) 2^-24 mean |g xhat|, dx by 6 roundings of its terms besides; dweight by as many
roundings as there are rows, in whatever order, and three for a product.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, FP, TYPES, U, assert_close, half_step, placed

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
LENGTHS = [1, 2, 3, 8, 31, 64, 100, 128, 129, 500, 768, 1024, 2048, 4096, 5003, 5120, 8192, 11008, 16384, 20001, 40960]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def adds(N):
    return max(64, N / 256) + 10


def rows(M, N, dt, seed, amplitude=True):
    gen = torch.Generator().manual_seed(seed * 7919 + N)
    x = torch.randn(M, N, generator=gen)
    if amplitude:
        x *= torch.exp(torch.randn(M, 1, generator=gen))
    return x.to(dt)


def weight(N, dt, seed=3):
    return (1 + 0.2 * torch.randn(N, generator=torch.Generator().manual_seed(seed))).to(dt)


def reference(x, w, r=None, eps=1e-6, offset=0.0):
    """h, rstd, y in 64 bits; h as the element type holds it."""
    dt = x.dtype
    h = x.double() if r is None else (x.double() + r.double()).to(dt).double()
    eps, offset = (float(torch.tensor(v, dtype=F32)) for v in (eps, offset))
    rstd = 1 / torch.sqrt(h.pow(2).mean(1) + eps)
    f = torch.ones(x.shape[1], dtype=torch.float64) if w is None else w.double() + offset
    return h, rstd, h * rstd[:, None] * f


def y_tol(y, N, dt):
    return (adds(N) / 2 + 6) * U * y.abs() + half_step(y, dt)


def check(x, w, r=None, eps=1e-6, offset=0.0, **kw):
    M, N = x.shape
    h, rstd, y = reference(x.cpu(), None if w is None else w.cpu(), None if r is None else r.cpu(), eps, offset)
    rs = torch.full((M,), math.nan, device="cuda")
    got, total = rwo.rms_norm_rows(x, w, r, rstd_out=rs, eps=eps, offset=offset, **kw)
    assert rwo.get_status() == rwo.OK
    if r is None:
        assert total is None
    else:
        assert torch.equal(total.double().cpu(), h)
    assert_close(rs, rstd, (adds(N) / 2 + 4) * U * rstd, "rstd")
    assert_close(got, y, y_tol(y, N, x.dtype), "y")
    return got, total, rs


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", LENGTHS)
def test_lengths(N, dt):
    M = 3 if N > 10000 else 19
    x, r, w = rows(M, N, dt, 1).cuda(), rows(M, N, dt, 2).cuda(), weight(N, dt).cuda()
    check(x, w)
    check(x, w, r)
    check(x, w.float(), r, offset=1.0)
    check(x, None, r, eps=1e-3)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", [64, 100, 1000, 4096, 9000])
@pytest.mark.parametrize("shift,pad", [(0, 8), (1, 0), (3, 5)])
def test_pitches_offsets_and_in_place(N, dt, shift, pad):
    x, r, w = rows(6, N, dt, 4), rows(6, N, dt, 5), weight(N, dt)
    want, h, _ = check(x.cuda(), w.cuda(), r.cuda())
    wp = placed(w[None], shift)[0]
    xp, rp = placed(x, shift, pad), placed(r, shift, pad)
    yp = placed(torch.zeros_like(x), shift, pad)
    a, ha = rwo.rms_norm_rows(xp, wp, rp, y=yp)
    assert_close(a, want.double(), 2 * y_tol(want.double().cpu(), N, dt) + half_step(want.double().cpu(), dt)) and torch.equal(ha, h)
    # the sum where the residual was, y where x was; and the other way round
    rwo.rms_norm_rows(xp, wp, rp, y=xp, sum_out=rp)
    assert torch.equal(xp, a) and torch.equal(rp, h)
    xp, rp = placed(x, shift, pad), placed(r, shift, pad)
    rwo.rms_norm_rows(xp, wp, rp, y=rp, sum_out=xp)
    assert torch.equal(rp, a) and torch.equal(xp, h)
    xp = placed(x, shift, pad)
    b, _ = rwo.rms_norm_rows(xp.clone(), w.cuda())
    rwo.rms_norm_rows(xp, w.cuda(), y=xp)
    assert_close(xp, b.double(), 2 * half_step(b.double().cpu(), dt) + 2 * y_tol(b.double().cpu(), N, dt))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N", [1, 5, 64, 127, 128, 129, 1000, 1024, 4096, 5003, 8192, 16384, 20001])
def test_e4m3(N, group, dt):
    M = 3 if N > 10000 else 11
    x, r, w = rows(M, N, dt, 6), rows(M, N, dt, 7), weight(N, dt)
    x[0] = 0
    r[0] = 0  # a row of zeros
    _, _, y = reference(x, w, r)
    got, scales, h = rwo.rms_norm_rows_e4m3(x.cuda(), w.cuda(), r.cuda(), group=group)
    assert rwo.get_status() == rwo.OK
    assert got.dtype is E4 and torch.equal(h.cpu(), (x.double() + r.double()).to(dt))
    size = group or N
    groups = -(-N // size)
    assert scales.shape == (M, groups)
    padded = torch.nn.functional.pad(y, (0, groups * size - N)).view(M, groups, size)
    want = (padded.abs().amax(2) / 448).clamp(min=2.0 ** -126)
    assert_close(scales, want, (adds(N) / 2 + 8) * U * want, "scales")
    s = scales.double().cpu().repeat_interleave(size, 1)[:, :N]
    tol = (adds(N) / 2 + 8) * U * y.abs() + torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s)
    assert_close(got.float().double().cpu() * s, y, tol, "y")
    assert got.float().abs().max() <= 448


@pytest.mark.parametrize("N", [4096, 1001])
def test_e4m3_uses_its_range(N):
    """The largest value of each group is code 448; doubling x changes nothing but nothing else (the norm takes it out)."""
    x, w = rows(9, N, F32, 8).cuda(), weight(N, F32).cuda()
    for group in (0, 128):
        y, s, h = rwo.rms_norm_rows_e4m3(x, w, group=group, eps=0.0)
        assert h is None
        size = group or N
        for g in range(s.shape[1]):
            assert (y[:, g * size: (g + 1) * size].float().abs().amax(1) == 448).all()
        y2, s2, _ = rwo.rms_norm_rows_e4m3(2 * x, w, group=group, eps=0.0)
        assert torch.equal(y.view(torch.uint8), y2.view(torch.uint8)) and torch.equal(s, s2)


def test_special_rows():
    """Zeros, tiny and huge values, NaN and infinity in a row: others stay as they are."""
    N = 4096
    x = rows(8, N, F32, 9)
    x[1] = 0
    x[2] *= 1e-15
    x[3] *= 1e15
    x[4, 7] = math.nan
    x[5, 9] = math.inf
    w = weight(N, F32)
    clean = [0, 1, 2, 3, 6, 7]
    y, _ = rwo.rms_norm_rows(x.cuda(), w.cuda())
    _, _, ref = reference(x, w)
    assert_close(y[clean], ref[clean], y_tol(ref[clean], N, F32))
    assert torch.isnan(y[4]).all() and torch.isnan(y[5, 9]) and not y[5, :9].any()
    y, s, _ = rwo.rms_norm_rows_e4m3(x.cuda(), w.cuda())
    assert not y[1].float().any() and (s[1] == 2.0 ** -126).all()


# ---- backward -------------------------------------------------------------------------------------------------


def grad_reference(dy, h, rstd, w, offset=0.0, sg=None):
    """dx, dweight and their tolerances before rounding."""
    dy, h, rstd = dy.double(), h.double(), rstd.double()[:, None]
    M, N = h.shape
    f = torch.ones(N, dtype=torch.float64) if w is None else w.double() + float(torch.tensor(offset, dtype=F32))
    xhat, g = h * rstd, dy * f
    c, ca = (g * xhat).mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True)
    dx = rstd * (g - xhat * c)
    tol = rstd * ((g.abs() + (xhat * c).abs()) * 6 * U + xhat.abs() * ca * (adds(N) + 4) * U)
    if sg is not None:
        dx = dx + sg.double()
        tol = tol + U * dx.abs()
    terms = dy * xhat
    return dx, terms.sum(0), tol, (M + 3) * U * terms.abs().sum(0)


def grad_check(dy, h, rstd, w, offset=0.0, sg=None, **kw):
    cpu = [None if t is None else t.cpu() for t in (dy, h, rstd, w, sg)]
    dx_ref, dw_ref, tol, dw_tol = grad_reference(*cpu[:4], offset, cpu[4])
    dx, dw = rwo.rms_norm_rows_backward(dy, h, rstd, w, offset=offset, sum_grad=sg, **kw)
    assert rwo.get_status() == rwo.OK
    assert_close(dx, dx_ref, tol + half_step(dx_ref, h.dtype), "dx")
    if w is None:
        assert dw is None
    else:
        assert_close(dw, dw_ref, dw_tol + 2.0 ** -140, "dweight")
    return dx, dw


def grad_inputs(M, N, dt, seed=11):
    h, dy, sg = rows(M, N, dt, seed), rows(M, N, dt, seed + 1, False), rows(M, N, dt, seed + 2, False)
    rstd = (1 / torch.sqrt(h.double().pow(2).mean(1) + 1e-6)).float()
    return dy, h, rstd, sg, weight(N, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_lengths(N, dt):
    M = 5 if N > 10000 else 70
    dy, h, rstd, sg, w = (t.cuda() for t in grad_inputs(M, N, dt))
    grad_check(dy, h, rstd, w)
    grad_check(dy, h, rstd, w.float(), 1.0, sg)
    grad_check(dy, h, rstd, None, 0.0, sg)


@pytest.mark.parametrize("M,N", [(1, 4096), (2, 64), (1000, 128), (5000, 768), (3001, 1000), (700, 8192), (20000, 33), (2500, 2500)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_backward_many_rows(M, N, dt):
    dy, h, rstd, sg, w = (t.cuda() for t in grad_inputs(M, N, dt, 20))
    a = grad_check(dy, h, rstd, w, 0.0, sg)
    b = rwo.rms_norm_rows_backward(dy, h, rstd, w, sum_grad=sg)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # one order of additions
    old = torch.randn(N, device="cuda")
    dw = old.clone()
    rwo.rms_norm_rows_backward(dy, h, rstd, w, sum_grad=sg, dweight=dw, accumulate=True)
    assert torch.equal(dw, old + a[1])


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("N", [100, 1024, 4099, 24000])
@pytest.mark.parametrize("shift,pad", [(0, 16), (1, 3)])
def test_backward_pitches_and_in_place(N, dt, shift, pad):
    dy, h, rstd, sg, w = grad_inputs(33, N, dt, 30)
    rs, wd = rstd.cuda(), w.cuda()
    want = grad_check(dy.cuda(), h.cuda(), rs, wd, 0.0, sg.cuda())
    tol = [2 * t for t in grad_reference(dy, h, rstd, w, 0.0, sg)[2:]]
    for place in range(4):
        p = [placed(t, shift, pad) for t in (dy, h, sg)]
        dx = p[place] if place < 3 else placed(torch.zeros_like(h), shift, pad)
        got = rwo.rms_norm_rows_backward(p[0], p[1], rs, wd, sum_grad=p[2], dx=dx)
        assert got[0] is dx
        assert_close(dx, want[0].double(), tol[0] + 2 * half_step(want[0].double().cpu(), dt), f"dx over {place}")
        assert_close(got[1], want[1].double(), tol[1] + 2.0 ** -140, f"dweight with dx over {place}")


def test_backward_against_differences():
    """The formula's gradients, which the kernel is held to above, against central differences in 64 bits."""
    M, N, k = 3, 17, 1e-6
    x, w, dy, sg = (rows(M, N, F32, s, False).double() for s in (40, 41, 42, 43))
    w = w[0] + 1

    def total(x, w):
        rstd = 1 / torch.sqrt(x.pow(2).mean(1, keepdim=True) + 1e-6)
        return float((dy * x * rstd * (w + 1)).sum() + (sg * x).sum())

    rstd = (1 / torch.sqrt(x.pow(2).mean(1) + 1e-6))
    dx, dw, _, _ = grad_reference(dy, x, rstd, w, 1.0, sg)
    got = rwo.rms_norm_rows_backward(dy.float().cuda(), x.float().cuda(), rstd.float().cuda(), w.float().cuda(), offset=1.0, sum_grad=sg.float().cuda())
    for i in range(M):
        for j in range(N):
            e = torch.zeros(M, N, dtype=torch.float64)
            e[i, j] = k
            diff = (total(x + e, w) - total(x - e, w)) / (2 * k)
            assert abs(diff - dx[i, j]) < 1e-7 and abs(diff - float(got[0][i, j])) < 1e-5 * (1 + abs(diff))
    for j in range(N):
        e = torch.zeros(N, dtype=torch.float64)
        e[j] = k
        diff = (total(x, w + e) - total(x, w - e)) / (2 * k)
        assert abs(diff - dw[j]) < 1e-7 and abs(diff - float(got[1][j])) < 1e-5 * (1 + abs(diff))


def test_empty_and_leading_dimensions():
    w = weight(64, BF).cuda()
    x = rows(12, 64, BF, 50).cuda()
    y, _ = rwo.rms_norm_rows(x.view(3, 4, 64), w)
    assert torch.equal(y.view(12, 64), rwo.rms_norm_rows(x, w)[0])
    y, s, h = rwo.rms_norm_rows_e4m3(x[:0], w, x[:0])
    assert y.shape == (0, 64) and s.shape == (0, 1) and h.shape == (0, 64)
    dx, dw = rwo.rms_norm_rows_backward(x[:0], x[:0], torch.empty(0, device="cuda"), w)
    assert dx.shape == (0, 64) and not dw.any()
    old = torch.ones(64, device="cuda")
    rwo.rms_norm_rows_backward(x[:0], x[:0], torch.empty(0, device="cuda"), w, dweight=old, accumulate=True)
    assert (old == 1).all()


def test_streams_and_graphs():
    """Calls with workspaces of their own on another stream and in a graph."""
    dy, h, rstd, sg, w = (t.cuda() for t in grad_inputs(500, 4096, BF, 60))
    want = rwo.rms_norm_rows_backward(dy, h, rstd, w, sum_grad=sg)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rwo.rms_norm_rows_backward(dy, h, rstd, w, sum_grad=sg, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    ws = rwo.rms_norm_backward_workspace(500, 4096, BF)
    dx, dw = torch.zeros_like(h), torch.zeros(4096, device="cuda")
    y, hs, rs = torch.zeros_like(h), torch.zeros_like(h), torch.zeros(500, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rwo.rms_norm_rows(h, w, sg, y=y, sum_out=hs, rstd_out=rs)
        rwo.rms_norm_rows_backward(dy, h, rstd, w, sum_grad=sg, dx=dx, dweight=dw, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    assert torch.equal(y, rwo.rms_norm_rows(h, w, sg)[0])


def framed(t, shift, pad):
    """t at a pitch of pad more, its storage's other elements NaN."""
    M, N = t.shape
    buf = torch.full((shift + M * (N + pad) + 8,), math.nan, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N", [(5000, 7), (3001, 333), (1700, 1501), (900, 5003), (400, 14001)])
@pytest.mark.parametrize("shift,pad,other", [(0, 0, 0), (1, 2, 0), (5, 0, 0), (3, 1, 1)])
def test_rows_on_no_boundary(M, N, dt, shift, pad, other):
    """Many rows that start anywhere, all matrices alike (other = 0) or one elsewhere; what lies between the rows stays."""
    dy, h, rstd, sg, w = grad_inputs(M, N, dt)
    (_, hv), (_, sv), (_, rv) = framed(h, shift, pad), framed(sg, shift + other, pad), framed(dy, shift, pad)
    buf, dv = framed(dy, shift, pad)
    gaps = torch.isnan(buf)
    dx, _ = grad_check(rv, hv, rstd.cuda(), w.cuda(), sg=sv, dx=framed(dy, shift, pad)[1])
    again, _ = rwo.rms_norm_rows_backward(dv, hv, rstd.cuda(), w.cuda(), sum_grad=sv, dx=dv)
    assert torch.equal(again, dx) and torch.equal(torch.isnan(buf), gaps)
    check(hv, w.cuda(), sv)
    buf, v = framed(h, shift, pad)
    y, _ = rwo.rms_norm_rows(v, w.cuda(), sv, y=framed(h, shift, pad)[1], sum_out=v)
    assert torch.equal(torch.isnan(buf), gaps)
    buf, v = framed(h, shift, pad)
    plain, _ = rwo.rms_norm_rows(v, w.cuda(), y=v)
    assert torch.equal(torch.isnan(buf), gaps)
    assert_close(plain, reference(h, w)[2], y_tol(reference(h, w)[2], N, dt))
    ref = reference(h, w, sg)[2]
    assert_close(y, ref, y_tol(ref, N, dt))
