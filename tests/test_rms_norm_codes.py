"""rms_norm_rows_e4m3: which code a value gets, and calls with tensors given, at pitches and at offsets.

A code is the nearest to 448 h w / max |h w| (rstd is in both).  With bf16 elements and weights h w has at most 16 bits, and 7 h w 19.
About one value in 2500 lies in the middle between two codes, the others at least 2^-21 of themselves from there, so the quotient
in 64 bits, rounded to fp32, falls on the right side everywhere, and the codes are compared for equality.  With fp16 h w has 22 bits
and 7 h w 25, one more than fp32 holds: like fp32 elements' it is rounded, as are the weight times 7/8 and the quotient, and the largest
value alike: six roundings of 2^-24, within which a code may be that of the quotient a little more or less.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from test_rms_norm import E4, adds, framed, reference, rows, weight
from train_util import BF, F32, FP, TYPES, U, assert_close, placed

pytestmark = pytest.mark.gpu
LENGTHS = [1, 5, 64, 127, 128, 129, 1000, 1024, 4096, 5003, 8192, 16384, 20001, 40960]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def grouped(t, size):
    N = t.shape[1]
    groups = -(-N // size)
    return torch.nn.functional.pad(t, (0, groups * size - N)).view(t.shape[0], groups, size)


def quotients(h, w, group):
    M, N = h.shape
    p = grouped(h.double() * w.double(), group or N)
    top = p.abs().amax(2, keepdim=True)
    return torch.where(top > 0, 448 * p / top, 0.0).view(M, -1)[:, :N]


def assert_codes(got, h, w, group):
    """got: the codes' values."""
    q = quotients(h, w, group)
    if h.dtype is BF:
        assert torch.equal(got.cpu(), q.float().to(E4).float())
    else:
        less, more = ((q * (1 + s * 6 * U)).clamp(-448, 448).float().to(E4).float() for s in (-1, 1))
        assert ((got.cpu() == less) | (got.cpu() == more)).all()


def scales_of(y, group):
    return (grouped(y, group or y.shape[1]).abs().amax(2) / 448).clamp(min=2.0 ** -126)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N", LENGTHS)
def test_codes_are_the_nearest(N, group, dt):
    """Every kernel: rows that start on 16-byte boundaries, at a pitch, anywhere, with and without a residual."""
    M = 5 if N > 10000 else 40
    x, r, w = rows(M, N, dt, 100), rows(M, N, dt, 101), weight(N, dt)
    x[0] = r[0] = 0
    h = (x.double() + r.double()).to(dt)
    for shift, pad in ((0, 0), (0, -N % 16 + 16), (3, 5)):
        xp, rp = placed(x, shift, pad), placed(r, shift, pad)
        got, scales, total = rwo.rms_norm_rows_e4m3(xp, w.cuda(), rp, group=group)
        assert rwo.get_status() == rwo.OK
        assert torch.equal(total.cpu(), h)
        assert_codes(got.float(), h, w, group)
        y = reference(x, w, r)[2]
        assert_close(scales, scales_of(y, group), (adds(N) / 2 + 8) * U * scales_of(y, group), "scales")
        assert_codes(rwo.rms_norm_rows_e4m3(xp, w.cuda(), group=group)[0].float(), x, w, group)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("group", [0, 128])
def test_codes_of_many_rows(group, dt):
    x, w = rows(3000, 2048, dt, 103), weight(2048, dt)
    got, _, _ = rwo.rms_norm_rows_e4m3(x.cuda(), w.cuda(), group=group)
    assert_codes(got.float(), x, w, group)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N", [128, 4096, 5003, 40960])
def test_codes_of_large_and_small_rows(N, group):
    """The codes do not depend on a row's magnitude, as long as the scales are above their least."""
    x, w = rows(6, N, BF, 104, False), weight(N, BF)
    x = (x.double() * torch.tensor([1.0, 2.0 ** 50, 2.0 ** -14, 2.0 ** -40, 2.0 ** 20, 2.0 ** -7], dtype=torch.float64)[:, None]).to(BF)
    got, scales, _ = rwo.rms_norm_rows_e4m3(x.cuda(), w.cuda(), group=group, eps=0.0)
    assert_codes(got.float(), x, w, group)
    y = reference(x, w, eps=0.0)[2]
    assert_close(scales, scales_of(y, group), (adds(N) / 2 + 8) * U * scales_of(y, group), "scales")


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N", [100, 4096, 5003, 40960])
def test_scales_at_their_least(N, group, dt):
    """y below 448 2^-126: the scale is 2^-126 and the codes are y 2^126."""
    x, w = rows(4, N, F32, 105, False).double(), weight(N, dt)
    x = (x * torch.tensor([2.0 ** -132, 2.0 ** -138, 2.0 ** -128, 1.0], dtype=torch.float64)[:, None]).to(dt)
    eps = 0.25  # rstd = 2
    got, scales, _ = rwo.rms_norm_rows_e4m3(x.cuda(), w.cuda(), group=group, eps=eps)
    y = reference(x, w, eps=eps)[2]
    assert_close(scales, scales_of(y, group), (adds(N) / 2 + 8) * U * scales_of(y, group), "scales")
    s = scales.double().cpu().repeat_interleave(group or N, 1)[:, :N]
    # h rstd weight of y's size may be below fp32's normal values, where a rounding is off by 2^-150
    tol = (adds(N) / 2 + 8) * U * y.abs() + torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s) + 2.0 ** -147
    assert_close(got.float().double().cpu() * s, y, tol, "y")


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("N,M", [(64, 50), (333, 70), (4096, 30), (5003, 20), (20001, 4)])
@pytest.mark.parametrize("shift,pad,yshift,ypad", [(0, 8, 0, 16), (0, 8, 1, 3), (1, 3, 0, 0), (5, 2, 7, 1)])
def test_tensors_given(N, M, group, dt, shift, pad, yshift, ypad):
    """y and the scales given, y at a pitch and at an offset; what lies between the rows stays; the sum over x or the residual."""
    x, r, w = rows(M, N, dt, 106), rows(M, N, dt, 107), weight(N, dt).cuda()
    parts = -(-N // group) if group else 1
    want = rwo.rms_norm_rows_e4m3(x.cuda(), w, r.cuda(), group=group)
    _, _, y = reference(x, w.cpu(), r)
    s = want[1].double().cpu().repeat_interleave(group or N, 1)[:, :N]
    assert_close(want[0].float().double().cpu() * s, y, (adds(N) / 2 + 8) * U * y.abs() + torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s), "y")
    for place in range(3):
        (_, xp), (_, rp) = framed(x, shift, pad), framed(r, shift, pad)
        buf = torch.full((yshift + M * (N + ypad) + 8,), 0x7F, dtype=torch.uint8, device="cuda")  # NaN between the rows
        yp = buf[yshift: yshift + M * (N + ypad)].view(M, N + ypad)[:, :N]
        sc, rs = torch.full((M, parts), math.nan, device="cuda"), torch.full((M,), math.nan, device="cuda")
        a, b, h = rwo.rms_norm_rows_e4m3(xp, w, rp, group=group, y=yp.view(E4), scales=sc, rstd_out=rs, sum_out=(None, xp, rp)[place])
        assert rwo.get_status() == rwo.OK and b is sc and a.data_ptr() == yp.data_ptr()
        assert torch.equal(h, want[2])
        # rows placed otherwise add their squares in another order: rstd may be off by its tolerance, bf16 rows' codes are not
        assert_close(sc, want[1].double(), 2 * (adds(N) / 2 + 8) * U * want[1].double().cpu(), "scales")
        got = yp.contiguous().view(E4).float().double().cpu()
        if dt is not BF:
            assert_close(got * s, y, 2 * (adds(N) / 2 + 8) * U * y.abs() + torch.maximum(2.0 ** -4 * y.abs(), 2.0 ** -10 * s), "y")
        else:
            assert torch.equal(got, want[0].float().double().cpu())
        buf.view(-1)[yshift: yshift + M * (N + ypad)].view(M, N + ypad)[:, :N] = 0x7F
        assert (buf == 0x7F).all()  # nothing else was written
