"""rms_norm_rows_backward of rows of large and small magnitude, in every kernel: rows on 16-byte boundaries and on none, alike and
elsewhere in their lines, held on chip and not.

Tolerances as in test_rms_norm.py: they are relative to the terms, whatever their magnitude.
"""
import pytest
import torch

import row_wise_online_gb300 as rwo
from test_rms_norm import adds, grad_reference, rows, weight
from train_util import BF, F32, U, assert_close, half_step, placed

pytestmark = pytest.mark.gpu
LENGTHS = [100, 1000, 4096, 5003, 8192, 16384, 20001]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def scaled(N, dt, amplitudes, seed, grads):
    """Rows of standard deviation ``amplitudes``, their rstd with eps = 0, and gradients of ``grads``."""
    a, g = (torch.tensor(v, dtype=torch.float64)[:, None] for v in (amplitudes, grads))
    h = (rows(len(a), N, F32, seed, False).double() * a).to(dt)
    dy = (rows(len(a), N, F32, seed + 1, False).double() * g).to(dt)
    sg = (rows(len(a), N, F32, seed + 2, False).double() * g / a).to(dt)
    return dy, h, (1 / torch.sqrt(h.double().pow(2).mean(1))).float(), sg, weight(N, dt)


def check(dy, h, rstd, w, sg, place):
    ref = grad_reference(dy, h, rstd, w, 0.0, sg)
    shifts = {"even": (0, 0, 0), "lines": (3, 3, 3), "elsewhere": (3, 1, 2)}[place]
    pad = -h.shape[1] % 8 if place == "even" else 1
    dyp, hp, sgp = (None if t is None else placed(t, s, pad) for t, s in zip((dy, h, sg), shifts))
    dx, dw = rwo.rms_norm_rows_backward(dyp, hp, rstd.cuda(), w.cuda(), sum_grad=sgp, dx=placed(torch.zeros_like(dy), shifts[0], pad))
    assert rwo.get_status() == rwo.OK
    assert_close(dx, ref[0], ref[2] + half_step(ref[0], h.dtype), "dx")
    assert_close(dw, ref[1], ref[3] + 2.0 ** -140, "dweight")


@pytest.mark.parametrize("place", ["even", "lines", "elsewhere"])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_of_large_and_small_rows(N, dt, place):
    amplitudes = [1e12, 1e14, 1e15, 1e16, 1.0, 1e-6, 1e-13, 1e-15]
    dy, h, rstd, sg, w = scaled(N, dt, amplitudes, 70, [1.0] * 8)
    check(dy, h, rstd, w, None, place)
    check(dy, h, rstd, w, sg, place)


@pytest.mark.parametrize("place", ["even", "lines", "elsewhere"])
@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_where_h_times_dy_leaves_the_range(N, dt, place):
    """dx is of ordinary size or near it, h dy of 1e40 or 1e-43 is not."""
    dy, h, rstd, sg, w = scaled(N, dt, [1e15, 1e-15, 1e15, 1e-15], 80, [1e25, 1e-28, 1e-10, 1e10])
    for r in range(4):  # by themselves: dweight is held to the terms of one magnitude
        check(dy[r: r + 1], h[r: r + 1], rstd[r: r + 1], w, sg[r: r + 1], place)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_backward_of_zero_rows(N, dt):
    """A row of zeros under a small eps: dx = rstd g."""
    dy, h, _, sg, w = scaled(N, dt, [1.0, 1.0, 1.0], 90, [1.0, 1.0, 1.0])
    h[1] = 0
    y, _ = rwo.rms_norm_rows(h.cuda(), w.cuda(), rstd_out=(rs := torch.empty(3, device="cuda")), eps=1e-30)
    assert not y[1].any()
    assert abs(float(rs[1]) - 1e15) <= (adds(N) / 2 + 4) * U * 1e15
    ref = grad_reference(dy, h, rs.cpu(), w)
    dx, dw = rwo.rms_norm_rows_backward(dy.cuda(), h.cuda(), rs, w.cuda())
    assert_close(dx, ref[0], ref[2] + half_step(ref[0], dt), "dx")
    assert_close(dw, ref[1], ref[3] + 2.0 ** -140, "dweight")
