"""The norm of rows of millions of elements, forward and backward: a thread's sum of thousands of values of one size.

Tolerances: a thread adds up 64 terms at a time, and those sums with what their additions round away: 64 + 2 2^-24 of the sum however
long it is, eight additions more join the warps and eight the lanes: 82 in all, half of that of rstd, with 6 more roundings for y; of the
backward pass's mean 82 and 4 for its terms, and 6 roundings of dx's terms.
"""
import pytest
import torch

import row_wise_online_gb300 as rwo
from test_rms_norm import reference
from train_util import BF, F32, U, assert_close, half_step

pytestmark = pytest.mark.gpu
ADDS = 82


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def alike(N, dt, values):
    """Rows of nearly equal elements: the rounding of a long plain sum goes one way for many additions."""
    return torch.stack([torch.full((N,), v) for v in values]).to(dt)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", [100_000, (1 << 22) + 3, 1 << 24])
def test_forward(N, dt):
    x = alike(N, dt, [1.1, 0.7, 3.3])
    h, rstd, y = reference(x, None)
    rs = torch.empty(3, device="cuda")
    got, _ = rwo.rms_norm_rows(x.cuda(), rstd_out=rs)
    assert rwo.get_status() == rwo.OK
    assert_close(rs, rstd, (ADDS / 2 + 4) * U * rstd, "rstd")
    assert_close(got, y, (ADDS / 2 + 6) * U * y.abs() + half_step(y, dt), "y")
    r = alike(N, dt, [0.2, 0.4, 0.6])
    h, rstd, y = reference(x, None, r)
    _, scales, total = rwo.rms_norm_rows_e4m3(x.cuda(), residual=r.cuda(), rstd_out=rs, group=0)
    assert torch.equal(total.double().cpu(), h)
    assert_close(rs, rstd, (ADDS / 2 + 4) * U * rstd, "rstd")
    top = y.abs().amax(1, keepdim=True) / 448
    assert_close(scales, top, (ADDS / 2 + 8) * U * top, "scales")


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", [100_000, (1 << 22) + 3, 1 << 24])
def test_backward(N, dt):
    h, dy = alike(N, dt, [1.1, 0.7]), alike(N, dt, [1.3, -0.9])
    rstd = (1 / torch.sqrt(h.double().pow(2).mean(1) + 1e-6)).float()
    dx, dw = rwo.rms_norm_rows_backward(dy.cuda(), h.cuda(), rstd.cuda())
    assert dw is None and rwo.get_status() == rwo.OK
    xhat, g = h.double() * rstd.double()[:, None], dy.double()
    c = (g * xhat).mean(1, keepdim=True)
    ref = rstd.double()[:, None] * (g - xhat * c)
    tol = rstd.double()[:, None] * ((g.abs() + (xhat * c).abs()) * 6 * U + xhat.abs() * c.abs() * (ADDS + 4) * U)
    assert_close(dx, ref, tol + half_step(ref, dt), "dx")


def test_infinities_in_long_rows():
    N = 100_000
    x = torch.randn(3, N, generator=torch.Generator().manual_seed(1))
    x[1, 7] = torch.inf
    x[1, 90_000] = -torch.inf
    rs = torch.empty(3, device="cuda")
    y, _ = rwo.rms_norm_rows(x.cuda(), rstd_out=rs)
    assert rs[1] == 0 and torch.isnan(y[1, [7, 90_000]]).all() and not y[1, 8:90_000].any()
    assert torch.isfinite(y[[0, 2]]).all() and torch.isfinite(rs).all()
