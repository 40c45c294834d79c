"""The sum that rms_norm_rows keeps beside y, for rows at pitches and offsets: to the bit, whatever is given and whatever it replaces."""
import pytest
import torch

import row_wise_online_gb300 as rwo
from test_rms_norm import framed, rows, weight
from train_util import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("M,N", [(6, 64), (6, 100), (700, 1000), (70, 4096), (300, 5003), (6, 9000), (4, 20001)])
@pytest.mark.parametrize("xs,rs,ss,pad", [(0, 0, 0, 8), (0, 0, 0, 0), (1, 1, 1, 0), (3, 3, 1, 5), (3, 2, 0, 5), (0, 1, 0, 3)])
def test_sum(M, N, xs, rs, ss, pad, dt):
    x, r, w = rows(M, N, dt, 110), rows(M, N, dt, 111), weight(N, dt).cuda()
    want = (x.double() + r.double()).to(dt).cuda()
    (_, xv), (_, rv) = framed(x, xs, pad), framed(r, rs, pad)
    y, h = rwo.rms_norm_rows(xv, w, rv)  # a new tensor
    assert torch.equal(h, want)
    buf, hv = framed(torch.zeros_like(x), ss, pad)
    gaps = torch.isnan(buf)
    y2, h = rwo.rms_norm_rows(xv, w, rv, sum_out=hv)
    assert h is hv and torch.equal(hv, want) and torch.equal(torch.isnan(buf), gaps) and torch.equal(y2, y)
    for place in range(2):  # in place of x, then of the residual
        (_, xv), (_, rv) = framed(x, xs, pad), framed(r, rs, pad)
        into = (xv, rv)[place]
        y2, h = rwo.rms_norm_rows(xv, w, rv, sum_out=into)
        assert h is into and torch.equal(into, want) and torch.equal(y2, y)
    assert rwo.get_status() == rwo.OK
