"""The loss and its gradient of rows of millions of entries, which are read twice.

Tolerances as for shorter rows: 1e-5 of the softmax and of the loss.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from test_loss_grad import check
from train_util import BF, F32, FP

pytestmark = pytest.mark.gpu
LENGTHS = [700_001, 1 << 22, (1 << 22) + 1, 1 << 24]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("dt", [F32, BF, FP])
@pytest.mark.parametrize("N", LENGTHS)
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_rising_entries(N, dt, eps):
    """Entries that rise along a row, so that nearly every one is the largest yet: by little, by much, and from a masked half."""
    x = torch.stack([torch.linspace(-17.0, 3.0, N), torch.linspace(0.0, 1.0, N), torch.linspace(-3e4, 3e4, N)])
    labels = torch.tensor([N - 1, 7, N // 2], device="cuda")
    check(x.to(dt).cuda(), labels, eps=eps)
    if not eps:
        x[0, : N // 2] = -torch.inf
        x[1, 5:] = -torch.inf
        x[2] = x[2].flip(0)
        check(x.to(dt).cuda(), labels)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("N", LENGTHS)
def test_smoothed_loss(N, dt):
    """Entries at one distance from the maximum, which every thread meets at the start, at the end, or is the only one not to."""
    x = torch.full((4, N), -11.7)
    x[0, :8192] = 0.0
    x[1, -8192:] = 0.0
    x[2] = -5.3
    x[2, N // 2] = 9.0
    x[3, :8192] = 1.4
    labels = torch.tensor([0, 5, N // 2, N - 1], device="cuda")
    check(x.to(dt).cuda(), labels, eps=0.9)
    check(x.to(dt).cuda(), labels, eps=0.1, z=1e-3)


def test_masked_entries():
    """A masked entry gives an infinite smoothed loss, in the first and in a later part of a thread's run; gradients stay finite."""
    N = 1 << 20
    x = torch.randn(3, N, generator=torch.Generator().manual_seed(2))
    x[0, 0] = x[1, N - 9] = -math.inf
    x[2, : N // 2] = -math.inf
    labels = torch.tensor([5, 5, N - 5], device="cuda")
    loss, g = rwo.cross_entropy_rows_grad(x.cuda(), labels, label_smoothing=0.1)
    assert (loss == math.inf).all() and torch.isfinite(g).all()
    check(x.cuda(), labels)


@pytest.mark.parametrize("dt", [F32, BF, FP])
@pytest.mark.parametrize("N", [(1 << 20) + 8, 1_100_001])
@pytest.mark.parametrize("eps", [0.0, 0.1])
def test_rows_with_little_left(N, dt, eps):
    """All but one, all but a few, and all entries masked: most threads meet nothing else."""
    x = torch.full((5, N), -math.inf)
    x[0, 77] = 2.5
    x[1, 1000:1100] = torch.randn(100, generator=torch.Generator().manual_seed(3))
    x[2, -1] = -4.0
    x[3] = 1.0
    x[3, : N - 5] = -math.inf
    labels = torch.tensor([77, 1050, 3, N - 1, 9], device="cuda")
    if eps:
        loss, g = rwo.cross_entropy_rows_grad(x.to(dt).cuda(), labels, label_smoothing=eps)
        assert (loss[:4] == math.inf).all() and torch.isnan(loss[4]) and torch.isfinite(g[:4]).all()
    check(x.to(dt).cuda(), labels, eps=eps)
