"""The loss and its gradient of rows of millions of entries, which are read twice.

Tolerances as for shorter rows: 1e-5 of the softmax and of the loss.
"""
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
