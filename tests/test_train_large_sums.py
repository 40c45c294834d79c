"""Sums of the training-step calls where offsets pass 32 bits, each one compared: dweight over more than a million rows, gradients of
tokens that come more than once.

Tolerances: dweight as many roundings of 2^-24 of the terms' magnitudes as a CTA has rows and parts there are; a gradient's row as many as
it has tokens, then half a step.
"""
import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, U, assert_close, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of device memory")


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def filled(shape, seed, scale=1.0):
    t = torch.empty(shape, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for c in t.view(-1).split(1 << 28):
        c.normal_(generator=gen).mul_(scale)
    return t


@pytest.mark.parametrize("N", [4096, 4095])
def test_dweight_of_many_rows(N):
    M = 1_100_000
    h, dy = filled((M, N), 1), filled((M, N), 2)
    rstd = torch.empty(M, device="cuda")
    want, mag = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for r in range(0, M, 50_000):
        x = h[r: r + 50_000].double()
        rstd[r: r + 50_000] = 1 / torch.sqrt(x.pow(2).mean(1) + 1e-6)
        terms = x.mul_(rstd[r: r + 50_000].double()[:, None]).mul_(dy[r: r + 50_000].double())
        want += terms.sum(0)
        mag += terms.abs_().sum(0)
    w = torch.ones(N, dtype=BF, device="cuda")
    old = torch.randn(N, device="cuda")
    dw = old.clone()
    rwo.rms_norm_rows_backward(dy, h, rstd, w, dx=dy, dweight=dw, accumulate=True)
    assert rwo.get_status() == rwo.OK
    # 152 CTAs at least: 7237 rows each, 304 parts, what was there; three roundings of a term
    tol = (7237 + 304 + 4) * U * mag + U * old.double().abs()
    assert_close(dw, want + old.double(), tol.cpu())
    # Roundings go both ways: a CTA's sums of up to 7237 terms of size 1 are off by some 60 2^-24 85 = 3e-4, 304 of them by 5e-3 a column, all
    # columns by 0.3.  A single row left out or taken twice is N^(1/2) = 64.
    assert float((dw.double() - want - old.double()).norm()) <= N ** 0.5 / 2


def test_gradient_of_repeated_tokens():
    V, D, T = 1_200_000, 4096, 40_000
    gen = torch.Generator(device="cuda").manual_seed(4)
    dy = filled((T, D), 3)
    tokens = torch.randint(0, V, (T,), device="cuda", generator=gen)
    tokens[::4] = torch.tensor([V - 1, 524288, 1048576, 0], device="cuda").repeat(T // 16)  # 2500 times each
    tokens[1::40] = V - 2
    grad = torch.full((V, D), 3.0, dtype=BF, device="cuda")
    g = rwo.embedding_rows_backward(dy, tokens, grad=grad, dtype=BF)
    assert rwo.get_status() == rwo.OK
    uniq, inv = tokens.unique(return_inverse=True)
    n = torch.bincount(inv).double()[:, None]
    ref = torch.zeros(len(uniq), D, dtype=torch.float64, device="cuda").index_add_(0, inv, dy.double())
    mag = torch.zeros(len(uniq), D, dtype=torch.float64, device="cuda").index_add_(0, inv, dy.double().abs())
    assert int((n >= 1000).sum()) == 5
    for c in range(0, len(uniq), 8000):
        at = slice(c, c + 8000)
        tol = (n[at] + 2) * U * mag[at] + half_step(ref[at], BF)
        assert_close(g[uniq[at]], ref[at], tol.cpu())
