"""embedding_rows_backward where a token's run goes over many chunks of the sorted list: written and added to, in every type, rows at pitches.

Tolerances: a chunk's 32 tokens in one chain, at most 256 chunks' sums in another, or the chunks' sums over 32 warps: fewer additions than
a run has tokens, 2^-24 of the magnitudes each, with a product and a sum with what was there; then half a step.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, TYPES, U, assert_close, half_step, placed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def batch(T, V, D, dt, runs, seed=3):
    """Tokens of which ``runs`` = {token: how many} stand all over the batch, and their gradients."""
    gen = torch.Generator().manual_seed(seed)
    tok = torch.randint(0, V, (T,), generator=gen)
    at = torch.randperm(T, generator=gen)
    for v, n in runs.items():
        tok[at[:n]], at = v, at[n:]
    tok[at[:50]] = -1
    return torch.randn(T, D, generator=gen).to(dt), tok


def reference(dy, tok, V, scale):
    keep = tok >= 0
    zero = torch.zeros(V, dy.shape[1], dtype=torch.float64)
    ref = zero.index_add(0, tok[keep], dy[keep].double()) * scale
    mag = zero.index_add(0, tok[keep], dy[keep].double().abs()) * abs(scale)
    n = torch.bincount(tok[keep], minlength=V).double()[:, None]
    return ref, (torch.clamp(n, max=32 + 256 + 32) + 2) * U * mag, n[:, 0] > 0


# chunks of 32 tokens: more than 256 of them from 8193 tokens on; runs of more than 16 chunks go to 32 warps
RUNS = [(20000, 500, 40, {7: 9000}), (20000, 500, 72, {0: 700, 499: 3000, 250: 512, 251: 513, 3: 545}), (9000, 1, 130, {0: 8000}),
        (50000, 60, 8, {59: 20000, 58: 20000}), (8200, 9, 300, {4: 4000}), (8192, 9, 300, {4: 4000})]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V,D,runs", RUNS)
def test_long_runs(T, V, D, runs, dt):
    dy, tok = batch(T, V, D, dt, runs)
    ref, tol, hit = reference(dy, tok, V, 0.5)
    for out in {F32, dt}:
        g = rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), V, scale=0.5, dtype=out)
        assert_close(g, ref, tol + torch.where(hit[:, None], half_step(ref, out), 0.0), "written")
        old = torch.randn(V, D, generator=torch.Generator().manual_seed(5)).to(out)
        old[~hit, 0] = math.nan
        for shift, pad in ((0, 0), (3, 5)):
            h = placed(old, shift, pad)
            gaps = torch.isnan(h._base if h._base is not None else h).sum()
            got = rwo.embedding_rows_backward(placed(dy, shift, pad), tok.cuda(), grad=h, scale=0.5, accumulate=True, dtype=out)
            assert got is h and rwo.get_status() == rwo.OK
            want = ref + old.double()
            where = hit.cuda()
            assert_close(h[where], want[hit], (tol + 2 * U * (old.double().abs() + ref.abs()))[hit] + half_step(want[hit], out), "added to")
            assert torch.equal(h[~where].nan_to_num(nan=7.0).cpu(), old[~hit].nan_to_num(nan=7.0))
            assert torch.isnan(h._base if h._base is not None else h).sum() == gaps


def test_accumulate_repeats():
    """The same bits for the same call, and twice the gradient for two calls where sums are exact."""
    dy, tok = batch(20000, 500, 64, F32, {7: 9000, 8: 600})
    dy = dy.mul(8).round() / 8  # sums of multiples of 1/8 below 2^21: exact in any order
    one = rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), 500)
    two = one.clone()
    rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), grad=two, accumulate=True)
    assert torch.equal(two, 2 * one)
    assert torch.equal(one.double().cpu(), reference(dy, tok, 500, 1.0)[0])
