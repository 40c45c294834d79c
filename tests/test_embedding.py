"""embedding_rows and embedding_rows_backward against float64.

Tolerances: a lookup is one fp32 product, rounded to the element type: half a step of each.  A gradient's row of n tokens is n
fp32 additions in any order, a product and a sum with what was there: (n + 2) 2^-24 of the magnitudes added up, then half a step.
"""
import math

import pytest
import torch

import row_wise_online_gb300 as rwo
from train_util import BF, F32, FP, TYPES, U, assert_close, half_step, placed

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from row_wise_online_gb300 import _build

    _build.build()
    torch.cuda.set_device(0)


def tokens_of(T, V, skew, seed=0, padding=0.05):
    gen = torch.Generator().manual_seed(seed * 31 + T)
    t = (V * torch.rand(T, generator=gen, dtype=torch.float64) ** skew).long().clamp(max=V - 1)
    t = t * 7919 % V if math.gcd(7919, V) == 1 else t
    t[torch.rand(T, generator=gen) < padding] = -1
    return t


def values(shape, dt, seed=1):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 50, 4096), (37, 100, 8), (300, 1000, 100), (1000, 7, 1), (513, 5003, 33), (64, 40, 5003), (3000, 2048, 768)])
def test_lookup(T, V, D, dt):
    table, tok = values((V, D), dt), tokens_of(T, V, 2.0)
    for scale in (1.0, 64.0, 0.3):
        ref = torch.where((tok >= 0)[:, None], table.double()[tok.clamp(min=0)] * float(torch.tensor(scale, dtype=F32)), 0.0)
        for kind in (torch.int64, torch.int32):
            y = rwo.embedding_rows(table.cuda(), tok.to(kind).cuda(), scale=scale)
            assert rwo.get_status() == rwo.OK
            assert_close(y, ref, (U * ref.abs() + half_step(ref, dt)) if scale not in (1.0,) else 0.0)
    for shift, pad in ((0, 8), (1, 3)):
        y = placed(torch.zeros(T, D, dtype=dt), shift, pad)
        got = rwo.embedding_rows(placed(table, shift, pad), tok.cuda(), y=y)
        assert got is y and torch.equal(got, rwo.embedding_rows(table.cuda(), tok.cuda()))


def test_lookup_shapes_and_bad_tokens():
    table = values((100, 64), BF).cuda()
    tok = tokens_of(24, 100, 1.0, padding=0).cuda()
    y = rwo.embedding_rows(table, tok.view(2, 3, 4))
    assert y.shape == (2, 3, 4, 64) and torch.equal(y.view(24, 64), table[tok])
    assert rwo.embedding_rows(table, tok[:0]).shape == (0, 64)
    tok[5], tok[7] = 100, 2 ** 33
    y = rwo.embedding_rows(table, tok)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG and rwo.get_status() == rwo.OK
    assert torch.isnan(y[[5, 7]]).all() and torch.equal(y[:5], table[tok[:5]])


def grad_reference(dy, tok, V, scale=1.0):
    scale = float(torch.tensor(scale, dtype=F32))
    keep = (tok >= 0) & (tok < V)
    ref = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, tok[keep], dy[keep].double()) * scale
    mag = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, tok[keep], dy[keep].double().abs()) * abs(scale)
    n = torch.bincount(tok[keep], minlength=V).double()[:, None]
    return ref, (n + 2) * U * mag, n


def check(dy, tok, V, scale=1.0, dtype=F32, dyd=None, tokd=None, **kw):
    ref, tol, _ = grad_reference(dy, tok, V, scale)
    g = rwo.embedding_rows_backward(dy.cuda() if dyd is None else dyd, tok.cuda() if tokd is None else tokd, V, scale=scale, dtype=dtype, **kw)
    assert rwo.get_status() == rwo.OK and g.dtype is dtype
    assert_close(g, ref, tol + torch.where(tol > 0, half_step(ref, dtype), 0.0))
    return g


SIZES = [(1, 1, 1), (1, 1000, 64), (2, 5, 3), (31, 40, 100), (32, 3, 256), (33, 3, 256), (64, 1, 512), (65, 1, 33), (1000, 50000, 768),
         (1500, 5003, 512), (4096, 4096, 128), (5000, 17, 1000), (8193, 300, 72), (40000, 131072, 40), (3000, 2000, 5003)]


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("T,V,D", SIZES)
@pytest.mark.parametrize("skew", [1.0, 6.0])
def test_gradient(T, V, D, dt, skew):
    dy, tok = values((T, D), dt), tokens_of(T, V, skew)
    a = check(dy, tok, V, scale=3.0)
    b = rwo.embedding_rows_backward(dy.cuda(), tok.int().cuda(), V, scale=3.0)
    assert torch.equal(a, b)  # int32 tokens, and the same order of additions
    if dt is not F32:
        check(dy, tok, V, dtype=dt)


@pytest.mark.parametrize("dt", [F32, BF])
@pytest.mark.parametrize("T,V,D", [(700, 300, 96), (2000, 64, 33), (1, 10, 8)])
def test_accumulate(T, V, D, dt):
    """Added to what is there; rows that no token names are not written, whatever they hold."""
    dy, tok = values((T, D), dt), tokens_of(T, V, 3.0)
    ref, tol, n = grad_reference(dy, tok, V, 0.5)
    for out in {F32, dt}:
        old = values((V, D), out, 5)
        old[n[:, 0] == 0, 0] = math.nan
        g = old.cuda()
        got = rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), grad=g, scale=0.5, accumulate=True)
        assert got is g and rwo.get_status() == rwo.OK
        hit = n[:, 0] > 0
        want = ref + old.double()
        assert_close(g[hit.cuda()], want[hit], (tol + 2 * U * (old.double().abs() + ref.abs()))[hit] + half_step(want[hit], out))
        assert torch.equal(g[~hit.cuda()].nan_to_num(nan=7.0).cpu(), old[~hit].nan_to_num(nan=7.0))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("shift,pad,D", [(0, 8, 256), (1, 0, 64), (3, 5, 200), (0, 7, 64)])
def test_pitches(shift, pad, D, dt):
    T, V = 900, 120
    dy, tok = values((T, D), dt), tokens_of(T, V, 3.0)
    check(dy, tok, V, dyd=placed(dy, shift, pad))
    for out in {F32, dt}:
        g = placed(torch.zeros(V, D, dtype=out), shift, pad)
        base = g._base if g._base is not None else g
        gaps = torch.isnan(base).sum()
        check(dy, tok, V, dtype=out, grad=g)
        assert torch.isnan(base).sum() == gaps


def test_gradient_edges():
    """All padding, all one token, every token once, no tokens; a token outside is recorded and gives nothing."""
    V, D = 77, 48
    dy = values((5000, D), F32)
    for tok in (torch.full((5000,), -1), torch.full((5000,), 76), torch.zeros(5000, dtype=torch.int64)):
        check(dy, tok.long(), V)
    check(dy[:77], torch.randperm(77, generator=torch.Generator().manual_seed(2)), V)
    g = rwo.embedding_rows_backward(dy[:0].cuda(), torch.empty(0, dtype=torch.int64, device="cuda"), V)
    assert g.shape == (V, D) and not g.any()
    tok = tokens_of(5000, V, 1.0)
    tok[17], tok[4000] = V, 2 ** 40
    ref, tol, _ = grad_reference(dy, tok, V)
    g = rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), V)
    assert rwo.get_status() == rwo.ERR_INVALID_ARG and rwo.get_status() == rwo.OK
    assert_close(g, ref, tol)


@pytest.mark.parametrize("V", [1, 2, 31, 32, 1023, 1024, 1025, 2 ** 20 - 1, 2 ** 20, 2 ** 20 + 5, 3_000_000])
def test_vocabularies_around_the_digits(V):
    T, D = 3000, 4
    tok = tokens_of(T, V, 1.0)
    tok[:3] = torch.tensor([0, V - 1, V // 2])
    check(values((T, D), F32), tok, V)


def test_large_batch_and_dimension():
    """More tokens than one CTA of the sort holds at once, a frequent token among them."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, V, D = 262144, 50021, 64
    dy = torch.randn(T, D, device="cuda", generator=gen)
    tok = (V * torch.rand(T, device="cuda", generator=gen, dtype=torch.float64) ** 4).long()
    tok[::3] = 4242
    g = rwo.embedding_rows_backward(dy, tok, V)
    ref = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, tok, dy.double())
    mag = torch.zeros(V, D, dtype=torch.float64, device="cuda").index_add_(0, tok, dy.double().abs())
    n = torch.bincount(tok, minlength=V).double()[:, None]
    # chunks of 32, eight sums of them, and the join: a token's additions are not one chain
    assert_close(g, ref, (torch.clamp(n, max=32 + T / 32 / 8 + 8) + 2) * U * mag)
    assert torch.equal(g, rwo.embedding_rows_backward(dy, tok, V))


def test_lookup_and_gradient_are_transposes():
    """<lookup(table), dy> = <table, gradient(dy)>, and the gradient against differences of the first."""
    T, V, D = 60, 11, 7
    table, dy, tok = values((V, D), F32, 3), values((T, D), F32, 4), tokens_of(T, V, 1.0)
    y = rwo.embedding_rows(table.cuda(), tok.cuda(), scale=2.0).double().cpu()
    g = rwo.embedding_rows_backward(dy.cuda(), tok.cuda(), V, scale=2.0).double().cpu()
    a, b = (y * dy.double()).sum(), (table.double() * g).sum()
    assert abs(a - b) <= (T + 4) * U * (y.abs() * dy.double().abs()).sum()
    for v in range(V):
        step = table.clone()
        step[v, 3] += 1.0
        diff = (rwo.embedding_rows(step.cuda(), tok.cuda(), scale=2.0).double().cpu() - y)[:, 3] * dy.double()[:, 3]
        assert abs(diff.sum() - g[v, 3]) <= 8 * U * (T + 4) * dy.double()[:, 3].abs().sum() * 4


def test_streams_and_graphs():
    T, V, D = 3000, 700, 256
    dy, tok = values((T, D), BF).cuda(), tokens_of(T, V, 4.0).cuda()
    want = rwo.embedding_rows_backward(dy, tok, V)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = rwo.embedding_rows_backward(dy, tok, V, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    ws = rwo.embedding_backward_workspace(T, V, D)
    grad, buf = torch.zeros_like(want), torch.zeros_like(tok)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rwo.embedding_rows_backward(dy, buf, grad=grad, workspace=ws)
    for t in (tok.flip(0).contiguous(), tok):
        buf.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, rwo.embedding_rows_backward(dy, t, V))
