"""The training-step calls where offsets pass 32 bits: rows picked from all over the output against 64 bits.

Tolerances as in the tests of each call.
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


def filled(shape, dt, scale=1.0):
    t = torch.empty(shape, dtype=dt, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    for c in t.view(-1).split(1 << 28):
        c.normal_(generator=gen).mul_(scale)
    return t


def test_loss():
    M, N = 36000, 131072
    x = filled((M, N), BF, 2.0)
    labels = torch.randint(0, N, (M,), device="cuda")
    pick = torch.tensor([0, 1, 16383, 16384, 32767, 32768, M - 1], device="cuda")
    rows = x[pick].double()
    loss, g = rwo.cross_entropy_rows_grad(x, labels, grad=x)
    assert rwo.get_status() == rwo.OK
    lse = torch.logsumexp(rows, 1, keepdim=True)
    ref = (rows - lse).exp()
    tol = 1e-5 * ref
    at = labels[pick][:, None]
    want = (lse - rows.gather(1, at))[:, 0]
    ref = ref.scatter_add(1, at, torch.full_like(at, -1.0, dtype=torch.float64))
    tol = tol.scatter_add(1, at, torch.full_like(at, 4 * U, dtype=torch.float64))
    assert_close(g[pick], ref, tol.cpu() + half_step(ref, BF).cpu())
    assert_close(loss[pick], want, 1e-5 * want.clamp(min=1))


@pytest.mark.parametrize("N", [4096, 4095])
def test_norm_and_its_gradient(N):
    M = 1_100_000
    x = filled((M, N), BF)
    w = filled((N,), BF, 0.1).add_(1)
    pick = torch.tensor([0, 1, 524287, 524288, 1048575, 1048576, M - 1], device="cuda")
    rows = x[pick].double()
    rs = torch.empty(M, device="cuda")
    y, _ = rwo.rms_norm_rows(x, w, rstd_out=rs)
    rstd = 1 / torch.sqrt(rows.pow(2).mean(1, keepdim=True) + 1e-6)
    ref = rows * rstd * w.double()
    assert_close(y[pick], ref, (43 * U * ref.abs() + half_step(ref, BF)).cpu())
    dx, dw = rwo.rms_norm_rows_backward(y, x, rs, w, dx=y)  # in place: dy = y
    assert rwo.get_status() == rwo.OK
    r = rs[pick].double()[:, None]
    y2, _ = rwo.rms_norm_rows(x[pick].contiguous(), w)
    g = y2.double() * w.double()
    xhat = rows * r
    c, ca = (g * xhat).mean(1, keepdim=True), (g * xhat).abs().mean(1, keepdim=True)
    want = r * (g - xhat * c)
    tol = r * ((g.abs() + (xhat * c).abs()) * 6 * U + xhat.abs() * ca * 80 * U) + half_step(want, BF)
    # y of the picked rows alone may round an entry the other way: half a step of dy, times its factor
    tol = tol + r * w.double().abs() * 2 * half_step(y2.double(), BF)
    assert_close(dx[pick], want, tol.cpu())
    assert torch.isfinite(dw).all()


def test_embedding_and_its_gradient():
    V, D, T = 1_200_000, 4096, 5000
    table = filled((V, D), BF)
    tokens = torch.randint(0, V, (T,), device="cuda")
    tokens[:4] = torch.tensor([0, V - 1, 524288, 1048576], device="cuda")
    y = rwo.embedding_rows(table, tokens)
    assert torch.equal(y, table[tokens])
    g = rwo.embedding_rows_backward(y, tokens, grad=table.fill_(3.0), dtype=BF)
    assert rwo.get_status() == rwo.OK
    ref = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    uniq, inv = tokens.unique(return_inverse=True)
    ref.index_add_(0, inv, y.double())
    n = torch.bincount(inv)
    once = uniq[n[: len(uniq)] == 1]
    assert torch.equal(g[once].double(), ref[: len(uniq)][n[: len(uniq)] == 1])
    hit = torch.zeros(V, dtype=torch.bool, device="cuda")
    hit[uniq] = True
    assert not any(bool(c.any()) for c in torch.where(hit[:, None], torch.zeros((), dtype=BF, device="cuda"), g).split(100000))


def test_gradient_norm():
    n = (1 << 32) + 12345
    flat = filled((n,), BF)
    ts = list(flat.split([7, n - 7 - 1000, 1000]))
    total = sum(float(c.double().pow(2).sum()) for c in flat.split(1 << 27))
    norm = rwo.clip_grad_norm(ts, 1.0)
    assert abs(float(norm) - total ** 0.5) <= 22 * U * total ** 0.5
    after = sum(float(c.double().pow(2).sum()) for c in flat.split(1 << 27))
    assert abs(after - 1.0) <= 2.0 ** -8 + 1e-3  # every element rounded to bf16 again
